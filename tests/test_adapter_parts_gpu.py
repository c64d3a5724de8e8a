"""Gradients asked for alone have the bits that they have beside the others, whatever the
alignment of the buffers."""
import pytest
import torch

import kronecker_sparse_matrix_b200 as ks
from kronecker_sparse_matrix_b200 import _lib
from tests.test_adapter_gpu import DEV, assert_backward, make

pytestmark = pytest.mark.gpu
NEEDS = ("need_dx", "need_da", "need_db")
# tensor-core products (H of 8, 16 and 24 ranks), fp32 products that take the adapters along (rank 1 and 8),
# few rows, and layers that take a second pass
CASES = [((1, 256, 64, 16), 3000, 16, torch.bfloat16), ((1, 64, 48, 8), 700, 5, torch.bfloat16),
         ((2, 96, 64, 1), 700, 24, torch.bfloat16), ((1, 192, 48, 8), 7400, 1, torch.float32),
         ((1, 192, 48, 8), 7300, 8, torch.float32), ((1, 64, 48, 8), 40, 16, torch.bfloat16),
         ((1, 64, 48, 8), 40, 16, torch.float32), ((5, 21, 23, 4), 700, 6, torch.bfloat16),
         ((2, 100, 48, 8), 900, 8, torch.float32)]


@pytest.mark.parametrize("p,n,r,dtype", CASES)
@pytest.mark.parametrize("odd", [(), ("x",), ("values",), ("dy",), ("A",), ("B",), ("x", "A"), ("x", "values", "dy", "A", "B")])
def test_parts(p, n, r, dtype, odd):
    q = make(p, n, 4, r, dtype, "segments", n)
    moved = make(p, n, 4, r, dtype, "segments", n, shift=1)
    q.update({name: moved[name] for name in odd})
    args = (q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"])
    whole = ks.adapter_backward(*args)
    assert_backward(q, p, whole)
    for wanted in (("need_dx",), ("need_da",), ("need_db",), ("need_da", "need_db"), ("need_dx", "need_db")):
        got = ks.adapter_backward(*args, **{m: m in wanted for m in NEEDS})
        for m, g, w in zip(NEEDS, got, whole):
            assert (g is not None) == (m in wanted) and (g is None or torch.equal(g, w)), (wanted, m)
    dx, _, _ = ks.adapter_backward(q["dy"], None, *args[2:], need_da=False, need_db=False)
    _, da, db = ks.adapter_backward(q["dy"], q["x"], None, *args[3:], need_dx=False)
    for got, w in zip((dx, da, db), whole):
        assert torch.equal(got, w)


@pytest.mark.parametrize("p,n,r,dtype", CASES)
def test_parts_beside_an_unaligned_dx(p, n, r, dtype):
    """dX one element into its storage, through the C entry point."""
    q = make(p, n, 4, r, dtype, "segments", n)
    a, b, c, d = p

    def run(dx):
        da, db = torch.empty_like(q["A"]), torch.empty_like(q["B"])
        code = {torch.float32: ks.KS_F32, torch.bfloat16: ks.KS_BF16}[dtype]
        _lib.check(_lib.load().ks_adapter_backward(
            q["dy"].data_ptr(), q["x"].data_ptr(), q["values"].data_ptr(), a, b, c, d, n, code, q["A"].data_ptr(),
            q["B"].data_ptr(), q["scales"].data_ptr(), q["ids"].data_ptr(), 4, r, None if dx is None else dx.data_ptr(),
            da.data_ptr(), db.data_ptr(), torch.cuda.current_stream().cuda_stream))
        return da, db

    odd = torch.empty(n * a * c * d + 1, dtype=dtype, device=DEV)[1:].view(n, -1)
    da, db = run(odd)
    assert_backward(q, p, (odd, da, db))
    for u, v in zip(run(None), (da, db)):
        assert torch.equal(u, v)

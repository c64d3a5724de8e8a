"""TF32 gradients of adapters (dX's KS product in TF32, everything else in fp32), against the
formulas in 64 bits.

Tolerances as in test_adapter_gpu.py; a TF32 product rounds both operands to 10 bits, 2^-10
relative each at most, so dX's product is off by 2^-9 |dY||K| more.  dA and dB know nothing of it.
"""
import pytest
import torch

import kronecker_sparse_matrix_b200 as ks
from tests.test_adapter_gpu import F64, backward64, dense_rows, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p", [(1, 192, 48, 8), (2, 64, 32, 2), (1, 256, 64, 16), (2, 96, 80, 1), (3, 20, 12, 5)])
@pytest.mark.parametrize("kind", ["rows", "segments", "one"])
def test_backward(p, kind):
    for n, r, shift in ((4, 16, 0), (260, 5, 0), (900, 20, 1)):
        q = make(p, n, 1 if kind == "one" else 3, r, torch.float32, kind, n, shift=shift)
        args = (q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"])
        got = ks.adapter_backward(*args, tf32=True)
        ks.sync_status()
        refs, tols = backward64(q, p)
        more = 2.0 ** -9 * dense_rows(q["values"].to(F64).abs(), p, q["dy"].to(F64).abs(), True)
        for name, g, ref, tol in zip(("dX", "dA", "dB"), got, refs, (tols[0] + more, tols[1], tols[2])):
            assert torch.isfinite(g).all()
            off = (g.to(F64) - ref).abs()
            assert (off <= tol + 1e-30).all(), f"{p} {name}: {(off / (tol + 1e-30)).max():.3g} of the tolerance"
        for k, name in enumerate(("need_dx", "need_da", "need_db")):  # alone as beside one another
            only = ks.adapter_backward(*args, tf32=True, **{m: m == name for m in ("need_dx", "need_da", "need_db")})
            assert torch.equal(only[k], got[k])


def test_bf16_is_refused():
    p = (1, 64, 48, 8)
    q = make(p, 6, 2, 8, torch.bfloat16, "rows", 1)
    with pytest.raises(ValueError, match="tf32"):
        ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"], tf32=True)

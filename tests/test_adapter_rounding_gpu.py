"""bf16 adapters of layers that no tensor-core product takes along: the KS product, the
adapters, the bias and the activation are summed in fp32 and rounded once.

Tolerances as in test_adapter_gpu.py, without a rounding of the KS product and of H:
fp32 sums, then half a step of bf16, 2^-8 relative, of the result (half of its smallest
spacing, 2^-134, beside zero).
"""
import pytest
import torch

import kronecker_sparse_matrix_b200 as ks
from tests.test_adapter_gpu import BF, DEV, F64, U, call, dense_rows, forward64, make, rows_of

pytestmark = pytest.mark.gpu

# c no multiple of 16 (whole vectors of c and l, and of l alone), odd d, blocks of the streaming
# kernels: weights in registers (l vectors, merged blocks), l vectors, single outputs, few rows or columns
PATTERNS = [(1, 96, 24, 8), (2, 32, 8, 4), (1, 64, 40, 2), (5, 21, 23, 4), (1, 104, 171, 4), (8, 2, 2, 16), (16, 2, 2, 1),
            (8, 4, 4, 2), (3, 3, 5, 8), (3, 7, 9, 5), (1, 15, 30, 8), (4, 19, 2, 13), (3, 8, 24, 24)]


def assert_rounded_once(got, ref, tol):
    tol = tol + BF * (ref.abs() + tol) + 2.0 ** -134
    off = (got.to(F64) - ref).abs()
    assert torch.isfinite(got).all()
    assert (off <= tol).all(), f"{(off / tol).max():.3g} of the tolerance"


def assert_forward_once(y, q, p, act):
    a, b, c, d = p
    ref, z, _, base_abs, low_abs = forward64(q, p, act)
    tol = (c + 4) * U * base_abs + (a * c * d + q["A"].shape[1] + 8) * U * low_abs + 8 * U * z.abs()
    if q["bias"] is not None:
        tol = tol + 4 * U * q["bias"].to(F64).abs()
    assert_rounded_once(y, ref, tol)


def assert_dx_once(dx, q, p):
    a, b, c, d = p
    v, A, B, dy = (q[k].to(F64) for k in ("values", "A", "B", "dy"))
    ref, base_abs = dense_rows(v, p, dy, True), dense_rows(v.abs(), p, dy.abs(), True)
    low_abs = torch.zeros_like(ref)
    for s in range(A.shape[0]):
        at, sc = rows_of(q, s), float(q["scales"][s])
        ref[at] += sc * dy[at] @ B[s] @ A[s]
        low_abs[at] = sc * (dy[at].abs() @ B[s].abs()) @ A[s].abs()
    assert_rounded_once(dx, ref, (b + 4) * U * base_abs + (a * b * d + A.shape[1] + 8) * U * low_abs + 8 * U * ref.abs())


def dx_of(q, p):
    dx, _, _ = ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"])
    ks.sync_status()
    return dx


@pytest.mark.parametrize("p", PATTERNS)
@pytest.mark.parametrize("kind", ["rows", "segments", "none"])
def test_one_rounding(p, kind):
    for n, r, act in ((300, 5, "none"), (1031, 16, "relu"), (2000, 20, "none")):
        q = make(p, n, 4, r, torch.bfloat16, kind, n + r, bias=True)
        assert_forward_once(call(q, p, act=act), q, p, act)
        if p[1] % 16 or p[1] * p[2] <= 64:  # (otherwise a tensor-core product takes dX)
            assert_dx_once(dx_of(q, p), q, p)


@pytest.mark.parametrize("p", [(1, 64, 48, 8), (2, 96, 64, 1), (1, 7, 9, 1), (8, 2, 2, 16)])
def test_one_rounding_of_unaligned_buffers(p):
    q = make(p, 700, 3, 16, torch.bfloat16, "segments", 5, bias=True, shift=1)
    assert_forward_once(call(q, p), q, p, "none")
    assert_dx_once(dx_of(q, p), q, p)
    out = torch.empty(700 * p[0] * p[1] * p[3] + 1, dtype=torch.bfloat16, device=DEV)[1:].view(700, -1)
    q = make(p, 700, 3, 16, torch.bfloat16, "segments", 5, bias=True)
    assert_forward_once(call(q, p, out=out), q, p, "none")


@pytest.mark.parametrize("p,n", [((1, 96, 24, 8), 90011), ((2, 50, 30, 20), 60003)])
def test_one_rounding_of_many_rows(p, n):
    """More rows than the fp32 sums are held for at a time."""
    q = make(p, n, 5, 8, torch.bfloat16, "segments", 7, bias=True)
    assert_forward_once(call(q, p), q, p, "none")
    assert_dx_once(dx_of(q, p), q, p)


def test_the_sum_of_a_product_and_its_opposite():
    """An adapter that takes the product away again, but for a part in 2^12: nothing of the
    product's own rounding may stay."""
    p = (1, 96, 24, 1)
    q = make(p, 400, 1, 24, torch.bfloat16, "one", 3)
    q["A"][0] = torch.eye(24, device=DEV)
    q["B"][0] = -q["values"].view(96, 24)
    q["scales"].fill_(1 - 2.0 ** -12)
    assert_forward_once(call(q, p), q, p, "none")


def test_alignment_of_a_alone_changes_nothing():
    p = (1, 64, 48, 8)
    q = make(p, 600, 3, 16, torch.bfloat16, "segments", 17, bias=True)
    odd = make(p, 600, 3, 16, torch.bfloat16, "segments", 17, bias=True, shift=1)
    assert torch.equal(call(dict(q, A=odd["A"]), p, act="gelu_tanh"), call(q, p, act="gelu_tanh"))


@pytest.mark.parametrize("p", [(1, 256, 64, 16), (1, 64, 48, 8), (2, 96, 64, 1), (3, 20, 12, 5), (8, 2, 2, 16)])
def test_one_rounding_of_few_rows(p):
    """The kernel of few rows holds H in fp32 too."""
    for n, r, shift in ((1, 16, 0), (9, 5, 0), (64, 16, 1)):
        q = make(p, n, 3, r, torch.bfloat16, "rows", n, bias=True, shift=shift)
        assert_forward_once(call(q, p, act="relu"), q, p, "relu")
        assert_dx_once(dx_of(q, p), q, p)


@pytest.mark.parametrize("p", [(1, 256, 64, 16), (1, 64, 48, 8), (2, 96, 64, 1), (2, 64, 32, 2), (2, 32, 48, 4)])
def test_tensor_core_products_round_h_and_the_result_alone(p):
    a, b, c, d = p
    for n, r in ((600, 16), (1031, 20)):
        q = make(p, n, 4, r, torch.bfloat16, "segments", n, bias=True)
        ref, z, _, base_abs, low_abs = forward64(q, p)
        tol = (c + 4) * U * base_abs + ((a * c * d + r + 8) * U + BF) * low_abs + 8 * U * z.abs() + 4 * U * q["bias"].to(F64).abs()
        assert_rounded_once(call(q, p), ref, tol)


def test_unaligned_calls_in_replayed_graphs():
    """A copy of A, and fp32 sums of a product, in workspaces of each graph's own."""
    runs = []
    for p, names in (((1, 64, 48, 8), ("A",)), ((1, 96, 24, 8), ()), ((5, 21, 23, 4), ("x",))):
        q, odd = (make(p, 700, 3, 16, torch.bfloat16, "segments", 5, bias=True, shift=s) for s in (0, 1))
        q.update({name: odd[name] for name in names})
        want = call(q, p), dx_of(q, p)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = ks.adapter_matmul(q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"], bias=q["bias"])
            dx, _, _ = ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"])
        runs.append((g, torch.cuda.Stream(), (y, dx), want, q))  # (a replay reads q again)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st, *_ in runs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    ks.sync_status()
    for _, _, got, want, _ in runs:
        assert all(torch.equal(u, v) for u, v in zip(got, want))

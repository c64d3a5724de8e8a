"""Low-rank adapters beside a KS product (ks_adapter_matmul) and their gradients
(ks_adapter_backward) against the formulas in 64 bits.

Tolerances, element by element.  With u = 2^-24, a fp32 sum of n products is off
by at most about n u times the sum of the products' magnitudes, so with |.| for
magnitudes (all in 64 bits)
    H:   (in + 2) u |X||A|^T scale
    Y:   (c + 4) u |X||K|^T + (in + rank + 8) u |H| |B|^T + 4 u |bias|
where |H| = scale |X||A|^T.  bf16 adds half a step, 2^-8 relative, for each
rounding: of Y, of the KS product where the adapters are added in a second pass,
and of H where it is a tensor-core operand.  TF32 products (dtype tf32) round
both operands to 10 bits, 2^-10 relative each at most.  The activations have
slopes of at most 1.13; their own evaluation is off by at most 2^-20 |z| in
fp32 and, with the hardware tanh of the tensor-core epilogue, 2^-11 |z|.
Gradients: the same with rows summed, n = rows of the adapter.
"""
import pytest
import torch

import kronecker_sparse_matrix_b200 as ks
from kronecker_sparse_matrix_b200 import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF = 2.0 ** -8
F64 = torch.float64

# CUDA-core and streaming patterns, tensor-core patterns with 1, 2, 4, 8 and 16 l, several k passes,
# several blocks, c that is no multiple of a chunk
PATTERNS = [(2, 4, 4, 2), (3, 20, 12, 5), (1, 7, 9, 1), (1, 96, 80, 1), (2, 64, 32, 2), (2, 32, 48, 4),
            (1, 192, 48, 8), (1, 256, 64, 16), (2, 48, 16, 24)]


def make_ids(kind, n, s, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        return None
    if kind == "none":
        return torch.full((n,), -1, dtype=torch.int32)
    if kind == "rows":
        return torch.randint(-1, s, (n,), generator=g, dtype=torch.int32)
    ids, at = torch.full((n,), -1, dtype=torch.int32), 0  # ragged segments in any order of the ids
    while at < n:
        k = int(torch.randint(1, max(2, n // 3), (1,), generator=g))
        ids[at:at + k] = int(torch.randint(-1, s, (1,), generator=g))
        at += k
    return ids


def make(p, n, s, r, dtype, kind, seed, bias=False, shift=0):
    """Inputs on the GPU; `shift` elements into their storage (no alignment beyond the element's)."""
    a, b, c, d = p
    g = torch.Generator().manual_seed(seed)

    def t(*shape, std=1.0):
        v = (torch.randn(*shape, generator=g) * std).to(dtype)
        buf = torch.empty(v.numel() + shift, dtype=dtype, device=DEV)
        buf[shift:].copy_(v.reshape(-1))
        return buf[shift:].view(*shape)

    fin, fout = a * c * d, a * b * d
    ids = make_ids(kind, n, s, seed + 1)
    return {"x": t(n, fin), "values": t(a, d, b, c, std=c ** -0.5), "A": t(s, r, fin, std=fin ** -0.5),
            "B": t(s, fout, r, std=r ** -0.5), "bias": t(fout) if bias else None, "dy": t(n, fout),
            "ids": None if ids is None else ids.to(DEV), "scales": (torch.rand(s, generator=g) + 0.5).to(DEV)}


def dense_rows(w, p, x, transpose=False):
    a, b, c, d = p
    n = x.shape[0]
    if transpose:
        return torch.einsum("nikl,ilkj->nijl", x.view(n, a, b, d), w).reshape(n, -1)
    return torch.einsum("nijl,ilkj->nikl", x.view(n, a, c, d), w).reshape(n, -1)


def rows_of(q, s):
    n = q["x"].shape[0]
    return torch.arange(n, device=DEV) if q["ids"] is None else torch.nonzero(q["ids"] == s).view(-1)


def act64(z, act):
    if act == "relu":
        return z.relu()
    if act == "none":
        return z
    return torch.nn.functional.gelu(z, approximate="tanh" if act == "gelu_tanh" else "none")


def forward64(q, p, act="none"):
    """Y and its tolerance's sums: base, |X||K|^T and |H||B|^T in 64 bits."""
    x, v, A, B = (q[k].to(F64) for k in ("x", "values", "A", "B"))
    base, base_abs = dense_rows(v, p, x), dense_rows(v.abs(), p, x.abs())
    low, low_abs = torch.zeros_like(base), torch.zeros_like(base)
    for s in range(A.shape[0]):
        at, sc = rows_of(q, s), float(q["scales"][s])
        low[at] = sc * (x[at] @ A[s].t()) @ B[s].t()
        low_abs[at] = sc * (x[at].abs() @ A[s].abs().t()) @ B[s].abs().t()
    z = base + low
    if q["bias"] is not None:
        z = z + q["bias"].to(F64)
    return act64(z, act), z, base, base_abs, low_abs


def assert_forward(y, q, p, act="none", tf32=False):
    a, b, c, d = p
    ref, z, base, base_abs, low_abs = forward64(q, p, act)
    fin, r = a * c * d, q["A"].shape[1]
    tol = (c + 4) * U * base_abs + (fin + r + 8) * U * low_abs + 8 * U * z.abs()
    if q["bias"] is not None:
        tol = tol + 4 * U * q["bias"].to(F64).abs()
    if q["x"].dtype == torch.bfloat16:
        tol = tol + BF * base.abs() + BF * low_abs  # the KS product's rounding, H's as an operand
    if tf32:
        tol = tol + 2.0 ** -9 * (base_abs + low_abs)
    if act != "none":
        low_bits = 2.0 ** -11 if tf32 or q["x"].dtype == torch.bfloat16 else 2.0 ** -20
        tol = 1.13 * tol + low_bits * z.abs()
    if q["x"].dtype == torch.bfloat16:
        tol = tol + BF * (ref.abs() + tol)
    off = (y.to(F64) - ref).abs()
    assert torch.isfinite(y).all()
    assert (off <= tol + 1e-30).all(), f"{p}: {(off / (tol + 1e-30)).max():.3g} of the tolerance"


def call(q, p, **kw):
    y = ks.adapter_matmul(q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"], bias=q["bias"], **kw)
    ks.sync_status()
    return y


@pytest.mark.parametrize("p", PATTERNS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["rows", "segments", "one", "none"])
def test_forward(p, dtype, kind):
    for n, s, r in ((1, 1, 1), (3, 2, 8), (40, 5, 16), (129, 3, 5), (300, 4, 20)):
        q = make(p, n, 1 if kind == "one" else s, r, dtype, kind, n + r)
        assert_forward(call(q, p), q, p)


@pytest.mark.parametrize("p", [(3, 20, 12, 5), (1, 96, 80, 1), (2, 64, 32, 2), (1, 192, 48, 8), (1, 256, 64, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh", "gelu_erf"])
def test_bias_and_activation(p, dtype, act):
    for n, kind, r in ((2, "rows", 16), (200, "segments", 16), (131, "none", 8)):
        q = make(p, n, 3, r, dtype, kind, n, bias=True)
        assert_forward(call(q, p, act=act), q, p, act)


@pytest.mark.parametrize("r", [1, 3, 8, 16, 24, 32, 64, 100, 128, 200])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ranks(r, dtype):
    for p in ((1, 64, 48, 8), (2, 96, 64, 1), (1, 10, 6, 3)):
        for n in (5, 150):
            q = make(p, n, 3, r, dtype, "segments", r)
            assert_forward(call(q, p), q, p)


@pytest.mark.parametrize("p", [(1, 192, 48, 8), (2, 64, 32, 2), (1, 256, 64, 16), (3, 20, 12, 5)])
def test_tf32(p):
    for n, kind in ((4, "rows"), (260, "segments")):
        q = make(p, n, 3, 16, torch.float32, kind, n, bias=True)
        assert_forward(call(q, p, tf32=True, act="gelu_tanh"), q, p, "gelu_tanh", tf32=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_unaligned_buffers(dtype):
    for p in ((1, 64, 48, 8), (2, 96, 64, 1), (1, 7, 9, 1)):
        for n in (3, 140):
            q = make(p, n, 3, 16, dtype, "segments", 5, bias=True, shift=1)
            assert_forward(call(q, p, act="relu"), q, p, "relu")


def test_many_adapters_in_one_tile():
    """Every row its own adapter, far more than a tile holds rows of one."""
    for dtype in (torch.float32, torch.bfloat16):
        q = make((1, 64, 48, 8), 300, 300, 8, dtype, "rows", 3)
        q["ids"] = torch.randperm(300, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(DEV)
        assert_forward(call(q, (1, 64, 48, 8)), q, (1, 64, 48, 8))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [3, 200])
def test_too_large_id_is_reported_and_takes_no_adapter(dtype, n):
    p = (1, 64, 48, 8)
    q = make(p, n, 2, 16, dtype, "rows", 9)
    bad = q["ids"].clone()
    bad[n // 2] = 2
    bad[0] = 2 ** 31 - 1
    y = ks.adapter_matmul(q["x"], q["values"], p, q["A"], q["B"], bad, q["scales"])
    with pytest.raises(ks.KsError, match="adapter id"):
        ks.sync_status()
    ks.sync_status()  # cleared
    q["ids"] = torch.where(bad > 1, -1, bad).to(torch.int32)
    assert_forward(y, q, p)
    ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], bad, q["scales"])
    with pytest.raises(ks.KsError, match="adapter id"):
        ks.sync_status()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_unused_weights_may_hold_anything(dtype):
    """Infinities and NaN in rows and adapters that no product uses stay there."""
    p = (1, 64, 48, 8)
    for n in (6, 200):
        q = make(p, n, 3, 16, dtype, "segments", 11)
        q["ids"].fill_(0)
        q["ids"][n // 2:] = -1
        clean = call(q, p)
        q["A"][1:] = float("nan")
        q["B"][1:] = float("inf")
        q["scales"][1:] = float("nan")
        assert torch.equal(call(q, p), clean)
        x = q["x"].clone()
        q["x"][n - 1] = float("inf")  # a row without an adapter
        y = call(q, p)
        assert torch.equal(y[:n - 1], clean[:n - 1])
        q["x"] = x
        da = ks.adapter_backward(q["dy"], x, q["values"], p, q["A"], q["B"], q["ids"], q["scales"])[1]
        q["dy"][n - 1] = float("nan")
        x[n - 1] = float("inf")
        da2, db2 = ks.adapter_backward(q["dy"], x, q["values"], p, q["A"], q["B"], q["ids"], q["scales"])[1:]
        assert torch.equal(da[0], da2[0]) and torch.isfinite(db2).all() and (da2[1:] == 0).all()


@pytest.mark.parametrize("p", [(1, 64, 48, 8), (1, 96, 80, 1), (2, 64, 32, 2), (1, 64, 64, 64), (3, 20, 12, 5)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_broken_adapter_harms_its_own_rows_only(p, dtype):
    """Infinities and NaN in one adapter's weights or scale, in a tile that it shares."""
    for n in (6, 200):
        q = make(p, n, 3, 16, dtype, "rows", 13)
        q["ids"][0] = 1
        args = (q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"])
        clean, (dx, da, db) = call(q, p), ks.adapter_backward(*args)
        other = q["ids"] != 1
        for name, value in (("A", float("inf")), ("B", float("nan")), ("scales", float("inf"))):
            kept = q[name].clone()
            q[name][1] = value
            y, (dx2, da2, db2) = call(q, p), ks.adapter_backward(*args)
            assert torch.equal(y[other], clean[other]) and torch.equal(dx2[other], dx[other])
            assert torch.equal(da2[::2], da[::2]) and torch.equal(db2[::2], db[::2])
            assert not torch.isfinite(y[0]).all()
            q[name].copy_(kept)


def test_without_ids_every_row_takes_the_first_adapter():
    for dtype in (torch.float32, torch.bfloat16):
        for p in ((1, 64, 48, 8), (1, 7, 9, 1)):
            q = make(p, 140, 3, 8, dtype, "one", 4)
            zero = dict(q, ids=torch.zeros(140, dtype=torch.int32, device=DEV))
            assert_forward(call(q, p), zero, p)
            assert_backward(zero, p, ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], None,
                                                         q["scales"]))


def test_scales_default_to_one_and_out_is_filled():
    p = (1, 64, 48, 8)
    q = make(p, 20, 2, 8, torch.float32, "rows", 2)
    q["scales"].fill_(1.0)
    out = torch.full((20, 512), float("nan"), device=DEV)
    assert ks.adapter_matmul(q["x"], q["values"], p, q["A"], q["B"], q["ids"], out=out) is out
    assert torch.equal(out, call(q, p))
    assert ks.adapter_matmul(q["x"][:0], q["values"], p, q["A"], q["B"], q["ids"][:0]).shape == (0, 512)


# ---------------------------------------------------------------- gradients


def backward64(q, p):
    a, b, c, d = p
    x, v, A, B, dy = (q[k].to(F64) for k in ("x", "values", "A", "B", "dy"))
    fin, fout, r = a * c * d, a * b * d, A.shape[1]
    bf = q["x"].dtype == torch.bfloat16
    dx, base_abs = dense_rows(v, p, dy, True), dense_rows(v.abs(), p, dy.abs(), True)
    low_abs = torch.zeros_like(dx)
    base = dx.clone()
    da, db = torch.zeros_like(A), torch.zeros_like(B)
    ta, tb = torch.zeros_like(A), torch.zeros_like(B)
    for s in range(A.shape[0]):
        at, sc = rows_of(q, s), float(q["scales"][s])
        G, Ga = sc * dy[at] @ B[s], sc * dy[at].abs() @ B[s].abs()
        H, Ha = sc * x[at] @ A[s].t(), sc * x[at].abs() @ A[s].abs().t()
        dx[at] += G @ A[s]
        low_abs[at] = Ga @ A[s].abs()
        da[s], db[s] = G.t() @ x[at], dy[at].t() @ H
        more = BF if bf else 0.0  # G and H as tensor-core operands
        ta[s] = ((fout + len(at) + 8) * U + more) * (Ga.t() @ x[at].abs())
        tb[s] = ((fin + len(at) + 8) * U + more) * (dy[at].abs().t() @ Ha)
    tx = (b + 4) * U * base_abs + (fout + r + 8) * U * low_abs
    if bf:
        tx = tx + BF * base.abs() + BF * low_abs
        tx, ta, tb = (t + BF * (g.abs() + t) for t, g in ((tx, dx), (ta, da), (tb, db)))
    return (dx, da, db), (tx, ta, tb)


def assert_backward(q, p, got=None):
    got = got or ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"])
    ks.sync_status()
    for name, g, ref, tol in zip(("dX", "dA", "dB"), got, *backward64(q, p)):
        assert g.shape == ref.shape and torch.isfinite(g).all(), name
        off = (g.to(F64) - ref).abs()
        assert (off <= tol + 1e-30).all(), f"{p} {name}: {(off / (tol + 1e-30)).max():.3g} of the tolerance"


@pytest.mark.parametrize("p", PATTERNS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["rows", "segments", "one", "none"])
def test_backward(p, dtype, kind):
    for n, s, r in ((1, 1, 1), (3, 2, 8), (40, 5, 16), (129, 3, 5), (700, 4, 20)):
        assert_backward(make(p, n, 1 if kind == "one" else s, r, dtype, kind, 3 * n + r), p)


@pytest.mark.parametrize("r", [1, 3, 8, 16, 24, 32, 64, 100, 128, 200])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward_ranks(r, dtype):
    for p in ((1, 64, 48, 8), (2, 96, 64, 1), (1, 10, 6, 3)):
        for n in (5, 450):
            assert_backward(make(p, n, 3, r, dtype, "segments", r), p)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward_unaligned_and_many_adapters(dtype):
    for p in ((1, 64, 48, 8), (1, 7, 9, 1)):
        assert_backward(make(p, 140, 3, 16, dtype, "segments", 5, shift=1), p)
        assert_backward(make(p, 260, 200, 8, dtype, "rows", 6), p)


@pytest.mark.parametrize("p,n", [((1, 192, 48, 8), 7300), ((2, 100, 48, 8), 7000), ((1, 64, 200, 16), 2700),
                                 ((1, 32, 256, 24), 2800)])
@pytest.mark.parametrize("kind", ["segments", "rows", "one"])
def test_fp32_products_large_enough_to_take_the_adapters_along(p, n, kind):
    """At least 2^30 flop: the adapters are stages of the fp32 product (64- and 128-row tiles, ragged rows and k)."""
    a, b, c, d = p
    assert 2 * n * a * b * c * d >= 1 << 30
    for r in (8, 5, 20):
        q = make(p, n, 1 if kind == "one" else 4, r, torch.float32, kind, n + r, bias=True)
        if kind == "rows":  # runs of a few rows, so that warps hold several adapters
            q["ids"] = q["ids"][:n // 3 + 1].repeat_interleave(3)[:n].contiguous()
        assert_forward(call(q, p, act="gelu_erf"), q, p, "gelu_erf")
        assert_backward(q, p)


def test_a_broken_adapter_in_a_large_fp32_product():
    p, n = (1, 192, 48, 8), 7300
    q = make(p, n, 3, 8, torch.float32, "segments", 3)
    q["ids"][5] = 1
    q["ids"][6] = 0
    clean, dx = call(q, p), ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"])[0]
    other = q["ids"] != 1
    q["B"][1] = float("inf")
    q["A"][1] = float("nan")
    assert torch.equal(call(q, p)[other], clean[other])
    dx2 = ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"])[0]
    assert torch.equal(dx2[other], dx[other]) and not torch.isfinite(dx2[5]).any()


def test_many_adapters_with_few_rows_each():
    for dtype in (torch.float32, torch.bfloat16):
        for p in ((1, 64, 48, 8), (1, 10, 6, 3)):
            q = make(p, 2000, 150, 16, dtype, "rows", 31)
            q["ids"] = q["ids"].sort().values
            assert_backward(q, p)
            assert_forward(call(q, p), q, p)


def test_backward_with_some_buffers_unaligned():
    """A fused dX beside an X and an A that take no vectors."""
    p = (1, 64, 48, 8)
    for names in (("A",), ("x",), ("x", "A"), ("B",), ("values",)):
        q = make(p, 600, 3, 16, torch.bfloat16, "segments", 17)
        odd = make(p, 600, 3, 16, torch.bfloat16, "segments", 17, shift=1)
        assert_backward(dict(q, **{n: odd[n] for n in names}), p)
        assert_forward(call(dict(q, **{n: odd[n] for n in names}), p), q, p)


def test_backward_parts_and_determinism():
    p = (1, 256, 64, 16)
    q = make(p, 3000, 6, 16, torch.bfloat16, "segments", 8)
    args = (q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"])
    whole = ks.adapter_backward(*args)
    again = ks.adapter_backward(*args)
    assert all(torch.equal(u, v) for u, v in zip(whole, again))
    for k, name in enumerate(("need_dx", "need_da", "need_db")):
        only = ks.adapter_backward(*args, **{m: m == name for m in ("need_dx", "need_da", "need_db")})
        assert [o is not None for o in only] == [j == k for j in range(3)]
        assert torch.equal(only[k], whole[k])
    dx, da, db = ks.adapter_backward(q["dy"], None, q["values"], p, q["A"], q["B"], q["ids"], q["scales"],
                                     need_da=False, need_db=False)
    assert da is None and db is None and torch.equal(dx, whole[0])
    dx, da, db = ks.adapter_backward(q["dy"][:0], q["x"][:0], q["values"], p, q["A"], q["B"], q["ids"][:0], q["scales"])
    assert dx.shape == (0, 1024) and not da.any() and not db.any()


def test_gradients_match_differences():
    """d/dt of <dY, Y(theta + t E)> against <grad, E>, differences in 64 bits of
    the 64-bit forward (the map is a product of two linear ones: central
    differences are exact for each alone)."""
    p = (2, 20, 12, 3)
    q = make(p, 50, 3, 4, torch.float32, "rows", 21)
    got = dict(zip(("x", "A", "B"), ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"],
                                                       q["scales"])))
    for name, grad in got.items():
        E = torch.randn(q[name].shape, generator=torch.Generator().manual_seed(4)).to(DEV)
        vals = []
        for sign in (1, -1):
            moved = dict(q, **{name: q[name].to(F64) + sign * 0.5 * E.to(F64)})
            vals.append((forward64(moved, p)[0] * q["dy"].to(F64)).sum())
        want, have = float(vals[0] - vals[1]), float((grad.to(F64) * E.to(F64)).sum())
        _, tols = backward64(q, p)
        tol = float((tols[("x", "A", "B").index(name)] * E.abs().to(F64)).sum())
        assert abs(want - have) <= tol


# ---------------------------------------------------------------- streams, graphs, the layer


def test_other_stream_and_two_graphs_at_once():
    p = (1, 256, 64, 16)
    qs = [make(p, n, 4, 16, torch.bfloat16, "segments", n) for n in (200, 333)]
    want = [(call(q, p), ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"]))
            for q in qs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = ks.adapter_matmul(qs[0]["x"], qs[0]["values"], p, qs[0]["A"], qs[0]["B"], qs[0]["ids"], qs[0]["scales"],
                          stream=side)
    side.synchronize()
    assert torch.equal(y, want[0][0])
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = ks.adapter_matmul(q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"])
            outs.append((y, ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"],
                                                q["scales"])))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(20):  # replays side by side, each with workspaces of its own
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    ks.sync_status()
    for (y, grads), (wy, wg) in zip(outs, want):
        assert torch.equal(y, wy) and all(torch.equal(u, v) for u, v in zip(grads, wg))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_gradients_through_autograd(dtype):
    p = (1, 64, 48, 8)
    torch.manual_seed(0)
    layer = ks.KSAdapterLinear(p, 3, 8, alpha=16, bias=True, dtype=dtype, device=DEV)
    assert layer.scales.dtype == torch.float32 and float(layer.scales[0]) == 2.0
    x = torch.randn(4, 30, 384, device=DEV, dtype=dtype, requires_grad=True)
    ids = torch.tensor([0, 2, -1, 0], dtype=torch.int32, device=DEV)  # one id for each sequence
    plain = ks.KSLinear(p, bias=True, dtype=dtype, device=DEV)
    plain.load_state_dict({"values": layer.values, "bias": layer.bias})
    base = plain(x)
    assert (layer(x, ids) - base).abs().max() <= BF * base.abs().max()  # B starts at zero
    with torch.no_grad():
        layer.B.normal_(std=0.3)
    y = layer(x, ids)
    dy = torch.randn_like(y)
    y.backward(dy)
    rows = ids.view(4, 1).expand(4, 30).reshape(-1).contiguous()
    q = {"x": x.detach().view(-1, 384), "values": layer.values.detach(), "A": layer.A.detach(),
         "B": layer.B.detach(), "dy": dy.view(-1, 512), "ids": rows, "scales": layer.scales}
    assert_backward(q, p, (x.grad.view(-1, 384), layer.A.grad, layer.B.grad))
    assert torch.equal(layer.values.grad, ks.matmul_dv(q["dy"], q["x"], p))
    assert torch.equal(layer.bias.grad, ks.bias_grad(q["dy"]))
    layer.freeze_base().zero_grad()
    layer(x.detach(), ids).backward(dy)
    assert layer.values.grad is None and layer.bias.grad is None and layer.A.grad is not None


def test_layer_refusals_and_types():
    layer = ks.KSAdapterLinear((1, 64, 48, 8), 2, 4, device=DEV)
    x = torch.randn(6, 384, device=DEV)
    with pytest.raises(ValueError, match="needs ids"):
        layer(x)
    with pytest.raises(ValueError, match="leading shape"):
        layer(x, torch.zeros(5, dtype=torch.int32, device=DEV))
    assert layer.to(torch.bfloat16).scales.dtype == torch.float32
    assert layer(x.bfloat16(), torch.zeros(6, dtype=torch.int32, device=DEV)).dtype == torch.bfloat16
    one = ks.KSAdapterLinear((1, 64, 48, 8), 1, 4, device=DEV)
    assert one(x).shape == (6, 512)


def test_binding_refusals():
    p = (1, 64, 48, 8)
    q = make(p, 6, 2, 8, torch.float32, "rows", 1)
    good = dict(A=q["A"], B=q["B"], ids=q["ids"], scales=q["scales"])
    for name, bad in (("A", q["A"][:, :, 1:]), ("A", q["A"].bfloat16()), ("B", q["B"].transpose(1, 2)),
                      ("B", q["B"][:1]), ("ids", q["ids"].long()), ("ids", q["ids"][:3]), ("ids", q["ids"].cpu()),
                      ("scales", q["scales"].double()), ("scales", q["scales"][:1])):
        with pytest.raises(ValueError):
            ks.adapter_matmul(q["x"], q["values"], p, **dict(good, **{name: bad}))
    with pytest.raises(ValueError):
        ks.adapter_matmul(q["x"][:, :100].contiguous(), q["values"], p, **good)
    with pytest.raises(ValueError):
        ks.adapter_matmul(q["x"], q["values"], p, **good, act="tanh")
    with pytest.raises(ValueError):
        ks.adapter_backward(q["dy"], None, q["values"], p, **good)
    with pytest.raises(ks.KsError, match="overlaps"):
        ks.adapter_matmul(q["x"], q["values"], p, **good, out=q["B"].view(-1)[:6 * 512].view(6, 512))


def layer_of(dtype):
    torch.manual_seed(5)
    layer = ks.KSAdapterLinear((1, 256, 64, 16), 3, 16, bias=True, dtype=dtype, device=DEV)
    with torch.no_grad():
        layer.B.normal_(std=0.1)
    ids = (torch.arange(300, device=DEV) // 70 - 1).clamp(max=2).to(torch.int32)
    return layer, ids, torch.randn(2, 300, 1024, device=DEV, dtype=dtype), torch.randn(2, 300, 4096, device=DEV, dtype=dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_captured_training_step_follows_its_inputs(dtype):
    layer, ids, xs, dys = layer_of(dtype)
    x, dy = xs[0].clone(), dys[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            layer.zero_grad(set_to_none=True)
            layer(x, ids).backward(dy)
    torch.cuda.current_stream().wait_stream(side)
    layer.zero_grad(set_to_none=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = layer(x, ids)
        y.backward(dy)
    for k in (1, 0):
        x.copy_(xs[k]), dy.copy_(dys[k])
        for p in layer.parameters():
            p.grad.zero_()
        g.replay()
        p = layer.pattern
        with torch.no_grad():
            assert torch.equal(y, ks.adapter_matmul(x, layer.values, p, layer.A, layer.B, ids, layer.scales,
                                                    bias=layer.bias))
            _, da, db = ks.adapter_backward(dy, x, layer.values, p, layer.A, layer.B, ids, layer.scales)
        # (a captured gradient is written where it was first made: zeroed or not, it holds this replay's alone)
        assert torch.equal(layer.A.grad, da) and torch.equal(layer.B.grad, db)
        assert torch.equal(layer.bias.grad, ks.bias_grad(dy))
        assert torch.equal(layer.values.grad, ks.matmul_dv(dy, x, p))


def test_capture_is_refused_while_an_eager_graph_of_the_leaves_lives():
    layer, ids, xs, dys = layer_of(torch.bfloat16)
    eager = layer(xs[0], ids)  # on the default stream, never differentiated
    with pytest.raises(RuntimeError, match="still lives"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            layer(xs[0], ids).backward(dys[0])
    with torch.cuda.graph(torch.cuda.CUDAGraph()), torch.no_grad():  # a forward pass has nothing to wait for
        layer(xs[0], ids)
    del eager
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(xs[0], ids).backward(dys[0])
    g.replay()
    _, da, _ = ks.adapter_backward(dys[0], xs[0], layer.values.detach(), layer.pattern, layer.A.detach(),
                                   layer.B.detach(), ids, layer.scales)
    assert torch.equal(layer.A.grad, da)


@pytest.mark.parametrize("p,r", [((1, 96, 80, 1), 17), ((1, 96, 80, 1), 40), ((1, 96, 80, 1), 100), ((2, 32, 48, 4), 64)])
@pytest.mark.parametrize("kind", ["rows", "segments", "one", "none"])
def test_many_rows_of_many_ranks(p, r, kind):
    """More rows than the small tiles of H take at once, in features and rows that no tile divides."""
    q = make(p, 9601, 1 if kind == "one" else 5, r, torch.bfloat16, kind, r, bias=True)
    assert_forward(call(q, p, act="gelu_tanh"), q, p, "gelu_tanh")
    assert_backward(q, p, ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"]))


def test_a_broken_adapter_among_many_rows_of_many_ranks():
    p = (1, 96, 80, 1)
    q = make(p, 9601, 5, 40, torch.bfloat16, "rows", 2)
    clean = call(q, p)
    other = q["ids"] != 1
    q["A"][1, 7] = float("inf")
    q["x"][~other] = float("nan")
    y = call(q, p)
    assert torch.equal(y[other], clean[other]) and torch.isnan(y[~other]).any()
    q["ids"][4000] = 5  # one past the last
    y = ks.adapter_matmul(q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"])
    with pytest.raises(ks.KsError, match="adapter id"):
        ks.sync_status()
    other[4000] = False
    assert torch.equal(y[other], clean[other])


@pytest.mark.parametrize("p", [(2, 162, 23, 8), (3, 38, 9, 5), (1, 150, 150, 1), (5, 33, 30, 9), (1, 200, 199, 20)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens_of_odd_layers(p, dtype):
    """Few rows, sizes of which no vector is a multiple; shift: buffers aligned to their elements alone."""
    for n, r, kind, shift in ((1, 4, "rows", 0), (5, 64, "rows", 0), (33, 13, "segments", 1), (64, 1, "one", 0)):
        q = make(p, n, 1 if kind == "one" else 3, r, dtype, kind, n, bias=True, shift=shift)
        assert_forward(call(q, p, act="gelu_erf"), q, p, "gelu_erf")


@pytest.mark.parametrize("p,n,r,s", [((8, 192, 40, 8), 131, 3, 20), ((4, 48, 48, 4), 2115, 20, 2), ((3, 38, 8, 5), 1203, 64, 2),
                                     ((3, 110, 57, 1), 999, 9, 2), ((4, 19, 2, 13), 289, 64, 1), ((3, 29, 4, 13), 700, 30, 40)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wide_and_odd_layers(p, n, r, s, dtype):
    for kind in ("segments", "rows"):
        q = make(p, n, s, r, dtype, kind, n, bias=True)
        assert_forward(call(q, p, act="relu"), q, p, "relu")
        assert_backward(q, p, ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"]))


@pytest.mark.parametrize("p,n", [((5, 21, 23, 4), 700), ((3, 90, 37, 2), 300), ((1, 16, 4, 1), 4097), ((2, 65, 17, 9), 129),
                                 ((1, 104, 171, 4), 300)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_products_of_odd_layers(p, n, dtype):
    """Blocks that no tile divides, in both directions."""
    q = make(p, n, 2, 6, dtype, "segments", n, bias=True, shift=1)
    assert_forward(call(q, p, act="gelu_tanh"), q, p, "gelu_tanh")
    assert_backward(q, p, ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"]))


def test_layer_scales_keep_their_value_and_empty_batches_their_shape():
    layer = ks.KSAdapterLinear((1, 64, 48, 8), 2, 3, alpha=1, bias=True, device=DEV).to(torch.bfloat16)
    assert torch.equal(layer.scales, torch.full((2,), 1 / 3, device=DEV))
    x = torch.zeros(2, 0, 384, device=DEV, dtype=torch.bfloat16, requires_grad=True)
    y = layer(x, torch.zeros(2, dtype=torch.int32, device=DEV))
    assert y.shape == (2, 0, 512)
    y.sum().backward()
    assert x.grad.shape == x.shape
    for p in layer.parameters():
        assert p.grad.shape == p.shape and not p.grad.any()


def test_two_streams_of_one_device_at_once():
    """Calls in flight beside one another, workspaces of each their own; few rows, stages and a second pass."""
    p = (1, 256, 64, 16)
    qs = [make(p, n, 3, 16, dt, "segments", n, bias=True) for n in (3, 500, 2000) for dt in (torch.bfloat16, torch.float32)]
    want = [(call(q, p), ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"]))
            for q in qs]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for k in range(24):
        q, st = qs[k % len(qs)], streams[k % len(streams)]
        y = ks.adapter_matmul(q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"], bias=q["bias"], stream=st)
        got.append((y, ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"],
                                           stream=st)))
    torch.cuda.synchronize()
    ks.sync_status()
    for k, (y, grads) in enumerate(got):
        assert torch.equal(y, want[k % len(qs)][0])
        assert all(torch.equal(u, v) for u, v in zip(grads, want[k % len(qs)][1]))

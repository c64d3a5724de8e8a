"""One AdamW step over many tensors (ks_adamw_step) and the AdamW optimizer
against the formula in 64 bits.

Tolerances.  A fp32 state is two products and a sum of fp32 numbers: 3 u of the
larger term, u = 2^-24, and v one more product.  The update is a quotient of
about ten fp32 operations: 16 u relative, times lr; p adds one rounding of each
of its terms.  bf16 parameters add half a step, 2^-8 relative.  An 8-bit state
is held to half a step of e4m3, 2^-4 relative of the value (2^-10 of a unit
below 2^-6, in units of the block's scale), and its scale to 4 u.
"""
import copy

import pytest
import torch

import kronecker_sparse_matrix_b200 as ks

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF = 2.0 ** -8
F64 = torch.float64
BLOCK = 256
HYPER = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


def shifted(t, shift):
    buf = torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)
    buf[shift:].copy_(t.reshape(-1))
    return buf[shift:].view(t.shape)


def make(sizes, dtype, bits, master=False, seed=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    q = {k: [] for k in ("p", "g", "m", "v", "master", "ms", "vs")}
    for n in sizes:
        size = torch.exp(2 * torch.randn(n, generator=g)) * 1e-2
        p = torch.randn(n, generator=g).to(dtype)
        grad = (torch.randn(n, generator=g) * size).to(dtype)
        m, v = torch.randn(n, generator=g) * size, size * size * (torch.rand(n, generator=g) + 0.1)
        if bits == 8:
            blocks = -(-n // BLOCK)
            m = (torch.randn(n, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
            v = (torch.rand(n, generator=g) * 448).to(torch.float8_e4m3fn)
            q["ms"].append(torch.rand(blocks, generator=g).mul(1e-4).to(DEV))
            q["vs"].append(torch.rand(blocks, generator=g).mul(1e-4).to(DEV))
        for k, t in (("p", p), ("g", grad), ("m", m), ("v", v)):
            q[k].append(shifted(t, shift))
        if master:
            q["master"].append(shifted(p.float() * (1 + 2 ** -10 * torch.rand(n, generator=g)), shift))
    return q


def step(q, bits, step=7, **more):
    kw = dict(HYPER, step=step, **more)
    if q["master"]:
        kw["masters"] = q["master"]
    if bits == 8:
        kw.update(exp_avg_scales=q["ms"], exp_avg_sq_scales=q["vs"])
    ks.adamw_step(q["p"], q["g"], q["m"], q["v"], **kw)


def spread(scale, n):
    return scale.to(F64).repeat_interleave(BLOCK)[:n]


def reference(q, k, bits, t, scale=1.0, lr=HYPER["lr"]):
    """(p, m, v or sqrt(v)) after the step, in 64 bits, and the tolerance of p."""
    n = q["p"][k].numel()
    b1, b2 = HYPER["betas"]
    g = q["g"][k].to(F64).view(-1) * scale
    p = (q["master"][k] if q["master"] else q["p"][k]).to(F64).view(-1)
    m, v = q["m"][k].to(F64).view(-1), q["v"][k].to(F64).view(-1)
    if bits == 8:
        m, v = m * spread(q["ms"][k], n), (v * spread(q["vs"][k], n)) ** 2
    tm = 4 * U * (b1 * m.abs() + (1 - b1) * g.abs())
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    root = v.sqrt()
    change = lr * (m / (1 - b1 ** t)) / (root / (1 - b2 ** t) ** 0.5 + HYPER["eps"])
    slack = lr * (tm / (1 - b1 ** t)) / (root / (1 - b2 ** t) ** 0.5 + HYPER["eps"])
    new = p * (1 - lr * HYPER["weight_decay"]) - change
    return new, m, (root if bits == 8 else v), tm, 4 * U * p.abs() + 16 * U * change.abs() + slack


def check(q, old, bits, t, **kw):
    for k in range(len(q["p"])):
        n = q["p"][k].numel()
        p, m, v, tm, tp = reference(old, k, bits, t, **kw)
        if q["master"]:
            assert ((q["master"][k].to(F64).view(-1) - p).abs() <= tp).all()
            assert torch.equal(q["p"][k], q["master"][k].to(torch.bfloat16))
        else:
            tol = tp + (BF * (p.abs() + tp) if q["p"][k].dtype == torch.bfloat16 else 0)
            assert ((q["p"][k].to(F64).view(-1) - p).abs() <= tol).all(), k
        for name, ref, tol in (("m", m, tm), ("v", v, 6 * U * v)):
            got = q[name][k].to(F64).view(-1)
            if bits == 8:
                scale = q[name + "s"][k].to(F64)
                pad = torch.zeros(scale.numel() * BLOCK, dtype=F64, device=DEV)
                pad[:n] = ref.abs()
                top = pad.view(-1, BLOCK).amax(1)
                assert ((scale * 448 - top).abs() <= 8 * U * top).all()
                unit = spread(q[name + "s"][k], n)
                # half a step of e4m3; a small sqrt(v) is held up to the smallest number
                half = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** (-9 if name == "v" else -10) * unit)
                assert ((got * unit - ref).abs() <= half * (1 + 1e-5) + tol).all(), (name, k)
                if name == "v":
                    assert ((got > 0) | (ref == 0) | (unit == 0)).all()
            else:
                assert ((got - ref).abs() <= tol).all(), (name, k)


def clone(q):
    return {k: [t.clone() for t in v] for k, v in q.items()}


SIZES = [[1], [255], [256], [257], [2048], [2049], [100003], [0, 5, 0], [1, 300, 4096, 17, 8191, 2, 65536],
         list(range(1, 40))]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtype,master", [(torch.float32, False), (torch.bfloat16, False), (torch.bfloat16, True)])
@pytest.mark.parametrize("bits", [32, 8])
def test_step(sizes, dtype, master, bits):
    for shift in (0, 1):
        q = make(sizes, dtype, bits, master, seed=len(sizes), shift=shift)
        old = clone(q)
        step(q, bits)
        check(q, old, bits, 7)


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_launch_takes(bits):
    q = make([(k * 37) % 700 + 1 for k in range(905)], torch.float32, bits, seed=2)
    old = clone(q)
    step(q, bits, step=1)
    check(q, old, bits, 1)


def test_two_dimensional_and_first_steps():
    """Fresh zero states, several steps: the states follow the recurrence."""
    p = torch.randn(40, 33, device=DEV)
    for bits in (32, 8):
        dt = torch.float32 if bits == 32 else torch.float8_e4m3fn
        q = {"p": [p.clone()], "g": [None], "m": [torch.zeros(40, 33, dtype=dt, device=DEV)],
             "v": [torch.zeros(40, 33, dtype=dt, device=DEV)], "master": [], "ms": [torch.zeros(6, device=DEV)],
             "vs": [torch.zeros(6, device=DEV)]}
        for t in (1, 2, 3):
            q["g"] = [torch.randn(40, 33, device=DEV)]
            old = clone(q)
            step(q, bits, step=t)
            check(q, old, bits, t)


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients_and_tiny_states(bits):
    """Zero gradients and states leave only the weight decay; states decay to
    nothing without NaN or infinities; no update is larger than its formula allows."""
    q = make([600], torch.float32, bits)
    for k in ("g", "m", "v"):
        q[k][0].zero_()
    p = q["p"][0].clone()
    step(q, bits)
    assert torch.allclose(q["p"][0], p * (1 - 1e-2 * 0.1), rtol=4 * U, atol=0)
    q = make([600], torch.float32, bits)
    q["g"][0].zero_()
    q["g"][0][3] = 1e-30  # beside a block of larger ones
    for t in range(1, 2500):
        step(q, bits, step=t)
    for k in ("p", "m", "v"):
        assert torch.isfinite(q[k][0].float()).all()


def test_small_second_state_never_becomes_zero():
    q = make([256], torch.float32, 8)
    q["m"][0].zero_(), q["v"][0].zero_()
    q["g"][0].fill_(1e-6)
    q["g"][0][0] = 1e3
    step(q, 8, step=1)
    assert (q["v"][0].float() > 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_second_state_below_the_normal_range_of_fp32_is_kept(dtype):
    """v is subnormal in fp32 here, about 4e-39; its root, 6e-20, is held."""
    q = make([512], dtype, 8)
    q["m"][0].zero_(), q["v"][0].zero_()
    q["g"][0].fill_(6e-19)
    step(q, 8, step=1)
    g = q["g"][0].double()
    root = spread(q["vs"][0], 512) * q["v"][0].double()
    want = ((1 - HYPER["betas"][1]) * g * g).sqrt()
    # half a step of e4m3; v to half a spacing (2^-149) of the subnormal numbers, 2e-7 of 4e-39
    assert ((root - want).abs() <= (2.0 ** -4 + 1e-5) * want).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_nan_and_infinite_gradients_stay_where_they_are(bits):
    q = make([1024], torch.float32, bits)
    q["g"][0][5], q["g"][0][600] = float("nan"), float("inf")
    old = clone(q)
    step(q, bits)
    ok = torch.ones(1024, dtype=torch.bool, device=DEV)
    ok[5] = ok[600] = False
    assert torch.isnan(q["p"][0][[5, 600]]).all() and torch.isfinite(q["p"][0][ok]).all()
    p = reference(old, 0, bits, 7)[0]
    assert torch.allclose(q["p"][0][ok].to(F64), p[ok], rtol=1e-4, atol=1e-6)
    bad = torch.isnan(q["m"][0].float() * (spread(q["ms"][0], 1024) if bits == 8 else 1))
    assert bad[5] and not bad[:256][ok[:256]].any() and not bad[256:512].any() and not bad[768:].any()
    if bits == 8:
        assert bad[512:768].all()


@pytest.mark.parametrize("bits", [32, 8])
def test_device_scalars_in_a_replayed_graph(bits):
    q = make([3000, 17], torch.bfloat16, bits, master=True)
    eager = clone(q)
    n, lr, gs = (torch.tensor([v], device=DEV, dtype=d) for v, d in ((5, torch.int64), (1e-2, torch.float32),
                                                                    (0.5, torch.float32)))
    kept = clone(q)
    g = torch.cuda.CUDAGraph()
    kw = dict(HYPER, lr=lr, step=n, grad_scale=gs, masters=q["master"])
    if bits == 8:
        kw.update(exp_avg_scales=q["ms"], exp_avg_sq_scales=q["vs"])
    with torch.cuda.graph(g):
        n.add_(1)
        ks.adamw_step(q["p"], q["g"], q["m"], q["v"], **kw)
    for k in q:  # the capture itself ran nothing
        assert all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(q[k], kept[k]))
    for t, rate, scale in ((6, 1e-2, 0.5), (7, 3e-3, 0.25), (8, 1e-3, 2.0)):
        lr.fill_(rate), gs.fill_(scale)
        old = clone(q)
        g.replay()
        torch.cuda.synchronize()
        check(q, old, bits, t, scale=scale, lr=rate)
    del eager


def test_neighbours_are_left_alone():
    """Tensors in one storage: nothing outside them changes."""
    for shift in (0, 1, 8):
        flat = {k: torch.full((4096 + shift,), 7.0, device=DEV) for k in ("p", "m", "v")}
        cut = {k: [f[shift + 16:shift + 16 + 300], f[shift + 1024:shift + 1024 + 2047]] for k, f in flat.items()}
        g = [torch.randn(300, device=DEV), torch.randn(2047, device=DEV)]
        ks.adamw_step(cut["p"], g, cut["m"], cut["v"], step=1, **HYPER)
        for k, f in flat.items():
            keep = torch.ones(4096 + shift, dtype=torch.bool, device=DEV)
            keep[shift + 16:shift + 316] = False
            keep[shift + 1024:shift + 3071] = False
            assert (f[keep] == 7.0).all() and not (f[~keep] == 7.0).all()


def test_refusals():
    q = make([300, 10], torch.float32, 32)
    kw = dict(HYPER, step=1)
    with pytest.raises(ks.KsError, match="overlaps"):
        ks.adamw_step([q["p"][0], q["p"][0]], q["g"][:1] * 2, q["m"][:1] * 2, q["v"][:1] * 2, **kw)
    with pytest.raises(ks.KsError, match="overlaps"):
        ks.adamw_step(q["p"][:1], q["p"][:1], q["m"][:1], q["v"][:1], **kw)
    with pytest.raises(ValueError):
        ks.adamw_step(q["p"], q["g"][:1], q["m"], q["v"], **kw)
    with pytest.raises(ValueError):
        ks.adamw_step(q["p"], q["g"][::-1], q["m"], q["v"], **kw)
    with pytest.raises(ValueError):
        ks.adamw_step(q["p"], [g.cpu() for g in q["g"]], q["m"], q["v"], **kw)
    with pytest.raises(ValueError):
        ks.adamw_step(q["p"], q["g"], q["m"], q["v"], **kw, exp_avg_scales=q["m"], exp_avg_sq_scales=q["v"])
    with pytest.raises(TypeError):
        ks.adamw_step([p.half() for p in q["p"]], q["g"], q["m"], q["v"], **kw)
    with pytest.raises(ks.KsError, match="masters are for bf16"):
        ks.adamw_step(q["p"], q["g"], q["m"], q["v"], **kw, masters=[p.clone() for p in q["p"]])
    ks.adamw_step([], [], [], [], **kw)


# ---------------------------------------------------------------- the optimizer


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_optimizer_follows_adamw_step(bits, dtype):
    torch.manual_seed(1)
    layer = ks.KSAdapterLinear((1, 64, 48, 8), 2, 4, bias=True, dtype=dtype, device=DEV)
    params = list(layer.parameters())
    opt = ks.AdamW(params, state_bits=bits, masters=True, **HYPER)
    assert isinstance(opt, torch.optim.Optimizer)
    x = torch.randn(20, 384, device=DEV, dtype=dtype)
    ids = torch.arange(20, device=DEV, dtype=torch.int32) % 2
    for t in range(1, 4):
        opt.zero_grad()
        if t == 2:  # a parameter that sits out a step keeps its own count
            layer.bias.requires_grad_(False)
        layer(x, ids).float().square().mean().backward()
        layer.bias.requires_grad_(True)
        state = {p: copy.deepcopy(opt.state[p]) if opt.state[p] else opt._init_state(p, opt.param_groups[0])
                 for p in params}
        before = {p: p.detach().clone() for p in params}
        opt.step()
        for p in params:
            if p.grad is None:
                assert torch.equal(p, before[p]) and opt.state[p]["step"] == 1
                continue
            n = state[p]["step"] + 1
            assert opt.state[p]["step"] == n
            q = {"p": [before[p]], "g": [p.grad], "m": [state[p]["exp_avg"]], "v": [state[p]["exp_avg_sq"]],
                 "master": [state[p]["master"]] if dtype == torch.bfloat16 else []}
            q["ms"], q["vs"] = ([state[p]["exp_avg_scale"]], [state[p]["exp_avg_sq_scale"]]) if bits == 8 else ([], [])
            step(q, bits, step=n)
            assert torch.equal(q["p"][0], p.detach())
            assert torch.equal(q["m"][0].view(torch.uint8), opt.state[p]["exp_avg"].view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
def test_optimizer_state_round_trip(bits):
    torch.manual_seed(2)
    a = [torch.nn.Parameter(torch.randn(n, device=DEV, dtype=torch.bfloat16)) for n in (300, 7)]
    opt = ks.AdamW(a, state_bits=bits, masters=True, **HYPER)
    grads = [[torch.randn_like(p) for p in a] for _ in range(4)]
    for g in grads[:2]:
        for p, d in zip(a, g):
            p.grad = d
        opt.step()
    b = [torch.nn.Parameter(p.detach().clone()) for p in a]
    other = ks.AdamW(b, state_bits=bits, masters=True, **HYPER)
    other.load_state_dict(copy.deepcopy(opt.state_dict()))
    for p, q in zip(a, b):
        for name, t in opt.state[p].items():
            if isinstance(t, torch.Tensor):
                u = other.state[q][name]
                assert u.dtype == t.dtype and u.data_ptr() != t.data_ptr()
    for g in grads[2:]:
        for ps, o in ((a, opt), (b, other)):
            for p, d in zip(ps, g):
                p.grad = d
            o.step()
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_optimizer_refuses_capture_and_marks_parameters_changed():
    p = torch.nn.Parameter(torch.randn(100, device=DEV))
    opt = ks.AdamW([p], **HYPER)
    p.grad = torch.randn_like(p)
    version = p._version
    opt.step()
    assert p._version > version
    g = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="adamw_step"):
        with torch.cuda.graph(g):
            opt.step()
    torch.cuda.synchronize()


def test_fine_tuning_step_as_used():
    """Adapters over a frozen layer, their gradients and the 8-bit step together:
    the step moves A and B by the formula and leaves the base alone."""
    torch.manual_seed(3)
    layer = ks.KSAdapterLinear((1, 256, 64, 16), 4, 16, bias=True, dtype=torch.bfloat16, device=DEV).freeze_base()
    with torch.no_grad():
        layer.B.normal_(std=0.1)
    opt = ks.AdamW([p for p in layer.parameters() if p.requires_grad], state_bits=8, masters=True, **HYPER)
    values = layer.values.detach().clone()
    x = torch.randn(500, 1024, device=DEV, dtype=torch.bfloat16)
    ids = torch.arange(500, device=DEV, dtype=torch.int32) // 125
    for _ in range(3):
        opt.zero_grad()
        y = layer(x, ids)
        y.backward(y.detach())
        opt.step(grad_scale=torch.tensor([0.5], device=DEV))
    ks.sync_status()
    assert torch.equal(values, layer.values) and all(torch.isfinite(p).all() for p in layer.parameters())
    assert all(opt.state[p]["step"] == 3 for p in (layer.A, layer.B))

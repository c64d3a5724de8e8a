"""Cases of the operators that fine-tune and serve Kronecker-sparse (KS) linear layers.

* adapter: low-rank adapters of many requests beside one shared KS projection,
      Y[n] = act(X[n] K^T + bias + scales[s] (X[n] A[s]^T) B[s]^T),  s = ids[n],
  a row whose id is negative taking none;
* adapter_grad: its gradients dX, dA, dB from dY (no activation);
* adamw: one AdamW step over many tensors, its two states in 32 bits or in 8 bits
  (e4m3 numbers with one fp32 scale for each 256 elements; the second state held as its square root).

``run`` computes a case in plain torch operations, or, with ``own`` set, through the package's entry points.
"""
import math

import torch

own = False

BLOCK = 256  # elements of a tensor that share a scale in an 8-bit state
TOP = 448.0  # largest e4m3 number
LOW = 2.0 ** -9  # smallest positive e4m3 number
NONE = 2.0 ** -100  # a block with nothing larger is held as zeros

_DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _adapter(op, pattern, batch, adapters, rank, ids, dtype, act="none", bias=False):
    a, b, c, d = pattern
    case = {"op": op, "a": a, "b": b, "c": c, "d": d, "batch": batch, "adapters": adapters, "rank": rank, "ids": ids,
            "dtype": dtype}
    if op == "adapter":
        case.update(act=act, bias=bias)
    return case


def _adamw(bits, count, small, large, dtype, master=False, shift=0):
    return {"op": "adamw", "bits": bits, "count": count, "small": small, "large": large, "dtype": dtype,
            "master": master, "shift": shift}


def listed():
    gpt2, vit = (1, 256, 64, 16), (1, 192, 48, 8)  # the MLP up-projections of the package's workloads
    cases = {
        # one token of one request: latency
        "fwd decode 1": _adapter("adapter", gpt2, 1, 4, 16, "rows", "bf16", "gelu_tanh", True),
        # one token of each of 32 requests, most with an adapter of their own
        "fwd decode 32": _adapter("adapter", gpt2, 32, 32, 16, "rows", "bf16", "gelu_tanh", True),
        # prompts of several requests packed into one batch, each with its adapter
        "fwd prefill": _adapter("adapter", gpt2, 8192, 8, 16, "segments", "bf16", "gelu_tanh", True),
        # a ViT layer in fp32 under four fine-tuned variants, ragged groups of images
        "fwd vit fp32": _adapter("adapter", vit, 25216, 4, 8, "segments", "fp32", "gelu_erf", True),
        # the widest layer of the pattern sweep, rank 64
        "fwd wide": _adapter("adapter", (4, 256, 64, 16), 8192, 4, 64, "segments", "bf16"),
        # an odd little layer: nothing a multiple of anything
        "bwd odd fp32": _adapter("adapter_grad", (3, 20, 12, 5), 77, 3, 5, "rows", "fp32"),
        # one training step of a GPT-2-shaped layer, eight adapters trained side by side
        "bwd gpt2": _adapter("adapter_grad", gpt2, 8192, 8, 16, "segments", "bf16"),
        # a ViT layer in fp32, one adapter
        "bwd vit fp32": _adapter("adapter_grad", vit, 25216, 1, 8, "one", "fp32"),
        # the twelve factors of the 4096-wide butterfly: many small tensors, latency
        "adamw butterfly": _adamw(32, 12, 8192, 8192, "fp32"),
        # values, biases and adapters of a stack of layers, bf16 with fp32 masters
        "adamw layers": _adamw(32, 144, 4096, 2097152, "bf16", master=True),
        # the same stack's odd-sized pieces with 8-bit states
        "adamw8 odd": _adamw(8, 60, 37, 300001, "fp32"),
        # a model's worth of parameters with 8-bit states
        "adamw8 large": _adamw(8, 40, 1048576, 8388608, "bf16"),
    }
    return [dict(case, name=name) for name, case in cases.items()]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    if rng.random() < 0.4:
        bits, dtype = rng.choice((8, 32)), rng.choice(("fp32", "bf16"))
        count, small = _log(rng, 1, 150), _log(rng, 1, 100000)
        large = _log(rng, small, max(small, min(8388608, 150000000 // count)))
        return _adamw(bits, count, small, large, dtype, dtype == "bf16" and rng.random() < 0.5, rng.choice((0, 0, 1)))
    op = rng.choice(("adapter", "adapter", "adapter_grad"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    while True:
        if rng.random() < 0.6:  # the sweep's patterns
            b, c = rng.choice(((48, 48), (64, 64), (96, 96), (128, 128), (192, 192), (256, 256), (192, 48), (256, 64)))
            a, d = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 8, 16))
        else:
            a, b, c, d = _log(rng, 1, 8), _log(rng, 2, 200), _log(rng, 2, 200), _log(rng, 1, 24)
        if a * b * d <= 16384 and a * c * d <= 4096:
            break
    rank = rng.choice((1, 4, 8, 8, 16, 16, 16, 32, 64, rng.randint(1, 64)))
    adapters = _log(rng, 1, 16 if rank > 16 else 32)
    # one draw in three is a batch of single tokens
    cells = 8192 * 16384 if dtype == "bf16" else 25216 * 1536
    most = max(64, min(25216, cells // max(a * b * d, a * c * d)))
    batch = _log(rng, 1, 64) if rng.random() < 0.33 else _log(rng, 64, most)
    ids = rng.choice(("rows", "one")) if batch <= 64 else rng.choice(("segments", "segments", "segments", "one"))
    return _adapter(op, (a, b, c, d), batch, 1 if ids == "one" else adapters, rank, ids, dtype,
                    rng.choice(("none", "relu", "gelu_tanh", "gelu_erf")), rng.random() < 0.5)


# ---------------------------------------------------------------- inputs


def _sizes(case):
    """Sizes of the tensors of an adamw case: spread over the logarithm of the range, large and small mixed."""
    n, lo, hi = case["count"], math.log(case["small"]), math.log(case["large"])
    return [int(round(math.exp(lo + (hi - lo) * ((7 * k) % n) / max(1, n - 1)))) for k in range(n)]


def _slots(case):
    """(start, size) of each tensor in the flat buffers, starts a multiple of BLOCK; and the buffers' length."""
    at, slots = 0, []
    for n in _sizes(case):
        slots.append((at, n))
        at += -(-n // BLOCK) * BLOCK
    return slots, at


def _ids(case, gen, dev):
    n, s = case["batch"], case["adapters"]
    if case["ids"] == "one":
        return None
    if case["ids"] == "rows":  # any row any adapter, about one in eight none
        r = torch.randint(0, s, (n,), generator=gen, device=dev)
        return torch.where(torch.rand(n, generator=gen, device=dev) < 0.125, -1, r).to(torch.int32)
    # requests of ragged lengths in the order they came, at least one without an adapter where there is room
    cuts = torch.sort(torch.randint(0, n, (2 * s,), generator=gen, device=dev)).values
    seg = torch.bucketize(torch.arange(n, device=dev), cuts, right=True)
    who = torch.randint(0, s, (2 * s + 1,), generator=gen, device=dev)
    who[torch.randint(0, 2 * s + 1, (1,), generator=gen, device=dev)] = -1
    return who[seg].to(torch.int32)


def _prepare_adapter(case, gen, dev):
    a, b, c, d = (case[k] for k in "abcd")
    n, s, r, dt = case["batch"], case["adapters"], case["rank"], _DT[case["dtype"]]
    fin, fout = a * c * d, a * b * d

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev).mul_(std).to(dt)

    st = {"x": normal(n, fin), "values": normal(a, d, b, c, std=c ** -0.5), "A": normal(s, r, fin, std=fin ** -0.5),
          "B": normal(s, fout, r, std=0.5 * r ** -0.5), "ids": _ids(case, gen, dev),
          "scales": torch.rand(s, generator=gen, device=dev).mul_(1.5).add_(0.5)}
    if case["op"] == "adapter":
        st["bias"] = normal(fout, std=0.1) if case["bias"] else None
    else:
        st["dy"] = normal(n, fout, std=0.01)
    return st


def _pack(t):
    """A flat fp32 state in 8 bits: e4m3 codes and a scale for each BLOCK (the largest magnitude is TOP)."""
    t = t.view(-1, BLOCK)
    top = t.abs().amax(1, keepdim=True)
    top = torch.where(top < NONE, torch.zeros_like(top), top)
    inverse = torch.where(top == 0, torch.zeros_like(top), TOP / top)
    code = (t * inverse).clamp(-TOP, TOP)
    return code, (top / TOP).view(-1)


def _prepare_adamw(case, gen, dev):
    slots, total = _slots(case)
    dt, shift = _DT[case["dtype"]], case["shift"]

    def flat(dtype):
        """A zeroed buffer that starts `shift` elements into its storage, and the tensors in it."""
        return torch.zeros(total + shift, dtype=dtype, device=dev)[shift:]

    def split(buf):
        return [buf[at:at + n] for at, n in slots]

    inside = torch.zeros(total, dtype=torch.bool, device=dev)
    for part in split(inside):
        part.fill_(True)

    def fill(dtype, t):
        buf = flat(dtype)
        buf.copy_(torch.where(inside, t, torch.zeros_like(t)))
        return buf

    def normal():
        return torch.randn(total, generator=gen, device=dev)

    # gradients over several orders of magnitude, some exactly zero; states of a run well under way
    size = torch.exp(1.5 * normal()) * 1e-3
    g = torch.where(torch.rand(total, generator=gen, device=dev) < 0.02, torch.zeros_like(size), normal() * size)
    p, m, v = normal() * 0.1, normal() * size * 0.3, size * size * (0.25 + torch.rand(total, generator=gen, device=dev))
    st = {"slots": slots, "p": fill(dt, p), "g": fill(dt, g)}
    st["master"] = fill(torch.float32, st["p"].float()) if case["master"] else None
    if case["master"]:
        st["master"].add_(torch.where(inside, st["master"] * (torch.rand(total, generator=gen, device=dev) - 0.5) * 2 ** -9, 0))
    if case["bits"] == 8:
        for name, t in (("m", m), ("v", v.sqrt())):
            code, scale = _pack(torch.where(inside, t, torch.zeros_like(t)))
            st[name] = flat(torch.float8_e4m3fn)
            st[name].copy_(code.reshape(-1).to(torch.float8_e4m3fn))
            st[name + "_scale"] = scale
    else:
        st["m"], st["v"] = fill(torch.float32, m), fill(torch.float32, v)
    for name in ("p", "g", "m", "v", "master"):
        st[name + "s"] = split(st[name]) if st[name] is not None else None
    if case["bits"] == 8:
        for name in ("m_scale", "v_scale"):
            st[name + "s"] = [st[name][at // BLOCK:at // BLOCK + -(-n // BLOCK)] for at, n in slots]
    st["hyper"] = {"lr": 2e-4, "betas": (0.9, 0.999), "eps": 1e-8, "weight_decay": 0.1, "step": 1000}
    return st


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    st = _prepare_adamw(case, gen, dev) if case["op"] == "adamw" else _prepare_adapter(case, gen, dev)
    return dict(st, case=case)


# ---------------------------------------------------------------- plain forms


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "gelu_erf":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _ks(x, values):
    """x (n, a*c*d) times the transposed KS factor with these values (a, d, b, c): a batch of a*d products."""
    a, d, b, c = values.shape
    n = x.shape[0]
    xs = x.view(n, a, c, d).permute(1, 3, 0, 2).reshape(a * d, n, c)
    y = torch.bmm(xs, values.reshape(a * d, b, c).transpose(1, 2))
    return y.view(a, d, n, b).permute(2, 0, 3, 1).reshape(n, a * b * d)


def _weights(st):
    """scales[s] where row n takes adapter s, 0 elsewhere: (n, adapters, 1)."""
    s = st["A"].shape[0]
    if st["ids"] is None:
        return st["scales"].view(1, s, 1).expand(st["x"].shape[0], s, 1)
    hit = st["ids"].view(-1, 1) == torch.arange(s, device=st["ids"].device).view(1, -1)
    return torch.where(hit, st["scales"].view(1, -1), 0.0).unsqueeze(2)


def _plain_adapter(st):
    x, A, B = st["x"].float(), st["A"].float(), st["B"].float()
    s, r, fin = A.shape
    h = ((x @ A.view(s * r, fin).t()).view(-1, s, r) * _weights(st)).view(-1, s * r)
    y = _ks(x, st["values"].float()) + h @ B.transpose(1, 2).reshape(s * r, -1)
    if st["bias"] is not None:
        y = y + st["bias"].float()
    return _act(y, st["case"]["act"]).to(st["x"].dtype)


def _plain_adapter_grad(st):
    x, dy, A, B = st["x"].float(), st["dy"].float(), st["A"].float(), st["B"].float()
    s, r, fin = A.shape
    w = _weights(st)
    Af, Bf = A.view(s * r, fin), B.transpose(1, 2).reshape(s * r, -1)
    h = ((x @ Af.t()).view(-1, s, r) * w).view(-1, s * r)
    g = ((dy @ Bf.t()).view(-1, s, r) * w).view(-1, s * r)
    dx = _ks(dy, st["values"].float().transpose(2, 3)) + g @ Af
    da = (g.t() @ x).view(s, r, fin)
    db = (h.t() @ dy).view(s, r, -1).transpose(1, 2)
    dt = st["x"].dtype
    return {"dx": dx.to(dt), "da": da.to(dt), "db": db.to(dt)}


def _plain_adamw(st):
    h, bits = st["hyper"], st["case"]["bits"]
    b1, b2 = h["betas"]
    g = st["g"].float()
    if bits == 8:
        m = st["m"].float().view(-1, BLOCK) * st["m_scale"].view(-1, 1)
        v = st["v"].float().view(-1, BLOCK) * st["v_scale"].view(-1, 1)
        m, v = m.view(-1), (v * v).view(-1)
    else:
        m, v = st["m"], st["v"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    root = v.sqrt()
    p = st["master"] if st["master"] is not None else st["p"].float()
    change = m / (root * (1 / math.sqrt(1 - b2 ** h["step"])) + h["eps"])
    p = p * (1 - h["lr"] * h["weight_decay"]) - change * (h["lr"] / (1 - b1 ** h["step"]))
    if st["master"] is not None:
        st["master"].copy_(p)
    st["p"].copy_(p)
    if bits == 8:
        code, scale = _pack(m)
        st["m"].copy_(code.view(-1).to(torch.float8_e4m3fn))
        st["m_scale"].copy_(scale)
        code, scale = _pack(root)
        # a second state above zero stays above zero, so that no step divides by eps alone
        code = torch.where(root.view(-1, BLOCK) > 0, code.clamp_min(LOW), code)
        st["v"].copy_(code.view(-1).to(torch.float8_e4m3fn))
        st["v_scale"].copy_(scale)
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)


def _adamw_outputs(st):
    names = ("p", "m", "v", "master") + (("m_scale", "v_scale") if st["case"]["bits"] == 8 else ())
    return {k: st[k] for k in names if st[k] is not None}


def run(st):
    op = st["case"]["op"]
    if own:
        import kronecker_sparse_matrix_b200 as ks
        pattern = tuple(st["case"][k] for k in "abcd") if op != "adamw" else None
        if op == "adapter":
            return ks.adapter_matmul(st["x"], st["values"], pattern, st["A"], st["B"], st["ids"], st["scales"],
                                     bias=st["bias"], act=st["case"]["act"])
        if op == "adapter_grad":
            dx, da, db = ks.adapter_backward(st["dy"], st["x"], st["values"], pattern, st["A"], st["B"], st["ids"],
                                             st["scales"])
            return {"dx": dx, "da": da, "db": db}
        more = {"exp_avg_scales": st["m_scales"], "exp_avg_sq_scales": st["v_scales"]} if st["case"]["bits"] == 8 else {}
        ks.adamw_step(st["ps"], st["gs"], st["ms"], st["vs"], masters=st["masters"], **more, **st["hyper"])
        return _adamw_outputs(st)
    if op == "adapter":
        return _plain_adapter(st)
    if op == "adapter_grad":
        return _plain_adapter_grad(st)
    _plain_adamw(st)
    return _adamw_outputs(st)


# ---------------------------------------------------------------- 64 bits


def _round_e4m3(t):
    """Nearest e4m3 number, ties to even, of float64 values in [-448, 448]."""
    _, e = torch.frexp(t)
    step = torch.exp2((e - 1).clamp_min(-6).to(torch.float64) - 3)
    return torch.round(t / step) * step


def _exact_adamw(st):
    h, bits = st["hyper"], st["case"]["bits"]
    f = torch.float64
    g, p = st["g"].to(f), (st["p"] if st["master"] is None else st["master"]).to(f)
    m, v = st["m"].to(f), st["v"].to(f)
    if bits == 8:
        m = m * st["m_scale"].to(f).repeat_interleave(BLOCK)
        v = (v * st["v_scale"].to(f).repeat_interleave(BLOCK)) ** 2
    b1, b2 = h["betas"]
    m += (1 - b1) * (g - m)
    v += (1 - b2) * (g ** 2 - v)
    mhat, vhat = m / (1 - b1 ** h["step"]), v / (1 - b2 ** h["step"])
    p = p - h["lr"] * h["weight_decay"] * p - h["lr"] * mhat / (vhat.sqrt() + h["eps"])
    out = {"p": p, "m": m, "v": v}
    if st["master"] is not None:
        out["master"] = p
    if bits == 8:
        for name, t in (("m", m), ("v", v.sqrt())):
            blocks = t.view(-1, BLOCK)
            scale = blocks.abs().max(1).values / TOP
            code = torch.nan_to_num(blocks / scale.view(-1, 1))
            code = _round_e4m3(code)
            if name == "v":
                code = torch.where((blocks > 0) & (code < LOW), LOW, code)
            out[name], out[name + "_scale"] = code.view(-1), scale
    return out


def _exact_adapter(st):
    f = torch.float64
    case = st["case"]
    a, b, c, d = (case[k] for k in "abcd")
    x, V, A, B = (st[k].to(f) for k in ("x", "values", "A", "B"))
    n, grad = x.shape[0], case["op"] == "adapter_grad"
    rows = [torch.nonzero(st["ids"] == s).view(-1) if st["ids"] is not None else torch.arange(n, device=x.device)
            for s in range(A.shape[0])]
    scales = st["scales"].to(f)
    if not grad:
        y = torch.einsum("nijl,ilkj->nikl", x.view(n, a, c, d), V).reshape(n, -1)
        for s, at in enumerate(rows):
            y[at] += scales[s] * torch.einsum("nr,fr->nf", torch.einsum("nf,rf->nr", x[at], A[s]), B[s])
        if st["bias"] is not None:
            y += st["bias"].to(f)
        if case["act"] == "relu":
            y = y.relu()
        elif case["act"] != "none":
            y = torch.nn.functional.gelu(y, approximate="tanh" if case["act"] == "gelu_tanh" else "none")
        return y
    dy = st["dy"].to(f)
    dx = torch.einsum("nikl,ilkj->nijl", dy.view(n, a, b, d), V).reshape(n, -1)
    da, db = torch.zeros_like(A), torch.zeros_like(B)
    for s, at in enumerate(rows):
        xs, ys = x[at], scales[s] * dy[at]
        dx[at] += torch.einsum("nf,fr,rg->ng", ys, B[s], A[s])
        da[s] = torch.einsum("nf,fr,ng->rg", ys, B[s], xs)
        db[s] = torch.einsum("nf,ng,rg->fr", ys, xs, A[s])
    return {"dx": dx, "da": da, "db": db}


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_adamw(st) if case["op"] == "adamw" else _exact_adapter(st)


# ---------------------------------------------------------------- work


def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        blocks = sum(-(-k // BLOCK) for k in _sizes(case))
        p = 3 * e if not case["master"] else 2 * e + 8  # p, g read, p written; a master replaces the read of p
        s = 4 if case["bits"] == 8 else 16
        return {"bytes": n * (p + s) + (16 * blocks if case["bits"] == 8 else 0), "flops": 15 * n}
    a, b, c, d = (case[k] for k in "abcd")
    n, s, r = case["batch"], case["adapters"], case["rank"]
    fin, fout = a * c * d, a * b * d
    params = a * b * c * d + min(s, n) * r * (fin + fout)
    base, low = 2 * n * a * b * c * d, 2 * n * r * (fin + fout)
    if case["op"] == "adapter":
        return {"bytes": e * (n * (fin + fout) + params + (fout if case["bias"] else 0)) + 4 * (n + s), "flops": base + low}
    grads = s * r * (fin + fout)
    return {"bytes": e * (n * (2 * fin + fout) + params + grads) + 4 * (n + s),
            "flops": base + 2 * low + 2 * n * r * fin}

"""Low-rank adapters of many requests beside one shared KS projection:
``adapter_matmul``, its gradients ``adapter_backward`` and the layer built on
them, ``KSAdapterLinear``.  As in the rest of the package, this module only
marshals torch tensors into the C ABI (ks_adapter_matmul, ks_adapter_backward).
"""
from __future__ import annotations

import threading
import weakref
from typing import Optional

import torch

from . import KS_BF16, KS_F32, KS_TF32, KSLinear, Pattern, _act, _lib, bias_grad, matmul_dv

_DTYPES, _DTYPES_TF32 = (KS_F32, KS_BF16), (KS_TF32, -1)


def _on_device(run, args, x, stream):
    """run(*args, stream) with x's device current; on a stream given, new tensors' memory belongs to it."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return run(*args, stream.cuda_stream)
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.get_device() == torch.cuda.current_device():
        return run(*args, None)
    with torch.cuda.device(x.get_device()):
        return run(*args, None)


def adapter_matmul(x: torch.Tensor, values: torch.Tensor, pattern: Pattern, A: torch.Tensor, B: torch.Tensor,
                   ids: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None, *,
                   bias: Optional[torch.Tensor] = None, act: str = "none", out: Optional[torch.Tensor] = None,
                   tf32: bool = False, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Y[n] = act(X[n] K^T + bias + scales[s] (X[n] A[s]^T) B[s]^T) with s = ids[n].

    x: (batch, a*c*d); values, bias and act as for ``matmul``; A: (adapters,
    rank, a*c*d); B: (adapters, a*b*d, rank), both of x's dtype; ids: int32, one
    per row (a negative id: no adapter; None: every row takes adapter 0);
    scales: float32, one per adapter (None: ones).  An id that is too large
    takes no adapter, and the next ``sync_status`` raises.  Rows of one adapter
    next to each other run fastest.  Sums are fp32, a bf16 Y is rounded once (and
    X A[s]^T where it is a tensor-core operand).  Asynchronous on ``stream``."""
    from ._ks_marshal import adapter_matmul as run  # built with the library
    a, b, c, d = pattern
    args = (_lib.address("ks_adapter_matmul"), x, values, A, B, ids, scales, bias, out, int(a), int(b), int(c), int(d),
            _act(act), _DTYPES_TF32 if tf32 else _DTYPES)
    if values is None:
        raise ValueError("values must be a tensor")
    given = out is not None
    status, out = _on_device(run, args, x, stream)
    if status:
        _lib.check(status)
    if given:
        torch.autograd.graph.increment_version(out)  # changed in place behind autograd's back
    return out


def adapter_backward(dy: torch.Tensor, x: Optional[torch.Tensor], values: Optional[torch.Tensor], pattern: Pattern,
                     A: torch.Tensor, B: torch.Tensor, ids: Optional[torch.Tensor] = None,
                     scales: Optional[torch.Tensor] = None, *, need_dx: bool = True, need_da: bool = True,
                     need_db: bool = True, tf32: bool = False, stream: Optional[torch.cuda.Stream] = None):
    """Gradients (dX, dA, dB) of ``adapter_matmul`` without an activation from
    dY (batch, a*b*d); None in the place of one that is not needed (values may
    be None without dX, x without dA and dB).  An adapter without rows gets
    zeros.  Deterministic; fp32 sums, bf16 gradients rounded once (and dY B[s] and
    X A[s]^T where they are tensor-core operands).  A gradient asked for alone has
    the bits it has beside the others."""
    from ._ks_marshal import adapter_backward as run  # built with the library
    a, b, c, d = pattern
    args = (_lib.address("ks_adapter_backward"), dy, values, A, B, ids, scales, x, int(a), int(b), int(c), int(d),
            need_dx, need_da, need_db, _DTYPES_TF32 if tf32 else _DTYPES)
    status, dx, da, db = _on_device(run, args, dy, stream)
    if status:
        _lib.check(status)
    return dx, da, db


class _EagerGraph:
    """The leaves of an autograd graph recorded on the default stream, while that graph lives.

    A leaf's gradient is accumulated on the stream where the first living graph of it was
    recorded.  Were that the default stream, a captured backward pass would have to
    wait there, which no capture allows: the engine's error can end the process.  So a
    backward pass refuses it before it starts."""
    __slots__ = ("leaves", "__weakref__")


_eager_graphs = weakref.WeakSet()
_eager_lock = threading.Lock()  # backward passes run in autograd's threads


class _KSAdapterFn(torch.autograd.Function):
    """y = x K^T + bias + the adapters' products; every gradient on the GPU."""

    @staticmethod
    def forward(ctx, x, values, bias, A, B, scales, ids, pattern):
        ctx.leaves = [weakref.ref(t) for t, need in zip((x, values, bias, A, B), ctx.needs_input_grad)
                      if need and t.is_leaf]
        if ctx.leaves and x.is_cuda and torch.cuda.current_stream(x.device).cuda_stream == 0:
            ctx.graph = _EagerGraph()
            ctx.graph.leaves = ctx.leaves
            with _eager_lock:
                _eager_graphs.add(ctx.graph)
        values, A, B = values.contiguous(), A.contiguous(), B.contiguous()
        ctx.pattern = pattern
        ctx.save_for_backward(x, values, A, B, scales, ids)
        return adapter_matmul(x, values, pattern, A, B, ids, scales, bias=bias)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, values, A, B, scales, ids = ctx.saved_tensors
        need = ctx.needs_input_grad
        if torch.cuda.is_current_stream_capturing():
            mine = {id(leaf()) for leaf in ctx.leaves} - {id(None)}
            with _eager_lock:
                graphs = list(_eager_graphs)
            if any(id(leaf()) in mine for graph in graphs for leaf in graph.leaves):
                raise RuntimeError("an autograd graph of the same tensors, recorded on the default stream, still lives: "
                                   "release its results before a backward pass is captured")
        dy = dy.contiguous()
        dx = da = db = None
        if need[0] or need[3] or need[4]:
            dx, da, db = adapter_backward(dy, x, values, ctx.pattern, A, B, ids, scales, need_dx=need[0],
                                          need_da=need[3], need_db=need[4])
        dv = matmul_dv(dy, x, ctx.pattern) if need[1] else None
        dbias = bias_grad(dy) if need[2] else None
        return dx, dv, dbias, da, db, None, None, None


class KSAdapterLinear(KSLinear):
    """A KSLinear with low-rank adapters beside it: y = x K^T (+ bias) +
    alpha/rank (x A[s]^T) B[s]^T, s the row's adapter.

    A (n_adapters, rank, in_features) is drawn N(0, 1/in_features), B
    (n_adapters, out_features, rank) starts at zero, so a fresh layer is its
    KSLinear.  ``scales`` is a buffer of alpha/rank per adapter (alpha defaults
    to rank).  ``freeze_base()`` leaves the adapters alone to be trained.  A
    training step can be captured into a CUDA graph once the results of earlier steps
    on the default stream are released (warm up on another stream)."""

    def __init__(self, pattern: Pattern, n_adapters: int, rank: int, alpha: Optional[float] = None, bias: bool = False,
                 dtype=torch.float32, device=None):
        super().__init__(pattern, bias=bias, dtype=dtype, device=device)
        if n_adapters < 1 or rank < 1:
            raise ValueError("n_adapters and rank must be positive")
        A = torch.randn(n_adapters, rank, self.in_features, dtype=dtype, device=device) * self.in_features ** -0.5
        self.A = torch.nn.Parameter(A)
        self.B = torch.nn.Parameter(torch.zeros(n_adapters, self.out_features, rank, dtype=dtype, device=device))
        self.register_buffer("scales", torch.full((n_adapters,), (rank if alpha is None else alpha) / rank,
                                                  dtype=torch.float32, device=device))

    def _apply(self, fn, recurse=True):
        scales = self.scales
        super()._apply(fn, recurse)
        if self.scales.dtype != torch.float32:  # the scales stay what they are under .to(dtype)
            self.scales = scales.to(self.scales.device)
        return self

    def freeze_base(self) -> "KSAdapterLinear":
        self.values.requires_grad_(False)
        if self.bias is not None:
            self.bias.requires_grad_(False)
        return self

    def forward(self, x: torch.Tensor, ids: Optional[torch.Tensor] = None) -> torch.Tensor:
        """ids: int32, of x's leading shape or of its first dimensions (one id
        for each sequence of a padded batch, say); None where the layer has a
        single adapter."""
        lead = x.shape[:-1]
        if ids is None:
            if self.A.shape[0] != 1:
                raise ValueError("a layer with several adapters needs ids")
        else:
            if ids.shape != lead[:ids.dim()]:
                raise ValueError(f"ids must have x's leading shape {tuple(lead)} or its first dimensions")
            ids = ids.reshape(ids.shape + (1,) * (len(lead) - ids.dim())).expand(lead).reshape(-1).contiguous()
        y = _KSAdapterFn.apply(x.reshape(-1, self.in_features).contiguous(), self.values, self.bias, self.A, self.B,
                               self.scales, ids, self.pattern)
        return y.reshape(*lead, self.out_features)

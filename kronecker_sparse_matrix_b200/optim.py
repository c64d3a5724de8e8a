"""AdamW over many tensors in one launch: ``adamw_step`` (ks_adamw_step) and the
optimizer class ``AdamW`` built on it, with states in 32 bits or in 8 bits."""
from __future__ import annotations

import array
import ctypes
from itertools import chain, repeat
from operator import attrgetter
from typing import Optional, Sequence, Tuple, Union

import torch

from . import KS_BF16, KS_F32, _lib, _stream_ptr

ADAMW_BLOCK = 256  # elements that share a scale in an 8-bit state

_dtype, _device = attrgetter("dtype"), attrgetter("device")
_ptr, _numel, _contiguous = torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.is_contiguous


def _pointers(name: str, tensors, count: int, dtype: torch.dtype, device: torch.device, numels=None):
    """The tensors' addresses, after checking them."""
    if len(tensors) != count:
        raise ValueError(f"{name} must have one tensor for each parameter")
    if set(map(_dtype, tensors)) != {dtype} or set(map(_device, tensors)) != {device}:
        raise ValueError(f"{name} must be {dtype} tensors on {device}")
    if not all(map(_contiguous, tensors)):
        raise ValueError(f"{name} must be contiguous")
    if numels is not None and list(map(_numel, tensors)) != numels:
        raise ValueError(f"{name} must have the parameters' element counts (scales: one for each {ADAMW_BLOCK})")
    return map(_ptr, tensors)


def _scalar(name: str, t: torch.Tensor, dtype: torch.dtype, device: torch.device) -> int:
    if t.dtype != dtype or t.device != device or t.numel() != 1:
        raise ValueError(f"{name} as a tensor must hold one {dtype} on {device}")
    return t.data_ptr()


def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], exp_avgs: Sequence[torch.Tensor],
               exp_avg_sqs: Sequence[torch.Tensor], *, step: Union[int, torch.Tensor],
               lr: Union[float, torch.Tensor], betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
               weight_decay: float = 1e-2, masters: Optional[Sequence[torch.Tensor]] = None,
               exp_avg_scales: Optional[Sequence[torch.Tensor]] = None,
               exp_avg_sq_scales: Optional[Sequence[torch.Tensor]] = None,
               grad_scale: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
    """One AdamW step, in place, over a list of tensors of one dtype (fp32 or
    bf16) and device: m = b1 m + (1-b1) g, v = b2 v + (1-b2) g^2, p = p (1 - lr wd)
    - lr m/(1-b1^t) / (sqrt(v/(1-b2^t)) + eps).

    States: fp32 tensors; or torch.float8_e4m3fn tensors holding m and sqrt(v)
    with ``exp_avg_scales`` and ``exp_avg_sq_scales``, fp32 tensors of
    ceil(numel/256) scales (zeros are valid fresh states of both kinds).
    ``masters``: fp32 masters of bf16 parameters.  step counts from 1.  step (int64), lr and
    grad_scale (float32) may be one-element CUDA tensors, read when the step
    runs: a captured step follows them.  Asynchronous on ``stream``."""
    count = len(params)
    if count == 0:
        return
    dt, dev = params[0].dtype, params[0].device
    if dt not in (torch.float32, torch.bfloat16):
        raise TypeError(f"unsupported dtype {dt}: use float32 or bfloat16")
    if dev.type != "cuda":
        raise ValueError("params must be CUDA tensors")
    numels = list(map(_numel, params))
    if len(exp_avgs) != count:
        raise ValueError("exp_avgs must have one tensor for each parameter")
    state = exp_avgs[0].dtype
    if state not in (torch.float32, torch.float8_e4m3fn):
        raise TypeError(f"unsupported state dtype {state}: use float32 or float8_e4m3fn")
    bits = 8 if state is torch.float8_e4m3fn else 32
    if (bits == 8) != (exp_avg_scales is not None) or (bits == 8) != (exp_avg_sq_scales is not None):
        raise ValueError("8-bit states need exp_avg_scales and exp_avg_sq_scales, 32-bit states take none")
    none = repeat(0, count)
    columns = [_pointers("params", params, count, dt, dev), _pointers("grads", grads, count, dt, dev, numels),
               _pointers("exp_avgs", exp_avgs, count, state, dev, numels),
               _pointers("exp_avg_sqs", exp_avg_sqs, count, state, dev, numels),
               none if masters is None else _pointers("masters", masters, count, torch.float32, dev, numels)]
    if bits == 8:
        blocks = [(n + ADAMW_BLOCK - 1) // ADAMW_BLOCK for n in numels]
        columns += [_pointers("exp_avg_scales", exp_avg_scales, count, torch.float32, dev, blocks),
                    _pointers("exp_avg_sq_scales", exp_avg_sq_scales, count, torch.float32, dev, blocks)]
    else:
        columns += [repeat(0, count), repeat(0, count)]
    table = array.array("Q", chain.from_iterable(zip(*columns, numels)))  # ks_adamw_tensor: eight 64-bit words
    opt = _lib.KsAdamwOptions(0.0, betas[0], betas[1], eps, weight_decay, 1)
    if isinstance(lr, torch.Tensor):
        opt.lr_ptr = _scalar("lr", lr, torch.float32, dev)
    else:
        opt.lr = lr
    if isinstance(step, torch.Tensor):
        opt.step_ptr = _scalar("step", step, torch.int64, dev)
    else:
        opt.step = step
    if grad_scale is not None:
        opt.grad_scale = _scalar("grad_scale", grad_scale, torch.float32, dev)
    with torch.cuda.device(dev):
        st = _lib.load().ks_adamw_step(table.buffer_info()[0], count, KS_F32 if dt is torch.float32 else KS_BF16, bits,
                                       ctypes.byref(opt), _stream_ptr(stream, dev))
    _lib.check(st)


class AdamW(torch.optim.Optimizer):
    """AdamW with decoupled weight decay on ``adamw_step``: the tensors of a
    group that share dtype, device and step number take one launch.

    state_bits: 32, or 8 for e4m3 states with a scale for each 256 elements.
    masters: keep an fp32 master of each bf16 parameter in the state.
    Parameters must be contiguous CUDA tensors, fp32 or bf16; one without a
    gradient is left out of the step.  ``step`` counts on the host: to capture
    steps into a CUDA graph, call ``adamw_step`` with a step tensor."""

    def __init__(self, params, lr: float = 1e-3, betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 1e-2, *, state_bits: int = 32, masters: bool = False):
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if not lr >= 0 or not eps >= 0 or not weight_decay >= 0 or not all(0 <= b < 1 for b in betas):
            raise ValueError("lr, eps and weight_decay must not be negative, betas must be in [0, 1)")
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, state_bits=state_bits,
                                      masters=masters))

    def _init_state(self, p: torch.Tensor, group) -> dict:
        st = {"step": 0}
        flat = {"dtype": torch.float32, "device": p.device}
        if group["state_bits"] == 8:
            flat["dtype"] = torch.float8_e4m3fn
            blocks = (p.numel() + ADAMW_BLOCK - 1) // ADAMW_BLOCK
            for name in ("exp_avg_scale", "exp_avg_sq_scale"):
                st[name] = torch.zeros(blocks, dtype=torch.float32, device=p.device)
        for name in ("exp_avg", "exp_avg_sq"):
            st[name] = torch.zeros(p.shape, **flat)
        if group["masters"] and p.dtype == torch.bfloat16:
            st["master"] = p.detach().float().contiguous()
        return st

    @torch.no_grad()
    def step(self, closure=None, *, grad_scale: Optional[torch.Tensor] = None):
        """One step; ``grad_scale``, a one-element float32 CUDA tensor, multiplies the gradients."""
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for group in self.param_groups:
            runs = {}
            for p in group["params"]:
                if p.grad is None:
                    continue
                if p.grad.is_sparse:
                    raise ValueError("sparse gradients are not supported")
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("this optimizer counts its steps on the host: capture adamw_step with a step "
                                       "tensor instead")
                st = self.state[p]
                if not st:
                    st.update(self._init_state(p, group))
                runs.setdefault((p.dtype, p.device, st["step"], "master" in st), []).append(p)
            for (_, _, done, master), ps in runs.items():
                states = [self.state[p] for p in ps]
                more = {"masters": [s["master"] for s in states]} if master else {}
                if group["state_bits"] == 8:
                    more["exp_avg_scales"] = [s["exp_avg_scale"] for s in states]
                    more["exp_avg_sq_scales"] = [s["exp_avg_sq_scale"] for s in states]
                adamw_step(ps, [p.grad.contiguous() for p in ps], [s["exp_avg"] for s in states],
                           [s["exp_avg_sq"] for s in states], step=done + 1, lr=group["lr"], betas=group["betas"],
                           eps=group["eps"], weight_decay=group["weight_decay"], grad_scale=grad_scale, **more)
                for p, s in zip(ps, states):
                    s["step"] = done + 1
                    torch.autograd.graph.increment_version(p)  # changed in place behind autograd's back
        return loss

    def load_state_dict(self, state_dict) -> None:
        """As torch's, but every state tensor keeps the type it was saved in
        (torch casts them to their parameter's)."""
        super().load_state_dict(state_dict)
        saved = state_dict["state"]
        indexes = chain.from_iterable(g["params"] for g in state_dict["param_groups"])
        params = chain.from_iterable(g["params"] for g in self.param_groups)
        for index, p in zip(indexes, params):
            for name, t in saved.get(index, {}).items():
                if isinstance(t, torch.Tensor):
                    self.state[p][name] = t.detach().to(p.device, copy=True)

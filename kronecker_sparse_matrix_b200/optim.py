"""AdamW over many tensors in one launch: ``adamw_step`` (ks_adamw_step) and the
optimizer class ``AdamW`` built on it, with states in 32 bits or in 8 bits."""
from __future__ import annotations

from itertools import chain
from typing import Optional, Sequence, Tuple, Union

import torch

from . import KS_BF16, KS_F32, _lib

ADAMW_BLOCK = 256  # elements that share a scale in an 8-bit state


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
    runs: a captured step follows them.  Autograd counts parameters and masters as
    changed in place.  Asynchronous on ``stream``."""
    if len(params) == 0:
        return
    from ._ks_marshal import adamw_step as run  # built with the library
    args = (_lib.address("ks_adamw_step"), params, grads, exp_avgs, exp_avg_sqs, masters, exp_avg_scales,
            exp_avg_sq_scales, lr, step, grad_scale, betas[0], betas[1], eps, weight_decay, (KS_F32, KS_BF16),
            None if stream is None else stream.cuda_stream)
    dev = params[0].get_device() if isinstance(params[0], torch.Tensor) else -1
    if dev < 0 or dev == torch.cuda.current_device():
        status = run(*args)
    else:
        with torch.cuda.device(dev):
            status = run(*args)
    if status:
        _lib.check(status)
    # changed in place behind autograd's back (the states are nobody's but the optimizer's)
    torch.autograd.graph.increment_version(params if masters is None else [*params, *masters])


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
                for s in states:
                    s["step"] = done + 1
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

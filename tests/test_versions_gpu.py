"""What a call changes in place counts as changed for autograd."""
import pytest
import torch

import kronecker_sparse_matrix_b200 as ks
from tests.test_adapter_gpu import DEV, make

pytestmark = pytest.mark.gpu
HYPER = dict(step=1, lr=1e-2)


def test_adamw_step_between_forward_and_backward_is_noticed():
    w = torch.randn(300, device=DEV, requires_grad=True)
    loss = (w * w).sum()
    ks.adamw_step([w.detach()], [torch.ones_like(w)], [torch.zeros(300, device=DEV)], [torch.zeros(300, device=DEV)], **HYPER)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_versions_of_parameters_and_masters():
    ps = [torch.randn(n, device=DEV, dtype=torch.bfloat16) for n in (5, 300)]
    masters = [p.float() for p in ps]
    states = [[torch.zeros(p.numel(), device=DEV) for p in ps] for _ in range(2)]
    grads = [torch.ones_like(p) for p in ps]
    before = [t._version for t in ps + masters + grads]
    ks.adamw_step(ps, grads, *states, masters=masters, **HYPER)
    after = [t._version for t in ps + masters + grads]
    assert [u > v for u, v in zip(after, before)] == [True] * 4 + [False] * 2
    kept = [t._version for t in ps]
    with pytest.raises(ValueError):
        ks.adamw_step(ps, grads[:1], *states, **HYPER)
    assert [t._version for t in ps] == kept
    with torch.inference_mode():
        p = torch.randn(300, device=DEV)
    ks.adamw_step([p], [torch.ones(300, device=DEV)], [torch.zeros(300, device=DEV)], [torch.zeros(300, device=DEV)], **HYPER)


def test_an_output_given_to_adapter_matmul():
    p = (1, 64, 48, 8)
    q = make(p, 20, 2, 8, torch.float32, "rows", 2)
    out = torch.zeros(20, 512, device=DEV)
    w = torch.ones_like(out, requires_grad=True)
    loss = (out * w).sum()
    ks.adapter_matmul(q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"], out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()

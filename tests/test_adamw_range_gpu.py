"""8-bit AdamW states at the ends of fp32's range: gradients that are infinite, whose square
is, or whose running mean lies above 2^126.

A state that cannot be held makes its whole block NaN, seen at once; a state that can is held to
half a step of e4m3, 2^-4 relative.
"""
import pytest
import torch

import kronecker_sparse_matrix_b200 as ks
from tests.test_adamw_gpu import BLOCK, DEV, F64, clone, make, reference, spread, step

pytestmark = pytest.mark.gpu


def held(q, name):
    return q[name][0].to(F64) * spread(q[name + "s"][0], q[name][0].numel())


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_an_infinite_gradient_makes_its_block_nan(dtype, shift):
    q = make([1000], dtype, 8, shift=shift)
    q["g"][0][600] = float("inf")
    q["g"][0][520], q["m"][0][520], q["v"][0][520] = 0, 0, 0  # zero states too
    old = clone(q)
    step(q, 8)
    block = torch.zeros(1000, dtype=torch.bool, device=DEV)
    block[512:768] = True
    for name in ("m", "v"):
        assert torch.isnan(held(q, name)[block]).all() and torch.isfinite(held(q, name)[~block]).all()
    ok = torch.arange(1000, device=DEV) != 600  # the step itself still knows the other elements' states
    assert torch.isfinite(q["p"][0][ok].float()).all() and torch.isnan(q["p"][0][600].float())
    q["g"][0].copy_(old["g"][0]), q["g"][0][600].zero_()
    step(q, 8, step=8)  # nothing of the block is stepped on quietly
    assert torch.isnan(q["p"][0][block].float()).all() and torch.isfinite(q["p"][0][~block].float()).all()


@pytest.mark.parametrize("value", [3e19, 2e20, -1e30])
def test_a_gradient_whose_square_is_infinite_makes_the_second_state_nan(value):
    q = make([1000], torch.float32, 8)
    q["g"][0][300] = value
    q["g"][0][301], q["v"][0][301] = 0, 0
    old = clone(q)
    step(q, 8)
    block = torch.zeros(1000, dtype=torch.bool, device=DEV)
    block[256:512] = True
    assert torch.isnan(held(q, "v")[block]).all() and torch.isfinite(held(q, "v")[~block]).all()
    p, m, _, tm, tp = reference(old, 0, 8, 7)
    unit = spread(q["ms"][0], 1000)
    assert ((held(q, "m") - m).abs() <= torch.maximum(2.0 ** -4 * m.abs(), 2.0 ** -10 * unit) * (1 + 1e-5) + tm).all()
    other = torch.arange(1000, device=DEV) != 300
    assert torch.isfinite(q["p"][0]).all()  # (an infinite root: no change but the decay)
    assert ((q["p"][0].to(F64) - p).abs() <= tp)[other].all()


@pytest.mark.parametrize("top", [2.0 ** 125, 2.0 ** 126, 1.5 * 2.0 ** 126, 2.0 ** 127, 3.4e38])
def test_a_first_state_near_the_largest_number_is_held(top):
    n = 3 * BLOCK
    p, g = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    g[BLOCK:2 * BLOCK] = torch.linspace(-1, 1, BLOCK, device=DEV) * top
    g[2 * BLOCK:] = 1.0
    m, v = (torch.zeros(n, device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
    ms, vs = torch.zeros(3, device=DEV), torch.zeros(3, device=DEV)
    ks.adamw_step([p], [g], [m], [v], step=1, lr=1e-3, betas=(0.0, 0.99), weight_decay=0.0, exp_avg_scales=[ms],
                  exp_avg_sq_scales=[vs])
    unit = ms.to(F64).repeat_interleave(BLOCK)
    off = (m.to(F64) * unit - g.to(F64)).abs()
    assert (off <= torch.maximum(2.0 ** -4 * g.to(F64).abs(), 2.0 ** -10 * unit) * (1 + 1e-5)).all()
    root = v.to(F64) * vs.to(F64).repeat_interleave(BLOCK)
    assert torch.isnan(root[BLOCK:2 * BLOCK]).all() and torch.isfinite(root[2 * BLOCK:]).all()

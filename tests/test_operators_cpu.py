"""Argument checks of the adapter and AdamW entry points without a GPU: every
call here is refused on the host, before any CUDA call."""
import ctypes

import pytest

from kronecker_sparse_matrix_b200 import _lib, build as ksbuild

P = 1 << 24  # fake 256-byte-aligned addresses, far apart; never dereferenced
FAR = 1 << 32


@pytest.fixture(scope="module")
def lib():
    ksbuild.build()
    return _lib.load()


def matmul(lib, X=P, V=P + FAR, pat=(1, 16, 8, 4), batch=4, Y=P + 2 * FAR, dtype=0, bias=None, act=0, A=P + 3 * FAR,
           B=P + 4 * FAR, scales=None, ids=None, s=2, r=8):
    return lib.ks_adapter_matmul(X, V, *pat, batch, Y, dtype, bias, act, A, B, scales, ids, s, r, None)


def backward(lib, dY=P, X=P + FAR, V=P + 2 * FAR, pat=(1, 16, 8, 4), batch=4, dtype=0, A=P + 3 * FAR, B=P + 4 * FAR,
             scales=None, ids=None, s=2, r=8, dX=P + 5 * FAR, dA=P + 6 * FAR, dB=P + 7 * FAR):
    return lib.ks_adapter_backward(dY, X, V, *pat, batch, dtype, A, B, scales, ids, s, r, dX, dA, dB, None)


@pytest.mark.parametrize("kw", [dict(s=0), dict(s=4097), dict(s=65536), dict(r=0), dict(r=1025), dict(A=None), dict(B=None),
                                dict(X=None), dict(Y=None), dict(V=None), dict(dtype=5), dict(act=4), dict(batch=-1),
                                dict(batch=(1 << 30) + 1), dict(pat=(1, 0, 8, 4)), dict(Y=P + 3 * FAR),
                                dict(Y=P + 4 * FAR), dict(Y=P), dict(Y=P + FAR), dict(ids=P + 2 * FAR + 4),
                                dict(scales=P + 2 * FAR), dict(bias=P + 2 * FAR)])
def test_adapter_matmul_invalid(lib, kw):
    assert matmul(lib, **kw) == 1


@pytest.mark.parametrize("kw", [dict(A=P + 3 * FAR + 2), dict(B=P + 4 * FAR + 1), dict(ids=P + 5 * FAR + 2),
                                dict(scales=P + 5 * FAR + 2), dict(X=P + 2), dict(bias=P + 5 * FAR + 2)])
def test_adapter_matmul_misaligned(lib, kw):
    assert matmul(lib, **kw) == 2


def test_adapter_matmul_empty_batch_is_a_noop(lib):
    assert matmul(lib, X=None, V=None, Y=None, A=None, B=None, batch=0) == 0


@pytest.mark.parametrize("kw", [dict(s=0), dict(r=0), dict(A=None), dict(dY=None), dict(X=None), dict(V=None),
                                dict(dtype=9), dict(dX=P), dict(dX=P + FAR), dict(dX=P + 2 * FAR),
                                dict(dA=P + 3 * FAR), dict(dB=P + 4 * FAR), dict(dA=P + 5 * FAR), dict(dB=P + 6 * FAR),
                                dict(dB=P), dict(ids=P + 7 * FAR)])
def test_adapter_backward_invalid(lib, kw):
    assert backward(lib, **kw) == 1


def test_adapter_backward_misaligned(lib):
    assert backward(lib, dA=P + 6 * FAR + 2) == 2
    assert backward(lib, dY=P + 1) == 2


def adamw(lib, tensors, dtype=0, bits=32, n=None, **kw):
    arr = (_lib.KsAdamwTensor * max(1, len(tensors)))(*tensors)
    o = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1)
    o.update(kw)
    return lib.ks_adamw_step(ctypes.cast(arr, ctypes.c_void_p), len(tensors) if n is None else n, dtype, bits,
                             ctypes.byref(_lib.KsAdamwOptions(**o)), None)


def tensor(k=0, n=1000, **kw):
    at = P + 16 * k * FAR
    f = dict(param=at, grad=at + FAR, exp_avg=at + 2 * FAR, exp_avg_sq=at + 3 * FAR, n=n)
    f.update(kw)
    return _lib.KsAdamwTensor(**f)


@pytest.mark.parametrize("kw", [dict(lr=-1.0), dict(lr=float("nan")), dict(lr=float("inf")), dict(beta1=1.0),
                                dict(beta2=-0.1), dict(beta1=float("nan")), dict(eps=-1e-8), dict(eps=float("nan")),
                                dict(weight_decay=-1.0), dict(step=0), dict(dtype=1), dict(bits=16), dict(n=-1)])
def test_adamw_invalid_numbers(lib, kw):
    assert adamw(lib, [tensor()], **kw) == 1


@pytest.mark.parametrize("kw", [dict(param=None), dict(grad=None), dict(exp_avg=None), dict(exp_avg_sq=None),
                                dict(n=-1), dict(grad=P), dict(exp_avg=P + 4 * 999), dict(exp_avg_sq=P + 2 * FAR),
                                dict(master=P + 5 * FAR)])
def test_adamw_invalid_tensor(lib, kw):
    assert adamw(lib, [tensor(**kw)]) == 1


def test_adamw_other_refusals(lib):
    assert adamw(lib, [tensor(0), tensor(0)]) == 1  # the same tensor twice
    assert b"overlaps" in lib.ks_last_error()
    assert adamw(lib, [tensor(0), tensor(1, exp_avg=P + 4)]) == 1
    assert adamw(lib, [tensor(0, master=P + 5 * FAR), tensor(1)], dtype=2) == 1  # masters for some only
    assert adamw(lib, [tensor()], bits=8) == 1  # no scales
    assert adamw(lib, [tensor(param=P + 2)]) == 2
    assert adamw(lib, [tensor()], step_ptr=P + 8 * FAR + 4) == 2
    assert adamw(lib, [tensor()], lr_ptr=P) == 1  # the rate inside a parameter
    assert lib.ks_adamw_step(None, 1, 0, 32, ctypes.byref(_lib.KsAdamwOptions()), None) == 1
    assert lib.ks_adamw_step(None, 0, 0, 32, None, None) == 1


def test_adamw_nothing_to_do(lib):
    assert adamw(lib, []) == 0
    assert adamw(lib, [_lib.KsAdamwTensor(n=0)]) == 0


def test_the_largest_batch(lib):
    """2^30 rows pass the check of the batch (and meet the next one), one more does not."""
    for call in (matmul, backward):
        assert call(lib, batch=1 << 30, A=None) == 1
        assert b"A and B" in lib.ks_last_error()
        assert call(lib, batch=(1 << 30) + 1, A=None) == 1
        assert b"2^30 rows" in lib.ks_last_error()

"""The erf form of GELU that the adapter kernels evaluate in packed fp32
(gelu_erf_f2 in ks_epilogue.cuh), modelled in numpy with the constants read from
the source, against z Phi(z) in 64 bits.  Bound: 0.75e-7 |z| of the formula (half
of Abramowitz and Stegun's 1.5e-7 for erf) and the fp32 operations: h <= 1/2 is off by
about ten units in the last place relative, the subtraction by one: 1.2e-6 |z| in all."""
import math
import os
import re

import numpy as np
import pytest

SRC = os.path.join(os.path.dirname(__file__), "..", "kronecker_sparse_matrix_b200", "csrc", "ks_epilogue.cuh")


def model(z):
    body = re.search(r"float2 gelu_erf_f2\(float2 z\) \{(.*?)\n\}", open(SRC).read(), flags=re.S).group(1)
    expr = [e.replace("f", "") for e in re.findall(r"both\(([-0-9.f* ]+)\)", body)]
    k = [np.float32(eval(e)) for e in expr]
    slope, one, c5, c4, c3, c2, c1, ex = k
    assert one == 1
    f = np.float32
    a = np.fmin(np.abs(z), f(32))  # as fminf: the number where one is NaN
    t = f(1) / (a * slope + f(1))
    q = t * c5 + c4
    for c in (c3, c2, c1):
        q = t * q + c
    h = (t * q) * np.exp2((a * a) * ex)
    return np.where(z < 0, f(0), z) - a * h


@pytest.mark.parametrize("lo,hi", [(-1e-3, 1e-3), (-1, 1), (-6, 6), (-40, 40), (-1e6, 1e6)])
def test_packed_erf_gelu(lo, hi):
    z = np.linspace(lo, hi, 20001, dtype=np.float32)
    ref = np.array([0.5 * v * math.erfc(-v / math.sqrt(2)) for v in z.astype(np.float64)])
    off = np.abs(model(z).astype(np.float64) - ref)
    assert (off <= 1.2e-6 * np.abs(z.astype(np.float64)) + 1e-38).all()


def test_ends():
    z = np.array([np.inf, -np.inf, np.nan, 0.0], dtype=np.float32)
    with np.errstate(invalid="ignore"):
        y = model(z)
    assert y[0] == np.inf and y[1] == 0 and np.isnan(y[2]) and y[3] == 0

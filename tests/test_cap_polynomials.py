"""The polynomials of the tanh cap, with the coefficients that the sources hold,
against tanh in 64 bits."""
import os
import re

import numpy as np
import pytest

from paged_kv_cache_234_gb300.build import CSRC


def coefficients(file, name, count):
    with open(os.path.join(CSRC, file)) as f:
        m = re.search(r"constexpr float %s\[%d\] = \{([^}]*)\}" % (name, count), f.read())
    c = [np.float32(x.strip().rstrip("f")) for x in m.group(1).split(",")]
    assert len(c) == count
    return c


def exact(c, u):
    p = np.zeros_like(u)
    for k in reversed(c):
        p = p * u * u + float(k)
    return u * p


def in_fp32(c, u):
    """u P(u^2) with fused steps: fp64 holds a product of fp32 values exactly."""
    w = u * u
    p = np.full_like(u, c[-1])
    for k in reversed(c[:-1]):
        p = (p.astype(np.float64) * w + float(k)).astype(np.float32)
    return u * p


POLYNOMIALS = {
    "degree 6": ("pkv_score.cuh", "c", 7, 1.0, 2.0 ** -23.1, 2.0 ** -22.2),
    "degree 3": ("pkv_prefill.cu", "near", 4, 0.35, 6.1e-8, 2.0 ** -22.6),
}


@pytest.mark.parametrize("which", POLYNOMIALS)
def test_relative_errors(which):
    file, name, count, end, bound, bound32 = POLYNOMIALS[which]
    c = coefficients(file, name, count)
    u = np.linspace(0.0, end, 1000001)[1:]
    assert np.max(np.abs(exact(c, u) / np.tanh(u) - 1)) <= bound
    u = np.concatenate([u, end * 10.0 ** -np.linspace(0.0, 6.0, 300000)]).astype(np.float32)
    u = u[u <= np.float32(end)]
    assert np.max(np.abs(in_fp32(c, u) / np.tanh(u.astype(np.float64)) - 1)) <= bound32

"""The polynomial of the tanh cap that tree attention takes inside half the cap,
against tanh in 64 bits."""
import numpy as np

from test_cap_polynomials import coefficients, exact, in_fp32


def test_relative_errors():
    c = coefficients("pkv_score.cuh", "close", 5)
    u = np.linspace(0.0, 0.5, 1000001)[1:]
    assert np.max(np.abs(exact(c, u) / np.tanh(u) - 1)) <= 2.0 ** -24.9
    u = np.concatenate([u, 0.5 * 10.0 ** -np.linspace(0.0, 6.0, 300000)]).astype(np.float32)
    # the product u P rounds once and P's last step once, 2^-24 each; what was rounded
    # before comes with the factor c[1] w <= 1 / 12, three times, w itself and two steps;
    # and the polynomial's own 2^-24.9
    tol = 2.0 ** -24 * (2 + 3 / 12) + 2.0 ** -24.9
    assert np.max(np.abs(in_fp32(c, u) / np.tanh(u.astype(np.float64)) - 1)) <= tol

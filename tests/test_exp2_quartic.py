"""The FMA-pipe 2^x of the sink-window kernels (one exponential pair in four): a quartic
in the fractional part, where the dual-window kernel has a cubic.

The coefficients come from the fit that tests/test_exp2_poly.py describes (Lawson's
algorithm for the relative error on Chebyshev nodes), one degree higher.  Pinned here:
the refit gives the committed coefficients, and an fp32 restatement of the kernel's
steps stays within 3e-6 of 2^x, so that a log-sum-exp keeps 32-bit quality."""
import os
import re

import numpy as np

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dual_window_attention_b200",
                   "csrc", "sink_attention_fwd.cuh")
BOUND = 3.0e-6  # 2.8e-6 of the quartic, 2^-23 of the last step of Horner's rule


def committed_coefficients():
    number = r"([0-9.eE+-]+)f"
    with open(SRC) as f:
        m = re.search(rf"C1 = {number}, C2 = {number},\s*C3 = {number}, C4 = {number}", f.read())
    assert m, "coefficients not found"
    return np.array([float(g) for g in m.groups()])


def lawson_fit(n_nodes=2001, iters=4000):
    """Minimax relative-error quartic with p(0) = 1 for 2^f on [-0.5, 0.5]."""
    f = 0.5 * np.cos(np.pi * (np.arange(n_nodes) + 0.5) / n_nodes)
    t = 2.0 ** f
    A = np.stack([f ** i / t for i in range(1, 5)], 1)
    b = 1.0 - 1.0 / t
    w = np.full(n_nodes, 1.0 / n_nodes)
    for _ in range(iters):
        sw = np.sqrt(w)
        c = np.linalg.lstsq(A * sw[:, None], b * sw, rcond=None)[0]
        w = w * np.abs(A @ c - b)
        w /= w.sum()
    return c


def test_refit_reproduces_committed_coefficients():
    np.testing.assert_allclose(committed_coefficients(), lawson_fit(), rtol=0, atol=1e-6)


def test_committed_quartic_relative_error():
    f = np.linspace(-0.5, 0.5, 400001)
    p = 1.0 + sum(c * f ** (i + 1) for i, c in enumerate(committed_coefficients()))
    err = np.abs(p / 2.0 ** f - 1.0)
    assert 2.5e-6 < err.max() <= 2.85e-6  # the minimax level


def restated(x):
    """Clamp, shifter rounding, Horner, exponent add, in fp32."""
    c = committed_coefficients().astype(np.float32)
    shift = np.float32(12582912.0)
    xc = np.maximum(x, np.float32(-127.0))
    t = (xc + shift).astype(np.float32)
    fr = (xc - (t - shift)).astype(np.float32)
    p = np.full_like(xc, c[3])
    for y in (c[2], c[1], c[0], np.float32(1.0)):  # each step rounded once, as a fused one is
        p = (p.astype(np.float64) * fr + y).astype(np.float32)
    return (p.view(np.int32) + (t.view(np.int32) << 23)).view(np.float32)


def test_restated_range_reduction():
    g = np.random.default_rng(0)
    x = np.concatenate([np.linspace(-126.0, 8.0, 200001), g.uniform(-126.0, 8.0, 100000),
                        np.arange(-126, 9) + 0.5, np.arange(-126, 9)]).astype(np.float32)
    # below -125, results of less than 2^-126 have lost bits
    err = np.abs(restated(x) / 2.0 ** x.astype(np.float64) - 1.0)[x >= -125]
    assert err.max() <= BOUND, err.max()


def test_restated_ends():
    """Masked scores weigh exactly 0, and what is near them nothing that is not tiny."""
    np.testing.assert_array_equal(restated(np.array([-np.inf, -1e30, -127.5, -127.0], np.float32)), 0.0)
    y = restated(np.linspace(-127.0, -125.5, 300001).astype(np.float32))
    assert (y >= 0).all() and y.max() <= 1.5 * 2.0 ** -126
    with open(SRC) as f:
        assert f.read().count("-127.0f") == 4  # the clamp of this restatement

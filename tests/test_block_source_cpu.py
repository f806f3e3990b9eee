"""What the layer operators' sources state, checked without a GPU."""
import os
import re

import numpy as np
from scipy.special import erfc, erfcx

from latent_projection_top_amd import block

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_cleared_part_of_a_workspace_matches_the_header():
    src = open(os.path.join(ROOT, "include", "block.h")).read()
    assert int(re.search(r"#define BLOCK_WORKSPACE_ZEROED (\d+)", src).group(1)) == block.WORKSPACE_ZEROED


def gelu_fit():
    """The device code's coefficients of Q, highest power first."""
    src = open(os.path.join(ROOT, "latent_projection_top_amd", "csrc", "block_device.h")).read()
    first = re.findall(r"float q = (-?[0-9.]+)f;", src)
    rest = re.findall(r"q = fmaf\(q, t, (-?[0-9.]+)f\);", src)
    assert len(first) == 1 and len(rest) == 7
    return [np.float32(c) for c in first + rest]


def test_gelu_fit_error():
    """Phi(-x) = exp(-x^2 / 2) t Q(t), t = 1 / (1 + 0.3 x): the fit's relative
    error with the coefficients as stored, in FP64, is the stated 2.3e-7 (the
    rounding of the eight coefficients, up to 2^-25 of each, is part of it)."""
    x = np.linspace(0.0, 14.5, 1000001)
    t = 1.0 / (1.0 + 0.3 * x)
    q = np.polyval([float(c) for c in gelu_fit()], t)
    assert np.abs(t * q / (0.5 * erfcx(x / np.sqrt(2.0))) - 1.0).max() <= 2.3e-7


def test_gelu_tail_in_fp32():
    """The same in FP32, each operation rounded once (fmaf once for both): the
    stated bounds. Beyond the fit's error the exponential's argument counts,
    up to x^2 / 2 log2(e) in base 2 with two roundings of 2^-24 (of the square
    and of the product), and 2^-24 for each of the ten other operations."""
    f = np.float32
    x = np.linspace(0.0, 13.0, 400001).astype(f)
    t = (1.0 / (np.float64(f(0.3)) * x + 1.0).astype(f)).astype(f)
    q = np.full_like(x, gelu_fit()[0])
    for c in gelu_fit()[1:]:
        q = (q.astype(np.float64) * t + np.float64(c)).astype(f)
    e = np.exp2((x * x * f(-0.72134752044448170)).astype(np.float64)).astype(f)
    tail = (e * (t * q)).astype(np.float64)
    x = x.astype(np.float64)
    want = 0.5 * erfc(x / np.sqrt(2.0))
    err = np.abs(tail / want - 1.0)
    assert (err <= 2.3e-7 + 2.0 ** -24 * (10.0 + x * x)).all()
    for most, bound in ((2.0, 6e-7), (6.0, 2.2e-6), (13.0, 8e-6)):
        assert err[x <= most].max() <= bound
    assert np.abs(tail - want).max() <= 2.15e-7

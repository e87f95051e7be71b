"""rms_norm_int8 with eps 0, where a row may have no finite reciprocal of its
root mean square."""
import numpy as np
import pytest
import torch

import bit_gemv_amd as bg
from gpu_helpers import assert_same_bits, dev, host, say
from oracle import serving


def _rows(k):
    """zeros, subnormal rows, the smallest normal ones, one element alone"""
    rng = np.random.default_rng(k)
    x = np.zeros((8, k), np.float32)
    for i, m in ((1, 1e-45), (2, 1e-41), (3, 1e-39), (4, 2e-38), (5, 1.0)):
        x[i] = rng.standard_normal(k) * m
    x[6, 3], x[7, 5] = 1e-43, -3e-39
    w = (1 + 0.2 * rng.standard_normal(k)).astype(np.float32)
    w[2] = -w[2]
    return x, w


@pytest.mark.parametrize("k", [256, 33024])
def test_oracle_is_finite(k):
    x, w = _rows(k)
    q, sx, _, y = serving.rms_norm_int8(x, w, 0.0)
    assert np.isfinite(y).all() and np.isfinite(sx).all()
    assert not q[0].any() and sx[0] == np.float32(1e-8) / np.float32(127)
    assert np.abs(q[1:]).max(-1).min() == 127                       # every other row uses its whole range


@pytest.mark.gpu
@pytest.mark.parametrize("k", [256, 8192, 33024])
def test_against_the_oracle(k):
    x, w = _rows(k)
    q, sx, _, _ = serving.rms_norm_int8(x, w, 0.0)
    say(f"rms_norm_int8 eps 0, k={k}")
    for res in (None, torch.zeros(x.shape, device="cuda")):
        gq, gs, _ = bg.rms_norm_int8(dev(x), dev(w), 0.0, res)
        assert_same_bits(host(gs), sx, "sx")
        assert_same_bits(host(gq), q, "qx")

"""rms_norm_int8 against the oracle: codes, scales and the new residual bit for
bit (the definition's roundings are all stated, and the sum of squares is in
64 bits on both sides)."""
import numpy as np
import pytest
import torch

import bit_gemv_amd as bg
from gpu_helpers import assert_same_bits, dev, host, say
from oracle import serving
from serving_helpers import bf16, dev_bf16f
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def _tensor(a, kind):
    return dev_bf16f(a) if kind == "bf16" else dev(a)


def _case(t, k, x, res, w, seed, eps=1e-5, x_scale=1.0, in_place=False):
    rng = np.random.default_rng(seed)
    r = (lambda a, kind: bf16(a) if kind == "bf16" else a.astype(np.float32))
    out = np.where(rng.random(k) < 0.01, 30.0, 1.0)
    xs = r(rng.standard_normal((t, k)) * out * x_scale, x)
    rs = None if res is None else r(rng.standard_normal((t, k)) * out * 2 * x_scale, res)
    ws = r(1 + 0.2 * rng.standard_normal(k), w)
    say(f"rms_norm_int8 t={t} k={k} x={x} res={res} w={w} in_place={in_place}")
    q, sx, h, _ = serving.rms_norm_int8(xs, ws, eps, rs)
    rd = None if rs is None else _tensor(rs, res)
    gq, gs, gr = bg.rms_norm_int8(_tensor(xs, x), _tensor(ws, w), eps, rd, rd if in_place else None)
    assert_same_bits(host(gs), sx, "sx")
    assert_same_bits(host(gq), q, "qx")
    if rs is None:
        assert gr is None
    elif res == "bf16":
        assert_same_bits(host(gr.view(torch.int16)), f32_to_bf16_bits(h).view(np.int16), "residual")
    else:
        assert_same_bits(host(gr), h, "residual")


@pytest.mark.parametrize("x", ["bf16", "fp32"])
@pytest.mark.parametrize("res", [None, "bf16", "fp32"])
@pytest.mark.parametrize("w", ["bf16", "fp32"])
def test_types(x, res, w):
    _case(5, 640, x, res, w, 1)


# one row to many, rows of less than a wave, one chunk exactly, past one chunk
# of each block size, and wide rows read in several passes
@pytest.mark.parametrize("t,k", [(1, 128), (3, 256), (1, 4096), (2, 8192), (7, 8320), (1, 11008), (2, 16384), (3, 28672),
                                 (1, 32768), (2, 32896), (1, 65536), (517, 4096), (4096, 128)])
@pytest.mark.parametrize("res", [None, "bf16"])
def test_sizes(t, k, res):
    _case(t, k, "bf16", res, "bf16", t + k)


@pytest.mark.parametrize("k", [4096, 32896])
@pytest.mark.parametrize("res", ["bf16", "fp32"])
def test_residual_in_place(k, res):
    _case(9, k, "fp32", res, "fp32", k, in_place=True)


@pytest.mark.parametrize("scale", [1e-18, 1e-6, 1e6, 1e15])
def test_magnitudes(scale):
    """Rows far below eps and far above it."""
    _case(4, 512, "fp32", "fp32", "fp32", 3, x_scale=scale)


def test_rows_past_one_launch():
    """More rows than a launch takes: as the same rows by themselves."""
    t, k = (1 << 21) + 5, 128
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((t, k), generator=g, device="cuda").bfloat16()
    w = torch.rand(k, generator=g, device="cuda")
    res = x.flip(0).contiguous()
    say(f"rms_norm_int8 t={t} k={k}")
    out = bg.rms_norm_int8(x, w, 1e-5, res)
    for at in (0, (1 << 21) - 3, t - 8):
        part = bg.rms_norm_int8(x[at : at + 8].clone(), w, 1e-5, res[at : at + 8].clone())
        assert all(torch.equal(a[at : at + 8], b) for a, b in zip(out, part))


def test_zero_rows_and_zero_eps():
    x = torch.zeros(3, 256, device="cuda")
    x[1] = 1
    say("rms_norm_int8 zero rows")
    q, s, _ = bg.rms_norm_int8(x, torch.ones(256, device="cuda"), 1e-5)
    assert int(q[0].abs().max()) == 0 and int(q[1].min()) == 127
    assert float(s[0]) == float(np.float32(1e-8) / np.float32(127))
    _case(2, 256, "fp32", None, "fp32", 4, eps=0.0)


def test_no_residual_out_pointer():
    """The C call without residual_out: same codes, residual untouched."""
    lib = bg.load_library()
    x, res, w = torch.randn(4, 256, device="cuda"), torch.randn(4, 256, device="cuda"), torch.ones(256, device="cuda")
    keep = res.clone()
    q, s = torch.empty(4, 256, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    say("rms_norm_int8 without residual_out")
    st = lib.rms_norm_int8(x.data_ptr(), 1, res.data_ptr(), 1, w.data_ptr(), 1, 4, 256, 1e-5, None, q.data_ptr(),
                           s.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    q2, s2, r2 = bg.rms_norm_int8(x, w, 1e-5, res)
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(res, keep) and torch.equal(r2, x + res)


def test_empty():
    q, s, r = bg.rms_norm_int8(torch.empty(0, 256, device="cuda"), torch.ones(256, device="cuda"))
    assert q.shape == (0, 256) and s.shape == (0,) and r is None

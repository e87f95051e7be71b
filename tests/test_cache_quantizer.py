"""The cache's codes, scales and zeros are the group quantizer's, bit for bit:
the oracle's against the C oracle's on the CPU, and kv_cache_write's against
quantize_groupwise's on the GPU."""
import numpy as np
import pytest
import torch

import bit_gemv_amd as bg
import oracle
from gpu_helpers import say
from oracle import serving
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

FORMATS = [(4, False), (4, True), (8, False), (8, True)]


def _rows(d, seed, n=1024):
    """bf16 bits: ordinary rows, constant ones, far from zero, tiny, huge."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, d)) * 10.0 ** rng.uniform(-3, 3, (n, 1))
    x[0], x[1], x[2] = 0, 2.5, -3e-10
    x[3:40] += 100
    x[40:60] = np.abs(x[40:60])
    x[60:80] *= 1e-12
    x[80:90] *= 1e20
    return f32_to_bf16_bits(x)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("bits,sym", FORMATS)
def test_oracles_agree(d, bits, sym):
    w = _rows(d, bits + d)
    q, s, z = serving.kv_quantize(bf16_bits_to_f32(w), bits, sym)
    c, s2, z2 = oracle.quantize(w, bits, sym, d)
    if bits == 4:
        c = np.stack((c & 15, c >> 4), -1).reshape(q.shape)
    elif sym:
        c = (c.view(np.int8).astype(np.int16) + 128).astype(np.uint8)
    assert np.array_equal(s.view(np.uint32), s2[:, 0].view(np.uint32))
    assert np.array_equal(q, c)
    if not sym:
        assert np.array_equal(z.view(np.uint32), z2[:, 0].view(np.uint32))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("bits,sym", FORMATS)
def test_write_gives_the_group_quantizers_codes(d, bits, sym):
    n, heads, page = 1024, 2, 16
    x = torch.from_numpy(_rows(d, bits + d + 1, n * heads).view(np.int16)).view(torch.bfloat16).cuda()
    say(f"kv_cache_write against quantize_groupwise D={d} bits={bits} sym={sym}")
    want = bg.quantize_groupwise(x, bits, sym, d)
    c = bg.KVCache.empty(n // page, page, heads, d, bits, sym)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.arange(n // page, dtype=torch.int32, device="cuda")[None]
    rows = x.view(n, heads, d)
    bg.kv_cache_write(rows, rows, c, table, i32(n), i32(0, n))
    codes = want.codes.view(torch.uint8).view(n, heads, -1)
    if sym and bits == 8:
        codes = codes ^ 128
    keys = c.k_codes.permute(0, 2, 1, 3).reshape(n, heads, -1)
    values = c.v_codes.permute(0, 2, 4, 1, 3).reshape(n, heads, -1)
    assert torch.equal(keys, codes) and torch.equal(values, codes)
    for got, ref in (("scales", want.scales),) + (() if sym else (("zeros", want.zeros),)):
        ref = ref.view(n, heads).view(torch.int32)
        for side in "kv":
            t = getattr(c, f"{side}_{got}").permute(0, 2, 1).reshape(n, heads)
            assert torch.equal(t.view(torch.int32), ref), (side, got)

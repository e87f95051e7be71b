"""kv_cache_write's codes, scales and zeros against the group quantizer's
formulas written in torch on the GPU, which divides a tensor by a number as a
product with the rounded reciprocal: bit for bit. Against quantize_groupwise,
which forms the quotient: one ulp of the scale, and the same codes and zeros
where the scale is the same."""
import numpy as np
import pytest
import torch

import bit_gemv_amd as bg
from gpu_helpers import say
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

FORMATS = [(4, False), (4, True), (8, False), (8, True)]


def _rows(d, seed, n):
    """bf16 rows: ordinary ones, constant ones, far from zero, tiny, huge."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, d)) * 10.0 ** rng.uniform(-3, 3, (n, 1))
    x[0], x[1], x[2] = 0, 2.5, -3e-10
    x[3:40] += 100
    x[40:60] = np.abs(x[40:60])
    x[60:80] *= 1e-12
    x[80:90] *= 1e20
    return torch.from_numpy(f32_to_bf16_bits(x).view(np.int16)).view(torch.bfloat16).cuda()


def _torch_quantizer(x, bits, sym):
    """(codes stored unsigned, scale, zero or None) of each row"""
    x = x.float()
    if sym:
        qmax = 2 ** (bits - 1) - 1
        s = x.abs().amax(-1, keepdim=True).clamp_min(1e-8) / qmax
        return (torch.round(x / s).clamp(-qmax, qmax) + 2 ** (bits - 1)).to(torch.uint8), s, None
    top = 2 ** bits - 1
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = (hi - lo).clamp_min(1e-8) / top
    z = torch.round(-lo / s) + 0.0
    return (torch.round(x / s) + z).clamp(0, top).to(torch.uint8), s, z


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("bits,sym", FORMATS)
def test_write_against_torch_and_the_group_quantizer(d, bits, sym):
    n, heads, page = 1024, 2, 16
    x = _rows(d, bits + d + 1, n * heads)
    say(f"kv_cache_write against the formulas in torch D={d} bits={bits} sym={sym}")
    q, s, z = _torch_quantizer(x, bits, sym)
    c = bg.KVCache.empty(n // page, page, heads, d, bits, sym)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.arange(n // page, dtype=torch.int32, device="cuda")[None]
    rows = x.view(n, heads, d)
    bg.kv_cache_write(rows, rows, c, table, i32(n), i32(0, n))
    packed = lambda t: t if bits == 8 else t[..., 0::2] | (t[..., 1::2] << 4)  # noqa: E731
    keys = c.k_codes.permute(0, 2, 1, 3).reshape(n * heads, -1)
    values = c.v_codes.permute(0, 2, 4, 1, 3).reshape(n * heads, -1)
    flat = lambda t: t.permute(0, 2, 1).reshape(n * heads, 1)  # noqa: E731
    bits_of = lambda t: t.contiguous().view(torch.int32)  # noqa: E731
    for side, codes in (("k", keys), ("v", values)):
        assert torch.equal(bits_of(flat(getattr(c, side + "_scales"))), bits_of(s)), side
        if not sym:
            assert torch.equal(bits_of(flat(getattr(c, side + "_zeros"))), bits_of(z)), side
        assert torch.equal(codes, packed(q)), side
    group = bg.quantize_groupwise(x, bits, sym, d)
    ulp = bits_of(s) - bits_of(group.scales)
    assert int(ulp.abs().max()) <= 1
    same = (ulp == 0).view(-1)
    assert bool(same.any()) and not bool(same.all())
    codes = group.codes.view(torch.uint8).view(n * heads, -1)
    assert torch.equal((codes ^ 128 if sym and bits == 8 else codes)[same], packed(q)[same])
    if not sym:
        assert torch.equal(bits_of(group.zeros)[same], bits_of(z)[same])

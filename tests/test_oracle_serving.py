"""Pins of the serving operators' oracle (oracle/serving.py). CPU only."""
import numpy as np
import pytest

import oracle
from oracle import serving
from workloads import bf16_bits_to_f32, f32_to_bf16_bits


def _bf16(rng, *shape, scale=1.0):
    return f32_to_bf16_bits(rng.standard_normal(shape) * scale)


def test_norm_of_a_unit_rms_row_is_the_weight():
    """h of +-1 has r = 1 / sqrt(1 + eps): with eps 0 y is w with h's signs."""
    rng = np.random.default_rng(1)
    h = np.where(rng.random((3, 256)) < 0.5, -1, 1).astype(np.float32)
    w = rng.random(256).astype(np.float32) + 0.5
    q, sx, hh, y = serving.rms_norm_int8(h - 2, w, 0.0, np.full((3, 256), 2, np.float32))
    assert np.array_equal(hh, h) and np.array_equal(y, h * w)
    assert np.allclose(sx, w.max() / 127) and np.array_equal(np.abs(q[:, w.argmax()]), [127, 127, 127])


def test_norm_codes_are_the_per_token_quantizers():
    rng = np.random.default_rng(2)
    x, w = bf16_bits_to_f32(_bf16(rng, 7, 384)), rng.random(384).astype(np.float32) + 0.5
    q, sx, _, y = serving.rms_norm_int8(x, w, 1e-5)
    q2, sx2 = oracle.quant_per_token_int8(y)
    assert np.array_equal(q, q2) and np.array_equal(sx.view(np.uint32), sx2.view(np.uint32))


@pytest.mark.parametrize("bits,sym", [(4, False), (4, True), (8, False), (8, True)])
def test_cache_quantizer_is_the_group_quantizer(bits, sym):
    """Rows of one 128-wide group each: quantize_groupwise's formulas."""
    rng = np.random.default_rng(bits + sym)
    w = _bf16(rng, 9, 128, scale=3.0)
    w[3] = f32_to_bf16_bits(np.full((1, 128), 2.5, np.float32))[0]       # a constant row
    w[4] = 0
    w[5] = f32_to_bf16_bits(np.abs(rng.standard_normal((1, 128))) + 4)[0]  # all positive
    q, s, z = serving.kv_quantize(bf16_bits_to_f32(w), bits, sym)
    c, s2, z2 = oracle.quantize(w, bits, sym, 128)
    if bits == 4:
        c = np.stack((c & 15, c >> 4), -1).reshape(9, 128)
    elif sym:
        c = (c.view(np.int8).astype(np.int16) + 128).astype(np.uint8)
    # the scale is the range times a rounded reciprocal: at most one ulp off
    # the quotient, and with the same scale the same codes and zeros
    ulp = s.view(np.int32).astype(np.int64) - s2[:, 0].view(np.int32)
    assert np.abs(ulp).max() <= 1
    same = ulp == 0
    assert same.any() and np.array_equal(q[same], c[same])
    if not sym:
        assert np.array_equal(z[same], z2[same, 0])
    # half a step of rounding each for the code and the zero point
    x = bf16_bits_to_f32(w)
    off = np.abs(serving.kv_dequantize(q, s, z, bits) - x)
    assert np.all(off <= s[:, None] * (0.5 if sym else 1.0) * (1 + 2.0 ** -16) + np.abs(x) * 2.0 ** -20)


@pytest.mark.parametrize("bits", [4, 8])
def test_cache_layout_byte_positions(bits):
    c = serving.Cache(2, 16, 3, 64, bits, True)
    codes = (np.arange(64) % (2 ** bits)).astype(np.uint8)
    for side in "kv":
        c.put(1, 6, 2, side, codes, 0.5, None)
        assert np.array_equal(c.codes(1, 2, side)[6], codes)
    row = 64 * bits // 8
    at = 37 if bits == 8 else 18
    want = 37 if bits == 8 else (36 % 16) | ((37 % 16) << 4)
    assert c.k_codes.reshape(-1)[((1 * 3 + 2) * 16 + 6) * row + at] == want
    assert c.v_codes.reshape(-1)[(((1 * 3 + 2) * 4 + 1) * row + at) * 4 + 2] == want


def _filled(rng, heads, d, bits, sym, lens, page=16):
    need = [(n + page - 1) // page for n in lens]
    cache = serving.Cache(sum(need) + 1, page, heads, d, bits, sym)
    table, at = [], 0
    for n, k in zip(lens, need):
        table.append(list(range(at, at + k)))
        for t in range(n):
            for side in "kv":
                cache.put_rows(table[-1][t // page], t % page, side, rng.standard_normal((heads, d)).astype(np.float32))
        at += k
    return cache, table


def test_attention_of_one_key_returns_its_value():
    rng = np.random.default_rng(5)
    cache, table = _filled(rng, 2, 64, 8, False, [1])
    q = rng.standard_normal((1, 6, 64))
    out, lse, _ = serving.attention(q, cache, table, [1], [0, 1], 0.3)
    for h in range(6):
        qv, s, z = cache.parts(table[0], h // 3, "v", 1)
        qk, sk, zk = cache.parts(table[0], h // 3, "k", 1)
        assert np.allclose(out[0, h], (qv[0] - z[0]) * s[0])
        assert np.isclose(lse[0, h], 0.3 * ((qk[0] - zk[0]) * sk[0]) @ q[0, h])


def test_attention_against_brute_force_and_empty_rows():
    """Two sequences, the second with more new rows than tokens held."""
    rng = np.random.default_rng(6)
    cache, table = _filled(rng, 1, 64, 4, True, [21, 3])
    q = rng.standard_normal((9, 2, 64))
    out, lse, _ = serving.attention(q, cache, table, [21, 3], [0, 4, 9], 0.125)
    assert np.all(out[4:6] == 0) and np.all(np.isneginf(lse[4:6])) and np.all(np.isfinite(lse[6:]))
    for seq, held, lo, hi in ((0, 21, 0, 4), (1, 3, 6, 9)):
        qk, sk, zk = cache.parts(table[seq], 0, "k", held)
        qv, sv, zv = cache.parts(table[seq], 0, "v", held)
        for r in range(lo, hi):
            for h in range(2):
                num, den = np.zeros(64), 0.0
                for j in range(held - (hi - r) + 1):
                    e = np.exp(0.125 * sum(q[r, h, i] * (qk[j, i] - zk[j]) * sk[j] for i in range(64)))
                    num, den = num + e * (qv[j] - zv[j]) * sv[j], den + e
                assert np.allclose(out[r, h], num / den) and np.isclose(lse[r, h], np.log(den))

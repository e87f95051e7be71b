"""CPU oracle of the serving operators: residual norm into INT8, the quantized
paged KV cache and attention over it. Plain numpy, loops over sequences and
heads; shares no code with the HIP library (TEST INFRASTRUCTURE, as the rest
of this package).

``tests/test_oracle_serving.py`` pins it: the per-token quantizer and the
group quantizer of ``oracle.c`` for the codes, hand-written byte positions for
the layout, closed forms and a brute-force softmax for the attention.
"""
from __future__ import annotations

import numpy as np

F32 = np.float32


def rms_norm_int8(x, weight, eps, residual=None):
    """float32 arrays x [t][k], weight [k] -> (qx int8, sx float32, h float32,
    y float32); fp32 roundings as defined, the sum of squares in fp64."""
    h = x.astype(F32) if residual is None else x.astype(F32) + residual.astype(F32)
    ss = (h.astype(np.float64) ** 2).sum(-1, keepdims=True)
    with np.errstate(divide="ignore", over="ignore"):
        r = np.minimum((1.0 / np.sqrt(ss / x.shape[1] + eps)).astype(F32), np.finfo(F32).max)
    y = (h * r) * weight.astype(F32)
    sx = np.maximum(np.abs(y).max(-1, keepdims=True), F32(1e-8)) / F32(127)
    q = np.clip(np.rint(y / sx), -127, 127).astype(np.int8)
    return q, sx[:, 0], h, y


def kv_quantize(x, bits, symmetric):
    """float32 [..., head_dim] -> (unsigned codes uint8, scale, zero or None): the
    group quantizer's formulas with the scale as a product with the rounded
    reciprocal of the level count."""
    x = x.astype(F32)
    if symmetric:
        qmax = F32(2 ** (bits - 1) - 1)
        s = np.maximum(np.abs(x).max(-1), F32(1e-8)) * (F32(1) / qmax)
        q = np.clip(np.rint(x / s[..., None]), -qmax, qmax) + F32(2 ** (bits - 1))
        return q.astype(np.uint8), s, None
    top = F32(2 ** bits - 1)
    lo, hi = x.min(-1), x.max(-1)
    s = np.maximum(hi - lo, F32(1e-8)) * (F32(1) / top)
    z = np.rint(-lo / s) + F32(0)
    q = np.clip(np.rint(x / s[..., None]) + z[..., None], 0, top)
    return q.astype(np.uint8), s, z


def kv_dequantize(q, s, z, bits):
    """fp32 values s (q - z) with one rounding of the product."""
    z = F32(2 ** (bits - 1)) if z is None else z[..., None]
    return (q.astype(F32) - z) * s[..., None]


class Cache:
    """The pool in its byte layout, and each slot's place in it."""

    def __init__(self, pages, page_size, heads, head_dim, bits, symmetric):
        self.page_size, self.heads, self.head_dim, self.bits, self.symmetric = page_size, heads, head_dim, bits, symmetric
        row = head_dim * bits // 8
        # slots nobody writes hold what must never show: NaN and stray codes
        self.k_codes = np.full((pages, heads, page_size, row), 0xA7, np.uint8)
        self.v_codes = np.full((pages, heads, page_size // 4, row, 4), 0xA7, np.uint8)
        n = (pages, heads, page_size)
        self.k_scales, self.v_scales = np.full(n, np.nan, F32), np.full(n, np.nan, F32)
        self.k_zeros = None if symmetric else np.full(n, np.nan, F32)
        self.v_zeros = None if symmetric else np.full(n, np.nan, F32)

    def put(self, page, offset, head, side, codes, s, z):
        if self.bits == 4:
            codes = codes[0::2] | (codes[1::2] << 4)
        if side == "k":
            self.k_codes[page, head, offset] = codes
        else:
            self.v_codes[page, head, offset // 4, :, offset % 4] = codes
        getattr(self, side + "_scales")[page, head, offset] = s
        if not self.symmetric:
            getattr(self, side + "_zeros")[page, head, offset] = z

    def put_rows(self, page, offset, side, x):
        """One token of float32 x [heads][head_dim]."""
        q, s, z = kv_quantize(x, self.bits, self.symmetric)
        for h in range(self.heads):
            self.put(page, offset, h, side, q[h], s[h], None if z is None else z[h])

    def codes(self, page, head, side):
        """Codes [page_size][head_dim] of a page and head."""
        b = self.k_codes[page, head] if side == "k" else np.swapaxes(self.v_codes[page, head], 1, 2).reshape(
            self.page_size, -1)
        if self.bits == 8:
            return b
        out = np.empty((self.page_size, self.head_dim), np.uint8)
        out[:, 0::2], out[:, 1::2] = b & 15, b >> 4
        return out

    def parts(self, pages, head, side, n):
        """codes, scale, zero (fp64) of the first n tokens of a list of pages"""
        q = np.concatenate([self.codes(p, head, side) for p in pages])[:n].astype(np.float64)
        s = np.concatenate([getattr(self, side + "_scales")[p, head] for p in pages])[:n].astype(np.float64)
        if self.symmetric:
            z = np.full(n, 2.0 ** (self.bits - 1))
        else:
            z = np.concatenate([getattr(self, side + "_zeros")[p, head] for p in pages])[:n].astype(np.float64)
        return q, s, z


def attention(q, cache, table, kv_lens, row_starts, scale):
    """float64 (out [rows][q_heads][head_dim], lse [rows][q_heads], bound like
    out). bound: how far a bf16 result of the stated arithmetic may be off,

      2^-8 |o|                       rounding the output to bf16
      (2^-11 + 2^-20 + 4 d) W        weights rounded to fp16, exp2, and scores
                                     off by d on both sides of the quotient
      n 2^-24 W'                     n fp32 additions per sum
      n 2^-27 max|v|                 weights below fp16's subnormals: half a step,
                                     2^-28 of the largest scale, times a code less
                                     a zero among the codes, at most twice max|v|
                                     over that scale

    with W = sum p |v| / sum p, W' the same of s (|c - mid| + |z - mid|), and
    d = (D + 8) 2^-24 max_j scale s_j sum |q| (|c - mid| + |z - mid|), the fp32
    rounding of a score."""
    rows, q_heads, d = q.shape
    group = q_heads // cache.heads
    mid = 2.0 ** (cache.bits - 1)
    out, bound = np.zeros((rows, q_heads, d)), np.zeros((rows, q_heads, d))
    lse = np.full((rows, q_heads), -np.inf)
    for b, held in enumerate(kv_lens):
        lo, hi = row_starts[b], row_starts[b + 1]
        if hi == lo or held <= 0:
            continue
        pages = table[b][:(held + cache.page_size - 1) // cache.page_size]
        for h in range(cache.heads):
            kq, ks, kz = cache.parts(pages, h, "k", held)
            vq, vs, vz = cache.parts(pages, h, "v", held)
            k, v = (kq - kz[:, None]) * ks[:, None], (vq - vz[:, None]) * vs[:, None]
            kabs = (np.abs(kq - mid) + np.abs(kz - mid)[:, None]) * ks[:, None]
            vabs = (np.abs(vq - mid) + np.abs(vz - mid)[:, None]) * vs[:, None]
            for r in range(lo, hi):
                n = held - (hi - r) + 1
                if n <= 0:
                    continue
                for j in range(h * group, (h + 1) * group):
                    x = q[r, j].astype(np.float64)
                    t = scale * (k[:n] @ x)
                    m = t.max()
                    p = np.exp(t - m)
                    out[r, j] = p @ v[:n] / p.sum()
                    lse[r, j] = m + np.log(p.sum())
                    delta = (d + 8) * 2.0 ** -24 * abs(scale) * (kabs[:n] @ np.abs(x)).max()
                    w, w2 = p @ np.abs(v[:n]) / p.sum(), p @ vabs[:n] / p.sum()
                    bound[r, j] = (2.0 ** -8 * np.abs(out[r, j]) + (2.0 ** -11 + 2.0 ** -20 + 4 * delta) * w
                                   + n * 2.0 ** -24 * w2 + n * 2.0 ** -27 * np.abs(v[:n]).max())
    return out, lse, bound

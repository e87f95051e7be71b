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


def attention_over(q, cache, sets, scale):
    """Attention of each row over the union of some sets of tokens: sets[r] is a
    list of (list of pages, tokens held in them), or None for a row that is left
    alone. float64 (out, lse, bound) as attention; 2^-19 in the place of 2^-20
    there: sets' results are joined in fp32 by two factors and a sum."""
    rows, q_heads, d = q.shape
    group, mid = q_heads // cache.heads, 2.0 ** (cache.bits - 1)
    out, bound = np.zeros((rows, q_heads, d)), np.zeros((rows, q_heads, d))
    lse, seen = np.full((rows, q_heads), -np.inf), {}

    def side(pages, h, name, n):
        key = tuple(pages), h, name
        if key not in seen:
            c, s, z = cache.parts(pages, h, name, len(pages) * cache.page_size)
            seen[key] = (c - z[:, None]) * s[:, None], (np.abs(c - mid) + np.abs(z - mid)[:, None]) * s[:, None]
        return seen[key][0][:n], seen[key][1][:n]

    for r in range(rows):
        live = [(pages[:(n + cache.page_size - 1) // cache.page_size], n) for pages, n in sets[r] or [] if n > 0]
        if not live:
            continue
        for h in range(cache.heads):
            k, kabs = (np.concatenate(x) for x in zip(*(side(p, h, "k", n) for p, n in live)))
            v, vabs = (np.concatenate(x) for x in zip(*(side(p, h, "v", n) for p, n in live)))
            for j in range(h * group, (h + 1) * group):
                x = q[r, j].astype(np.float64)
                t = scale * (k @ x)
                m = t.max()
                p = np.exp(t - m)
                out[r, j] = p @ v / p.sum()
                lse[r, j] = m + np.log(p.sum())
                delta = (d + 8) * 2.0 ** -24 * abs(scale) * (kabs @ np.abs(x)).max()
                w, w2 = p @ np.abs(v) / p.sum(), p @ vabs / p.sum()
                bound[r, j] = (2.0 ** -8 * np.abs(out[r, j]) + (2.0 ** -11 + 2.0 ** -19 + 4 * delta) * w
                               + len(t) * (2.0 ** -24 * w2 + 2.0 ** -27 * np.abs(v).max()))
    return out, lse, bound


def weigh(q, lse, cache, weights, table, kv_lens, row_starts, scale, causal=True):
    """float64 weights after a call over float32 weights [pages][heads][page_size]
    (NaN in, NaN out where nothing is written) and a bound like them of what fp32
    may be off. With p a row's weight and x its score, p is off by
      (D + 8) 2^-24 scale s sum |q| (|c - mid| + |z - mid|)    the score's product
      6 2^-24 (|x| + |lse|) + 2^-21       its scaling, the difference and exp2
    relative to itself, and the sum of n of them by n 2^-24, the old weight's
    addition by 2^-24."""
    rows, q_heads, d = q.shape
    group, mid, ps = q_heads // cache.heads, 2.0 ** (cache.bits - 1), cache.page_size
    out, bound = weights.astype(np.float64), np.zeros(weights.shape)
    for b, held in enumerate(kv_lens):
        lo, hi = row_starts[b], row_starts[b + 1]
        if hi == lo or held <= 0:
            continue
        pages, pos = table[b][:(held + ps - 1) // ps], np.arange(held)
        at = np.asarray(pages)[pos // ps], pos % ps
        for h in range(cache.heads):
            c, s, z = cache.parts(pages, h, "k", held)
            k, kabs = (c - z[:, None]) * s[:, None], (np.abs(c - mid) + np.abs(z - mid)[:, None]) * s[:, None]
            total, off = np.zeros(held), np.zeros(held)
            for r in range(lo, hi):
                n = max(0, held - (hi - r) + 1) if causal else held
                for j in range(h * group, (h + 1) * group):
                    if not np.isfinite(lse[r, j]):
                        continue
                    y = q[r, j].astype(np.float64)
                    x = scale * (k[:n] @ y)
                    p = np.exp(x - lse[r, j])
                    rel = ((d + 8) * abs(scale) * (kabs[:n] @ np.abs(y)) + 6 * (np.abs(x) + abs(lse[r, j]))) * 2.0 ** -24
                    total[:n] += p
                    off[:n] += p * (np.expm1(rel) + 2.0 ** -21)
            was = out[at[0], h, at[1]]
            if causal:
                was = np.where(pos < held - (hi - lo), was, 0.0)
            out[at[0], h, at[1]] = was + total
            bound[at[0], h, at[1]] = off + ((hi - lo) * group + 8) * 2.0 ** -24 * (total + np.abs(was))
    return out, bound


def evict(cache, weights, table, kv_lens, keep, recent, to_table=None):
    """Evicts in place of the oracle's cache and weights; table, to_table: lists of
    pages of each sequence. Returns (kept [b][heads][keep], new lengths)."""
    to_table, ps = to_table or table, cache.page_size
    kept, lens = np.full((len(kv_lens), cache.heads, keep), -1, np.int32), []
    names = ["k_scales", "v_scales"] + ([] if cache.symmetric else ["k_zeros", "v_zeros"])
    for b, held in enumerate(kv_lens):
        lens.append(min(max(held, 0), keep))
        for h in range(cache.heads):
            pos = np.arange(max(held, 0))
            if held > keep:
                w = np.array([weights[table[b][i // ps], h, i % ps] for i in range(held - recent)], np.float64)
                # NaN is heaviest; a stable sort of the negatives keeps the earlier of equal ones
                best = np.argsort(np.where(np.isnan(w), -np.inf, -w), kind="stable")
                nan_first = np.concatenate([best[np.isnan(w[best])], best[~np.isnan(w[best])]])
                pos = np.concatenate([np.sort(nan_first[:keep - recent]), np.arange(held - recent, held)])
            kept[b, h, :len(pos)] = pos
            src = [(table[b][i // ps], i % ps) for i in pos]
            k = [cache.k_codes[p, h, o].copy() for p, o in src]
            v = [cache.v_codes[p, h, o // 4, :, o % 4].copy() for p, o in src]
            numbers = [[a[p, h, o] for p, o in src] for a in [weights] + [getattr(cache, n) for n in names]]
            for j in range(len(pos)):
                p, o = to_table[b][j // ps], j % ps
                cache.k_codes[p, h, o], cache.v_codes[p, h, o // 4, :, o % 4] = k[j], v[j]
                for a, x in zip([weights] + [getattr(cache, n) for n in names], numbers):
                    a[p, h, o] = x[j]
    return kept, lens

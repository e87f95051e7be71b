"""Shared by the serving operators' GPU tests: batches with ragged lengths and
scattered pages, built on the host by the oracle."""
import numpy as np
import torch

import bit_gemv_amd as bg
from gpu_helpers import dev
from oracle import serving
from workloads import bf16_bits_to_f32, f32_to_bf16_bits


def bf16(a):
    """float array -> the nearest bf16 values, as float32"""
    return bf16_bits_to_f32(f32_to_bf16_bits(np.asarray(a, np.float32)))


def dev_bf16f(a):
    """float32 array of bf16 values -> bf16 GPU tensor"""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(torch.bfloat16)


class Batch:
    """Sequences (tokens held, new rows) over scattered pages. Table entries
    past a sequence's pages are out of the pool on purpose."""

    def __init__(self, seqs, page, rng, spare=2, lead=0, wide=0):
        self.kv = [s[0] for s in seqs]
        self.starts = [lead]
        for s in seqs:
            self.starts.append(self.starts[-1] + s[1])
        self.rows = self.starts[-1]
        need = [(n + page - 1) // page for n in self.kv]
        self.pages = sum(need) + spare
        order, at = rng.permutation(self.pages), 0
        wide = max(need + [1, wide]) + 1
        self.table = np.where(rng.random((len(seqs), wide)) < 0.5, -1, 1 << 30).astype(np.int32)
        self.lists = []
        for i, n in enumerate(need):
            self.lists.append([int(x) for x in order[at:at + n]])
            self.table[i, :n] = self.lists[-1]
            at += n

    def on_gpu(self):
        return dev(self.table), dev(np.asarray(self.kv, np.int32)), dev(np.asarray(self.starts, np.int32))

    def positions(self):
        """(row, sequence, position) of every row that belongs to a sequence"""
        for i, held in enumerate(self.kv):
            for r in range(self.starts[i], self.starts[i + 1]):
                yield r, i, held - (self.starts[i + 1] - r)


def fill(cache, batch, rng, k_scale=1.0, v_scale=1.0, skip_new=False):
    """Writes every held token into the oracle's cache; k_scale, v_scale: a
    factor, or a function of (sequence, position)."""
    f = lambda s, i, t: s(i, t) if callable(s) else s  # noqa: E731
    shape = (cache.heads, cache.head_dim)
    for i, held in enumerate(batch.kv):
        n = held - (batch.starts[i + 1] - batch.starts[i]) if skip_new else held
        for t in range(max(0, n)):
            at = batch.lists[i][t // cache.page_size], t % cache.page_size
            cache.put_rows(*at, "k", rng.standard_normal(shape) * f(k_scale, i, t))
            cache.put_rows(*at, "v", rng.standard_normal(shape) * f(v_scale, i, t))


def to_gpu(c):
    z = lambda a: None if a is None else dev(a)  # noqa: E731
    return bg.KVCache(dev(c.k_codes), dev(c.v_codes), dev(c.k_scales), dev(c.v_scales), z(c.k_zeros), z(c.v_zeros),
                      c.head_dim, c.bits)


def new_cache(batch, page, heads, d, bits, sym):
    return serving.Cache(batch.pages, page, heads, d, bits, sym)


def check_attention(got, lse, want, want_lse, bound, what, rows=slice(None)):
    """Every element of a bf16 result within the bound derived in
    oracle.serving.attention; the log-sum-exp (fp32) within 2^-20 of its own
    size plus 1e-5 (fp32 scores, sums of positive terms, exp2 and log)."""
    got = got.float().cpu().numpy().astype(np.float64)[rows]
    assert np.all(np.isfinite(got)), what
    err, b = np.abs(got - want[rows]), bound[rows]
    bad = err > b
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst {(err / np.maximum(b, 1e-300)).max():.2f} times "
                           f"the bound at {np.argwhere(bad)[0]}: {got[tuple(np.argwhere(bad)[0])]} for "
                           f"{want[rows][tuple(np.argwhere(bad)[0])]}")
    if lse is not None:
        lse, wl = lse.cpu().numpy().astype(np.float64)[rows], want_lse[rows]
        assert np.array_equal(np.isneginf(lse), np.isneginf(wl)), what
        ok = np.isfinite(wl)
        assert np.all(np.abs(lse[ok] - wl[ok]) <= 1e-5 + 2.0 ** -20 * np.abs(wl[ok])), what

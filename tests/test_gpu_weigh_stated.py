"""What libquant.h states of kv_cache_weigh beside its formula: how a new prompt is
weighed in pages that held other tokens, and the error where a score's terms
cancel."""
import numpy as np
import pytest
import torch

import bit_gemv_amd as bg
from gpu_helpers import dev, host, say
from oracle import serving
from serving_helpers import Batch, bf16, dev_bf16f, fill, new_cache, to_gpu
from test_gpu_weigh_evict import FORMATS, _check_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hints", [(0, 0), (1, 0)])
def test_a_prompt_weighed_by_its_last_rows_in_pages_that_held_others(hints):
    """The weights in recycled pages are others' and huge. Weighed from NULL, as
    the header says of a new prompt, no slot keeps any of them, and the next
    call's additions in place go on from there; in place from the start they
    would count."""
    rng = np.random.default_rng(39)
    b = Batch([(100, 8), (37, 3)], 16, rng)
    ref = new_cache(b, 16, 1, 64, 8, True)
    fill(ref, b, rng)
    q = bf16(rng.standard_normal((b.rows, 12, 64)))
    gpu, gq = to_gpu(ref), dev_bf16f(q)
    stale = np.full(ref.k_scales.shape, 1e6, np.float32)
    batch, lse = b.on_gpu(), torch.empty(q.shape[:2], device="cuda")
    say("recycled pages", hints)
    bg.paged_attention(gq, gpu, *batch, scale=0.125, lse=lse)
    w = dev(stale)
    args = dict(scale=0.125, max_rows=hints[0], max_kv=hints[1])
    bg.kv_cache_weigh(gq, lse, gpu, None, *batch, out=w, **args)
    fresh, bound = serving.weigh(q, host(lse), ref, np.zeros_like(stale), b.lists, b.kv, b.starts, 0.125)
    _check_weights(w, stale, np.where(bound > 0, fresh, stale), bound, "from NULL")
    first = host(w)
    bg.kv_cache_weigh(gq, lse, gpu, w, *batch, **args)
    want, bound = serving.weigh(q, host(lse), ref, first, b.lists, b.kv, b.starts, 0.125)
    _check_weights(w, first, want, bound, "in place")
    w = dev(stale)
    bg.kv_cache_weigh(gq, lse, gpu, w, *batch, **args)
    for i, n in enumerate(b.kv):
        old = [(b.lists[i][t // 16], 0, t % 16) for t in range(n - (8, 3)[i])]
        assert all(host(w)[at] >= 1e6 for at in old)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bits,sym", FORMATS)
def test_scores_whose_terms_cancel(bits, sym, d):
    """Query elements of 500 to 1000 that cancel over keys of nearly one value,
    beside some of about 1: the sums on the way are rounded at their own size,
    180 to 400 times 2^-24 of the scores and log-sums (128-wide), and stay within
    the bound on the terms' magnitudes that the header gives."""
    rng = np.random.default_rng(d + bits)
    b = Batch([(200, 40), (90, 3)], 16, rng)
    ref = new_cache(b, 16, 1, d, bits, sym)
    fill(ref, b, rng)
    for i, held in enumerate(b.kv):
        for t in range(held):
            ref.put_rows(b.lists[i][t // 16], t % 16, "k", np.where(np.arange(d) % 2, 3.0, 2.9)[None])
    big, small = bf16(rng.uniform(500, 1000, (b.rows, 3, d // 4))), bf16(rng.standard_normal((b.rows, 3, d // 2)))
    q = np.concatenate((big, small, -big), -1)
    sets = [None] * b.rows
    for r, i, pos in b.positions():
        sets[r] = [(b.lists[i], pos + 1)]
    lse = serving.attention_over(q, ref, sets, d ** -0.5)[1].astype(np.float32)
    zero = np.zeros(ref.k_scales.shape, np.float32)
    want, bound = serving.weigh(q, lse, ref, zero, b.lists, b.kv, b.starts, d ** -0.5)
    for max_rows in (40, 1):
        say(f"cancelling scores D={d} bits={bits} sym={sym} max_rows {max_rows}")
        got = bg.kv_cache_weigh(dev_bf16f(q), dev(lse), to_gpu(ref), None, *b.on_gpu(), max_rows=max_rows)
        _check_weights(got, zero, want, bound, f"max_rows {max_rows}")

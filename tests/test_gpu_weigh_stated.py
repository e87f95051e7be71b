"""What libquant.h states of kv_cache_weigh beside its formula: how a new prompt is
weighed in pages that held other tokens."""
import numpy as np
import pytest
import torch

import bit_gemv_amd as bg
from gpu_helpers import dev, host, say
from oracle import serving
from serving_helpers import Batch, bf16, dev_bf16f, fill, new_cache, to_gpu
from test_gpu_weigh_evict import _check_weights

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

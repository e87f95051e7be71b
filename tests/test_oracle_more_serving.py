"""Pins of the oracle of attention over several sets of tokens, weights and
eviction (oracle/serving.py). CPU only."""
import numpy as np
import pytest

from oracle import serving


def _cache(rng, pages=6, heads=2, d=64, bits=8, sym=False):
    c = serving.Cache(pages, 16, heads, d, bits, sym)
    for p in range(pages):
        for o in range(16):
            for side in "kv":
                c.put_rows(p, o, side, rng.standard_normal((heads, d)))
    return c


@pytest.mark.parametrize("bits,sym", [(4, False), (8, True)])
def test_over_one_set_it_is_attention(bits, sym):
    """Causal attention by the older oracle, its own positions as the set."""
    rng = np.random.default_rng(1)
    c = _cache(rng, bits=bits, sym=sym)
    q = rng.standard_normal((5, 4, 64)).astype(np.float32)
    want, wl, _ = serving.attention(q, c, [[3, 1], [0, 5, 2]], [20, 40], [0, 2, 5], 0.125)
    sets = [[([3, 1], 19 + r)] for r in range(2)] + [[([0, 5, 2], 38 + r)] for r in range(3)]
    got, gl, _ = serving.attention_over(q, c, sets, 0.125)
    assert np.allclose(got, want, rtol=1e-12, atol=1e-12) and np.allclose(gl, wl, rtol=1e-12)


def test_cutting_a_set_changes_nothing_and_no_set_gives_zeros():
    rng = np.random.default_rng(2)
    c, q = _cache(rng), rng.standard_normal((4, 4, 64)).astype(np.float32)
    sets = [[([3, 1, 2], 37)], [([3], 16), ([1], 16), ([2], 5)], [([3], 0)], None]
    out, lse, _ = serving.attention_over(np.repeat(q[:1], 4, 0), c, sets, 0.125)
    assert np.allclose(out[0], out[1], rtol=1e-12, atol=1e-12) and np.allclose(lse[0], lse[1])
    assert not out[2:].any() and np.isneginf(lse[2:]).all()


def test_weights_are_the_softmax_summed_over_rows_and_heads():
    rng = np.random.default_rng(3)
    c, q = _cache(rng), rng.standard_normal((3, 4, 64)).astype(np.float32)
    sets = [[([4, 0], 18 + r)] for r in range(3)]
    lse = serving.attention_over(q, c, sets, 0.125)[1].astype(np.float32)
    w = np.full(c.k_scales.shape, 2.0, np.float32)
    out, bound = serving.weigh(q, lse, c, w, [[4, 0]], [20], [0, 3], 0.125)
    for h in range(2):
        k, s, z = c.parts([4, 0], h, "k", 20)
        t = 0.125 * np.einsum("rjd,kd->rjk", q[:, 2 * h:2 * h + 2].astype(np.float64), (k - z[:, None]) * s[:, None])
        for r in range(3):
            t[r, :, 18 + r:] = -np.inf
        p = np.exp(t - t.max(-1, keepdims=True))
        p = (p / p.sum(-1, keepdims=True)).sum((0, 1))
        got = np.concatenate([out[4, h], out[0, h]])[:20]
        assert np.allclose(got, p + np.where(np.arange(20) < 17, 2.0, 0.0), rtol=1e-6)   # lse rounded to fp32
    assert np.all(out[[1, 2, 3, 5]] == 2.0) and np.all(out[0, :, 4:] == 2.0) and not bound[[1, 2, 3, 5]].any()
    whole, _ = serving.weigh(q, lse, c, w, [[4, 0]], [20], [0, 3], 0.125, causal=False)
    assert np.all(whole[4] >= 2.0) and np.all(whole[0, :, :4] > 2.0)
    lse[1] = -np.inf
    less, _ = serving.weigh(q, lse, c, w, [[4, 0]], [20], [0, 3], 0.125)
    assert np.all(less <= out) and np.all(less[4] < out[4])


def test_eviction_by_hand():
    """Six tokens to four, the last always kept: by weight, ties to the earlier,
    each head its own; codes, numbers and weights follow."""
    rng = np.random.default_rng(4)
    c = _cache(rng)
    w = np.zeros(c.k_scales.shape, np.float32)
    w[3, 0, :6] = [1, 5, 1, 7, 1, 0]
    w[3, 1, :6] = [np.nan, -1, np.inf, 0, 2, 9]
    k, v, s = c.k_codes.copy(), c.v_codes.copy(), c.v_zeros.copy()
    kept, lens = serving.evict(c, w, [[3], [5]], [6, 4], 4, 1)
    assert lens == [4, 4]
    assert kept[0].tolist() == [[0, 1, 3, 5], [0, 2, 4, 5]] and kept[1].tolist() == [[0, 1, 2, 3]] * 2
    for h in range(2):
        for j, i in enumerate(kept[0, h]):
            assert np.array_equal(c.k_codes[3, h, j], k[3, h, i]) and c.v_zeros[3, h, j] == s[3, h, i]
            assert np.array_equal(c.v_codes[3, h, j // 4, :, j % 4], v[3, h, i // 4, :, i % 4])
    assert w[3, 0, :4].tolist() == [1, 5, 7, 0]
    assert np.array_equal(c.k_codes[[0, 1, 2, 4, 5]], k[[0, 1, 2, 4, 5]])
    kept, lens = serving.evict(c, w, [[3]], [4], 2, 0, [[0]])
    assert kept[0, 0].tolist() == [1, 2] and lens == [2] and w[0, 0, :2].tolist() == [5, 7]

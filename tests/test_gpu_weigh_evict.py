"""kv_cache_weigh against the oracle in 64 bits within a derived bound
(oracle.serving.weigh), kv_cache_evict against it bit for bit, and both in a
run of calls as a server makes them."""
import ctypes

import numpy as np
import pytest
import torch

import bit_gemv_amd as bg
from gpu_helpers import assert_same_bits, dev, host, say
from oracle import serving
from serving_helpers import Batch, bf16, check_attention, dev_bf16f, fill, new_cache, to_gpu
from test_gpu_guard import Guarded, _ok, _p, _st

pytestmark = pytest.mark.gpu

FORMATS = [(4, False), (4, True), (8, False), (8, True)]
SEQS = [(1, 1), (17, 1), (16, 16), (33, 5), (70, 70), (261, 3), (3, 6), (0, 2), (40, 0), (129, 1)]


def _i32(v):
    return dev(np.asarray(v, np.int32))


def _weights(ref, rng):
    """Weights summed up before: heavy-tailed, a quarter exactly zero."""
    shape = ref.k_scales.shape
    return (np.exp(2 * rng.standard_normal(shape)) * (rng.random(shape) > 0.25)).astype(np.float32)


def _check_weights(got, before, want, bound, what):
    got = got.cpu().numpy().astype(np.float64)
    touched = bound > 0
    assert np.array_equal(got[~touched], before[~touched].astype(np.float64), equal_nan=True), f"{what}: other slots changed"
    err = np.abs(got - want)[touched]
    assert np.all(np.isfinite(got[touched])), what
    worst = (err / bound[touched]).max() if err.size else 0
    assert worst <= 1, f"{what}: {worst:.2f} times the bound"


def _weigh(seqs, d, bits, sym, page=16, heads=2, group=4, seed=0, causal=True, hints=((0, 0),), scale=None, q_scale=1.0,
           gap=0, lead=0, wide=0, k_scale=1.0, what="", far=False):
    rng = np.random.default_rng(seed)
    b = Batch(seqs, page, rng, lead=lead, wide=wide)
    ref = new_cache(b, page, heads, d, bits, sym)
    fill(ref, b, rng, k_scale)
    if far:  # keys far from zero for their range: zeros outside the codes
        for i, held in enumerate(b.kv):
            for t in range(i % 3, held, 5):
                x = (5 + 0.01 * rng.standard_normal((heads, d)), np.full((heads, d), 0.03125), -7 - rng.random((heads, d)))
                ref.put_rows(b.lists[i][t // page], t % page, "k", x[t % 3])
    gpu = to_gpu(ref)
    rows, qh, sc = b.rows + 1, heads * group, d ** -0.5 if scale is None else scale
    q = bf16(rng.standard_normal((rows, qh, d)) * q_scale)
    sets = [None] * rows
    for r, i, pos in b.positions():
        sets[r] = [(b.lists[i], min(pos + 1, b.kv[i]) if causal else b.kv[i])]
    lse = serving.attention_over(q, ref, sets, sc)[1].astype(np.float32)
    w = _weights(ref, rng)
    want, bound = serving.weigh(q, lse, ref, w, b.lists, b.kv, b.starts, sc, causal)
    zero, zero_bound = serving.weigh(q, lse, ref, np.zeros_like(w), b.lists, b.kv, b.starts, sc, causal)
    pad = torch.full((rows, qh + gap, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    pad[:, :qh] = dev_bf16f(q)
    for max_rows, max_kv in hints:
        name = f"kv_cache_weigh {what} D={d} bits={bits} sym={sym} page={page} group={group} causal={causal} {max_rows, max_kv}"
        say(name)
        args = dict(scale=scale, causal=causal, max_rows=max_rows, max_kv=max_kv)
        batch = b.on_gpu()
        out = torch.full(w.shape, 7.0, device="cuda")
        bg.kv_cache_weigh(pad[:, :qh], dev(lse), gpu, dev(w), *batch, out=out, **args)
        _check_weights(out, np.full_like(w, 7.0), want, bound, name)
        here = dev(w)
        assert bg.kv_cache_weigh(pad[:, :qh], dev(lse), gpu, here, *batch, **args) is here
        _check_weights(here, w, want, bound, name + " in place")
        _check_weights(bg.kv_cache_weigh(pad[:, :qh], dev(lse), gpu, None, *batch, **args), np.zeros_like(w), zero, zero_bound,
                       name + " from zero")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("bits,sym", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_weigh_formats(d, bits, sym, causal):
    """Bounds that choose each kernel, right and wrong: rows streamed past keys,
    shared by blocks and (a wide table and no bound) not; keys past 16 rows."""
    _weigh(SEQS, d, bits, sym, seed=d + bits, causal=causal, hints=((0, 0), (70, 261), (4, 261), (1, 17)))
    _weigh(SEQS, d, bits, sym, seed=d + bits, causal=causal, wide=512, hints=((0, 0), (1, 0)))


@pytest.mark.parametrize("bits,sym", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_weigh_single_tokens(d, bits, sym):
    _weigh([(1, 1), (2, 1), (31, 1), (32, 1), (33, 1), (128, 1), (300, 1), (16, 1), (0, 1)], d, bits, sym, seed=d + 1,
           hints=((1, 300), (1, 0)))


@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 16, 20, 33])
@pytest.mark.parametrize("bits,sym", [(4, False), (8, True)])
def test_weigh_head_layouts(group, bits, sym):
    _weigh([(37, 1), (50, 11), (20, 20)], 64, bits, sym, heads=1 if group > 8 else 3, group=group, seed=group,
           hints=((20, 50), (1, 50)), gap=2, lead=3)


@pytest.mark.parametrize("page", [16, 64, 256])
def test_weigh_pages_and_long_sequences(page):
    _weigh([(1300, 1), (270, 18), (257, 257), (5, 2)], 64, 8, True, page=page, heads=1, group=2, seed=page,
           hints=((0, 0), (1, 1300)))
    _weigh([(9001, 2)], 64, 4, False, page=page, heads=1, group=1, seed=page, hints=((2, 9001), (40, 9001)))


@pytest.mark.parametrize("d,bits,sym", [(64, 8, True), (128, 4, False), (256, 8, False)])
def test_weigh_shared_rows(d, bits, sym):
    """Runs of keys whose rows several blocks share: whole prompts, chunks, rows
    that see all; bounds of the lengths too small, so that only some runs are."""
    seqs = [(300, 300), (500, 130), (40, 40), (700, 7), (0, 3)]
    for causal in (True, False):
        _weigh(seqs, d, bits, sym, seed=d, heads=1, group=3, causal=causal, hints=((0, 0), (300, 700), (300, 200), (40, 1)),
               wide=64)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_weigh_zeros_far_from_the_codes(bits, d):
    _weigh([(200, 40), (90, 3), (70, 1)], d, bits, False, seed=9, heads=1, q_scale=0.2, far=True,
           hints=((40, 200), (40, 9000), (1, 200)), wide=512)


@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0, 1e-4])
def test_weigh_scale(scale):
    _weigh([(33, 5), (200, 1)], 64, 8, True, seed=8, scale=scale, hints=((5, 200), (1, 200)))


def test_weights_of_one_step_add_up_to_the_number_of_rows():
    """The rows' weights are their softmax: over keys they sum to 1 each. bf16 of
    attention has no part in it: 2^-20 relative a weight and fp32 sums."""
    rng = np.random.default_rng(3)
    b = Batch([(900, 1), (70, 70), (300, 9)], 16, rng)
    ref = new_cache(b, 16, 2, 128, 8, True)
    fill(ref, b, rng)
    gpu, q = to_gpu(ref), torch.randn((b.rows, 8, 128), device="cuda").bfloat16()
    lse = torch.empty((b.rows, 8), device="cuda")
    bg.paged_attention(q, gpu, *b.on_gpu(), lse=lse)
    w = bg.kv_cache_weigh(q, lse, gpu, None, *b.on_gpu())
    for i, n in enumerate((1, 70, 9)):
        total = w[b.lists[i]].double().sum((0, 2)).cpu().numpy()
        assert np.all(np.abs(total - 4 * n) <= 4 * n * 1e-4), (i, total)


def test_rows_without_a_finite_log_sum_add_nothing():
    rng = np.random.default_rng(4)
    b = Batch([(40, 3), (90, 20)], 16, rng)
    ref = new_cache(b, 16, 1, 64, 8, True)
    fill(ref, b, rng)
    gpu, q = to_gpu(ref), torch.randn((b.rows, 2, 64), device="cuda").bfloat16()
    lse = torch.full((b.rows, 2), 3.0, device="cuda")
    for max_rows in (0, 1):
        say("lse not finite", max_rows)
        bad_q, bad = q.clone(), lse.clone()
        bad_q[1, 1], bad[1, 1] = float("nan"), float("nan")
        bad_q[7, 0], bad[7, 0], bad[9, 1] = float("inf"), float("inf"), -float("inf")
        zero_q = q.clone()
        got = bg.kv_cache_weigh(bad_q, bad, gpu, None, *b.on_gpu(), max_rows=max_rows)
        away = lse.clone()
        for r, h in ((1, 1), (7, 0), (9, 1)):
            away[r, h] = 1e4                       # exp(x - 1e4) is 0 in fp32
        want = bg.kv_cache_weigh(zero_q, away, gpu, None, *b.on_gpu(), max_rows=max_rows)
        assert torch.equal(got, want) and bool(torch.isfinite(got).all())


def _state(ref, w):
    names = ["k_codes", "v_codes", "k_scales", "v_scales"] + ([] if ref.symmetric else ["k_zeros", "v_zeros"])
    return {n: getattr(ref, n).copy() for n in names} | {"weights": w.copy()}


def _evict(lens, keep, recent, d=64, bits=8, sym=True, page=16, heads=2, seed=0, elsewhere=False, weights=None, hints=(0,)):
    rng = np.random.default_rng(seed)
    room = [(min(n, keep), 0) for n in lens] if elsewhere else []
    b = Batch([(n, 0) for n in lens] + room, page, rng)
    ref = new_cache(b, page, heads, d, bits, sym)
    n = len(lens)
    for t in (ref.k_codes, ref.v_codes):
        t[:] = rng.integers(0, 256, t.shape, dtype=np.uint8)
    for t in (ref.k_scales, ref.v_scales, ref.k_zeros, ref.v_zeros):
        if t is not None:
            t[:] = rng.random(t.shape, dtype=np.float32)
    w = _weights(ref, rng)
    if weights is not None:
        w[:] = weights(rng, w.shape)
    table, lists, to = dev(b.table[:n]), b.lists[:n], b.lists[n:]
    to_table = dev(np.ascontiguousarray(b.table[n:])) if elsewhere else None
    start = _state(ref, w)
    first = to_gpu(ref)
    want_kept, want_lens = serving.evict(ref, w, lists, lens, keep, recent, to if elsewhere else None)
    want = _state(ref, w)
    for max_kv in hints:
        gpu, wg = to_gpu(ref), dev(start["weights"])
        for name in start:
            if name != "weights":
                getattr(gpu, name).copy_(getattr(first, name))
        say(f"kv_cache_evict lens {lens[:6]} keep {keep} recent {recent} D={d} bits={bits} sym={sym} page={page} heads={heads} "
            f"elsewhere={elsewhere} max_kv {max_kv}")
        got_lens, kept = bg.kv_cache_evict(gpu, wg, table, _i32(lens), keep, recent, to_table=to_table, max_kv=max_kv)
        assert host(got_lens).tolist() == want_lens
        assert_same_bits(host(kept), want_kept, "kept")
        got = {name: host(wg if name == "weights" else getattr(gpu, name)) for name in start}
        # what stayed, and (of the rest) what no page of the target holds
        free = np.ones(ref.k_scales.shape, bool)
        for i, pages in enumerate(to if elsewhere else lists):
            free[pages] = False
            for j in range(want_lens[i]):
                p, o = pages[j // page], j % page
                for name in start:
                    at = (p, slice(None), o // 4, slice(None), o % 4) if name == "v_codes" else (p, slice(None), o)
                    assert np.array_equal(got[name][at], want[name][at], equal_nan=True), (name, i, j)
        for name in start:
            rest = free[:, 0, 0]
            assert np.array_equal(got[name][rest], start[name][rest], equal_nan=True), f"{name}: other pages changed"


@pytest.mark.parametrize("elsewhere", [False, True])
@pytest.mark.parametrize("bits,sym", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_evict_formats(d, bits, sym, elsewhere):
    _evict([100, 33, 17, 16, 1, 0, 257], 17, 5, d, bits, sym, seed=d + bits, elsewhere=elsewhere)


@pytest.mark.parametrize("elsewhere", [False, True])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (5, 0), (64, 64), (99, 3), (100, 0), (255, 128), (300, 300), (1000, 7)])
def test_evict_budgets(keep, recent, elsewhere):
    """All budgets from one token to more than there are; only recent ones; none."""
    _evict([300, 99, 100, 101, 1024], keep, recent, seed=keep, elsewhere=elsewhere)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("heads", [1, 5])
def test_evict_pages_and_heads(page, heads):
    _evict([700, 255, 1025], 301, 40, page=page, heads=heads, seed=page, bits=4)


def test_evict_ties_and_odd_values():
    """All weights alike, all zero, of both zeros, negative, infinite, NaN,
    subnormal, neighbours in the last bit."""
    one = np.float32(1.0)
    for f in (lambda r, s: np.zeros(s, np.float32), lambda r, s: np.full(s, 0.5, np.float32),
              lambda r, s: np.where(r.random(s) < 0.5, np.float32(-0.0), np.float32(0.0)),
              lambda r, s: r.standard_normal(s).astype(np.float32),
              lambda r, s: r.choice(np.array([np.nan, np.inf, -np.inf, 0.0, -1.0, 1e-40, 3e38], np.float32), s),
              lambda r, s: np.where(r.random(s) < 0.3, np.nextafter(one, np.float32(2)), one),
              lambda r, s: r.choice(np.array([one, np.nextafter(one, np.float32(0)), np.nextafter(one, np.float32(2))]), s)):
        _evict([500, 130, 65], 64, 10, seed=5, weights=f)


@pytest.mark.parametrize("n", [4095, 4097, 32768, 32900, 50001])
def test_evict_long_sequences(n):
    """Past what a block holds at once."""
    _evict([n, n // 3], n // 5, 100, heads=1, bits=4, seed=n, hints=(0, n))
    _evict([n], n - 7, 0, heads=1, bits=4, seed=n, weights=lambda r, s: r.integers(0, 3, s).astype(np.float32), hints=(n, 1))


def test_evict_ignores_pages_outside_the_pool():
    """They go first; the others' choice and place do not change."""
    c = bg.KVCache.empty(8, 16, 1, 64)
    for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
        t.fill_(1)
    w = torch.arange(128, device="cuda", dtype=torch.float32).view(8, 1, 16) + 1
    say("evict, bad pages")
    table = _i32([[0, -1, 2, 99, 4]])
    lens, kept = bg.kv_cache_evict(c, w.clone(), table, _i32([75]), 40, 3)
    assert host(lens).tolist() == [40]
    # 43 positions of the pool (0-15, 32-47, 64-74); the last three stay, and the 37 heaviest of the other 40
    assert host(kept)[0, 0].tolist() == list(range(3, 16)) + list(range(32, 48)) + list(range(64, 75))
    lens, kept = bg.kv_cache_evict(c, w, table, _i32([75]), 50, 0)
    pos = host(kept)[0, 0]
    assert np.all(np.diff(pos) > 0) and set(range(16)) | set(range(32, 48)) | set(range(64, 75)) <= set(pos.tolist())
    lens, kept = bg.kv_cache_evict(c, w, table, _i32([-5]), 4, 0)
    assert host(lens).tolist() == [0] and bool((kept == -1).all())
    lens, kept = bg.kv_cache_evict(c, w, table, _i32([1 << 30]), 100, 0)     # cut to the table
    assert host(lens).tolist() == [80]


def test_lengths_updated_in_place_by_many_sequences():
    """More blocks than run at once read the lengths that others replace."""
    heads, d, n, keep = 8, 64, 260, 20
    rng = np.random.default_rng(2)
    b = Batch([(40 + i % 30, 0) for i in range(n)], 16, rng)
    c = bg.KVCache.empty(b.pages, 16, heads, d)
    c.k_codes.copy_(torch.from_numpy(rng.integers(0, 256, c.k_codes.shape, dtype=np.uint8)))
    for t in (c.v_codes, c.k_scales, c.v_scales):
        t.fill_(3)
    w = dev(rng.random(c.k_scales.shape, dtype=np.float32))
    table, lens, _ = b.on_gpu()
    before, k0, w0 = lens.clone(), host(c.k_codes).copy(), host(w).copy()
    say("evict, lengths in place")
    _, kept = bg.kv_cache_evict(c, w, table, lens, keep, 3, new_lens=lens)
    assert bool((lens == keep).all())
    kept, k1, w1 = host(kept), host(c.k_codes), host(w)
    for i in range(n):
        for h in range(heads):
            old = [w0[b.lists[i][t // 16], h, t % 16] for t in range(b.kv[i])]
            best = sorted(range(b.kv[i] - 3), key=lambda t: (-old[t], t))[:keep - 3]
            assert kept[i, h].tolist() == sorted(best) + list(range(b.kv[i] - 3, b.kv[i])), (i, h)
            for j, t in enumerate(kept[i, h]):
                at, src = (b.lists[i][j // 16], h, j % 16), (b.lists[i][t // 16], h, t % 16)
                assert np.array_equal(k1[at], k0[src]) and w1[at] == w0[src], (i, h, j)
    assert host(before).tolist() == b.kv


def test_shared_pages_are_read_only_when_moved_elsewhere():
    """Two sequences over the same pages, evicted into pages of their own."""
    rng = np.random.default_rng(1)
    b = Batch([(90, 0), (30, 0), (30, 0)], 16, rng)
    ref = new_cache(b, 16, 2, 64, 8, True)
    fill(ref, b, rng)
    w = np.abs(rng.standard_normal(ref.k_scales.shape)).astype(np.float32)
    gpu, wg = to_gpu(ref), dev(w)
    table = _i32([b.lists[0], b.lists[0]])
    to = _i32([b.lists[1], b.lists[2]])
    say("evict, shared")
    lens = _i32([90, 70])
    got, kept = bg.kv_cache_evict(gpu, wg, table, lens, 30, 4, to_table=to, new_lens=lens)
    assert got is lens and host(lens).tolist() == [30, 30]
    want_kept, _ = serving.evict(ref, w, [b.lists[0]] * 2, [90, 70], 30, 4, b.lists[1:])
    assert_same_bits(host(kept), want_kept, "kept")
    for n in ("k_codes", "k_scales", "v_scales"):
        assert_same_bits(host(getattr(gpu, n))[b.lists[0]], getattr(ref, n)[b.lists[0]], n)


@pytest.mark.parametrize("bits,sym", FORMATS)
def test_some_pages_stay_in_their_place(bits, sym):
    """to_table with fresh pages beside some of the sequence's own: batches of
    tokens are then moved in order, beside a sequence that moves altogether."""
    rng = np.random.default_rng(bits)
    page, keep = 16, 4000
    b = Batch([(9000, 0), (5000, 0), (keep, 0), (keep, 0)], page, rng)
    ref = new_cache(b, page, 2, 64, bits, sym)
    for t in (ref.k_codes, ref.v_codes):
        t[:] = rng.integers(0, 256, t.shape, dtype=np.uint8)
    for t in (ref.k_scales, ref.v_scales, ref.k_zeros, ref.v_zeros):
        if t is not None:
            t[:] = rng.random(t.shape, dtype=np.float32)
    w = _weights(ref, rng)
    mixed = [old if i % 3 else new for i, (old, new) in enumerate(zip(b.lists[0], b.lists[2]))]
    to = [mixed, b.lists[3]]
    gpu, wg = to_gpu(ref), dev(w)
    say(f"evict, some pages stay, bits={bits} sym={sym}")
    table = dev(np.ascontiguousarray(b.table[:2]))
    lens, kept = bg.kv_cache_evict(gpu, wg, table, _i32([9000, 5000]), keep, 100, to_table=_i32(to))
    want_kept, want_lens = serving.evict(ref, w, b.lists[:2], [9000, 5000], keep, 100, to)
    assert host(lens).tolist() == want_lens
    assert_same_bits(host(kept), want_kept, "kept")
    want = _state(ref, w)
    for name in want:
        got = host(wg if name == "weights" else getattr(gpu, name))
        for pages in to:
            assert np.array_equal(got[pages], want[name][pages], equal_nan=True), name


def test_graph_of_a_decode_step_with_eviction():
    """Write, attention, weigh and evict captured once and replayed while lengths
    grow and shrink in device memory: every replay gives the eager calls' bits."""
    rng = np.random.default_rng(6)
    b = Batch([(64, 1), (40, 1), (80, 1)], 16, rng, wide=8)
    ref = new_cache(b, 16, 2, 64, 8, True)
    fill(ref, b, rng)
    q, k, v = torch.randn((b.rows, 4, 64), device="cuda").bfloat16(), *torch.randn((2, b.rows, 2, 64), device="cuda")
    table, lens0, starts = b.on_gpu()
    w0 = dev(_weights(ref, rng))

    def step(c, w, lens, lse, out, kept):
        bg.kv_cache_write(k, v, c, table, lens, starts, max_rows=1)
        bg.paged_attention(q, c, table, lens, starts, max_rows=1, lse=lse, out=out)
        bg.kv_cache_weigh(q, lse, c, w, table, lens, starts, max_rows=1)
        bg.kv_cache_evict(c, w, table, lens, 40, 8, kept=kept, new_lens=lens)
        lens += 1

    def fresh():
        return [to_gpu(ref), w0.clone(), lens0.clone(), torch.empty((b.rows, 4), device="cuda"), torch.empty_like(q),
                torch.empty((3, 2, 40), dtype=torch.int32, device="cuda")]

    eager, graph = fresh(), fresh()
    step(*fresh())
    torch.cuda.synchronize()
    say("graph of a decode step")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*graph)
    for i in range(4):
        step(*eager)
        g.replay()
        torch.cuda.synchronize()
        for a, x in zip(eager[1:], graph[1:]):
            assert torch.equal(a, x), i
    assert host(eager[2]).tolist() == [41, 41, 41]


@pytest.mark.parametrize("d,bits,sym", [(64, 4, True), (128, 8, False), (256, 8, True)])
def test_guard(d, bits, sym):
    """Weights, kept positions, lengths and the pool between canaries."""
    lib, rng = bg.load_library(), np.random.default_rng(d)
    b = Batch([(300, 1), (37, 30), (1, 1), (90, 1)], 16, rng, spare=0)
    row, meta = d * bits // 8, (b.pages, 2, 16)
    g = {"k_codes": Guarded((*meta, row), torch.uint8), "v_codes": Guarded((b.pages, 2, 4, row, 4), torch.uint8)}
    for n in ("k_scales", "v_scales") + (() if sym else ("k_zeros", "v_zeros")):
        g[n] = Guarded(meta, torch.float32)
    z = lambda n: g[n].t if n in g else None  # noqa: E731
    c = bg.KVCache(g["k_codes"].t, g["v_codes"].t, g["k_scales"].t, g["v_scales"].t, z("k_zeros"), z("v_zeros"), d, bits)
    for t in g.values():
        t.t.fill_(1)
    q, lse = torch.randn((b.rows, 6, d), device="cuda").bfloat16(), torch.zeros((b.rows, 6), device="cuda")
    table, lens, starts = b.on_gpu()
    for mr, mk in ((0, 0), (30, 300), (1, 300), (1, 1), (30, 1 << 20)):
        w = Guarded(meta, torch.float32)
        w.t.zero_()
        say(f"guard kv_cache_weigh D={d} {mr, mk}")
        need = bg.kv_cache_weigh_workspace(b.rows, 6, c, 4, table.shape[1], mr, mk)
        ws = Guarded((max(need, 256),), torch.uint8)
        for causal in (1, 0):
            _ok(lib.kv_cache_weigh(c._ref, _p(q), b.rows, 6, 6 * d, ctypes.c_float(d ** -0.5), _p(lse), _p(table),
                                   table.shape[1], _p(lens), _p(starts), 4, causal, mr, mk, w.ptr(), w.ptr(), ws.ptr(), need,
                                   _st()), "weigh")
        w.check("weights")
        ws.check("workspace")
    kept, new = Guarded((4, 2, 77), torch.int32), Guarded((4,), torch.int32)
    say(f"guard kv_cache_evict D={d}")
    _ok(lib.kv_cache_evict(c._ref, w.ptr(), _p(table), table.shape[1], _p(lens), 4, 77, 9, None, 0, 0, kept.ptr(), new.ptr(),
                           _st()), "evict")
    for t, n in [(w, "weights"), (kept, "kept"), (new, "new_lens")] + [(t, n) for n, t in g.items()]:
        t.check(n)


def test_two_streams_at_once():
    """Equal calls on two streams over one cache, each with weights of its own."""
    rng = np.random.default_rng(8)
    b = Batch([(900, 1), (70, 70), (300, 9)], 16, rng)
    ref = new_cache(b, 16, 2, 64, 4, False)
    fill(ref, b, rng)
    gpu, q = to_gpu(ref), torch.randn((b.rows, 8, 64), device="cuda").bfloat16()
    lse, batch = torch.zeros((b.rows, 8), device="cuda"), b.on_gpu()
    want = [bg.kv_cache_weigh(q, lse, gpu, None, *batch, max_rows=n) for n in (0, 1)]
    torch.cuda.synchronize()
    say("two streams")
    got = []
    for st in [torch.cuda.Stream() for _ in range(2)]:
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got += [[bg.kv_cache_weigh(q, lse, gpu, None, *batch, max_rows=n) for n in (0, 1)] for _ in range(4)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(x, y) for x, y in zip(g, want))


def test_a_server_with_shared_prefixes_and_a_budget():
    """Prompts behind a shared prefix, then decode steps: cache writes, attention
    over prefix and own tokens, weights of both, eviction of the own ones to a
    budget; every step's attention and weights against the oracle on the step's
    own cache."""
    rng = np.random.default_rng(7)
    page, heads, group, d, keep, recent = 16, 2, 4, 64, 24, 6
    n, prefix, room = 3, 50, 64
    b = Batch([(room, 0)] * n + [(prefix, 0)], page, rng)
    ref = new_cache(b, page, heads, d, 8, False)
    for t in range(prefix):
        for side in "kv":
            ref.put_rows(b.lists[n][t // page], t % page, side, rng.standard_normal((heads, d)))
    gpu, lists = to_gpu(ref), b.lists[:n]
    table = dev(b.table)
    pre = (table[n:].contiguous(), _i32([prefix]))
    own = table[:n].contiguous()
    w_ref = np.zeros(ref.k_scales.shape, np.float32)
    wg, held = dev(w_ref), [0] * n
    for step in range(4):
        new = [20, 9, 31] if step == 0 else [1, 1, 1] if step < 3 else [5, 1, 2]
        held = [a + x for a, x in zip(held, new)]
        starts = [0] + np.cumsum(new).tolist()
        rows = starts[-1]
        k, v = rng.standard_normal((2, rows, heads, d)).astype(np.float32)
        q = bf16(rng.standard_normal((rows, heads * group, d)))
        sets = []
        for i in range(n):
            for x in range(new[i]):
                pos = held[i] - new[i] + x
                ref.put_rows(lists[i][pos // page], pos % page, "k", k[starts[i] + x])
                ref.put_rows(lists[i][pos // page], pos % page, "v", v[starts[i] + x])
                sets.append([(b.lists[n], prefix), (lists[i], pos + 1)])
        batch, whole = (own, _i32(held), _i32(starts)), _i32([0, rows])
        say(f"server step {step}: {held}")
        bg.kv_cache_write(dev(k), dev(v), gpu, *batch)
        lse = torch.empty((rows, heads * group), device="cuda")
        out = bg.prefix_attention(dev_bf16f(q), gpu, *pre, whole, *batch, lse=lse)
        want, wl, bound = serving.attention_over(q, ref, sets, d ** -0.5)
        check_attention(out, lse, want, wl, bound, f"step {step}")
        before = host(wg)
        bg.kv_cache_weigh(dev_bf16f(q), lse, gpu, wg, *batch)
        bg.kv_cache_weigh(dev_bf16f(q), lse, gpu, wg, *pre, whole, causal=False)
        lse = host(lse)
        a, ba = serving.weigh(q, lse, ref, before, lists, held, starts, d ** -0.5)
        p, bp = serving.weigh(q, lse, ref, before, [b.lists[n]], [prefix], [0, rows], d ** -0.5, causal=False)
        _check_weights(wg, before, np.where(ba > 0, a, p), ba + bp, f"weights {step}")
        w_ref = host(wg).copy()
        lens, kept = bg.kv_cache_evict(gpu, wg, own, batch[1], keep, recent)
        want_kept, held = serving.evict(ref, w_ref, lists, held, keep, recent)
        assert host(lens).tolist() == held
        assert_same_bits(host(kept), want_kept, "kept")
        for i in range(n):
            for j in range(held[i]):
                at = lists[i][j // page], slice(None), j % page
                assert np.array_equal(host(gpu.k_codes)[at], ref.k_codes[at]) and host(wg)[at].tolist() == w_ref[at].tolist()

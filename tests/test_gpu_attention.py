"""paged_attention against the oracle in 64 bits, each element within a bound
derived from the stated arithmetic (oracle.serving.attention)."""
import numpy as np
import pytest
import torch

import bit_gemv_amd as bg
from gpu_helpers import dev, say
from oracle import serving
from serving_helpers import Batch, bf16, check_attention, dev_bf16f, fill, new_cache, to_gpu

pytestmark = pytest.mark.gpu

FORMATS = [(4, False), (4, True), (8, False), (8, True)]
# tokens held, new rows: one token, single tokens of odd contexts, whole
# prompts, chunks, rows without any token to see, no rows, no tokens
SEQS = [(1, 1), (17, 1), (16, 16), (33, 5), (70, 70), (261, 3), (3, 6), (0, 2), (40, 0), (129, 1)]


def _run(seqs, d, bits, sym, page=16, heads=2, group=4, seed=0, q_scale=1.0, k_scale=1.0, v_scale=1.0, gap=0, lead=0,
         scale=None, hints=((0, 0),), what="", room=0):
    rng = np.random.default_rng(seed)
    b = Batch(seqs, page, rng, lead=lead, wide=room // page)
    ref = new_cache(b, page, heads, d, bits, sym)
    fill(ref, b, rng, k_scale, v_scale)
    gpu = to_gpu(ref)
    rows, qh = b.rows + 1, heads * group
    q = bf16(rng.standard_normal((rows, qh, d)) * q_scale)
    wide = torch.full((rows, qh + gap, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :qh] = dev_bf16f(q)
    want, want_lse, bound = serving.attention(q, ref, b.lists, b.kv, b.starts, d ** -0.5 if scale is None else scale)
    mine = [r for r, _, _ in b.positions()]
    for max_rows, max_kv in hints:
        say(f"paged_attention {what} D={d} bits={bits} sym={sym} page={page} heads={heads} group={group} rows={b.rows} "
            f"hints {max_rows} {max_kv}")
        out = torch.full((rows, qh, d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((rows, qh), 7.0, device="cuda")
        bg.paged_attention(wide[:, :qh], gpu, *b.on_gpu(), scale=scale, max_rows=max_rows, max_kv=max_kv, out=out, lse=lse)
        check_attention(out, lse, want, want_lse, bound, what, mine)
        rest = [r for r in range(rows) if r not in mine]
        assert bool((out[rest] == 7.0).all()) and bool((lse[rest] == 7.0).all()), "rows of no sequence changed"
    return out


@pytest.mark.parametrize("bits,sym", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_formats(d, bits, sym):
    # bounds that choose each kernel: 256, 128, 16 and 8 rows a tile
    _run(SEQS, d, bits, sym, seed=d + bits, hints=((0, 0), (20, 0), (4, 261), (2, 0)))


@pytest.mark.parametrize("bits,sym", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_formats_cut_into_spans(d, bits, sym):
    """A table wide enough for long contexts: every kernel cuts its work into
    spans and joins the parts."""
    seqs = [(40, 40), (300, 70), (3, 6), (0, 2), (500, 33), (40, 0)]
    _run(seqs, d, bits, sym, seed=d + bits + 2, room=8192, hints=((70, 0), (4, 0), (2, 0)))
    _run([(300, 200)], d, bits, sym, heads=1, group=8, seed=d + bits + 3, room=8192)


@pytest.mark.parametrize("bits,sym", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_single_tokens(d, bits, sym):
    """A decode batch: the single-token form, split and whole."""
    _run([(1, 1), (2, 1), (31, 1), (32, 1), (33, 1), (128, 1), (300, 1), (16, 1)], d, bits, sym, seed=d + bits + 1,
         hints=((1, 300), (1, 0), (0, 0)))


@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 16, 20, 33])
@pytest.mark.parametrize("bits,sym", [(4, False), (8, True)])
def test_head_layouts(group, bits, sym):
    _run([(37, 1), (50, 11), (20, 20)], 64, bits, sym, heads=1 if group > 8 else 3, group=group, seed=group)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("bits,sym", [(4, True), (8, False)])
def test_pages(page, bits, sym):
    _run([(300, 1), (270, 18), (257, 257), (5, 2)], 64, bits, sym, page=page, heads=1, group=2, seed=page)


@pytest.mark.parametrize("bits,sym", [(4, False), (8, True)])
def test_hints_change_nothing_that_counts(bits, sym):
    """Bounds that are exact, loose, unknown or too small."""
    _run(SEQS, 128, bits, sym, seed=21, hints=((70, 261), (1, 1), (3, 50), (1 << 20, 1 << 20), (0, 17), (2, 0)))


@pytest.mark.parametrize("held", [1, 127, 128, 129, 1000, 8191])
@pytest.mark.parametrize("bits,sym", [(4, False), (8, True)])
def test_long_single_sequence(held, bits, sym):
    """One row over many splits, odd ends."""
    _run([(held, 1)], 64, bits, sym, page=32, heads=1, group=2, seed=held)


def test_long_chunk():
    _run([(1500, 130), (900, 64)], 128, 8, True, page=64, heads=1, group=2, seed=5)
    _run([(1500, 130), (900, 64)], 128, 4, False, page=16, heads=1, group=2, seed=6)


@pytest.mark.parametrize("bits,sym", FORMATS)
@pytest.mark.parametrize("group", [1, 4, 5])
def test_single_tokens_beside_a_chunk(bits, sym, group):
    """A batch whose single tokens go to a launch of their own, whole and split."""
    seqs = [(150, 100)] + [(n, 1) for n in (1, 40, 257, 600, 33)] + [(9, 9), (3, 4)]
    _run(seqs, 64, bits, sym, heads=2, group=group, seed=group, hints=((100, 600), (100, 5000)))
    _run(seqs, 64, bits, sym, page=256, heads=1, group=group, seed=group, hints=((100, 0),))


def test_rows_apart_and_leading_rows():
    _run(SEQS, 128, 8, True, seed=7, gap=5, lead=3)


@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0, 1e-4])
def test_scale(scale):
    _run([(33, 5), (200, 1)], 64, 8, True, seed=8, scale=scale)


def test_sharp_and_flat_softmax():
    """Scores far apart (one key takes all) and all alike."""
    _run([(300, 2), (90, 40)], 128, 8, True, seed=9, q_scale=8.0)
    _run([(300, 2), (90, 40)], 128, 4, False, seed=9, q_scale=8.0)
    _run([(300, 2), (90, 40)], 128, 8, False, seed=9, q_scale=1e-3)


def test_rising_scores():
    """The running maximum is raised again and again along the context."""
    _run([(600, 2), (600, 33)], 64, 8, True, seed=10, k_scale=lambda i, t: 0.1 + t / 60, q_scale=3.0)


@pytest.mark.parametrize("bits,sym", FORMATS)
def test_uneven_value_scales(bits, sym):
    """Value scales that grow, shrink and jump by many powers of two."""
    for f in (lambda i, t: 2.0 ** (t / 20), lambda i, t: 2.0 ** (-t / 20), lambda i, t: 2.0 ** ((t * 7) % 23 - 11)):
        _run([(300, 1), (200, 20)], 64, bits, sym, seed=11, v_scale=f)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_zeros_far_from_the_codes(bits, d):
    """Keys and values far from zero for their range (zeros of thousands), all
    alike (zeros of 1e8 and more) and on one side, among ordinary ones."""
    rng = np.random.default_rng(20)
    b = Batch([(200, 40), (90, 3), (70, 1)], 16, rng, wide=512)
    ref = new_cache(b, 16, 1, d, bits, False)
    fill(ref, b, rng)
    for i, (held, every) in enumerate(((200, 5), (90, 1), (70, 33))):
        for t in range(0, held, every):
            at = b.lists[i][t // 16], t % 16
            kind = (t // every) % 4
            for side in "kv":
                x = (5 + 0.01 * rng.standard_normal((1, d)), np.full((1, d), 0.03125), -7 - rng.random((1, d)),
                     rng.standard_normal((1, d)))[kind]
                ref.put_rows(*at, side, x)
    q = bf16(0.2 * rng.standard_normal((44, 5, d)))
    want, wl, bound = serving.attention(q, ref, b.lists, b.kv, b.starts, d ** -0.5)
    for hints in ((0, 0), (40, 500), (40, 5000), (3, 5000), (1, 5000)):
        say(f"paged_attention far zeros bits={bits} d={d} hints {hints}")
        out = bg.paged_attention(dev_bf16f(q), to_gpu(ref), *b.on_gpu(), max_rows=hints[0], max_kv=hints[1])
        check_attention(out, None, want, wl, bound, f"far zeros {hints}")


@pytest.mark.parametrize("q_scale,k_scale", [(1e-30, 1.0), (1e30, 1e-30), (1e-5, 1e5), (1e18, 1e-18)])
def test_magnitudes_of_q(q_scale, k_scale):
    """q far outside fp16's range, tiny or huge."""
    # key scales have a floor of 1e-8 / 127: below it a key is all zeros
    _run([(90, 3), (40, 1)], 64, 8, True, seed=12, q_scale=q_scale, k_scale=k_scale)


def test_heads_of_different_size_in_one_tile():
    """Rows of one 16-row tile whose q differ by 2^14: each within its own
    bound, as the power of two that scales q is the row's own."""
    rng = np.random.default_rng(13)
    b = Batch([(64, 1)], 16, rng)
    ref = new_cache(b, 16, 1, 64, 8, True)
    fill(ref, b, rng)
    q = bf16(rng.standard_normal((1, 8, 64)) * np.float32(2.0) ** (-2 * np.arange(8))[None, :, None])
    want, wl, bound = serving.attention(q, ref, b.lists, b.kv, b.starts, 0.125)
    say("paged_attention uneven heads")
    out = bg.paged_attention(dev_bf16f(q), to_gpu(ref), *b.on_gpu())
    check_attention(out, None, want, wl, bound, "uneven heads")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("bits,sym", [(4, False), (8, True)])
def test_a_row_that_is_not_finite_changes_no_other(bad, bits, sym):
    """In tiles of 8, 16 and 128 rows, whole and in parts; a NaN reaches its
    row's result, split or not."""
    rng = np.random.default_rng(19)
    b = Batch([(700, 3), (40, 30), (9, 1)], 16, rng, wide=512)
    ref = new_cache(b, 16, 1, 64, bits, sym)
    fill(ref, b, rng)
    q = bf16(rng.standard_normal((34, 4, 64)))
    want, wl, bound = serving.attention(q, ref, b.lists, b.kv, b.starts, 0.125)
    hit = [(0, 1), (2, 3), (7, 0), (33, 2)]
    gq = dev_bf16f(q)
    for i, (r, h) in enumerate(hit):
        gq[r, h, 5 * i] = bad
    keep = np.ones((34, 4), bool)
    keep[tuple(np.array(hit).T)] = False
    for hints in ((0, 0), (30, 700), (30, 5000), (3, 5000), (2, 5000), (2, 700)):
        say(f"paged_attention q {bad} bits={bits} hints {hints}")
        lse = torch.empty((34, 4), device="cuda")
        out = bg.paged_attention(gq, to_gpu(ref), *b.on_gpu(), max_rows=hints[0], max_kv=hints[1], lse=lse)
        k = torch.from_numpy(keep).cuda()
        check_attention(out[k], lse[k], want[keep], wl[keep], bound[keep], f"{bad} {hints}")
        if bad != bad:
            assert bool(out[~k].isnan().all()) and bool(lse[~k].isnan().all())


def test_pages_outside_the_pool_are_not_attended_to():
    rng = np.random.default_rng(14)
    b = Batch([(80, 1), (80, 20)], 16, rng)
    ref = new_cache(b, 16, 1, 64, 8, True)
    fill(ref, b, rng)
    q = bf16(rng.standard_normal((21, 2, 64)))
    for bad in (-1, b.pages, (1 << 31) - 1, -(1 << 31)):
        table = b.table.copy()
        table[0, 2] = table[1, 0] = bad
        say(f"paged_attention page {bad}")
        out = bg.paged_attention(dev_bf16f(q), to_gpu(ref), dev(table), *b.on_gpu()[1:])
        want = np.zeros((21, 2, 64))
        for r, i, pos in b.positions():
            keep = [t for t in range(pos + 1) if table[i, t // 16] != bad]
            qk, sk, zk = ref.parts(b.lists[i], 0, "k", 80)
            qv, sv, zv = ref.parts(b.lists[i], 0, "v", 80)
            k, v = ((qk - 128) * sk[:, None])[keep], ((qv - 128) * sv[:, None])[keep]
            for h in range(2):
                p = np.exp(0.125 * (k @ q[r, h].astype(np.float64)))
                want[r, h] = p @ v / p.sum()
        err = np.abs(out.float().cpu().numpy() - want)
        # the bound's leading terms; values are at most about 5
        assert err.max() <= 2.0 ** -8 * np.abs(want).max() + 2.0 ** -10 * 5, err.max()


def test_odd_lengths_and_starts_touch_nothing_outside():
    rng = np.random.default_rng(15)
    b = Batch([(30, 5), (9, 4)], 16, rng)
    ref = new_cache(b, 16, 1, 64, 8, True)
    fill(ref, b, rng)
    gpu, q = to_gpu(ref), dev_bf16f(rng.standard_normal((9, 2, 64)))
    for kv, starts in (([1 << 30, 9], [0, 5, 9]), ([-5, 9], [0, 5, 9]), ([30, 9], [-7, 5, 9]), ([30, 9], [0, 5, 1 << 30]),
                       ([30, 9], [9, 5, 0])):
        say(f"paged_attention kv={kv} starts={starts}")
        bg.paged_attention(q, gpu, b.on_gpu()[0], dev(np.asarray(kv, np.int32)), dev(np.asarray(starts, np.int32)))
    torch.cuda.synchronize()


def test_shared_prefix_pages():
    """Two sequences over the same first pages, the second with more."""
    rng = np.random.default_rng(17)
    b = Batch([(32, 1), (50, 1)], 16, rng)
    ref = new_cache(b, 16, 1, 64, 8, True)
    fill(ref, b, rng)
    b.lists[0] = b.lists[1][:2]
    b.table[0, :2] = b.lists[0]
    q = bf16(rng.standard_normal((2, 4, 64)))
    want, wl, bound = serving.attention(q, ref, b.lists, b.kv, b.starts, 0.125)
    say("paged_attention shared prefix")
    check_attention(bg.paged_attention(dev_bf16f(q), to_gpu(ref), *b.on_gpu()), None, want, wl, bound, "shared prefix")


@pytest.mark.parametrize("single", [True, False])
def test_many_sequences(single):
    """Past 64 sequences the sharing-out adds them up in several rounds."""
    seqs = [(1 + (i * 37) % 90, 1 if single else 1 + (i % 3) * 7) for i in range(150)]
    _run(seqs, 64, 4, True, heads=1, group=2, seed=18, hints=((0, 0), (15, 90), (15, 4000), (1, 4000)))


def test_empty_calls():
    gpu = bg.KVCache.empty(2, 16, 1, 64)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    none = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert bg.paged_attention(none, gpu, z(0, 1), z(0), z(1)).shape == (0, 4, 64)
    assert bg.paged_attention(none, gpu, z(2, 1), z(2), z(3)).shape == (0, 4, 64)
    one = torch.ones((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    starts = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    assert float(bg.paged_attention(one, gpu, z(1, 0), z(1), starts).abs().max()) == 0   # a table without pages


def test_equal_calls_give_equal_bits():
    rng = np.random.default_rng(16)
    b = Batch([(3000, 1), (100, 40)], 16, rng)
    ref = new_cache(b, 16, 1, 64, 4, False)
    fill(ref, b, rng)
    gpu, q = to_gpu(ref), dev_bf16f(rng.standard_normal((41, 4, 64)))
    say("paged_attention repeated")
    outs = [bg.paged_attention(q, gpu, *b.on_gpu()) for _ in range(4)]
    assert all(torch.equal(outs[0], o) for o in outs[1:])

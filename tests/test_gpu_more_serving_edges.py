"""What the calls beside paged attention do with pages outside the pool, with
lengths and starts that no batch should have, and with rows of 128 and 256 code
bytes over several batches of an eviction. Every result against the oracle,
outputs of the former between canaries."""
import numpy as np
import pytest
import torch

import bit_gemv_amd as bg
from gpu_helpers import assert_same_bits, dev, host, say
from oracle import serving
from serving_helpers import Batch, bf16, check_attention, dev_bf16f, fill, new_cache, to_gpu
from test_gpu_guard import Guarded
from test_gpu_weigh_evict import FORMATS, _check_weights, _evict, _i32, _state, _weights

pytestmark = pytest.mark.gpu

BAD = [-1, 1 << 20, (1 << 31) - 1, -(1 << 31)]
# 12 heads a group: the kernels for few rows are reached by wrong bounds only.
# Bounds and a table's width that choose each form of the weights: rows shared by
# blocks, not shared, keys past 16 rows.
WEIGH_FORMS = [((0, 0), 0), ((20, 0), 2048), ((1, 0), 0), ((1, 17), 2048)]
# and of attention: 128 rows a tile in whole units and in spans, 16, a wrong length
ATTN_FORMS = [((0, 0), 0), ((5, 0), 4096), ((1, 0), 4096), ((1, 17), 0)]


def _case(seqs, rng, d=64, bits=8, sym=True, heads=1, group=12, wide=0):
    b = Batch(seqs, 16, rng, wide=wide // 16)
    ref = new_cache(b, 16, heads, d, bits, sym)
    fill(ref, b, rng)
    return b, ref, bf16(rng.standard_normal((b.rows, heads * group, d)))


def _run_weigh(q, lse, gpu, w, table, kv, starts, hints, causal):
    """weights between canaries, the call's workspace as well"""
    out = Guarded(w.shape, torch.float32)
    out.t.copy_(dev(w))
    rows, qh, _ = q.shape
    need = bg.kv_cache_weigh_workspace(rows, qh, gpu, len(kv), table.shape[1], *hints)
    ws = Guarded((max(need, 256),), torch.uint8)
    say(f"kv_cache_weigh kv={kv} starts={starts} hints={hints} causal={causal}")
    bg.kv_cache_weigh(dev_bf16f(q), dev(lse), gpu, out.t, dev(table), _i32(kv), _i32(starts), scale=0.125, causal=causal,
                      max_rows=hints[0], max_kv=hints[1], workspace=ws.t)
    out.check("weights")
    ws.check("workspace")
    return out.t


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hints,wide", WEIGH_FORMS)
def test_weights_of_pages_outside_the_pool(hints, wide, causal):
    """Their tokens have no slot; every other token's weight is what it was, as
    a weight depends on its own key and the row's log-sum alone."""
    rng = np.random.default_rng(31)
    b, ref, q = _case([(80, 1), (200, 20), (40, 3)], rng, bits=4, sym=False, wide=wide)
    gpu, w = to_gpu(ref), _weights(ref, rng)
    lse = rng.standard_normal(q.shape[:2]).astype(np.float32) + 6
    want, bound = serving.weigh(q, lse, ref, w, b.lists, b.kv, b.starts, 0.125, causal)
    gone = [(0, 2), (1, 0), (1, 5), (1, 12), (2, 2)]
    for seq, i in gone:
        page = b.lists[seq][i]
        want[page], bound[page] = w[page], 0
    for bad in BAD + [b.pages]:
        table = b.table.copy()
        for seq, i in gone:
            table[seq, i] = bad
        got = _run_weigh(q, lse, gpu, w, table, b.kv, b.starts, hints, causal)
        _check_weights(got, w, want, bound, f"page {bad} hints {hints}")


# kv_lens, row_starts, and of each of two sequences that hold 32 and 16 tokens and
# have 5 and 4 rows what a causal call sees: its "own" positions, "all" that the
# table holds, "none" of it, or (no rows) "left"
ODD = [([1 << 30, 16], [0, 5, 9], ["all", "own"]), ([(1 << 31) - 1, 16], [0, 5, 9], ["all", "own"]),
       ([-5, 16], [0, 5, 9], ["none", "own"]), ([-(1 << 31), 16], [0, 5, 9], ["none", "own"]),
       ([32, 16], [-7, 5, 9], ["own", "own"]), ([32, 16], [0, 5, 1 << 30], ["own", "none"]),
       ([32, 16], [9, 5, 0], ["left", "left"]), ([32, 16], [-(1 << 31), -3, 0], ["left", "left"])]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hints,wide", WEIGH_FORMS)
def test_weights_of_odd_lengths_and_starts(hints, wide, causal):
    rng = np.random.default_rng(32)
    b, ref, q = _case([(32, 5), (16, 4)], rng, wide=wide)
    gpu, w = to_gpu(ref), _weights(ref, rng)
    lse = rng.standard_normal(q.shape[:2]).astype(np.float32) + 4
    own = {c: serving.weigh(q, lse, ref, w, b.lists, b.kv, b.starts, 0.125, c) for c in (True, False)}
    for kv, starts, kinds in ODD:
        want, bound = w.astype(np.float64), np.zeros(w.shape)
        for i, kind in enumerate(kinds):
            if kind == "left" or kv[i] <= 0:
                continue
            at = b.lists[i]
            if causal and kind == "none":             # tokens of rows that stand before the first position:
                want[at], bound[at] = 0, 1e-30        # their weights start from 0, and no row sees them
            else:
                source = own[causal and kind == "own"]
                want[at], bound[at] = source[0][at], source[1][at]
        got = _run_weigh(q, lse, gpu, w, b.table, kv, starts, hints, causal)
        _check_weights(got, w, want, bound, f"kv {kv} starts {starts} hints {hints}")


def _pieces(ref, pages, n):
    """n tokens of a list of pages as sets of attention_over, pages that are not
    in the pool left out"""
    return [([p], min(16, n - 16 * i)) for i, p in enumerate(pages) if 0 <= p < len(ref.k_scales) and n > 16 * i]


def _run_attention(q, ref, sets, need, call, what):
    """One call between canaries; rows whose set is None stay as they were."""
    rows, qh, d = q.shape
    want, wl, bound = serving.attention_over(q, ref, sets, 0.125)
    ws, out, lse = Guarded((max(need, 256),), torch.uint8), Guarded(q.shape, torch.bfloat16), Guarded((rows, qh), torch.float32)
    out.t.fill_(7.0)
    lse.t.fill_(7.0)
    say(what)
    call(dev_bf16f(q), workspace=ws.t, out=out.t, lse=lse.t, scale=0.125)
    for t, n in ((ws, "workspace"), (out, "out"), (lse, "lse")):
        t.check(n)
    mine, rest = ([r for r in range(rows) if (sets[r] is None) == left] for left in (False, True))
    check_attention(out.t, lse.t, want, wl, bound, what, mine)
    assert bool((out.t[rest] == 7.0).all()) and bool((lse.t[rest] == 7.0).all()), what


def _cross(b, gpu, q, ref, table, kv, starts, sets, hints):
    need = bg.cross_attention_workspace(len(q), q.shape[1], gpu, len(kv), table.shape[1], *hints)
    _run_attention(q, ref, sets, need, lambda x, **a: bg.cross_attention(
        x, gpu, dev(table), _i32(kv), _i32(starts), max_rows=hints[0], max_kv=hints[1], **a),
        f"cross_attention kv={kv} starts={starts} hints={hints}")


def _prefix(gpu, q, ref, prefix, batch, sets, hints, bounds=(0, 0)):
    (pt, pl, ps), (table, kv, starts) = prefix, batch
    need = bg.prefix_attention_workspace(len(q), q.shape[1], gpu, len(pl), pt.shape[1], len(kv), table.shape[1], *bounds, *hints)
    _run_attention(q, ref, sets, need, lambda x, **a: bg.prefix_attention(
        x, gpu, dev(pt), _i32(pl), _i32(ps), dev(table), _i32(kv), _i32(starts), max_prefix_rows=bounds[0],
        max_prefix=bounds[1], max_rows=hints[0], max_kv=hints[1], **a),
        f"prefix_attention prefix {pl, ps} kv={kv} starts={starts} hints={hints} {bounds}")


@pytest.mark.parametrize("bits,sym", [(4, False), (8, True)])
@pytest.mark.parametrize("hints,wide", ATTN_FORMS)
def test_cross_attention_passes_over_pages_outside_the_pool(hints, wide, bits, sym):
    rng = np.random.default_rng(33)
    b, ref, q = _case([(80, 1), (75, 20), (16, 2)], rng, bits=bits, sym=sym, wide=wide)
    gpu = to_gpu(ref)
    for bad in BAD:
        table = b.table.copy()
        table[0, 2] = table[1, 0] = table[1, 4] = table[2, 0] = bad
        sets = [None] * b.rows
        for r, i, _ in b.positions():
            sets[r] = _pieces(ref, table[i], b.kv[i])
        _cross(b, gpu, q, ref, table, b.kv, b.starts, sets, hints)


@pytest.mark.parametrize("hints,wide", ATTN_FORMS)
def test_cross_attention_of_odd_lengths_and_starts(hints, wide):
    """Rows that see everything see it wherever they stand; rows of no tokens are
    zeros, rows of no sequence are left alone."""
    rng = np.random.default_rng(34)
    b, ref, q = _case([(32, 5), (16, 4)], rng, wide=wide)
    gpu = to_gpu(ref)
    for kv, starts, kinds in ODD:
        sets = [None] * 9
        for i, kind in enumerate(kinds):
            for r in range(b.starts[i], b.starts[i + 1]):
                if kind != "left":
                    sets[r] = [(b.lists[i], b.kv[i])] if kv[i] > 0 else []
        _cross(b, gpu, q, ref, b.table, kv, starts, sets, hints)


@pytest.mark.parametrize("hints,wide", ATTN_FORMS)
@pytest.mark.parametrize("bounds", [(0, 0), (1, 17)])
def test_prefix_attention_passes_over_pages_outside_the_pool(hints, wide, bounds):
    rng = np.random.default_rng(35)
    b, ref, q = _case([(80, 1), (75, 20), (30, 3), (100, 0), (40, 0)], rng, wide=wide)
    gpu = to_gpu(ref)
    for bad in BAD:
        table = b.table.copy()
        for i, j in ((0, 2), (1, 0), (1, 4), (2, 0), (2, 1), (3, 0), (3, 6), (4, 1)):
            table[i, j] = bad
        sets = [None] * b.rows
        for r, i, pos in b.positions():
            sets[r] = _pieces(ref, table[3 if i < 2 else 4], 100 if i < 2 else 40) + _pieces(ref, table[i], pos + 1)
        prefix = table[3:], [100, 40], [0, b.starts[2], b.starts[3]]
        _prefix(gpu, q, ref, prefix, (table[:3], b.kv[:3], b.starts[:4]), sets, hints, bounds)


@pytest.mark.parametrize("hints,wide", ATTN_FORMS)
def test_prefix_attention_of_odd_lengths_and_starts(hints, wide):
    """Of the own tokens, and of the prefix: its tokens cut to its table, none of
    them, and rows that no prefix has."""
    rng = np.random.default_rng(36)
    b, ref, q = _case([(32, 5), (16, 4), (48, 0), (32, 0)], rng, wide=wide)
    gpu = to_gpu(ref)
    pos = {r: (i, p) for r, i, p in b.positions()}

    def own(r, kind):
        i, p = pos[r]
        return {"own": [(b.lists[i], p + 1)], "all": [(b.lists[i], b.kv[i])], "none": []}[kind]

    front = [[(b.lists[2], 48)], [(b.lists[3], 32)]]
    for kv, starts, kinds in ODD:
        sets = [None if kinds[i] == "left" else front[i] + own(r, kinds[i]) for r, (i, _) in sorted(pos.items())]
        prefix = np.ascontiguousarray(b.table[2:]), [48, 32], [0, 5, 9]
        _prefix(gpu, q, ref, prefix, (b.table[:2], kv, starts), sets, hints)
    for pl, ps, has in (([1 << 30, 32], [0, 5, 9], (1, 1)), ([-5, 32], [0, 5, 9], (0, 1)), ([-(1 << 31), 0], [0, 5, 9], (0, 0)),
                        ([48, 32], [-7, 5, 9], (1, 1)), ([48, 32], [0, 5, 1 << 30], (1, 1)), ([48, 32], [9, 5, 0], (0, 0)),
                        ([48, 32], [-(1 << 31), -3, 0], (0, 0))):
        sets = [(front[i] if has[i] else []) + own(r, "own") for r, (i, _) in sorted(pos.items())]
        for bounds in ((0, 0), (1, 17)):
            _prefix(gpu, q, ref, (np.ascontiguousarray(b.table[2:]), pl, ps), (b.table[:2], b.kv[:2], b.starts[:3]), sets, hints,
                    bounds)


def test_prefix_attention_over_tables_without_pages():
    rng = np.random.default_rng(37)
    b, ref, q = _case([(32, 5), (16, 4)], rng)
    gpu, none = to_gpu(ref), np.zeros((1, 0), np.int32)
    pos = {r: (i, p) for r, i, p in b.positions()}
    sets = [[(b.lists[i], p + 1)] for _, (i, p) in sorted(pos.items())]
    for hints in ((0, 0), (1, 0)):
        _prefix(gpu, q, ref, (none, [7], [0, 9]), (b.table, b.kv, b.starts), sets, hints)
        _prefix(gpu, q, ref, (b.table[:1], [32], [0, 5]), (np.zeros((2, 0), np.int32), [3, 3], b.starts),
                [[(b.lists[0], 32)]] * 5 + [[]] * 4, hints)


@pytest.mark.parametrize("bits,sym", FORMATS)
def test_the_weights_of_a_row_add_up_to_one(bits, sym):
    """Each row's weights are its softmax, if its log-sum is attention's. Each is
    off by its own bound (oracle.serving.weigh) and by the log-sum's error, at
    most 1e-5 + 2^-20 of it (serving_helpers.check_attention), as exp has it."""
    rng = np.random.default_rng(38)
    b = Batch([(900, 1), (70, 70), (300, 9)], 16, rng)
    ref = new_cache(b, 16, 2, 128, bits, sym)
    fill(ref, b, rng)
    q = bf16(rng.standard_normal((b.rows, 8, 128)))
    gpu, gq, lse = to_gpu(ref), dev_bf16f(q), torch.empty((b.rows, 8), device="cuda")
    say(f"weights add up bits={bits} sym={sym}")
    bg.paged_attention(gq, gpu, *b.on_gpu(), lse=lse)
    got = host(bg.kv_cache_weigh(gq, lse, gpu, None, *b.on_gpu())).astype(np.float64)
    zero = np.zeros(ref.k_scales.shape, np.float32)
    _, bound = serving.weigh(q, host(lse), ref, zero, b.lists, b.kv, b.starts, 128 ** -0.5)
    off = np.expm1(1e-5 + 2.0 ** -20 * float(lse.abs().max()))
    for i, n in enumerate((1, 70, 9)):
        total, room = got[b.lists[i]].sum((0, 2)), bound[b.lists[i]].sum((0, 2))
        assert np.all(np.abs(total - 4 * n) <= room + 4 * n * off), (i, total - 4 * n, room, off)


@pytest.mark.parametrize("elsewhere", [False, True])
@pytest.mark.parametrize("d,bits", [(128, 8), (256, 4), (256, 8)])
@pytest.mark.parametrize("sym", [True, False])
def test_evict_rows_of_128_and_256_bytes_over_several_batches(d, bits, sym, elsewhere):
    """More than two batches of 1024 tokens, of one head (the most parts of a
    token) and of several."""
    _evict([5000, 2600, 1500], 2300, 100, d, bits, sym, heads=1, seed=d + bits, elsewhere=elsewhere, hints=(0, 5000))
    _evict([3000, 1100], 2100, 0, d, bits, sym, page=64, heads=3, seed=d, elsewhere=elsewhere)


@pytest.mark.parametrize("d,bits,sym", [(128, 8, False), (256, 8, True)])
def test_some_pages_of_wide_rows_stay_in_their_place(d, bits, sym):
    rng = np.random.default_rng(d)
    page, keep = 16, 3000
    b = Batch([(7000, 0), (4000, 0), (keep, 0), (keep, 0)], page, rng)
    ref = new_cache(b, page, 1, d, bits, sym)
    for t in (ref.k_codes, ref.v_codes):
        t[:] = rng.integers(0, 256, t.shape, dtype=np.uint8)
    for t in (ref.k_scales, ref.v_scales, ref.k_zeros, ref.v_zeros):
        if t is not None:
            t[:] = rng.random(t.shape, dtype=np.float32)
    w = _weights(ref, rng)
    mixed = [old if i % 3 else new for i, (old, new) in enumerate(zip(b.lists[0], b.lists[2]))]
    to = [mixed, b.lists[3]]
    gpu, wg = to_gpu(ref), dev(w)
    say(f"evict, some pages stay, D={d} bits={bits} sym={sym}")
    lens, kept = bg.kv_cache_evict(gpu, wg, dev(np.ascontiguousarray(b.table[:2])), _i32([7000, 4000]), keep, 100,
                                   to_table=_i32(to))
    want_kept, want_lens = serving.evict(ref, w, b.lists[:2], [7000, 4000], keep, 100, to)
    assert host(lens).tolist() == want_lens
    assert_same_bits(host(kept), want_kept, "kept")
    for name, want in _state(ref, w).items():
        got = host(wg if name == "weights" else getattr(gpu, name))
        for pages in to:
            whole = pages[:keep // page]                # slots behind the last token may hold anything
            assert np.array_equal(got[whole], want[whole], equal_nan=True), name


@pytest.mark.parametrize("call", ["paged", "prefix"])
@pytest.mark.parametrize("last", [(1 << 31) - 1, (1 << 31) - 200, (1 << 31) - 300])
def test_rows_past_any_table_pass_over_pages_outside_the_pool(call, last):
    """Of single rows that stand at the ends of what int32 holds, over tiles of 32
    keys whose first half is in no page: positions there are not attended to."""
    rng = np.random.default_rng(40)
    b, ref, q = _case([(128, 1), (64, 1)], rng, group=4)
    gpu, table = to_gpu(ref), b.table.copy()
    table[0, 0] = table[0, 4] = table[1, 2] = -1
    kv, starts = [last, last], [0, 1, 2]
    sets = [_pieces(ref, table[i], 16 * table.shape[1]) for i in range(2)]
    for hints in ((1, 0), (1, 128)):
        if call == "prefix":
            _prefix(gpu, q, ref, (table[:1], [128], [0, 2]), (table, kv, starts), [_pieces(ref, table[0], 128) + s for s in sets],
                    hints)
        else:
            need = bg.paged_attention_workspace(2, 4, gpu, 2, table.shape[1], *hints)
            _run_attention(q, ref, sets, need, lambda x, **a: bg.paged_attention(
                x, gpu, dev(table), _i32(kv), _i32(starts), max_rows=hints[0], max_kv=hints[1], **a), f"paged {kv} {hints}")

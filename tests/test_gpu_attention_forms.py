"""paged_attention against the oracle in every form its work takes: parts of many
steps, blocks with two parts, tiles of 8, 16, 128 and 256 rows, single tokens
beside chunks with one join for both, whole units past the page look-ahead, and
many sequences. Each test names its form (attention_forms.forms, held to the
library's own workspace), so that another rule of dispatch shows here. Every
output lies between canaries. The oracle takes some of the key heads."""
import numpy as np
import pytest
import torch

import bit_gemv_amd as bg
from attention_forms import forms
from gpu_helpers import dev, say
from oracle import serving
from serving_helpers import Batch, bf16, check_attention, dev_bf16f, new_cache, to_gpu
from test_gpu_guard import Guarded

pytestmark = pytest.mark.gpu

FORMATS = [(4, False), (4, True), (8, False), (8, True)]
# every format at 64 and 128 wide, two at 256
WIDE = [(d, *f) for d in (64, 128) for f in FORMATS] + [(256, 4, False), (256, 8, True)]
ROOM = 8192
SINGLE = [(1500, 1), (700, 1), (2300, 1), (0, 1), (1, 1)]


def _random_cache(b, page, heads, d, bits, sym, rng, far=False):
    """Random codes and scales in every held slot, zeros among the codes (far:
    every third key or value's outside of them, with a small scale); the other
    slots keep the NaN that new_cache gives them."""
    c = new_cache(b, page, heads, d, bits, sym)
    c.k_codes[:] = rng.integers(0, 256, c.k_codes.shape, np.uint8)
    c.v_codes[:] = rng.integers(0, 256, c.v_codes.shape, np.uint8)
    step = 2.0 / 2 ** bits
    for i, held in enumerate(b.kv):
        for p, page_of in enumerate(b.lists[i]):
            n = min(page, held - p * page)
            for side in "kv":
                s = rng.uniform(0.5, 1.5, (heads, n)) * step
                z = rng.integers(0, 2 ** bits, (heads, n)).astype(np.float32)
                if far:
                    t = (p * page + np.arange(n)) % 3 == 0
                    z[:, t] = rng.choice([-5e4, -300.0, 2000.0, 7e6], (heads, int(t.sum())))
                    s[:, t] = rng.uniform(-2, 2, (heads, int(t.sum()))).clip(0.5) / np.abs(z[:, t])
                getattr(c, side + "_scales")[page_of, :, :n] = s
                if not sym:
                    getattr(c, side + "_zeros")[page_of, :, :n] = z
    return c


def _some_heads(c, heads):
    """The oracle's cache of some key heads"""
    part = serving.Cache.__new__(serving.Cache)
    part.__dict__.update(c.__dict__)
    part.heads = len(heads)
    for n in ("k_codes", "v_codes", "k_scales", "v_scales", "k_zeros", "v_zeros"):
        if getattr(c, n) is not None:
            setattr(part, n, getattr(c, n)[:, heads])
    return part


def _run(seqs, d, bits, sym, heads, group, hints, form, room=ROOM, page=16, seed=0, q_scale=1.0, far=False, lead=0, bad=None):
    """form: what the launches of this call must be, given as a check of
    forms()' result. bad: (row, query head) pairs whose q holds a NaN."""
    rng = np.random.default_rng(seed + d + bits)
    b = Batch(seqs, page, rng, lead=lead, wide=room // page - 1)
    rows, qh = b.rows + 1, heads * group
    launches = forms(seqs, d, bits, heads, group, b.table.shape[1] * page, *hints, rows)
    assert b.table.shape[1] * page == room
    assert form(launches), launches
    ref = _random_cache(b, page, heads, d, bits, sym, rng, far)
    q = bf16(rng.standard_normal((rows, qh, d)) * q_scale)
    gq = dev_bf16f(q)
    keep = np.ones((rows, qh), bool)
    for r, h in bad or ():
        gq[r, h, (r + h) % d] = float("nan")
        keep[r, h] = False
    gpu, batch = to_gpu(ref), b.on_gpu()
    need = bg.paged_attention_workspace(rows, qh, gpu, len(seqs), batch[0].shape[1], *hints)
    ws, out, lse = Guarded((max(need, 256),), torch.uint8), Guarded((rows, qh, d), torch.bfloat16), Guarded((rows, qh), torch.float32)
    out.t.fill_(7.0)
    lse.t.fill_(7.0)
    say(f"paged_attention D={d} bits={bits} sym={sym} heads={heads} group={group} hints={hints} {launches}")
    bg.paged_attention(gq, gpu, *batch, max_rows=hints[0], max_kv=hints[1], out=out.t, lse=lse.t, workspace=ws.t)
    for t, n in ((ws, "workspace"), (out, "out"), (lse, "lse")):
        t.check(n)
    mine = np.array([r for r, _, _ in b.positions()])
    rest = [r for r in range(rows) if r not in set(mine.tolist())]
    assert bool((out.t[rest] == 7.0).all()) and bool((lse.t[rest] == 7.0).all()), "rows of no sequence changed"
    for h in sorted({0, heads - 1, int(rng.integers(heads))} if heads > 2 else set(range(heads))):
        cols = slice(h * group, (h + 1) * group)
        want, wl, bound = serving.attention(q[:, cols], _some_heads(ref, [h]), b.lists, b.kv, b.starts, d ** -0.5)
        pick = np.zeros((rows, group), bool)
        pick[mine] = keep[mine, cols]
        on = torch.from_numpy(pick).cuda()
        check_attention(out.t[:, cols][on], lse.t[:, cols][on], want[pick], wl[pick], bound[pick], f"key head {h} {launches}")
    gone = torch.from_numpy(~keep).cuda()
    assert bool(out.t[gone].isnan().all()) and bool(lse.t[gone].isnan().all())


def _cut(p, tile):
    """Spans of several steps, some with two parts in a block"""
    return p.tile == tile and not p.by_unit and p.longest > 1 and p.parts and p.share > 1


def _cut_twice(p, tile):
    return _cut(p, tile) and p.second > 0 and any(len(x) > 1 for x in p.parts)


@pytest.mark.parametrize("d,bits,sym", WIDE)
def test_single_tokens_in_long_spans(d, bits, sym):
    _run(SINGLE, d, bits, sym, 64, 4, (1, 0), lambda f: len(f) == 1 and _cut_twice(f[0], 8), seed=1)
    _run([(h, 2 if h > 5 else n) for h, n in SINGLE], d, bits, sym, 64, 7, (2, 0),
         lambda f: len(f) == 1 and _cut_twice(f[0], 16), seed=2)


@pytest.mark.parametrize("d,bits,sym", WIDE)
def test_chunks_in_long_spans(d, bits, sym):
    _run([(700, 90), (310, 40), (33, 33)], d, bits, sym, 32, 4, (90, 0), lambda f: len(f) == 1 and _cut_twice(f[0], 128), seed=3)
    if d < 256:
        _run([(900, 230), (310, 200), (300, 300)], d, bits, sym, 32, 4, (300, 0),
             lambda f: len(f) == 1 and _cut_twice(f[0], 256), seed=4)


@pytest.mark.parametrize("d,bits,sym", WIDE)
def test_chunks_beside_single_tokens_joined_at_once(d, bits, sym):
    """Both launches cut, one join: tiles of 256 (128 for 256-wide heads) and
    of 128 rows beside those of 16."""
    _run([(1100, 290)] + SINGLE[:3], d, bits, sym, 32, 4, (290, 0),
         lambda f: len(f) == 2 and _cut_twice(f[0], 128 if d == 256 else 256) and _cut(f[1], 16), seed=5)
    _run([(700, 90), (310, 40)] + SINGLE, d, bits, sym, 32, 2, (90, 0),
         lambda f: len(f) == 2 and _cut_twice(f[0], 128) and _cut(f[1], 16), seed=6, lead=2)


@pytest.mark.parametrize("d,bits,sym", WIDE)
def test_whole_units_of_chunks(d, bits, sym):
    """Several sequences, 256 rows a tile: blocks take units, the largest first."""
    _run([(1100, 290), (333, 150)], d, bits, sym, 8, 4, (290, 1100),
         lambda f: len(f) == 1 and f[0].by_unit and f[0].tile == (128 if d == 256 else 256), room=1120, seed=7)


@pytest.mark.parametrize("d,bits,sym", WIDE)
def test_units_past_the_page_look_ahead(d, bits, sym):
    """Pages are read 64 groups of 16 keys ahead for many rows (1024 keys) and 64
    steps ahead for few (8192): units longer than that, taken whole because the
    hint says less."""
    units = lambda tile: lambda f: len(f) == 1 and f[0].by_unit and f[0].tile == tile  # noqa: E731
    _run([(2200, 70), (1300, 75)], d, bits, sym, 1, 3, (0, 300), units(128), room=2224, seed=8)
    if d < 256:
        _run([(2200, 120), (1300, 150)], d, bits, sym, 1, 4, (0, 300), units(256), room=2224, seed=9)
    _run([(8500, 1), (16600, 2)], d, bits, sym, 1, 2, (2, 1000), units(8), room=16640, page=32, seed=10)
    _run([(8500, 2), (16600, 2)], d, bits, sym, 1, 8, (2, 1000), units(16), room=16640, page=32, seed=11)


@pytest.mark.parametrize("bits,sym", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
def test_more_than_64_sequences_in_spans(d, bits, sym):
    """The sequences are added up in several rounds."""
    lens = [90 + (i * 37) % 60 for i in range(150)]
    _run([(n, 1) for n in lens], d, bits, sym, 8, 4, (1, 0), lambda f: len(f) == 1 and _cut_twice(f[0], 8), seed=12)
    _run([(n, 1 + (i % 3) * 7) for i, n in enumerate(lens)], d, bits, sym, 8, 2, (15, 0),
         lambda f: len(f) == 2 and _cut_twice(f[0], 128) and _cut_twice(f[1], 16), seed=13)


@pytest.mark.parametrize("hints", [(1, 0), (1, 40), (0, 0), (3, 40)])
def test_a_thousand_sequences(hints):
    _run([(1 + (i * 7) % 40, 1) for i in range(1000)], 64, 8, True, 2, 4, hints, lambda f: True, seed=14, room=64 if hints[1] else ROOM)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_zeros_far_from_the_codes_in_every_tile(d, bits):
    kw = dict(far=True, q_scale=0.2)
    _run([(900, 230), (310, 200), (300, 300)], d, bits, False, 32, 4, (300, 0), lambda f: _cut_twice(f[0], 256), seed=15, **kw)
    _run([(1100, 290)] + SINGLE[:3], d, bits, False, 32, 4, (290, 0),
         lambda f: _cut_twice(f[0], 256) and _cut(f[1], 16), seed=16, **kw)
    _run([(333, 150)], d, bits, False, 2, 4, (150, 333), lambda f: f[0].by_unit and f[0].tile == 256, seed=17, room=352, **kw)
    _run(SINGLE, d, bits, False, 64, 4, (1, 0), lambda f: _cut_twice(f[0], 8), seed=18, **kw)


@pytest.mark.parametrize("d,bits,sym", WIDE)
def test_a_nan_row_changes_no_other_in_every_tile(d, bits, sym):
    big = 128 if d == 256 else 256
    _run([(1100, 290)] + SINGLE[:3], d, bits, sym, 32, 4, (290, 0), lambda f: _cut_twice(f[0], big) and _cut(f[1], 16),
         seed=19, bad=[(0, 0), (130, 127), (289, 2), (291, 1), (292, 126)])
    _run([(1100, 290), (333, 150)], d, bits, sym, 8, 4, (290, 1100), lambda f: f[0].by_unit and f[0].tile == big,
         room=1120, seed=20, bad=[(0, 0), (200, 31), (439, 3)])
    _run(SINGLE, d, bits, sym, 64, 4, (1, 0), lambda f: _cut_twice(f[0], 8), seed=21, bad=[(0, 0), (2, 255), (2, 3)])


def _sees_all(c, pages, q, group, scale):
    """Attention of rows q to every token of `pages`, in 64 bits; and the largest value"""
    out, lse, top = np.zeros(q.shape), np.zeros(q.shape[:2]), 0.0
    for h in range(q.shape[1]):
        n = len(pages) * c.page_size
        (kq, ks, kz), (vq, vs, vz) = c.parts(pages, h // group, "k", n), c.parts(pages, h // group, "v", n)
        k, v = (kq - kz[:, None]) * ks[:, None], (vq - vz[:, None]) * vs[:, None]
        t = scale * q[:, h].astype(np.float64) @ k.T
        p = np.exp(t - t.max(-1, keepdims=True))
        out[:, h] = p @ v / p.sum(-1, keepdims=True)
        lse[:, h] = t.max(-1) + np.log(p.sum(-1))
        top = max(top, np.abs(v).max())
    return out, lse, top


@pytest.mark.parametrize("hints,room", [((0, 0), 48), ((5, 32), 48), ((5, 0), ROOM), ((1, 0), ROOM), ((1, 17), 48)])
def test_odd_lengths_and_starts_between_canaries(hints, room):
    """Lengths and starts that no batch should have: rows see what the table
    holds at positions up to their own, or nothing, and rows that they give to
    no sequence are left alone."""
    rng = np.random.default_rng(22)
    b = Batch([(32, 5), (16, 4)], 16, rng, wide=room // 16 - 1)
    ref = _random_cache(b, 16, 1, 64, 8, True, rng)
    q = bf16(rng.standard_normal((9, 12, 64)))
    gpu, gq, scale = to_gpu(ref), dev_bf16f(q), 0.125
    want, wl, bound = serving.attention(q, ref, b.lists, b.kv, b.starts, scale)
    tops = [_sees_all(ref, b.lists[i], q, 12, scale) for i in range(2)]
    cases = [([1 << 30, 16], [0, 5, 9], {0: "all", 1: "own"}), ([(1 << 31) - 1, 16], [0, 5, 9], {0: "all", 1: "own"}),
             ([-5, 16], [0, 5, 9], {0: "none", 1: "own"}), ([-(1 << 31), 16], [0, 5, 9], {0: "none", 1: "own"}),
             ([32, 16], [-7, 5, 9], {0: "own", 1: "own"}), ([32, 16], [0, 5, 1 << 30], {0: "own", 1: "none"}),
             ([32, 16], [9, 5, 0], {0: "left", 1: "left"}), ([32, 16], [-(1 << 31), -3, 0], {0: "left", 1: "left"})]
    for kv, starts, kinds in cases:
        need = bg.paged_attention_workspace(9, 12, gpu, 2, b.table.shape[1], *hints)
        ws, out, lse = Guarded((max(need, 256),), torch.uint8), Guarded((9, 12, 64), torch.bfloat16), Guarded((9, 12), torch.float32)
        out.t.fill_(7.0)
        lse.t.fill_(7.0)
        say(f"paged_attention kv={kv} starts={starts} hints={hints}")
        bg.paged_attention(gq, gpu, b.on_gpu()[0], dev(np.asarray(kv, np.int32)), dev(np.asarray(starts, np.int32)),
                           max_rows=hints[0], max_kv=hints[1], out=out.t, lse=lse.t, workspace=ws.t)
        for t, n in ((ws, "workspace"), (out, "out"), (lse, "lse")):
            t.check(n)
        for i, rows in ((0, slice(0, 5)), (1, slice(5, 9))):
            o, ll = out.t[rows], lse.t[rows]
            if kinds[i] == "own":
                check_attention(o, ll, want[rows], wl[rows], bound[rows], f"{kv} {starts}")
            elif kinds[i] == "none":
                assert bool((o == 0).all()) and bool(torch.isneginf(ll).all()), (kv, starts)
            elif kinds[i] == "left":
                assert bool((o == 7.0).all()) and bool((ll == 7.0).all()), (kv, starts)
            else:
                # every element's bound (oracle.serving.attention) is at most
                # (2^-8 + 2^-10) of the largest value: the result's own rounding,
                # the weights', and what is left of the other terms below 2^-11
                all_out, all_lse, top = tops[i]
                err = np.abs(o.float().cpu().numpy() - all_out[rows])
                assert err.max() <= (2.0 ** -8 + 2.0 ** -10) * top, err.max()
                assert np.abs(ll.cpu().numpy() - all_lse[rows]).max() <= 1e-5 + 2.0 ** -20 * np.abs(all_lse).max()


@pytest.mark.parametrize("bits,sym", FORMATS)
def test_written_slots_after_a_replay(bits, sym):
    """The cache's bytes after a captured write are those of an eager one, on
    every replay, and no other byte moves."""
    rng = np.random.default_rng(23)
    b = Batch([(40, 40), (19, 3), (64, 1), (0, 2)], 16, rng)
    c = to_gpu(new_cache(b, 16, 2, 128, bits, sym))
    k, v = torch.randn((2, b.rows, 2, 128), device="cuda")
    batch, pool = b.on_gpu(), [t for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales, c.k_zeros, c.v_zeros) if t is not None]
    first = [t.clone() for t in pool]
    say(f"kv_cache_write captured bits={bits} sym={sym}")
    bg.kv_cache_write(k, v, c, *batch)
    want = [t.clone() for t in pool]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bg.kv_cache_write(k, v, c, *batch)
    for _ in range(3):
        for t, f in zip(pool, first):
            t.copy_(f)
        g.replay()
        torch.cuda.synchronize()
        for t, w, f in zip(pool, want, first):
            assert torch.equal(t.view(torch.uint8), w.view(torch.uint8)) and not torch.equal(t.view(torch.uint8), f.view(torch.uint8))
        (k * v).sum().item()                        # the program's own work between replays

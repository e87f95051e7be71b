"""prefix_attention and cross_attention against the oracle in 64 bits, each
element within a bound derived from the stated arithmetic
(oracle.serving.attention_over)."""
import ctypes

import numpy as np
import pytest
import torch

import bit_gemv_amd as bg
from gpu_helpers import dev, say
from oracle import serving
from serving_helpers import Batch, bf16, check_attention, dev_bf16f, fill, new_cache, to_gpu
from test_gpu_graphs import _check_graph
from test_gpu_guard import Guarded, _ok, _p, _st

pytestmark = pytest.mark.gpu

FORMATS = [(4, False), (4, True), (8, False), (8, True)]


def _i32(v):
    return dev(np.asarray(v, np.int32))


class Shared:
    """Sequences (own tokens, rows), each prefix (tokens, sequences) before as
    many of them, in one pool; `skip` sequences at the front have no prefix."""

    def __init__(self, seqs, prefixes, page, rng, skip=0, lead=0, wide=0):
        self.b = b = Batch(list(seqs) + [(n, 0) for n, _ in prefixes], page, rng, lead=lead, wide=wide)
        n = len(seqs)
        self.kv, self.starts, self.lists = b.kv[:n], b.starts[:n + 1], b.lists[:n]
        first = [skip]
        for _, m in prefixes:
            first.append(first[-1] + m)
        assert first[-1] <= n
        self.prefix_lens = [m for m, _ in prefixes]
        self.prefix_starts = [self.starts[i] for i in first]
        self.sets = [None] * (b.rows + 1)                       # a row behind the last sequence
        for r, i, pos in b.positions():
            front = [(b.lists[n + j], m) for j, (m, _) in enumerate(prefixes) if first[j] <= i < first[j + 1]]
            self.sets[r] = front + [(self.lists[i], min(pos + 1, self.kv[i]))]
        table = dev(b.table)
        self.args = (table[n:].contiguous(), _i32(self.prefix_lens), _i32(self.prefix_starts), table[:n].contiguous(),
                     _i32(self.kv), _i32(self.starts))


def _compare(name, call, ref, sets, rows, qh, d, rng, hints, scale, q_scale, gap, what):
    q = bf16(rng.standard_normal((rows, qh, d)) * q_scale)
    wide = torch.full((rows, qh + gap, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :qh] = dev_bf16f(q)
    want, want_lse, bound = serving.attention_over(q, ref, sets, d ** -0.5 if scale is None else scale)
    mine = [r for r in range(rows) if sets[r] is not None]
    rest = [r for r in range(rows) if sets[r] is None]
    for h in hints:
        say(f"{name} {what} D={d} bits={ref.bits} sym={ref.symmetric} page={ref.page_size} heads={ref.heads} q heads {qh} "
            f"rows {rows} hints {h}")
        out = torch.full((rows, qh, d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((rows, qh), 7.0, device="cuda")
        call(wide[:, :qh], out=out, lse=lse, scale=scale, **h)
        check_attention(out, lse, want, want_lse, bound, f"{name} {what} {h}", mine)
        assert bool((out[rest] == 7.0).all()) and bool((lse[rest] == 7.0).all()), "rows of no sequence changed"


def _prefix(seqs, prefixes, d, bits, sym, page=16, heads=2, group=4, seed=0, hints=({},), scale=None, q_scale=1.0, gap=0,
            what="", k_scale=1.0, v_scale=1.0, **kw):
    rng = np.random.default_rng(seed)
    s = Shared(seqs, prefixes, page, rng, **kw)
    ref = new_cache(s.b, page, heads, d, bits, sym)
    fill(ref, s.b, rng, k_scale, v_scale)
    gpu = to_gpu(ref)
    _compare("prefix_attention", lambda q, **a: bg.prefix_attention(q, gpu, *s.args, **a), ref, s.sets, s.b.rows + 1,
             heads * group, d, rng, hints, scale, q_scale, gap, what)


def _cross(seqs, d, bits, sym, page=16, heads=2, group=4, seed=0, hints=({},), scale=None, q_scale=1.0, gap=0, lead=0, room=0,
           what="", k_scale=1.0, v_scale=1.0):
    rng = np.random.default_rng(seed)
    b = Batch(seqs, page, rng, lead=lead, wide=room // page)
    ref = new_cache(b, page, heads, d, bits, sym)
    fill(ref, b, rng, k_scale, v_scale)
    gpu = to_gpu(ref)
    sets = [None] * (b.rows + 1)
    for r, i, _ in b.positions():
        sets[r] = [(b.lists[i], b.kv[i])]
    _compare("cross_attention", lambda q, **a: bg.cross_attention(q, gpu, *b.on_gpu(), **a), ref, sets, b.rows + 1,
             heads * group, d, rng, hints, scale, q_scale, gap, what)


# encoder tokens, rows: one of each, more rows than tokens, none, odd ends
STATES = [(1, 1), (17, 1), (5, 40), (33, 5), (261, 3), (0, 4), (40, 0), (129, 2), (70, 70)]


@pytest.mark.parametrize("bits,sym", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_cross_formats(d, bits, sym):
    """Bounds that choose each kernel: 256, 128, 16 and 8 rows a tile; whole units
    and, over a wide table, spans."""
    hints = ({}, dict(max_rows=70), dict(max_rows=4, max_kv=261), dict(max_rows=2))
    _cross(STATES, d, bits, sym, seed=d + bits, hints=hints)
    _cross(STATES, d, bits, sym, seed=d + bits, hints=hints, room=8192)


@pytest.mark.parametrize("bits,sym", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_cross_single_tokens(d, bits, sym):
    _cross([(1, 1), (2, 1), (31, 1), (32, 1), (33, 1), (128, 1), (0, 1), (300, 1), (16, 1)], d, bits, sym, seed=d + bits + 1,
           hints=(dict(max_rows=1, max_kv=300), dict(max_rows=1), {}), group=1)


@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 16, 20])
@pytest.mark.parametrize("bits,sym", [(4, False), (8, True)])
def test_cross_head_layouts(group, bits, sym):
    _cross([(37, 1), (50, 11), (9, 30)], 64, bits, sym, heads=1 if group > 8 else 3, group=group, seed=group)


@pytest.mark.parametrize("bits,sym", [(4, True), (8, False)])
def test_cross_pages_beams_and_a_long_input(bits, sym):
    for page in (16, 64, 256):
        _cross([(300, 5), (270, 5), (257, 5), (3, 5)], 64, bits, sym, page=page, heads=1, group=2, seed=page, gap=3, lead=2)
    _cross([(4001, 2), (77, 150)], 64, bits, sym, page=32, heads=1, group=2, seed=5,
           hints=({}, dict(max_rows=2, max_kv=4001)))


@pytest.mark.parametrize("bits,sym", [(4, False), (8, True)])
def test_cross_beside_single_tokens_and_with_wrong_bounds(bits, sym):
    """A batch whose single rows go to a launch of their own; bounds too small."""
    seqs = [(150, 100)] + [(n, 1) for n in (1, 40, 257, 600, 0)] + [(9, 9), (4, 4)]
    _cross(seqs, 64, bits, sym, seed=6, hints=(dict(max_rows=100, max_kv=600), dict(max_rows=100, max_kv=9000),
                                               dict(max_rows=1, max_kv=1)), room=9000 // 16 * 16)


# own tokens, rows: behind the prefix nothing but the row itself, rows before
# the sequence's first position, no rows, nothing of their own
OWN = [(1, 1), (17, 1), (16, 16), (33, 5), (3, 6), (40, 0), (0, 2), (129, 1), (70, 70)]


@pytest.mark.parametrize("bits,sym", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefix_formats(d, bits, sym):
    """Every kernel for the prefix and for the own tokens; whole units and, where
    lengths are not known and the table is wide, spans."""
    hints = ({}, dict(max_rows=70, max_kv=129, max_prefix=300, max_prefix_rows=110),
             dict(max_rows=1, max_kv=129, max_prefix=300, max_prefix_rows=3),
             dict(max_rows=4, max_kv=8000, max_prefix=8000, max_prefix_rows=1))
    _prefix(OWN, [(300, 4), (33, 5)], d, bits, sym, seed=d + bits, hints=hints)
    _prefix(OWN, [(300, 4), (33, 5)], d, bits, sym, seed=d + bits, hints=hints, wide=512)


@pytest.mark.parametrize("bits,sym", FORMATS)
def test_prefix_decode(bits, sym):
    """A decode batch behind one long prefix, in 8-, 16- and 128-row tiles."""
    for n, group, d in ((2, 4, 64), (4, 4, 128), (20, 8, 128)):
        seqs = [(1 + (37 * i) % 90, 1) for i in range(n)]
        _prefix(seqs, [(700, n)], d, bits, sym, heads=1, group=group, seed=n, page=64,
                hints=({}, dict(max_rows=1, max_kv=90, max_prefix=700, max_prefix_rows=n)))


@pytest.mark.parametrize("group,d", [(7, 64), (5, 128), (3, 256)])
def test_prefix_tiles_end_inside_a_group(group, d):
    """Rows beside each other in different tiles, units cut into parts and whole
    ones, of the prefix and of the own tokens, one prefix and several."""
    seqs = [(90, 70), (60, 50), (300, 90), (40, 40), (33, 1)]
    for prefixes in ([(500, 5)], [(500, 2), (260, 3)]):
        _prefix(seqs, prefixes, d, 8, False, heads=1, group=group, seed=group, wide=512,
                hints=({}, dict(max_rows=90, max_kv=300), dict(max_prefix=500, max_prefix_rows=260)))


def test_prefix_of_more_than_64_sequences():
    """Past what a wave looks up at once: single rows, and a few chunks."""
    for page, n in ((16, 70), (64, 150)):
        seqs = [(1 + (7 * i) % 40, 3 if i % 40 == 1 else 1) for i in range(n)]
        _prefix(seqs, [(130, 20), (70, n - 25)], 64, 8, True, page=page, heads=1, group=2, seed=n, skip=5,
                hints=({}, dict(max_rows=3, max_kv=40, max_prefix=130, max_prefix_rows=n)))
        many = [(0, 0)] * 66 + [(20, 2), (30, 1)]
        _prefix(many, [(10, 1)] * 66 + [(200, 2)], 64, 8, True, page=page, heads=1, group=2, seed=n)


@pytest.mark.parametrize("group", [1, 3, 7, 16, 20])
def test_prefix_head_layouts(group):
    _prefix([(37, 1), (50, 11), (20, 20)], [(90, 2), (17, 1)], 64, 8, True, heads=1 if group > 8 else 3, group=group, seed=group)


def test_prefix_of_some_rows_only_and_empty_ones():
    """Sequences without a prefix before and behind those with one, a prefix of
    no tokens, one of no sequences, leading rows and rows apart."""
    _prefix([(20, 2), (30, 1), (5, 5), (60, 3), (9, 1)], [(50, 1), (0, 1), (100, 0), (16, 1)], 128, 8, True, skip=1, lead=3,
            gap=2, seed=3)
    _prefix([(0, 2), (0, 1)], [(0, 2)], 64, 4, False, seed=4)


def test_prefix_scales_and_sharp_softmax():
    for scale in (1.0, -0.3, 0.0):
        _prefix([(33, 5), (20, 1)], [(100, 2)], 64, 8, True, seed=8, scale=scale)
    # all weight in the prefix, all of it in the own tokens, and value scales
    # that differ between them by many powers of two
    for f in (lambda i, t: 30.0 if i == 2 else 0.1, lambda i, t: 0.1 if i == 2 else 30.0):
        _prefix([(90, 4), (70, 40)], [(200, 2)], 64, 8, True, seed=9, k_scale=f, q_scale=2.0)
        _prefix([(90, 4), (70, 40)], [(200, 2)], 64, 4, False, seed=9, v_scale=f)


def test_without_a_prefix_it_is_paged_attention():
    rng = np.random.default_rng(1)
    b = Batch([(33, 5), (200, 1), (40, 40)], 16, rng)
    ref = new_cache(b, 16, 2, 64, 8, True)
    fill(ref, b, rng)
    gpu, q = to_gpu(ref), torch.randn((b.rows, 8, 64), device="cuda").bfloat16()
    say("prefix_attention p=0")
    none = torch.zeros((0, 3), dtype=torch.int32, device="cuda"), _i32([]), _i32([0])
    assert torch.equal(bg.prefix_attention(q, gpu, *none, *b.on_gpu()), bg.paged_attention(q, gpu, *b.on_gpu()))


def test_a_shared_prefix_is_what_each_sequence_alone_has():
    """The prefix's pages at the front of every sequence's own table
    (paged_attention) and shared give the same attention."""
    rng = np.random.default_rng(2)
    s = Shared([(20, 1), (37, 9), (1, 1)], [(96, 3)], 16, rng)
    ref = new_cache(s.b, 16, 2, 128, 8, False)
    fill(ref, s.b, rng)
    gpu, q = to_gpu(ref), dev_bf16f(bf16(rng.standard_normal((s.b.rows, 8, 128))))
    front = s.b.lists[3]
    table = np.full((3, 20), -1, np.int32)
    for i, pages in enumerate(s.lists):
        table[i, :len(front) + len(pages)] = front + pages
    say("shared and alone")
    alone = bg.paged_attention(q, gpu, dev(table), _i32([n + 96 for n in s.kv]), s.args[5])
    _, _, bound = serving.attention_over(q.float().cpu().numpy(), ref, s.sets[:-1], 128 ** -0.5)
    off = (bg.prefix_attention(q, gpu, *s.args).double() - alone.double()).abs().cpu().numpy()
    assert np.all(off <= 2 * bound)


def test_a_nan_stays_in_its_row():
    rng = np.random.default_rng(3)
    s = Shared([(20, 1), (37, 9), (1, 1)], [(96, 3)], 16, rng)
    ref = new_cache(s.b, 16, 2, 64, 8, True)
    fill(ref, s.b, rng)
    gpu, q = to_gpu(ref), torch.randn((s.b.rows, 4, 64), device="cuda").bfloat16()
    bad = q.clone()
    bad[4, 2, 7] = float("nan")
    for name, call in (("prefix", lambda x, l: bg.prefix_attention(x, gpu, *s.args, lse=l)),
                       ("cross", lambda x, l: bg.cross_attention(x, gpu, *s.args[3:], lse=l))):
        say(name, "NaN")
        l0, l1 = torch.empty((2, s.b.rows, 4), device="cuda")
        want, got = call(q, l0), call(bad, l1)
        assert bool(got[4, 2].isnan().all()) and bool(l1[4, 2].isnan())
        got[4, 2], l1[4, 2] = want[4, 2], l0[4, 2]
        assert torch.equal(got, want) and torch.equal(l1, l0)


@pytest.mark.parametrize("bits,sym", [(4, False), (8, True)])
def test_graphs(bits, sym):
    """Captured and replayed, one after another with workspaces of their own."""
    rng = np.random.default_rng(7)
    s = Shared([(300, 1), (37, 30), (1, 1), (90, 1)], [(900, 2), (70, 2)], 16, rng, wide=512)
    ref = new_cache(s.b, 16, 2, 128, bits, sym)
    fill(ref, s.b, rng)
    gpu, q = to_gpu(ref), torch.randn((s.b.rows, 8, 128), device="cuda").bfloat16()
    out, lse, cross = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"), torch.empty_like(q)
    for hints in ({}, dict(max_rows=30, max_kv=300, max_prefix=900, max_prefix_rows=40)):
        def both():
            bg.prefix_attention(q, gpu, *s.args, out=out, lse=lse, **hints)
            bg.cross_attention(q, gpu, *s.args[3:], out=cross, max_rows=hints.get("max_rows", 0))
        _check_graph(f"prefix and cross {hints}", both, [out, lse, cross])


@pytest.mark.parametrize("d,bits,sym", [(64, 4, True), (128, 8, True), (256, 4, False)])
def test_guard(d, bits, sym):
    """Outputs and workspace between canaries, in every launch form."""
    lib, rng = bg.load_library(), np.random.default_rng(d)
    s = Shared([(300, 1), (37, 30), (1, 1), (90, 1), (40, 2)], [(900, 2), (70, 2)], 16, rng, wide=512)
    ref = new_cache(s.b, 16, 2, d, bits, sym)
    fill(ref, s.b, rng)
    gpu, rows, qh = to_gpu(ref), s.b.rows, 6
    q = torch.randn((rows, qh, d), device="cuda").bfloat16()
    pt, pl, ps, bt, kl, rs = s.args
    for pr, pk, mr, mk in ((0, 0, 0, 0), (31, 900, 30, 300), (1, 900, 1, 300), (3, 4000, 1, 1), (1 << 20, 1 << 20, 3, 0)):
        need = bg.prefix_attention_workspace(rows, qh, gpu, 2, pt.shape[1], 5, bt.shape[1], pr, pk, mr, mk)
        ws, out, lse = Guarded((need,), torch.uint8), Guarded((rows, qh, d), torch.bfloat16), Guarded((rows, qh), torch.float32)
        say(f"guard prefix_attention D={d} {pr, pk, mr, mk} workspace {need}")
        _ok(lib.prefix_attention(gpu._ref, _p(q), rows, qh, qh * d, ctypes.c_float(d ** -0.5), _p(pt), pt.shape[1], _p(pl),
                                 _p(ps), 2, pr, pk, _p(bt), bt.shape[1], _p(kl), _p(rs), 5, mr, mk, ws.ptr(), need, out.ptr(),
                                 lse.ptr(), _st()), "prefix_attention")
        for t, n in ((ws, "workspace"), (out, "out"), (lse, "lse")):
            t.check(n)
        assert bool(torch.isfinite(out.t.float()).all()) and bool(torch.isfinite(lse.t).all())
        need = bg.cross_attention_workspace(rows, qh, gpu, 5, bt.shape[1], mr, mk)
        ws, out = Guarded((max(256, need),), torch.uint8), Guarded((rows, qh, d), torch.bfloat16)
        say(f"guard cross_attention {mr, mk} workspace {need}")
        _ok(lib.cross_attention(gpu._ref, _p(q), rows, qh, qh * d, ctypes.c_float(d ** -0.5), _p(bt), bt.shape[1], _p(kl),
                                _p(rs), 5, mr, mk, ws.ptr(), need, out.ptr(), None, _st()), "cross_attention")
        ws.check("workspace")
        out.check("out")
        assert bool(torch.isfinite(out.t.float()).all())


def test_two_streams_at_once():
    rng = np.random.default_rng(11)
    s = Shared([(300, 1), (37, 30), (1, 1), (90, 1)], [(900, 2), (70, 2)], 16, rng, wide=512)
    ref = new_cache(s.b, 16, 2, 64, 8, True)
    fill(ref, s.b, rng)
    gpu, q = to_gpu(ref), torch.randn((s.b.rows, 8, 64), device="cuda").bfloat16()
    calls = (lambda: bg.prefix_attention(q, gpu, *s.args), lambda: bg.cross_attention(q, gpu, *s.args[3:]))
    want = [c() for c in calls]
    torch.cuda.synchronize()
    say("two streams")
    got = []
    for st in [torch.cuda.Stream() for _ in range(2)]:
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got += [[c() for c in calls] for _ in range(4)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))

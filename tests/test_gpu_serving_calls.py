"""The serving operators as a program calls them: captured and replayed, on
other streams and side by side, writing nothing around their outputs, and one
after another through a decoder layer's attention half."""
import ctypes

import numpy as np
import pytest
import torch

import bit_gemv_amd as bg
import oracle
from gpu_helpers import assert_same_bits, dev, host, say
from oracle import serving
from serving_helpers import Batch, bf16, check_attention, dev_bf16f, fill, new_cache, to_gpu
from test_gpu_graphs import _check_graph
from test_gpu_guard import Guarded, _ok, _p, _st
from workloads import bf16_bits_to_f32

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _setup(seqs, heads=2, group=4, d=128, bits=8, sym=True, page=16, seed=0, wide=0):
    """A filled GPU cache of random codes, its batch and q."""
    rng = np.random.default_rng(seed)
    b = Batch(seqs, page, rng, wide=wide)
    c = bg.KVCache.empty(b.pages, page, heads, d, bits, sym)
    g = _gen(seed)
    for t in (c.k_codes, c.v_codes):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    for t in (c.k_scales, c.v_scales):
        t.copy_(torch.rand(t.shape, generator=g, device="cuda") * 0.02 + 0.01)
    if not sym:
        for t in (c.k_zeros, c.v_zeros):
            t.copy_(torch.randint(0, 2 ** bits, t.shape, generator=g, device="cuda").float())
    q = torch.randn((b.rows, heads * group, d), generator=g, device="cuda").bfloat16()
    return b, c, q


def test_norm_graph():
    x, res = torch.randn(33, 4096, device="cuda"), torch.randn(33, 4096, device="cuda").bfloat16()
    w = torch.rand(4096, device="cuda") + 0.5
    q, s, r = bg.rms_norm_int8(x, w, 1e-5, res)
    _check_graph("rms_norm_int8", lambda: bg.rms_norm_int8(x, w, 1e-5, res, r, q, s), [q, s, r])


@pytest.mark.parametrize("bits,sym", [(4, False), (8, True)])
def test_cache_graph(bits, sym):
    b, c, _ = _setup([(40, 40), (19, 3), (64, 1)], bits=bits, sym=sym)
    k, v = torch.randn((2, b.rows, 2, 128), device="cuda")
    batch = b.on_gpu()
    outs = [c.k_codes, c.v_codes, c.k_scales, c.v_scales]
    # slots outside the batch keep what the poison puts there: compare the read
    ko, vo = torch.empty_like(k), torch.empty_like(v)

    def both():
        bg.kv_cache_write(k, v, c, *batch)
        bg.kv_cache_read(c, *batch, rows=b.rows, dtype=torch.float32, k=ko, v=vo)

    _check_graph(f"kv_cache write and read bits={bits}", both, [ko, vo])
    assert all(bool(torch.isfinite(o.float()).any()) for o in outs)


@pytest.mark.parametrize("seqs,hints", [
    ([(900, 1), (17, 1), (300, 1)], (1, 900)),       # whole sequences per block
    ([(5000, 1), (700, 1)], (1, 5000)),              # spans, joined
    ([(700, 130), (260, 260)], (260, 700)),          # chunks, whole units
    ([(700, 130), (260, 260)], (260, 8000)),         # chunks, joined
    ([(300, 200)] + [(90, 1)] * 6, (200, 300)),      # two launches
    ([(300, 200)] + [(90, 1)] * 6, (200, 8000)),     # two launches of each kind
])
def test_attention_graph(seqs, hints):
    b, c, q = _setup(seqs, wide=512)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    batch = b.on_gpu()
    need = bg.paged_attention_workspace(b.rows, q.shape[1], c, len(seqs), batch[0].shape[1], *hints)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    for workspace in (ws, None):
        _check_graph(f"paged_attention {seqs[:2]}",
                     lambda: bg.paged_attention(q, c, *batch, max_rows=hints[0], max_kv=hints[1], out=out, lse=lse,
                                                workspace=workspace), [out, lse])


def test_two_graphs_and_growing_lengths():
    """Two captured decode steps over one cache, replayed in turn while the
    lengths in device memory grow: the launches depend on none of them."""
    b, c, q = _setup([(200, 1), (37, 1)], page=64)
    room = b.table.shape[1] * 64
    table = torch.zeros((2, b.table.shape[1]), dtype=torch.int32, device="cuda")
    table[0], table[1] = torch.arange(b.table.shape[1], device="cuda") % b.pages, (b.pages - 1)
    lens, starts = b.on_gpu()[1:]
    outs, graphs = [torch.empty_like(q) for _ in range(2)], []
    bg.paged_attention(q, c, table, lens, starts, max_rows=1)
    torch.cuda.synchronize()
    for i, qq in enumerate((q, -q)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            bg.paged_attention(qq, c, table, lens, starts, max_rows=1, out=outs[i])
        graphs.append((g, qq))
    say("two graphs")
    for n in (1, 64, 129, room):
        lens.fill_(n)
        for i in (0, 1, 1, 0):
            outs[i].fill_(float("nan"))
            graphs[i][0].replay()
            want = bg.paged_attention(graphs[i][1], c, table, lens, starts, max_rows=1)
            torch.cuda.synchronize()
            assert torch.equal(outs[i], want), (n, i)


def test_other_streams_side_by_side():
    """The same calls on two streams at once give the bits of calls in order."""
    sets = [_setup([(3000, 1), (500, 1)], seed=s) for s in (1, 2)] + [_setup([(400, 70)], seed=3, wide=512)]
    xs = [torch.randn(64, 2048, device="cuda") for _ in range(2)]
    w = torch.ones(2048, device="cuda")
    want = [bg.paged_attention(q, c, *b.on_gpu()) for b, c, q in sets] + [bg.rms_norm_int8(x, w)[0] for x in xs]
    batches = [b.on_gpu() for b, _, _ in sets]
    torch.cuda.synchronize()
    say("two streams")
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for i, st in enumerate(streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            for _ in range(5):
                got[i].append([bg.paged_attention(q, c, *bt) for (_, c, q), bt in zip(sets, batches)]
                              + [bg.rms_norm_int8(x, w)[0] for x in xs])
    torch.cuda.synchronize()
    for g in got[0] + got[1]:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


@pytest.mark.parametrize("k", [640, 8320])
def test_norm_guard(k):
    lib, t = bg.load_library(), 7
    x, res, w = torch.randn(t, k, device="cuda"), torch.randn(t, k, device="cuda").bfloat16(), torch.ones(k, device="cuda")
    q, s, r = Guarded((t, k), torch.int8), Guarded((t,), torch.float32), Guarded((t, k), torch.bfloat16)
    say(f"guard rms_norm_int8 k={k}")
    _ok(lib.rms_norm_int8(_p(x), 1, _p(res), 0, _p(w), 1, t, k, 1e-5, r.ptr(), q.ptr(), s.ptr(), _st()), "rms_norm_int8")
    for g, n in ((q, "qx"), (s, "sx"), (r, "residual_out")):
        g.check(n)
    q2, s2, r2 = bg.rms_norm_int8(x, w, 1e-5, res)
    assert torch.equal(q.t, q2) and torch.equal(s.t, s2) and torch.equal(r.t, r2)


@pytest.mark.parametrize("bits,sym", [(4, False), (8, True)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_cache_and_attention_guard(d, bits, sym):
    """Pool tensors, read outputs, attention's output, lse and workspace, each
    between canaries, over every launch form."""
    lib, page, heads = bg.load_library(), 16, 2
    b = Batch([(300, 20), (33, 1), (1300, 1), (5, 5), (40, 1)], page, np.random.default_rng(d), spare=0, wide=512)
    row = d * bits // 8
    meta = (b.pages, heads, page)
    g = {"k_codes": Guarded((*meta, row), torch.uint8),
         "v_codes": Guarded((b.pages, heads, page // 4, row, 4), torch.uint8)}
    for n in ("k_scales", "v_scales") + (() if sym else ("k_zeros", "v_zeros")):
        g[n] = Guarded(meta, torch.float32)
    z = lambda n: g[n].t if n in g else None  # noqa: E731
    c = bg.KVCache(g["k_codes"].t, g["v_codes"].t, g["k_scales"].t, g["v_scales"].t, z("k_zeros"), z("v_zeros"), d, bits)
    full = Batch.__new__(Batch)
    full.__dict__.update(b.__dict__)
    full.starts = [0]
    for n in b.kv:
        full.starts.append(full.starts[-1] + n)
    rows = full.starts[-1]
    k, v = torch.randn((2, rows, heads, d), device="cuda")
    say(f"guard cache D={d} bits={bits} sym={sym}")
    bg.kv_cache_write(k, v, c, *full.on_gpu())
    for n, t in g.items():
        t.check(n)
    ko, vo = Guarded((rows, heads, d), torch.bfloat16), Guarded((rows, heads, d), torch.bfloat16)
    bg.kv_cache_read(c, *full.on_gpu(), rows=rows, k=ko.t, v=vo.t)
    ko.check("read k")
    vo.check("read v")
    qh = 3 * heads
    q = torch.randn((b.rows, qh, d), device="cuda").bfloat16()
    ref = None
    for hints in ((0, 0), (20, 1300), (1, 1300), (1, 1), (3, 0), (1000, 1 << 20)):
        batch = b.on_gpu()
        need = bg.paged_attention_workspace(b.rows, qh, c, len(b.kv), batch[0].shape[1], *hints)
        ws, out, lse = Guarded((max(need, 256),), torch.uint8), Guarded((b.rows, qh, d), torch.bfloat16), Guarded(
            (b.rows, qh), torch.float32)
        say(f"  attention hints {hints} workspace {need}")
        st = lib.paged_attention(c._ref, _p(q), b.rows, qh, qh * d, ctypes.c_float(d ** -0.5), _p(batch[0]),
                                 batch[0].shape[1], _p(batch[1]), _p(batch[2]), len(b.kv), *hints, ws.ptr(), need,
                                 out.ptr(), lse.ptr(), _st())
        _ok(st, "paged_attention")
        for t, n in ((ws, "workspace"), (out, "out"), (lse, "lse")):
            t.check(n)
        assert bool(torch.isfinite(out.t.float()).all()) and bool(torch.isfinite(lse.t).all())
        ref = out.t.clone() if ref is None else ref
        # another order of sums and other tiles' powers of two: the fp16 weights
        # and the bf16 result may round the other way, 2^-10 + 2^-8 of the values
        assert float((out.t.float() - ref.float()).abs().max()) <= (2.0 ** -10 + 2.0 ** -8) * 5
    for n, t in g.items():
        t.check(n + " after attention")


def test_chunks_and_single_tokens_agree_with_one_prompt():
    """The same 75 tokens as one prompt, in three chunks and token by token:
    each within the bound of the one 64-bit result; the cache's bytes equal."""
    rng = np.random.default_rng(4)
    n, heads, group, d = 75, 2, 4, 64
    b = Batch([(n, n)], 16, rng)
    x = bf16(rng.standard_normal((2, n, heads, d)))
    q = bf16(rng.standard_normal((n, heads * group, d)))
    ref = new_cache(b, 16, heads, d, 8, True)
    for t in range(n):
        ref.put_rows(b.lists[0][t // 16], t % 16, "k", x[0, t])
        ref.put_rows(b.lists[0][t // 16], t % 16, "v", x[1, t])
    want, want_lse, bound = serving.attention(q, ref, b.lists, [n], [0, n], d ** -0.5)
    kd, vd, qd = dev_bf16f(x[0]), dev_bf16f(x[1]), dev_bf16f(q)
    table = b.on_gpu()[0]
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for cuts in ([n], [31, 64, n], list(range(1, n + 1))):
        c = to_gpu(new_cache(b, 16, heads, d, 8, True))
        out, at = torch.empty_like(qd), 0
        say(f"{len(cuts)} calls")
        for to in cuts:
            batch = (table, i32(to), i32(0, to - at))
            bg.kv_cache_write(kd[at:to], vd[at:to], c, *batch)
            out[at:to] = bg.paged_attention(qd[at:to], c, *batch, max_rows=to - at)
            at = to
        assert_same_bits(host(c.k_codes), ref.k_codes, "k_codes")
        assert_same_bits(host(c.v_codes), ref.v_codes, "v_codes")
        check_attention(out, None, want, want_lse, bound, f"{len(cuts)} calls")


def test_attention_half_of_a_w8a8_layer():
    """Norm into INT8, the fused q|k|v product, the cache written from slices of
    its fp32 rows, attention, per-token INT8, the output product and the next
    norm with the residual: every step against its oracle on the step's own
    inputs, for a ragged batch of prompts and then a decode step."""
    rng = np.random.default_rng(5)
    hidden, heads, group, d = 512, 2, 2, 128
    qh = heads * group
    wqkv = dev_bf16f(bf16(rng.standard_normal(((qh + 2 * heads) * d, hidden)) * 0.05))
    wo = dev_bf16f(bf16(rng.standard_normal((hidden, qh * d)) * 0.05))
    pq, po = bg.quantize_groupwise(wqkv, 8, True, hidden), bg.quantize_groupwise(wo, 8, True, qh * d)
    norm_w = bf16(1 + 0.1 * rng.standard_normal(hidden))
    final = Batch([(41, 1), (18, 1), (70, 1)], 16, rng)
    ref = new_cache(final, 16, heads, d, 8, True)
    cache = to_gpu(ref)
    for step in ("prompts", "decode"):
        held = [n - 1 for n in final.kv] if step == "prompts" else final.kv
        new = held if step == "prompts" else [1, 1, 1]
        starts = np.cumsum([0] + new).astype(np.int32)
        rows = int(starts[-1])
        batch = (final.on_gpu()[0], dev(np.asarray(held, np.int32)), dev(starts))
        x, res = rng.standard_normal((rows, hidden)).astype(np.float32), bf16(rng.standard_normal((rows, hidden)))
        say(f"layer {step}: {rows} rows")
        qx, sx, res1 = bg.rms_norm_int8(dev(x), dev_bf16f(norm_w), 1e-5, dev_bf16f(res))
        oq, osx, _, _ = serving.rms_norm_int8(x, norm_w, 1e-5, res)
        assert_same_bits(host(qx), oq, "norm codes")
        assert_same_bits(host(sx), osx, "norm scales")
        qkv, acc = bg.w8a8_gemm(qx, sx, pq.codes.view(torch.int8), pq.scales.view(-1), want_acc=True)
        assert_same_bits(host(acc), oracle.w8a8_gemm(oq, osx, host(pq.codes).view(np.int8), host(pq.scales)[:, 0])[0], "qkv")
        kv = qkv.view(rows, -1, d)
        bg.kv_cache_write(kv[:, qh:qh + heads], kv[:, qh + heads:], cache, *batch)
        hkv = host(qkv).reshape(rows, -1, d)
        for i in range(3):
            for r in range(starts[i], starts[i + 1]):
                pos = held[i] - int(starts[i + 1] - r)
                ref.put_rows(final.lists[i][pos // 16], pos % 16, "k", hkv[r, qh:qh + heads])
                ref.put_rows(final.lists[i][pos // 16], pos % 16, "v", hkv[r, qh + heads:])
        for n in ("k_codes", "v_codes", "k_scales", "v_scales"):
            assert_same_bits(host(getattr(cache, n)), getattr(ref, n), n)
        q = kv[:, :qh].bfloat16()
        out = bg.paged_attention(q, cache, *batch)
        want, wl, bound = serving.attention(q.float().cpu().numpy(), ref, final.lists, held, list(starts), d ** -0.5)
        check_attention(out, None, want, wl, bound, step)
        flat = out.view(rows, -1)
        qa, sa = bg.quant_per_token_int8(flat)
        oqa, osa = oracle.quant_per_token_int8(host(flat.view(torch.int16)).view(np.uint16))
        assert_same_bits(host(qa), oqa, "attention codes")
        y, _ = bg.w8a8_gemm(qa, sa, po.codes.view(torch.int8), po.scales.view(-1))
        q2, s2, _ = bg.rms_norm_int8(y, dev_bf16f(norm_w), 1e-5, res1, res1)
        r1 = bf16(x + res)
        o2, os2, h2, _ = serving.rms_norm_int8(host(y), norm_w, 1e-5, r1)
        assert_same_bits(host(q2), o2, "second norm codes")
        assert_same_bits(host(s2), os2, "second norm scales")
        assert_same_bits(host(res1.float()), bf16(h2), "residual")


def test_calls_refuse_another_devices_tensors():
    """Tensors on the CPU among GPU ones are named."""
    c = bg.KVCache.empty(2, 16, 1, 64)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    k = torch.zeros((1, 1, 64), device="cuda")
    with pytest.raises(ValueError, match="kv_lens"):
        bg.kv_cache_write(k, k, c, z(1, 1), torch.zeros(1, dtype=torch.int32), z(2))
    with pytest.raises(ValueError, match="q is on"):
        bg.paged_attention(torch.zeros((1, 2, 64), dtype=torch.bfloat16), c, z(1, 1), z(1), z(2))
    with pytest.raises(TypeError, match="q must be"):
        bg.paged_attention(torch.zeros((1, 2, 64), device="cuda"), c, z(1, 1), z(1), z(2))
    with pytest.raises(ValueError, match="row_starts"):
        bg.kv_cache_read(c, z(1, 1), z(1), z(1), rows=1)
    with pytest.raises(bg.LibquantError, match="multiple of heads"):
        c3 = bg.KVCache.empty(2, 16, 3, 64)
        bg.paged_attention(torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda"), c3, z(1, 1), z(1), z(2))
    with pytest.raises(ValueError, match="contiguous"):
        bg.kv_cache_write(torch.zeros((1, 1, 128), device="cuda")[..., ::2], k, c, z(1, 1), z(1), z(2))

"""kv_cache_write and kv_cache_read against the oracle: every byte of the pool
(written slots bit for bit, all others as they were) and the values read."""
import numpy as np
import pytest
import torch

import bit_gemv_amd as bg
from gpu_helpers import assert_same_bits, dev, host, say
from oracle import serving
from serving_helpers import Batch, bf16, dev_bf16f, fill, new_cache, to_gpu

pytestmark = pytest.mark.gpu

FORMATS = [(4, False), (4, True), (8, False), (8, True)]
# tokens held, new rows: single tokens at each place of a quad, chunks that
# start and end inside quads and pages, more rows than tokens, none
SEQS = [(1, 1), (2, 1), (3, 1), (64, 1), (17, 16), (16, 16), (33, 5), (50, 50), (39, 2), (3, 6), (0, 3), (20, 0)]


def _same_pool(gpu, ref, what):
    for n in ("k_codes", "v_codes", "k_scales", "v_scales", "k_zeros", "v_zeros"):
        if getattr(ref, n) is not None:
            assert_same_bits(host(getattr(gpu, n)), getattr(ref, n), f"{what} {n}")


def _run(d, bits, sym, page, heads, seqs, kind, seed, max_rows=0, gap=0, scale=1.0, lead=0, offset=0.0):
    rng = np.random.default_rng(seed)
    b = Batch(seqs, page, rng, lead=lead)
    ref = new_cache(b, page, heads, d, bits, sym)
    fill(ref, b, rng, skip_new=True)
    gpu = to_gpu(ref)
    rows = b.rows + 2                                       # two rows behind the last sequence
    x = rng.standard_normal((2, rows, heads, d)).astype(np.float32) * np.float32(scale) + np.float32(offset)
    if kind == "bf16":
        x = bf16(x)
    wide = torch.empty((rows, 2 * heads + gap, d), dtype=torch.bfloat16 if kind == "bf16" else torch.float32,
                       device="cuda").fill_(float("nan"))
    wide[:, :heads], wide[:, heads:2 * heads] = dev(x[0]).to(wide.dtype), dev(x[1]).to(wide.dtype)
    say(f"kv_cache D={d} bits={bits} sym={sym} page={page} heads={heads} {kind} gap={gap} max_rows={max_rows}")
    batch = b.on_gpu()
    bg.kv_cache_write(wide[:, :heads], wide[:, heads:2 * heads], gpu, *batch, max_rows=max_rows)
    for r, i, pos in b.positions():
        if pos >= 0:
            for s, side in enumerate("kv"):
                ref.put_rows(b.lists[i][pos // page], pos % page, side, x[s, r])
    _same_pool(gpu, ref, "after the write")
    for dtype in (torch.float32, torch.bfloat16):
        k = torch.full((rows, heads, d), 7.0, dtype=dtype, device="cuda")
        v = torch.full_like(k, 7.0)
        bg.kv_cache_read(gpu, *batch, rows=rows, dtype=dtype, max_rows=max_rows, k=k, v=v)
        for s, got in enumerate((k, v)):
            want = np.full((rows, heads, d), 7.0, np.float32)
            for r, i, pos in b.positions():
                want[r] = serving.kv_dequantize(*serving.kv_quantize(x[s, r], bits, sym), bits) if pos >= 0 else 0.0
            if dtype == torch.bfloat16:
                want = bf16(want)
            assert_same_bits(host(got.float()), want, f"read {dtype} {'kv'[s]}")


@pytest.mark.parametrize("bits,sym", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_formats(d, bits, sym, kind):
    _run(d, bits, sym, 16, 2, SEQS, kind, d + bits)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("heads", [1, 3, 8])
def test_pages_and_heads(page, heads):
    _run(64, 8, True, page, heads, [(300, 1), (257, 257), (19, 7)], "bf16", page + heads)
    _run(64, 4, False, page, heads, [(300, 1), (257, 257), (19, 7)], "bf16", page + heads)


@pytest.mark.parametrize("max_rows", [1, 3, 50, 1000])
def test_hint_changes_nothing(max_rows):
    _run(128, 4, False, 16, 2, SEQS, "bf16", 11, max_rows=max_rows)


@pytest.mark.parametrize("max_rows", [0, 90])
def test_one_chunk_among_many_single_tokens(max_rows):
    """Enough sequences for the flat grid, past 64 of them."""
    seqs = [(5 + i, 1) for i in range(70)] + [(100, 90), (3, 5), (0, 1), (30, 0), (33, 1)] + [(7, 2)] * 60
    _run(64, 8, True, 16, 1, seqs, "bf16", 17, max_rows=max_rows)
    _run(64, 4, False, 32, 3, seqs, "fp32", 18, max_rows=max_rows, lead=2)


def test_rows_apart_and_leading_rows():
    """k and v as slices of a fused product's rows; rows before the first sequence."""
    _run(128, 8, True, 16, 2, SEQS, "fp32", 12, gap=5)
    _run(128, 4, True, 16, 2, SEQS, "bf16", 13, gap=3, lead=4)


@pytest.mark.parametrize("bits,sym", FORMATS)
@pytest.mark.parametrize("scale,offset", [(0.0, 0.0), (0.0, 2.5), (1e-12, 0.0), (1e12, 0.0), (0.01, 50.0), (1.0, -9.0),
                                          (1e25, 0.0)])
def test_magnitudes(bits, sym, scale, offset):
    """Constant vectors, vectors that do not span zero, tiny and huge ones."""
    _run(64, bits, sym, 16, 1, [(21, 21)], "fp32", 14, scale=scale, offset=offset)


def test_rounding_ties():
    """Values on half codes of a scale that is a power of two."""
    d = 64
    x = (np.arange(d, dtype=np.float32) - 32) / 2 + 0.5
    x[0], x[1] = 127, -127
    for bits, top in ((8, 127.0), (4, 7.0)):
        y = np.clip(x, -top, top)[None, None].repeat(4, 0)
        b = Batch([(4, 4)], 16, np.random.default_rng(0))
        ref = new_cache(b, 16, 1, d, bits, True)
        gpu = to_gpu(ref)
        say(f"kv_cache ties bits={bits}")
        bg.kv_cache_write(dev_bf16f(y), dev_bf16f(y), gpu, *b.on_gpu())
        for t in range(4):
            ref.put_rows(b.lists[0][0], t, "k", y[t])
            ref.put_rows(b.lists[0][0], t, "v", y[t])
        _same_pool(gpu, ref, f"ties bits={bits}")


def test_pages_outside_the_pool():
    """Rows in such pages are dropped, read as zeros, and nothing else moves."""
    rng = np.random.default_rng(15)
    b = Batch([(40, 40), (20, 20)], 16, rng)
    ref = new_cache(b, 16, 2, 64, 8, True)
    fill(ref, b, rng)
    gpu = to_gpu(ref)
    x = bf16(rng.standard_normal((60, 2, 64)))
    for bad in (-1, -(1 << 31), b.pages, (1 << 31) - 1):
        table = b.table.copy()
        table[0, 1] = bad
        batch = (dev(table), *b.on_gpu()[1:])
        say(f"kv_cache page {bad}")
        bg.kv_cache_write(dev_bf16f(x), dev_bf16f(x), gpu, *batch)
        for r, i, pos in b.positions():
            if not (i == 0 and 16 <= pos < 32):
                for side in "kv":
                    ref.put_rows(b.lists[i][pos // 16], pos % 16, side, x[r])
        _same_pool(gpu, ref, f"page {bad}")
        k, v = bg.kv_cache_read(gpu, *batch, rows=60)
        assert float(k[16:32].abs().max()) == 0 and float(v[16:32].abs().max()) == 0
        assert float(k[:16].abs().min(-1).values.max()) > 0 or float(k[:16].abs().max()) > 0


def test_lengths_past_the_table_and_odd_starts():
    """Lengths and starts that do not fit the tensors touch nothing outside."""
    rng = np.random.default_rng(16)
    b = Batch([(30, 5), (9, 4)], 16, rng)
    ref = new_cache(b, 16, 1, 64, 8, True)
    fill(ref, b, rng)
    x = dev_bf16f(rng.standard_normal((9, 1, 64)))
    for kv, starts in (([1 << 30, 9], [0, 5, 9]), ([-5, 9], [0, 5, 9]), ([30, 9], [-7, 5, 9]), ([30, 9], [0, 5, 1 << 30]),
                       ([30, 9], [9, 5, 0])):
        gpu = to_gpu(ref)
        batch = (b.on_gpu()[0], dev(np.asarray(kv, np.int32)), dev(np.asarray(starts, np.int32)))
        say(f"kv_cache kv={kv} starts={starts}")
        bg.kv_cache_write(x, x, gpu, *batch)
        bg.kv_cache_read(gpu, *batch, rows=9)
        torch.cuda.synchronize()
        spare = [p for p in range(b.pages) if p not in b.lists[0] + b.lists[1]]
        assert bool(torch.isnan(gpu.k_scales[spare]).all())


def test_large_offsets():
    """A pool past 4 GiB of codes: the last page is addressed beyond 32 bits."""
    pages, heads, d, page = 70000, 8, 128, 64
    if torch.cuda.mem_get_info()[0] < 14 << 30:
        pytest.skip("needs 14 GiB of GPU memory")
    gpu = bg.KVCache.empty(pages, page, heads, d)
    assert gpu.k_codes.numel() > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((130, heads, d), generator=g, device="cuda")
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    lens, starts = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([130], [0, 130]))
    say("kv_cache large offsets")
    bg.kv_cache_write(x, -x, gpu, table, lens, starts)
    k, v = bg.kv_cache_read(gpu, table, lens, starts, rows=130, dtype=torch.float32)
    s = x.abs().amax(-1, keepdim=True)
    # half a step of the code, and the fp32 rounding of code and product
    assert bool(((k - x).abs() <= s / 127 * 0.5 + s * 2.0 ** -22).all())
    assert torch.equal(v, -k)
    # attention over those pages: the bits of the same pages in a small pool
    at = [pages - 1, 3, pages - 2]
    small = bg.KVCache(*(t[at].clone() for t in (gpu.k_codes, gpu.v_codes, gpu.k_scales, gpu.v_scales)), None, None, d, 8)
    tiny = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    q = torch.randn((130, 2 * heads, d), generator=g, device="cuda").bfloat16()
    for n in (130, 1):
        s1 = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        assert torch.equal(bg.paged_attention(q[:n], gpu, table, lens, s1), bg.paged_attention(q[:n], small, tiny, lens, s1))


def test_empty_calls():
    gpu = bg.KVCache.empty(2, 16, 1, 64)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    none = torch.empty((0, 1, 64), device="cuda")
    bg.kv_cache_write(none, none, gpu, z(0, 1), z(0), z(1))
    bg.kv_cache_write(none, none, gpu, z(2, 1), z(2), z(3))
    k, v = bg.kv_cache_read(gpu, z(2, 1), z(2), z(3), rows=0)
    assert k.shape == v.shape == (0, 1, 64)

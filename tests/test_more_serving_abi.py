"""CPU checks of the calls beside paged_attention over the cache: arguments are
refused before any HIP call."""
import ctypes

import pytest
import torch

import bit_gemv_amd as bg
from test_serving_abi import CACHE_REFUSALS, MIS, NO_GPU, A, B, C, D, E, F, G, H, I, J, K, P, _cache

L, M, N = (P((i + 20) << 32) for i in range(3))


@pytest.fixture(scope="module")
def lib():
    return bg.load_library()


def _cross(lib, q=E, rows=4, qh=8, qs=1024, scale=0.1, table=G, mp=3, lens=H, starts=I, b=2, mr=0, mk=0, ws=K,
           wsb=1 << 31, out=F, lse=None, **kw):
    c = _cache(**kw)
    return lib.cross_attention(ctypes.byref(c), q, rows, qh, qs, scale, table, mp, lens, starts, b, mr, mk, ws, wsb, out, lse,
                               None)


def _prefix(lib, q=E, rows=4, qh=8, qs=1024, scale=0.1, pt=L, pp=5, pl=M, ps=N, p=1, mpr=0, mpk=0, table=G, mp=3, lens=H,
            starts=I, b=2, mr=0, mk=0, ws=K, wsb=1 << 31, out=F, lse=None, **kw):
    c = _cache(**kw)
    return lib.prefix_attention(ctypes.byref(c), q, rows, qh, qs, scale, pt, pp, pl, ps, p, mpr, mpk, table, mp, lens, starts,
                                b, mr, mk, ws, wsb, out, lse, None)


BATCH_REFUSALS = [
    (dict(rows=-1), 1), (dict(b=-1), 1), (dict(mp=-1), 1), (dict(mr=-1), 1), (dict(b=65536), 2), (dict(mp=1 << 30), 2),
    (dict(table=None), 1), (dict(lens=None), 1), (dict(starts=None), 1), (dict(starts=P((9 << 32) + 2)), 1),
]


@pytest.mark.parametrize("call", [_cross, _prefix])
@pytest.mark.parametrize("kwargs,status", CACHE_REFUSALS + BATCH_REFUSALS + [
    (dict(qh=7), 1), (dict(qh=0), 1), (dict(qs=1023), 1), (dict(qs=512), 1), (dict(mk=-1), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(q=None), 1), (dict(q=MIS), 1), (dict(out=None), 1), (dict(out=MIS), 1), (dict(lse=P((12 << 32) + 2)), 1),
    (dict(out=E), 1), (dict(out=A), 1), (dict(lse=F), 1), (dict(out=G), 1), (dict(qh=1 << 17, qs=1 << 24), 2),
    (dict(rows=(1 << 30) + 1, qh=1, qs=128, heads=1), 2),
])
def test_attention_calls_refuse(lib, call, kwargs, status):
    assert call(lib, **kwargs) == status
    assert lib.lq_last_error() != b""


@pytest.mark.parametrize("kwargs,status", [
    (dict(p=-1), 1), (dict(pp=-1), 1), (dict(mpr=-1), 1), (dict(mpk=-1), 1), (dict(p=65536), 2), (dict(pp=1 << 30), 2),
    (dict(pt=None), 1), (dict(pl=None), 1), (dict(ps=None), 1), (dict(ps=P((9 << 32) + 2)), 1), (dict(out=L), 1),
    (dict(out=M), 1), (dict(lse=N), 1), (dict(ws=L), 1), (dict(ws=None), 1), (dict(ws=MIS), 1), (dict(wsb=100), 1),
])
def test_prefix_refuses(lib, kwargs, status):
    assert _prefix(lib, **kwargs) == status
    assert lib.lq_last_error() != b""


@pytest.mark.parametrize("call", [_cross, _prefix])
def test_attention_calls_empty_and_no_device(lib, call):
    assert call(lib, rows=0, table=None, lens=None, starts=None) == 0
    assert call(lib, b=0, table=None, lens=None, starts=None) == 0
    if NO_GPU:
        assert call(lib) == 4
        assert call(lib, mp=0, table=None) == 4
        assert call(lib, symmetric=0, k_zeros=J, v_zeros=P(13 << 32), bits=4, head_dim=64) == 4


def test_attention_workspaces(lib):
    f, g = lib.cross_attention_workspace_bytes, lib.prefix_attention_workspace_bytes
    for bad in ((-1, 8, 2, 128, 2, 3, 16, 0, 0), (4, 7, 2, 128, 2, 3, 16, 0, 0), (4, 8, 2, 128, -1, 3, 16, 0, 0),
                (4, 8, 2, 128, 2, 3, 16, -1, 0), (4, 8, 2, 128, 2, 3, 0, 0, 0), ((1 << 30) + 1, 1, 1, 128, 2, 3, 16, 0, 0)):
        assert f(*bad) == -1
        rows, qh, h, d, b, mp, ps, mr, mk = bad
        assert g(rows, qh, h, d, ps, 1, 3, 0, 0, b, mp, mr, mk) == -1
    for bad in ((-1, 3, 0, 0), (1, -1, 0, 0), (1, 3, -1, 0), (1, 3, 0, -1), (65536, 3, 0, 0), (1, 1 << 30, 0, 0)):
        assert g(4, 8, 2, 128, 16, *bad, 2, 3, 0, 0) == -1
    assert f(0, 8, 2, 128, 2, 3, 16, 0, 0) == 0 and g(0, 8, 2, 128, 16, 1, 3, 0, 0, 2, 3, 0, 0) == 0
    need = f(1, 8, 1, 128, 1, 1024, 16, 1, 0)
    assert need > 0                              # one row over a long input is split
    c = dict(rows=1, qh=8, heads=1, mp=1024, b=1, mr=1, pages=2048)
    assert _cross(lib, **c, wsb=need - 1) == 1 and _cross(lib, **c, ws=None) == 1 and _cross(lib, **c, ws=E) == 1
    # without a prefix the call is paged_attention's, workspace included
    sizes = (3, 8, 1, 128, 2, 1024, 16, 0, 0)
    assert g(3, 8, 1, 128, 16, 0, 0, 0, 0, 2, 1024, 0, 0) == lib.paged_attention_workspace_bytes(*sizes)
    if NO_GPU:
        assert _prefix(lib, p=0, pt=None, pl=None, ps=None, mp=0, table=None, ws=None, wsb=0) == 4


def _weigh(lib, q=E, rows=4, qh=8, qs=1024, scale=0.1, lse=F, table=G, mp=3, lens=H, starts=I, b=2, causal=1, mr=0, mk=0,
           w=K, out=K, ws=N, wsb=1 << 31, **kw):
    c = _cache(**kw)
    return lib.kv_cache_weigh(ctypes.byref(c), q, rows, qh, qs, scale, lse, table, mp, lens, starts, b, causal, mr, mk, w, out,
                              ws, wsb, None)


@pytest.mark.parametrize("kwargs,status", CACHE_REFUSALS + BATCH_REFUSALS + [
    (dict(qh=7), 1), (dict(qh=0), 1), (dict(qs=1023), 1), (dict(qs=512), 1), (dict(qs=1 << 50), 2), (dict(mk=-1), 1),
    (dict(scale=float("nan")), 1), (dict(causal=2), 1), (dict(causal=-1), 1), (dict(q=None), 1), (dict(q=MIS), 1),
    (dict(lse=None), 1), (dict(lse=P((12 << 32) + 2)), 1), (dict(w=MIS), 1), (dict(out=None), 1), (dict(out=MIS), 1),
    (dict(out=A), 1), (dict(out=C), 1), (dict(out=E), 1), (dict(out=F), 1), (dict(out=G), 1), (dict(out=H), 1),
    (dict(out=P((11 << 32) + 256)), 1),         # partly over the weights
    (dict(rows=(1 << 30) + 1, qh=1, qs=128, heads=1), 2),
])
def test_weigh_refuses(lib, kwargs, status):
    assert _weigh(lib, **kwargs) == status
    assert lib.lq_last_error() != b""


def test_weigh_workspace(lib):
    f = lib.kv_cache_weigh_workspace_bytes
    for bad in ((-1, 8, 2, 128, 2, 3, 16, 0, 0), (4, 7, 2, 128, 2, 3, 16, 0, 0), (4, 8, 2, 128, -1, 3, 16, 0, 0),
                (4, 8, 2, 128, 2, 3, 16, -1, 0), (4, 8, 2, 128, 2, 3, 0, 0, 0), ((1 << 30) + 1, 1, 1, 128, 2, 3, 16, 0, 0)):
        assert f(*bad) == -1
    assert f(0, 8, 2, 128, 2, 3, 16, 0, 0) == 0 and f(4, 8, 2, 128, 2, 0, 16, 0, 0) == 0
    assert f(1000, 8, 8, 128, 1000, 100, 16, 1, 0) == 0         # single rows: no sums to add up
    need = f(400, 8, 1, 128, 1, 64, 16, 0, 0)                    # 4 steps of 256 keys, 25 runs of 128 rows
    assert need == 4 * 25 * 256 * 4
    c = dict(rows=400, qh=8, heads=1, mp=64, b=1, pages=2048)
    assert _weigh(lib, **c, wsb=need - 1) == 1 and _weigh(lib, **c, ws=None) == 1 and _weigh(lib, **c, ws=MIS) == 1
    assert _weigh(lib, **c, ws=E) == 1 and _weigh(lib, **c, ws=K) == 1 and _weigh(lib, **c, ws=K, out=L) == 1
    if NO_GPU:
        assert _weigh(lib, **c, wsb=need) == 4


def test_weigh_empty_and_no_device(lib):
    assert _weigh(lib, rows=0, table=None, lens=None, starts=None) == 0
    assert _weigh(lib, b=0, table=None, lens=None, starts=None) == 0
    assert _weigh(lib, mp=0, table=None) == 0
    if NO_GPU:
        for kw in (dict(), dict(w=None), dict(out=L), dict(causal=0), dict(symmetric=0, k_zeros=J, v_zeros=P(13 << 32))):
            assert _weigh(lib, **kw) == 4


def _evict(lib, w=E, table=G, mp=3, lens=H, b=2, keep=20, recent=4, to=None, tp=0, mk=0, kept=I, new=K, **kw):
    c = _cache(**kw)
    return lib.kv_cache_evict(ctypes.byref(c), w, table, mp, lens, b, keep, recent, to, tp, mk, kept, new, None)


@pytest.mark.parametrize("kwargs,status", CACHE_REFUSALS + [
    (dict(b=-1), 1), (dict(mp=-1), 1), (dict(b=65536), 2), (dict(mp=1 << 30), 2), (dict(mk=-1), 1),
    (dict(keep=0), 1), (dict(keep=-3), 1), (dict(recent=-1), 1), (dict(recent=21), 1), (dict(keep=1 << 31), 2),
    (dict(b=65535, heads=128, pages=1), 2),
    (dict(table=None), 1), (dict(lens=None), 1), (dict(lens=P((9 << 32) + 2)), 1), (dict(w=None), 1), (dict(w=MIS), 1),
    (dict(kept=None), 1), (dict(new=None), 1), (dict(new=P((9 << 32) + 2)), 1),
    (dict(to=L, tp=1), 1),                      # room for 16 of 20 tokens
    (dict(to=L, tp=-1), 1), (dict(to=L, tp=1 << 30), 2), (dict(to=P((9 << 32) + 2), tp=3), 1),
    (dict(kept=G), 1), (dict(kept=H), 1), (dict(kept=K), 1), (dict(new=G), 1), (dict(w=A), 1), (dict(w=G), 1),
    (dict(new=P((8 << 32) + 4)), 1),            # partly over kv_lens
    (dict(to=L, tp=2, new=L), 1),
])
def test_evict_refuses(lib, kwargs, status):
    assert _evict(lib, **kwargs) == status
    assert lib.lq_last_error() != b""


def test_evict_empty_and_no_device(lib):
    assert _evict(lib, b=0, table=None, lens=None, w=None) == 0
    if NO_GPU:
        for kw in (dict(), dict(new=H), dict(to=L, tp=2), dict(mp=0, table=None), dict(keep=20, mp=1), dict(keep=1 << 20)):
            assert _evict(lib, **kw) == 4


def test_binding_refuses_tensors_on_the_cpu():
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    t = torch.zeros((1, 1), dtype=torch.int32)

    class Cache:
        _index, head_dim, heads, device, k_scales = 0, 64, 1, "cuda:0", torch.zeros((1, 1, 16))

    for call in (lambda: bg.cross_attention(q, Cache, t, t[0], t[0]),
                 lambda: bg.kv_cache_weigh(q, q[..., 0].float(), Cache, None, t, t[0], t[0]),
                 lambda: bg.kv_cache_evict(Cache, Cache.k_scales, t, t[0], 4),
                 lambda: bg.prefix_attention(q, Cache, t, t[0], t[0], t, t[0], t[0])):
        with pytest.raises(ValueError, match="GPU|the cache"):
            call()
    for bad in (lambda: bg.kv_cache_evict(Cache, q, t[0], t[0], 4), lambda: bg.prefix_attention(q, Cache, t[0], t, t, t, t, t)):
        with pytest.raises(ValueError, match="must be a tensor"):
            bad()

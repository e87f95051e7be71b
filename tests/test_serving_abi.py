"""CPU checks of the serving entry points: arguments are refused before any
HIP call, and the binding's own checks name what is wrong."""
import ctypes

import pytest
import torch

import bit_gemv_amd as bg

P = ctypes.c_void_p
A, B, C, D, E, F, G, H, I, J, K = (P((i + 1) << 32) for i in range(11))  # 16-byte-aligned fake addresses
MIS = P((12 << 32) + 8)
NO_GPU = torch.cuda.device_count() == 0


@pytest.fixture(scope="module")
def lib():
    return bg.load_library()


def _norm(lib, x=A, xt=0, res=B, rt=0, w=C, wt=0, t=4, k=256, eps=1e-5, ro=D, qx=E, sx=F):
    return lib.rms_norm_int8(x, xt, res, rt, w, wt, t, k, eps, ro, qx, sx, None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(xt=2), 1), (dict(wt=-1), 1), (dict(rt=7), 1),
    (dict(t=-1), 1), (dict(k=0), 1), (dict(k=200), 2),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(x=None), 1), (dict(x=MIS), 1), (dict(w=None), 1), (dict(w=MIS), 1), (dict(res=MIS), 1), (dict(ro=MIS), 1),
    (dict(qx=None), 1), (dict(sx=None), 1),
    (dict(res=None), 1),                        # residual_out without residual
    (dict(ro=P((2 << 32) + 256)), 1),           # residual_out partly over residual
    (dict(ro=A), 1), (dict(qx=A), 1), (dict(qx=B), 1), (dict(sx=E), 1), (dict(qx=D), 1),
    (dict(t=1 << 33, k=1 << 20), 2),
])
def test_norm_refuses(lib, kwargs, status):
    assert _norm(lib, **kwargs) == status
    assert lib.lq_last_error() != b""


def test_norm_empty_in_place_and_no_device(lib):
    assert _norm(lib, t=0, x=None, w=None, qx=None, sx=None, res=None, ro=None) == 0
    if NO_GPU:
        assert _norm(lib) == 4
        assert _norm(lib, ro=B) == 4            # residual updated in place
        assert _norm(lib, res=None, ro=None) == 4
        assert _norm(lib, ro=None) == 4


def _cache(**kw):
    f = dict(k_codes=A, v_codes=B, k_scales=C, k_zeros=None, v_scales=D, v_zeros=None, pages=8, page_size=16, heads=2,
             head_dim=128, bits=8, symmetric=1)
    f.update(kw)
    return bg._KvCacheRecord(*(f[n] for n, _ in bg._KvCacheRecord._fields_))


CACHE_REFUSALS = [
    (dict(bits=5), 1), (dict(bits=0), 1), (dict(pages=0), 1), (dict(heads=-1), 1), (dict(head_dim=0), 1),
    (dict(head_dim=96), 2), (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=512), 2),
    (dict(pages=1 << 31), 2), (dict(heads=1 << 20), 2),
    (dict(k_codes=None), 1), (dict(v_codes=MIS), 1), (dict(k_scales=MIS), 1), (dict(v_scales=None), 1),
    (dict(k_zeros=J), 1),                       # zeros of a symmetric cache
    (dict(symmetric=0), 1), (dict(symmetric=0, k_zeros=J), 1), (dict(symmetric=0, k_zeros=J, v_zeros=MIS), 1),
]


def _write(lib, cache=None, k=E, v=F, t=0, rows=4, ks=256, vs=256, table=G, mp=3, lens=H, starts=I, b=2, mr=0, **kw):
    c = _cache(**kw)
    return lib.kv_cache_write(ctypes.byref(c), k, v, t, rows, ks, vs, table, mp, lens, starts, b, mr, None)


def _read(lib, k=E, v=F, t=0, rows=4, table=G, mp=3, lens=H, starts=I, b=2, mr=0, **kw):
    c = _cache(**kw)
    return lib.kv_cache_read(ctypes.byref(c), k, v, t, rows, table, mp, lens, starts, b, mr, None)


def _attn(lib, q=E, rows=4, qh=8, qs=1024, scale=0.1, table=G, mp=3, lens=H, starts=I, b=2, mr=0, mk=0, ws=K,
          wsb=1 << 31, out=F, lse=None, **kw):
    c = _cache(**kw)
    return lib.paged_attention(ctypes.byref(c), q, rows, qh, qs, scale, table, mp, lens, starts, b, mr, mk, ws, wsb,
                               out, lse, None)


@pytest.mark.parametrize("call", [_write, _read, _attn])
@pytest.mark.parametrize("kwargs,status", CACHE_REFUSALS + [
    (dict(rows=-1), 1), (dict(b=-1), 1), (dict(mp=-1), 1), (dict(mr=-1), 1), (dict(b=65536), 2), (dict(mp=1 << 30), 2),
    (dict(table=None), 1), (dict(lens=None), 1), (dict(starts=None), 1), (dict(starts=P((9 << 32) + 2)), 1),
])
def test_cache_calls_refuse(lib, call, kwargs, status):
    assert call(lib, **kwargs) == status
    assert lib.lq_last_error() != b""


@pytest.mark.parametrize("call", [_write, _read, _attn])
def test_cache_calls_empty_and_no_device(lib, call):
    assert call(lib, rows=0, table=None, lens=None, starts=None) == 0
    assert call(lib, b=0, table=None, lens=None, starts=None) == 0
    if NO_GPU:
        assert call(lib) == 4
        assert call(lib, symmetric=0, k_zeros=J, v_zeros=P(13 << 32), bits=4, head_dim=64) == 4


def test_cache_null_record(lib):
    assert lib.kv_cache_write(None, E, F, 0, 4, 256, 256, G, 3, H, I, 2, 0, None) == 1


@pytest.mark.parametrize("kwargs,status", [
    (dict(t=2), 1), (dict(ks=255), 1), (dict(vs=260), 1), (dict(ks=128), 1), (dict(ks=1 << 50), 2),
    (dict(k=None), 1), (dict(v=MIS), 1), (dict(k=A), 1), (dict(v=C), 1), (dict(table=A), 1), (dict(v_codes=A), 1),
])
def test_write_refuses(lib, kwargs, status):
    assert _write(lib, **kwargs) == status


@pytest.mark.parametrize("kwargs,status", [
    (dict(t=2), 1), (dict(k=None, v=None), 1), (dict(k=MIS), 1), (dict(k=A), 1), (dict(v=E), 1), (dict(v=D), 1),
])
def test_read_refuses(lib, kwargs, status):
    assert _read(lib, **kwargs) == status


@pytest.mark.parametrize("kwargs,status", [
    (dict(qh=7), 1), (dict(qh=0), 1), (dict(qs=1023), 1), (dict(qs=512), 1), (dict(mk=-1), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(q=None), 1), (dict(q=MIS), 1), (dict(out=None), 1), (dict(out=MIS), 1), (dict(lse=P((12 << 32) + 2)), 1),
    (dict(out=E), 1), (dict(out=A), 1), (dict(lse=F), 1), (dict(qh=1 << 17, qs=1 << 24), 2),
])
def test_attention_refuses(lib, kwargs, status):
    assert _attn(lib, **kwargs) == status


def test_attention_workspace(lib):
    f = lib.paged_attention_workspace_bytes
    for bad in ((-1, 8, 2, 128, 2, 3, 16, 0, 0), (4, 7, 2, 128, 2, 3, 16, 0, 0), (4, 8, 2, 128, -1, 3, 16, 0, 0),
                (4, 8, 2, 128, 2, 3, 16, -1, 0), (4, 8, 2, 128, 2, 3, 0, 0, 0), (4, 8, 2, 512, 2, 3, 16, 0, 0)):
        assert f(*bad) == -1
    assert f(0, 8, 2, 128, 2, 3, 16, 0, 0) == 0
    need = f(1, 8, 1, 128, 1, 1024, 16, 1, 0)
    assert need > 0                              # one row over a long context is split
    c = dict(rows=1, qh=8, heads=1, mp=1024, b=1, mr=1, pages=2048)
    assert _attn(lib, **c, wsb=need - 1) == 1 and _attn(lib, **c, ws=None) == 1 and _attn(lib, **c, ws=MIS) == 1
    assert _attn(lib, **c, ws=E) == 1            # the workspace over q
    if NO_GPU:
        assert _attn(lib, **c, wsb=need) == 4


def test_binding_refuses_what_is_not_on_the_gpu():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        bg.rms_norm_int8(x, x[0])
    with pytest.raises(TypeError):
        bg.rms_norm_int8(None, x)
    with pytest.raises(ValueError, match="GPU"):
        bg.KVCache.empty(2, 16, 1, 64, device="cpu")
    with pytest.raises(ValueError, match="bits"):
        bg.KVCache(x, x, x, x, None, None, 64, 5)
    with pytest.raises(ValueError, match="together"):
        bg.KVCache(x, x, x, x, x, None, 64, 8)

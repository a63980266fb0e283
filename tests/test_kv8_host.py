"""Prompt attention and the 8-bit cache: what the calls refuse, before anything reaches a GPU (CPU),
and what their Python side refuses."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE, HIP = 0, 1, 2, 3, 4
P = ctypes.c_void_p(256)          # a non-null address that no refused call may touch
I2 = ctypes.c_int64 * 2
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def fk():
    import exact_means_clustering_flashassign_amd as mod

    mod.load()
    return mod


@pytest.fixture(scope="module")
def lib(fk):
    return fk.load()


def _cache(kind, **kw):
    from exact_means_clustering_flashassign_amd import _binding

    t = getattr(_binding, kind)
    d = dict(k=256, v=256, k_scale=256, v_scale=256, key_bias=None, pages=4, page=16, heads=2, dim=64,
             k_stride=(2048, 128, 64), v_stride=(2048, 128, 64), k_scale_stride=(32, 2, 1),
             v_scale_stride=(32, 2, 1), bias_stride=(32, 2, 1))
    d.update(kw)
    return t(*(d[n] for n, _ in t._fields_))


BAD_CACHES = [dict(pages=-1), dict(page=0), dict(pages=1 << 20, page=1 << 11), dict(k=None), dict(v=None),
              dict(heads=0), dict(dim=0), dict(k_stride=(-1, 128, 64)), dict(v_stride=(1 << 62, 128, 64)),
              dict(key_bias=256, bias_stride=(-1, 2, 1))]
BAD_CACHES8 = BAD_CACHES + [dict(k_scale=None), dict(v_scale=None), dict(k_scale_stride=(-1, 2, 1)),
                            dict(v_scale_stride=(32, 1 << 62, 1))]
BAD_ATTN = [dict(dt=-1), dict(dt=3), dict(B=-1), dict(Hq=0), dict(Hq=3), dict(cache=None), dict(ld=7),
            dict(width=-1), dict(max_len=-1), dict(scale=NAN), dict(scale=INF), dict(cap=-1.0), dict(cap=NAN),
            dict(cap=INF), dict(q=None), dict(lens=None), dict(out=None), dict(table=None), dict(qs=None),
            dict(qs=I2(-1, 64)), dict(qs=I2(1 << 62, 64))]


def test_prompt_attn_refusals(fk, lib):
    c = _cache("fk_kv_cache_t")
    need = lib.fk_workspace_size_prompt(1, 5, 3, 4, 2, 64)

    def call(**kw):
        d = dict(q=P, qs=I2(256, 64), dt=1, T=5, B=3, Hq=4, cache=ctypes.byref(c), table=P, ld=8, width=8,
                 lens=P, cu=P, max_len=0, scale=0.1, cap=0.0, out=P, lse=None, ws=P, wsb=need, stream=None)
        d.update(kw)
        return lib.fk_prompt_attn(*d.values())

    for bad in BAD_ATTN + [dict(T=-1), dict(T=1 << 31), dict(cu=None), dict(T=1 << 30, Hq=1 << 30)]:
        assert call(**bad) == INVALID, bad
    for bad in BAD_CACHES:
        b = _cache("fk_kv_cache_t", **bad)
        assert call(cache=ctypes.byref(b)) == INVALID, bad
    assert call(ws=None) == WORKSPACE and call(wsb=need - 1) == WORKSPACE
    assert call(ws=ctypes.c_void_p(264)) == WORKSPACE
    wide = _cache("fk_kv_cache_t", dim=1025, k_stride=(65600, 2050, 1025), v_stride=(65600, 2050, 1025))
    assert call(cache=ctypes.byref(wide)) == UNSUPPORTED
    assert call(T=0, q=None, lens=None, cu=None, out=None, ws=None, wsb=0) == OK
    assert call(B=0, q=None, lens=None, cu=None, out=None, ws=None, wsb=0) == OK
    for bad in [(5, 1, 1, 4, 2, 64), (1, -1, 1, 4, 2, 64), (1, 1, -1, 4, 2, 64), (1, 1, 1, 0, 2, 64),
                (1, 1, 1, 4, 3, 64), (1, 1, 1, 4, 0, 64), (1, 1, 1, 4, 2, 0)]:
        assert lib.fk_workspace_size_prompt(*bad) == 0, bad
    assert lib.fk_workspace_size_prompt(1, 0, 0, 4, 2, 64) >= 256


def test_store_and_load_refusals(fk, lib):
    c = _cache("fk_kv_cache8_t")

    def store(**kw):
        d = dict(k=P, ks=I2(128, 64), v=P, vs=I2(128, 64), dt=1, T=3, slots=P, cache=ctypes.byref(c), stream=None)
        d.update(kw)
        return lib.fk_kv_store8(*d.values())

    def load(**kw):
        d = dict(cache=ctypes.byref(c), slots=P, dt=1, T=3, ko=P, vo=P, stream=None)
        d.update(kw)
        return lib.fk_kv_load8(*d.values())

    for bad in [dict(dt=3), dict(T=-1), dict(T=1 << 31), dict(k=None), dict(v=None), dict(ks=None), dict(vs=None),
                dict(ks=I2(-1, 64)), dict(vs=I2(1 << 62, 64)), dict(slots=None), dict(cache=None)]:
        assert store(**bad) == INVALID, bad
    for bad in [dict(dt=-1), dict(T=-1), dict(T=1 << 31), dict(slots=None), dict(cache=None), dict(ko=None),
                dict(vo=None)]:
        assert load(**bad) == INVALID, bad
    for bad in BAD_CACHES8:
        b = ctypes.byref(_cache("fk_kv_cache8_t", **bad))
        assert store(cache=b) == INVALID and load(cache=b) == INVALID, bad
    assert store(T=0, k=None, v=None, slots=None) == OK and load(T=0, slots=None, ko=None, vo=None) == OK
    none = _cache("fk_kv_cache8_t", pages=0, k=None, v=None, k_scale=None, v_scale=None)
    assert store(cache=ctypes.byref(none)) == OK       # every slot is outside


def test_paged_attn8_refusals(fk, lib):
    c = _cache("fk_kv_cache8_t")
    need = lib.fk_workspace_size_attn8(1, 3, 4, 2, 64)

    def call(**kw):
        d = dict(q=P, qs=I2(256, 64), dt=1, B=3, Hq=4, cache=ctypes.byref(c), table=P, ld=8, width=8, lens=P,
                 max_len=0, scale=0.1, cap=0.0, out=P, lse=None, ws=P, wsb=need, stream=None)
        d.update(kw)
        return lib.fk_paged_attn8(*d.values())

    for bad in BAD_ATTN:
        assert call(**bad) == INVALID, bad
    for bad in BAD_CACHES8:
        b = _cache("fk_kv_cache8_t", **bad)
        assert call(cache=ctypes.byref(b)) == INVALID, bad
    assert call(ws=None) == WORKSPACE and call(wsb=need - 1) == WORKSPACE
    assert call(ws=ctypes.c_void_p(264)) == WORKSPACE
    wide = _cache("fk_kv_cache8_t", dim=1025, k_stride=(65600, 2050, 1025), v_stride=(65600, 2050, 1025))
    assert call(cache=ctypes.byref(wide)) == UNSUPPORTED
    assert call(B=0, q=None, lens=None, out=None, ws=None, wsb=0) == OK
    for bad in [(5, 1, 4, 2, 64), (1, -1, 4, 2, 64), (1, 1, 0, 2, 64), (1, 1, 4, 3, 64), (1, 1, 4, 0, 64),
                (1, 1, 4, 2, 0)]:
        assert lib.fk_workspace_size_attn8(*bad) == 0, bad


def test_without_a_gpu_valid_calls_report_an_error(fk, lib):
    """Arguments in order but no device: a status, not a crash."""
    import torch

    if torch.cuda.is_available():
        pytest.skip("the addresses here are made up: only for machines without a GPU")
    c, c8 = _cache("fk_kv_cache_t"), _cache("fk_kv_cache8_t")
    for dt in (0, 1, 2):
        for width in (8, 4000):
            assert lib.fk_prompt_attn(P, I2(256, 64), dt, 5, 3, 4, ctypes.byref(c), P, width, width, P, P, 0, 0.1,
                                      0.0, P, None, P, lib.fk_workspace_size_prompt(dt, 5, 3, 4, 2, 64), None) == HIP
            assert lib.fk_paged_attn8(P, I2(256, 64), dt, 3, 4, ctypes.byref(c8), P, width, width, P, 0, 0.1, 0.0,
                                      P, None, P, lib.fk_workspace_size_attn8(dt, 3, 4, 2, 64), None) == HIP
        assert lib.fk_kv_store8(P, I2(128, 64), P, I2(128, 64), dt, 3, P, ctypes.byref(c8), None) == HIP
        assert lib.fk_kv_load8(ctypes.byref(c8), P, dt, 3, P, P, None) == HIP


def test_python_refusals(fk):
    import torch

    z, i32 = torch.zeros, torch.int32
    e = z(2, 16, 2, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = z(2, 16, 2)
    with pytest.raises(ValueError, match="device"):
        fk.fk_prompt_attn(z(3, 4, 64), z(2, 16, 2, 64), z(2, 16, 2, 64), z(1, 2, dtype=i32), z(1, dtype=i32),
                          z(2, dtype=i32))
    with pytest.raises(ValueError, match="device"):
        fk.fk_kv_store8(z(3, 2, 64), z(3, 2, 64), z(3, dtype=i32), e, e, s, s)
    with pytest.raises(ValueError, match="device"):
        fk.fk_kv_load8(z(3, dtype=i32), e, e, s, s, torch.float32)
    with pytest.raises(ValueError, match="device"):
        fk.fk_paged_attn8(z(3, 4, 64), e, e, s, s, z(3, 2, dtype=i32), z(3, dtype=i32))


@pytest.mark.gpu
def test_python_refusals_on_device(fk):
    import torch

    def z(*s, dtype=torch.float16):
        return torch.zeros(*s, dtype=dtype, device="cuda")

    def e(*s):
        return z(*s, dtype=torch.uint8).view(torch.float8_e4m3fn)

    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    base = dict(q=z(5, 4, 64), k_cache=z(2, 16, 2, 64), v_cache=z(2, 16, 2, 64), table=z(2, 2, dtype=i32),
                lens=z(2, dtype=i32), cu_tokens=z(3, dtype=i32))
    fk.fk_prompt_attn(**base)
    q = base["q"]
    big = z(4 << 20, dtype=u8)
    for bad in [dict(q=z(5, 4, 32)), dict(q=z(5, 5, 64)), dict(q=z(5, 4, 64, dtype=f32)), dict(q=z(5, 4, 128)[:, :, ::2]),
                dict(q=z(5, 4, 64).requires_grad_()), dict(v_cache=z(2, 16, 2, 32)), dict(table=z(2, 2, dtype=torch.int64)),
                dict(lens=z(3, dtype=i32)), dict(lens=z(2, dtype=torch.int64)), dict(cu_tokens=z(2, dtype=i32)),
                dict(cu_tokens=z(3, dtype=torch.int64)), dict(key_bias=z(2, 16, 2)), dict(key_bias=z(2, 16, 1, dtype=f32)),
                dict(out=z(5, 4, 32)), dict(out=q), dict(lse=z(5, 4)), dict(ws=z(8, dtype=u8)), dict(softcap=-1.0),
                dict(max_len=-1), dict(out=base["k_cache"].view(-1)[:1280].view(5, 4, 64)),
                dict(out=z(5, 4, 64), ws=big, lse=big[:80].view(f32).view(5, 4)), dict(q=z(5, 4, 64, dtype=torch.float64))]:
        with pytest.raises((ValueError, fk.FKError)):
            fk.fk_prompt_attn(**{**base, **bad})
    base = dict(k=z(3, 2, 64), v=z(3, 2, 64), slots=torch.arange(3, dtype=i32, device="cuda"), k_cache=e(2, 16, 2, 64),
                v_cache=e(2, 16, 2, 64), k_scale=z(2, 16, 2, dtype=f32), v_scale=z(2, 16, 2, dtype=f32))
    fk.fk_kv_store8(**base)
    arena = z(1 << 16, dtype=u8)
    for bad in [dict(k=z(3, 2, 32)), dict(k=z(3, 1, 64)), dict(v=z(3, 2, 64, dtype=f32)), dict(v=z(2, 2, 64)),
                dict(slots=z(2, dtype=i32)), dict(slots=z(3, dtype=torch.int64)), dict(k_cache=z(2, 16, 2, 64)),
                dict(k_cache=z(2, 16, 2, 64, dtype=u8)), dict(v_cache=e(2, 16, 2, 32)), dict(k_scale=z(2, 16, 2)),
                dict(v_scale=z(2, 16, 1, dtype=f32)), dict(key_bias=z(2, 16, dtype=f32)), dict(v_cache=base["k_cache"]),
                dict(v_scale=base["k_scale"]), dict(key_bias=base["v_scale"]), dict(k=z(3, 2, 64).requires_grad_()),
                dict(k=z(3, 2, 64, dtype=torch.float64), v=z(3, 2, 64, dtype=torch.float64)),
                dict(k_scale=z(2, 16, 2, dtype=f32).requires_grad_()),
                dict(k=arena[:768].view(torch.float16).view(3, 2, 64),
                     k_cache=arena[:4096].view(torch.float8_e4m3fn).view(2, 16, 2, 64))]:
        with pytest.raises((ValueError, fk.FKError)):
            fk.fk_kv_store8(**{**base, **bad})
    cache = {n: base[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    load = dict(slots=base["slots"], dtype=torch.float16, **cache)
    fk.fk_kv_load8(**load)
    one = z(3, 2, 64)
    for bad in [dict(dtype=torch.float64), dict(slots=z(3, dtype=torch.int64)), dict(k_out=z(3, 2, 32)),
                dict(v_out=z(3, 2, 64, dtype=f32)), dict(k_out=one, v_out=one),
                dict(k_out=base["k_cache"].view(-1).view(torch.float16)[:384].view(3, 2, 64))]:
        with pytest.raises((ValueError, fk.FKError)):
            fk.fk_kv_load8(**{**load, **bad})
    base = dict(q=z(3, 4, 64), table=z(3, 2, dtype=i32), lens=z(3, dtype=i32), **cache)
    q = base["q"]
    want = fk.fk_paged_attn8(**base)
    assert torch.equal(fk.fk_paged_attn8(**{**base, "q": q.clone()}, out=q), want)     # q itself may be out
    for bad in [dict(q=z(3, 4, 32)), dict(q=z(3, 5, 64)), dict(table=z(2, 2, dtype=i32)), dict(lens=z(2, dtype=i32)),
                dict(k_cache=z(2, 16, 2, 64)), dict(k_scale=z(2, 16, 2)), dict(out=z(3, 4, 32)), dict(ws=z(8, dtype=u8)),
                dict(q=z(3, 4, 64).requires_grad_()), dict(softcap=NAN), dict(lse=z(3, 4)),
                dict(out=big[:1536].view(torch.float16).view(3, 4, 64), ws=big)]:
        with pytest.raises((ValueError, fk.FKError)):
            fk.fk_paged_attn8(**{**base, **bad})

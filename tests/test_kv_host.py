"""Paged-cache calls: what they refuse, before anything reaches a GPU (CPU)."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = ctypes.c_void_p(256)          # a non-null address that no refused call may touch
I2 = ctypes.c_int64 * 2


@pytest.fixture(scope="module")
def fk():
    import exact_means_clustering_flashassign_amd as mod

    mod.load()
    return mod


@pytest.fixture(scope="module")
def lib(fk):
    return fk.load()


def _cache(fk, **kw):
    from exact_means_clustering_flashassign_amd._binding import fk_kv_cache_t

    d = dict(k=256, v=256, key_bias=None, pages=4, page=16, heads=2, dim=64,
             k_stride=(2048, 128, 64), v_stride=(2048, 128, 64), bias_stride=(32, 2, 1))
    d.update(kw)
    return fk_kv_cache_t(*(d[n] for n, _ in fk_kv_cache_t._fields_))


def test_page_tables_refusals(lib):
    def call(**kw):
        d = dict(old=P, new=P, tin=None, win=0, free=P, nf=4, B=2, page=16, width=8, tokens=2,
                 table=P, lens=P, ct=P, cp=P, slots=P, pos=P, stream=None)
        d.update(kw)
        return lib.fk_page_tables(*d.values())

    for bad in [dict(B=-1), dict(page=0), dict(page=-4), dict(width=0), dict(win=-1), dict(nf=-1),
                dict(tokens=-1), dict(B=1 << 31), dict(page=1 << 31), dict(width=1 << 40),
                dict(old=None), dict(new=None), dict(win=3), dict(free=None), dict(table=None),
                dict(lens=None), dict(ct=None), dict(cp=None), dict(slots=None), dict(pos=None),
                dict(tin=P, win=7)]:
        assert call(**bad) == INVALID, bad


def test_norm_rope_refusals(fk, lib):
    c = _cache(fk)

    def call(**kw):
        d = dict(q=P, qs=I2(256, 64), k=P, ks=I2(128, 64), v=P, vs=I2(128, 64), dt=1, T=3, Hq=4, Hkv=2,
                 D=64, qw=P, kw=P, eps=1e-6, rope=P, mp=9, rot=64, inter=0, pos=P, slots=P,
                 cache=ctypes.byref(c), qo=P, ko=None, stream=None)
        d.update(kw)
        return lib.fk_qk_norm_rope(*d.values())

    for bad in [dict(dt=3), dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(D=0), dict(rot=-2), dict(rot=63),
                dict(rot=66), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(qw=None), dict(kw=None), dict(qs=None), dict(ks=None), dict(vs=None),
                dict(qs=I2(-1, 64)), dict(ks=I2(1 << 62, 64)), dict(q=None), dict(k=None), dict(v=None),
                dict(qo=None), dict(slots=None), dict(cache=None), dict(rope=None), dict(pos=None),
                dict(mp=0), dict(slots=None, cache=None), dict(Hkv=1), dict(D=32, rot=32),
                dict(T=1 << 30, Hq=1 << 30, D=1 << 20)]:
        assert call(**bad) == INVALID, bad
    for bad in [dict(pages=-1), dict(page=0), dict(pages=1 << 20, page=1 << 11), dict(k=None), dict(v=None),
                dict(k_stride=(-1, 128, 64)), dict(v_stride=(1 << 62, 128, 64)),
                dict(key_bias=256, bias_stride=(-1, 2, 1))]:
        b = _cache(fk, **bad)
        assert call(cache=ctypes.byref(b)) == INVALID, bad
    assert call(T=0, q=None, k=None, qo=None) == OK


def test_paged_attn_refusals(fk, lib):
    c = _cache(fk)
    need = lib.fk_workspace_size_attn(1, 3, 4, 2, 64)

    def call(**kw):
        d = dict(q=P, qs=I2(256, 64), dt=1, B=3, Hq=4, cache=ctypes.byref(c), table=P, ld=8, width=8, lens=P,
                 max_len=0, scale=0.1, cap=0.0, out=P, lse=None, ws=P, wsb=need, stream=None)
        d.update(kw)
        return lib.fk_paged_attn(*d.values())

    for bad in [dict(dt=-1), dict(B=-1), dict(Hq=0), dict(Hq=3), dict(cache=None), dict(ld=7), dict(width=-1),
                dict(max_len=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(cap=-1.0),
                dict(cap=float("nan")), dict(cap=float("inf")), dict(q=None), dict(lens=None), dict(out=None),
                dict(table=None), dict(qs=None), dict(qs=I2(-1, 64))]:
        assert call(**bad) == INVALID, bad
    assert call(ws=None) == WORKSPACE and call(wsb=need - 1) == WORKSPACE
    assert call(ws=ctypes.c_void_p(264)) == WORKSPACE
    wide = _cache(fk, dim=1025, k_stride=(65600, 2050, 1025), v_stride=(65600, 2050, 1025))
    assert call(cache=ctypes.byref(wide)) == UNSUPPORTED
    assert call(B=0, q=None, lens=None, out=None, ws=None, wsb=0) == OK
    for bad in [(5, 1, 4, 2, 64), (1, -1, 4, 2, 64), (1, 1, 0, 2, 64), (1, 1, 4, 3, 64), (1, 1, 4, 0, 64),
                (1, 1, 4, 2, 0)]:
        assert lib.fk_workspace_size_attn(*bad) == 0, bad
    assert lib.fk_workspace_size_attn(1, 0, 4, 2, 64) >= 256


def test_without_a_gpu_valid_calls_report_an_error(fk, lib):
    """Arguments in order but no device: a status, not a crash."""
    import torch

    if torch.cuda.is_available():
        pytest.skip("the addresses here are made up: only for machines without a GPU")
    c = _cache(fk)
    HIP = 4
    assert lib.fk_page_tables(P, P, None, 0, P, 4, 2, 16, 8, 2, P, P, P, P, P, P, None) == HIP
    assert lib.fk_qk_norm_rope(P, I2(256, 64), P, I2(128, 64), P, I2(128, 64), 1, 3, 4, 2, 64, P, P, 1e-6, P, 9,
                               64, 0, P, P, ctypes.byref(c), P, None, None) == HIP
    for width in (8, 4000):
        assert lib.fk_paged_attn(P, I2(256, 64), 1, 3, 4, ctypes.byref(c), P, width, width, P, 0, 0.1, 0.0, P,
                                 None, P, lib.fk_workspace_size_attn(1, 3, 4, 2, 64), None) == HIP


def test_python_refusals(fk):
    import torch

    i32 = torch.int32
    z = torch.zeros
    with pytest.raises(ValueError, match="device"):
        fk.fk_page_tables(z(2, dtype=i32), z(2, dtype=i32), z(4, dtype=i32), 16, 4, 2)
    with pytest.raises(ValueError, match="device"):
        fk.fk_qk_norm_rope(z(3, 4, 64), z(3, 2, 64))
    with pytest.raises(ValueError, match="device"):
        fk.fk_paged_attn(z(3, 4, 64), z(2, 16, 2, 64), z(2, 16, 2, 64), z(3, 2, dtype=i32), z(3, dtype=i32))
    with pytest.raises(ValueError, match="element type"):
        fk.dtype_code(torch.float64)


@pytest.mark.gpu
def test_python_refusals_on_device(fk):
    import torch

    def z(*s, dtype=torch.float16):
        return torch.zeros(*s, dtype=dtype, device="cuda")

    i32 = torch.int32
    q, kc, vc, tb, ln = z(3, 4, 64), z(2, 16, 2, 64), z(2, 16, 2, 64), z(3, 2, dtype=i32), z(3, dtype=i32)
    fk.fk_paged_attn(q, kc, vc, tb, ln)
    for bad in [dict(q=z(3, 4, 32)), dict(q=z(3, 5, 64)), dict(q=z(3, 4, 64, dtype=torch.float32)),
                dict(vc=z(2, 16, 2, 32)), dict(tb=z(2, 2, dtype=i32)), dict(tb=z(3, 2, dtype=torch.int64)),
                dict(ln=z(2, dtype=i32)), dict(ln=z(3, dtype=torch.int64)), dict(kb=z(2, 16, 2)),
                dict(kb=z(2, 16, 1, dtype=torch.float32)), dict(q=z(3, 4, 128)[:, :, ::2]),
                dict(q=z(3, 4, 64).requires_grad_()), dict(out=z(3, 4, 32)), dict(ws=z(8, dtype=torch.uint8))]:
        d = dict(q=q, kc=kc, vc=vc, tb=tb, ln=ln, kb=None, out=None, ws=None)
        d.update(bad)
        with pytest.raises((ValueError, fk.FKError)):
            fk.fk_paged_attn(d["q"], d["kc"], d["vc"], d["tb"], d["ln"], key_bias=d["kb"], out=d["out"], ws=d["ws"])
    k, v, sl = z(3, 2, 64), z(3, 2, 64), z(3, dtype=i32)
    fk.fk_qk_norm_rope(q, k, v, slots=sl, k_cache=kc, v_cache=vc)
    rope, pos = z(9, 64, dtype=torch.float32), z(3, dtype=i32)
    for bad in [dict(k=z(2, 2, 64)), dict(v=None), dict(v=z(3, 1, 64)), dict(slots=None), dict(k_cache=None),
                dict(q_weight=z(64)), dict(q_weight=z(64), k_weight=z(32)), dict(rope=rope),
                dict(rope=rope[:, :63].contiguous(), positions=pos), dict(rope=z(9, 66, dtype=torch.float32), positions=pos),
                dict(rope=rope, positions=z(2, dtype=i32)), dict(eps=-1.0), dict(q_out=z(3, 4, 32)),
                dict(k=k.clone().requires_grad_())]:
        d = dict(k=k, v=v, slots=sl, k_cache=kc, v_cache=vc)
        d.update(bad)
        with pytest.raises((ValueError, fk.FKError)):
            fk.fk_qk_norm_rope(q, **d)
    old, new, free = z(3, dtype=i32), z(3, dtype=i32), z(4, dtype=i32)
    for bad in [dict(page=0), dict(width=0), dict(tokens=-1), dict(table=z(2, 4, dtype=i32)), dict(new=z(2, dtype=i32)),
                dict(free=z(2, 2, dtype=i32)), dict(out=(old,) * 5), dict(out=(old,) * 6)]:
        d = dict(old=old, new=new, free=free, page=16, width=4, tokens=3)
        d.update(bad)
        with pytest.raises((ValueError, fk.FKError)):
            fk.fk_page_tables(d["old"], d["new"], d["free"], d["page"], d["width"], d["tokens"],
                              table=d.get("table"), out=d.get("out"))

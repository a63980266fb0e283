"""The 8-bit cache on the GPU against the fp64 oracle: codes, scales and what is read back
(exact: a scale is a power of two, so there is one rounding and it is defined), single-token
attention over it.

Error bounds of the attention (u = 2^-24; U = 2^-11 fp16, 2^-8 bf16, 2^-24 fp32): a score is off
by e_s = (D + 10) u S + cap 2^-20, S the largest scale * sum |q_i k_i|; a weight relatively by 2 e_s, by
its rounding as two 16-bit numbers (three for fp32 results), 2^-16 (2^-22), by 2^-20 for the
exponentials, 2 u for the value's scale, and sums over n keys by (n + 16) u. With R the sum of
these, the result is off by E = 2 R V + U (|out| + 2 R V), V the largest |v|; lse by e_s + R +
2^-22 |lse|.
"""
import math

import numpy as np
import pytest

import oracle
import synthdata
from gpu_helpers import host_f64, to_dev, torch_dtype

pytestmark = pytest.mark.gpu

UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
LARGEST = {"f16": 65504.0, "bf16": (2 - 2.0 ** -7) * 2.0 ** 127, "f32": (2 - 2.0 ** -23) * 2.0 ** 127}
U32 = 2.0 ** -24
DTYPES = ["f16", "bf16", "f32"]


def _torch():
    import torch
    return torch


def _dev(a):
    return _torch().from_numpy(np.ascontiguousarray(a)).cuda()


def _rand(rng, shape, dtype, scale=1.0):
    return synthdata.to_storage((rng.standard_normal(shape) * scale).astype(np.float32), dtype)


def _numbers():
    """What the 256 codes stand for."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    x = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0)) * np.where(c & 128, -1.0, 1.0)
    x[[127, 255]] = np.nan
    return x


def _cache(pages, page, H, D, how, fill=0):
    """k, v (e4m3), k_scale, v_scale, key_bias of a layout, codes all `fill`, numbers NaN."""
    torch = _torch()

    def codes():
        if how == "heads":
            t = torch.full((pages, H, page, D), fill, dtype=torch.uint8, device="cuda").transpose(1, 2)
        elif how == "odd":
            s = (page * H * (D + 1) + 1, H * (D + 1), D + 1, 1)
            t = torch.full((pages * s[0] + 9,), fill, dtype=torch.uint8, device="cuda").as_strided(
                (pages, page, H, D), s, 3)
        else:
            t = torch.full((pages, page, H, D), fill, dtype=torch.uint8, device="cuda")
        return t.view(torch.float8_e4m3fn)

    def numbers():
        if how == "plain":
            return torch.full((pages, page, H), math.nan, device="cuda")
        return torch.full((pages, H, page + 1), math.nan, device="cuda").transpose(1, 2)[:, :page]

    return codes(), codes(), numbers(), numbers(), numbers()


STORE = [
    # T, heads, D, page, layout
    (1, 1, 64, 1, "plain"),
    (32, 8, 128, 16, "plain"),
    (77, 5, 80, 20, "heads"),
    (130, 2, 96, 7, "plain"),
    (9, 3, 33, 4, "odd"),
    (40, 1, 256, 16, "plain"),
    (11, 2, 1000, 3, "plain"),
    (5, 1, 1, 2, "plain"),
    (1000, 4, 32, 64, "heads"),
    (21, 20, 192, 8, "plain"),
    (3, 1, 4096, 2, "plain"),
    (17, 2, 520, 2, "odd"),
    (700, 7, 8, 16, "plain"),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", STORE, ids=[f"t{c[0]}h{c[1]}d{c[2]}{c[4]}" for c in STORE])
def test_store_and_load(fk, case, dtype):
    torch = _torch()
    T, H, D, page, how = case
    rng = np.random.default_rng(T + D)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    if T > 4:
        slots[1], slots[3] = -1, pages * page          # outside: skipped
    # rows of every size the type holds, zeros and borders of the scale among them
    span = {"f16": (-24, 12), "bf16": (-140, 125), "f32": (-145, 125)}[dtype]
    x = rng.standard_normal((2, T, H, D)) * np.exp2(rng.integers(*span, (2, T, H, 1)).astype(float))
    x[:, ::5] = rng.integers(-64, 65, x[:, ::5].shape) * 7.0          # many ties
    x[0, T // 2], x[1, 0, 0] = 0.0, 448.0
    x = np.clip(x, -LARGEST[dtype], LARGEST[dtype])
    x = [synthdata.to_storage(a.astype(np.float32), dtype) for a in x]
    xd = [to_dev(a, dtype) for a in x]
    if how == "plain" and T > 2:                       # one projection's output, side by side
        both = torch.cat(xd, 1)
        xd = [both[:, :H], both[:, H:]]
    kc, vc, ks, vs, kb = _cache(pages, page, H, D, how, fill=0x5A)
    fk.fk_kv_store8(xd[0], xd[1], _dev(slots), kc, vc, ks, vs, kb)
    live = (slots >= 0) & (slots < pages * page)
    at = slots[live] // page, slots[live] % page
    k_out, v_out = fk.fk_kv_load8(_dev(slots), kc, vc, ks, vs, torch_dtype(dtype))
    for a, codes, scales, back in ((x[0], kc, ks, k_out), (x[1], vc, vs, v_out)):
        want, scale = oracle.quantise(synthdata.to_f64(a, dtype))
        codes, scales = codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy().astype(np.float64)
        got = _numbers()[codes[at]] * scales[at][..., None]
        assert np.array_equal(scales[at], scale[live]) and np.array_equal(got, want[live])
        other = np.ones(codes.shape[:2], bool)
        other[at] = False
        assert (codes[other] == 0x5A).all() and np.isnan(scales[other]).all()     # nothing else is touched
        want = np.clip(np.where(live[:, None, None], want, 0.0), -LARGEST[dtype], LARGEST[dtype])
        want = synthdata.to_f64(synthdata.to_storage(want.astype(np.float32), dtype), dtype)
        assert np.array_equal(host_f64(back, dtype), want)
    bias = kb.cpu().numpy()
    assert (bias[at] == 0).all() and np.isnan(bias).sum() == (pages * page - live.sum()) * H


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 33])
def test_rows_that_are_not_finite(fk, D, dtype):
    torch = _torch()
    x = torch.randn(6, 2, D, device="cuda").to(torch_dtype(dtype))
    x[0, 0, 3], x[1, 1, 0], x[2, 0, D - 1] = math.inf, -math.inf, math.nan
    x[3, 1] = math.nan
    kc, vc, ks, vs, _ = _cache(2, 4, 2, D, "plain")
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    fk.fk_kv_store8(x, x, slots, kc, vc, ks, vs)
    k, v = fk.fk_kv_load8(slots, kc, vc, ks, vs, torch_dtype(dtype))
    want, scale = oracle.quantise(x.double().cpu().numpy())
    for back, scales in ((k, ks), (v, vs)):
        assert np.array_equal(scales.flatten(0, 1)[:6].cpu().numpy(), scale)
        assert np.array_equal(np.isnan(want), back.isnan().cpu().numpy())
        assert np.array_equal(np.nan_to_num(want), np.nan_to_num(host_f64(back, dtype)))


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_code_is_read_exactly(fk, dtype):
    torch = _torch()
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(1, 1, 1, 256)
    for D in (256, 255):
        kc = codes[..., :D].contiguous().view(torch.float8_e4m3fn)
        vc = codes[..., 256 - D:].contiguous().view(torch.float8_e4m3fn)
        for s in (1.0, 0.25, 3.0, 2.0 ** 8):
            sc = torch.full((1, 1, 1), s, device="cuda")
            slot = torch.zeros(3, dtype=torch.int32, device="cuda")       # the same slot again and again
            k, v = fk.fk_kv_load8(slot, kc, vc, sc, sc.clone(), torch_dtype(dtype))
            for got, want in ((k, _numbers()[:D] * s), (v, _numbers()[256 - D:] * s)):
                want = torch.from_numpy(want.clip(-LARGEST[dtype], LARGEST[dtype])).to(torch_dtype(dtype))
                got = got.cpu()
                assert all(torch.equal(got[i, 0].nan_to_num(), want.nan_to_num()) for i in range(3))
                assert torch.equal(got[0, 0].isnan(), want.isnan())


def _attn_case(case, dtype, seed):
    """Inputs with codes of NaN and scales of NaN wherever nothing may be read from."""
    torch = _torch()
    Hq, Hkv, D, page, lens, bias, cap, how = case
    rng = np.random.default_rng(seed)
    B = len(lens)
    held = [-(-n // page) for n in lens]
    width = max(1, max(held)) + 1
    pages = sum(held) + 3
    perm = rng.permutation(pages).astype(np.int32)
    table = np.where(rng.random((B, width)) < 0.5, -1, pages + 5).astype(np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = perm[at:at + h]
        at += h
    if B > 2 and held[0] > 2:
        table[0, 1], table[0, 2] = -1, pages           # holes: their keys are left out
    used = np.zeros((pages, page), bool)
    for b, n in enumerate(lens):
        for j in range(n):
            if 0 <= table[b, j // page] < pages:
                used[table[b, j // page], j % page] = True
    kb = None
    if bias:
        kb = np.zeros((pages, page, Hkv), np.float32)
        counts = rng.integers(0, 6, kb.shape)
        kb[counts > 0] = np.log(counts[counts > 0])
        kb[counts == 0] = -np.inf
        if bias == "none":
            kb[:] = -np.inf
            kb[table[0, 0], page // 2] = 0.5
        if bias == "lowest":
            kb = np.where(rng.random(kb.shape) < 0.5, np.finfo(np.float32).min, kb).astype(np.float32)
            for j in range(lens[1]):
                kb[table[1, j // page], j % page] = np.finfo(np.float32).min
    dead = np.broadcast_to(~used[:, :, None], (pages, page, Hkv)).copy()
    if kb is not None:
        dead |= kb == -np.inf
    kc, vc, ks, vs, kbd = _cache(pages, page, Hkv, D, how)
    rows = []
    for codes, scales in ((kc, ks), (vc, vs)):
        c = rng.integers(0, 127, (pages, page, Hkv, D)) + 128 * rng.integers(0, 2, (pages, page, Hkv, D))
        s = np.exp2(rng.uniform(-8, -6, (pages, page, Hkv))).astype(np.float32)
        rows.append(_numbers()[c] * s[..., None].astype(np.float64))
        c[dead], s = 127, np.where(dead, np.nan, s)
        codes.view(torch.uint8).copy_(_dev(c.astype(np.uint8)))
        scales.copy_(_dev(s.astype(np.float32)))
    if kb is not None:
        kbd.copy_(_dev(np.where(used[:, :, None], kb, np.nan).astype(np.float32)))
    q = _rand(rng, (B, Hq, D), dtype, 2.0)
    want = oracle.paged_attn(synthdata.to_f64(q, dtype), *rows, table, lens, D ** -0.5, cap,
                             None if kb is None else kb.astype(np.float64))
    args = dict(q=to_dev(q, dtype), k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, table=_dev(table),
                lens=_dev(np.array(lens, np.int32)), softcap=cap, key_bias=None if kb is None else kbd,
                return_lse=True)
    return args, want


def _check_attn(got, want, dtype, D, cap, where=""):
    out, lse = host_f64(got[0], dtype), got[1].double().cpu().numpy()
    ref, rlse, info = want
    S, V, n = (info[..., i][..., None] for i in (1, 2, 3))
    e_s = (D + 10) * U32 * S + cap * 2.0 ** -20
    R = 2 * e_s + (2.0 ** -22 if dtype == "f32" else 2.0 ** -16) + 2.0 ** -20 + (n + 18) * U32
    tol = 2 * R * V + UNIT[dtype] * (np.abs(ref) + 2 * R * V) + (2.0 ** -25 if dtype == "f16" else 0)
    err = np.abs(out - ref)
    assert (err <= tol).all(), (where, "out", float((err / np.maximum(tol, 1e-300)).max()))
    none = rlse == -np.inf
    assert np.array_equal(none, lse == -np.inf), where
    assert (out[none] == 0).all(), where
    err = np.abs(lse[~none] - rlse[~none])
    tol = (e_s + R)[..., 0][~none] + 2.0 ** -22 * np.abs(rlse[~none])
    assert (err <= tol).all(), (where, "lse", float((err / tol).max()))


ATTN = [
    # Hq, Hkv, D, page, lens, bias, cap, layout
    (4, 2, 64, 16, [1, 0, 40], None, 0.0, "plain"),
    (8, 2, 128, 16, [300, 33, 64, 17], None, 0.0, "plain"),
    (32, 4, 128, 24, [700, 5], "log", 30.0, "plain"),
    (20, 1, 80, 20, [130, 77], "log", 0.0, "plain"),
    (6, 6, 96, 1, [100, 31], None, 12.0, "heads"),
    (2, 2, 32, 7, [64, 0, 63], "none", 0.0, "plain"),
    (16, 1, 256, 16, [290, 64], None, 0.0, "plain"),
    (3, 1, 192, 64, [65, 31], "lowest", 0.0, "heads"),
    (40, 1, 64, 16, [600, 4], "log", 0.0, "plain"),
    (34, 2, 128, 16, [2500, 1, 900], None, 20.0, "plain"),
    (3, 3, 33, 4, [50, 20, 0], "log", 10.0, "plain"),
    (2, 1, 72, 16, [90, 5], None, 0.0, "plain"),
    (2, 1, 20, 3, [65, 9], None, 0.0, "odd"),
    (2, 1, 320, 16, [50, 20], "log", 0.0, "plain"),
    (2, 2, 1000, 16, [20, 3], None, 0.0, "plain"),
    (8, 8, 128, 16, [3000, 2049, 64], None, 0.0, "plain"),
    (4, 1, 64, 256, [3, 5000, 0, 700, 0, 1], None, 0.0, "plain"),
]
ATTN_IDS = [f"{c[0]}x{c[1]}d{c[2]}p{c[3]}n{max(c[4])}{c[5] or ''}{c[7]}" for c in ATTN]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", ATTN, ids=ATTN_IDS)
def test_paged_attn8(fk, case, dtype):
    torch = _torch()
    args, want = _attn_case(case, dtype, seed=len(case[4]) * 100 + case[2])
    for hint in (1, max(case[4]), 0):                  # how the work is split goes by max_len
        got = fk.fk_paged_attn8(max_len=hint, **args)
        _check_attn(got, want, dtype, case[2], case[6], f"max_len {hint}")
    table = args["table"]                              # room for 2^20 keys a request, most of it unused
    args["table"] = torch.cat([table, table.new_full((table.shape[0], (1 << 20) // case[3]), -1)], 1)
    _check_attn(fk.fk_paged_attn8(**args), want, dtype, case[2], case[6], "wide table")


def test_paged_attn8_many_ragged_requests(fk):
    rng = np.random.default_rng(5)
    lens = [int(n) for n in np.exp(rng.uniform(0, np.log(3000), 90))]
    lens[::9] = [0] * len(lens[::9])
    args, want = _attn_case((4, 2, 64, 16, lens, None, 0.0, "plain"), "bf16", 6)
    for hint in (0, max(lens)):
        _check_attn(fk.fk_paged_attn8(max_len=hint, **args), want, "bf16", 64, 0.0)
    lens = [int(n) for n in np.exp(rng.uniform(0, np.log(600), 700))]
    lens[::7] = [0] * len(lens[::7])
    args, want = _attn_case((4, 4, 128, 8, lens, None, 0.0, "plain"), "f16", 7)
    for hint in (0, 200, 32):
        _check_attn(fk.fk_paged_attn8(max_len=hint, **args), want, "f16", 128, 0.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dims", [(4, 2, 64), (40, 2, 96), (2, 1, 256), (3, 3, 33)], ids=["d64", "g20d96", "d256", "d33"])
def test_paged_attn8_numbers_that_are_not_finite(fk, dims, dtype):
    """NaN codes that count reach their request, head and element; nothing else does; masked keys and
    queries of nothing left stay out."""
    torch = _torch()
    Hq, Hkv, D = dims
    lens = [70, 5, 700, 40]
    args, want = _attn_case((Hq, Hkv, D, 16, lens, None, 0.0, "plain"), dtype, D + 3)
    table, G = args["table"], Hq // Hkv
    page, tok = int(table[2, 20]), 9
    args["v_cache"].view(torch.uint8)[page, tok, Hkv - 1, 5] = 127
    out, lse = (t.clone() for t in fk.fk_paged_attn8(**args))
    assert out[2, -G:, 5].isnan().all() and out.isnan().sum() == G
    out[2, -G:, 5] = torch.from_numpy(want[0][2, -G:, 5]).to(out)
    _check_attn((out, lse), want, dtype, D, 0.0)
    args["v_cache"].view(torch.uint8)[page, tok, Hkv - 1, 5] = 0
    args["k_cache"].view(torch.uint8)[page, tok, 0, D - 1] = 255
    out, lse = fk.fk_paged_attn8(**args)
    assert out[2, :G].isnan().all() and lse[2, :G].isnan().all()
    assert out.isnan().sum() == G * D and lse.isnan().sum() == G
    # a query that is not finite and has no keys
    args["q"][1], args["table"][1] = math.nan, -1
    out, lse = fk.fk_paged_attn8(**args)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
    args["q"][3, 0, 0] = math.inf                      # and one that has some
    out, lse = fk.fk_paged_attn8(**args)
    assert not out[3, 0].isfinite().any() and out[3, 1:].isfinite().all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 33])
def test_captured_and_replayed(fk, D, dtype):
    """Store, read back and attention in one graph, replayed over other rows and lengths, with eager
    calls between the replays, on a stream of its own."""
    torch = _torch()
    B, H, page, T = 3, 2, 8, 40
    made = []
    for seed in range(3):
        rng = np.random.default_rng(seed)
        rows = [to_dev(_rand(rng, (T, H, D), dtype), dtype) for _ in range(2)]
        slots = rng.permutation(9 * page)[:T].astype(np.int32)
        slots[3] = -1
        lens = rng.integers(0, 3 * page + 1, B).astype(np.int32)
        table = rng.permutation(9).reshape(B, 3).astype(np.int32)
        made.append((*rows, _dev(slots), _dev(lens), _dev(table), to_dev(_rand(rng, (B, 4 * H, D), dtype), dtype)))
    k, v, slots, lens, table, q = (t.clone() for t in made[0])

    def fresh():
        c = _cache(9, page, H, D, "plain")
        for t in c[2:]:
            t.fill_(1.0)
        return c

    def step(c, k, v, slots, lens, table, q, **kw):
        fk.fk_kv_store8(k, v, slots, *c)
        back = fk.fk_kv_load8(slots, *c[:4], k.dtype)
        return (*back, *fk.fk_paged_attn8(q, *c[:4], table, lens, key_bias=c[4], return_lse=True, **kw))

    held = fresh()
    ws = torch.empty(fk.fk_workspace_size_attn8(q.dtype, B, 4 * H, H, D), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(held, k, v, slots, lens, table, q, ws=ws)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step(held, k, v, slots, lens, table, q, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    for i in (1, 0, 2, 2, 1):
        for a, b in zip((k, v, slots, lens, table, q), made[i]):
            a.copy_(b)
        for a, b in zip(held, fresh()):
            a.view(torch.uint8).copy_(b.view(torch.uint8)) if a.dtype == torch.float8_e4m3fn else a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        want = step(fresh(), *made[i])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


def test_nothing_to_do(fk):
    torch = _torch()
    kc, vc, ks, vs, kb = _cache(2, 4, 2, 64, "plain")
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.zeros((0, 2, 64), device="cuda")
    fk.fk_kv_store8(x, x, torch.zeros(0, **i32), kc, vc, ks, vs, kb)
    assert ks.isnan().all() and kb.isnan().all()
    k, v = fk.fk_kv_load8(torch.zeros(0, **i32), kc, vc, ks, vs, torch.float16)
    assert k.shape == v.shape == (0, 2, 64)
    none = [t[:0] for t in (kc, vc, ks, vs)]           # a cache without pages
    y = torch.ones((3, 2, 64), device="cuda")
    fk.fk_kv_store8(y, y, torch.zeros(3, **i32), *none)
    k, v = fk.fk_kv_load8(torch.arange(3, **i32), *none, torch.float32)
    assert (k == 0).all() and (v == 0).all()
    out, lse = fk.fk_paged_attn8(torch.ones((2, 4, 64), device="cuda"), *none, torch.zeros((2, 3), **i32),
                                 torch.full((2,), 9, **i32), return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    out = fk.fk_paged_attn8(torch.ones((0, 4, 64), device="cuda"), kc, vc, ks, vs, torch.zeros((0, 3), **i32),
                            torch.zeros(0, **i32))
    assert out.shape == (0, 4, 64)

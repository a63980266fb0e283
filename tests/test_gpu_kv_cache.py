"""Paged key-value cache on the GPU against the fp64 oracle: page tables (exact),
query/key norm with rotation and stores, single-token attention.

Error bounds (u = 2^-24, the fp32 unit; U = the output type's, 2^-11 fp16,
2^-8 bf16, 2^-24 fp32), from the arithmetic the header promises:
  * norm + rotation: y is a sum of at most two products whose magnitudes sum to
    M (from the oracle). The mean of D squares is off by at most D u / 2 + 4 u
    relatively after the square root, each product by 4 u more, so the fp32 value
    is off by E = (D / 2 + 10) u M and the stored one by E + U (|y| + E), plus half the
    smallest fp16 subnormal, 2^-25.
  * attention: a score is off by e_s = (D + 8) u S + cap 2^-20, S the largest
    scale * sum |q_i k_i|; a weight relatively by 2 e_s, by the rounding of the
    probabilities to 16 bits or more (2^-16, and 2^-38 of the largest one for
    each key), 2^-20 for the exponentials, and sums over at most n / 4 + 16 keys in a
    row by (n / 4 + 16) u. With R the sum of these, the result is off by
    E = 2 R V + U (|out| + 2 R V), V the largest |v|; lse by e_s + R + 2^-22 |lse|.
"""
import math

import numpy as np
import pytest

import oracle
import synthdata
from gpu_helpers import host_f64, to_dev, torch_dtype

pytestmark = pytest.mark.gpu

UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U32 = 2.0 ** -24


def _torch():
    import torch
    return torch


def _dev(a):
    return _torch().from_numpy(np.ascontiguousarray(a)).cuda()


def _rand(rng, shape, dtype, scale=1.0):
    return synthdata.to_storage((rng.standard_normal(shape) * scale).astype(np.float32), dtype)


# ---------------------------------------------------------------------------
# page tables
# ---------------------------------------------------------------------------
TABLES = [
    # B, page, width, width_in, free, pad, old up to, new up to
    (1, 1, 1, 1, 4, 0, 0, 1),
    (1, 16, 8, 8, 40, 3, 100, 1),
    (3, 4, 5, 2, 3, 2, 12, 9),             # free list too short, held pages past table_in
    (7, 48, 9, 9, 90, 0, 300, 200),        # rows too narrow for some
    (64, 16, 200, 128, 9000, 17, 2000, 1),
    (255, 8, 33, 33, 9000, 5, 150, 130),
    (1000, 1, 70, 64, 70000, 0, 40, 33),
    (1025, 64, 20, 20, 20000, 1, 700, 600),
    (5000, 16, 7, 7, 30000, 9, 60, 60),
    (2048, 4, 9, 9, 30000, 3, 20, 12),     # the most whose sums every block forms for itself
    (2049, 4, 9, 9, 30000, 3, 20, 12),
    (2, 16, 5000, 5000, 10000, 0, 40000, 38000),
]


@pytest.mark.parametrize("case", TABLES, ids=[f"B{c[0]}p{c[1]}w{c[2]}" for c in TABLES])
def test_page_tables(fk, case):
    B, page, width, width_in, n_free, pad, most_old, most_new = case
    rng = np.random.default_rng(B * 31 + page)
    old = rng.integers(0, most_old + 1, B).astype(np.int32)
    new = rng.integers(0, most_new + 1, B).astype(np.int32)
    old[rng.random(B) < 0.15] = 0
    new[rng.random(B) < 0.15] = 0
    if B > 4:
        old[1], new[2] = -3, -7                 # counts as 0
    tin = rng.integers(-1, 1 << 20, (B, width_in)).astype(np.int32)
    free = rng.permutation(n_free).astype(np.int32)
    tokens = int(np.maximum(new, 0).sum()) + pad
    want = oracle.page_tables(old, new, tin, free, page, width, tokens)
    got = fk.fk_page_tables(_dev(old), _dev(new), _dev(free), page, width, tokens, table=_dev(tin))
    for g, w, name in zip(got, want, ("table", "lens", "cu_tokens", "cu_pages", "slots", "positions")):
        assert np.array_equal(g.cpu().numpy(), w), name
    if tokens > 5:                              # fewer token places than tokens, and no table before
        want = oracle.page_tables(old, new, None, free, page, width, tokens // 2)
        got = fk.fk_page_tables(_dev(old), _dev(new), _dev(free), page, width, tokens // 2)
        for g, w in zip(got, want):
            assert np.array_equal(g.cpu().numpy(), w)


def test_page_tables_in_place_empty_and_huge_lengths(fk):
    torch = _torch()
    i32 = torch.int32
    z = torch.zeros(0, dtype=i32, device="cuda")
    out = fk.fk_page_tables(z, z, z, 16, 4, 3)
    assert out[0].shape == (0, 4) and out[2].tolist() == [0] and out[3].tolist() == [0]
    assert out[4].tolist() == [-1] * 3 and out[5].tolist() == [0] * 3
    # sums past 2^31 - 1 stop there; nothing outside the outputs is touched
    old, new = _dev(np.full(3, 2 ** 31 - 1, np.int32)), _dev(np.full(3, 2 ** 31 - 1, np.int32))
    out = fk.fk_page_tables(old, new, z, 1, 2, 2)
    top = 2 ** 31 - 1
    assert out[1].tolist() == [top] * 3 and out[2].tolist() == [0, top, top, top]
    assert (out[0] == -1).all() and out[4].tolist() == [-1, -1]
    # table updated in place over several steps equals one long step
    rng = np.random.default_rng(3)
    B, page, width = 9, 8, 16
    free = torch.arange(200, dtype=i32, device="cuda")
    lens = torch.zeros(B, dtype=i32, device="cuda")
    table = torch.full((B, width), -1, dtype=i32, device="cuda")
    taken, seen = 0, [[] for _ in range(B)]
    for step in range(5):
        n = rng.integers(0, 20, B).astype(np.int32)
        bufs = (table, torch.empty_like(lens), *(torch.empty(B + 1, dtype=i32, device="cuda") for _ in range(2)),
                *(torch.empty(int(n.sum()), dtype=i32, device="cuda") for _ in range(2)))
        _, lens, ct, cp, slots, pos = fk.fk_page_tables(lens, _dev(n), free[taken:], page, width,
                                                        int(n.sum()), table=table, out=bufs)
        taken += int(cp[-1])
        for b in range(B):
            seen[b] += slots[ct[b]:ct[b + 1]].tolist()
    rows, ls = table.cpu().numpy(), lens.tolist()
    for b in range(B):
        assert seen[b] == [rows[b, i // page] * page + i % page for i in range(ls[b])]


# ---------------------------------------------------------------------------
# norm + rotation
# ---------------------------------------------------------------------------
ROPE = [
    # T, Hq, Hkv, D, rot, interleaved, norm, page (0: no cache), layout
    (1, 1, 1, 2, 2, False, True, 0, "plain"),
    (1, 8, 2, 128, 128, False, True, 16, "packed"),
    (5, 32, 8, 128, 128, False, True, 16, "packed"),
    (3, 4, 4, 64, 64, True, True, 1, "packed"),
    (33, 3, 1, 256, 256, False, False, 7, "plain"),
    (17, 6, 2, 96, 40, True, True, 8, "packed"),
    (17, 6, 2, 96, 40, False, True, 8, "packed"),
    (9, 5, 5, 80, 80, False, True, 4, "heads"),
    (12, 2, 1, 72, 12, False, True, 4, "plain"),      # pairs that no 8-element group holds whole
    (12, 2, 1, 72, 12, True, True, 4, "plain"),
    (7, 3, 3, 33, 20, False, True, 3, "plain"),       # odd rows
    (7, 3, 3, 33, 20, True, False, 3, "odd"),
    (6, 2, 2, 64, 0, False, True, 5, "odd"),
    (4, 2, 1, 1000, 96, False, True, 2, "plain"),
    (300, 7, 1, 192, 64, False, True, 20, "packed"),
    (2800, 32, 8, 128, 96, False, True, 16, "packed"),     # waves that take several passes
    (9000, 4, 1, 32, 32, False, True, 0, "packed"),
    (40, 12, 2, 200, 36, False, True, 16, "packed"),
]


def _layout(t, how, gap):
    """The tensor's values in other strides: heads before tokens, or rows at odd offsets."""
    torch = _torch()
    if how == "heads":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    if how == "odd":
        T, H, D = t.shape
        buf = torch.zeros(T * (H * (D + 1) + 3) + 5, dtype=t.dtype, device=t.device)
        v = buf.as_strided((T, H, D), (H * (D + 1) + 3, D + 1, 1), gap)
        v.copy_(t)
        return v
    return t


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("case", ROPE, ids=[f"T{c[0]}D{c[3]}r{c[4]}{'i' if c[5] else 'h'}{c[8]}" for c in ROPE])
def test_norm_rope(fk, case, dtype):
    torch = _torch()
    T, Hq, Hkv, D, rot, inter, norm, page, how = case
    rng = np.random.default_rng(T * 7 + D)
    x = _rand(rng, (T, Hq + 2 * Hkv, D), dtype, 2.0)
    x64 = synthdata.to_f64(x, dtype)
    xd = to_dev(x, dtype)
    q, k, v = xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:]
    if how != "packed":
        q, k, v = (_layout(t.contiguous(), how, i) for i, t in enumerate((q, k, v)))
    w = [_rand(rng, D, dtype) for _ in range(2)] if norm else [None, None]
    w64 = [None if a is None else synthdata.to_f64(a, dtype) for a in w]
    wd = [None if a is None else to_dev(a, dtype) for a in w]
    rope = rng.uniform(-1, 1, (50, rot)).astype(np.float32) if rot else None
    pos = rng.integers(-2, 53, T).astype(np.int32)      # some outside: taken as the nearest inside
    kw = dict(rope=_dev(rope), positions=_dev(pos)) if rot else {}
    eps = 1e-5
    want = [oracle.norm_rope(x64[:, a:b], w64[i], eps, None if rope is None else rope.astype(np.float64),
                             pos, inter) for i, (a, b) in enumerate(((0, Hq), (Hq, Hq + Hkv)))]

    def check(got, y, m, name):
        e = (D / 2 + 10) * U32 * m
        tol = e + UNIT[dtype] * (np.abs(y) + e) + (2.0 ** -25 if dtype == "f16" else 0.0)
        err = np.abs(host_f64(got, dtype) - y)
        assert (err <= tol).all(), (name, float((err / np.maximum(tol, 1e-300)).max()))

    if not page:
        qo, ko = fk.fk_qk_norm_rope(q, k, None, *wd, eps, interleaved=inter, **kw)
        check(qo, *want[0], "q")
        check(ko, *want[1], "k")
        return
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    if T > 4:
        slots[1], slots[2] = -1, pages * page           # outside: skipped
    filler = _rand(rng, (pages, page, Hkv, D), dtype)
    kc, vc = to_dev(filler, dtype), to_dev(filler, dtype)
    if how == "heads":                                  # heads before tokens in a page
        kc = kc.transpose(1, 2).contiguous().transpose(1, 2)
    bias = torch.full((pages, page, Hkv), 7.0, device="cuda")
    k_out = torch.empty((T, Hkv, D), dtype=xd.dtype, device="cuda") if T % 2 else None
    qo, ko = fk.fk_qk_norm_rope(q, k, v, *wd, eps, interleaved=inter, slots=_dev(slots), k_cache=kc,
                                v_cache=vc, key_bias=bias, k_out=k_out, **kw)
    check(qo, *want[0], "q")
    if k_out is None:
        assert ko is None
    else:
        check(ko, *want[1], "k_out")
    f64 = synthdata.to_f64(filler, dtype).reshape(pages * page, Hkv, D)
    yk, mk, yv = f64.copy(), np.zeros_like(f64), f64.copy()
    yb = np.full((pages * page, Hkv), 7.0)
    ok = (slots >= 0) & (slots < pages * page)
    yk[slots[ok]], mk[slots[ok]], yv[slots[ok]] = want[1][0][ok], want[1][1][ok], x64[ok, Hq + Hkv:]
    yb[slots[ok]] = 0.0
    check(kc.contiguous(), yk.reshape(kc.shape), mk.reshape(kc.shape), "k_cache")
    assert np.array_equal(host_f64(vc, dtype).reshape(yv.shape), yv)
    assert np.array_equal(bias.cpu().numpy().reshape(yb.shape), yb)


def test_norm_rope_no_tokens_and_zero_rows(fk):
    torch = _torch()
    q, k = torch.zeros(0, 4, 64, device="cuda"), torch.zeros(0, 2, 64, device="cuda")
    qo, ko = fk.fk_qk_norm_rope(q, k)
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 2, 64)
    # an all-zero row has no direction: eps keeps it at zero
    q, k, w = torch.zeros(3, 4, 64, device="cuda"), torch.zeros(3, 2, 64, device="cuda"), torch.ones(64, device="cuda")
    qo, ko = fk.fk_qk_norm_rope(q, k, None, w, w, 1e-6)
    assert (qo == 0).all() and (ko == 0).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
ATTN = [
    # Hq, Hkv, D, page, lens, bias, cap, layout
    (1, 1, 64, 16, [1], None, 0.0, "plain"),
    (4, 4, 128, 16, [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65], None, 0.0, "plain"),
    (8, 2, 128, 16, [127, 128, 129, 0, 255, 256, 257, 500], None, 0.0, "heads"),
    (32, 8, 128, 48, [700, 1, 333], None, 0.0, "plain"),
    (16, 1, 256, 64, [1000, 3], None, 0.0, "plain"),
    (17, 1, 64, 5, [200, 77], None, 30.0, "plain"),           # more query heads than one tile
    (64, 2, 128, 1, [300, 150], None, 0.0, "plain"),
    (6, 2, 96, 20, [90, 41, 0], "log", 0.0, "plain"),
    (5, 5, 80, 8, [64, 100], "log", 20.0, "heads"),
    (3, 1, 192, 7, [129, 64], "lowest", 0.0, "plain"),
    (2, 2, 32, 16, [64, 40, 16, 33], "none", 0.0, "plain"),
    (4, 2, 72, 12, [100, 9], "log", 0.0, "wide"),
    (3, 3, 33, 4, [50, 5, 0], "log", 10.0, "plain"),           # odd rows
    (2, 1, 20, 3, [65, 1], None, 0.0, "odd"),
    (2, 1, 320, 16, [130, 31], "log", 0.0, "plain"),           # wide heads
    (2, 2, 1000, 16, [70, 2], None, 0.0, "plain"),
    (8, 8, 128, 16, [5000, 2049, 64], None, 0.0, "plain"),
    (8, 1, 128, 16, [20000], "log", 50.0, "plain"),
    (4, 1, 64, 256, [3, 9000, 0, 700, 0, 1], None, 0.0, "plain"),
    (80, 2, 128, 16, [400, 33, 700], "log", 0.0, "plain"),     # 40 query heads a key head
    (33, 1, 256, 16, [300, 1], None, 0.0, "plain"),
    (24, 1, 32, 16, [600, 40], None, 15.0, "heads"),
]


def _attn_case(case, dtype, seed):
    """Inputs of a case with NaN wherever nothing may be read from: unused
    slots, tokens past a request's end and keys with bias -inf."""
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
        table[0, 1] = -1                     # a hole: its keys are left out
        if how == "plain":
            table[0, 2] = pages              # and so is a page past the cache
    used = np.zeros((pages, page), bool)
    for b, n in enumerate(lens):
        for j in range(n):
            if 0 <= table[b, j // page] < pages:
                used[table[b, j // page], j % page] = True
    kb = None
    if bias:
        kb = np.log(rng.integers(0, 6, (pages, page, Hkv)).astype(np.float32), where=True,
                    out=np.zeros((pages, page, Hkv), np.float32))
        if bias == "none":                   # whole requests with nothing left
            kb[:] = -np.inf
            kb[table[0, 0], 3] = 0.5
        if bias == "lowest":                 # the type's lowest value masks by absorbing the score
            kb = np.where(rng.random(kb.shape) < 0.5, np.finfo(np.float32).min, kb).astype(np.float32)
            for j in range(lens[1]):
                kb[table[1, j // page], j % page] = np.finfo(np.float32).min
    q = _rand(rng, (B, Hq, D), dtype, 2.0)
    k, v = (_rand(rng, (pages, page, Hkv, D), dtype) for _ in range(2))
    qd, kd, vd = (to_dev(t, dtype) for t in (q, k, v))
    k64, v64 = synthdata.to_f64(k, dtype), synthdata.to_f64(v, dtype)
    dead = torch.from_numpy(~used).cuda()[:, :, None].expand(pages, page, Hkv).clone()
    if kb is not None:
        dead |= torch.from_numpy(kb == -np.inf).cuda()
    kd[dead] = math.nan
    vd[dead] = math.nan
    kbd = None if kb is None else _dev(np.where(used[:, :, None], kb, np.nan).astype(np.float32))
    td = _dev(table)
    if how == "heads":                       # heads before tokens in memory
        kd, vd = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (kd, vd))
    elif how == "wide":                      # keys and values side by side, a table inside a wider one
        both = torch.cat([kd, vd], -1)
        kd, vd = both[..., :D], both[..., D:]
        td = torch.cat([td, torch.full_like(td, 1 << 30)], 1)[:, :width]
    elif how == "odd":
        def odd(t, gap):
            s = (page * Hkv * (D + 1) + 1, Hkv * (D + 1), D + 1, 1)
            buf = torch.full((pages * s[0] + 9,), math.nan, dtype=t.dtype, device="cuda")
            o = buf.as_strided(t.shape, s, gap)
            o.copy_(t)
            return o
        kd, vd = odd(kd, 1), odd(vd, 3)
    scale = 1.0 / math.sqrt(D)
    want = oracle.paged_attn(synthdata.to_f64(q, dtype), k64, v64, table, lens, scale, cap,
                             None if kb is None else kb.astype(np.float64))
    args = dict(q=qd, k_cache=kd, v_cache=vd, table=td, lens=_dev(np.array(lens, np.int32)),
                softcap=cap, key_bias=kbd, return_lse=True)
    return args, want


def _check_attn(got, want, dtype, D, cap, where=""):
    out, lse = host_f64(got[0], dtype), got[1].double().cpu().numpy()
    ref, rlse, info = want
    S, V, n = (info[..., i][..., None] for i in (1, 2, 3))
    e_s = (D + 8) * U32 * S + cap * 2.0 ** -20
    R = 2 * e_s + 2.0 ** -16 + n * 2.0 ** -38 + 2.0 ** -20 + (n / 4 + 16) * U32
    tol = 2 * R * V + UNIT[dtype] * (np.abs(ref) + 2 * R * V) + (2.0 ** -25 if dtype == "f16" else 0)
    err = np.abs(out - ref)
    assert (err <= tol).all(), (where, "out", float((err / np.maximum(tol, 1e-300)).max()))
    none = rlse == -np.inf
    assert np.array_equal(none, lse == -np.inf), where
    assert (out[none] == 0).all(), where
    err = np.abs(lse[~none] - rlse[~none])
    tol = (e_s + R)[..., 0][~none] + 2.0 ** -22 * np.abs(rlse[~none])
    assert (err <= tol).all(), (where, "lse", float((err / tol).max()))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("case", ATTN, ids=[f"{c[0]}x{c[1]}d{c[2]}p{c[3]}n{max(c[4])}{c[5] or ''}" for c in ATTN])
def test_paged_attn(fk, case, dtype):
    args, want = _attn_case(case, dtype, seed=len(case[4]) * 100 + case[2])
    # how the work is split goes by max_len: a short hint, the true one and none
    for hint in (1, max(case[4]), 0):
        got = fk.fk_paged_attn(max_len=hint, **args)
        _check_attn(got, want, dtype, case[2], case[6], f"max_len {hint}")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("case", ATTN, ids=[f"{c[0]}x{c[1]}d{c[2]}p{c[3]}n{max(c[4])}{c[5] or ''}" for c in ATTN])
def test_paged_attn_wide_tables(fk, case, dtype):
    """Tables with room for 2^20 keys a request, most of it unused: the split and
    the loads are those of large caches."""
    torch = _torch()
    args, want = _attn_case(case, dtype, seed=len(case[4]) * 100 + case[2])
    table = args["table"]
    args["table"] = torch.cat([table, table.new_full((table.shape[0], (1 << 20) // case[3]), -1)], 1)
    _check_attn(fk.fk_paged_attn(**args), want, dtype, case[2], case[6])


def test_paged_attn_many_ragged_requests(fk):
    rng = np.random.default_rng(5)
    lens = [int(n) for n in np.exp(rng.uniform(0, np.log(3000), 90))]
    lens[::9] = [0] * len(lens[::9])
    case = (4, 2, 64, 16, lens, None, 0.0, "plain")
    args, want = _attn_case(case, "bf16", 6)
    _check_attn(fk.fk_paged_attn(**args), want, "bf16", 64, 0.0)
    _check_attn(fk.fk_paged_attn(max_len=max(lens), **args), want, "bf16", 64, 0.0)
    # more requests than a block has threads, cut and whole
    lens = [int(n) for n in np.exp(rng.uniform(0, np.log(600), 700))]
    lens[::7] = [0] * len(lens[::7])
    args, want = _attn_case((4, 4, 128, 8, lens, None, 0.0, "plain"), "f16", 7)
    for hint in (0, 200, 32):
        _check_attn(fk.fk_paged_attn(max_len=hint, **args), want, "f16", 128, 0.0)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("case", [(64, 32, 128, 16, [900, 1, 0, 640, 77], "log", 30.0, "plain"),
                                  (80, 4, 64, 7, [5 * i for i in range(40)] + [700], None, 0.0, "heads"),
                                  (8, 8, 32, 16, [13 * i % 600 for i in range(20)], None, 0.0, "plain")],
                         ids=["heads32", "g20", "d32"])
def test_paged_attn_a_block_for_every_cu(fk, case, dtype):
    """Middle lengths and about as many (request, head) pairs as CUs."""
    args, want = _attn_case(case, dtype, seed=17)
    _check_attn(fk.fk_paged_attn(max_len=max(case[4]), **args), want, dtype, case[2], case[6])


def test_paged_attn_same_bits_any_workspace_and_stream(fk):
    torch = _torch()
    args, want = _attn_case((8, 2, 128, 16, [6000, 0, 37, 900], "log", 0.0, "plain"), "bf16", 8)
    n = fk.fk_workspace_size_attn(torch.bfloat16, 4, 8, 2, 128)
    first = None
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = fk.fk_paged_attn(ws=ws, **args)
        torch.cuda.current_stream().wait_stream(side)
        _check_attn(got, want, "bf16", 128, 0.0)
        if first is not None:
            assert torch.equal(first[0].view(torch.int16), got[0].view(torch.int16))
            assert torch.equal(first[1], got[1])
        first = got


@pytest.mark.parametrize("D", [64, 33])
def test_paged_attn_nothing_to_do(fk, D):
    """No requests, tables without columns, caches without pages, lengths below zero."""
    torch = _torch()
    z = lambda *s, t=torch.float16: torch.zeros(s, dtype=t, device="cuda")      # noqa: E731
    i32 = torch.int32
    kc = z(3, 16, 2, D)
    out, lse = fk.fk_paged_attn(z(0, 4, D), kc, kc, z(0, 5, t=i32), z(0, t=i32), return_lse=True)
    assert out.shape == (0, 4, D) and lse.shape == (0, 4)
    q, lens = torch.ones(2, 4, D, dtype=torch.float16, device="cuda"), _dev(np.array([7, -3], np.int32))
    for cache, table in ((kc, z(2, 0, t=i32)), (z(0, 16, 2, D), z(2, 100, t=i32)),
                         (kc, torch.full((2, 100), -1, dtype=i32, device="cuda"))):
        out, lse = fk.fk_paged_attn(q, cache, cache, table, lens, return_lse=True)
        assert (out == 0).all() and (lse == -math.inf).all()
    x = z(5, 6, D)
    _, ko = fk.fk_qk_norm_rope(x[:, :4], x[:, 4:], x[:, 4:], slots=z(5, t=i32), k_cache=z(0, 16, 2, D),
                               v_cache=z(0, 16, 2, D))
    assert ko is None


def test_paged_attn_offsets_past_32_bits(fk):
    """Pages 3 * 2^30 elements apart: offsets of 12 GB and more."""
    torch = _torch()
    pages, page, Hkv, D, gap = 3, 4, 2, 64, 3 << 30
    if torch.cuda.mem_get_info()[0] < (30 << 30):
        pytest.skip("needs 30 GB of free device memory")
    rng = np.random.default_rng(9)
    k, v = (_rand(rng, (pages, page, Hkv, D), "f16") for _ in range(2))
    raw = torch.empty(2 * gap + 2 * page * Hkv * D, dtype=torch.float16, device="cuda")
    kd = raw.as_strided((pages, page, Hkv, D), (gap, Hkv * D, D, 1))
    vd = raw.as_strided((pages, page, Hkv, D), (gap, Hkv * D, D, 1), page * Hkv * D)
    kd.copy_(to_dev(k, "f16"))
    vd.copy_(to_dev(v, "f16"))
    q, table, lens = _rand(rng, (1, 4, D), "f16"), np.array([[2, 0, 1]], np.int32), [11]
    want = oracle.paged_attn(*(synthdata.to_f64(t, "f16") for t in (q, k, v)), table, lens, 0.125)
    got = fk.fk_paged_attn(to_dev(q, "f16"), kd, vd, _dev(table), _dev(np.array(lens, np.int32)),
                           return_lse=True)
    _check_attn(got, want, "f16", D, 0.0)
    # and stores to them
    x = to_dev(_rand(rng, (3, 4 + 2 * Hkv, D), "f16"), "f16")
    slots = _dev(np.array([9, 2, 4], np.int32))
    _, ko = fk.fk_qk_norm_rope(x[:, :4], x[:, 4:6], x[:, 6:], slots=slots, k_cache=kd, v_cache=vd,
                               k_out=torch.empty(3, Hkv, D, dtype=torch.float16, device="cuda"))
    for t, s in enumerate((9, 2, 4)):
        assert torch.equal(kd[s // page, s % page], ko[t]) and torch.equal(vd[s // page, s % page], x[t, 6:])


def test_step_in_a_graph(fk):
    """A decode step (tables, norm + rotation + stores, attention) captured once
    and replayed with new lengths and inputs, against the same calls run eagerly."""
    torch = _torch()
    i32, dt = torch.int32, torch.bfloat16
    B, Hq, Hkv, D, page, width = 5, 8, 2, 128, 16, 24
    pages = B * width
    rng = np.random.default_rng(11)
    gen = torch.Generator(device="cuda").manual_seed(12)

    def state():
        return dict(kc=torch.zeros(pages, page, Hkv, D, dtype=dt, device="cuda"),
                    vc=torch.zeros(pages, page, Hkv, D, dtype=dt, device="cuda"),
                    old=torch.zeros(B, dtype=i32, device="cuda"), new=torch.zeros(B, dtype=i32, device="cuda"),
                    table=torch.full((B, width), -1, dtype=i32, device="cuda"),
                    free=torch.zeros(B, dtype=i32, device="cuda"),
                    qkv=torch.zeros(B, Hq + 2 * Hkv, D, dtype=dt, device="cuda"),
                    out=[torch.empty(s, dtype=i32, device="cuda") for s in ((B, width), (B,), (B + 1,), (B + 1,), (B,), (B,))])

    w = torch.ones(D, dtype=dt, device="cuda")
    rope = torch.rand(page * width, D, device="cuda", generator=gen)

    def step(s):
        table, lens, _, _, slots, pos = fk.fk_page_tables(s["old"], s["new"], s["free"], page, width, B,
                                                          table=s["table"], out=s["out"])
        q, _ = fk.fk_qk_norm_rope(s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hkv], s["qkv"][:, Hq + Hkv:], w, w,
                                  1e-6, rope, pos, False, slots, s["kc"], s["vc"])
        return fk.fk_paged_attn(q, s["kc"], s["vc"], table, lens, return_lse=True)

    a, b = state(), state()
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step(a)
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(a)
    a2 = state()                             # what the capture warmed up is undone
    for n in ("kc", "vc", "old", "table"):
        a[n].copy_(a2[n])
    old, taken = np.zeros(B, np.int32), 0
    for it in range(40):
        new = (rng.random(B) < 0.8).astype(np.int32)
        need = int((-(-(old + new) // page) - -(-old // page)).sum())
        free = torch.arange(taken, taken + B, dtype=i32, device="cuda") % pages
        qkv = torch.randn(B, Hq + 2 * Hkv, D, device="cuda", generator=gen).to(dt)
        for s in (a, b):
            s["new"].copy_(_dev(new))
            s["free"].copy_(free)
            s["qkv"].copy_(qkv)
        graph.replay()
        want = step(b)
        torch.cuda.synchronize()
        assert torch.equal(held[0], want[0]) and torch.equal(held[1], want[1]), it
        assert torch.equal(a["kc"], b["kc"]) and torch.equal(a["out"][0], b["out"][0])
        for s in (a, b):
            s["table"].copy_(s["out"][0])
            s["old"].copy_(s["out"][1])
        old, taken = old + new, taken + need

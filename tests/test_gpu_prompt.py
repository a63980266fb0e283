"""Prompt attention on the GPU against the fp64 oracle.

Error bounds as for single-token attention (u = 2^-24; U = 2^-11 fp16, 2^-8 bf16,
2^-24 fp32), with one more term: a score is off by e_s = (D + 8) u S + cap 2^-20, S the
largest scale * sum |q_i k_i|; a weight relatively by 2 e_s, by 2^-20 for the
exponentials, by one rounding to the cache's type P (2^-8 bf16, 2^-11 fp16 and 2^-38 of
the largest for each key, 0 fp32), and sums over n keys by (n + 16) u. With R the sum
of these, the result is off by E = 2 R V + U (|out| + 2 R V), V the largest |v|; lse,
whose sum takes the probabilities before they are rounded, by e_s + R + 2^-22 |lse|.
"""
import math

import numpy as np
import pytest

import oracle
import synthdata
from gpu_helpers import host_f64, to_dev

pytestmark = pytest.mark.gpu

UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U32 = 2.0 ** -24
DTYPES = ["f16", "bf16", "f32"]


def _torch():
    import torch
    return torch


def _dev(a):
    return _torch().from_numpy(np.ascontiguousarray(a)).cuda()


def _rand(rng, shape, dtype, scale=1.0):
    return synthdata.to_storage((rng.standard_normal(shape) * scale).astype(np.float32), dtype)


def _case(case, dtype, seed):
    """Inputs with NaN wherever nothing may be read from: unused slots, tokens past a request's
    end, keys with bias -inf, rows of q that no request has."""
    torch = _torch()
    Hq, Hkv, D, page, reqs, bias, cap, how = case
    rng = np.random.default_rng(seed)
    B, lens = len(reqs), [max(a + n, 0) for a, n in reqs]
    cu = np.concatenate([[0], np.cumsum([n for _, n in reqs])]).astype(np.int32)
    T = int(cu[-1]) + 3
    held = [-(-n // page) for n in lens]
    width = max(1, max(held)) + 1
    pages = sum(held) + 3
    perm = rng.permutation(pages).astype(np.int32)
    table = np.where(rng.random((B, width)) < 0.5, -1, pages + 5).astype(np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = perm[at:at + h]
        at += h
    if how == "holes" and held[0] > 2:
        table[0, 1], table[0, 2] = -1, pages         # their keys are left out
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
        if bias == "none":                           # next to nothing left
            kb[:] = -np.inf
            kb[table[0, 0], page // 2] = 0.5
        if bias == "lowest":                         # the type's lowest value masks by absorbing the score
            kb = np.where(rng.random(kb.shape) < 0.5, np.finfo(np.float32).min, kb).astype(np.float32)
            for j in range(lens[-1]):
                kb[table[-1, j // page], j % page] = np.finfo(np.float32).min
    q = _rand(rng, (T, Hq, D), dtype, 2.0)
    k, v = (_rand(rng, (pages, page, Hkv, D), dtype) for _ in range(2))
    qd, kd, vd = (to_dev(t, dtype) for t in (q, k, v))
    qd[int(cu[-1]):] = math.nan
    dead = torch.from_numpy(~used).cuda()[:, :, None].expand(pages, page, Hkv).clone()
    if kb is not None:
        dead |= torch.from_numpy(kb == -np.inf).cuda()
    kd[dead] = math.nan
    vd[dead] = math.nan
    kbd = None if kb is None else _dev(np.where(used[:, :, None], kb, np.nan).astype(np.float32))
    td = _dev(table)
    if how == "heads":                               # heads before tokens in memory
        kd, vd = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (kd, vd))
        qd = qd.transpose(0, 1).contiguous().transpose(0, 1)
    elif how == "wide":                              # keys and values side by side, q inside a projection
        both = torch.cat([kd, vd], -1)
        kd, vd = both[..., :D], both[..., D:]
        td = torch.cat([td, torch.full_like(td, 1 << 30)], 1)[:, :width]
        qd = torch.cat([torch.full_like(qd, math.nan), qd], 1)[:, Hq:]
    elif how == "odd":
        def odd(t, gap):
            s = (page * Hkv * (D + 1) + 1, Hkv * (D + 1), D + 1, 1)
            buf = torch.full((pages * s[0] + 9,), math.nan, dtype=t.dtype, device="cuda")
            o = buf.as_strided(t.shape, s, gap)
            o.copy_(t)
            return o
        kd, vd = odd(kd, 1), odd(vd, 3)
    scale = 1.0 / math.sqrt(D)
    want = oracle.prompt_attn(synthdata.to_f64(q, dtype), synthdata.to_f64(k, dtype), synthdata.to_f64(v, dtype),
                              table, lens, cu, scale, cap, None if kb is None else kb.astype(np.float64))
    args = dict(q=qd, k_cache=kd, v_cache=vd, table=td, lens=_dev(np.array([a + n for a, n in reqs], np.int32)),
                cu_tokens=_dev(cu), softcap=cap, key_bias=kbd)
    return args, want


def _call(fk, args, dtype, **kw):
    """A call whose outputs hold a mark before it: (out, lse), rows of no request checked."""
    torch = _torch()
    T, Hq, D = args["q"].shape
    out = torch.full((T, Hq, D), 7.0, dtype=args["q"].dtype, device="cuda")
    lse = torch.full((T, Hq), 7.0, dtype=torch.float32, device="cuda")
    got = fk.fk_prompt_attn(out=out, lse=lse, **args, **kw)
    end = int(args["cu_tokens"][-1])
    assert (out[end:] == 7).all() and (lse[end:] == 7).all()
    return got


def _check(got, want, dtype, D, cap, where=""):
    ref, rlse, info = want
    own = ~np.isnan(rlse[:, 0])
    out, lse = host_f64(got[0], dtype)[own], got[1].double().cpu().numpy()[own]
    ref, rlse, info = ref[own], rlse[own], info[own]
    S, V, n = (info[..., i][..., None] for i in (1, 2, 3))
    e_s = (D + 8) * U32 * S + cap * 2.0 ** -20
    P = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11 + n * 2.0 ** -38, "f32": 0.0}[dtype]
    R = 2 * e_s + P + 2.0 ** -20 + (n + 16) * U32
    tol = 2 * R * V + UNIT[dtype] * (np.abs(ref) + 2 * R * V) + (2.0 ** -25 if dtype == "f16" else 0)
    err = np.abs(out - ref)
    assert (err <= tol).all(), (where, "out", float((err / np.maximum(tol, 1e-300)).max()),
                                np.argwhere(~(err <= tol))[:4].tolist())
    none = rlse == -np.inf
    assert np.array_equal(none, lse == -np.inf), where
    assert (out[none] == 0).all(), where
    err = np.abs(lse[~none] - rlse[~none])
    tol = (e_s + R)[..., 0][~none] + 2.0 ** -22 * np.abs(rlse[~none])
    assert (err <= tol).all(), (where, "lse", float((err / tol).max()))


CASES = [
    # Hq, Hkv, D, page, [(held before, new)], bias, cap, layout
    (1, 1, 64, 16, [(0, 1)], None, 0.0, "plain"),
    (4, 2, 64, 16, [(0, 33), (7, 0), (100, 1), (0, 64)], None, 0.0, "plain"),
    (8, 2, 128, 16, [(0, 130), (60, 5), (3, 70)], None, 0.0, "holes"),
    (8, 2, 128, 24, [(200, 40), (0, 100)], "log", 30.0, "wide"),
    (5, 1, 80, 20, [(0, 77), (130, 3)], "log", 0.0, "plain"),
    (6, 6, 96, 1, [(0, 100), (31, 1)], None, 12.0, "heads"),
    (2, 2, 32, 7, [(64, 64), (0, 0), (0, 63)], "none", 0.0, "plain"),
    (3, 1, 256, 16, [(0, 90), (64, 2)], None, 0.0, "plain"),
    (3, 1, 192, 64, [(1, 65), (0, 31)], "lowest", 0.0, "heads"),
    (40, 2, 64, 16, [(0, 30), (90, 4)], "log", 0.0, "plain"),       # 20 query heads a key head
    (16, 1, 128, 48, [(300, 7), (0, 20)], None, 20.0, "plain"),
    (300, 1, 64, 16, [(10, 3), (0, 2)], None, 0.0, "plain"),        # more than a block's rows a token
    (4, 4, 128, 16, [(-5, 40), (0, 20)], None, 0.0, "plain"),       # fewer keys held than tokens new
    (3, 3, 33, 4, [(0, 50), (20, 5)], "log", 10.0, "plain"),        # odd rows
    (2, 1, 20, 3, [(0, 65), (9, 1)], None, 0.0, "odd"),
    (2, 1, 320, 16, [(20, 30)], "log", 0.0, "plain"),               # wide heads
    (2, 2, 1000, 16, [(0, 20)], None, 0.0, "plain"),
    (2, 1, 128, 16, [(0, 600), (1500, 3)], None, 0.0, "plain"),
    (1, 1, 72, 16, [(2000, 70)], "lowest", 0.0, "wide"),
]
IDS = [f"{c[0]}x{c[1]}d{c[2]}p{c[3]}{c[5] or ''}{c[7]}" for c in CASES]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_prompt_attn(fk, case, dtype):
    args, want = _case(case, dtype, seed=case[2] + len(case[4]))
    for hint in (0, 1, max(a + n for a, n in case[4])):     # how the work is split goes by max_len
        _check(_call(fk, args, dtype, max_len=hint), want, dtype, case[2], case[6], f"max_len {hint}")

"""Paged attention, and norm + rotation, where what counts is infinite or NaN, against
what the formulas give for it in IEEE arithmetic:

  * a key whose score is -inf has weight 0 and drops out: the result is the one
    without it (the oracle's, with that key masked);
  * a request whose keys are all masked gives 0 and -inf, whatever its query holds;
  * an infinite value gives an infinite element, a NaN one NaN, and the others stay as they are;
  * NaN in a key reaches its request and the query heads of its cache head, and no others;
  * a row that is not finite spoils itself, unnormed only its pairs, and values keep their bits.

Error bounds of the finite results are those of test_gpu_kv_cache.py.
"""
import math

import numpy as np
import pytest

import oracle
import synthdata
from gpu_helpers import host_f64, to_dev
from test_gpu_kv_cache import _check_attn, _dev, _rand

pytestmark = pytest.mark.gpu

DTYPES = ["f16", "bf16", "f32"]
# rows narrower than the tile that holds them, rows that fill it, and rows of odd size
DIMS = [(2, 1, 24), (6, 2, 72), (4, 2, 80), (17, 1, 96), (2, 1, 160), (3, 1, 200), (4, 2, 64), (8, 2, 128),
        (2, 1, 256), (3, 3, 33), (2, 1, 320)]
LENS = [70, 5, 700]


def _case(Hq, Hkv, D, dtype, lens, seed):
    """Inputs with one page per 16 tokens, in order of requests, and their fp64 values."""
    rng = np.random.default_rng(seed)
    page, B = 16, len(lens)
    held = [-(-n // page) for n in lens]
    table = np.full((B, max(held)), -1, np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = np.arange(at, at + h)
        at += h
    q, k, v = _rand(rng, (B, Hq, D), dtype), *(_rand(rng, (at, page, Hkv, D), dtype) for _ in range(2))
    f64 = [synthdata.to_f64(t, dtype) for t in (q, k, v)]
    dev = [to_dev(t, dtype) for t in (q, k, v)]
    return dev, f64, table


def _wide(table):
    """Room for 2^20 keys a request: the plan of large caches."""
    return np.concatenate([table, np.full((table.shape[0], 1 << 16), -1, np.int32)], 1)


def _all_plans(fk, q, k, v, table, lens, D, check, **kw):
    ls = _dev(np.array(lens, np.int32))
    for tab, hint in ((table, 1), (table, max(lens)), (table, 0), (_wide(table), 0)):
        check(fk.fk_paged_attn(q, k, v, _dev(tab), ls, max_len=hint, return_lse=True, **kw))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dims", DIMS, ids=[f"{a}x{b}d{d}" for a, b, d in DIMS])
def test_keys_of_score_minus_infinity_drop_out(fk, dims, dtype):
    Hq, Hkv, D = dims
    (q, k, v), (q64, k64, v64), table = _case(Hq, Hkv, D, dtype, LENS, D)
    q[..., :2] = q[..., :2].abs() + 0.5             # -inf times these is -inf for every head
    q64 = host_f64(q, dtype)
    bias = np.zeros(k64.shape[:3])
    for page, tok, e in ((0, 0, 0), (1, 3, 1), (4, 2, 0), (table[1, 0], 4, 1), (table[2, 20], 15, 0)):
        k[page, tok, :, e] = -math.inf
        bias[page, tok] = -math.inf
    want = oracle.paged_attn(q64, k64, v64, table, LENS, D ** -0.5, 0.0, bias)
    _all_plans(fk, q, k, v, table, LENS, D, lambda got: _check_attn(got, want, dtype, D, 0.0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("masked", ["pages", "bias"])
@pytest.mark.parametrize("dims", [(4, 2, 64), (8, 2, 128), (40, 2, 96), (2, 1, 256), (3, 3, 33)],
                         ids=["d64", "d128", "g20d96", "d256", "d33"])
def test_nothing_left_whatever_the_query_holds(fk, dims, masked, dtype):
    import torch

    Hq, Hkv, D = dims
    lens = [70, 5, 700, 40]
    (q, k, v), (q64, k64, v64), table = _case(Hq, Hkv, D, dtype, lens, D + 1)
    q[0], q[2, :, 1] = math.nan, math.inf
    bias = np.zeros(k64.shape[:3], np.float32)
    if masked == "pages":
        table = np.where(np.isin(np.arange(4), (0, 2))[:, None], -1, table).astype(np.int32)
    else:
        for b in (0, 2):
            bias[table[b, :-(-lens[b] // 16)]] = -np.inf
    want = oracle.paged_attn(np.nan_to_num(q64), k64, v64, table, lens, D ** -0.5, 0.0, bias.astype(np.float64))
    assert (want[1][[0, 2]] == -np.inf).all()
    for kw in ({}, dict(softcap=9.0)):
        if masked == "bias" or kw:
            kw["key_bias"] = _dev(bias)
        if kw.get("softcap"):
            want = oracle.paged_attn(np.nan_to_num(q64), k64, v64, table, lens, D ** -0.5, 9.0,
                                     bias.astype(np.float64))
        _all_plans(fk, q, k, v, table, lens, D,
                   lambda got: _check_attn(got, want, dtype, D, kw.get("softcap", 0.0)), **kw)
    # a query that is NaN and has keys is NaN, and no other request is
    q2 = torch.zeros_like(q)
    q2[1, 0, 0] = math.nan
    out, lse = fk.fk_paged_attn(q2, k, v, _dev(table), _dev(np.array(lens, np.int32)), key_bias=_dev(bias),
                                return_lse=True)
    assert out[1, 0].isnan().all() and lse[1, 0].isnan()
    assert not out[1, 1:].isnan().any() and not out[[0, 2, 3]].isnan().any() and not lse[[0, 2, 3]].isnan().any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dims", DIMS, ids=[f"{a}x{b}d{d}" for a, b, d in DIMS])
def test_infinite_and_nan_values_stay_in_their_element(fk, dims, dtype):
    Hq, Hkv, D = dims
    (q, k, v), (q64, k64, v64), table = _case(Hq, Hkv, D, dtype, LENS, D + 2)
    q *= 0.125                                       # scores of a few tenths: no weight underflows
    q64 = host_f64(q, dtype)
    want = oracle.paged_attn(q64, k64, v64, table, LENS, D ** -0.5)
    put = {0: (0, 1, 3, math.inf), 1: (table[1, 0], 4, D - 1, -math.inf), 2: (table[2, 40], 0, D // 2, math.nan)}
    for page, tok, e, x in put.values():
        v[page, tok, :, e] = x
    for b in range(len(LENS)):
        for at in range(0, LENS[b], 9):              # and, in one element, an infinity at many keys
            v[table[b, at // 16], at % 16, :, 5] = math.inf

    def check(got):
        out = got[0].double().cpu().numpy()
        for b, (_, _, e, x) in put.items():
            assert np.isnan(out[b, :, e]).all() if x != x else (out[b, :, e] == x).all(), (b, e)
            assert (out[b, :, 5] == np.inf).all(), b
            out[b, :, [e, 5]] = want[0][b, :, [e, 5]]
        fixed = to_dev(synthdata.to_storage(out.astype(np.float32), dtype), dtype)
        _check_attn((fixed, got[1]), want, dtype, D, 0.0)

    _all_plans(fk, q, k, v, table, LENS, D, check)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dims", DIMS, ids=[f"{a}x{b}d{d}" for a, b, d in DIMS])
def test_nan_keys_reach_their_request_and_head_only(fk, dims, dtype):
    Hq, Hkv, D = dims
    (q, k, v), (q64, k64, v64), table = _case(Hq, Hkv, D, dtype, LENS, D + 3)
    want = oracle.paged_attn(q64, k64, v64, table, LENS, D ** -0.5)
    k[table[2, 3], 7, Hkv - 1, D - 1] = math.nan

    def check(got):
        G = Hq // Hkv
        assert got[0][2, -G:].isnan().all() and got[1][2, -G:].isnan().all()
        out, lse = got[0].clone(), got[1].clone()
        out[2, -G:], lse[2, -G:] = (_like(w[2, -G:], t) for w, t in zip(want, (out, lse)))
        _check_attn((out, lse), want, dtype, D, 0.0)

    _all_plans(fk, q, k, v, table, LENS, D, check)


def _like(a, t):
    import torch
    return torch.from_numpy(a).to(t.dtype).to(t.device)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(128, 128, False), (128, 12, False), (96, 40, True), (33, 20, False), (64, 0, False)],
                         ids=["whole", "exchange", "sides", "odd", "none"])
def test_rotation_of_rows_that_are_not_finite(fk, shape, dtype):
    """Infinities and NaN stay in their row, and unnormed in their pair; values keep their bits."""
    import torch

    D, rot, inter = shape
    rng = np.random.default_rng(D + rot)
    T, Hq, Hkv = 9, 5, 2
    x = to_dev(_rand(rng, (T, Hq + 2 * Hkv, D), dtype), dtype)
    bad = x.clone()
    bad[2, 1, 1], bad[4, 3, D - 1], bad[7, Hq, 0], bad[3, -1, 2] = math.nan, math.inf, -math.inf, math.nan
    w = to_dev(_rand(rng, D, dtype), dtype)
    kw = dict(interleaved=inter, slots=_dev(np.arange(T, dtype=np.int32)))
    if rot:
        kw.update(rope=_dev(rng.uniform(0.2, 0.9, (T, rot)).astype(np.float32)),
                  positions=_dev(np.arange(T, dtype=np.int32)))
    for ws in ((w, w), (None, None)):
        res = []
        for src in (x, bad):
            kc, vc = (torch.zeros(T, 1, Hkv, D, dtype=x.dtype, device="cuda") for _ in range(2))
            q, _ = fk.fk_qk_norm_rope(src[:, :Hq], src[:, Hq:Hq + Hkv], src[:, Hq + Hkv:], None, None, 1e-6,
                                      k_cache=kc, v_cache=vc, **kw) if ws[0] is None else \
                fk.fk_qk_norm_rope(src[:, :Hq], src[:, Hq:Hq + Hkv], src[:, Hq + Hkv:], *ws, k_cache=kc, v_cache=vc, **kw)
            res.append(torch.cat([q, kc[:, 0], vc[:, 0]], 1))
        same = (res[0] == res[1])
        rows = {(2, 1): 1, (4, 3): D - 1, (7, Hq): 0, (3, Hq + 2 * Hkv - 1): 2}
        for (t, h), e in rows.items():
            assert not res[1][t, h, e].isfinite()
            if ws[0] is None:                            # the element and its partner at most
                assert (~same[t, h]).sum() <= 2
            same[t, h] = True
        assert same.all()
        assert torch.equal(res[1][:, Hq + Hkv:].isnan(), bad[:, Hq + Hkv:].isnan())

"""How exact prompts and attention over 8 bits are, beyond the worst-case bounds of test_gpu_prompt.py and
test_gpu_cache8.py: root mean square errors over a call, as test_kv_accuracy.py holds fk_paged_attn to.
  * fp32 results and every lse: to a plain fp32 evaluation (numpy) of the same inputs, as there.
  * 16-bit results over 8 bits: 1.05 times the exact result's own rounding, as there (probabilities enter
    as two numbers).
  * 16-bit prompts: a probability is rounded once to the type, independently of the others: with values of
    unit variance the error is sqrt(sum p^2) of a rounding's, and so is the result's size, so it adds a rounding
    like the result's own: sqrt(2) times that, 1.05 allowed for again.
Tests on the CPU plant what these checks are for and see them fail.
"""
import math

import numpy as np
import pytest

from test_kv_accuracy import DTYPES, F, _rms, _round


def _inputs(seed, n, T, heads, groups, D, dtype):
    rng = np.random.default_rng(seed)
    return [_round(rng.standard_normal(s) * x, dtype)
            for s, x in (((heads, groups * T, D), 1.5), ((heads, n, D), 1.0), ((heads, n, D), 1.0))]


def _seen(n, T, groups):
    """Keys of row (group, token): the last T of n keys are the tokens'."""
    return np.arange(n)[None] <= np.tile(np.arange(n - T, n), groups)[:, None]


def _attend(q, k, v, seen, f):
    out, lse = np.empty(q.shape), np.empty(q.shape[:2])
    for h in range(q.shape[0]):
        s = (q[h].astype(f) * f(1 / math.sqrt(q.shape[-1]))) @ np.ascontiguousarray(k[h].T.astype(f))
        s = np.where(seen, s, f(-np.inf))
        top = s.max(-1, keepdims=True)
        p = np.exp(s - top)
        total = p.sum(-1, keepdims=True)
        out[h], lse[h] = p @ v[h].astype(f) / total, (top + np.log(total))[:, 0]
    return out, lse


def _check(out, lse, q, k, v, seen, dtype, roundings, where=""):
    ref, rlse = _attend(q, k, v, seen, np.float64)
    plain, plse = _attend(q, k, v, seen, F)
    if dtype == "f32":
        most = 2 * _rms(plain - ref)
    else:
        most = 1.05 * math.sqrt(roundings) * _rms(_round(ref, dtype) - ref)
    assert _rms(out - ref) <= most, (where, "out", _rms(out - ref) / most)
    most = 3 * _rms(plse - rlse) + 2.0 ** -24 * np.abs(rlse).max() + (2.0 ** -21 if dtype == "f16" else 0)
    assert _rms(lse - rlse) <= most, (where, "lse", _rms(lse - rlse) / most)


@pytest.mark.parametrize("dtype", DTYPES)
def test_planted_mistakes_are_seen(dtype):
    n, T, G, D = 500, 60, 2, 64
    q, k, v = _inputs(1, n, T, 2, G, D, dtype)
    seen = _seen(n, T, G)
    ref, rlse = _attend(q, k, v, seen, np.float64)
    lse32 = rlse.astype(F).astype(np.float64)
    _check(_round(ref, dtype), lse32, q, k, v, seen, dtype, 1)

    def rounded(values, sums):                           # the weights of values and of the sum as given
        out, lse = np.empty(q.shape), np.empty(q.shape[:2])
        for h in range(2):
            s = np.where(seen, q[h] @ k[h].T / math.sqrt(D), -np.inf)
            top = s.max(-1, keepdims=True)
            p = np.exp(s - top)
            out[h] = values(p) @ v[h] / sums(p).sum(-1, keepdims=True)
            lse[h] = (top + np.log(sums(p).sum(-1, keepdims=True)))[:, 0]
        return _round(out, dtype), lse.astype(F).astype(np.float64)

    same, narrow = lambda p: p, "f16" if dtype == "f32" else dtype
    once = rounded(lambda p: _round(p, narrow), same)
    with pytest.raises(AssertionError, match="out"):
        _check(*once, q, k, v, seen, dtype, 1)
    if dtype != "f32":
        _check(*once, q, k, v, seen, dtype, 2)
    with pytest.raises(AssertionError, match="lse"):
        _check(ref if dtype == "f32" else _round(ref, dtype), rounded(same, lambda p: _round(p, narrow))[1], q, k, v, seen, dtype, 2)
    if dtype == "f16":                                   # fewer bits than the type's
        with pytest.raises(AssertionError, match="out"):
            _check(*rounded(lambda p: _round(p, "bf16"), same), q, k, v, seen, dtype, 2)
    with pytest.raises(AssertionError):                  # values narrowed on the way
        wrong = v * (1 + 2.0 ** -8) if dtype == "bf16" else _round(v, "bf16")
        _check(_round(_attend(q, k, wrong, seen, np.float64)[0], dtype), lse32, q, k, v, seen, dtype, 2)


CASES = [  # query heads, cache heads, elements, keys, tokens
    (16, 4, 128, 700, 300), (8, 2, 64, 500, 500), (16, 1, 256, 900, 64), (6, 2, 96, 1500, 33), (6, 2, 192, 300, 300),
    (4, 4, 32, 600, 257), (8, 2, 33, 500, 60), (6, 2, 90, 1200, 9), (4, 2, 320, 300, 80), (8, 8, 80, 64, 64)]


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}x{c[1]}d{c[2]}n{c[3]}t{c[4]}" for c in CASES])
def test_prompts(fk, case, dtype):
    import torch
    from gpu_helpers import torch_dtype

    Hq, Hkv, D, n, T = case
    G, page, dt = Hq // Hkv, 16, torch_dtype(dtype)
    q, k, v = _inputs(D + n, n, T, Hkv, G, D, dtype)
    pages = -(-n // page)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda()      # noqa: E731

    def cache(a):
        return dev(np.concatenate([a.transpose(1, 0, 2), np.zeros((pages * page - n, Hkv, D))]).reshape(pages, page, Hkv, D))

    qd = dev(q.reshape(Hq, T, D).transpose(1, 0, 2))
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages)
    for hint in (0, 1):
        out, lse = fk.fk_prompt_attn(qd, cache(k), cache(v), table, _i32([n]), _i32([0, T]), max_len=hint, return_lse=True)
        _check(out.double().cpu().numpy().transpose(1, 0, 2).reshape(q.shape), lse.double().cpu().numpy().T.reshape(q.shape[:2]),
               q, k, v, _seen(n, T, G), dtype, 2, f"max_len {hint}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", [(16, 4, 128, 3000), (8, 2, 64, 700), (16, 1, 256, 1500), (6, 2, 96, 900), (6, 2, 192, 500),
                                  (40, 2, 128, 600), (8, 2, 33, 500), (4, 2, 320, 300)], ids=lambda c: f"{c[0]}x{c[1]}d{c[2]}")
def test_8bit_cache(fk, case, dtype):
    import torch
    from gpu_helpers import torch_dtype

    Hq, Hkv, D, n = case
    G, page, dt = Hq // Hkv, 16, torch_dtype(dtype)
    q, k, v = _inputs(D + n, n, 1, Hkv, G, D, dtype)
    pages = -(-n // page)
    code = lambda a: torch.from_numpy(np.concatenate([a.transpose(1, 0, 2), np.zeros((pages * page - n, Hkv, D))])      # noqa: E731
                                      .reshape(pages, page, Hkv, D)).float().cuda().to(torch.float8_e4m3fn)
    kc, vc = code(k), code(v)
    k, v = (c.double().cpu().numpy().reshape(-1, Hkv, D)[:n].transpose(1, 0, 2) for c in (kc, vc))
    one = torch.ones((pages, page, Hkv), device="cuda")
    qd = torch.from_numpy(q.reshape(1, Hq, D)).to(dt).cuda()
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages)
    for hint in (0, 1, n):
        out, lse = fk.fk_paged_attn8(qd, kc, vc, one, one, table, _i32([n]), max_len=hint, return_lse=True)
        _check(out.double().cpu().numpy().reshape(q.shape), lse.double().cpu().numpy().reshape(q.shape[:2]), q, k, v,
               _seen(n, 1, G), dtype, 1, f"max_len {hint}")

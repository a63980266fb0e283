"""How exact single-token attention is, beyond the worst-case bounds of test_gpu_kv_cache.py.

Those bounds hold for any input and are far above the usual error: probabilities of 8 or 11
bits would pass them. Here the error's root mean square over a request is held against
  * 16-bit results: that of the exact result rounded once, times 1.05. An error of a fifth
    of that rounding, independent of it, is 1.02; probabilities rounded once to the type
    are as large as the rounding itself and give 1.4.
  * fp32 results: that of a plain fp32 evaluation (numpy) of the same inputs, times 2. In an
    emulation of the kernel's order of operations the ratio is 0.5 to 1.15.
  * lse, fp32 whatever the type: the plain evaluation's times 3, plus a rounding of its own
    size, plus for fp16, whose sums are scaled by 2^14, half a unit of the scaled log, 2^-21.
Scores under a large cap: the score's own rounding, (D + 24) 2^-24 of it, not the cap's.
Tests on the CPU plant the mistakes that these checks are for and see them fail.
"""
import math

import numpy as np
import pytest

DTYPES = ["f16", "bf16", "f32"]
F = np.float32


def _round(a, dtype):
    import torch
    t = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    return torch.from_numpy(np.ascontiguousarray(a)).to(t).double().numpy()


def _rms(a):
    return math.sqrt(float((np.asarray(a, np.float64) ** 2).mean()))


def _inputs(seed, n, heads, groups, D, dtype):
    """q (heads, groups, D), k and v (n, heads, D), values of the type, in float64."""
    rng = np.random.default_rng(seed)
    return (_round(rng.standard_normal(s) * x, dtype)
            for s, x in (((heads, groups, D), 1.5), ((n, heads, D), 1.0), ((n, heads, D), 1.0)))


def _exact(q, k, v):
    s = np.einsum("hgd,nhd->hgn", q, k) / math.sqrt(q.shape[-1])
    top = s.max(-1, keepdims=True)
    w = np.exp(s - top)
    total = w.sum(-1, keepdims=True)
    return np.einsum("hgn,nhd->hgd", w / total, v), (top + np.log(total))[..., 0]


def _plain32(q, k, v):
    out, lse = np.empty(q.shape), np.empty(q.shape[:2])
    for h in range(q.shape[0]):
        s = (q[h].astype(F) * F(1 / math.sqrt(q.shape[-1]))) @ np.ascontiguousarray(k[:, h].T.astype(F))
        top = s.max(-1, keepdims=True)
        p = np.exp(s - top)
        total = p.sum(-1, keepdims=True)
        out[h], lse[h] = p @ np.ascontiguousarray(v[:, h].astype(F)) / total, (top + np.log(total))[:, 0]
    return out, lse


def _check(out, lse, q, k, v, dtype, where=""):
    ref, rlse = _exact(q, k, v)
    plain, plse = _plain32(q, k, v)
    if dtype == "f32":
        most = 2 * _rms(plain - ref)
    else:
        most = 1.05 * _rms(_round(ref, dtype) - ref)
    assert _rms(out - ref) <= most, (where, "out", _rms(out - ref) / most)
    most = 3 * _rms(plse - rlse) + 2.0 ** -24 * np.abs(rlse).max() + (2.0 ** -21 if dtype == "f16" else 0)
    assert _rms(lse - rlse) <= most, (where, "lse", _rms(lse - rlse) / most)


# ---------------------------------------------------------------------------
# mistakes, on the CPU
# ---------------------------------------------------------------------------
def _with(q, k, v, dtype, value_weight=lambda p: p, sum_weight=lambda p: p):
    """The formula with the weights of values and of the sum rounded as given."""
    s = np.einsum("hgd,nhd->hgn", q, k) / math.sqrt(q.shape[-1])
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    total = sum_weight(p).sum(-1, keepdims=True)
    out = np.einsum("hgn,nhd->hgd", value_weight(p), v) / total
    return _round(out, dtype), (top + np.log(total))[..., 0].astype(F).astype(np.float64)


def _two(p, dtype):
    """hi rounded down and lo to nearest, fp16 scaled by 2^14: the sum the kernel multiplies."""
    scale = 2.0 ** 14 if dtype == "f16" else 1.0
    hi = _round(p * scale, dtype)
    step = 2.0 ** (np.floor(np.log2(p * scale)) - (10 if dtype == "f16" else 7))
    hi = np.where(hi > p * scale, hi - step, hi)
    return (hi + _round(p * scale - hi, dtype)) / scale


@pytest.mark.parametrize("n", [40, 900])
@pytest.mark.parametrize("dtype", DTYPES)
def test_planted_mistakes_are_seen(dtype, n):
    q, k, v = _inputs(n, n, 2, 8, 128, dtype)
    narrow = "f16" if dtype == "f32" else dtype
    args = (q, k, v, dtype)
    _check(*_with(*args), *args)
    if dtype != "f32":
        _check(*_with(*args, value_weight=lambda p: _two(p, dtype)), *args)
    with pytest.raises(AssertionError, match="out"):
        _check(*_with(*args, value_weight=lambda p: _round(p, narrow)), *args)
    with pytest.raises(AssertionError, match="lse"):
        _check(_with(*args)[0], _with(*args, sum_weight=lambda p: _round(p, narrow))[1], *args)
    with pytest.raises(AssertionError):          # values narrowed on the way
        _check(*_with(q, k, _round(v, "bf16") if dtype != "bf16" else v * (1 + 2.0 ** -9), dtype), *args)


def _small_scores(D, n, dtype):
    """Queries and keys above 0, so that scores have no cancellation: 1e-3 to 1."""
    rng = np.random.default_rng(D)
    q = _round(rng.uniform(0.5, 1.0, (n, 1, D)) * 10.0 ** rng.uniform(-3, 0, (n, 1, 1)), dtype)
    k = _round(rng.uniform(0.5, 1.0, (n, 1, D)) / math.sqrt(D), dtype)
    return q, k, (q * k).sum(-1) / math.sqrt(D)


def _check_small(lse, raw, cap, D, dtype):
    want = cap * np.tanh(raw / cap)
    tol = (D + 24) * 2.0 ** -24 * want + (2.0 ** -19 if dtype == "f16" else 0)
    assert (np.abs(lse - want) <= tol).all(), float((np.abs(lse - want) / tol).max())


def test_planted_cap_rounding_is_seen():
    _, _, raw = _small_scores(128, 64, "f32")
    _check_small((50 * np.tanh(raw / 50)).astype(F).astype(np.float64), raw, 50.0, 128, "f32")
    e = np.exp(F(2) * raw.astype(F) / F(50))
    with pytest.raises(AssertionError):
        _check_small((F(50) - F(100) / (e + F(1))).astype(np.float64), raw, 50.0, 128, "f32")


# ---------------------------------------------------------------------------
# the kernels
# ---------------------------------------------------------------------------
CASES = [  # query heads, cache heads, elements, lengths
    (16, 4, 128, [3000, 40]), (8, 2, 64, [700, 12]), (16, 1, 256, [1500, 64]), (6, 2, 96, [900, 33]),
    (6, 2, 192, [500, 20]), (40, 2, 128, [600, 100]), (16, 4, 32, [2000, 17]), (8, 2, 33, [500, 60]),
    (4, 2, 320, [300, 40])]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}x{c[1]}d{c[2]}" for c in CASES])
def test_rms_error(fk, case, dtype):
    import torch
    from gpu_helpers import torch_dtype

    Hq, Hkv, D, lens = case
    sets = [list(_inputs(D + n, n, Hkv, Hq // Hkv, D, dtype)) for n in lens]
    page, dt = 16, torch_dtype(dtype)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda()      # noqa: E731
    held = [-(-n // page) for n in lens]
    table = np.full((len(lens), max(held)), -1, np.int32)
    pad = lambda a: np.concatenate([a, np.zeros((-len(a) % page,) + a.shape[1:])])  # noqa: E731
    for b, h in enumerate(held):
        table[b, :h] = sum(held[:b]) + np.arange(h)
    q = dev(np.stack([s[0].reshape(Hq, D) for s in sets]))
    kc, vc = (dev(np.concatenate([pad(s[i]) for s in sets]).reshape(-1, page, Hkv, D)) for i in (1, 2))
    ls, tb = (torch.from_numpy(np.asarray(a, np.int32)).cuda() for a in (lens, table))
    for hint in (0, 1, max(lens)):
        out, lse = fk.fk_paged_attn(q, kc, vc, tb, ls, max_len=hint, return_lse=True)
        for b, (q64, k64, v64) in enumerate(sets):
            _check(out[b].double().cpu().numpy().reshape(q64.shape), lse[b].double().cpu().numpy().reshape(q64.shape[:2]),
                   q64, k64, v64, dtype, f"{lens[b]} keys, max_len {hint}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128, 256, 33])
def test_small_scores_under_a_large_cap(fk, D, dtype):
    """One key a request, so that lse is its score."""
    import torch
    from gpu_helpers import torch_dtype

    n, dt = 64, torch_dtype(dtype)
    q, k, raw = _small_scores(D, n, dtype)
    dev = lambda a: torch.from_numpy(a).to(dt).cuda()      # noqa: E731
    kc = dev(k)[:, None]
    table, lens = torch.arange(n, dtype=torch.int32, device="cuda")[:, None], torch.ones(n, dtype=torch.int32, device="cuda")
    for cap in (30.0, 50.0, 1000.0):
        _, lse = fk.fk_paged_attn(dev(q), kc, kc, table, lens, softcap=cap, return_lse=True)
        _check_small(lse.double().cpu().numpy(), raw, cap, D, dtype)

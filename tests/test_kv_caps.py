"""Scores under large caps, in prompts and over the 8-bit cache, for every type.

cap tanh(s / cap) has to carry the rounding of the score and not that of the cap, as
fk_paged_attn's does: with one key a request lse is the score, off by (D + 24) 2^-24 of it and for
fp16, whose sums are scaled by a power of two, by 2^-19 (test_kv_accuracy.py). 16-bit prompts and 16-bit
queries over 8 bits take a cheaper form below a cap of 64 (the header says so), which is off by up to 8
units of 2^-24 of the cap: an exponential and a reciprocal of one unit in the last place, 2^-23, each, and
the sum e + 1 rounded, through 1 - 2 / (e + 1).
"""
import math

import numpy as np
import pytest

from test_kv_accuracy import DTYPES, _check_small, _small_scores

pytestmark = pytest.mark.gpu

LARGE = (65.0, 1000.0, 1e4, 1e6, 1e8)
SMALL = (1.0, 30.0, 64.0)


def _check(lse, raw, cap, D, dtype):
    if cap > 64 or dtype == "f32":
        _check_small(lse, raw, cap, D, dtype)
    else:
        want = cap * np.tanh(raw / cap)
        tol = (D + 24) * 2.0 ** -24 * want + cap * 2.0 ** -21 + (2.0 ** -19 if dtype == "f16" else 0)
        assert (np.abs(lse - want) <= tol).all(), (cap, float((np.abs(lse - want) / tol).max()))


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [32, 64, 128, 192, 256, 33, 320])
def test_prompts(fk, D, dtype):
    """n requests of one token and one key."""
    import torch
    from gpu_helpers import torch_dtype

    n, dt = 64, torch_dtype(dtype)
    q, k, raw = _small_scores(D, n, dtype)
    qd, kc = (torch.from_numpy(a).to(dt).cuda() for a in (q, k[:, None]))
    for cap in LARGE + SMALL:
        _, lse = fk.fk_prompt_attn(qd, kc, kc.clone(), _i32([[i] for i in range(n)]), _i32([1] * n),
                                   _i32(list(range(n + 1))), softcap=cap, return_lse=True)
        _check(lse.double().cpu().numpy(), raw, cap, D, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128, 192, 256, 33, 320])
def test_8bit_cache(fk, D, dtype):
    import torch
    from gpu_helpers import torch_dtype

    n, dt = 64, torch_dtype(dtype)
    q, k, _ = _small_scores(D, n, dtype)
    codes = torch.from_numpy(k * math.sqrt(D)).float().cuda().to(torch.float8_e4m3fn)[:, None]
    raw = (q * codes.double().cpu().numpy()[:, 0]).sum(-1) * 0.125 / math.sqrt(D)
    scales = torch.full((n, 1, 1), 0.125, device="cuda")
    for cap in LARGE + SMALL:
        _, lse = fk.fk_paged_attn8(torch.from_numpy(q).to(dt).cuda(), codes, codes.clone(), scales, scales.clone(),
                                   _i32([[i] for i in range(n)]), _i32([1] * n), softcap=cap, return_lse=True)
        _check(lse.double().cpu().numpy(), raw, cap, D, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dims", [(8, 2, 128), (4, 1, 64), (3, 1, 200), (3, 3, 33)], ids=["d128", "d64", "d200", "d33"])
def test_prompts_of_many_keys(fk, dims, dtype):
    """Results under caps that leave the scores nearly as they are, held to the bound of a call
    without a cap."""
    import test_gpu_prompt as tp

    for cap in (100.0, 1e5, 1e7):
        args, want = tp._case((*dims, 16, [(0, 130), (300, 40), (0, 0), (70, 1)], "log", cap, "plain"), dtype, dims[2])
        tp._check(tp._call(fk, args, dtype), want, dtype, dims[2], 0.0, f"cap {cap}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dims", [(8, 2, 128), (40, 1, 64), (3, 1, 200), (3, 3, 33)], ids=["d128", "d64", "d200", "d33"])
def test_8bit_cache_of_many_keys(fk, dims, dtype):
    import test_gpu_cache8 as tc

    for cap in (100.0, 1e5, 1e7):
        args, want = tc._attn_case((*dims, 16, [700, 5, 0], "log", cap, "plain"), dtype, dims[2])
        tc._check_attn(fk.fk_paged_attn8(**args), want, dtype, dims[2], 0.0, f"cap {cap}")

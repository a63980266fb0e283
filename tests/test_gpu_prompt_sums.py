"""Prompt attention: fp32 sums over long keys, which are held apart in runs."""
import math

import numpy as np
import pytest

from gpu_helpers import host_f64

pytestmark = pytest.mark.gpu


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("D,heads", [(8, 1), (72, 1), (72, 128)], ids=["d8", "d72", "parts"])
def test_a_last_key_above_all_others(fk, D, heads):
    """One token over two runs of more than 2^15 steps, no multiple of it, none of which hides a key; the last
    key of all, and of the first run where two parts share the keys (128 heads), has a score 12 above the
    rest. Scores are 0 and 12, values quarters up to 1.25 and for the last keys 3 to 4: the sums of 2^15
    steps of up to 64 keys are whole quarters below 2^24 of them, exact in fp32. What is left are the
    exponential, 2^-20, and the scaling and joining of a few sums."""
    import torch
    step = 64 if D <= 64 else 32
    run, x = (1 << 15) + 40, 12.0
    n = 2 * run * step
    g = torch.Generator(device="cuda").manual_seed(D)
    k = torch.zeros((2, step, heads, D), device="cuda")
    k[1, step - 1, :, 0] = x
    v = (torch.randint(2, 6, (1, 1, heads, D), device="cuda", generator=g) * 0.25).repeat(2, step, 1, 1)
    v[1, step - 1] = torch.randint(12, 17, (heads, D), device="cuda", generator=g) * 0.25
    q = torch.zeros((1, heads, D), device="cuda")
    q[..., 0] = 1.0
    table = torch.zeros((1, 2 * run), dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    if heads > 1:
        table[0, run - 1] = 1
    out, lse = fk.fk_prompt_attn(q, k, v, table, _i32([n]), _i32([0, 1]), 1.0, max_len=1 if heads == 1 else 0,
                                 return_lse=True)
    count = 1 if heads == 1 else 2
    w = count * math.exp(x)
    v64 = host_f64(v, "f32")
    want = ((n - count) * v64[0, 0] + w * v64[1, -1]) / (n - count + w)
    assert np.abs(host_f64(out[0], "f32") / want - 1).max() <= 2.0 ** -16
    assert np.abs(lse.double().cpu().numpy() - math.log(n - count + w)).max() <= 2.0 ** -16


@pytest.mark.parametrize("D", [8, 72, 200])
def test_values_that_are_alike(fk, D):
    """One token over 2^22 keys and some, equal scores below the first key's and for each element equal values,
    so that every addition may round the same way: a run of up to 2^15 terms is off by 2^-10 of itself at
    most, 2^7 runs and their join by 2^-17, the exponential by 2^-20; the weights' sum, of up to 2^17 steps,
    by 2^-8."""
    import torch
    step, n = 64, (1 << 22) + 39
    x = 1.21484375
    g = torch.Generator(device="cuda").manual_seed(D)
    k = torch.zeros((2, step, 1, D), device="cuda")
    k[..., 0] = -x
    k[1, 0] = 0.0
    v = torch.rand((1, 1, 1, D), device="cuda", generator=g).add(0.5).repeat(2, step, 1, 1)
    q = torch.zeros((1, 1, D), device="cuda")
    q[..., 0] = 1.0
    table = torch.zeros((1, n // step + 1), dtype=torch.int32, device="cuda")
    table[0, 0] = 1
    for hint in (1, 0):
        out, lse = fk.fk_prompt_attn(q, k, v, table, _i32([n]), _i32([0, 1]), 1.0, max_len=hint, return_lse=True)
        assert np.abs(host_f64(out[0, 0], "f32") / host_f64(v[0, 0, 0], "f32") - 1).max() <= 2.0 ** -8 + 2.0 ** -9
        assert abs(float(lse) - math.log(1.0 + (n - 1) * math.exp(-x))) <= 2.0 ** -8

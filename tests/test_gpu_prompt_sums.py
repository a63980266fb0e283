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

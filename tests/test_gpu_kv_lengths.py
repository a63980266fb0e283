"""Paged attention at the largest lengths: 2^31 - 1 keys, more than the longest length
less a step's keys, through one page that every entry of the table repeats.

All keys of the page are one row and all values one row (token stride 0), so the result
is that value and lse is the score plus the log of the number of keys that count. A lane's
sums run over fewer than 2^24 equal terms and are whole multiples of them, exact in fp32;
partial results are joined in at most 1024 additions, 2^-14 relatively.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

PAGE = (1 << 23) + 1                     # a page's tokens: just over a power of two
N = (1 << 31) - 1


def _longest(fk, dtype, live=None):
    import torch

    torch.cuda.synchronize()
    width, D = 256, 32
    k, v = (torch.randint(1, 5, (1, 1, 1, D), device="cuda").to(dtype).expand(1, PAGE, 1, D) for _ in range(2))
    q = torch.randint(-2, 3, (2, 2, D), device="cuda").to(dtype)
    table = torch.zeros((2, width), dtype=torch.int32, device="cuda")
    lens = torch.tensor([N, 5], dtype=torch.int32, device="cuda")
    bias = None if live is None else torch.where(live, 0.0, -math.inf).view(1, PAGE, 1)
    out, lse = fk.fk_paged_attn(q, k, v, table, lens, 0.125, key_bias=bias, return_lse=True)
    live = torch.ones(PAGE, dtype=torch.bool, device="cuda") if live is None else live
    count = [int(live.sum()) * (N // PAGE) + int(live[:N % PAGE].sum()), int(live[:5].sum())]
    score = 0.125 * (q.double() * k[0, 0].double()).sum(-1).cpu().numpy()
    want = score + np.log(np.array(count, np.float64))[:, None]
    assert np.abs(lse.double().cpu().numpy() - want).max() <= 2.0 ** -14 + 2.0 ** -22 * np.abs(want).max()
    err = (out.double() - v[0, 0].double()).abs() / v[0, 0].double()
    assert err.max() <= 2.0 ** -14 + {torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}[dtype]


@pytest.mark.parametrize("dtype", ["float16", "float32"])
def test_longest_request(fk, dtype):
    import torch
    _longest(fk, getattr(torch, dtype))


@pytest.mark.parametrize("dtype", ["float16", "float32"])
def test_longest_request_with_bias(fk, dtype):
    """The bias of the steps asked for beyond the end is read inside the page."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(4)
    live = torch.rand(PAGE, device="cuda", generator=g) < 0.5
    live[0] = True
    _longest(fk, getattr(torch, dtype), live)

"""Single-token attention of any layout: sums over long keys."""
import math

import numpy as np
import pytest

from gpu_helpers import host_f64, torch_dtype

pytestmark = pytest.mark.gpu

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("call", ["fk_paged_attn", "fk_paged_attn8"])
def test_long_sums_of_any_layout(fk, call, dtype):
    """2^22 keys of one weight, 0.2968 of the largest, which a wave adds a quarter of one by one: in one
    run the last half of them would be added as multiples of 2^-5 (0.28125 or 0.3125). Runs of at most
    2^12 terms are off by 2^-13, 2^8 runs and their join by 2^-16, the exponential by 2^-20."""
    import torch
    D, page, n = 33, 1 << 10, 1 << 22
    dt = torch_dtype(dtype)
    x = 1.21484375                                   # a score below the largest
    k, v = torch.zeros((2, page, 1, D), device="cuda"), torch.ones((2, page, 1, D), device="cuda")
    k[..., 0] = -1.0
    k[1, 0] = 0.0
    v[..., 1:20], v[..., 20:] = 3.0, 0.625           # (e4m3 numbers all)
    q = torch.zeros((1, 1, D), dtype=dt, device="cuda")
    q[..., 0] = 1.0
    table = torch.zeros((1, n // page), dtype=torch.int32, device="cuda")
    table[0, 0] = 1
    if call == "fk_paged_attn":
        cache = (k.to(dt), v.to(dt))
    else:
        one = torch.ones((2, page, 1), device="cuda")
        cache = (k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), one, one.clone())
    out, lse = getattr(fk, call)(q, *cache, table, _i32([n]), x, max_len=1, return_lse=True)
    want = host_f64(v[0, 0, 0], "f32")
    assert abs(float(lse) - math.log(1.0 + (n - 1) * math.exp(-x))) <= 2.0 ** -12
    assert np.abs(host_f64(out[0, 0], dtype) / want - 1).max() <= 2.0 ** -12 + U[dtype]

"""The largest launches of prompt attention and of single-token attention over 8 bits: what the header's
limit allows is taken, what would hold 2^32 threads is refused before anything is enqueued."""
import ctypes

import pytest

from test_kv8_host import HIP, I2, P, UNSUPPORTED, _cache

I3 = ctypes.c_int64 * 3


@pytest.fixture(scope="module")
def lib():
    import torch

    import exact_means_clustering_flashassign_amd as mod

    if torch.cuda.is_available():
        pytest.skip("the addresses here are made up: only for machines without a GPU")
    return mod.load()


def _prompt(lib, dt, T, B, Hq, Hkv, D, width=1, page=16):
    c = _cache("fk_kv_cache_t", heads=Hkv, dim=D, page=page, k_stride=(page * Hkv * D, Hkv * D, D),
               v_stride=(page * Hkv * D, Hkv * D, D))
    ws = lib.fk_workspace_size_prompt(dt, T, B, Hq, Hkv, D)
    assert ws > 0
    return lib.fk_prompt_attn(P, I2(Hq * D, D), dt, T, B, Hq, ctypes.byref(c), P, width, width, P, P, 0, 0.1, 0.0, P,
                              None, P, ws, None)


@pytest.mark.parametrize("dt", [0, 1, 2])
@pytest.mark.parametrize("D", [64, 128, 192, 256, 33, 320])
def test_prompts(lib, dt, D):
    """A call that is in order ends with the status of a machine without a GPU."""
    # T Hq below 2^26 and T Hq + 8 B Hkv below 2^27
    for T, B, Hq, Hkv in ((70000, 70000, 128, 128), ((1 << 26) - 9, 1, 1, 1), (1, (1 << 24) - 1, 1, 1),
                          (1, 1 << 19, 31, 31), ((1 << 18) - 9, 1, 256, 1), ((1 << 18) - 1, 64, 256, 16),
                          (600, 1 << 20, 8, 8)):
        assert T * Hq < 1 << 26 and T * Hq + 8 * B * Hkv < 1 << 27
        for width in (1, 1 << 20):                   # (long keys: blocks of several parts)
            assert _prompt(lib, dt, T, B, Hq, Hkv, D, width) == HIP, (T, B, Hq, Hkv, width)
    for T, B, Hq, Hkv in ((1, 1 << 25, 1, 1), (1 << 20, 1 << 20, 32, 32), (0x7FFFFFF0, 1, 4, 2),
                          (1 << 30, 1, 1 << 10, 1)):                 # (2^33 tiles)
        assert _prompt(lib, dt, T, B, Hq, Hkv, D) == UNSUPPORTED, (T, B, Hq, Hkv)


@pytest.mark.parametrize("dt", [0, 1, 2])
@pytest.mark.parametrize("D", [64, 33])
def test_single_tokens(lib, dt, D):
    def call8(B, H, width=1):
        c = _cache("fk_kv_cache8_t", heads=H, dim=D, k_stride=(16 * H * D, H * D, D), v_stride=(16 * H * D, H * D, D))
        return lib.fk_paged_attn8(P, I2(H * D, D), dt, B, H, ctypes.byref(c), P, width, width, P, 0, 0.1, 0.0, P, None, P,
                                  lib.fk_workspace_size_attn8(dt, B, H, H, D), None)

    def call(B, H, width=1):
        c = _cache("fk_kv_cache_t", heads=H, dim=D, k_stride=(16 * H * D, H * D, D), v_stride=(16 * H * D, H * D, D))
        return lib.fk_paged_attn(P, I2(H * D, D), dt, B, H, ctypes.byref(c), P, width, width, P, 0, 0.1, 0.0, P, None, P,
                                 lib.fk_workspace_size_attn(dt, B, H, H, D), None)

    for f in (call, call8):
        for width in (1, 1 << 12):
            assert f((1 << 24) - 1, 1, width) == HIP and f(1 << 16, 255, width) == HIP
            assert f(1 << 28, 1, width) == UNSUPPORTED and f(1 << 20, 1 << 8, width) == UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_requests_of_many_heads(fk, dtype):
    """70000 requests of one token with 128 heads: nine million blocks."""
    import torch
    from gpu_helpers import torch_dtype

    B, H, D, page = 70000, 128, 8, 4
    dt = torch_dtype(dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((5, page, H, D), device="cuda", generator=g).to(dt) for _ in range(2))
    q = torch.randn((B, H, D), device="cuda", generator=g).to(dt)
    table = torch.randint(0, 5, (B, 2), device="cuda", generator=g).int()
    lens = torch.randint(1, 2 * page + 1, (B,), device="cuda", generator=g).int()
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    out, lse = fk.fk_prompt_attn(q, k, v, table, lens, cu, return_lse=True)
    for b in (0, 1, 35000, B - 2, B - 1):
        n = int(lens[b])
        at = table[b].long()
        kb, vb = (c[at].flatten(0, 1)[:n].double() for c in (k, v))
        s = (q[b].double()[None] * kb).sum(-1) / D ** 0.5
        want = (s.softmax(0)[..., None] * vb).sum(0)
        # one rounding of a weight and one of the result, of values below 5
        assert (out[b].double() - want).abs().max() <= {"bf16": 10 * 2.0 ** -8, "f32": 2.0 ** -18}[dtype]
        assert (lse[b].double() - s.logsumexp(0)).abs().max() <= 2.0 ** -18
    assert not out.isnan().any() and not lse.isnan().any()

"""Prompt attention and the 8-bit cache at the ends of their ranges: 2^31 - 1 keys, offsets past 32
bits, two captured graphs with one workspace, rounding of results.

Lengths: one page that every entry of the table repeats, all its keys one row and all its values
one row, so the result is that value and lse is the score plus the log of the number of keys.
Sums of up to 2^25 equal terms a part are whole multiples of a power of two times the value,
below 2^24 of what each step adds: exact in fp32. Partial results are joined in at most
1024 additions, 2^-14 relatively.
"""
import math

import numpy as np
import pytest

import oracle
from gpu_helpers import host_f64, torch_dtype

pytestmark = pytest.mark.gpu

PAGE = (1 << 23) + 1                     # a page's tokens: just over a power of two
N = (1 << 31) - 1
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _near(lse, out, score, counts, v, dtype):
    want = score + np.log(np.array(counts, np.float64))[:, None]
    assert np.abs(lse.double().cpu().numpy() - want).max() <= 2.0 ** -14 + 2.0 ** -22 * np.abs(want).max()
    err = (host_f64(out, dtype) - v) / v
    assert np.abs(err).max() <= 2.0 ** -14 + U[dtype]


@pytest.mark.parametrize("bias", [False, True], ids=["", "bias"])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_longest_prompt(fk, dtype, bias):
    """The last tokens of a request of 2^31 - 1, next to a short one."""
    import torch
    D, T = 32, 5
    k, v = (torch.randint(1, 5, (1, 1, 1, D), device="cuda").to(torch_dtype(dtype)).expand(1, PAGE, 1, D) for _ in range(2))
    q = torch.randint(-2, 3, (T, 2, D), device="cuda").to(torch_dtype(dtype))
    kb = torch.zeros((1, PAGE, 1), device="cuda") if bias else None
    out, lse = fk.fk_prompt_attn(q, k, v, torch.zeros((2, 256), dtype=torch.int32, device="cuda"), _i32([N, 5]),
                                 _i32([0, 3, 5]), 0.125, key_bias=kb, return_lse=True)
    score = 0.125 * (q.double() * k[0, 0].double()).sum(-1).cpu().numpy()
    _near(lse, out, score, [N - 2, N - 1, N, 4, 5], host_f64(v[0, 0].contiguous(), dtype), dtype)


@pytest.mark.parametrize("bias", [False, True], ids=["", "bias"])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_longest_8bit_request(fk, dtype, bias):
    import torch
    D = 32
    k, v = (torch.randint(1, 5, (1, 1, 1, D), device="cuda").float().to(torch.float8_e4m3fn).expand(1, PAGE, 1, D)
            for _ in range(2))
    ks, vs = (torch.full((1, PAGE, 1), s, device="cuda") for s in (0.5, 2.0))
    kb = torch.zeros((1, PAGE, 1), device="cuda") if bias else None
    q = torch.randint(-2, 3, (2, 2, D), device="cuda").to(torch_dtype(dtype))
    out, lse = fk.fk_paged_attn8(q, k, v, ks, vs, torch.zeros((2, 256), dtype=torch.int32, device="cuda"),
                                 _i32([N, 5]), 0.25, key_bias=kb, return_lse=True)
    score = 0.125 * (q.double() * k[0, 0].double()).sum(-1).cpu().numpy()
    _near(lse, out, score, [N, 5], 2.0 * v[0, 0].double().cpu().numpy(), dtype)


@pytest.mark.parametrize("cut", [False, True], ids=["whole", "parts"])
def test_long_fp32_sums_are_held_apart(fk, cut):
    """2^22 and 2^27 keys whose scores grow, over pages that the table repeats. Roundings of 2^19 sums
    of random sign are off by 2^9.5 halves of u = 2^-24 in the mean, 2^-15.5 of the largest value; 2^-11
    is more than 16 times that."""
    import torch
    Hq, Hkv, D, T, page, pages = (2, 1, 8, 3, 1 << 13, 4) if cut else (512, 8, 8, 128, 512, 4)
    width = 1 << (14 if cut else 13)
    n = width * page - 77
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(s, device="cuda", generator=g) for s in ((T, Hq, D), (pages, page, Hkv, D), (pages, page, Hkv, D)))
    k[..., 0] = torch.arange(pages, device="cuda").view(pages, 1, 1) * 3.0      # a query with a large
    q[..., 0] = torch.randn((T, Hq), device="cuda", generator=g)                # first element prefers late pages
    table = torch.div(torch.arange(width, device="cuda") * pages, width, rounding_mode="floor").int()
    out, lse = fk.fk_prompt_attn(q, k, v, table.view(1, width), _i32([n]), _i32([0, T]), 1.0, return_lse=True)
    k64, v64 = (host_f64(t, "f32").reshape(pages * page, Hkv, D) for t in (k, v))
    reps = np.bincount(table.cpu().numpy(), minlength=pages).astype(np.float64)
    for t, h in ((0, 0), (1, Hq - 1), (T - 1, Hq // 2), (T - 1, 0), (T // 2, Hq // 3)):
        hk = h // (Hq // Hkv)
        counts = np.repeat(reps, page)
        counts[pages * page - (width * page - n) - (T - 1 - t):] -= 1.0        # what the row does not see
        s = k64[:, hk] @ host_f64(q[t, h], "f32")
        w = counts * np.exp(s - s.max())
        want, big = w @ v64[:, hk] / w.sum(), np.abs(v64).max()
        assert np.abs(host_f64(out[t, h], "f32") - want).max() <= 2.0 ** -11 * big
        assert abs(float(lse[t, h]) - (s.max() + np.log(w.sum()))) <= 2.0 ** -11


PAST = (1 << 17) + 64                    # pages of 16 tokens, 16 rows of 128: 2^32 elements and more


def _pages(rng, B, width):
    """A table over the first pages and the same one over pages at the end of a long cache."""
    low = rng.permutation(B * width).reshape(B, width)
    return _i32(low.tolist()), _i32((PAST - 1 - low).tolist()), PAST - 1 - np.arange(B * width)


@pytest.mark.parametrize("D", [128, 127])
def test_prompt_past_32_bits(fk, D):
    """The same bits as over a short cache."""
    import torch
    B, width = 2, 12
    low, high, at = _pages(np.random.default_rng(1), B, width)
    far = torch.empty((PAST, 16, 16, 128), dtype=torch.float16, device="cuda")
    near = torch.randn((B * width, 16, 16, 128), device="cuda").half()
    far[_i32(at.tolist()).long()] = near
    q = torch.randn((150, 32, D), device="cuda").half()
    got = [fk.fk_prompt_attn(q, c[:, :, :8, :D], c[:, :, 8:, :D], t, _i32([190, 100]), _i32([0, 100, 150]),
                             return_lse=True, max_len=190) for c, t in ((near, low), (far, high))]
    assert all(torch.equal(a, b) for a, b in zip(*got)) and not got[0][0].isnan().any()


@pytest.mark.parametrize("D", [128, 127])
def test_8bit_past_32_bits(fk, D):
    import torch
    B, width = 2, 12
    low, high, at = _pages(np.random.default_rng(2), B, width)
    T = B * width * 16
    k, v = (torch.randn((T, 8, D), device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((B, 32, D), device="cuda").bfloat16()
    order = torch.arange(T, device="cuda")
    slots = [order, (PAST - 1 - order // 16) * 16 + order % 16]
    got = []
    for pages, slot, table in ((B * width, slots[0], low), (PAST, slots[1], high)):
        codes = torch.empty((pages, 16, 16, 128), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        numbers = torch.empty((2, pages, 16, 8), device="cuda")
        cache = (codes[:, :, :8, :D], codes[:, :, 8:, :D], numbers[0], numbers[1])
        fk.fk_kv_store8(k, v, slot.int(), *cache)
        got.append(fk.fk_kv_load8(slot.int(), *cache, torch.bfloat16)
                   + fk.fk_paged_attn8(q, *cache, table, _i32([190, 100]), return_lse=True))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and not got[0][2].isnan().any()
    assert np.array_equal(host_f64(got[0][0], "bf16"), oracle.quantise(host_f64(k, "bf16"))[0])


def test_two_graphs_one_workspace(fk):
    """A prompt's attention and a step's over the 8-bit cache, captured by themselves with one
    workspace and replayed in turn, with eager calls between that use it as well."""
    import torch
    Hq, Hkv, D, page, B, width = 8, 2, 128, 16, 2, 256
    pages = B * width
    table = torch.randperm(pages, device="cuda").int().view(B, width)
    k, v = (torch.randn((pages, page, Hkv, D), device="cuda").half() for _ in range(2))
    slots = torch.arange(pages * page, device="cuda").int()
    k8, v8 = (torch.zeros((pages, page, Hkv, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.empty((pages, page, Hkv), device="cuda") for _ in range(2))
    fk.fk_kv_store8(k.view(-1, Hkv, D), v.view(-1, Hkv, D), slots, k8, v8, ks, vs)
    lens, cu = _i32([4000, 3500]), _i32([0, 40, 70])
    q, q1 = torch.randn((70, Hq, D), device="cuda").half(), torch.randn((B, Hq, D), device="cuda").half()
    need = max(fk.fk_workspace_size_prompt(q.dtype, 70, B, Hq, Hkv, D), fk.fk_workspace_size_attn8(q.dtype, B, Hq, Hkv, D))
    ws = torch.zeros(need + 256, dtype=torch.uint8, device="cuda")
    ws = ws[-ws.data_ptr() % 256:][:need]
    out, out1 = torch.empty_like(q), torch.empty_like(q1)
    prompt = lambda o: fk.fk_prompt_attn(q, k, v, table, lens, cu, out=o, ws=ws, max_len=4096)
    step = lambda o: fk.fk_paged_attn8(q1, k8, v8, ks, vs, table, lens, out=o, ws=ws)
    prompt(out), step(out1)
    torch.cuda.synchronize()
    graphs = []
    for call, o in ((prompt, out), (step, out1)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(o)
        graphs.append(graph)
    for i in range(5):
        q.normal_(), q1.normal_()
        lens.copy_(_i32([4000 - 300 * i, 3500 - 1000 * (i % 3)]))
        want = prompt(torch.empty_like(q)), step(torch.empty_like(q1))
        out.fill_(math.nan), out1.fill_(math.nan), ws.fill_(255)
        for g in graphs if i % 2 else graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(out1, want[1]), i


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_mean_rounding(fk, dtype):
    """Root mean square errors next to the type's own rounding of exact results: an error of at most U
    |x| for the result, uniform, is U |x| / sqrt(3) in the mean; probabilities rounded to the
    type once, one by one, add at most U sqrt(sum p^2 v^2) / sqrt(3), values of unit variance:
    U sqrt(sum p^2), no more than U times the spread of the results themselves. So twice U |x|,
    with |x| the root mean square, holds for prompts, and U |x| for the 8-bit cache, whose
    probabilities are not rounded to the type."""
    import torch
    Hq, Hkv, D, n = 8, 2, 128, 700
    q, k, v = (torch.randn(s, device="cuda").to(torch_dtype(dtype)) for s in ((n, Hq, D), (44, 16, Hkv, D), (44, 16, Hkv, D)))
    table = torch.arange(44, device="cuda").int().view(1, 44)
    out = fk.fk_prompt_attn(q, k, v, table, _i32([n]), _i32([0, n]))
    want, *_ = oracle.prompt_attn(host_f64(q, dtype), host_f64(k, dtype), host_f64(v, dtype), table.cpu().numpy(),
                                 [n], [0, n], 1.0 / math.sqrt(D))
    rms = lambda x: float(np.sqrt(np.mean(np.square(x))))
    assert rms(host_f64(out, dtype) - want) <= 2.0 * U[dtype] * rms(want)

    k8, v8 = (torch.zeros((44, 16, Hkv, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.empty((44, 16, Hkv), device="cuda") for _ in range(2))
    slots = torch.arange(44 * 16, device="cuda").int()
    fk.fk_kv_store8(k.view(-1, Hkv, D), v.view(-1, Hkv, D), slots, k8, v8, ks, vs)
    kd, vd = (oracle.quantise(host_f64(t.view(-1, Hkv, D), dtype))[0].reshape(44, 16, Hkv, D) for t in (k, v))
    out = fk.fk_paged_attn8(q[:1], k8, v8, ks, vs, table, _i32([n]))
    want, *_ = oracle.prompt_attn(host_f64(q[:1], dtype), kd, vd, table.cpu().numpy(), [n], [0, 1], 1.0 / math.sqrt(D))
    assert rms(host_f64(out, dtype) - want) <= U[dtype] * rms(want)


@pytest.mark.parametrize("dims", [(2, 1, 33), (3, 3, 130), (2, 2, 300)], ids=["d33", "d130", "d300"])
def test_long_sums_of_any_layout(fk, dims):
    """2^20 keys whose scores grow, in rows that the vector units take; bound as above."""
    import torch
    Hq, Hkv, D = dims
    T, page, pages, width = 3, 1 << 10, 4, 1 << 10
    n = width * page - 77
    g = torch.Generator(device="cuda").manual_seed(D)
    q, k, v = (torch.randn(s, device="cuda", generator=g) for s in ((T, Hq, D), (pages, page, Hkv, D + 1), (pages, page, Hkv, D + 1)))
    k[..., 0] = torch.arange(pages, device="cuda").view(pages, 1, 1) * 3.0
    k, v, q = k[..., :D], v[..., 1:], q * 0.25
    table = torch.div(torch.arange(width, device="cuda") * pages, width, rounding_mode="floor").int()
    out, lse = fk.fk_prompt_attn(q, k, v, table.view(1, width), _i32([n]), _i32([0, T]), 1.0, return_lse=True)
    k64, v64 = (host_f64(t.contiguous(), "f32").reshape(pages * page, Hkv, D) for t in (k, v))
    for t in range(T):
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            counts = np.repeat(np.bincount(table.cpu().numpy(), minlength=pages).astype(np.float64), page)
            counts[pages * page - (width * page - n) - (T - 1 - t):] -= 1.0
            s = k64[:, hk] @ host_f64(q[t, h], "f32")
            w = counts * np.exp(s - s.max())
            want, big = w @ v64[:, hk] / w.sum(), np.abs(v64).max()
            assert np.abs(host_f64(out[t, h], "f32") - want).max() <= 2.0 ** -11 * big
            assert abs(float(lse[t, h]) - (s.max() + np.log(w.sum()))) <= 2.0 ** -11

"""ClusteredKVCache: tables, norm + rotation + stores, attention and clustering
together, as a server of one layer runs them, against the fp64 oracle."""
import math

import numpy as np
import pytest

import oracle
import synthdata
from gpu_helpers import host_f64, to_dev, torch_dtype
from test_gpu_kv_cache import _check_attn, _dev, _rand


def _rope(rng, positions, rot):
    ang = rng.uniform(0, 6.28, (positions, rot // 2))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _dense(cache, b, dtype):
    """Keys, values and bias a request holds, read back in order."""
    n = cache.lens[b]
    rows = cache.table[b, :-(-n // cache.page)].long()
    pick = lambda c: c[rows].flatten(0, 1)[:n]           # noqa: E731
    return (host_f64(pick(cache.k), dtype), host_f64(pick(cache.v), dtype),
            pick(cache.key_bias).cpu().numpy().astype(np.float64))


def _check(cache, q, got, dtype, dim, dense=None):
    """attend()'s result against the oracle over what is held (one page per token)."""
    for b in range(q.shape[0]):
        k, v, bias = dense[b] if dense else _dense(cache, b, dtype)
        want = oracle.paged_attn(host_f64(q[b:b + 1], dtype), k[:, None], v[:, None],
                                 np.arange(len(k))[None], [len(k)], dim ** -0.5, 0.0, bias[:, None])
        _check_attn((got[0][b:b + 1], got[1][b:b + 1]), want, dtype, dim, 0.0, f"request {b}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_prompt_and_steps(fk, dtype):
    rng = np.random.default_rng(21)
    B, Hq, Hkv, D, page = 3, 6, 2, 64, 8
    cache = fk.ClusteredKVCache(B, 60, page, Hkv, D, 100, torch_dtype(dtype))
    rope, w = _rope(rng, 200, D), [_rand(rng, D, dtype) for _ in range(2)]
    wd, rd = [to_dev(a, dtype) for a in w], _dev(rope)
    seen = [[] for _ in range(B)]
    for new in ([37, 0, 9], [1, 1, 1], [1, 1, 1], [0, 20, 0], [1, 1, 1]):
        T = sum(new)
        x = _rand(rng, (T, Hq + 2 * Hkv, D), dtype)
        x64, xd = synthdata.to_f64(x, dtype), to_dev(x, dtype)
        q = cache.append(xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], new, *wd, 1e-6, rd)
        at, pos = 0, []
        for b, n in enumerate(new):
            pos += range(len(seen[b]), len(seen[b]) + n)
            seen[b] += list(x64[at:at + n])
            at += n
        want, m = oracle.norm_rope(x64[:, :Hq], synthdata.to_f64(w[0], dtype), 1e-6,
                                   rope.astype(np.float64), np.array(pos), False)
        unit = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}[dtype]
        e = (D / 2 + 10) * 2.0 ** -24 * m                # the norm + rotation bound
        assert (np.abs(host_f64(q, dtype) - want) <= e + unit * (np.abs(want) + e) + 2.0 ** -25).all()
        if max(new) == 1:
            _check(cache, q, cache.attend(q, return_lse=True), dtype, D)
    assert cache.lens == [len(s) for s in seen] == cache.seen == cache.lens_dev.tolist()
    for b in range(B):                                   # values are as given, in order
        assert np.array_equal(_dense(cache, b, dtype)[1], np.array(seen[b])[:, Hq + Hkv:])


@pytest.mark.gpu
def test_compress_keeps_equal_keys_exactly(fk):
    """Tokens that are copies of a few keys lose nothing: the compressed cache's
    attention meets the bound of the exact one over all tokens."""
    import torch
    rng = np.random.default_rng(22)
    H, D, page, n, K, keep = 2, 64, 16, 150, 12, 10
    cache = fk.ClusteredKVCache(2, 40, page, H, D, 200, torch.float16)
    kinds = [_rand(rng, (K, H, D), "f16") for _ in range(2)]
    which = np.concatenate([np.arange(K), rng.integers(0, K, n - keep - K)])
    x = _rand(rng, (2 * n, 3 * H, D), "f16")
    for r in range(2):
        x[r * n:r * n + n - keep, H:2 * H] = kinds[0][which]
        x[r * n:r * n + n - keep, 2 * H:] = kinds[1][which]
    xd = to_dev(x, "f16")
    cache.append(xd[:, :H], xd[:, H:2 * H], xd[:, 2 * H:], [n, n])
    full = [_dense(cache, b, "f16") for b in range(2)]
    before = cache.free.numel()
    init = to_dev(np.ascontiguousarray(kinds[0].transpose(1, 0, 2)), "f16")
    assert cache.compress(1, K, keep, niter=3, init=init) == K + keep
    assert cache.lens == [n, K + keep] and cache.seen == [n, n] and cache.centres == [0, K]
    assert cache.free.numel() == before + (-(-n // page) - -(-(K + keep) // page))
    q = to_dev(_rand(rng, (2, 4 * H, D), "f16"), "f16")
    _check(cache, q, cache.attend(q, return_lse=True), "f16", D, full)
    # the next token goes behind what is kept, at the position after all that was seen
    rope = _dev(_rope(rng, 300, D))
    x1 = to_dev(_rand(rng, (2, 3 * H, D), "f16"), "f16")
    q1 = cache.append(x1[:, :H], x1[:, H:2 * H], x1[:, 2 * H:], [1, 1], rope=rope)
    same, _ = fk.fk_qk_norm_rope(x1[:, :H], x1[:, H:2 * H], rope=rope,
                                 positions=_dev(np.array([n, n], np.int32)))
    assert torch.equal(q1, same)
    _check(cache, q1, cache.attend(q1, return_lse=True), "f16", D)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_compress_attends_over_centres(fk, dtype):
    """Random keys: centres, counts and mean values against fp64 sums over the
    clusters, then attention against the oracle over what is held; a second
    compression leaves the first one's centres; freed pages are used again."""
    import torch
    rng = np.random.default_rng(23)
    H, D, page, n, K, keep = 3, 32, 4, 90, 20, 7
    cache = fk.ClusteredKVCache(1, 25, page, H, D, 100, torch_dtype(dtype))
    x = to_dev(_rand(rng, (n, 3 * H, D), dtype), dtype)
    cache.append(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], [n])
    k, v, _ = _dense(cache, 0, dtype)
    cache.compress(0, K, keep, niter=4)
    ck, cv, bias = _dense(cache, 0, dtype)
    assert np.array_equal(ck[K:], k[n - keep:]) and np.array_equal(cv[K:], v[n - keep:])
    assert (bias[K:] == 0).all()
    unit = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}[dtype]
    for h in range(H):
        d = ((k[:n - keep, None, h] - ck[None, :K, h]) ** 2).sum(-1)
        near = np.sort(d, 1)[:, :2]
        assert ((near[:, 1] - near[:, 0]) > 1e-4 * near[:, 1]).mean() > 0.9
        ids = d.argmin(1)
        cnt = np.bincount(ids, minlength=K)
        got = np.rint(np.exp(bias[:K, h])).astype(int)
        assert got.sum() == n - keep
        if np.array_equal(got, cnt):                     # no point inside the near-tie band moved
            for c in range(K):
                m = v[:n - keep, h][ids == c].mean(0) if cnt[c] else np.zeros(D)
                assert (np.abs(cv[c, h] - m) <= unit * np.abs(m) + 2e-3 * max(np.abs(m).max(), 1e-6)).all()
    q = to_dev(_rand(rng, (1, 2 * H, D), dtype), dtype)
    _check(cache, q, cache.attend(q, return_lse=True), dtype, D)
    x = to_dev(_rand(rng, (60, 3 * H, D), dtype), dtype)
    cache.append(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], [60])
    assert len(set(cache.table[0, :-(-cache.lens[0] // page)].tolist()) | set(cache.free.tolist())) == 25
    cache.compress(0, 5, 3)
    assert cache.lens == [K + 5 + 3] and cache.centres == [K + 5] and cache.seen == [n + 60]
    again = _dense(cache, 0, dtype)
    assert np.array_equal(again[0][:K], ck[:K]) and np.array_equal(again[2][:K], bias[:K])
    _check(cache, q, cache.attend(q, return_lse=True), dtype, D)


def test_refusals_on_host():
    import exact_means_clustering_flashassign_amd as fk
    import torch

    with pytest.raises(ValueError):
        fk.ClusteredKVCache(1, 0, 16, 2, 64, 100, torch.float16, device="cpu")
    c = fk.ClusteredKVCache(2, 3, 16, 2, 64, 100, torch.float16, device="cpu")
    x = torch.zeros(60, 2, 64, dtype=torch.float16)
    for new in ([60], [61, -1], [30, 20], [0, 0]):
        with pytest.raises(ValueError):
            c.append(x, x, x, new)
    with pytest.raises(RuntimeError):                    # four pages, three free
        c.append(x, x, x, [60, 0])
    with pytest.raises(ValueError):
        fk.ClusteredKVCache(1, 9, 16, 2, 64, 50, torch.float16, device="cpu").append(x, x, x, [60])
    with pytest.raises(ValueError):
        c.compress(0, 4)
    assert c.lens == [0, 0] and c.free.numel() == 3

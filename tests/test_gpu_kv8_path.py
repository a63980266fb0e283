"""ClusteredKVCache with prompts and in 8 bits: append, prompt attention, single tokens and
clustering run together, against the fp64 oracle over what is held."""
import numpy as np
import pytest

import oracle
import test_gpu_cache8 as c8
from gpu_helpers import host_f64, to_dev, torch_dtype
from test_gpu_kv_cache import _rand
from test_gpu_prompt import _check


def _held(cache, b):
    """Keys, values and bias a request holds, in order, as float64."""
    import torch

    n = cache.lens[b]
    rows = cache.table[b, :-(-n // cache.page)].long()

    def pick(c):
        return c[rows].flatten(0, 1)[:n]

    if cache.quantised:
        numbers = torch.from_numpy(c8._numbers()).cuda()
        k, v = (numbers[pick(c.view(torch.uint8)).long()] * pick(s).double()[..., None]
                for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    else:
        k, v = pick(cache.k).double(), pick(cache.v).double()
    return k.cpu().numpy(), v.cpu().numpy(), pick(cache.key_bias).double().cpu().numpy()


def _prompts(cache, q, new, dtype):
    """The oracle's result of a step's tokens, one page per token."""
    Hq, D = q.shape[1:]
    parts, t = [], 0
    for b, n in enumerate(new):
        k, v, bias = _held(cache, b)
        if n:
            parts.append(oracle.prompt_attn(host_f64(q[t:t + n], dtype), k[:, None], v[:, None],
                                            np.arange(len(k))[None], [len(k)], [0, n], D ** -0.5, 0.0,
                                            bias[:, None]))
        t += n
    return tuple(np.concatenate([p[i] for p in parts]) for i in range(3))


@pytest.mark.gpu
@pytest.mark.parametrize("quantised", [False, True], ids=["plain", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_prompts_steps_and_clusters(fk, dtype, quantised):
    rng = np.random.default_rng(31)
    B, Hq, Hkv, D, page = 3, 6, 2, 64, 8
    cache = fk.ClusteredKVCache(B, 90, page, Hkv, D, 200, torch_dtype(dtype), quantised=quantised)
    w = [to_dev(_rand(rng, D, dtype), dtype) for _ in range(2)]

    def step(new):
        x = to_dev(_rand(rng, (sum(new), Hq + 2 * Hkv, D), dtype), dtype)
        return cache.append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], new, *w)

    for new in ([70, 0, 33], [1, 1, 1], [0, 90, 20], [1, 1, 1]):
        q = step(new)
        got = cache.attend_prompts(q, return_lse=True)
        _check(got, _prompts(cache, q, new, dtype), dtype, D, 0.0, f"prompts {new}")
        if max(new) == 1:                              # the same tokens by the other kernel
            one = cache.attend(q, return_lse=True)
            want = _prompts(cache, q, new, dtype)
            c8._check_attn(one, want, dtype, D, 0.0, f"tokens {new}")
    # older tokens become centres; new prompts attend to centres and tokens
    before = [_held(cache, b) for b in range(B)]
    assert cache.compress(1, 9, 12) == 21 and cache.lens[1] == 21
    after = _held(cache, 1)
    for a, b in zip(after, before[1]):                 # what is kept is kept exactly
        assert np.array_equal(a[9:], b[-12:])
    assert (np.exp(after[2][:9]).sum(0).round() == len(before[1][0]) - 12).all()
    with pytest.raises(ValueError, match="no step"):
        cache.attend_prompts(q)
    q = step([0, 17, 3])
    _check(cache.attend_prompts(q, return_lse=True), _prompts(cache, q, [0, 17, 3], dtype), dtype, D, 0.0)
    cache.release(0)
    with pytest.raises(ValueError, match="no step"):
        cache.attend_prompts(q)
    q = step([40, 0, 0])
    _check(cache.attend_prompts(q, return_lse=True), _prompts(cache, q, [40, 0, 0], dtype), dtype, D, 0.0)
    with pytest.raises(ValueError, match="tokens"):
        cache.attend_prompts(q[:39])


@pytest.mark.gpu
def test_stored_rows_are_the_nearest_codes(fk):
    """What a quantised cache holds is the oracle's rounding of the rows given to it."""
    rng = np.random.default_rng(32)
    cache = fk.ClusteredKVCache(1, 9, 16, 3, 64, 100, torch_dtype("bf16"), quantised=True)
    x = to_dev(_rand(rng, (50, 9, 64), "bf16"), "bf16")
    cache.append(x[:, :3], x[:, 3:6], x[:, 6:], [50])
    k, v, _ = _held(cache, 0)
    assert np.array_equal(k, oracle.quantise(host_f64(x[:, 3:6], "bf16"))[0])
    assert np.array_equal(v, oracle.quantise(host_f64(x[:, 6:], "bf16"))[0])


def test_quantised_refusals_on_host():
    import exact_means_clustering_flashassign_amd as fk
    import torch

    with pytest.raises(ValueError, match="element type"):
        fk.ClusteredKVCache(1, 9, 16, 2, 64, 100, torch.float64, device="cpu", quantised=True)
    c = fk.ClusteredKVCache(2, 3, 16, 2, 64, 100, torch.float16, device="cpu", quantised=True)
    x = torch.zeros(10, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="no step"):
        c.attend_prompts(x)
    with pytest.raises(RuntimeError):
        c.append(torch.zeros(60, 2, 64), torch.zeros(60, 2, 64), torch.zeros(60, 2, 64), [60, 0])
    assert c.lens == [0, 0] and c.free.numel() == 3

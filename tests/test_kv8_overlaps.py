"""The tensors of an 8-bit cache that is stored to: none may hold an element of another, however they
lie; those that lie between one another's elements are taken."""
import random

import pytest


def test_share_is_exact():
    """Overlap of two strided tensors, against marks on every byte."""
    import torch
    from exact_means_clustering_flashassign_amd._binding import _share

    rng = random.Random(2)

    def one(base, dtype, size):
        shape = [rng.randint(1, 4) for _ in range(4)]
        order = list(range(3))
        rng.shuffle(order)
        strides, at = [0, 0, 0, 1], shape[3] + rng.choice((0, 0, 3, 9))
        for i in order:
            strides[i], at = at, at * shape[i] + rng.choice((0, 0, 5))
        if rng.random() < 0.1:
            strides[rng.randrange(3)] = rng.randint(0, 9)            # any strides at all
        off = rng.randint(0, 600)
        return base.view(dtype).as_strided(shape, strides, off // size), size

    seen = [0, 0]
    base = torch.zeros(1 << 15, dtype=torch.uint8)
    for _ in range(3000):
        (a, sa), (b, sb) = (one(base, *rng.choice(((torch.uint8, 1), (torch.float32, 4)))) for _ in range(2))
        if rng.random() < 0.4:                           # halves of one tensor, side by side
            d = rng.randrange(4)
            b, sb = a.narrow(d, a.shape[d] // 2, a.shape[d] - a.shape[d] // 2), sa
            a = a.narrow(d, 0, a.shape[d] // 2)
        if not a.numel() or not b.numel():
            continue
        marks = []
        for t, s in ((a, sa), (b, sb)):
            m = torch.zeros(1 << 15, dtype=torch.bool)
            at = torch.tensor([t.data_ptr() - base.data_ptr()])
            for n, st in zip(t.shape, t.stride()):
                at = (at[:, None] + torch.arange(n) * st * s).flatten()
            for i in range(s):
                m[at + i] = True
            marks.append(m)
        want = bool((marks[0] & marks[1]).any())
        assert _share(a, b) == want, (a.shape, a.stride(), a.data_ptr(), b.shape, b.stride(), b.data_ptr())
        seen[want] += 1
    assert min(seen) > 200, seen


def test_share_of_large_tensors_ends():
    """Caches of realistic sizes, in layouts that users have, without a walk over their rows."""
    import time

    import torch
    from exact_means_clustering_flashassign_amd._binding import _share

    big = torch.empty(1, dtype=torch.uint8, device="meta").expand(1 << 34)
    both = big.as_strided((100000, 2, 16, 8, 128), (32768, 16384, 1024, 128, 1))
    t = time.perf_counter()
    for a, b, want in [(both[:, 0], both[:, 1], False), (both[:, 0], both[:, 0, :, 4:], True)]:
        for x, y in ((a, b), (b, a), (a.transpose(1, 2), b)):
            assert _share(x, y, 0, y.storage_offset() - x.storage_offset()) == want
    assert time.perf_counter() - t < 1.0


@pytest.mark.gpu
def test_store8(fk):
    import torch

    def z(*s, dtype=torch.float16):
        return torch.zeros(*s, dtype=dtype, device="cuda")

    u8, f32, e4m3 = torch.uint8, torch.float32, torch.float8_e4m3fn
    pages, page, H, D = 3, 16, 2, 64
    x = torch.randn((5, H, D), dtype=torch.float16, device="cuda")
    slots = torch.arange(5, dtype=torch.int32, device="cuda") * 7
    n, s = pages * page * H * D, pages * page * H
    codes, numbers = z(3 * n, dtype=u8), z(4 * s, dtype=f32)
    shape = (pages, page, H, D)

    def cache(at=(0, n), ns=(0, s, 2 * s)):
        return [codes[a:a + n].view(e4m3).view(shape) for a in at] + [numbers[a:a + s].view(shape[:3]) for a in ns]

    fk.fk_kv_store8(x, x, slots, *cache())
    want = [t.clone() for t in fk.fk_kv_load8(slots, *cache()[:4], torch.float16)]
    for bad in (cache(at=(0, n - 64)), cache(at=(8, 0)), cache(ns=(0, s - 1, 2 * s)), cache(ns=(0, s, 1)),
                cache(ns=(5, s, 0)), cache(ns=(2 * s, 0, s - 3)), cache(at=(0, 0)), cache(ns=(0, 0, s)), cache(ns=(0, s, s))):
        before = codes.clone(), numbers.clone()
        with pytest.raises(ValueError, match="overlaps"):
            fk.fk_kv_store8(x, x, slots, *bad)
        assert torch.equal(before[0], codes) and torch.equal(before[1], numbers)
    mixed = cache()                                      # scales inside the codes
    mixed[2] = codes[n:2 * n].view(f32)[:s].view(shape[:3])
    with pytest.raises(ValueError, match="overlaps"):
        fk.fk_kv_store8(x, x, slots, *mixed)
    # side by side in one allocation: keys and values of a page, of a token, of a head
    for split in (1, 2, 3):
        lay = list(shape)
        lay.insert(split, 2)
        both = z(*lay, dtype=u8).view(e4m3)
        nums = torch.ones((*lay[:-1], 2), device="cuda") if split < 4 else None
        kc, vc = both.unbind(split)
        ks, kb = nums.select(split, 0).unbind(-1)
        vs = nums.select(split, 1)[..., 0]
        fk.fk_kv_store8(x, x, slots, kc, vc, ks, vs, kb)
        got = fk.fk_kv_load8(slots, kc, vc, ks, vs, torch.float16)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        used = (slots // page).long(), (slots % page).long()
        assert (kb[used] == 0).all() and kb.sum() == kb.numel() - 5 * H

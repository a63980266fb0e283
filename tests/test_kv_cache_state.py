"""ClusteredKVCache's own books: what a refused step leaves behind. The CPU tests put the
oracle's tables and plain stores in place of the kernels."""
import numpy as np
import pytest

import oracle
from exact_means_clustering_flashassign_amd import _binding


def _tables(len_old, len_new, free_pages, page, width, tokens, table=None, out=None):
    import torch

    r = oracle.page_tables(len_old.numpy(), len_new.numpy(), None if table is None else table.numpy(),
                           free_pages.numpy(), page, width, tokens)
    return tuple(torch.from_numpy(a.astype(np.int32)) for a in r)


def _store(q, k, v, q_weight, k_weight, eps, rope, positions, interleaved, slots, k_cache, v_cache, key_bias):
    for t, s in enumerate(slots.tolist()):
        at = s // k_cache.shape[1], s % k_cache.shape[1]
        k_cache[at], v_cache[at], key_bias[at] = k[t], v[t], 0.0
    _store.positions = positions.tolist()
    return q, None


@pytest.fixture()
def cpu_cache(monkeypatch):
    import exact_means_clustering_flashassign_amd as fk

    monkeypatch.setattr(_binding, "fk_page_tables", _tables)
    monkeypatch.setattr(_binding, "fk_qk_norm_rope", _store)

    def make(*sizes):
        import torch
        return fk.ClusteredKVCache(*sizes, torch.float32, device="cpu")

    return make


def _books(c):
    return [t.clone() for t in (c.table, c.lens_dev, c.free, c.shift)], list(c.lens), list(c.seen), list(c.centres)


def _same(a, b):
    return all(x.equal(y) for x, y in zip(a[0], b[0])) and a[1:] == b[1:]


def _consistent(c, pages):
    """Device and host lengths agree, and every page is in one request's row or free."""
    assert c.lens_dev.tolist() == c.lens
    held = [c.table[b, :-(-n // c.page)].tolist() for b, n in enumerate(c.lens)]
    assert sorted(sum(held, []) + c.free.tolist()) == list(range(pages))


def test_refused_append_changes_nothing(cpu_cache, monkeypatch):
    import torch

    c = cpu_cache(2, 12, 4, 2, 8, 20)
    x = torch.arange(10 * 2 * 8, dtype=torch.float32).view(10, 2, 8)
    c.append(x[:3], x[:3], x[:3], [2, 1])
    before = _books(c)

    def refuse(*_):
        raise ValueError("refused")

    with monkeypatch.context() as m:
        m.setattr(_binding, "fk_qk_norm_rope", refuse)
        with pytest.raises(ValueError, match="refused"):
            c.append(x[:6], x[:6], x[:6], [6, 0])
    assert _same(before, _books(c))
    # the step again, and one more for the other request: no page is given twice
    c.append(x[:6], x[:6], x[:6], [6, 0])
    assert _store.positions == [2, 3, 4, 5, 6, 7]
    c.append(x[:5], x[:5], x[:5], [0, 5])
    assert c.lens == [8, 6] == c.seen
    _consistent(c, 12)
    assert torch.equal(c.k[c.table[0, :2].long()].flatten(0, 1), torch.cat([x[:2], x[:6]]))


@pytest.mark.gpu
def test_refused_append_then_steps_match_the_oracle(fk):
    import torch
    from test_gpu_kv_path import _check

    Hq, H, D, page = 4, 2, 64, 8
    c = fk.ClusteredKVCache(2, 12, page, H, D, 40, torch.float16)
    g = torch.Generator(device="cuda").manual_seed(3)

    def step(T):
        x = torch.randn(T, Hq + 2 * H, D, device="cuda", generator=g).half()
        return x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]

    c.append(*step(13), [13, 0])
    before = _books(c)
    q, k, v = step(6)
    w = torch.ones(D, dtype=torch.float16, device="cuda")
    rope = torch.ones(50, D, device="cuda")
    for bad in [dict(q=q.clone().requires_grad_()), dict(k=k[:, :1]), dict(v=v.float()), dict(q_weight=w),
                dict(q_weight=w, k_weight=w[:32]), dict(rope=rope.half()), dict(rope=rope[:, :63].contiguous()),
                dict(eps=-1.0)]:
        with pytest.raises((ValueError, fk.FKError)):
            c.append(**dict(dict(q=q, k=k, v=v, new=[3, 3]), **bad))
        assert _same(before, _books(c)), bad
    c.append(q, k, v, [3, 3])
    for _ in range(6):
        q, k, v = step(2)
        got = c.attend(c.append(q, k, v, [1, 1]), return_lse=True)
        _consistent(c, 12)
        _check(c, q, got, "f16", D)
    assert c.lens == [22, 9]


def test_positions_past_the_rotation_table_are_refused(cpu_cache):
    """Positions go on counting what compression took out: they can pass max_len."""
    import torch

    c = cpu_cache(2, 12, 4, 2, 8, 20)
    x, rope = torch.zeros(9, 2, 8), torch.zeros(24, 8)
    c.append(x[:9], x[:9], x[:9], [9, 0], rope=rope)
    c.lens[0], c.lens_dev[0], c.shift[0] = 3, 3, 6       # as a compression leaves it: 3 held of 9 seen
    c.free = torch.cat([c.free, c.table[0, 1:3]])
    c.append(x[:9], x[:9], x[:9], [9, 0], rope=rope)
    assert _store.positions == list(range(9, 18)) and c.seen == [18, 0]
    before = _books(c)
    with pytest.raises(ValueError, match="25 positions, .* 24"):
        c.append(x[:7], x[:7], x[:7], [7, 0], rope=rope)
    assert _same(before, _books(c))
    c.append(x[:6], x[:6], x[:6], [6, 0], rope=rope)     # the last row of the table
    assert _store.positions == list(range(18, 24))
    c.append(x[:8], x[:8], x[:8], [0, 8], rope=rope)     # the full request gets nothing: fine
    c.append(x[:1], x[:1], x[:1], [1, 0])                # and no rotation needs no table


def test_release_gives_the_pages_back(cpu_cache):
    import torch

    c = cpu_cache(2, 6, 4, 2, 8, 20)
    x = torch.arange(20 * 2 * 8, dtype=torch.float32).view(20, 2, 8)
    for turn in range(4):                                # more tokens in all than there are pages for
        c.append(x[:14], x[:14], x[:14], [13, 1])
        _consistent(c, 6)
        c.release(0)
        assert c.lens == [0, turn + 1] and c.seen == [0, turn + 1]
        assert (c.table[0] == -1).all()
        _consistent(c, 6)
    c.lens[1], c.centres[1], c.shift[1] = 4, 2, 3        # as a compression leaves it
    c.lens_dev[1] = 4
    c.release(1)
    assert c.lens == c.seen == c.centres == [0, 0] and c.shift.tolist() == [0, 0]
    _consistent(c, 6)
    c.append(x[:2], x[:2], x[:2], [0, 2], rope=torch.zeros(5, 8))
    assert _store.positions == [0, 1]
    c.release(0)                                         # nothing held: nothing happens
    _consistent(c, 6)


@pytest.mark.gpu
def test_release_then_another_request_matches_the_oracle(fk):
    import torch
    from test_gpu_kv_path import _check

    H, D, page = 2, 64, 8
    c = fk.ClusteredKVCache(2, 14, page, H, D, 60, torch.float16)
    g = torch.Generator(device="cuda").manual_seed(5)
    for turn in range(3):
        x = torch.randn(70 - turn, 3 * H, D, device="cuda", generator=g).half()
        c.append(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], [60 - turn, 10])
        if turn == 0:
            c.compress(1, 4, keep=3, niter=2)
        _consistent(c, 14)
        q = torch.randn(2, 2 * H, D, device="cuda", generator=g).half()
        _check(c, q, c.attend(q, return_lse=True), "f16", D)
        c.release(0)
        out, lse = c.attend(q, return_lse=True)
        assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()

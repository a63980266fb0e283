"""The paged-cache oracle against closed forms and independent formulas (CPU)."""
import numpy as np
import pytest

import oracle


def test_tables_worked_example():
    # page 4: request 0 holds 5 tokens on pages 7, 3 and gets 4 (9 -> 3 pages),
    # request 1 is empty and gets 0, request 2 is new with 5 (2 pages)
    table, lens, ct, cp, slots, pos = oracle.page_tables(
        [5, 0, 0], [4, 0, 5], np.array([[7, 3], [-1, -1], [-1, -1]]), [9, 2, 5], 4, 3, 11)
    assert table.tolist() == [[7, 3, 9], [-1, -1, -1], [2, 5, -1]]
    assert lens.tolist() == [9, 0, 5] and ct.tolist() == [0, 4, 4, 9] and cp.tolist() == [0, 1, 1, 3]
    assert slots.tolist() == [13, 14, 15, 36, 8, 9, 10, 11, 20, -1, -1]
    assert pos.tolist() == [5, 6, 7, 8, 0, 1, 2, 3, 4, 0, 0]


def test_tables_short_list_and_narrow_row():
    table, _, _, cp, slots, _ = oracle.page_tables([0, 0], [3, 9], None, [4], 2, 3, 12)
    assert cp.tolist() == [0, 2, 5] and table.tolist() == [[4, -1, -1], [-1, -1, -1]]
    assert slots.tolist() == [8, 9] + [-1] * 10


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_keeps_norms_and_relative_position(interleaved):
    rng = np.random.default_rng(1)
    T, D, rot = 6, 12, 8
    ang = np.arange(40)[:, None] * 10.0 ** -np.arange(rot // 2)[None]
    rope = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    x = np.broadcast_to(rng.standard_normal((1, 2, D)), (T, 2, D)).copy()
    w = rng.standard_normal(D)
    flat, _ = oracle.norm_rope(x, w, 0.0, None, None, interleaved)
    assert np.allclose(((flat / w) ** 2).mean(-1), 1.0)
    y, m = oracle.norm_rope(x, w, 0.0, rope, np.arange(T), interleaved)
    assert np.allclose((y ** 2).sum(-1), (flat ** 2).sum(-1))        # a rotation
    assert np.array_equal(y[0], flat[0]) and np.array_equal(y[..., rot:], flat[..., rot:])
    a, b = y[1, 0] @ y[3, 1], y[3, 0] @ y[5, 1]                      # same distance, same product
    assert np.isclose(a, b) and (m >= np.abs(y) - 1e-12).all()
    assert np.array_equal(oracle.norm_rope(x, w, 0.0, rope, np.full(T, 99), interleaved)[0],
                          oracle.norm_rope(x, w, 0.0, rope, np.full(T, 39), interleaved)[0])


def test_attn_closed_forms():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((3, 2, 1, 4)), rng.standard_normal((3, 2, 1, 4))
    table = np.array([[2, 0], [1, -1], [1, 2]])
    q = rng.standard_normal((3, 2, 4))
    # zero queries: the mean of the values and log of their number
    out, lse, _ = oracle.paged_attn(q * 0, k, v, table, [3, 4, 0], 1.0)
    assert np.allclose(out[0, 0], (v[2, 0, 0] + v[2, 1, 0] + v[0, 0, 0]) / 3)
    assert np.allclose(lse[0], np.log(3)) and np.allclose(lse[1], np.log(2))   # page -1 is absent
    assert (out[2] == 0).all() and (lse[2] == -np.inf).all()
    # a bias of log n stands for n equal keys
    bias = np.full((3, 2, 1), -np.inf)
    bias[2, 0], bias[0, 0] = np.log(5), np.log(2)
    out, lse, _ = oracle.paged_attn(q, k, v, table, [3, 0, 0], 0.7, 0.0, bias)
    kk = np.concatenate([np.repeat(k[2, 0], 5, 0), np.repeat(k[0, 0], 2, 0)])
    vv = np.concatenate([np.repeat(v[2, 0], 5, 0), np.repeat(v[0, 0], 2, 0)])
    for h in range(2):
        s = 0.7 * kk @ q[0, h]
        assert np.isclose(lse[0, h], np.log(np.exp(s).sum()))
        assert np.allclose(out[0, h], np.exp(s) @ vv / np.exp(s).sum())
    # the cap bounds scores and leaves small ones
    _, lse, _ = oracle.paged_attn(q * 1e6, k, v, table, [1, 0, 0], 1.0, 3.0)
    assert (np.abs(lse[0]) <= 3.0).all()

"""The oracles of prompt attention and of e4m3 rows against closed forms and enumeration (CPU)."""
import numpy as np

import oracle


def test_e4m3_numbers_by_enumeration():
    """All 127 non-negative numbers from their bits, and rounding as a search among them."""
    codes = np.arange(127)
    e, f = codes >> 3, codes & 7
    numbers = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    assert numbers.max() == 448 and (np.diff(numbers) > 0).all()
    assert np.array_equal(oracle.e4m3_round(numbers), numbers)
    mid = (numbers[1:] + numbers[:-1]) / 2
    even = np.where(codes[:-1] % 2 == 0, numbers[:-1], numbers[1:])
    assert np.array_equal(oracle.e4m3_round(mid), even) and np.array_equal(oracle.e4m3_round(-mid), -even)
    x = np.random.default_rng(0).uniform(0, 448, 4000)
    near = numbers[np.abs(x[:, None] - numbers[None]).argmin(1)]
    assert np.array_equal(oracle.e4m3_round(x), near)


def test_quantise_worked_rows():
    x = np.array([[448.0, 1.0, 0.0], [449.0, 1.0, -3.0], [0.0, 0.0, 0.0], [2.0 ** -140, 0, 0],
                  [np.inf, 224.5, -1.0], [np.nan, -224.0, 2.0 ** -12]])
    y, s = oracle.quantise(x)
    assert s.tolist() == [1.0, 2.0, 1.0, 2.0 ** -126, 1.0, 0.5]
    assert y[0].tolist() == [448, 1, 0] and y[1].tolist() == [448, 1, -3]
    assert np.isnan(y[4, 0]) and y[4, 1:].tolist() == [224, -1]
    assert np.isnan(y[5, 0]) and y[5, 1] == -224
    assert (y[2] == 0).all() and y[3, 0] == 0


def test_prompt_rows_are_single_token_calls():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((4, 3, 2, 5)), rng.standard_normal((4, 3, 2, 5))
    table = np.array([[2, 0], [1, 3]])
    q = rng.standard_normal((7, 4, 5))
    out, lse, _ = oracle.prompt_attn(q, k, v, table, [5, 3], [0, 2, 6], 0.6)
    for t, (b, n) in enumerate([(0, 4), (0, 5), (1, 0), (1, 1), (1, 2), (1, 3)]):
        o, s, _ = oracle.paged_attn(q[t:t + 1], k, v, table[b:b + 1], [n], 0.6)
        assert np.array_equal(out[t], o[0]) and np.array_equal(lse[t], s[0])
    assert (lse[2] == -np.inf).all() and (out[2] == 0).all()        # fewer keys than new tokens
    assert np.isnan(out[6]).all()                                   # a row of no request
    assert np.allclose(out[3, 0], v[1, 0, 0])                       # one key: its value

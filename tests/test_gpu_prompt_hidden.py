"""Prompt attention: infinite values that a row sees next to hidden ones in the same element."""
import math

import numpy as np
import pytest

import oracle
import synthdata
from gpu_helpers import host_f64, to_dev
from test_gpu_prompt import DTYPES, _call, _case, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("req", [(0, 300), (700, 70)], ids=["prompt", "chunk"])
@pytest.mark.parametrize("dims", [(4, 2, 64), (2, 1, 128), (40, 2, 96), (3, 1, 256), (3, 3, 33), (2, 1, 320)],
                         ids=lambda d: f"{d[0]}x{d[1]}d{d[2]}")
def test_hidden_values_beside_an_infinite_one(fk, dims, req, dtype):
    """A value that is infinite for all, and later ones in the same element that are not finite either:
    rows before these keep the infinity."""
    Hq, Hkv, D = dims
    old, n = req
    args, _ = _case((Hq, Hkv, D, 16, [req], None, 0.0, "plain"), dtype, D + n)
    args["q"] *= 0.0625                              # scores of a few tenths: no weight underflows
    k64, v64 = (np.nan_to_num(host_f64(args[c].nan_to_num(), dtype)) for c in ("k_cache", "v_cache"))
    want = oracle.prompt_attn(host_f64(args["q"].nan_to_num(), dtype), k64, v64, args["table"].cpu().numpy(),
                              [old + n], [0, n], 1.0 / math.sqrt(D))
    inf, nan = math.inf, math.nan
    column = np.zeros((n, 4))                        # what elements 3, 4, 5 and D - 1 are
    at = lambda i: args["v_cache"][int(args["table"][0, (old + i) // 16]), (old + i) % 16]      # noqa: E731
    for c, (e, first, later) in enumerate([(3, inf, {n // 3: inf, n - 20: inf}), (4, inf, {n // 3: nan}),
                                           (5, inf, {n - 20: -inf}), (D - 1, -inf, {n - 1: nan, n // 2: -inf})]):
        seen = 5 if old == 0 else -old + 3           # new token 5, or a key held before
        at(seen)[:, e] = first
        column[max(seen, 0):, c] = first
        for i, x in later.items():
            at(i)[:, e] = x
            with np.errstate(invalid="ignore"):
                column[i:, c] += x
    for hint in (0, 1):
        got = _call(fk, args, dtype, max_len=hint)
        out = got[0].double().cpu().numpy()
        for c, e in enumerate((3, 4, 5, D - 1)):
            rows = slice(5 if old == 0 else 0, n)
            exp = column[rows, c][:, None]
            assert np.array_equal(out[rows, :, e], np.broadcast_to(exp, out[rows, :, e].shape), equal_nan=True), (hint, e)
            out[rows, :, e] = want[0][rows, :, e]
        fixed = to_dev(synthdata.to_storage(out.astype(np.float32), dtype), dtype)
        _check((fixed, got[1]), want, dtype, D, 0.0, f"max_len {hint}")

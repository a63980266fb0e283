"""Prompts of 16-bit rows that are not whole 16-byte units, few rows over long keys and many: the kernel
goes by the number of rows and keys, the result does not. Bounds as in test_gpu_prompt.py."""
import math

import pytest

from test_gpu_prompt import _call, _case, _check

pytestmark = pytest.mark.gpu

FEW, MANY = [(600, 7), (0, 0), (300, 1), (0, 40)], [(600, 130), (0, 0), (300, 1), (0, 300)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("reqs", [FEW, MANY], ids=["few", "many"])
@pytest.mark.parametrize("case", [(4, 2, 33, 16, None, 0.0, "plain"), (8, 1, 90, 7, "log", 20.0, "odd"),
                                  (3, 3, 130, 16, "lowest", 0.0, "wide"), (6, 2, 250, 24, "log", 0.0, "heads"),
                                  (2, 1, 7, 1, None, 100.0, "odd"), (2, 2, 66, 16, None, 0.0, "holes")],
                         ids=lambda c: f"{c[0]}x{c[1]}d{c[2]}{c[6]}")
def test_few_and_many_rows(fk, case, reqs, dtype):
    Hq, Hkv, D, page, bias, cap, how = case
    args, want = _case((Hq, Hkv, D, page, reqs, bias, cap, how), dtype, D)
    for hint in (0, 100, 1 << 20):
        _check(_call(fk, args, dtype, max_len=hint), want, dtype, D, cap, f"max_len {hint}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_thousands_of_keys(fk, dtype):
    """Single tokens and a few over keys of more than one round of a block's waves, in a wide table."""
    import torch
    args, want = _case((4, 1, 90, 16, [(5000, 1), (0, 1), (2600, 9)], None, 0.0, "plain"), dtype, 4)
    _check(_call(fk, args, dtype), want, dtype, 90, 0.0)
    table = args["table"]
    args["table"] = torch.cat([table, table.new_full((3, 1 << 16), -1)], 1)
    first = _call(fk, args, dtype)
    _check(first, want, dtype, 90, 0.0)
    again = _call(fk, args, dtype)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    args["q"][0, 0, 3] = math.nan                        # a row of its own
    out, lse = _call(fk, args, dtype)
    assert out.isnan().sum() == 90 and lse.isnan().sum() == 1 and out[0, 0].isnan().all()

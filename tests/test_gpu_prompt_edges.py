"""Prompt attention: numbers that are not finite, long caches cut into parts, streams, captured
graphs, workspaces of any content, rows of no request."""
import math

import numpy as np
import pytest

import oracle
import synthdata
from gpu_helpers import host_f64, to_dev
from test_gpu_prompt import DTYPES, _call, _case, _check, _dev

pytestmark = pytest.mark.gpu

DIMS = [(4, 2, 64), (8, 2, 128), (40, 2, 96), (3, 1, 256), (3, 3, 33)]
IDS = [f"{a}x{b}d{d}" for a, b, d in DIMS]


def _at(args, b, j):
    """Page and token of key j of request b."""
    page = args["k_cache"].shape[1]
    return int(args["table"][b, j // page]), j % page


def _like(a, t):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(t.dtype).to(t.device)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("reqs", [[(0, 150), (70, 40)], [(700, 30), (1000, 20)]], ids=["prompts", "chunks"])
@pytest.mark.parametrize("dims", DIMS, ids=IDS)
def test_values_reach_only_the_rows_that_see_them(fk, dims, reqs, dtype):
    """Infinities and NaN in values: rows before them stay as they were, later ones get them
    in their element."""
    Hq, Hkv, D = dims
    args, _ = _case((Hq, Hkv, D, 16, reqs, None, 0.0, "plain"), dtype, D)
    args["q"] *= 0.0625                              # scores of a few tenths: no weight underflows
    scale = 1.0 / math.sqrt(D)
    lens = [a + n for a, n in reqs]
    k64, v64 = (np.nan_to_num(host_f64(args[c].nan_to_num(), dtype)) for c in ("k_cache", "v_cache"))
    want = oracle.prompt_attn(host_f64(args["q"].nan_to_num(), dtype), k64, v64, args["table"].cpu().numpy(),
                              lens, args["cu_tokens"].tolist(), scale)
    put = []
    for b, (old, n) in enumerate(reqs):
        for i, e, x in ((n // 2, 3, math.inf), (n - 1, D - 1, math.nan), (1, D // 2, -math.inf),
                        (n // 2 + 1, 7, math.inf), (n // 2 + 1, 8, -math.inf)):
            args["v_cache"][_at(args, b, old + i)][:, e] = x
            put.append((b, i, e, x))
    for hint in (0, 1):
        got = _call(fk, args, dtype, max_len=hint)
        out = got[0].double().cpu().numpy()
        cu = args["cu_tokens"].tolist()
        for b, i, e, x in put:
            rows = slice(cu[b] + i, cu[b + 1])
            bad = out[rows, :, e]
            assert np.isnan(bad).all() if x != x else (bad == x).all(), (b, i, e, x)
            out[rows, :, e] = want[0][rows, :, e]
        fixed = to_dev(synthdata.to_storage(out.astype(np.float32), dtype), dtype)
        _check((fixed, got[1]), want, dtype, D, 0.0, f"max_len {hint}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dims", DIMS, ids=IDS)
def test_keys_reach_only_the_rows_and_heads_that_see_them(fk, dims, dtype):
    Hq, Hkv, D = dims
    args, want = _case((Hq, Hkv, D, 16, [(0, 90), (40, 70)], None, 0.0, "plain"), dtype, D + 1)
    args["k_cache"][_at(args, 1, 40 + 30)][Hkv - 1, D - 1] = math.nan
    out, lse = _call(fk, args, dtype)
    G, rows = Hq // Hkv, slice(90 + 30, 160)
    assert out[rows, -G:].isnan().all() and lse[rows, -G:].isnan().all()
    out[rows, -G:], lse[rows, -G:] = (_like(x[rows, -G:], t) for x, t in zip(want, (out, lse)))
    _check((out, lse), want, dtype, D, 0.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dims", DIMS, ids=IDS)
def test_scores_of_minus_infinity_and_queries_that_are_not_finite(fk, dims, dtype):
    Hq, Hkv, D = dims
    reqs = [(0, 60), (10, 20), (0, 5)]
    args, _ = _case((Hq, Hkv, D, 16, reqs, None, 0.0, "plain"), dtype, D + 2)
    q = args["q"]
    q[:85, :, :2] = q[:85, :, :2].abs() + 0.5        # -inf times these is -inf for every head
    lens = [a + n for a, n in reqs]
    bias = np.zeros(args["k_cache"].shape[:3])
    for b, j, e in ((0, 0, 0), (0, 7, 1), (1, 12, 0), (2, 4, 1)):
        at = _at(args, b, j)
        args["k_cache"][at][:, e] = -math.inf
        bias[at] = -math.inf
    k64, v64 = (host_f64(args[c], dtype) for c in ("k_cache", "v_cache"))
    want = oracle.prompt_attn(host_f64(q.nan_to_num(), dtype), k64, v64, args["table"].cpu().numpy(), lens,
                              args["cu_tokens"].tolist(), 1 / math.sqrt(D), 0.0, bias)
    assert (want[1][0] == -np.inf).all()             # the first token's only key is out
    _check(_call(fk, args, dtype), want, dtype, D, 0.0)
    # a query that is NaN makes its row NaN and no other
    q[3, 0, 0] = math.nan
    out, lse = _call(fk, args, dtype)
    assert out[3, 0].isnan().all() and lse[3, 0].isnan()
    keep = lse.isnan().sum()
    assert keep == 1 and out[:85].isnan().sum() == D


LONG = [
    (8, 2, 128, 16, [(5000, 33), (0, 700), (2500, 1)], None, 0.0, "plain"),
    (4, 1, 64, 48, [(9000, 5)], "log", 0.0, "plain"),
    (2, 1, 96, 1, [(0, 1300)], None, 20.0, "plain"),
    (1, 1, 256, 16, [(3000, 2), (10, 0), (1, 1)], None, 0.0, "plain"),
    (6, 2, 192, 16, [(2000, 70)], "none", 0.0, "plain"),
    (16, 1, 128, 256, [(4000, 3)] + [(i * 37, i % 5) for i in range(12)], None, 0.0, "plain"),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", LONG, ids=[f"{c[0]}x{c[1]}d{c[2]}" for c in LONG])
def test_long_keys_cut_into_parts(fk, case, dtype):
    torch = pytest.importorskip("torch")
    args, want = _case(case, dtype, seed=case[2])
    most = max(a + n for a, n in case[4])
    for hint in (0, most, most // 3, 1):
        _check(_call(fk, args, dtype, max_len=hint), want, dtype, case[2], case[6], f"max_len {hint}")
    # a table with room for 2^20 keys a request, most of it unused
    table = args["table"]
    args["table"] = torch.cat([table, table.new_full((table.shape[0], (1 << 20) // case[3]), -1)], 1)
    _check(_call(fk, args, dtype), want, dtype, case[2], case[6], "wide table")


def test_many_requests(fk):
    rng = np.random.default_rng(4)
    reqs = [(int(rng.integers(0, 90)), int(rng.integers(0, 40))) for _ in range(150)]
    reqs[5] = (0, 400)
    for case in ((4, 2, 64, 16, reqs, None, 0.0, "plain"), (2, 2, 128, 8, reqs, "log", 0.0, "plain")):
        args, want = _case(case, "bf16", 3)
        _check(_call(fk, args, "bf16"), want, "bf16", case[2], 0.0)


def test_same_bits_any_workspace_and_stream(fk):
    import torch

    args, want = _case((8, 2, 128, 16, [(3000, 20), (0, 0), (37, 90)], "log", 0.0, "plain"), "bf16", 8)
    T, Hq, D = args["q"].shape
    n = fk.fk_workspace_size_prompt(torch.bfloat16, T, 3, 8, 2, 128)
    first = None
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = _call(fk, args, "bf16", ws=ws)
        torch.cuda.current_stream().wait_stream(side)
        _check(got, want, "bf16", D, 0.0)
        if first is not None:
            assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1])
        first = got


@pytest.mark.parametrize("D", [64, 33])
def test_captured_and_replayed(fk, D):
    """A step in a graph, replayed over other lengths, tokens and caches, with eager calls between."""
    import torch

    cases = [(4, 2, D, 16, [(1200, 20), (0, 44), (3, 6)], None, 0.0, "plain"),
             (4, 2, D, 16, [(900, 1), (40, 59), (0, 10)], None, 0.0, "plain"),
             (4, 2, D, 16, [(0, 64), (0, 0), (1220, 6)], None, 0.0, "plain")]
    made = [_case(c, "f16", i) for i, c in enumerate(cases)]
    pages = max(m[0]["k_cache"].shape[0] for m in made)
    width = max(m[0]["table"].shape[1] for m in made)
    kc = torch.zeros((pages, 16, 2, D), dtype=torch.float16, device="cuda")
    vc, table = torch.zeros_like(kc), torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    q, lens, cu = made[0][0]["q"].clone(), made[0][0]["lens"].clone(), made[0][0]["cu_tokens"].clone()
    assert all(m[0]["q"].shape == q.shape for m in made)
    ws = torch.empty(fk.fk_workspace_size_prompt(torch.float16, q.shape[0], 3, 4, 2, D), dtype=torch.uint8,
                     device="cuda")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")

    def step():
        fk.fk_prompt_attn(q, kc, vc, table, lens, cu, out=out, lse=lse, ws=ws)

    def fill(args):
        kc[:args["k_cache"].shape[0]] = args["k_cache"]
        vc[:args["v_cache"].shape[0]] = args["v_cache"]
        table.fill_(-1)
        table[:, :args["table"].shape[1]] = args["table"].clamp(max=args["k_cache"].shape[0])
        table[table >= args["k_cache"].shape[0]] = -1
        for a, b in ((q, "q"), (lens, "lens"), (cu, "cu_tokens")):
            a.copy_(args[b])

    fill(made[0][0])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (1, 0, 2, 1, 1):
        args, want = made[i]
        fill(args)
        out.fill_(7), lse.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        _check((out, lse), want, "f16", D, 0.0, f"replay {i}")
        eager = _call(fk, args, "f16")
        _check(eager, want, "f16", D, 0.0, f"eager {i}")


def test_nothing_to_do(fk):
    import torch

    z = dict(dtype=torch.float16, device="cuda")
    kc = torch.zeros((2, 16, 2, 64), **z)
    i32 = dict(dtype=torch.int32, device="cuda")
    out = fk.fk_prompt_attn(torch.zeros((0, 4, 64), **z), kc, kc.clone(), torch.zeros((3, 2), **i32),
                            torch.zeros(3, **i32), torch.zeros(4, **i32))
    assert out.shape == (0, 4, 64)
    mark = torch.full((5, 4, 64), 3.0, **z)          # tokens, but no request has them
    q = torch.randn((5, 4, 64), **z)
    fk.fk_prompt_attn(q, kc, kc.clone(), torch.zeros((0, 2), **i32), torch.zeros(0, **i32),
                      torch.zeros(1, **i32), out=mark)
    assert (mark == 3).all()
    fk.fk_prompt_attn(q, kc, kc.clone(), torch.zeros((2, 2), **i32), torch.zeros(2, **i32),
                      torch.zeros(3, **i32), out=mark)
    assert (mark == 3).all()
    for width, pages in ((0, 2), (2, 0)):            # no keys at all: zeros and -inf
        none = kc[:pages]
        got, lse = fk.fk_prompt_attn(q, none, none.clone(), torch.zeros((1, width), **i32),
                                     torch.full((1,), 5, **i32), torch.tensor([0, 5], **i32), return_lse=True)
        assert (got == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("dims", [(4, 2, 64), (3, 1, 33)], ids=["d64", "d33"])
def test_thousands_of_requests(fk, dims):
    """More requests than one or two rounds of the search for a block's request take, most of them
    with nothing new."""
    rng = np.random.default_rng(9)
    for n in (65, 4097, 9000):
        reqs = [(int(a), int(b)) for a, b in zip(rng.integers(0, 4, n), rng.integers(-12, 3, n).clip(0))]
        reqs[n // 2], reqs[-1], reqs[0] = (40, 90), (3, 0), (0, 2)
        args, want = _case((*dims, 8, reqs, None, 0.0, "plain"), "f16", n)
        _check(_call(fk, args, "f16"), want, "f16", dims[2], 0.0, f"{n} requests")

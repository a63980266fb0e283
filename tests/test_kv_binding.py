"""What the paged-cache calls' Python side refuses beyond types and shapes."""
import pytest


@pytest.mark.gpu
def test_trained_weights_are_refused_unless_no_gradient_is_asked_for(fk):
    import torch

    q, k = torch.randn(3, 4, 64, device="cuda"), torch.randn(3, 2, 64, device="cuda")
    w = torch.rand(64, device="cuda")
    par = torch.nn.Parameter(w.clone())
    rope, pos = torch.rand(9, 64, device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda")
    turn = torch.nn.Parameter(rope.clone())
    want = fk.fk_qk_norm_rope(q, k, None, w, w, rope=rope, positions=pos)
    for ws, r, name in (((par, w), rope, "q_weight"), ((w, par), rope, "k_weight"), ((w, w), turn, "rope")):
        with pytest.raises(ValueError, match=f"{name} requires grad"):
            fk.fk_qk_norm_rope(q, k, None, *ws, rope=r, positions=pos)
        with torch.no_grad():
            got = fk.fk_qk_norm_rope(q, k, None, *ws, rope=r, positions=pos)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_meets_is_exact():
    """Overlap of a byte range with a strided tensor, against marks on every byte."""
    import random

    import torch
    from exact_means_clustering_flashassign_amd._binding import _meets

    rng, buf = random.Random(1), torch.zeros(4000, dtype=torch.int16)
    for _ in range(400):
        shape = [rng.randint(1, 4) for _ in range(3)]
        inner = [1, shape[2] + rng.randint(0, 3)]
        inner.append((shape[1] - 1) * inner[1] + shape[2] + rng.randint(0, 40))
        strides = [inner[2], inner[1], 1]
        if rng.random() < 0.3:                           # heads outside tokens
            shape[0], shape[1], strides[0], strides[1] = shape[1], shape[0], strides[1], strides[0]
        t = buf.as_strided(shape, strides)
        used = torch.zeros(4000, dtype=torch.bool)
        used.as_strided(shape, strides).fill_(True)
        used = used.repeat_interleave(2)
        lo = rng.randint(-30, 300)
        hi = lo + rng.randint(0, 60)
        assert _meets(lo, hi, t) == bool(used[max(lo, 0):max(hi, 0)].any()), (shape, strides, lo, hi)


def _tables(fk, B=40, page=4, width=9):
    import torch

    i32 = dict(dtype=torch.int32, device="cuda")
    old, new = torch.arange(B, **i32) % 20, torch.arange(B, **i32) % 7
    T = int(new.sum())
    free, table = torch.arange(500, **i32), torch.full((B, width), 3, **i32)
    out = [torch.empty(s, **i32) for s in ((B, width), (B,), (B + 1,), (B + 1,), (T,), (T,))]
    return (old, new, free, page, width, T), table, out


@pytest.mark.gpu
def test_page_tables_outputs_apart(fk):
    import torch

    args, table, out = _tables(fk)
    want = fk.fk_page_tables(*args, table=table)
    assert all(torch.equal(a, b) for a, b in zip(want, fk.fk_page_tables(*args, table=table, out=out)))
    big = torch.zeros(2000, dtype=torch.int32, device="cuda")
    B, T, width = 40, args[5], 9
    shifted = big[:B * width + 7]
    for bad, kw, name in [
            ({1: args[0]}, {}, r"out\[1\] overlaps len_old"), ({1: args[1]}, {}, r"out\[1\] overlaps len_new"),
            ({4: args[2][:T]}, {}, r"out\[4\] overlaps free_pages"), ({5: out[4]}, {}, r"out\[5\] overlaps out\[4\]"),
            ({2: big[:B + 1], 3: big[B:2 * B + 1]}, {}, r"out\[3\] overlaps out\[2\]"),
            ({0: shifted[7:].view(B, width)}, dict(table=shifted[:B * width].view(B, width)), r"out\[0\] overlaps table"),
            ({1: table.view(-1)[:B]}, {}, r"out\[1\] overlaps table")]:
        outs = [bad.get(i, t) for i, t in enumerate(out)]
        with pytest.raises(ValueError, match=name):
            fk.fk_page_tables(*args, **dict(dict(table=table), **kw), out=outs)
    got = fk.fk_page_tables(*args, table=table, out=[table] + out[1:])
    assert got[0] is table and all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 33])
def test_norm_rope_outputs_apart(fk, D):
    import torch

    T, Hq, H, page = 3, 4, 2, 4
    gen = torch.Generator(device="cuda").manual_seed(6)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)      # noqa: E731
    qkv, w, rot = rnd(T, Hq + 2 * H, D), rnd(D), D // 2 * 2
    rope, pos = rnd(T * Hq * D // rot + 2, rot), torch.arange(T, dtype=torch.int32, device="cuda")
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    kc, vc = torch.zeros(8, page, H, D, device="cuda"), torch.zeros(8, page, H, D, device="cuda")
    kw = dict(rope=rope, positions=pos, slots=torch.arange(T, dtype=torch.int32, device="cuda"), k_cache=kc, v_cache=vc)
    want = fk.fk_qk_norm_rope(q, k, v, w, w, **kw, k_out=torch.empty(T, H, D, device="cuda"))
    qc, n, m = q.contiguous(), T * Hq * D, T * H * D
    flat = qkv.view(-1)
    one = torch.empty(n + m - 1, device="cuda")
    for q_, bad, name in [(qc, dict(q_out=qc), "q_out overlaps q,"), (q, dict(q_out=flat[:n].view(T, Hq, D)), "q_out overlaps"),
                          (q, dict(k_out=flat[-m:].view(T, H, D)), "k_out overlaps"),
                          (q, dict(q_out=rope.view(-1)[:n].view(T, Hq, D)), "q_out overlaps rope"),
                          (q, dict(q_out=kc.view(-1)[:n].view(T, Hq, D)), "q_out overlaps k_cache"),
                          (q, dict(k_out=vc.view(-1)[-m:].view(T, H, D)), "k_out overlaps v_cache"),
                          (q, dict(q_out=one[:n].view(T, Hq, D), k_out=one[-m:].view(T, H, D)), "overlaps k_out")]:
        with pytest.raises(ValueError, match=name):
            fk.fk_qk_norm_rope(q_, k, v, w, w, **kw, **bad)
    # outputs in the gaps of an input are apart from it
    row = Hq * D + T * Hq * D
    buf = torch.zeros(T * row, device="cuda")
    wide = buf.as_strided((T, Hq, D), (row, D, 1))
    wide.copy_(q)
    got = fk.fk_qk_norm_rope(wide, k, v, w, w, **kw, q_out=buf[Hq * D:row].view(T, Hq, D),
                             k_out=buf[row + Hq * D:row + Hq * D + m].view(T, H, D))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(wide, q)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 33])
def test_paged_attn_in_place_or_apart(fk, D):
    """out over q: the same bits where it is q, refused where it is a part of it."""
    import torch

    gen = torch.Generator(device="cuda").manual_seed(7)
    B, Hq, H, page, width = 3, 8, 2, 16, 400
    kc, vc = (torch.randn(60, page, H, D, device="cuda", generator=gen).half() for _ in range(2))
    table = torch.randint(0, 60, (B, width), device="cuda", generator=gen, dtype=torch.int32)
    lens = torch.tensor([width * page, 0, 77], dtype=torch.int32, device="cuda")
    buf = torch.randn((2 * B + 1) * Hq * D, device="cuda", generator=gen).half()
    n = B * Hq * D
    q = buf[:n].view(B, Hq, D)
    for hint in (0, 40, 700):
        want = fk.fk_paged_attn(q, kc, vc, table, lens, max_len=hint, return_lse=True)
        mine = q.clone()
        got = fk.fk_paged_attn(mine, kc, vc, table, lens, max_len=hint, out=mine, return_lse=True)
        assert got[0] is mine and torch.equal(mine, want[0]) and torch.equal(got[1], want[1])
    for q_, out in ((q, buf[D:n + D].view(B, Hq, D)), (buf.as_strided((B, Hq, D), (Hq * D, D, 1), 8), buf[:n].view(B, Hq, D)),
                    (buf.as_strided((B, Hq, D), (2 * Hq * D, D, 1)), q)):
        with pytest.raises(ValueError, match="out overlaps q"):
            fk.fk_paged_attn(q_, kc, vc, table, lens, out=out)
    gaps = buf.as_strided((2, Hq, D), (4 * Hq * D, D, 1))
    got = fk.fk_paged_attn(gaps, kc, vc, table[:2], lens[:2], out=buf[Hq * D:3 * Hq * D].view(2, Hq, D))
    assert torch.equal(got, fk.fk_paged_attn(gaps, kc, vc, table[:2], lens[:2]))


def test_empty_ranges_overlap_nothing():
    from exact_means_clustering_flashassign_amd._binding import _apart

    _apart([("out", 100, 200)], [("free_pages", 150, 150), ("q", 200, 300), ("k", 0, 100)])
    _apart([("out", 100, 200), ("lens", 150, 150)], [])
    for other in ((150, 151), (0, 101), (199, 300), (0, 300)):
        with pytest.raises(ValueError, match="out overlaps x, which the call reads"):
            _apart([("out", 100, 200)], [("x", *other)])
        with pytest.raises(ValueError, match="out overlaps x"):
            _apart([("x", *other), ("out", 100, 200)], [])

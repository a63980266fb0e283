"""Measured cases of the paged key-value-cache operators.

Three operators, called as a program that serves attention over a clustered or
plain paged cache calls them:

  tables  fk_page_tables:   block tables, token slots and positions of a step,
                            built on the GPU from request lengths;
  rope    fk_qk_norm_rope:  per-head RMS norm of queries and keys with the
                            position rotation, keys and values written to
                            their slots of the cache;
  attn    fk_paged_attn:    attention of one new token per request over the
                            paged cache, with a per-key bias (log of cluster
                            counts) and a tanh cap.

``run`` computes each in its plain form (elementary torch operations, 32-bit
arithmetic, one rounding at the end) unless ``own`` is set, when it calls the
library. ``exact`` computes the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a batch of 32 long requests: every request gains
        # one token, a few of them a page; latency counts
        _tables("tables_decode_b32", B=32, page=16, old=75600, new=1, pad=0),
        # chunked prompts of many requests at once, ragged, some with nothing new
        _tables("tables_prompts_b1024", B=1024, page=64, old=4096, new=2048, pad=777),
        # one-token pages (token lists of routed attention), few requests
        _tables("tables_page1_b8", B=8, page=1, old=30000, new=32768, pad=5),
        # the new tokens of one decode step, 32 requests
        _rope("rope_decode_t32", T=32, Hq=32, Hkv=8, D=128, rot=128, inter=False, norm=True,
              page=16, packed=True, dtype="bf16"),
        # one long prompt
        _rope("rope_prompt_t75600", T=75600, Hq=32, Hkv=8, D=128, rot=128, inter=False,
              norm=True, page=16, packed=True, dtype="f16"),
        # odd sizes: interleaved pairs over part of the head, fp32, no cache
        _rope("rope_partial_f32_t8191", T=8191, Hq=12, Hkv=4, D=96, rot=40, inter=True,
              norm=True, page=0, packed=False, dtype="f32"),
        # one short request alone: launch and dependent-load latency
        _attn("attn_one_2048", B=1, Hq=16, Hkv=4, D=64, len=2048, spread="equal", page=16,
              bias=False, cap=0.0, dtype="f16"),
        # one long request alone: the cache's length is the only axis to split
        _attn("attn_one_131072", B=1, Hq=32, Hkv=8, D=128, len=131072, spread="equal", page=64,
              bias=False, cap=0.0, dtype="bf16"),
        # a serving batch from empty to long, most of them short
        _attn("attn_ragged_b32", B=32, Hq=32, Hkv=8, D=128, len=16384, spread="log", page=16,
              bias=False, cap=0.0, dtype="bf16"),
        # a compressed cache: 1000 cluster centres weighted by log count (some
        # clusters empty) and 56 recent tokens, one query head per key head, scores capped
        _attn("attn_clusters_b32", B=32, Hq=32, Hkv=32, D=128, len=1056, spread="equal", page=32,
              bias=True, cap=30.0, dtype="f16"),
        # one key head for 16 query heads, wide head, fp32
        _attn("attn_mqa_f32_b4", B=4, Hq=16, Hkv=1, D=256, len=32768, spread="linear", page=48,
              bias=False, cap=0.0, dtype="f32"),
        # the largest: a batch of long requests
        _attn("attn_long_b32", B=32, Hq=32, Hkv=8, D=128, len=65536, spread="linear", page=16,
              bias=False, cap=0.0, dtype="bf16"),
    ]


def _tables(name, **kw):
    return dict({"name": name, "op": "tables"}, **kw)


def _rope(name, **kw):
    return dict({"name": name, "op": "rope"}, **kw)


def _attn(name, **kw):
    return dict({"name": name, "op": "attn"}, **kw)


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "rope", "attn", "attn", "attn"])
    if op == "tables":
        B, page = _log(rng, 1, 4096), rng.choice([1, 8, 16, 24, 64, 256])
        new = rng.choice([1, _log(rng, 1, 32768)])
        new = max(1, min(new, (1 << 22) // B))
        old = max(1, min(_log(rng, 1, 131072), (1 << 24) * page // B))
        return {"op": op, "B": B, "page": page, "old": old, "new": new,
                "pad": rng.choice([0, rng.randint(1, 999)])}
    dtype = rng.choice(["f32", "f16", "bf16"])
    D = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
    Hkv, G = rng.choice([1, 2, 4, 8, 8, 20, 32]), rng.choice([1, 1, 2, 4, 4, 7, 8, 16, 32])
    if op == "rope":
        T = _log(rng, 1, 100000)
        T = max(1, min(T, 75600 * 48 * 128 * 2 // ((Hkv * G + 2 * Hkv) * D * BYTES[dtype])))
        inter = rng.random() < 0.4
        rot = rng.choice([0, D, D, D // 2, 16 if inter else 12])
        return {"op": op, "T": T, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "rot": rot, "inter": inter,
                "norm": rng.random() < 0.7, "page": rng.choice([0, 1, 16, 20, 64]),
                "packed": rng.random() < 0.6, "dtype": dtype}
    B, n = _log(rng, 1, 256), _log(rng, 1, 131072)
    # bytes of keys: under half of the largest listed case, less with more query heads
    room = (1 << 31) * 4 // max(4, G)
    B = max(1, min(B, room // (Hkv * D * BYTES[dtype] * n)))
    n = max(1, min(n, room // (Hkv * D * BYTES[dtype] * B)))
    return {"op": op, "B": B, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "len": n,
            "spread": rng.choice(["equal", "log", "linear"]), "page": rng.choice([1, 8, 16, 20, 64, 256]),
            "bias": rng.random() < 0.4, "cap": rng.choice([0.0, 0.0, 20.0, 50.0]), "dtype": dtype}


def _lengths(case):
    """Request lengths of a case (their order goes by the seed): all the same,
    spread evenly, or spread evenly over the logarithm with an empty request."""
    B, n = case["B"], case["len"]
    if case["spread"] == "equal":
        return [n] * B
    if case["spread"] == "linear":
        return [max(1, (n * (i + 1)) // B) for i in range(B)]
    ls = [int(round(n ** ((i + 1) / B))) for i in range(B)]
    if B > 1:
        ls[0] = 0
    return ls


def _table_lengths(case):
    """(old, new) of every request: old evenly spread up to case["old"], every
    seventh request new (old 0); new evenly spread up to case["new"], every
    fifth request with none unless all get one token."""
    B = case["B"]
    old = [0 if i % 7 == 3 else max(1, case["old"] * (i + 1) // B) for i in range(B)]
    new = [case["new"] if case["new"] == 1 else
           (0 if i % 5 == 2 else max(1, case["new"] * (B - i) // B)) for i in range(B)]
    return old, new


def _ceil(a, b):
    return -(-a // b)


def _table_sizes(case):
    old, new = _table_lengths(case)
    P = case["page"]
    width = max(_ceil(o + n, P) for o, n in zip(old, new))
    held = [_ceil(o, P) for o in old]
    need = [_ceil(o + n, P) for o, n in zip(old, new)]
    return old, new, width, held, need


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _randn(g, shape, dtype, scale=1.0):
    x = torch.empty(shape, dtype=DTYPES[dtype], device="cuda").normal_(generator=g)
    return x if scale == 1.0 else x * scale


def _shuffled(values, seed):
    order = np.random.RandomState(seed % (1 << 32)).permutation(len(values))
    return [values[i] for i in order]


def prepare(case, seed):
    g = _gen(seed)
    return {"tables": _prepare_tables, "rope": _prepare_rope, "attn": _prepare_attn}[case["op"]](
        case, seed, g)


def _prepare_tables(case, seed, g):
    old, new, width, held, need = _table_sizes(case)
    order = _shuffled(list(range(case["B"])), seed)
    old, new, held = ([v[i] for i in order] for v in (old, new, held))
    total, want = sum(held), sum(need) - sum(held)
    pages = torch.randperm(total + want + 16, generator=g, device="cuda").to(torch.int32)
    held_t = torch.tensor(held, device="cuda")
    at = torch.cumsum(held_t, 0) - held_t
    col = torch.arange(width, device="cuda")
    idx = (at[:, None] + col[None, :]).clamp_(max=pages.numel() - 1)
    table = torch.where(col[None, :] < held_t[:, None], pages[idx], pages.new_tensor(-1))
    return {"op": "tables", "len_old": _i32(old), "len_new": _i32(new), "table": table.contiguous(),
            "free": pages[total:].contiguous(), "page": case["page"], "width": width,
            "tokens": sum(new) + case["pad"]}


def _rope_table(positions, rot):
    half = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    ang = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * \
        (10000.0 ** (-2.0 * half / rot))[None, :]
    return torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32)


def _prepare_rope(case, seed, g):
    T, Hq, Hkv, D, dt = case["T"], case["Hq"], case["Hkv"], case["D"], case["dtype"]
    if case["packed"]:            # one projection's output, queries, keys and values side by side
        qkv = _randn(g, (T, Hq + 2 * Hkv, D), dt)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = (_randn(g, (T, h, D), dt) for h in (Hq, Hkv, Hkv))
    s = {"op": "rope", "q": q, "k": k, "v": v if case["page"] else None, "inter": case["inter"]}
    for name in ("q_weight", "k_weight"):
        s[name] = (1 + 0.1 * _randn(g, (D,), "f32")).to(DTYPES[dt]) if case["norm"] else None
    most = max(T, 4096)
    s["rope"] = _rope_table(most, case["rot"]) if case["rot"] else None
    s["positions"] = (torch.arange(T, device="cuda", dtype=torch.int32) if T > 256 else
                      torch.randint(0, most, (T,), generator=g, device="cuda", dtype=torch.int32))
    s["slots"] = s["k_cache"] = s["v_cache"] = None
    if case["page"]:
        P = case["page"]
        n = _ceil(T, P) + 1
        pages = torch.randperm(n, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        slots = (pages[t // P] * P + t % P).to(torch.int32)
        if T > 8:                 # two padding tokens of the step
            slots[T - 2:] = -1
        s["slots"] = slots
        s["k_cache"] = torch.zeros((n, P, Hkv, D), dtype=DTYPES[dt], device="cuda")
        s["v_cache"] = torch.zeros((n, P, Hkv, D), dtype=DTYPES[dt], device="cuda")
    return s


def _prepare_attn(case, seed, g):
    B, Hq, Hkv, D, P, dt = (case[n] for n in ("B", "Hq", "Hkv", "D", "page", "dtype"))
    lens = _shuffled(_lengths(case), seed)
    width = max(1, _ceil(max(lens), P))
    held = [_ceil(n, P) for n in lens]
    pages = sum(held) + 1
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    held_t = torch.tensor(held, device="cuda")
    at = torch.cumsum(held_t, 0) - held_t
    col = torch.arange(width, device="cuda")
    idx = (at[:, None] + col[None, :]).clamp_(max=pages - 1)
    table = torch.where(col[None, :] < held_t[:, None], perm[idx], perm.new_tensor(-1))
    s = {"op": "attn", "q": _randn(g, (B, Hq, D), dt, 3.0), "table": table.contiguous(),
         "k_cache": _randn(g, (pages, P, Hkv, D), dt), "v_cache": _randn(g, (pages, P, Hkv, D), dt),
         "lens": _i32(lens), "scale": 1.0 / math.sqrt(D), "cap": case["cap"], "bias": None}
    if case["bias"]:              # log of cluster counts, empty clusters at -inf
        counts = torch.randint(0, 150, (pages, P, Hkv), generator=g, device="cuda")
        s["bias"] = counts.to(torch.float32).log()
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        import exact_means_clustering_flashassign_amd as fk

        if s["op"] == "tables":
            r = fk.fk_page_tables(s["len_old"], s["len_new"], s["free"], s["page"], s["width"],
                                  s["tokens"], table=s["table"])
            return dict(zip(("table", "lens", "cu_tokens", "cu_pages", "slots", "positions"), r))
        if s["op"] == "rope":
            q, k = fk.fk_qk_norm_rope(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], EPS,
                                      s["rope"], s["positions"], s["inter"], s["slots"],
                                      s["k_cache"], s["v_cache"])
            if s["slots"] is None:
                return {"q": q, "k": k}
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        out, lse = fk.fk_paged_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                    s["scale"], s["cap"], s["bias"], return_lse=True)
        return {"out": out, "lse": lse}
    return {"tables": _plain_tables, "rope": _plain_rope, "attn": _plain_attn}[s["op"]](s)


def _plain_tables(s):
    P, W, F = s["page"], s["width"], s["free"].numel()
    old, new = s["len_old"].long(), s["len_new"].long()
    zero = old.new_zeros(1)
    held, need = (old + P - 1) // P, (old + new + P - 1) // P
    cu_tokens = torch.cat([zero, new.cumsum(0)])
    cu_pages = torch.cat([zero, (need - held).cumsum(0)])
    col = torch.arange(W, device=old.device)[None, :]
    at = cu_pages[:-1, None] + col - held[:, None]
    fresh = torch.where(at < F, s["free"][at.clamp(0, F - 1)], -1)
    table = torch.where(col < held[:, None], s["table"][:, :W],
                        torch.where(col < need[:, None], fresh, -1))
    t = torch.arange(s["tokens"], device=old.device)
    b = torch.searchsorted(cu_tokens[1:], t, right=True)
    live = b < old.numel()
    b = b.clamp(max=old.numel() - 1)
    pos = old[b] + t - cu_tokens[b]
    page = table[b, (pos // P).clamp(0, W - 1)].long()
    slots = torch.where(live & (page >= 0), page * P + pos % P, -1)
    pos = torch.where(live, pos, 0)
    out = {"table": table, "lens": old + new, "cu_tokens": cu_tokens, "cu_pages": cu_pages,
           "slots": slots, "positions": pos}
    return {k: v.to(torch.int32) for k, v in out.items()}


def _plain_norm_rope(x, weight, rope, positions, inter):
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * weight.float()
    if rope is not None:
        rot = rope.shape[1]
        cos, sin = (c[:, None, :] for c in rope[positions.long()].chunk(2, 1))
        z = y[..., :rot]
        a, b = (z[..., 0::2], z[..., 1::2]) if inter else z.chunk(2, -1)
        p, r = a * cos - b * sin, b * cos + a * sin
        z = torch.stack([p, r], -1).flatten(-2) if inter else torch.cat([p, r], -1)
        y = torch.cat([z, y[..., rot:]], -1)
    return y.to(x.dtype)


def _plain_rope(s):
    q = _plain_norm_rope(s["q"], s["q_weight"], s["rope"], s["positions"], s["inter"])
    k = _plain_norm_rope(s["k"], s["k_weight"], s["rope"], s["positions"], s["inter"])
    if s["slots"] is None:
        return {"q": q, "k": k}
    # rows without a slot go to a spare row past the cache's end, which is dropped
    rows = s["k_cache"].shape[0] * s["k_cache"].shape[1]
    at = torch.where(s["slots"] >= 0, s["slots"].long(), rows)
    out = {"q": q}
    for name, new in (("k_cache", k), ("v_cache", s["v"])):
        c = s[name]
        flat = torch.cat([c.flatten(0, 1), c.new_zeros((1,) + c.shape[2:])])
        flat[at] = new
        out[name] = flat[:rows].view(c.shape)
    return out


def _plain_attn(s):
    q, kc, vc, table = s["q"], s["k_cache"], s["v_cache"], s["table"]
    B, Hq, D = q.shape
    P, Hkv = kc.shape[1], kc.shape[2]
    G, L = Hq // Hkv, table.shape[1] * P
    page = table.clamp(min=0).long()

    def rows(c):                  # (B, Hkv, L, D) fp32
        return c[page].view(B, L, Hkv, -1).transpose(1, 2).float().contiguous()

    pos = torch.arange(L, device=q.device)
    live = (pos[None, :] < s["lens"][:, None])[:, None, None, :]
    qt = (q.float() * s["scale"]).view(B, Hkv, G, D).transpose(2, 3).contiguous()
    score = torch.matmul(rows(kc), qt).transpose(2, 3)         # (B, Hkv, G, L)
    if s["cap"] > 0:
        score = s["cap"] * torch.tanh(score / s["cap"])
    if s["bias"] is not None:
        score = score + s["bias"][page].view(B, L, Hkv).transpose(1, 2)[:, :, None, :]
    score = torch.where(live, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(top > -math.inf, torch.exp(score - top), 0.0)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.contiguous(), rows(vc)) / total.clamp(min=1e-30)
    lse = torch.where(total > 0, top + total.log(), -math.inf)
    return {"out": out.view(B, Hq, D).to(q.dtype), "lse": lse.reshape(B, Hq)}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "tables":
        _, new, width, held, need = _table_sizes(case)
        B, T = case["B"], sum(new) + case["pad"]
        read = 2 * B + sum(need)                       # lengths, held pages, free pages
        write = B * width + B + 2 * (B + 1) + 2 * T
        return {"bytes": 4 * (read + write), "flops": 0}
    if case["op"] == "rope":
        T, Hq, Hkv, D, e = case["T"], case["Hq"], case["Hkv"], case["D"], BYTES[case["dtype"]]
        heads = Hq + (2 if case["page"] else 1) * Hkv
        small = 4 * T * (bool(case["rot"]) + bool(case["page"])) + 4 * T * case["rot"]
        per = (4 if case["norm"] else 0) * D + 3 * case["rot"]
        return {"bytes": 2 * T * heads * D * e + small, "flops": T * (Hq + Hkv) * per}
    lens = _lengths(case)
    n, B, Hq, Hkv, D, e = sum(lens), case["B"], case["Hq"], case["Hkv"], case["D"], BYTES[case["dtype"]]
    pages = sum(_ceil(x, case["page"]) for x in lens)
    b = 2 * n * Hkv * D * e + 2 * B * Hq * D * e + 4 * B * Hq + 4 * B + 4 * pages
    return {"bytes": b + (4 * n * Hkv if case["bias"] else 0), "flops": 4 * n * Hq * D}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "tables":
        return None               # whole numbers only
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope" else _exact_attn(s)


def _exact_row(x, weight, rope, positions, inter):
    """RMS norm and rotation with every pair as one complex number."""
    y = x.double()
    if weight is not None:
        y = y / (y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + EPS).sqrt() * weight.double()
    if rope is None:
        return y
    rot = rope.shape[1]
    turn = rope.double()[positions.long()]
    turn = torch.complex(turn[:, :rot // 2], turn[:, rot // 2:]).unsqueeze(1)
    y = y.clone()
    if inter:
        z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * turn
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_rope(s):
    q = _exact_row(s["q"], s["q_weight"], s["rope"], s["positions"], s["inter"])
    k = _exact_row(s["k"], s["k_weight"], s["rope"], s["positions"], s["inter"])
    if s["slots"] is None:
        return {"q": q, "k": k}
    out, keep = {"q": q}, s["slots"] >= 0
    at = s["slots"][keep].long()
    for name, new in (("k_cache", k), ("v_cache", s["v"].double())):
        c = s[name].double()
        c.view(-1, *c.shape[2:])[at] = new[keep]
        out[name] = c
    return out


def _exact_attn(s):
    """Request by request and key head by key head, over the tokens it has."""
    B, Hq, D = s["q"].shape
    P, Hkv = s["k_cache"].shape[1], s["k_cache"].shape[2]
    G = Hq // Hkv
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        page = s["table"][b, :_ceil(n, P)].long()
        for h in range(Hkv):
            k = s["k_cache"][page, :, h].reshape(-1, D)[:n].double()
            v = s["v_cache"][page, :, h].reshape(-1, D)[:n].double()
            g = slice(h * G, (h + 1) * G)
            w = torch.mm(k, s["q"][b, g].double().t().contiguous()) * s["scale"]     # (n, G)
            if s["cap"] > 0:
                w = torch.tanh(w / s["cap"]) * s["cap"]
            if s["bias"] is not None:
                w = w + s["bias"][page, :, h].reshape(-1, 1)[:n].double()
            lse[b, g] = torch.logsumexp(w, 0)
            p = torch.where(lse[b, g] > -math.inf, (w - lse[b, g]).exp(), 0.0)
            out[b, g] = torch.mm(p.t().contiguous(), v)
    return {"out": out, "lse": lse}

"""Measured cases of prompt attention and of the 8-bit paged cache.

Three paths over four calls, as a program that serves attention over a
clustered or plain paged cache makes them:

  prompt  fk_prompt_attn:   causal attention of a step's packed prompts, each
                            over all that its request holds in the cache;
  quant   fk_kv_store8 and  keys and values quantised to e4m3 as they are
          fk_kv_load8:      written, one scale per token and head, and read back;
  attn8   fk_paged_attn8:   attention of one new token per request over the
                            8-bit cache, with a per-key bias and a tanh cap.

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
E4M3 = torch.float8_e4m3fn
CHUNK = 1 << 29                    # scores that the reference forms hold at once


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a short prompt alone: launch and dependent-load latency
        _prompt("prompt_one_t128", B=1, Hq=16, Hkv=4, D=64, new=128, spread="equal", old=0,
                page=16, bias=False, cap=0.0, dtype="f16"),
        # one chunk of a long prompt: few rows over a long cache
        _prompt("prompt_chunk_t512", B=1, Hq=32, Hkv=8, D=128, new=512, spread="equal", old=32768,
                page=64, bias=False, cap=0.0, dtype="bf16"),
        # prompts of many users in one step, from none to 4096 tokens, odd head sizes
        _prompt("prompt_ragged_b16", B=16, Hq=20, Hkv=4, D=80, new=4096, spread="log", old=0,
                page=24, bias=False, cap=0.0, dtype="f16"),
        # follow-up prompts of four users over cluster centres (log counts, some empty), capped, fp32
        _prompt("prompt_clusters_f32_b4", B=4, Hq=8, Hkv=8, D=64, new=999, spread="linear",
                old=1056, page=32, bias=True, cap=30.0, dtype="f32"),
        # the largest: one whole long prompt
        _prompt("prompt_long_t32768", B=1, Hq=32, Hkv=8, D=128, new=32768, spread="equal", old=0,
                page=16, bias=False, cap=0.0, dtype="bf16"),
        # the new tokens of one decode step of 32 requests, stored and read back
        _quant("quant_decode_t32", T=32, Hkv=8, D=128, page=16, packed=True, dtype="bf16"),
        # one long prompt
        _quant("quant_prompt_t75600", T=75600, Hkv=8, D=128, page=16, packed=True, dtype="f16"),
        # odd sizes, fp32
        _quant("quant_f32_t4099", T=4099, Hkv=5, D=80, page=20, packed=False, dtype="f32"),
        # one short request alone
        _attn8("attn8_one_2048", B=1, Hq=16, Hkv=4, D=64, len=2048, spread="equal", page=16,
               bias=False, cap=0.0, dtype="f16"),
        # a compressed cache: 1000 centres with log counts and 56 recent tokens
        _attn8("attn8_clusters_b32", B=32, Hq=32, Hkv=32, D=128, len=1056, spread="equal", page=32,
               bias=True, cap=30.0, dtype="f16"),
        # one key head for 16 query heads, wide head, fp32 queries
        _attn8("attn8_mqa_f32_b4", B=4, Hq=16, Hkv=1, D=256, len=32768, spread="linear", page=48,
               bias=False, cap=0.0, dtype="f32"),
        # a batch of long requests
        _attn8("attn8_long_b32", B=32, Hq=32, Hkv=8, D=128, len=65536, spread="linear", page=16,
               bias=False, cap=0.0, dtype="bf16"),
    ]


def _prompt(name, **kw):
    return dict({"name": name, "op": "prompt"}, **kw)


def _quant(name, **kw):
    return dict({"name": name, "op": "quant"}, **kw)


def _attn8(name, **kw):
    return dict({"name": name, "op": "attn8"}, **kw)


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "quant", "attn8", "attn8"])
    dtype = rng.choice(["f32", "f16", "bf16"] if op != "prompt" else ["f32", "f16", "f16", "bf16", "bf16"])
    D = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
    Hkv = rng.choice([1, 2, 4, 5, 8, 8, 20, 32])
    if op == "quant":
        most = 75600 * 8 * 128 * 2
        T = min(_log(rng, 1, 200000), max(1, most // (Hkv * D * BYTES[dtype])))
        return {"op": op, "T": T, "Hkv": Hkv, "D": D, "page": rng.choice([1, 16, 20, 64]),
                "packed": rng.random() < 0.6, "dtype": dtype}
    G = rng.choice([1, 1, 2, 4, 4, 7, 8, 16, 32])
    page, bias = rng.choice([1, 8, 16, 20, 64, 256]), rng.random() < 0.4
    cap, spread = rng.choice([0.0, 0.0, 20.0, 50.0]), rng.choice(["equal", "log", "linear"])
    if op == "prompt":
        # scores under a quarter of the largest listed case's (fp32: a 32nd), as is their
        # product with D; keys under 2^31 bytes
        room = (32 * 32768 * 32768) // (32 if dtype == "f32" else 4)
        room = room * 128 // max(128, D)
        B, new = _log(rng, 1, 64), _log(rng, 1, 32768)
        old = rng.choice([0, _log(rng, 1, 65536)])
        B = max(1, min(B, room // (Hkv * G * new * new)))
        new = max(1, min(new, math.isqrt(room // (Hkv * G * B))))
        old = max(0, min(old, room // (Hkv * G * B * new) - new,
                         (1 << 30) // (Hkv * D * BYTES[dtype] * B) - new))
        return {"op": op, "B": B, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "new": new, "spread": spread,
                "old": old, "page": page, "bias": bias, "cap": cap, "dtype": dtype}
    B, n = _log(rng, 1, 256), _log(rng, 1, 131072)
    # elements of keys: under half of the largest such case, less with more query heads
    room = (1 << 29) * 4 // max(4, G)
    B = max(1, min(B, room // (Hkv * D * n)))
    n = max(1, min(n, room // (Hkv * D * B)))
    return {"op": op, "B": B, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "len": n, "spread": spread,
            "page": page, "bias": bias, "cap": cap, "dtype": dtype}


def _spread(n, B, spread):
    """B lengths up to n: all the same, spread evenly, or spread evenly over the
    logarithm with an empty one."""
    if spread == "equal":
        return [n] * B
    if spread == "linear":
        return [max(1, (n * (i + 1)) // B) for i in range(B)]
    ls = [int(round(n ** ((i + 1) / B))) for i in range(B)]
    if B > 1:
        ls[0] = 0
    return ls


def _prompt_lengths(case):
    """(held before, new) of every request; every third one starts from nothing."""
    B, old = case["B"], case["old"]
    new = _spread(case["new"], B, case["spread"])
    return [0 if i % 3 == 2 else old * (B - i) // B for i in range(B)], new


def _ceil(a, b):
    return -(-a // b)


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


def _order(n, seed):
    return np.random.RandomState(seed % (1 << 32)).permutation(n).tolist()


def _block_table(lens, page, g):
    """Block table of requests of these lengths, pages in random order, and their number."""
    width = max(1, _ceil(max(lens), page))
    held = [_ceil(n, page) for n in lens]
    pages = sum(held) + 1
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    held_t = torch.tensor(held, device="cuda")
    at = torch.cumsum(held_t, 0) - held_t
    col = torch.arange(width, device="cuda")
    idx = (at[:, None] + col[None, :]).clamp_(max=pages - 1)
    table = torch.where(col[None, :] < held_t[:, None], perm[idx], perm.new_tensor(-1))
    return table.contiguous(), pages


def _log_counts(g, shape):
    """Log of cluster counts, empty clusters at -inf."""
    return torch.randint(0, 150, shape, generator=g, device="cuda").to(torch.float32).log()


def prepare(case, seed):
    g = _gen(seed)
    return {"prompt": _prepare_prompt, "quant": _prepare_quant, "attn8": _prepare_attn8}[case["op"]](
        case, seed, g)


def _prepare_prompt(case, seed, g):
    Hq, Hkv, D, P, dt = (case[n] for n in ("Hq", "Hkv", "D", "page", "dtype"))
    old, new = _prompt_lengths(case)
    order = _order(case["B"], seed)
    old, new = [old[i] for i in order], [new[i] for i in order]
    lens = [a + b for a, b in zip(old, new)]
    table, pages = _block_table(lens, P, g)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return {"op": "prompt", "q": _randn(g, (cu[-1], Hq, D), dt, 3.0), "table": table,
            "k_cache": _randn(g, (pages, P, Hkv, D), dt), "v_cache": _randn(g, (pages, P, Hkv, D), dt),
            "lens": _i32(lens), "cu": _i32(cu), "scale": 1.0 / math.sqrt(D), "cap": case["cap"],
            "bias": _log_counts(g, (pages, P, Hkv)) if case["bias"] else None,
            # a server knows the lengths of its requests
            "host": list(zip(lens, new)), "max_len": max(lens)}


def _prepare_quant(case, seed, g):
    T, Hkv, D, P, dt = (case[n] for n in ("T", "Hkv", "D", "page", "dtype"))
    if case["packed"]:            # one projection's output, keys and values side by side
        kv = _randn(g, (T, 2 * Hkv, D), dt)
        k, v = kv[:, :Hkv], kv[:, Hkv:]
    else:
        k, v = _randn(g, (T, Hkv, D), dt), _randn(g, (T, Hkv, D), dt, 0.02)
    n = _ceil(T, P) + 1
    pages = torch.randperm(n, generator=g, device="cuda")
    t = torch.arange(T, device="cuda")
    slots = (pages[t // P] * P + t % P).to(torch.int32)
    if T > 8:                     # two padding tokens of the step
        slots[T - 2:] = -1
    s = {"op": "quant", "k": k, "v": v, "slots": slots}
    for name in ("k", "v"):
        s[name + "_cache"] = torch.zeros((n, P, Hkv, D), dtype=torch.uint8, device="cuda").view(E4M3)
        s[name + "_scale"] = torch.zeros((n, P, Hkv), dtype=torch.float32, device="cuda")
    return s


def _codes(g, shape):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(std=100.0, generator=g)
    return x.clamp_(-448, 448).to(E4M3)


def _prepare_attn8(case, seed, g):
    B, Hq, Hkv, D, P, dt = (case[n] for n in ("B", "Hq", "Hkv", "D", "page", "dtype"))
    lens = _spread(case["len"], B, case["spread"])
    lens = [lens[i] for i in _order(B, seed)]
    table, pages = _block_table(lens, P, g)
    s = {"op": "attn8", "q": _randn(g, (B, Hq, D), dt, 3.0), "table": table, "lens": _i32(lens),
         "scale": 1.0 / math.sqrt(D), "cap": case["cap"],
         "bias": _log_counts(g, (pages, P, Hkv)) if case["bias"] else None}
    for name in ("k", "v"):       # rows of different sizes
        s[name + "_cache"] = _codes(g, (pages, P, Hkv, D))
        e = torch.randint(-8, -5, (pages, P, Hkv), generator=g, device="cuda")
        s[name + "_scale"] = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        import exact_means_clustering_flashassign_amd as fk

        if s["op"] == "prompt":
            out, lse = fk.fk_prompt_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                         s["cu"], s["scale"], s["cap"], s["bias"],
                                         max_len=s["max_len"], return_lse=True)
            return {"out": out, "lse": lse}
        cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        if s["op"] == "quant":
            fk.fk_kv_store8(s["k"], s["v"], s["slots"], *cache)
            k, v = fk.fk_kv_load8(s["slots"], *cache, s["k"].dtype)
            return {"k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
        out, lse = fk.fk_paged_attn8(s["q"], *cache, s["table"], s["lens"], s["scale"], s["cap"],
                                     s["bias"], return_lse=True)
        return {"out": out, "lse": lse}
    return {"prompt": _plain_prompt, "quant": _plain_quant, "attn8": _plain_attn8}[s["op"]](s)


def _request_rows(c, table, b, n):
    """Rows of a request's first n tokens, (heads, n, ...)."""
    P = c.shape[1]
    page = table[b, :_ceil(n, P)].long()
    return c[page].flatten(0, 1)[:n].transpose(0, 1)


def _plain_prompt(s):
    q, cap = s["q"], s["cap"]
    T, Hq, D = q.shape
    Hkv = s["k_cache"].shape[2]
    G = Hq // Hkv
    out = torch.zeros_like(q)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float32, device=q.device)
    t = 0
    for b, (L, n) in enumerate(s["host"]):
        if n == 0:
            continue
        k = _request_rows(s["k_cache"], s["table"], b, L).float().transpose(1, 2).contiguous()
        v = _request_rows(s["v_cache"], s["table"], b, L).float().contiguous()
        key = torch.arange(L, device=q.device)
        rows = max(1, min(n, CHUNK // (Hq * L)))
        for i in range(0, n, rows):
            m = min(rows, n - i)
            x = (q[t + i:t + i + m].float() * s["scale"]).view(m, Hkv, G, D)
            x = x.permute(1, 2, 0, 3).reshape(Hkv, G * m, D)
            score = torch.matmul(x, k).view(Hkv, G, m, L)
            if cap > 0:
                score = cap * torch.tanh(score / cap)
            if s["bias"] is not None:
                score = score + _request_rows(s["bias"], s["table"], b, L)[:, None, None, :]
            at = L - n + i + torch.arange(m, device=q.device)
            score = torch.where(key[None, :] <= at[:, None], score, -math.inf)
            top = score.amax(-1, keepdim=True)
            p = torch.where(top > -math.inf, torch.exp(score - top), 0.0)
            del score
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p.view(Hkv, G * m, L), v).view(Hkv, G, m, D) / total.clamp(min=1e-30)
            out[t + i:t + i + m] = o.permute(2, 0, 1, 3).reshape(m, Hq, D).to(q.dtype)
            r = torch.where(total > 0, top + total.log(), -math.inf)
            lse[t + i:t + i + m] = r[..., 0].permute(2, 0, 1).reshape(m, Hq)
        t += n
    return {"out": out, "lse": lse}


def _plain_quant(s):
    # rows without a slot go to a spare row past the cache's end, which is dropped
    n = s["k_scale"].shape[0] * s["k_scale"].shape[1]
    slots = s["slots"].long()
    live = (slots >= 0) & (slots < n)
    at = torch.where(live, slots, n)
    out = {}
    for name in ("k", "v"):
        x, codes, scales = s[name], s[name + "_cache"].view(torch.uint8), s[name + "_scale"]
        y = x.float()
        # the smallest power of two that takes the row's largest element to 448 at most
        part, e = torch.frexp(y.abs().amax(-1))
        e = torch.where(part > 0, e - 9 + (part > 0.875).int(), 0).clamp(min=-126)
        scale = torch.ldexp(torch.ones_like(part), e)
        y = torch.ldexp(y, -e[..., None]).to(E4M3).view(torch.uint8)
        codes = torch.cat([codes.flatten(0, 1), codes.new_zeros((1,) + codes.shape[2:])])
        scales = torch.cat([scales.flatten(0, 1), scales.new_zeros((1,) + scales.shape[2:])])
        codes[at], scales[at] = y, scale
        out[name + "_scale"] = scales[:n].view(s[name + "_scale"].shape)
        back = codes[at].view(E4M3).float() * scales[at][..., None]
        most = torch.finfo(x.dtype).max
        out[name] = torch.where(live[:, None, None], back.clamp(-most, most), 0.0).to(x.dtype)
    return {k: out[k] for k in ("k", "v", "k_scale", "v_scale")}


def _plain_attn8(s):
    q, table = s["q"], s["table"]
    B, Hq, D = q.shape
    P, Hkv = s["k_cache"].shape[1], s["k_cache"].shape[2]
    G, L = Hq // Hkv, table.shape[1] * P
    page = table.clamp(min=0).long()

    def rows(name):               # (B, Hkv, L, D) fp32
        x = s[name + "_cache"].view(torch.uint8)[page].view(E4M3).float()
        x = x * s[name + "_scale"][page][..., None]
        return x.view(B, L, Hkv, -1).transpose(1, 2).contiguous()

    pos = torch.arange(L, device=q.device)
    live = (pos[None, :] < s["lens"][:, None])[:, None, None, :]
    qt = (q.float() * s["scale"]).view(B, Hkv, G, D).transpose(2, 3).contiguous()
    score = torch.matmul(rows("k"), qt).transpose(2, 3)        # (B, Hkv, G, L)
    if s["cap"] > 0:
        score = s["cap"] * torch.tanh(score / s["cap"])
    if s["bias"] is not None:
        score = score + s["bias"][page].view(B, L, Hkv).transpose(1, 2)[:, :, None, :]
    score = torch.where(live, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(top > -math.inf, torch.exp(score - top), 0.0)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.contiguous(), rows("v")) / total.clamp(min=1e-30)
    lse = torch.where(total > 0, top + total.log(), -math.inf)
    return {"out": out.view(B, Hq, D).to(q.dtype), "lse": lse.reshape(B, Hq)}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "quant":     # store: rows in, codes and scales out; load: the reverse
        rows, D, e = 2 * case["T"] * case["Hkv"], case["D"], BYTES[case["dtype"]]
        return {"bytes": 2 * rows * (D * e + D + 4) + 2 * 4 * case["T"], "flops": 3 * rows * D}
    B, Hq, Hkv, D, P = (case[n] for n in ("B", "Hq", "Hkv", "D", "page"))
    e = BYTES[case["dtype"]]
    if case["op"] == "prompt":
        old, new = _prompt_lengths(case)
        lens, tokens, held = [a + n for a, n in zip(old, new) if n], sum(new), e
        scores = sum(a * n + n * (n + 1) // 2 for a, n in zip(old, new))
    else:
        lens, tokens, held = _spread(case["len"], B, case["spread"]), B, 1
        scores = sum(lens)
    n, pages = sum(lens), sum(_ceil(x, P) for x in lens)
    b = 2 * tokens * Hq * D * e + 4 * tokens * Hq + 4 * B + 4 * pages + 2 * n * Hkv * D * held
    b += 4 * n * Hkv if case["bias"] else 0
    b += 8 * n * Hkv if case["op"] == "attn8" else 0           # scales
    return {"bytes": b, "flops": 4 * scores * Hq * D}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "quant": _exact_quant, "attn8": _exact_attn8}[case["op"]](s)


def _attend64(x, k, v, scale, cap, bias, hidden):
    """Rows x (m,D) over keys k and values v (n,D), 64 bits: softmax by way of
    its logarithm; keys where hidden (m,n or none) is true are left out."""
    w = torch.mm(x, k.t().contiguous()) * scale
    if cap > 0:
        w = torch.tanh(w / cap) * cap
    if bias is not None:
        w = w + bias[None, :]
    if hidden is not None:
        w.masked_fill_(hidden, -math.inf)
    lse = torch.logsumexp(w, 1)
    w = torch.where(lse[:, None] > -math.inf, (w - lse[:, None]).exp(), 0.0)
    return torch.mm(w, v), lse


def _exact_prompt(s):
    """Request by request and query head by query head."""
    T, Hq, D = s["q"].shape
    G = Hq // s["k_cache"].shape[2]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    t = 0
    for b, (L, n) in enumerate(s["host"]):
        rows = max(1, min(n, CHUNK // (2 * max(L, 1))))
        for h in range(Hq if n else 0):
            k, v = (_request_rows(s[c], s["table"], b, L)[h // G].double() for c in ("k_cache", "v_cache"))
            bias = None if s["bias"] is None else \
                _request_rows(s["bias"], s["table"], b, L)[h // G].double()
            for i in range(0, n, rows):
                m = min(rows, n - i)
                hidden = torch.ones((m, L), dtype=torch.bool, device="cuda").triu_(L - n + i + 1)
                at = slice(t + i, t + i + m)
                out[at, h], lse[at, h] = _attend64(s["q"][at, h].double(), k, v, s["scale"], s["cap"],
                                                   bias, hidden)
        t += n
    return {"out": out, "lse": lse}


def _exact_quant(s):
    """Codes from the definition of the numbers e4m3 holds: multiples of 2^(e-3)
    with 2^e <= |y| < 2^(e+1), of 2^-9 below 2^-6; halves go to the even one."""
    out, slots = {}, s["slots"].long()
    keep = slots >= 0
    for name in ("k", "v"):
        x = s[name].double()
        most = x.abs().amax(-1)
        scale = torch.exp2(torch.floor(torch.log2(most)) - 8)
        scale = torch.where(most > 448 * scale, 2 * scale, torch.where(most <= 224 * scale, scale / 2, scale))
        scale = torch.where(most > 0, scale.clamp(min=2.0 ** -126), 1.0)
        y = x / scale[..., None]
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        y = torch.round(y / step) * step * scale[..., None]
        top = torch.finfo(s[name].dtype).max
        out[name] = torch.where(keep[:, None, None], y.clamp(-top, top), 0.0)
        held = s[name + "_scale"].double()
        held.view(-1, held.shape[2])[slots[keep]] = scale[keep]
        out[name + "_scale"] = held
    return {k: out[k] for k in ("k", "v", "k_scale", "v_scale")}


def _exact_attn8(s):
    """Request by request and key head by key head, over the tokens it has."""
    B, Hq, D = s["q"].shape
    Hkv = s["k_cache"].shape[2]
    G = Hq // Hkv
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        for h in range(Hkv if n else 0):
            k, v = (_request_rows(s[c + "_cache"].view(torch.uint8), s["table"], b, n)[h].contiguous()
                    .view(E4M3).double() *
                    _request_rows(s[c + "_scale"], s["table"], b, n)[h].double()[:, None]
                    for c in ("k", "v"))
            bias = None if s["bias"] is None else \
                _request_rows(s["bias"], s["table"], b, n)[h].double()
            g = slice(h * G, (h + 1) * G)
            out[b, g], lse[b, g] = _attend64(s["q"][b, g].double(), k, v, s["scale"], s["cap"], bias,
                                             None)
    return {"out": out, "lse": lse}

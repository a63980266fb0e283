"""A paged key-value cache whose old tokens can be replaced by cluster centres.

The pages name KV-cache compression and attention routing as uses of fast
exact K-Means ("flash-kmeans and the return of exact K-Means on the GPU",
introduction; paixiangai.cn, section on use cases). This module runs the
library's calls together as a server of one attention layer would:

* a step places its new tokens (``fk_page_tables``), makes their queries and
  keys and stores keys and values (``fk_qk_norm_rope``), and attends: one token
  per request (``fk_paged_attn``) or whole prompts (``fk_prompt_attn``);
* ``compress`` clusters the keys of a request's older tokens, head by head
  (``fk_lloyd``), takes the mean value of each cluster with the sort-inverse
  update (``fk_update``), and keeps the centres in the tokens' place, each with
  the bias log n of the n keys it stands for. A softmax over n equal keys with
  mean value v equals one key with that bias and value v, so what is lost is
  only how far keys lie from their centres.

A quantised cache holds keys and values in 8 bits (``fk_kv_store8``): single tokens
attend to them as they are (``fk_paged_attn8``), for prompts and for clustering they are read
back (``fk_kv_load8``).
"""
from __future__ import annotations

from . import _binding as fk
from .api import batch_kmeans_Euclid


class ClusteredKVCache:
    """Keys and values of `requests` requests of one layer, in pages.

    pages, page: number of pages and tokens per page; heads, dim: key-value
    heads and elements per head; max_len: most tokens a request may hold.
    Compressed requests hold fewer tokens than they have seen: `lens` counts
    what is held, `centres` how many of those are cluster centres (they come
    first), `seen` the tokens there were, which gives the next one's position. Lists of lengths are host integers: a server knows them.
    quantised: keys and values are held as e4m3 codes with a scale per token and head; dtype is
    then the type they come in and are read back in."""

    def __init__(self, requests: int, pages: int, page: int, heads: int, dim: int, max_len: int,
                 dtype, device="cuda:0", quantised: bool = False):
        torch = fk._torch()
        if min(requests, pages, page, heads, dim, max_len) < 1:
            raise ValueError("every size must be at least 1")
        i32 = dict(dtype=torch.int32, device=device)
        self.page, self.max_len, self.width = page, max_len, -(-max_len // page)
        self.dtype, self.quantised = dtype, quantised
        held = torch.uint8 if quantised else dtype
        self.k = torch.zeros((pages, page, heads, dim), dtype=held, device=device)
        self.v = torch.zeros_like(self.k)
        self.key_bias = torch.zeros((pages, page, heads), dtype=torch.float32, device=device)
        if quantised:
            fk.dtype_code(dtype)                       # says what is supported
            self.k, self.v = (c.view(torch.float8_e4m3fn) for c in (self.k, self.v))
            self.k_scale, self.v_scale = torch.zeros_like(self.key_bias), torch.zeros_like(self.key_bias)
        self.table = torch.full((requests, self.width), -1, **i32)
        self.lens_dev = torch.zeros(requests, **i32)
        self.shift = torch.zeros(requests, **i32)      # position minus place in the cache
        self.free = torch.arange(pages, **i32)         # pages not in use
        self.lens, self.seen, self.centres = ([0] * requests for _ in range(3))
        self.cu_tokens, self.new = None, []            # of the last step

    def _pages(self, n: int) -> int:
        return -(-n // self.page)

    def append(self, q, k, v, new, q_weight=None, k_weight=None, eps: float = 1e-6, rope=None,
               interleaved: bool = False):
        """Store a step's tokens: new[b] tokens of request b, in order of requests, as
        q (T,Hq,D), k and v (T,Hkv,D). Returns the normed and rotated queries. Positions
        count all tokens a request has seen, and have to be inside rope's rows."""
        torch = fk._torch()
        T = int(q.shape[0])
        if len(new) != len(self.lens) or min(new) < 0 or sum(new) != T:
            raise ValueError(f"new must hold {len(self.lens)} lengths that sum to {T}")
        lens = [a + n for a, n in zip(self.lens, new)]
        if max(lens) > self.max_len:
            raise ValueError(f"a request would hold {max(lens)} tokens, more than {self.max_len}")
        most = max((s + n for s, n in zip(self.seen, new) if n), default=0)
        if rope is not None and most > rope.shape[0]:
            raise ValueError(f"a request would have {most} positions, more than rope's {rope.shape[0]}")
        taken = sum(self._pages(b) - self._pages(a) for a, b in zip(self.lens, lens))
        if taken > self.free.numel():
            raise RuntimeError(f"{taken} pages needed, {self.free.numel()} free")
        n = torch.tensor(new, dtype=torch.int32).to(self.k.device)
        table, lens_dev, cu_tokens, _, slots, pos = fk.fk_page_tables(
            self.lens_dev, n, self.free, self.page, self.width, T, table=self.table)
        if rope is not None:
            pos = pos + torch.repeat_interleave(self.shift, n, output_size=T)
        if self.quantised:
            if q.dtype != self.dtype or v.dtype != self.dtype:
                raise ValueError(f"queries, keys and values must be {self.dtype}")
            out, k = fk.fk_qk_norm_rope(q, k, None, q_weight, k_weight, eps, rope, pos, interleaved)
            fk.fk_kv_store8(k, v, slots, self.k, self.v, self.k_scale, self.v_scale, self.key_bias)
        else:
            out, _ = fk.fk_qk_norm_rope(q, k, v, q_weight, k_weight, eps, rope, pos, interleaved,
                                        slots, self.k, self.v, self.key_bias)
        # only now: a refused call leaves the cache as it was
        self.table, self.lens_dev, self.free = table, lens_dev, self.free[taken:]
        self.lens, self.cu_tokens, self.new = lens, cu_tokens, list(new)
        self.seen = [a + b for a, b in zip(self.seen, new)]
        return out

    def attend(self, q, scale=None, softcap: float = 0.0, return_lse: bool = False):
        """Attention of one token per request, q (B,Hq,D), over everything held."""
        if self.quantised:
            return fk.fk_paged_attn8(q, self.k, self.v, self.k_scale, self.v_scale, self.table, self.lens_dev,
                                     scale, softcap, self.key_bias, max(max(self.lens), 1),
                                     return_lse=return_lse)
        return fk.fk_paged_attn(q, self.k, self.v, self.table, self.lens_dev, scale, softcap,
                                self.key_bias, max(max(self.lens), 1), return_lse=return_lse)

    def attend_prompts(self, q, scale=None, softcap: float = 0.0, return_lse: bool = False):
        """Attention of the last step's tokens, q (T,Hq,D) as `append` returned them, each over
        what its request holds up to and with itself. Nothing may have been compressed or
        released since."""
        torch = fk._torch()
        if self.cu_tokens is None:
            raise ValueError("no step since the last change of the cache")
        if q.shape[0] != sum(self.new):
            raise ValueError(f"the last step had {sum(self.new)} tokens, got {q.shape[0]}")
        k, v, bias, table = self.k, self.v, self.key_bias, self.table
        if self.quantised:                             # what the step's requests hold, read back
            rows = [self._pages(n) if new else 0 for n, new in zip(self.lens, self.new)]
            pages = torch.cat([table[b, :n] for b, n in enumerate(rows)])
            k, v = self._read(pages)
            bias = bias[pages.long()]
            number = torch.full_like(table, -1)
            at = 0
            for b, n in enumerate(rows):
                number[b, :n] = torch.arange(at, at + n, dtype=torch.int32, device=table.device)
                at += n
            table = number
        return fk.fk_prompt_attn(q, k, v, table, self.lens_dev, self.cu_tokens, scale, softcap, bias,
                                 max(max(self.lens), 1), return_lse=return_lse)

    def _read(self, pages):
        """Keys and values of pages of a quantised cache, as a cache of those pages."""
        torch = fk._torch()
        tok = torch.arange(self.page, dtype=torch.int32, device=pages.device)
        slots = (pages[:, None] * self.page + tok).flatten()
        return tuple(t.view(-1, self.page, *t.shape[1:]) for t in
                     fk.fk_kv_load8(slots, self.k, self.v, self.k_scale, self.v_scale, self.dtype))

    def compress(self, request: int, n_clusters: int, keep: int = 0, niter: int = 10,
                 init=None, seed: int = 0) -> int:
        """Replace a request's tokens, but for the last `keep`, by n_clusters
        centres per head; the pages that frees go back to the list. Centres of an earlier
        call stay as they are, in front. init: (heads, n_clusters, dim) starting centres.
        Returns the tokens the request now holds."""
        torch = fk._torch()
        n, c0 = self.lens[request], self.centres[request]
        old = n - int(keep)
        if keep < 0 or n_clusters < 1 or old - c0 < n_clusters:
            raise ValueError(f"cannot make {n_clusters} clusters of {max(old - c0, 0)} tokens")
        held = c0 + n_clusters + keep
        rows = self.table[request, :self._pages(n)].long()
        heads, dim = self.k.shape[2:]
        held_k, held_v = self._read(rows.int()) if self.quantised else (self.k[rows], self.v[rows])

        def tokens(c, first, last):                    # (heads, last - first, ...) in order
            return c.flatten(0, 1)[first:last].transpose(0, 1).contiguous()

        keys, values = tokens(held_k, c0, old), tokens(held_v, c0, old)
        _, centers, _ = batch_kmeans_Euclid(keys, n_clusters, 0.0, False, niter, init, seed)
        # one more assignment: keys, counts and mean values of the same clusters
        c_lp, cnorm = fk.fk_norms(centers, keys.dtype)
        means = torch.zeros((heads, n_clusters, dim), dtype=torch.float32, device=keys.device)
        _, counts, _ = fk.fk_update(values, fk.fk_assign(keys, c_lp, cnorm), means)
        new_k = torch.cat([c_lp, tokens(held_k, old, n)], 1)
        new_v = torch.cat([means.to(values.dtype), tokens(held_v, old, n)], 1)
        bias = torch.cat([counts.float().log(), tokens(self.key_bias[rows], old, n)], 1)
        at = torch.arange(c0, held, device=keys.device)
        page, tok = rows[at // self.page], at % self.page
        if self.quantised:                             # (what was read back is stored without a loss)
            fk.fk_kv_store8(new_k.transpose(0, 1).contiguous(), new_v.transpose(0, 1).contiguous(),
                            (page * self.page + tok).int(), self.k, self.v, self.k_scale, self.v_scale)
        else:
            self.k[page, tok], self.v[page, tok] = new_k.transpose(0, 1), new_v.transpose(0, 1)
        self.key_bias[page, tok] = bias.transpose(0, 1)
        self.free = torch.cat([self.free, rows[self._pages(held):].to(torch.int32)])
        self.table[request, self._pages(held):] = -1
        self.lens_dev[request] = held
        self.shift[request] = self.seen[request] - held
        self.lens[request], self.centres[request] = held, c0 + n_clusters
        self.cu_tokens = None
        return held

    def release(self, request: int) -> None:
        """End a request: its pages go back to the list, and its row is empty for another."""
        torch = fk._torch()
        self.free = torch.cat([self.free, self.table[request, :self._pages(self.lens[request])]])
        self.table[request] = -1
        self.lens_dev[request] = self.shift[request] = 0
        self.lens[request] = self.seen[request] = self.centres[request] = 0
        self.cu_tokens = None

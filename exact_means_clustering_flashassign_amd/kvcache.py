"""A paged key-value cache whose old tokens can be replaced by cluster centres.

The pages name KV-cache compression and attention routing as uses of fast
exact K-Means ("flash-kmeans and the return of exact K-Means on the GPU",
introduction; paixiangai.cn, section on use cases). This module runs the
library's calls together as a server of one attention layer would:

* a step places its new tokens (``fk_page_tables``), makes their queries and
  keys and stores keys and values (``fk_qk_norm_rope``), and attends
  (``fk_paged_attn``);
* ``compress`` clusters the keys of a request's older tokens, head by head
  (``fk_lloyd``), takes the mean value of each cluster with the sort-inverse
  update (``fk_update``), and keeps the centres in the tokens' place, each with
  the bias log n of the n keys it stands for. A softmax over n equal keys with
  mean value v equals one key with that bias and value v, so what is lost is
  only how far keys lie from their centres.
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
    first), `seen` the tokens there were, which gives the next one's position. Lists of lengths are host integers: a server knows them."""

    def __init__(self, requests: int, pages: int, page: int, heads: int, dim: int, max_len: int,
                 dtype, device="cuda:0"):
        torch = fk._torch()
        if min(requests, pages, page, heads, dim, max_len) < 1:
            raise ValueError("every size must be at least 1")
        i32 = dict(dtype=torch.int32, device=device)
        self.page, self.max_len, self.width = page, max_len, -(-max_len // page)
        self.k = torch.zeros((pages, page, heads, dim), dtype=dtype, device=device)
        self.v = torch.zeros_like(self.k)
        self.key_bias = torch.zeros((pages, page, heads), dtype=torch.float32, device=device)
        self.table = torch.full((requests, self.width), -1, **i32)
        self.lens_dev = torch.zeros(requests, **i32)
        self.shift = torch.zeros(requests, **i32)      # position minus place in the cache
        self.free = torch.arange(pages, **i32)         # pages not in use
        self.lens, self.seen, self.centres = ([0] * requests for _ in range(3))

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
        table, lens_dev, _, _, slots, pos = fk.fk_page_tables(
            self.lens_dev, n, self.free, self.page, self.width, T, table=self.table)
        if rope is not None:
            pos = pos + torch.repeat_interleave(self.shift, n, output_size=T)
        out, _ = fk.fk_qk_norm_rope(q, k, v, q_weight, k_weight, eps, rope, pos, interleaved,
                                    slots, self.k, self.v, self.key_bias)
        # only now: a refused call leaves the cache as it was
        self.table, self.lens_dev, self.free = table, lens_dev, self.free[taken:]
        self.lens = lens
        self.seen = [a + b for a, b in zip(self.seen, new)]
        return out

    def attend(self, q, scale=None, softcap: float = 0.0, return_lse: bool = False):
        """Attention of one token per request, q (B,Hq,D), over everything held."""
        return fk.fk_paged_attn(q, self.k, self.v, self.table, self.lens_dev, scale, softcap,
                                self.key_bias, max(max(self.lens), 1), return_lse=return_lse)

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

        def tokens(c, first, last):                    # (heads, last - first, ...) in order
            return c[rows].flatten(0, 1)[first:last].transpose(0, 1).contiguous()

        keys, values = tokens(self.k, c0, old), tokens(self.v, c0, old)
        _, centers, _ = batch_kmeans_Euclid(keys, n_clusters, 0.0, False, niter, init, seed)
        # one more assignment: keys, counts and mean values of the same clusters
        c_lp, cnorm = fk.fk_norms(centers, keys.dtype)
        means = torch.zeros((heads, n_clusters, dim), dtype=torch.float32, device=keys.device)
        _, counts, _ = fk.fk_update(values, fk.fk_assign(keys, c_lp, cnorm), means)
        new_k = torch.cat([c_lp, tokens(self.k, old, n)], 1)
        new_v = torch.cat([means.to(values.dtype), tokens(self.v, old, n)], 1)
        bias = torch.cat([counts.float().log(), tokens(self.key_bias, old, n)], 1)
        at = torch.arange(c0, held, device=keys.device)
        page, tok = rows[at // self.page], at % self.page
        self.k[page, tok], self.v[page, tok] = new_k.transpose(0, 1), new_v.transpose(0, 1)
        self.key_bias[page, tok] = bias.transpose(0, 1)
        self.free = torch.cat([self.free, rows[self._pages(held):].to(torch.int32)])
        self.table[request, self._pages(held):] = -1
        self.lens_dev[request] = held
        self.shift[request] = self.seen[request] - held
        self.lens[request], self.centres[request] = held, c0 + n_clusters
        return held

    def release(self, request: int) -> None:
        """End a request: its pages go back to the list, and its row is empty for another."""
        torch = fk._torch()
        self.free = torch.cat([self.free, self.table[request, :self._pages(self.lens[request])]])
        self.table[request] = -1
        self.lens_dev[request] = self.shift[request] = 0
        self.lens[request] = self.seen[request] = self.centres[request] = 0

"""ctypes binding over libfkmeans.so: argument marshalling only.

Every function has the name of the C entry point it calls. Tensors are
PyTorch tensors on the current HIP device; work is enqueued on torch's
current stream. Nothing here computes: a missing or broken library raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import Optional, Tuple

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfkmeans.so")

FK_F32, FK_F16, FK_BF16 = 0, 1, 2
FK_OK = 0
STATUS = {0: "FK_OK", 1: "FK_ERR_INVALID", 2: "FK_ERR_UNSUPPORTED", 3: "FK_ERR_WORKSPACE",
          4: "FK_ERR_HIP"}

_lib = None


class FKError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {fk_status_string(status)}")


class fk_trace_t(ctypes.Structure):
    _fields_ = [("iterations", ctypes.c_int32), ("norms_ms", ctypes.c_double),
                ("assign_ms", ctypes.c_double), ("update_ms", ctypes.c_double)]


class fk_kv_cache_t(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("key_bias", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("page", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("k_stride", ctypes.c_int64 * 3),
                ("v_stride", ctypes.c_int64 * 3), ("bias_stride", ctypes.c_int64 * 3)]


def load(path: Optional[str] = None):
    """Load libfkmeans.so (once) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first "
                           "(python -m exact_means_clustering_flashassign_amd.build)")
    lib = ctypes.CDLL(path)
    P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    sig = {
        "fk_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "fk_version": (I32, []),
        "fk_workspace_size": (SZ, [ctypes.c_int, I64, I64, I64, I64]),
        "fk_norms": (ctypes.c_int, [P, P, P, ctypes.c_int, I64, I64, I64, P]),
        "fk_assign": (ctypes.c_int, [P, P, P, ctypes.c_int, I64, I64, I64, I64, P, P]),
        "fk_update": (ctypes.c_int, [P, P, ctypes.c_int, I64, I64, I64, I64, P, P, P, P, SZ, P]),
        "fk_update_noalloc": (ctypes.c_int, [P, P, ctypes.c_int, I64, I64, I64, I64, P, P, P, P]),
        "fk_update_partial": (ctypes.c_int, [P, P, ctypes.c_int, I64, I64, I64, I64, P, P, P, SZ,
                                             P]),
        "fk_lloyd": (ctypes.c_int, [P, ctypes.c_int, I64, I64, I64, I64, P, I32, ctypes.c_float,
                                    P, P, ctypes.POINTER(I32), P, SZ, P]),
        "fk_workspace_size_host": (SZ, [ctypes.c_int, I64, I64, I64, I64]),
        "fk_lloyd_host": (ctypes.c_int, [P, ctypes.c_int, I64, I64, I64, I64, P, I32,
                                         ctypes.c_float, I64, P, P, ctypes.POINTER(I32), P, SZ,
                                         P]),
        "fk_page_tables": (ctypes.c_int, [P, P, P, I64, P, I64, I64, I64, I64, I64, P, P, P, P, P,
                                          P, P]),
        "fk_qk_norm_rope": (ctypes.c_int, [P, P, P, P, P, P, ctypes.c_int, I64, I64, I64, I64, P,
                                           P, ctypes.c_float, P, I64, I64, I32, P, P, P, P, P,
                                           P]),
        "fk_paged_attn": (ctypes.c_int, [P, P, ctypes.c_int, I64, I64, P, P, I64, I64, P, I64,
                                         ctypes.c_float, ctypes.c_float, P, P, P, SZ, P]),
        "fk_workspace_size_attn": (SZ, [ctypes.c_int, I64, I64, I64, I64]),
        "fk_trace_begin": (ctypes.c_int, [I32]),
        "fk_trace_end": (ctypes.c_int, [ctypes.POINTER(fk_trace_t)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    _lib = lib
    return lib


def fk_status_string(status: int) -> str:
    return load().fk_status_string(int(status)).decode()


def fk_version() -> int:
    return int(load().fk_version())


# ---------------------------------------------------------------------------
# tensor helpers
# ---------------------------------------------------------------------------
def _torch():
    import torch
    return torch


def dtype_code(dtype) -> int:
    torch = _torch()
    codes = {torch.float32: FK_F32, torch.float16: FK_F16, torch.bfloat16: FK_BF16}
    if dtype not in codes:
        raise ValueError(f"unsupported element type {dtype}; use float32, float16 or bfloat16")
    return codes[dtype]


def torch_dtype(code: int):
    torch = _torch()
    return {FK_F32: torch.float32, FK_F16: torch.float16, FK_BF16: torch.bfloat16}[code]


def _dev(t, name, dtype=None, shape=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(t):
    return ctypes.c_void_p(_torch().cuda.current_stream(t.device).cuda_stream)


def _check(st: int, where: str):
    if st != FK_OK:
        raise FKError(st, where)


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------
def fk_workspace_size(dtype, B: int, N: int, d: int, K: int) -> int:
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    return int(load().fk_workspace_size(code, B, N, d, K))


def workspace(dtype, B: int, N: int, d: int, K: int, device):
    """A device workspace tensor of fk_workspace_size bytes (256-byte aligned)."""
    torch = _torch()
    n = fk_workspace_size(dtype, B, N, d, K)
    if n == 0:
        raise ValueError("invalid problem size")
    ws = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + n]


def fk_norms(c, dtype, c_lp=None, cnorm=None) -> Tuple[object, object]:
    """c (B,K,d) fp32 -> (c_lp (B,K,d) dtype, cnorm (B,K) fp32)."""
    torch = _torch()
    code = dtype_code(dtype)
    B, K, d = c.shape
    if c_lp is None:
        c_lp = torch.empty((B, K, d), dtype=dtype, device=c.device)
    if cnorm is None:
        cnorm = torch.empty((B, K), dtype=torch.float32, device=c.device)
    st = load().fk_norms(_dev(c, "c", torch.float32), _dev(c_lp, "c_lp", dtype, (B, K, d)),
                         _dev(cnorm, "cnorm", torch.float32, (B, K)), code, B, K, d, _stream(c))
    _check(st, "fk_norms")
    return c_lp, cnorm


def fk_assign(x, c_lp, cnorm, ids=None):
    """x (B,N,d), c_lp (B,K,d) same dtype, cnorm (B,K) fp32 -> ids (B,N) int32."""
    torch = _torch()
    code = dtype_code(x.dtype)
    B, N, d = x.shape
    K = c_lp.shape[1]
    if ids is None:
        ids = torch.empty((B, N), dtype=torch.int32, device=x.device)
    st = load().fk_assign(_dev(x, "x"), _dev(c_lp, "c_lp", x.dtype, (B, K, d)),
                          _dev(cnorm, "cnorm", torch.float32, (B, K)), code, B, N, d, K,
                          _dev(ids, "ids", torch.int32, (B, N)), _stream(x))
    _check(st, "fk_assign")
    return ids


def fk_update(x, ids, c, counts=None, shift=None, ws=None):
    """In-place centroid update of c (B,K,d) fp32; returns (c, counts, shift)."""
    torch = _torch()
    code = dtype_code(x.dtype)
    B, N, d = x.shape
    K = c.shape[1]
    if counts is None:
        counts = torch.empty((B, K), dtype=torch.int32, device=x.device)
    if shift is None:
        shift = torch.empty((B,), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(x.dtype, B, N, d, K, x.device)
    st = load().fk_update(_dev(x, "x"), _dev(ids, "ids", torch.int32, (B, N)), code, B, N, d, K,
                          _dev(c, "c", torch.float32, (B, K, d)),
                          _dev(counts, "counts", torch.int32, (B, K)),
                          _dev(shift, "shift", torch.float32, (B,)), _dev(ws, "ws", torch.uint8),
                          ws.numel(), _stream(x))
    _check(st, "fk_update")
    return c, counts, shift


FK_NOALLOC_SCRATCH_BYTES = 64 << 20


def fk_update_noalloc(x, ids, c, counts, shift):
    """fk_update with the library's own device scratch (no workspace); the
    caller passes every output. In-place update of c; returns (c, counts, shift)."""
    torch = _torch()
    code = dtype_code(x.dtype)
    B, N, d = x.shape
    K = c.shape[1]
    st = load().fk_update_noalloc(_dev(x, "x"), _dev(ids, "ids", torch.int32, (B, N)), code, B,
                                  N, d, K, _dev(c, "c", torch.float32, (B, K, d)),
                                  _dev(counts, "counts", torch.int32, (B, K)),
                                  _dev(shift, "shift", torch.float32, (B,)), _stream(x))
    _check(st, "fk_update_noalloc")
    return c, counts, shift


def fk_update_partial(x, ids, sums, counts, ws=None):
    """Add this block of points' per-cluster sums (B,K,d) fp32 and counts
    (B,K) int32 into sums and counts (one shard's part of an update)."""
    torch = _torch()
    code = dtype_code(x.dtype)
    B, N, d = x.shape
    K = sums.shape[1]
    if ws is None:
        ws = workspace(x.dtype, B, N, d, K, x.device)
    st = load().fk_update_partial(_dev(x, "x"), _dev(ids, "ids", torch.int32, (B, N)), code, B,
                                  N, d, K, _dev(sums, "sums", torch.float32, (B, K, d)),
                                  _dev(counts, "counts", torch.int32, (B, K)),
                                  _dev(ws, "ws", torch.uint8), ws.numel(), _stream(x))
    _check(st, "fk_update_partial")
    return sums, counts


def fk_lloyd(x, init, max_iter: int, tol: float, ids=None, centers=None, ws=None):
    """Lloyd's loop from init (B,K,d) in x's dtype -> (ids, centers fp32, n_iter).
    init=None resumes from the fp32 centres in `centers` (updated in place)."""
    torch = _torch()
    code = dtype_code(x.dtype)
    B, N, d = x.shape
    if init is None and centers is None:
        raise ValueError("resuming (init=None) needs the fp32 centers to start from")
    K = (init if init is not None else centers).shape[1]
    if ids is None:
        ids = torch.empty((B, N), dtype=torch.int32, device=x.device)
    if centers is None:
        centers = torch.empty((B, K, d), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(x.dtype, B, N, d, K, x.device)
    n_iter = ctypes.c_int32(0)
    ip = None if init is None else _dev(init, "init", x.dtype, (B, K, d))
    st = load().fk_lloyd(_dev(x, "x"), code, B, N, d, K, ip,
                         int(max_iter), float(tol), _dev(ids, "ids", torch.int32, (B, N)),
                         _dev(centers, "centers", torch.float32, (B, K, d)),
                         ctypes.byref(n_iter), _dev(ws, "ws", torch.uint8), ws.numel(),
                         _stream(x))
    _check(st, "fk_lloyd")
    return ids, centers, int(n_iter.value)


def fk_workspace_size_host(dtype, B: int, chunk: int, d: int, K: int) -> int:
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    return int(load().fk_workspace_size_host(code, B, chunk, d, K))


def fk_lloyd_host(x_host, init, max_iter: int, tol: float, chunk: int, ids=None, centers=None,
                  ws=None):
    """Lloyd's loop over points in host memory, streamed in chunks of `chunk`
    points per problem -> (ids, centers fp32, n_iter). x_host: a contiguous
    CPU tensor (B,N,d), best page-locked (pin_memory); init (B,K,d) on the GPU,
    or None to resume from the fp32 centres in `centers`."""
    torch = _torch()
    if not isinstance(x_host, torch.Tensor) or x_host.device.type != "cpu":
        raise ValueError("x_host must be a CPU tensor")
    if not x_host.is_contiguous() or x_host.dim() != 3:
        raise ValueError("x_host must be a contiguous (B, N, d) tensor")
    if init is None and centers is None:
        raise ValueError("resuming (init=None) needs the fp32 centers to start from")
    code = dtype_code(x_host.dtype)
    B, N, d = x_host.shape
    start = init if init is not None else centers
    K = start.shape[1]
    dev = start.device
    if ids is None:
        ids = torch.empty((B, N), dtype=torch.int32, device=dev)
    if centers is None:
        centers = torch.empty((B, K, d), dtype=torch.float32, device=dev)
    if ws is None:
        n = fk_workspace_size_host(code, B, chunk, d, K)
        if n == 0:
            raise ValueError("invalid problem size or chunk")
        raw = torch.empty(n + 256, dtype=torch.uint8, device=dev)
        off = (-raw.data_ptr()) % 256
        ws = raw[off:off + n]
    n_iter = ctypes.c_int32(0)
    st = load().fk_lloyd_host(x_host.data_ptr(), code, B, N, d, K,
                              None if init is None else _dev(init, "init", x_host.dtype,
                                                             (B, K, d)), int(max_iter),
                              float(tol), int(chunk), _dev(ids, "ids", torch.int32, (B, N)),
                              _dev(centers, "centers", torch.float32, (B, K, d)),
                              ctypes.byref(n_iter), _dev(ws, "ws", torch.uint8), ws.numel(),
                              _stream(start))
    _check(st, "fk_lloyd_host")
    return ids, centers, int(n_iter.value)


# ---------------------------------------------------------------------------
# paged key-value cache
# These run once per layer and generated token, where a few microseconds of
# argument handling show: attributes are read once, structures and strides are
# packed as bytes, and the words of an error are only made when there is one.
# ---------------------------------------------------------------------------
_pack2 = struct.Struct("2q").pack
_pack_cache = struct.Struct("3P4q9q").pack      # the layout of fk_kv_cache_t


_tc = None


class _TorchCalls:
    """What the calls below need of torch, looked up once."""

    def __init__(self):
        torch = _torch()
        self.empty, self.empty_like = torch.empty, torch.empty_like
        self.i32, self.f32, self.u8 = torch.int32, torch.float32, torch.uint8
        self.codes = {torch.float32: FK_F32, torch.float16: FK_F16, torch.bfloat16: FK_BF16}
        self.stream = torch._C._cuda_getCurrentRawStream
        self.grad = torch.is_grad_enabled


def _calls():
    global _tc
    if _tc is None:
        load()
        _tc = _TorchCalls()
    return _tc


def _gpu_index(t, name) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a device tensor")
    return index


def _on(t, name, dtype, shape, index):
    """Checks of a contiguous tensor on device `index`; its address."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or \
            not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"cuda:{index}, got {t.dtype} {tuple(t.shape)} strides {t.stride()} on "
                         f"{t.device}")
    return t.data_ptr()


def _rows(t, name, dtype, dims, index):
    """Checks of a tensor with contiguous rows, for the forward-only calls; its strides."""
    s = t.stride()
    if len(s) != dims or t.dtype is not dtype or t.get_device() != index or t.requires_grad or \
            (s[-1] != 1 and t.shape[-1] > 1):
        if t.requires_grad:
            raise ValueError(f"{name} requires grad: the call has no backward pass, detach it first")
        raise ValueError(f"{name} must be a {dims}-dimensional {dtype} tensor with contiguous rows "
                         f"on cuda:{index}, got {t.dtype} {tuple(t.shape)} strides {s} on "
                         f"{t.device}")
    return s


def _apart(outs, ins):
    """Refuses outputs (name, address, end) that overlap one another or an input (name, address,
    end of its extent, and the tensor where that may have gaps)."""
    for i, (name, lo, hi) in enumerate(outs):
        for other, a, b in outs[:i]:
            if max(lo, a) < min(hi, b):
                raise ValueError(f"{name} overlaps {other}")
        for other, a, b, *t in ins:
            if max(lo, a) < min(hi, b) and (not t or _meets(lo - a, hi - a, t[0])):
                raise ValueError(f"{name} overlaps {other}, which the call reads")


def _span(name, t, stride, size):
    """An input for _apart with its extent; its gaps are looked into where that is met."""
    p = t.data_ptr()
    if not t.numel():
        return name, p, p
    return name, p, p + (sum((n - 1) * s for n, s in zip(t.shape, stride)) + 1) * size, t


def _meets(lo, hi, t):
    """Whether bytes lo to hi from a tensor's address hold any of its elements."""
    size = t.element_size()

    def within(lo, hi, axes, extent):
        if not axes:
            return lo < size and hi > 0
        (s, n), *rest = axes
        extent -= (n - 1) * s                    # of one index
        first = max(0, (lo - extent) // s + 1) if s else 0
        last = min(n - 1, (hi - 1) // s) if s else 0
        # three indices in a row: the middle one lies between lo and hi whole
        return last - first >= 2 or any(within(lo - i * s, hi - i * s, rest, extent)
                                        for i in range(first, last + 1))

    axes = sorted(((s * size, n) for s, n in zip(t.stride(), t.shape) if n > 1), reverse=True)
    return lo < hi and within(lo, hi, axes, sum((n - 1) * s for s, n in axes) + size)


def _no_grad(t, name):
    """Parameters may be given where no gradient is asked for; else it would be lost."""
    if t.requires_grad and _tc.grad():
        raise ValueError(f"{name} requires grad: the call has no backward pass, detach it or use "
                         f"torch.no_grad()")


def _kv_cache(k_cache, v_cache, key_bias, dtype, heads, dim, index):
    """fk_kv_cache_t (as bytes) of (pages, page, heads, dim) tensors in any axis order of
    memory, and its number of heads."""
    sk = _rows(k_cache, "k_cache", dtype, 4, index)
    sv = _rows(v_cache, "v_cache", dtype, 4, index)
    shape = k_cache.shape
    if v_cache.shape != shape or shape[3] != dim or (heads and shape[2] != heads):
        raise ValueError(f"k_cache and v_cache must have shape (pages, page, {heads or 'heads'}, "
                         f"{dim}), got {tuple(shape)} and {tuple(v_cache.shape)}")
    bp, sb = None, (0, 0, 0)
    if key_bias is not None:
        sb = key_bias.stride()
        if key_bias.shape != shape[:3] or key_bias.dtype is not _calls().f32 or \
                key_bias.get_device() != index or key_bias.requires_grad:
            raise ValueError(f"key_bias must be float32 of shape {tuple(shape[:3])} on "
                             f"cuda:{index} without grad, got {key_bias.dtype} "
                             f"{tuple(key_bias.shape)} on {key_bias.device}")
        bp = key_bias.data_ptr()
    return _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), bp or 0, *shape, *sk[:3], *sv[:3],
                       *sb), shape[2]


def fk_page_tables(len_old, len_new, free_pages, page: int, width: int, tokens: int, table=None,
                   out=None):
    """Block tables and slots of a step: requests of len_old (B) tokens get
    len_new (B) more, pages taken from free_pages (F) in order; table (B,W)
    holds the pages they have (None: none). All int32 on the GPU. Returns
    (table (B,width), lens (B), cu_tokens (B+1), cu_pages (B+1), slots (tokens),
    positions (tokens)), views of one buffer; `out`: those six tensors, to
    write into: the first may be `table` itself, else none may overlap
    another or an input."""
    tc = _tc or _calls()
    i32, index = tc.i32, _gpu_index(len_old, "len_old")
    B = len_old.numel()
    p_old = _on(len_old, "len_old", i32, (B,), index)
    p_new = _on(len_new, "len_new", i32, (B,), index)
    n_free = free_pages.numel()
    p_free = _on(free_pages, "free_pages", i32, (n_free,), index)
    p_in, width_in = None, 0
    if table is not None:
        width_in = table.shape[-1]
        p_in = _on(table, "table", i32, (B, width_in), index)
    if out is None:
        if width < 1 or tokens < 0:
            raise ValueError("width must be at least 1 and tokens non-negative")
        n = B * width
        buf = tc.empty(n + 3 * B + 2 + 2 * tokens, dtype=i32, device=len_old.device)
        rows, *rest = buf.split_with_sizes((n, B, B + 1, B + 1, tokens, tokens))
        out = (rows.view(B, width), *rest)
        p = buf.data_ptr()
        n, B4, T4 = 4 * n, 4 * B, 4 * tokens
        ps = (p, p + n, p + n + B4, p + n + 2 * B4 + 4, p + n + 3 * B4 + 8, p + n + 3 * B4 + 8 + T4)
    else:
        if len(out) != 6:
            raise ValueError("out must hold table, lens, cu_tokens, cu_pages, slots, positions")
        shapes = ((B, width), (B,), (B + 1,), (B + 1,), (tokens,), (tokens,))
        ps = [_on(t, f"out[{i}]", i32, s, index) for i, (t, s) in enumerate(zip(out, shapes))]
        out = tuple(out)
        ins = [("len_old", p_old, p_old + 4 * B), ("len_new", p_new, p_new + 4 * B),
               ("free_pages", p_free, p_free + 4 * n_free)]
        if p_in is not None and (p_in != ps[0] or width_in != width):
            ins.append(("table", p_in, p_in + 4 * B * width_in))
        _apart([(f"out[{i}]", p, p + 4 * t.numel()) for i, (p, t) in enumerate(zip(ps, out))
                if t.numel()], ins)
    st = _lib.fk_page_tables(p_old, p_new, p_in, width_in, p_free, n_free, B, page, width, tokens,
                             *ps, tc.stream(index))
    if st:
        _check(st, "fk_page_tables")
    return out


def fk_qk_norm_rope(q, k, v=None, q_weight=None, k_weight=None, eps: float = 1e-6, rope=None,
                    positions=None, interleaved: bool = False, slots=None, k_cache=None,
                    v_cache=None, key_bias=None, q_out=None, k_out=None):
    """q (T,Hq,D), k and v (T,Hkv,D): per-head RMS norm with the weights (D)
    (none: no norm) and rotation of the first rot elements by rope (max_pos,
    rot) fp32, cosines then sines, at positions (T) int32 (none: no rotation).
    Weights and rope that require grad are taken under torch.no_grad() only.
    With slots (T) int32, distinct where they are inside the cache, keys and
    values are stored in k_cache and v_cache (pages, page, Hkv, D), with a
    key_bias (pages, page, Hkv) of 0; others are skipped. Returns
    (q_out, k_out); k_out is None with a cache unless given. q_out and k_out
    given may not overlap each other, the cache or an input (not even q itself)."""
    tc = _tc or _calls()
    dt, index = q.dtype, _gpu_index(q, "q")
    code = tc.codes.get(dt)
    if code is None:
        code = dtype_code(dt)            # says what is supported
    sq, sk = _rows(q, "q", dt, 3, index), _rows(k, "k", dt, 3, index)
    T, Hq, D = q.shape
    ks = k.shape
    Hkv = ks[1]
    if ks != (T, Hkv, D):
        raise ValueError(f"k must have shape {(T, 'Hkv', D)}, got {tuple(ks)}")
    cache = vp = sv = sp = p_ko = None
    if slots is not None:
        if v is None or k_cache is None or v_cache is None:
            raise ValueError("slots need v, k_cache and v_cache")
        sv = _rows(v, "v", dt, 3, index)
        if v.shape != ks:
            raise ValueError(f"v must have k's shape {tuple(ks)}, got {tuple(v.shape)}")
        vp, sv = v.data_ptr(), _pack2(sv[0], sv[1])
        sp = _on(slots, "slots", tc.i32, (T,), index)
        cache = _kv_cache(k_cache, v_cache, key_bias, dt, Hkv, D, index)[0]
    elif v is not None or k_cache is not None or v_cache is not None or key_bias is not None:
        raise ValueError("v and the cache need slots")
    elif k_out is None:
        k_out = tc.empty((T, Hkv, D), dtype=dt, device=q.device)
        p_ko = k_out.data_ptr()
    given = []                           # outputs of the caller's
    if k_out is not None and p_ko is None:
        p_ko = _on(k_out, "k_out", dt, (T, Hkv, D), index)
        given.append(("k_out", p_ko, k_out))
    if q_out is None:
        q_out = tc.empty((T, Hq, D), dtype=dt, device=q.device)
        p_qo = q_out.data_ptr()
    else:
        p_qo = _on(q_out, "q_out", dt, (T, Hq, D), index)
        given.append(("q_out", p_qo, q_out))
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight go together")
    p_qw = p_kw = rp = pp = None
    if q_weight is not None:
        p_qw = _on(q_weight, "q_weight", dt, (D,), index)
        p_kw = _on(k_weight, "k_weight", dt, (D,), index)
        _no_grad(q_weight, "q_weight")
        _no_grad(k_weight, "k_weight")
    rot = max_pos = 0
    if rope is not None:
        if rope.dim() != 2 or positions is None:
            raise ValueError("rope must be (max_pos, rot), with positions")
        max_pos, rot = rope.shape
        rp = _on(rope, "rope", tc.f32, (max_pos, rot), index)
        _no_grad(rope, "rope")
        pp = _on(positions, "positions", tc.i32, (T,), index)
    if given:
        e = q.element_size()
        outs = [(n, p, p + t.numel() * e) for n, p, t in given if t.numel()]
        ins = [_span("q", q, sq, e), _span("k", k, sk, e)]
        if cache:
            ins += [_span("v", v, v.stride(), e), ("slots", sp, sp + 4 * T),
                    _span("k_cache", k_cache, k_cache.stride(), e),
                    _span("v_cache", v_cache, v_cache.stride(), e)]
        if p_qw:
            ins += [("q_weight", p_qw, p_qw + D * e), ("k_weight", p_kw, p_kw + D * e)]
        if rp:
            ins += [("rope", rp, rp + 4 * rope.numel()), ("positions", pp, pp + 4 * T)]
        _apart(outs, ins)
    st = _lib.fk_qk_norm_rope(
        q.data_ptr(), _pack2(sq[0], sq[1]), k.data_ptr(), _pack2(sk[0], sk[1]), vp, sv, code, T,
        Hq, Hkv, D, p_qw, p_kw, eps, rp, max_pos, rot, interleaved, pp, sp, cache,
        p_qo, p_ko, tc.stream(index))
    if st:
        _check(st, "fk_qk_norm_rope")
    return q_out, k_out


@functools.lru_cache(256)
def _attn_ws(code, B, Hq, Hkv, D):
    return int(load().fk_workspace_size_attn(code, B, Hq, Hkv, D))


def fk_workspace_size_attn(dtype, B: int, Hq: int, Hkv: int, D: int) -> int:
    return _attn_ws(dtype if isinstance(dtype, int) else dtype_code(dtype), B, Hq, Hkv, D)


def fk_paged_attn(q, k_cache, v_cache, table, lens, scale: Optional[float] = None,
                  softcap: float = 0.0, key_bias=None, max_len: int = 0, out=None, lse=None,
                  return_lse: bool = False, ws=None):
    """Attention of one token per request, q (B,Hq,D), over lens (B) int32 keys
    of k_cache and v_cache (pages, page, Hkv, D) found through table (B,W)
    int32: softmax(softcap(scale q.k) + key_bias) v, with scale 1/sqrt(D) by
    default. Returns out (B,Hq,D), and with return_lse (or lse given) the
    natural log of the softmax's sum, (B,Hq) fp32. out, lse and ws given may not
    overlap each other or an input, but out may be a contiguous q itself."""
    tc = _tc or _calls()
    dt, index = q.dtype, _gpu_index(q, "q")
    code = tc.codes.get(dt)
    if code is None:
        code = dtype_code(dt)            # says what is supported
    sq = _rows(q, "q", dt, 3, index)
    B, Hq, D = q.shape
    cache, heads = _kv_cache(k_cache, v_cache, key_bias, dt, 0, D, index)
    st2 = _rows(table, "table", tc.i32, 2, index)
    rows, width = table.shape
    if rows != B:
        raise ValueError(f"table must have {B} rows, got {tuple(table.shape)}")
    p_lens = _on(lens, "lens", tc.i32, (B,), index)
    need = _attn_ws(code, B, Hq, heads, D)
    if need == 0:
        raise ValueError(f"{Hq} query heads of {D} do not go with {heads} cache heads")
    dev = q.device
    if out is None:
        if q.is_contiguous():
            out = tc.empty_like(q)
        else:
            out = tc.empty((B, Hq, D), dtype=dt, device=dev)
        p_out = out.data_ptr()
    else:
        p_out = _on(out, "out", dt, (B, Hq, D), index)
        if p_out != q.data_ptr() or not q.is_contiguous():
            _apart([("out", p_out, p_out + out.numel() * q.element_size())],
                   [_span("q", q, sq, q.element_size())])
    p_lse = None
    if lse is not None:
        p_lse = _on(lse, "lse", tc.f32, (B, Hq), index)
    elif return_lse:
        lse = tc.empty((B, Hq), dtype=tc.f32, device=dev)
        p_lse = lse.data_ptr()
    if ws is None:
        ws = tc.empty(need, dtype=tc.u8, device=dev)
        p_ws = ws.data_ptr()
    else:
        need = ws.numel()
        p_ws = _on(ws, "ws", tc.u8, (need,), index)
    st = _lib.fk_paged_attn(
        q.data_ptr(), _pack2(sq[0], sq[1]), code, B, Hq, cache, table.data_ptr(),
        st2[0] if B > 1 else width, width, p_lens, max_len, D ** -0.5 if scale is None else scale,
        softcap, p_out, p_lse, p_ws, need, tc.stream(index))
    if st:
        _check(st, "fk_paged_attn")
    return out if lse is None else (out, lse)


def fk_trace_begin(capacity: int) -> None:
    _check(load().fk_trace_begin(int(capacity)), "fk_trace_begin")


def fk_trace_end() -> dict:
    out = fk_trace_t()
    _check(load().fk_trace_end(ctypes.byref(out)), "fk_trace_end")
    return {"iterations": out.iterations, "norms_ms": out.norms_ms,
            "assign_ms": out.assign_ms, "update_ms": out.update_ms}


# ---------------------------------------------------------------------------
# libfkbaseline: the materialised-distance assign and the scatter-atomic
# update (include/fkmeans_baselines.h), for contrast measurements only.
# ---------------------------------------------------------------------------
BASELINE_LIB_PATH = os.path.join(HERE, "libfkbaseline.so")
_blib = None


def load_baseline(path: Optional[str] = None):
    """Load libfkbaseline.so (once) and declare its signatures."""
    global _blib
    if _blib is not None:
        return _blib
    path = path or BASELINE_LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first "
                           "(python -m exact_means_clustering_flashassign_amd.build)")
    lib = ctypes.CDLL(path)
    P, I64 = ctypes.c_void_p, ctypes.c_int64
    lib.fkb_assign_materialized.restype = ctypes.c_int
    lib.fkb_assign_materialized.argtypes = [P, P, P, ctypes.c_int, I64, I64, I64, I64, P, P, P]
    lib.fkb_update_atomic.restype = ctypes.c_int
    lib.fkb_update_atomic.argtypes = [P, P, ctypes.c_int, I64, I64, I64, I64, P, P, P, P]
    lib.fkb_mfma_peak.restype = ctypes.c_int
    lib.fkb_mfma_peak.argtypes = [I64, ctypes.c_int32, ctypes.c_uint32, P, P, P]
    lib.fkb_wall_clock_khz.restype = ctypes.c_int32
    lib.fkb_wall_clock_khz.argtypes = []
    _blib = lib
    return lib


def fkb_assign_materialized(x, c_lp, cnorm, dist=None, ids=None):
    """Standard assign: the (B,N,K) fp32 matrix -2 x.c (rocBLAS), then argmin."""
    torch = _torch()
    code = dtype_code(x.dtype)
    B, N, d = x.shape
    K = c_lp.shape[1]
    if dist is None:
        dist = torch.empty((B, N, K), dtype=torch.float32, device=x.device)
    if ids is None:
        ids = torch.empty((B, N), dtype=torch.int32, device=x.device)
    st = load_baseline().fkb_assign_materialized(
        _dev(x, "x"), _dev(c_lp, "c_lp", x.dtype, (B, K, d)),
        _dev(cnorm, "cnorm", torch.float32, (B, K)), code, B, N, d, K,
        _dev(dist, "dist", torch.float32, (B, N, K)), _dev(ids, "ids", torch.int32, (B, N)),
        _stream(x))
    _check(st, "fkb_assign_materialized")
    return ids


def fkb_update_atomic(x, ids, c, counts=None, sums=None):
    """Standard update: scatter atomics into sums, then divide; c updated in place."""
    torch = _torch()
    code = dtype_code(x.dtype)
    B, N, d = x.shape
    K = c.shape[1]
    if counts is None:
        counts = torch.empty((B, K), dtype=torch.int32, device=x.device)
    if sums is None:
        sums = torch.empty((B, K, d), dtype=torch.float32, device=x.device)
    st = load_baseline().fkb_update_atomic(
        _dev(x, "x"), _dev(ids, "ids", torch.int32, (B, N)), code, B, N, d, K,
        _dev(c, "c", torch.float32, (B, K, d)), _dev(counts, "counts", torch.int32, (B, K)),
        _dev(sums, "sums", torch.float32, (B, K, d)), _stream(x))
    _check(st, "fkb_update_atomic")
    return c, counts


def fkb_mfma_peak(blocks: int, iters: int, seed: int, out=None, stamps=None, device="cuda"):
    """MFMA peak probe: blocks x 4 waves, each iters x 32 v_mfma_f32_32x32x16_f16.
    Returns (out, stamps); stamps (blocks, 4) int64 = memtime start/end,
    realtime start/end per block."""
    torch = _torch()
    if out is None:
        out = torch.empty(blocks * 256, dtype=torch.float32, device=device)
    if stamps is None:
        stamps = torch.empty((blocks, 4), dtype=torch.int64, device=device)
    st = load_baseline().fkb_mfma_peak(int(blocks), int(iters), int(seed) & 0xFFFFFFFF,
                                       _dev(out, "out", torch.float32, (blocks * 256,)),
                                       _dev(stamps, "stamps", torch.int64, (blocks, 4)),
                                       _stream(out))
    _check(st, "fkb_mfma_peak")
    return out, stamps


def fkb_wall_clock_khz() -> int:
    return int(load_baseline().fkb_wall_clock_khz())

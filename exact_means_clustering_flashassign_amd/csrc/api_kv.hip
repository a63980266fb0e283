// C ABI of the paged key-value cache: argument validation before anything is
// enqueued. The kernels are in kvtables.hip, qkrope.hip, attn.hip, prompt.hip,
// cache8.hip and attn8.hip.
#include <math.h>

#include "fk_kv.hpp"

namespace {

constexpr int64_t kI32Max = 0x7FFFFFFF;
constexpr int64_t kElemLimit = (int64_t)1 << 62;

bool valid_dt(int dt) { return dt == FK_F32 || dt == FK_F16 || dt == FK_BF16; }

bool below(int64_t v, int64_t lo) { return v < lo || v >= kI32Max; }

// a * b (both >= 0) stays under the element limit.
bool mul_ok(int64_t a, int64_t b) { return a == 0 || b <= kElemLimit / a; }

// Offsets i0*s0 + i1*s1 + i2*s2 + dim over the given extents stay addressable.
bool extent_ok(const int64_t* n, const int64_t* s, int axes, int64_t dim) {
  int64_t total = dim;
  for (int i = 0; i < axes; ++i) {
    if (s[i] < 0) return false;
    const int64_t last = n[i] > 0 ? n[i] - 1 : 0;
    if (!mul_ok(last, s[i]) || (total += last * s[i]) > kElemLimit) return false;
  }
  return true;
}

bool valid_cache(const fk_kv_cache_t* c) {
  if (!c || below(c->pages, 0) || below(c->page, 1) || below(c->heads, 1) || below(c->dim, 1))
    return false;
  if (c->pages * c->page >= ((int64_t)1 << 31)) return false;
  if (c->pages > 0 && (!c->k || !c->v)) return false;
  const int64_t n[3] = {c->pages, c->page, c->heads};
  return extent_ok(n, c->k_stride, 3, c->dim) && extent_ok(n, c->v_stride, 3, c->dim) &&
         (!c->key_bias || extent_ok(n, c->bias_stride, 3, 1));
}

bool valid_cache8(const fk_kv_cache8_t* c) {
  if (!c || below(c->pages, 0) || below(c->page, 1) || below(c->heads, 1) || below(c->dim, 1))
    return false;
  if (c->pages * c->page >= ((int64_t)1 << 31)) return false;
  if (c->pages > 0 && (!c->k || !c->v || !c->k_scale || !c->v_scale)) return false;
  const int64_t n[3] = {c->pages, c->page, c->heads};
  return extent_ok(n, c->k_stride, 3, c->dim) && extent_ok(n, c->v_stride, 3, c->dim) &&
         extent_ok(n, c->k_scale_stride, 3, 1) && extent_ok(n, c->v_scale_stride, 3, 1) &&
         (!c->key_bias || extent_ok(n, c->bias_stride, 3, 1));
}

bool valid_rows(const int64_t* stride, int64_t n, int64_t heads, int64_t dim) {
  const int64_t ext[2] = {n, heads};
  return stride && extent_ok(ext, stride, 2, dim);
}

fk_status_t status_of(hipError_t e) {
  if (e == hipErrorInvalidConfiguration || e == hipErrorNotSupported) return FK_ERR_UNSUPPORTED;
  return e == hipSuccess ? FK_OK : FK_ERR_HIP;
}

}  // namespace

extern "C" {

fk_status_t fk_page_tables(const int32_t* len_old, const int32_t* len_new,
                           const int32_t* table_in, int64_t width_in, const int32_t* free_pages,
                           int64_t n_free, int64_t B, int64_t page, int64_t width, int64_t tokens,
                           int32_t* table, int32_t* lens, int32_t* cu_tokens, int32_t* cu_pages,
                           int32_t* slots, int32_t* positions, hipStream_t stream) {
  if (below(B, 0) || below(page, 1) || below(width, 1) || below(width_in, 0) ||
      below(n_free, 0) || below(tokens, 0) || !mul_ok(B, width))
    return FK_ERR_INVALID;
  if (!cu_tokens || !cu_pages) return FK_ERR_INVALID;
  if (B > 0 && (!len_old || !len_new || !table || !lens)) return FK_ERR_INVALID;
  if (B > 0 && width_in > 0 && !table_in) return FK_ERR_INVALID;
  if (B > 0 && table_in && table_in == table && width_in != width) return FK_ERR_INVALID;
  if (n_free > 0 && !free_pages) return FK_ERR_INVALID;
  if (tokens > 0 && (!slots || !positions)) return FK_ERR_INVALID;
  fk::TablesArgs a{len_old, len_new, table_in, free_pages, width_in, n_free, B, page, width,
                   tokens, table, lens, cu_tokens, cu_pages, slots, positions};
  return status_of(fk::launch_page_tables(a, stream));
}

fk_status_t fk_qk_norm_rope(const void* q, const int64_t q_stride[2], const void* k,
                            const int64_t k_stride[2], const void* v, const int64_t v_stride[2],
                            fk_dtype_t dt, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                            const void* q_weight, const void* k_weight, float eps,
                            const float* rope, int64_t max_pos, int64_t rot, int32_t interleaved,
                            const int32_t* positions, const int32_t* slots,
                            const fk_kv_cache_t* cache, void* q_out, void* k_out,
                            hipStream_t stream) {
  if (!valid_dt(dt) || below(T, 0) || below(Hq, 1) || below(Hkv, 1) || below(D, 1))
    return FK_ERR_INVALID;
  if (rot < 0 || rot > D || (rot & 1) || !(eps >= 0.f) || isinf(eps)) return FK_ERR_INVALID;
  if ((q_weight == nullptr) != (k_weight == nullptr)) return FK_ERR_INVALID;
  if (!valid_rows(q_stride, T, Hq, D) || !valid_rows(k_stride, T, Hkv, D)) return FK_ERR_INVALID;
  if (T > 0 && (cache == nullptr) != (slots == nullptr)) return FK_ERR_INVALID;
  if (cache) {
    if (!valid_cache(cache) || cache->heads != Hkv || cache->dim != D) return FK_ERR_INVALID;
    if (!valid_rows(v_stride, T, Hkv, D)) return FK_ERR_INVALID;
  }
  if (!mul_ok(T, Hq) || !mul_ok(T * Hq, D) || !mul_ok(T, Hkv) || !mul_ok(T * Hkv, D))
    return FK_ERR_INVALID;
  if (T == 0) return FK_OK;
  if (!q || !k || !q_out || (cache && !v) || (!cache && !k_out)) return FK_ERR_INVALID;
  if (rot > 0 && (!rope || !positions || below(max_pos, 1))) return FK_ERR_INVALID;
  fk::RopeArgs a{};
  a.q = q, a.k = k, a.v = v;
  for (int i = 0; i < 2; ++i) {
    a.q_stride[i] = q_stride[i];
    a.k_stride[i] = k_stride[i];
    a.v_stride[i] = cache ? v_stride[i] : 0;
  }
  a.T = T, a.Hq = Hq, a.Hkv = Hkv, a.D = D;
  a.q_weight = q_weight, a.k_weight = k_weight, a.eps = eps;
  a.rope = rope, a.max_pos = max_pos, a.rot = rot, a.interleaved = interleaved != 0;
  a.positions = positions, a.slots = slots;
  if (cache && cache->pages > 0) a.cache = *cache;   // no pages: every slot is outside
  a.q_out = q_out, a.k_out = k_out;
  return status_of(fk::launch_qk_norm_rope(a, dt, stream));
}

size_t fk_workspace_size_attn(fk_dtype_t dt, int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  if (!valid_dt(dt) || below(B, 0) || below(Hq, 1) || below(Hkv, 1) || Hq % Hkv || below(D, 1))
    return 0;
  const size_t n = fk::attn_ws_bytes(dt, B, Hq, Hkv, D);
  return n < 256 ? 256 : n;
}

fk_status_t fk_paged_attn(const void* q, const int64_t q_stride[2], fk_dtype_t dt, int64_t B,
                          int64_t Hq, const fk_kv_cache_t* cache, const int32_t* table,
                          int64_t ld_table, int64_t width, const int32_t* lens, int64_t max_len,
                          float scale, float softcap, void* out, float* lse, void* ws,
                          size_t ws_bytes, hipStream_t stream) {
  if (!valid_dt(dt) || below(B, 0) || below(Hq, 1) || !valid_cache(cache)) return FK_ERR_INVALID;
  if (Hq % cache->heads || below(width, 0) || ld_table < width || max_len < 0)
    return FK_ERR_INVALID;
  if (!isfinite(scale) || !(softcap >= 0.f) || isinf(softcap)) return FK_ERR_INVALID;
  if (!valid_rows(q_stride, B, Hq, cache->dim) || !mul_ok(B, Hq) ||
      !mul_ok(B * Hq, cache->dim) || !mul_ok(B, ld_table))
    return FK_ERR_INVALID;
  if (cache->dim > fk::kAttnMaxDim) return FK_ERR_UNSUPPORTED;
  if (B == 0) return FK_OK;
  if (!q || !lens || !out || (width > 0 && !table)) return FK_ERR_INVALID;
  if (!ws || ((uintptr_t)ws & 255) ||
      ws_bytes < fk_workspace_size_attn(dt, B, Hq, cache->heads, cache->dim))
    return FK_ERR_WORKSPACE;
  fk::AttnArgs a{};
  a.q = q, a.q_stride[0] = q_stride[0], a.q_stride[1] = q_stride[1];
  a.B = B, a.Hq = Hq, a.cache = *cache;
  a.table = table, a.ld_table = ld_table, a.width = width, a.lens = lens, a.max_len = max_len;
  a.scale = scale, a.softcap = softcap, a.out = out, a.lse = lse;
  return status_of(fk::launch_paged_attn(a, dt, ws, stream));
}

size_t fk_workspace_size_prompt(fk_dtype_t dt, int64_t T, int64_t B, int64_t Hq, int64_t Hkv,
                                int64_t D) {
  if (!valid_dt(dt) || below(T, 0) || below(B, 0) || below(Hq, 1) || below(Hkv, 1) || Hq % Hkv ||
      below(D, 1) || !mul_ok(T, Hq) || !mul_ok(T * Hq, 64 * D))
    return 0;
  const size_t n = fk::prompt_ws_bytes(dt, T, B, Hq, Hkv, D);
  return n < 256 ? 256 : n;
}

fk_status_t fk_prompt_attn(const void* q, const int64_t q_stride[2], fk_dtype_t dt, int64_t T,
                           int64_t B, int64_t Hq, const fk_kv_cache_t* cache,
                           const int32_t* table, int64_t ld_table, int64_t width,
                           const int32_t* lens, const int32_t* cu_tokens, int64_t max_len,
                           float scale, float softcap, void* out, float* lse, void* ws,
                           size_t ws_bytes, hipStream_t stream) {
  if (!valid_dt(dt) || below(T, 0) || below(B, 0) || below(Hq, 1) || !valid_cache(cache))
    return FK_ERR_INVALID;
  if (Hq % cache->heads || below(width, 0) || ld_table < width || max_len < 0)
    return FK_ERR_INVALID;
  if (!isfinite(scale) || !(softcap >= 0.f) || isinf(softcap)) return FK_ERR_INVALID;
  if (!valid_rows(q_stride, T, Hq, cache->dim) || !mul_ok(T, Hq) ||
      !mul_ok(T * Hq, 64 * cache->dim) || !mul_ok(B, ld_table))
    return FK_ERR_INVALID;
  if (cache->dim > fk::kAttnMaxDim) return FK_ERR_UNSUPPORTED;
  if (T == 0 || B == 0) return FK_OK;
  if (!q || !lens || !cu_tokens || !out || (width > 0 && !table)) return FK_ERR_INVALID;
  if (!ws || ((uintptr_t)ws & 255) ||
      ws_bytes < fk_workspace_size_prompt(dt, T, B, Hq, cache->heads, cache->dim))
    return FK_ERR_WORKSPACE;
  fk::PromptArgs a{};
  a.q = q, a.q_stride[0] = q_stride[0], a.q_stride[1] = q_stride[1];
  a.T = T, a.B = B, a.Hq = Hq, a.cache = *cache;
  a.table = table, a.ld_table = ld_table, a.width = width, a.lens = lens, a.cu = cu_tokens;
  a.max_len = max_len, a.scale = scale, a.softcap = softcap, a.out = out, a.lse = lse;
  return status_of(fk::launch_prompt_attn(a, dt, ws, stream));
}

fk_status_t fk_kv_store8(const void* k, const int64_t k_stride[2], const void* v,
                         const int64_t v_stride[2], fk_dtype_t dt, int64_t T,
                         const int32_t* slots, const fk_kv_cache8_t* cache, hipStream_t stream) {
  if (!valid_dt(dt) || below(T, 0) || !valid_cache8(cache)) return FK_ERR_INVALID;
  if (!valid_rows(k_stride, T, cache->heads, cache->dim) ||
      !valid_rows(v_stride, T, cache->heads, cache->dim) || !mul_ok(T, cache->heads) ||
      !mul_ok(T * cache->heads, cache->dim))
    return FK_ERR_INVALID;
  if (T == 0) return FK_OK;
  if (!k || !v || !slots) return FK_ERR_INVALID;
  if (cache->pages == 0) return FK_OK;               // every slot is outside
  fk::Cache8Args a{};
  a.k = k, a.v = v, a.T = T, a.slots = slots, a.cache = *cache;
  for (int i = 0; i < 2; ++i) a.k_stride[i] = k_stride[i], a.v_stride[i] = v_stride[i];
  return status_of(fk::launch_kv_store8(a, dt, stream));
}

fk_status_t fk_kv_load8(const fk_kv_cache8_t* cache, const int32_t* slots, fk_dtype_t dt,
                        int64_t T, void* k_out, void* v_out, hipStream_t stream) {
  if (!valid_dt(dt) || below(T, 0) || !valid_cache8(cache)) return FK_ERR_INVALID;
  if (!mul_ok(T, cache->heads) || !mul_ok(T * cache->heads, cache->dim)) return FK_ERR_INVALID;
  if (T == 0) return FK_OK;
  if (!slots || !k_out || !v_out) return FK_ERR_INVALID;
  fk::Cache8Args a{};
  a.T = T, a.slots = slots, a.cache = *cache, a.k_out = k_out, a.v_out = v_out;
  return status_of(fk::launch_kv_load8(a, dt, stream));
}

size_t fk_workspace_size_attn8(fk_dtype_t dt, int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  if (!valid_dt(dt) || below(B, 0) || below(Hq, 1) || below(Hkv, 1) || Hq % Hkv || below(D, 1))
    return 0;
  const size_t n = fk::attn8_ws_bytes(dt, B, Hq, Hkv, D);
  return n < 256 ? 256 : n;
}

fk_status_t fk_paged_attn8(const void* q, const int64_t q_stride[2], fk_dtype_t dt, int64_t B,
                           int64_t Hq, const fk_kv_cache8_t* cache, const int32_t* table,
                           int64_t ld_table, int64_t width, const int32_t* lens, int64_t max_len,
                           float scale, float softcap, void* out, float* lse, void* ws,
                           size_t ws_bytes, hipStream_t stream) {
  if (!valid_dt(dt) || below(B, 0) || below(Hq, 1) || !valid_cache8(cache)) return FK_ERR_INVALID;
  if (Hq % cache->heads || below(width, 0) || ld_table < width || max_len < 0)
    return FK_ERR_INVALID;
  if (!isfinite(scale) || !(softcap >= 0.f) || isinf(softcap)) return FK_ERR_INVALID;
  if (!valid_rows(q_stride, B, Hq, cache->dim) || !mul_ok(B, Hq) ||
      !mul_ok(B * Hq, cache->dim) || !mul_ok(B, ld_table))
    return FK_ERR_INVALID;
  if (cache->dim > fk::kAttnMaxDim) return FK_ERR_UNSUPPORTED;
  if (B == 0) return FK_OK;
  if (!q || !lens || !out || (width > 0 && !table)) return FK_ERR_INVALID;
  if (!ws || ((uintptr_t)ws & 255) ||
      ws_bytes < fk_workspace_size_attn8(dt, B, Hq, cache->heads, cache->dim))
    return FK_ERR_WORKSPACE;
  fk::AttnArgs8 a{};
  a.q = q, a.q_stride[0] = q_stride[0], a.q_stride[1] = q_stride[1];
  a.B = B, a.Hq = Hq;
  fk_kv_cache_t& c = a.cache;
  c.k = cache->k, c.v = cache->v, c.key_bias = cache->key_bias;
  c.pages = cache->pages, c.page = cache->page, c.heads = cache->heads, c.dim = cache->dim;
  a.k_scale = cache->k_scale, a.v_scale = cache->v_scale;
  for (int i = 0; i < 3; ++i) {
    c.k_stride[i] = cache->k_stride[i], c.v_stride[i] = cache->v_stride[i];
    c.bias_stride[i] = cache->bias_stride[i];
    a.ks_stride[i] = cache->k_scale_stride[i], a.vs_stride[i] = cache->v_scale_stride[i];
  }
  a.table = table, a.ld_table = ld_table, a.width = width, a.lens = lens, a.max_len = max_len;
  a.scale = scale, a.softcap = softcap, a.out = out, a.lse = lse;
  return status_of(fk::launch_paged_attn8(a, dt, ws, stream));
}

}  // extern "C"

// Keys and values quantised to e4m3 as they are written to a paged cache, and read
// back. Rows of (token, key or value, head) are independent: one pass over each.
#include <math.h>

#include "e4m3.hpp"

namespace fk {
namespace {

// A row's place in the cache.
struct Row {
  bool value;
  int64_t t, page, tok, h;
};

__device__ __forceinline__ bool row_of(const Cache8Args& a, int64_t r, Row& o) {
  const int64_t H = a.cache.heads;
  o.t = r / (2 * H);
  const int64_t i = r - o.t * 2 * H;
  o.value = i >= H;
  o.h = o.value ? i - H : i;
  const int64_t s = a.slots[o.t];
  o.page = s / a.cache.page;
  o.tok = s - o.page * a.cache.page;
  return s >= 0 && o.page < a.cache.pages;
}

// Any size, stride and alignment: a row a wave.
template <int DT> __global__ __launch_bounds__(256) void store8_any_kernel(Cache8Args a) {
  const int lane = threadIdx.x & 63;
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  Row o;
  if (r >= a.T * 2 * a.cache.heads || !row_of(a, r, o)) return;
  const fk_kv_cache8_t& c = a.cache;
  const int64_t* xs = o.value ? a.v_stride : a.k_stride;
  const int64_t* cs = o.value ? c.v_stride : c.k_stride;
  const int64_t* ss = o.value ? c.v_scale_stride : c.k_scale_stride;
  const auto* x = (const typename Val<DT>::type*)(o.value ? a.v : a.k) + o.t * xs[0] + o.h * xs[1];
  uint8_t* to = (uint8_t*)(o.value ? c.v : c.k) + o.page * cs[0] + o.tok * cs[1] + o.h * cs[2];
  float most = 0.f;
  for (int64_t e = lane; e < c.dim; e += 64) {
    const float y = fabsf(Val<DT>::get(x + e));
    most = y < INFINITY ? fmaxf(most, y) : most;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) most = fmaxf(most, __shfl_xor(most, off, 64));
  const int ex = scale_exponent(most);
  const float inv = pow2(-ex);
  for (int64_t e = lane; e < c.dim; e += 64) {
    const float y = Val<DT>::get(x + e);
    to[e] = (uint8_t)e4m3_codes(is_finite(y) ? y * inv : NAN, 0.f, 0.f, 0.f);
  }
  if (lane != 0) return;
  (o.value ? c.v_scale : c.k_scale)[o.page * ss[0] + o.tok * ss[1] + o.h * ss[2]] = pow2(ex);
  if (!o.value && c.key_bias)
    c.key_bias[o.page * c.bias_stride[0] + o.tok * c.bias_stride[1] + o.h * c.bias_stride[2]] = 0.f;
}

template <int DT> __global__ __launch_bounds__(256) void load8_any_kernel(Cache8Args a) {
  const int lane = threadIdx.x & 63;
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= a.T * 2 * a.cache.heads) return;
  const fk_kv_cache8_t& c = a.cache;
  Row o;
  const bool live = row_of(a, r, o);
  const int64_t* cs = o.value ? c.v_stride : c.k_stride;
  const int64_t* ss = o.value ? c.v_scale_stride : c.k_scale_stride;
  auto* y = (typename Val<DT>::type*)(o.value ? a.v_out : a.k_out) + (o.t * c.heads + o.h) * c.dim;
  if (!live) {
    for (int64_t e = lane; e < c.dim; e += 64) Val<DT>::put(y + e, 0.f);
    return;
  }
  const uint8_t* x = (const uint8_t*)(o.value ? c.v : c.k) + o.page * cs[0] + o.tok * cs[1] + o.h * cs[2];
  const float s = (o.value ? c.v_scale : c.k_scale)[o.page * ss[0] + o.tok * ss[1] + o.h * ss[2]];
  for (int64_t e = lane; e < c.dim; e += 64) Val<DT>::put(y + e, clamp_to<DT>(e4m3_get(x[e]) * s));
}

template <int DT> hipError_t run_store(const Cache8Args& a, hipStream_t s) {
  const int64_t rows = a.T * 2 * a.cache.heads, blocks = (rows + 3) / 4;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  store8_any_kernel<DT><<<(unsigned)blocks, 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int DT> hipError_t run_load(const Cache8Args& a, hipStream_t s) {
  const int64_t rows = a.T * 2 * a.cache.heads, blocks = (rows + 3) / 4;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  load8_any_kernel<DT><<<(unsigned)blocks, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_store8(const Cache8Args& a, int dt, hipStream_t s) {
  return dt == FK_F32 ? run_store<FK_F32>(a, s) : dt == FK_F16 ? run_store<FK_F16>(a, s) : run_store<FK_BF16>(a, s);
}

hipError_t launch_kv_load8(const Cache8Args& a, int dt, hipStream_t s) {
  return dt == FK_F32 ? run_load<FK_F32>(a, s) : dt == FK_F16 ? run_load<FK_F16>(a, s) : run_load<FK_BF16>(a, s);
}

}  // namespace fk

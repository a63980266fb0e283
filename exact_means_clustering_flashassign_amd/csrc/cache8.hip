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

constexpr int64_t kMostBlocks = 0xFFFFFF;            // of 256 threads: fewer than 2^32 in a launch

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

// ---------------------------------------------------------------------------
// Rows of whole, aligned units of 8 elements, up to 64 of them
// ---------------------------------------------------------------------------
// LPR lanes take a row, a unit each, and a wave 64 / LPR rows at a time, U times: all of a lane's
// loads go out before the first maximum is formed. Bound by bytes: 75600 tokens of 8 heads of
// 128, fp16, stored and read back in 218 us, 4.3 TB/s (a large copy: 4.9); 32 tokens take 11 us a
// call, nearly all of it the launch's.
typedef uint32_t w4 __attribute__((ext_vector_type(4)));
typedef uint32_t w2 __attribute__((ext_vector_type(2)));
typedef const __attribute__((address_space(1))) w4* src16;
typedef const __attribute__((address_space(1))) w2* src8;
typedef __attribute__((address_space(1))) w4* dst16;
typedef __attribute__((address_space(1))) w2* dst8;

template <int DT> struct Unit {            // 8 elements
  w4 w[DT == FK_F32 ? 2 : 1];
  __device__ __forceinline__ void load(uint64_t at) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(w) / 16); ++i) w[i] = *(src16)(at + 16 * i);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (DT == FK_F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t u = w[i >> 2][i & 3];
        x[i] = __builtin_bit_cast(float, u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint16_t u = (uint16_t)(w[0][i >> 1] >> (16 * (i & 1)));
        x[i] = Val<DT>::get(&u);
      }
    }
  }
  __device__ __forceinline__ void put(uint64_t at, const float (&x)[8]) {
    if constexpr (DT == FK_F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i >> 2][i & 3] = __builtin_bit_cast(uint32_t, x[i]);
    } else {
      typedef typename Val<DT>::arith T;
      typedef T T8 __attribute__((ext_vector_type(8)));
      T8 v;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (T)x[i];
      w[0] = __builtin_bit_cast(w4, v);
    }
#pragma unroll
    for (int i = 0; i < (int)(sizeof(w) / 16); ++i) *(dst16)(at + 16 * i) = w[i];
  }
};

struct Rows {
  uint32_t n;                 // of (token, key or value, head)
  FastDiv by_heads2, by_page;
};

// Row r's place.
struct Place {
  bool inside, value;
  uint32_t t, h;
  int64_t code, number;       // of its first code and its scale, from the cache's first
};
__device__ __forceinline__ Place place_of(const Cache8Args& a, const Rows& rows, uint32_t r) {
  const fk_kv_cache8_t& c = a.cache;
  Place o;
  o.t = div_by(r, rows.by_heads2);
  const uint32_t i = r - o.t * 2 * (uint32_t)c.heads;
  o.value = i >= c.heads;
  o.h = o.value ? i - (uint32_t)c.heads : i;
  const int32_t s = a.slots[o.t];
  const uint32_t page = div_by(s < 0 ? 0 : s, rows.by_page), tok = (s < 0 ? 0 : s) - page * rows.by_page.d;
  o.inside = s >= 0 && page < c.pages;
  const int64_t* cs = o.value ? c.v_stride : c.k_stride;
  const int64_t* ss = o.value ? c.v_scale_stride : c.k_scale_stride;
  o.code = page * cs[0] + tok * cs[1] + o.h * cs[2];
  o.number = page * ss[0] + tok * ss[1] + o.h * ss[2];
  return o;
}

template <int DT, int LPR, int U> __global__ __launch_bounds__(256) void store8_kernel(Cache8Args a, Rows rows) {
  constexpr int per = 64 / LPR;
  const fk_kv_cache8_t& c = a.cache;
  const int lane = threadIdx.x & 63, unit = lane & (LPR - 1);
  const uint32_t r0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * (per * U) + lane / LPR;
  const bool held = unit * 8 < c.dim;
  Unit<DT> in[U];
  Place at[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t r = r0 + u * per;
    at[u].inside = false;
    if (r >= rows.n) continue;
    at[u] = place_of(a, rows, r);
    const int64_t* xs = at[u].value ? a.v_stride : a.k_stride;
    const uint64_t from = (uint64_t)(at[u].value ? a.v : a.k) +
                          (uint64_t)(at[u].t * xs[0] + at[u].h * xs[1] + unit * 8) * Val<DT>::bytes;
    if (held) in[u].load(from);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float x[8], most = 0.f;
    in[u].get(x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = fabsf(x[i]);
      most = held && y < INFINITY ? fmaxf(most, y) : most;
    }
#pragma unroll
    for (int off = LPR / 2; off >= 1; off >>= 1) most = fmaxf(most, __shfl_xor(most, off, 64));
    const int ex = scale_exponent(most);
    const float inv = pow2(-ex);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = is_finite(x[i]) ? x[i] * inv : NAN;
    if (!at[u].inside) continue;
    if (held)
      *(dst8)((uint64_t)(at[u].value ? c.v : c.k) + at[u].code + unit * 8) =
          w2{e4m3_codes(x[0], x[1], x[2], x[3]), e4m3_codes(x[4], x[5], x[6], x[7])};
    if (unit != 0) continue;
    (at[u].value ? c.v_scale : c.k_scale)[at[u].number] = pow2(ex);
    if (!at[u].value && c.key_bias) {
      const int32_t s = a.slots[at[u].t];
      const uint32_t page = div_by(s, rows.by_page), tok = s - page * rows.by_page.d;
      c.key_bias[page * c.bias_stride[0] + tok * c.bias_stride[1] + at[u].h * c.bias_stride[2]] = 0.f;
    }
  }
}

template <int DT, int LPR, int U> __global__ __launch_bounds__(256) void load8_kernel(Cache8Args a, Rows rows) {
  constexpr int per = 64 / LPR;
  const fk_kv_cache8_t& c = a.cache;
  const int lane = threadIdx.x & 63, unit = lane & (LPR - 1);
  const uint32_t r0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * (per * U) + lane / LPR;
  const bool held = unit * 8 < c.dim;
  w2 in[U];
  float scale[U];
  Place at[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t r = r0 + u * per;
    in[u] = w2{0, 0}, scale[u] = 0.f;
    if (r >= rows.n) continue;
    at[u] = place_of(a, rows, r);
    if (!at[u].inside) continue;
    if (held) in[u] = *(src8)((uint64_t)(at[u].value ? c.v : c.k) + at[u].code + unit * 8);
    scale[u] = (at[u].value ? c.v_scale : c.k_scale)[at[u].number];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (r0 + u * per >= rows.n || !held) continue;
    float x[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w = in[u][i];
      const floatx2_t lo = e4m3_pair<false>(w), hi = e4m3_pair<true>(w);
      x[4 * i] = lo.x, x[4 * i + 1] = lo.y, x[4 * i + 2] = hi.x, x[4 * i + 3] = hi.y;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = clamp_to<DT>(x[i] * scale[u]);
    Unit<DT> out;
    out.put((uint64_t)(at[u].value ? a.v_out : a.k_out) +
                (uint64_t)(((int64_t)at[u].t * c.heads + at[u].h) * c.dim + unit * 8) * Val<DT>::bytes, x);
  }
}

// Whether rows hold whole units that start where a unit may.
bool whole_units(const Cache8Args& a, int eb) {
  const fk_kv_cache8_t& c = a.cache;
  if (c.dim % 8 || c.dim > 512 || a.T * 2 * c.heads >= ((int64_t)1 << 31)) return false;
  for (int i = 0; i < 3; ++i)
    if ((c.k_stride[i] | c.v_stride[i]) % 8) return false;
  for (int i = 0; i < 2; ++i)
    if ((a.k_stride[i] | a.v_stride[i]) * eb % 16) return false;      // (0 for loads)
  if (((uintptr_t)c.k | (uintptr_t)c.v) & 7) return false;
  return !(((uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.k_out | (uintptr_t)a.v_out) & 15);
}

template <int DT, int LPR> hipError_t run_units(const Cache8Args& a, bool store, hipStream_t s) {
  const uint32_t n = (uint32_t)(a.T * 2 * a.cache.heads);
  const Rows rows{n, fast_div((uint32_t)(2 * a.cache.heads)), fast_div((uint32_t)a.cache.page)};
  // four rows a lane where there is work for every wave of the chip all the same
  const bool many = (int64_t)n * LPR >= (int64_t)4 * 64 * 8 * 4 * kMaxCus;
  const uint32_t per_block = 4 * (64 / LPR) * (many ? 4 : 1), blocks = n / per_block + (n % per_block != 0);
  if (blocks > kMostBlocks) return hipErrorInvalidConfiguration;
  const auto kernel = store ? (many ? store8_kernel<DT, LPR, 4> : store8_kernel<DT, LPR, 1>)
                            : (many ? load8_kernel<DT, LPR, 4> : load8_kernel<DT, LPR, 1>);
  kernel<<<blocks, 256, 0, s>>>(a, rows);
  return hipGetLastError();
}

template <int DT> hipError_t run(const Cache8Args& a, bool store, hipStream_t s) {
  const int64_t n = a.T * 2 * a.cache.heads, blocks = (n + 3) / 4, D = a.cache.dim;
  if (whole_units(a, Val<DT>::bytes))
    return D <= 32    ? run_units<DT, 4>(a, store, s)
           : D <= 64  ? run_units<DT, 8>(a, store, s)
           : D <= 128 ? run_units<DT, 16>(a, store, s)
           : D <= 256 ? run_units<DT, 32>(a, store, s)
                      : run_units<DT, 64>(a, store, s);
  if (blocks > kMostBlocks) return hipErrorInvalidConfiguration;
  if (store) store8_any_kernel<DT><<<(unsigned)blocks, 256, 0, s>>>(a);
  else load8_any_kernel<DT><<<(unsigned)blocks, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_store8(const Cache8Args& a, int dt, hipStream_t s) {
  return dt == FK_F32 ? run<FK_F32>(a, true, s) : dt == FK_F16 ? run<FK_F16>(a, true, s) : run<FK_BF16>(a, true, s);
}

hipError_t launch_kv_load8(const Cache8Args& a, int dt, hipStream_t s) {
  return dt == FK_F32 ? run<FK_F32>(a, false, s) : dt == FK_F16 ? run<FK_F16>(a, false, s) : run<FK_BF16>(a, false, s);
}

}  // namespace fk

// Attention of a step's prompts over a paged key-value cache: every new token over
// its request's keys up to itself.
#include "attn_parts.hpp"

namespace fk {
namespace {

// Request of token t: the last one that starts at or before it and is not empty; -1: none.
__device__ __forceinline__ int64_t request_of(const PromptArgs& a, int64_t t) {
  int64_t lo = 0, hi = a.B;                // first b with cu[b + 1] > t
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (a.cu[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo < a.B && a.cu[lo] <= t ? lo : -1;
}

// Keys that token t of request b sees.
__device__ __forceinline__ int64_t seen_by(const PromptArgs& a, int64_t b, int64_t t) {
  const int64_t held = a.width * a.cache.page;
  const int64_t n = (int64_t)a.lens[b] - a.cu[b + 1] + t + 1;
  return n < 0 ? 0 : (n < held ? n : held);
}

// One row (token, query head), any size, stride and alignment, by one wave: a lane holds
// every 64th element.
template <int DT, int EPL>
__device__ __forceinline__ void attend_row(const PromptArgs& a, int64_t t, int64_t h) {
  using E = typename Val<DT>::type;
  const int64_t b = request_of(a, t);
  if (b < 0) return;
  const int lane = threadIdx.x & 63;
  const fk_kv_cache_t& c = a.cache;
  const int D = (int)c.dim;
  const int64_t hk = h / (a.Hq / c.heads), n = seen_by(a, b, t);
  const E* q = (const E*)a.q + t * a.q_stride[0] + h * a.q_stride[1];
  float qf[EPL], o[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    qf[i] = e < D ? Val<DT>::get(q + e) : 0.f;
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t j = 0; j < n; ++j) {
    const int64_t page = a.table[b * a.ld_table + j / c.page], tok = j % c.page;
    if (page < 0 || page >= c.pages) continue;
    float bias = 0.f;
    if (c.key_bias) {
      bias = c.key_bias[page * c.bias_stride[0] + tok * c.bias_stride[1] + hk * c.bias_stride[2]];
      if (bias == -INFINITY) continue;
    }
    const E* k = (const E*)c.k + page * c.k_stride[0] + tok * c.k_stride[1] + hk * c.k_stride[2];
    const E* v = (const E*)c.v + page * c.v_stride[0] + tok * c.v_stride[1] + hk * c.v_stride[2];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      if (e < D) s = fmaf(qf[i], Val<DT>::get(k + e), s);
    }
    s = wave_sum(s) * a.scale;
    if (a.softcap > 0.f) s = capped(s, a.softcap, 1.f / a.softcap);
    s += bias;
    const float mn = fmaxf(m, s);
    const float alpha = m == -INFINITY ? 0.f : fast_exp2((m - mn) * kLog2e);
    const float p = s == -INFINITY ? 0.f : fast_exp2((s - mn) * kLog2e);   // NaN stays NaN
    l = l * alpha + p;
    m = mn;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      if (e < D) o[i] = fmaf(p, Val<DT>::get(v + e), o[i] * alpha);
    }
  }
  const bool any = l != 0.f;             // true for NaN: it has to reach the result
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    if (e < D) Val<DT>::put((E*)a.out + (t * a.Hq + h) * D + e, any ? o[i] / l : 0.f);
  }
  if (a.lse && lane == 0) a.lse[t * a.Hq + h] = any ? m + logf(l) : -INFINITY;
}

template <int DT, int EPL>
__global__ __launch_bounds__(kWaves * 64) void prompt_any_kernel(PromptArgs a) {
  const int64_t r = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  const int64_t t = r / a.Hq;
  if (t < a.T) attend_row<DT, EPL>(a, t, r - t * a.Hq);
}

template <int DT> hipError_t run_any(const PromptArgs& a, hipStream_t s) {
  const int64_t D = a.cache.dim, blocks = (a.T * a.Hq + kWaves - 1) / kWaves;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const auto kernel = D <= 64    ? prompt_any_kernel<DT, 1>
                      : D <= 128 ? prompt_any_kernel<DT, 2>
                      : D <= 256 ? prompt_any_kernel<DT, 4>
                                 : prompt_any_kernel<DT, 16>;
  kernel<<<(unsigned)blocks, kWaves * 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t prompt_ws_bytes(int dt, int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  return 0;
}

hipError_t launch_prompt_attn(const PromptArgs& a, int dt, void* ws, hipStream_t s) {
  return dt == FK_F32   ? run_any<FK_F32>(a, s)
         : dt == FK_F16 ? run_any<FK_F16>(a, s)
                        : run_any<FK_BF16>(a, s);
}

}  // namespace fk

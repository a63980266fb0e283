// Attention of one new token per request over a paged key-value cache.
//
// Online softmax: a running maximum m, the sum l of e^(s - m) and the sums
// o = sum e^(s - m) v; a new maximum scales l and o by e^(m_old - m_new), and two
// partial results join the same way.
#include <math.h>

#include "fk_kv.hpp"

namespace fk {
namespace {

constexpr int kWaves = 4;

__device__ __forceinline__ float capped(float s, float cap) {
  if (!(cap > 0.f)) return s;
  // tanh(x) = 1 - 2 / (e^(2x) + 1): saturates to +-1 without overflowing to NaN
  return cap * (1.f - 2.f / (__expf(2.f * (s / cap)) + 1.f));
}

// Any size, stride and alignment. One block per (request, query head); a wave
// takes every fourth key, a lane every 64th element of a row.
template <int DT, int EPL>
__global__ __launch_bounds__(kWaves * 64) void attn_any_kernel(AttnArgs a) {
  using E = typename Val<DT>::type;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t b = blockIdx.x / a.Hq, h = blockIdx.x - b * a.Hq;
  const fk_kv_cache_t& c = a.cache;
  const int D = (int)c.dim;
  const int64_t hk = h / (a.Hq / c.heads);
  const E* q = (const E*)a.q + b * a.q_stride[0] + h * a.q_stride[1];
  float qf[EPL], o[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    qf[i] = e < D ? Val<DT>::get(q + e) : 0.f;
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int64_t cap_len = a.width * c.page;
  const int64_t len = a.lens[b] < cap_len ? a.lens[b] : cap_len;
  for (int64_t j = w; j < len; j += kWaves) {
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
    s = capped(wave_sum(s) * a.scale, a.softcap) + bias;
    const float mn = fmaxf(m, s);
    const float alpha = m == -INFINITY ? 0.f : __expf(m - mn);
    const float p = s == -INFINITY ? 0.f : __expf(s - mn);   // a NaN score stays one
    l = l * alpha + p;
    m = mn;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      if (e < D) o[i] = fmaf(p, Val<DT>::get(v + e), o[i] * alpha);
    }
  }
  __shared__ float sm[kWaves], sl[kWaves], so[kWaves][EPL * 64];
  if (lane == 0) sm[w] = m, sl[w] = l;
#pragma unroll
  for (int i = 0; i < EPL; ++i) so[w][lane + 64 * i] = o[i];
  __syncthreads();
  float top = sm[0];
  for (int i = 1; i < kWaves; ++i) top = fmaxf(top, sm[i]);
  float f[kWaves], total = 0.f;
  for (int i = 0; i < kWaves; ++i) {
    f[i] = sl[i] == 0.f ? 0.f : __expf(sm[i] - top);
    total += f[i] * sl[i];
  }
  const bool any = total != 0.f;         // true for NaN: it has to reach the result
  for (int e = threadIdx.x; e < D; e += kWaves * 64) {
    float t = 0.f;
    for (int i = 0; i < kWaves; ++i) t += f[i] * so[i][e];
    Val<DT>::put((E*)a.out + (b * a.Hq + h) * D + e, any ? t / total : 0.f);
  }
  if (a.lse && threadIdx.x == 0) a.lse[b * a.Hq + h] = any ? top + logf(total) : -INFINITY;
}

template <int DT>
hipError_t run_any(const AttnArgs& a, hipStream_t s) {
  const int64_t blocks = a.B * a.Hq;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const int64_t D = a.cache.dim;
  const auto kernel = D <= 64    ? attn_any_kernel<DT, 1>
                      : D <= 128 ? attn_any_kernel<DT, 2>
                      : D <= 256 ? attn_any_kernel<DT, 4>
                                 : attn_any_kernel<DT, 16>;
  kernel<<<(unsigned)blocks, kWaves * 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t attn_ws_bytes(int64_t, int64_t, int64_t, int64_t) { return 256; }

hipError_t launch_paged_attn(const AttnArgs& a, int dt, void*, hipStream_t s) {
  if (a.B == 0) return hipSuccess;
  return dt == FK_F32 ? run_any<FK_F32>(a, s)
         : dt == FK_F16 ? run_any<FK_F16>(a, s)
                        : run_any<FK_BF16>(a, s);
}

}  // namespace fk

// Attention of one new token per request over a paged cache of e4m3 codes.
#include "attn_parts.hpp"
#include "e4m3.hpp"

namespace fk {
namespace {

// Any size, stride and alignment, as attn_any_kernel: one block per (request, query head,
// part of the request's keys), a wave every fourth key, a lane every 64th element.
template <int DT, int EPL>
__global__ __launch_bounds__(kWaves * 64) void attn8_any_kernel(AttnArgs8 a, int parts, float* po,
                                                                float* pml) {
  using E = typename Val<DT>::type;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t bh = blockIdx.x / parts, b = bh / a.Hq, h = bh - b * a.Hq;
  const int part = (int)(blockIdx.x - bh * parts);
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
  const int64_t len = a.lens[b] < 0 ? 0 : (a.lens[b] < cap_len ? a.lens[b] : cap_len);
  const int64_t last = len * (part + 1) / parts;
  for (int64_t j = len * part / parts + w; j < last; j += kWaves) {
    const int64_t page = a.table[b * a.ld_table + j / c.page], tok = j % c.page;
    if (page < 0 || page >= c.pages) continue;
    float bias = 0.f;
    if (c.key_bias) {
      bias = c.key_bias[page * c.bias_stride[0] + tok * c.bias_stride[1] + hk * c.bias_stride[2]];
      if (bias == -INFINITY) continue;
    }
    const uint8_t* k = (const uint8_t*)c.k + page * c.k_stride[0] + tok * c.k_stride[1] + hk * c.k_stride[2];
    const uint8_t* v = (const uint8_t*)c.v + page * c.v_stride[0] + tok * c.v_stride[1] + hk * c.v_stride[2];
    const float ks = a.k_scale[page * a.ks_stride[0] + tok * a.ks_stride[1] + hk * a.ks_stride[2]];
    const float vs = a.v_scale[page * a.vs_stride[0] + tok * a.vs_stride[1] + hk * a.vs_stride[2]];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      if (e < D) s = fmaf(qf[i], e4m3_get(k[e]), s);
    }
    s = wave_sum(s) * ks * a.scale;
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
      if (e < D) o[i] = fmaf(p, e4m3_get(v[e]) * vs, o[i] * alpha);
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
    f[i] = join_factor(sm[i], sl[i], top);
    total += f[i] * sl[i];
  }
  const bool any = total != 0.f;         // true for NaN: it has to reach the result
  for (int e = threadIdx.x; e < D; e += kWaves * 64) {
    float t = 0.f;
    for (int i = 0; i < kWaves; ++i) t += f[i] * so[i][e];
    if (parts > 1) {
      po[(bh * parts + part) * D + e] = t;
    } else {
      Val<DT>::put((E*)a.out + bh * D + e, any ? t / total : 0.f);
    }
  }
  if (threadIdx.x != 0) return;
  if (parts > 1) pml[(bh * parts + part) * 2] = top, pml[(bh * parts + part) * 2 + 1] = total;
  else if (a.lse) a.lse[bh] = any ? top + logf(total) : -INFINITY;
}

template <int DT>
hipError_t run_any(const AttnArgs8& a, int64_t most, void* ws, hipStream_t s) {
  const int parts = most > 128 ? (int)any_parts(a.B, a.Hq) : 1;
  const int64_t heads = a.B * a.Hq, blocks = heads * parts;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const int64_t D = a.cache.dim;
  float* po = (float*)ws;
  float* pml = po + blocks * D;
  const auto kernel = D <= 64    ? attn8_any_kernel<DT, 1>
                      : D <= 128 ? attn8_any_kernel<DT, 2>
                      : D <= 256 ? attn8_any_kernel<DT, 4>
                                 : attn8_any_kernel<DT, 16>;
  kernel<<<(unsigned)blocks, kWaves * 64, 0, s>>>(a, parts, po, pml);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || parts == 1) return e;
  attn_any_join_kernel<DT><<<(unsigned)heads, kWaves * 64, 0, s>>>(a, parts, po, pml);
  return hipGetLastError();
}

}  // namespace

size_t attn8_ws_bytes(int dt, int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  return (size_t)(B * Hq * any_parts(B, Hq)) * (D + 2) * 4;
}

hipError_t launch_paged_attn8(const AttnArgs8& a, int dt, void* ws, hipStream_t s) {
  return dt == FK_F32   ? run_any<FK_F32>(a, longest(a), ws, s)
         : dt == FK_F16 ? run_any<FK_F16>(a, longest(a), ws, s)
                        : run_any<FK_BF16>(a, longest(a), ws, s);
}

}  // namespace fk

// Per-head RMS norm of queries and keys with the position rotation in the same
// pass, keys and values stored to their slots of a paged cache.
#include "fk_kv.hpp"

namespace fk {
namespace {

constexpr int kWaves = 4;

__device__ __forceinline__ int64_t clamp_pos(int64_t p, int64_t n) {
  return p < 0 ? 0 : (p >= n ? n - 1 : p);
}

// One wave per row (token, head); rows 0..Hq-1 of a token are its queries, the
// next Hkv its keys, the next Hkv (with a cache) its values. Any size, stride
// and alignment: a lane takes every 64th element, and reads a rotated
// element's partner from memory again.
template <int DT>
__global__ __launch_bounds__(kWaves * 64) void rope_any_kernel(RopeArgs a, int64_t rows) {
  using E = typename Val<DT>::type;
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (row >= rows) return;
  const bool store = a.cache.k != nullptr;
  const int64_t per = a.Hq + a.Hkv * (store ? 2 : 1);
  const int64_t t = row / per;
  int64_t h = row - t * per;
  const int64_t D = a.D;
  const int kind = h < a.Hq ? 0 : (h < a.Hq + a.Hkv ? 1 : 2);
  h -= kind == 0 ? 0 : (kind == 1 ? a.Hq : a.Hq + a.Hkv);

  int64_t page = 0, tok = 0;
  bool slot_ok = false;
  if (store && kind) {
    const int64_t slot = a.slots[t];
    slot_ok = slot >= 0 && slot < a.cache.pages * a.cache.page;
    if (slot_ok) page = slot / a.cache.page, tok = slot - page * a.cache.page;
  }
  if (kind == 2) {
    if (!slot_ok) return;
    const E* x = (const E*)a.v + t * a.v_stride[0] + h * a.v_stride[1];
    E* y = (E*)a.cache.v + page * a.cache.v_stride[0] + tok * a.cache.v_stride[1] +
           h * a.cache.v_stride[2];
    for (int64_t i = lane; i < D; i += 64) y[i] = x[i];
    return;
  }
  const E* x = kind == 0 ? (const E*)a.q + t * a.q_stride[0] + h * a.q_stride[1]
                         : (const E*)a.k + t * a.k_stride[0] + h * a.k_stride[1];
  const E* w = (const E*)(kind == 0 ? a.q_weight : a.k_weight);
  E* y0 = kind == 0 ? (E*)a.q_out + (t * a.Hq + h) * D
                    : (a.k_out ? (E*)a.k_out + (t * a.Hkv + h) * D : nullptr);
  E* y1 = slot_ok ? (E*)a.cache.k + page * a.cache.k_stride[0] + tok * a.cache.k_stride[1] +
                        h * a.cache.k_stride[2]
                  : nullptr;
  if (kind == 1 && slot_ok && a.cache.key_bias && lane == 0)
    a.cache.key_bias[page * a.cache.bias_stride[0] + tok * a.cache.bias_stride[1] +
                     h * a.cache.bias_stride[2]] = 0.f;
  float r = 1.f;
  if (w) {
    float ss = 0.f;
    for (int64_t i = lane; i < D; i += 64) {
      const float f = Val<DT>::get(x + i);
      ss = fmaf(f, f, ss);
    }
    ss = wave_sum(ss);
    r = 1.f / sqrtf(ss / (float)D + a.eps);
  }
  const int64_t half = a.rot / 2;
  const float* cs = half ? a.rope + clamp_pos(a.positions[t], a.max_pos) * a.rot : nullptr;
  for (int64_t i = lane; i < D; i += 64) {
    float f = Val<DT>::get(x + i) * r;
    if (w) f *= Val<DT>::get(w + i);
    if (i < a.rot) {
      const bool second = a.interleaved ? (i & 1) : i >= half;
      const int64_t j = a.interleaved ? (i ^ 1) : (second ? i - half : i + half);
      const int64_t pair = a.interleaved ? i >> 1 : (second ? i - half : i);
      float g = Val<DT>::get(x + j) * r;
      if (w) g *= Val<DT>::get(w + j);
      const float c = cs[pair], sn = cs[half + pair];
      f = second ? f * c + g * sn : f * c - g * sn;
    }
    if (y0) Val<DT>::put(y0 + i, f);
    if (y1) Val<DT>::put(y1 + i, f);
  }
}

}  // namespace

hipError_t launch_qk_norm_rope(const RopeArgs& a, int dt, hipStream_t s) {
  const int64_t rows = a.T * (a.Hq + a.Hkv * (a.cache.k ? 2 : 1));
  if (rows == 0) return hipSuccess;
  const int64_t blocks = (rows + kWaves - 1) / kWaves;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const auto kernel = dt == FK_F32   ? rope_any_kernel<FK_F32>
                      : dt == FK_F16 ? rope_any_kernel<FK_F16>
                                     : rope_any_kernel<FK_BF16>;
  kernel<<<(unsigned)blocks, kWaves * 64, 0, s>>>(a, rows);
  return hipGetLastError();
}

}  // namespace fk

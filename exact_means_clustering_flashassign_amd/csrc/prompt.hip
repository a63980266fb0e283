// Attention of a step's prompts: rows of any layout, and the choice of kernel.
#include "prompt.hpp"

#include <algorithm>

namespace fk {
namespace {

template <int DT, int EPL>
__global__ __launch_bounds__(kWaves * 64) void prompt_any_kernel(PromptArgs a) {
  const int64_t r = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  const int64_t t = r / a.Hq, b = t < a.T ? request_of(a, t) : -1;
  if (b < 0) return;
  float m, l, o[EPL];
  row_sums<DT, EPL>(a, b, t, r - t * a.Hq, 0, seen_by(a, b, t), m, l, o);
  put_row<DT, EPL>(a, r, m, l, o);
}

template <int DT> hipError_t run_any(const PromptArgs& a, hipStream_t s) {
  const int64_t D = a.cache.dim, blocks = (a.T * a.Hq + kWaves - 1) / kWaves;
  if (blocks > 0xFFFFFF) return hipErrorInvalidConfiguration;        // (fewer than 2^32 threads)
  const auto kernel = D <= 64    ? prompt_any_kernel<DT, 1>
                      : D <= 128 ? prompt_any_kernel<DT, 2>
                      : D <= 256 ? prompt_any_kernel<DT, 4>
                                 : prompt_any_kernel<DT, 16>;
  kernel<<<(unsigned)blocks, kWaves * 64, 0, s>>>(a);
  return hipGetLastError();
}

// Rows the matrix-core kernel can load: whole, aligned 16-byte units.
bool aligned16(const PromptArgs& a, int eb) {
  const fk_kv_cache_t& c = a.cache;
  const int64_t s[] = {a.q_stride[0], a.q_stride[1], c.k_stride[0], c.k_stride[1], c.k_stride[2],
                       c.v_stride[0], c.v_stride[1], c.v_stride[2], c.dim};
  for (int64_t v : s)
    if (v * eb % 16) return false;
  return !(((uintptr_t)a.q | (uintptr_t)c.k | (uintptr_t)c.v | (uintptr_t)a.out) & 15);
}

template <int DT> hipError_t run(const PromptArgs& a, void* ws, hipStream_t s) {
  const int64_t D = a.cache.dim;
  if (D > 256 || !aligned16(a, Val<DT>::bytes)) return run_any<DT>(a, s);
  return D <= 128 ? launch_prompt_narrow<DT>(a, ws, s) : launch_prompt_wide(a, DT, ws, s);
}

}  // namespace

size_t prompt_ws_bytes(int dt, int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  if (D > 256) return 0;
  int64_t parts = most_parts(T, Hq / Hkv, Hkv, 128);
  if (!only_four(dt, (int)D)) parts = std::max(parts, most_parts(T, Hq / Hkv, Hkv, 256));
  return parts == 1 ? 0 : (size_t)(parts * T * Hq) * (D + 2) * 4;
}

hipError_t launch_prompt_attn(const PromptArgs& a, int dt, void* ws, hipStream_t s) {
  return dt == FK_F32   ? run<FK_F32>(a, ws, s)
         : dt == FK_F16 ? run<FK_F16>(a, ws, s)
                        : run<FK_BF16>(a, ws, s);
}

}  // namespace fk

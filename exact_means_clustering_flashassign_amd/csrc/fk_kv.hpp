// Declarations shared by the paged key-value-cache units (tables, norm +
// rotation, attention) and their API layer.
#pragma once

#include "fk_internal.hpp"

namespace fk {

// Element i of a dt array, widened to fp32 (exact), and back (nearest-even).
template <int DT> struct Val;
template <> struct Val<FK_F32> {
  using type = float;
  using arith = float;      // the type as the compiler's conversions know it
  static constexpr int bytes = 4;
  __device__ static __forceinline__ float get(const float* p) { return *p; }
  __device__ static __forceinline__ void put(float* p, float f) { *p = f; }
};
template <> struct Val<FK_F16> {
  using type = uint16_t;
  using arith = _Float16;
  static constexpr int bytes = 2;
  __device__ static __forceinline__ float get(const uint16_t* p) { return f16_bits_to_f32(*p); }
  __device__ static __forceinline__ void put(uint16_t* p, float f) { *p = f32_to_f16_bits(f); }
};
template <> struct Val<FK_BF16> {
  using type = uint16_t;
  using arith = __bf16;
  static constexpr int bytes = 2;
  __device__ static __forceinline__ float get(const uint16_t* p) { return bf16_bits_to_f32(*p); }
  __device__ static __forceinline__ void put(uint16_t* p, float f) {
    // the integer rounding would carry a NaN's payload into infinity
    *p = f == f ? f32_to_bf16_bits(f) : (uint16_t)0x7FC0;
  }
};

// n / d for n < 2^31 by a multiplication (Granlund and Montgomery's method).
struct FastDiv {
  uint32_t mul, shift, d;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while (((uint64_t)1 << l) < d) ++l;
  return {(uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << l) - d)) / d + 1), l, d};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv& f) {
  return (__umulhi(n, f.mul) + n) >> f.shift;
}

struct TablesArgs {
  const int32_t *len_old, *len_new, *table_in, *free_pages;
  int64_t width_in, n_free, B, page, width, tokens;
  int32_t *table, *lens, *cu_tokens, *cu_pages, *slots, *positions;
};
hipError_t launch_page_tables(const TablesArgs& a, hipStream_t s);

struct RopeArgs {
  const void *q, *k, *v;
  int64_t q_stride[2], k_stride[2], v_stride[2];
  int64_t T, Hq, Hkv, D;
  const void *q_weight, *k_weight;
  float eps;
  const float* rope;
  int64_t max_pos, rot;
  int interleaved;
  const int32_t *positions, *slots;
  fk_kv_cache_t cache;   // k null: nothing is stored
  void *q_out, *k_out;
};
hipError_t launch_qk_norm_rope(const RopeArgs& a, int dt, hipStream_t s);

struct AttnArgs {
  const void* q;
  int64_t q_stride[2];
  int64_t B, Hq;
  fk_kv_cache_t cache;
  const int32_t* table;
  int64_t ld_table, width;
  const int32_t* lens;
  int64_t max_len;
  float scale, softcap;
  void* out;
  float* lse;
};
constexpr int64_t kAttnMaxDim = 1024;
size_t attn_ws_bytes(int dt, int64_t B, int64_t Hq, int64_t Hkv, int64_t D);
hipError_t launch_paged_attn(const AttnArgs& a, int dt, void* ws, hipStream_t s);


// The 8-bit cache: k and v of `cache` are e4m3 codes.
struct AttnArgs8 : AttnArgs {
  const float *k_scale, *v_scale;
  int64_t ks_stride[3], vs_stride[3];
};
size_t attn8_ws_bytes(int dt, int64_t B, int64_t Hq, int64_t Hkv, int64_t D);
hipError_t launch_paged_attn8(const AttnArgs8& a, int dt, void* ws, hipStream_t s);

struct Cache8Args {
  const void *k, *v;          // store: rows in
  int64_t k_stride[2], v_stride[2];
  int64_t T;
  const int32_t* slots;
  fk_kv_cache8_t cache;
  void *k_out, *v_out;        // load: rows out
};
hipError_t launch_kv_store8(const Cache8Args& a, int dt, hipStream_t s);
hipError_t launch_kv_load8(const Cache8Args& a, int dt, hipStream_t s);

struct PromptArgs {
  const void* q;
  int64_t q_stride[2];
  int64_t T, B, Hq;
  fk_kv_cache_t cache;
  const int32_t* table;
  int64_t ld_table, width;
  const int32_t *lens, *cu;
  int64_t max_len;
  float scale, softcap;
  void* out;
  float* lse;
};
size_t prompt_ws_bytes(int dt, int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D);
hipError_t launch_prompt_attn(const PromptArgs& a, int dt, void* ws, hipStream_t s);
// rows of up to 128 elements (a unit for each type), and of 129 to 256
template <int DT> hipError_t launch_prompt_narrow(const PromptArgs& a, void* ws, hipStream_t s);
template <> hipError_t launch_prompt_narrow<FK_F16>(const PromptArgs& a, void* ws, hipStream_t s);
template <> hipError_t launch_prompt_narrow<FK_BF16>(const PromptArgs& a, void* ws, hipStream_t s);
template <> hipError_t launch_prompt_narrow<FK_F32>(const PromptArgs& a, void* ws, hipStream_t s);
hipError_t launch_prompt_wide(const PromptArgs& a, int dt, void* ws, hipStream_t s);

}  // namespace fk

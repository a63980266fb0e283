// What the attention kernels share: the softmax's arithmetic, loads by address,
// the sharing-out of requests of any lengths and the joining of partial results.
#pragma once

#include <math.h>

#include "fk_kv.hpp"

namespace fk {
namespace {

constexpr int kWaves = 4;

// Blocks of so many waves that a launch may have: fewer than 2^32 threads.
constexpr int64_t most_blocks(int waves) { return 0xFFFFFFFF / (waves * 64); }

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLog2eRest = 1.92596299112661746887e-8f;    // log2 e - kLog2e
constexpr float kLn2 = 0.69314718055994530942f;

// cap * tanh(s / cap) to a few units in the last place of its own size (scores of a few
// units under a cap of tens must not carry the cap's rounding): below 1 the
// quotient of Lambert's continued fraction cut after six terms (4e-10 off at 1), above
// it (e^2x - 1) / (e^2x + 1), where the difference loses nothing.
__device__ __forceinline__ float capped(float s, float cap, float inv_cap) {
  const float x = fminf(fmaxf(s * inv_cap, -20.f), 20.f), y = x * x;
  const float e = fast_exp2(x * (2.f * kLog2e));
  const bool small = y < 1.f;
  const float num = small ? x * fmaf(fmaf(21.f, y, 1260.f), y, 10395.f) : e - 1.f;
  const float den = small ? fmaf(fmaf(y + 210.f, y, 4725.f), y, 10395.f) : e + 1.f;
  const float r = cap * (num * __builtin_amdgcn_rcpf(den));
  return s == s ? r : s;     // the clamp drops a NaN
}

// cap * tanh(s / cap) within 2^-21 of the cap, a third of capped()'s instructions: for 16-bit types up
// to a cap of kNearCap, where that is at most 2^-15 of a weight, an eighth of the least that half a step of
// fp16 can be. Under a larger cap it would show. (8192 tokens, 32 heads of 128 on 8, bf16: 804 us, with
// capped() 1175; 32 requests of up to 8192 keys in 8 bits, the same heads: 68 and 70.)
constexpr float kNearCap = 64.f;
__device__ __forceinline__ float cap_16bit(float s, float cap, float inv_cap) {
  const float e = fast_exp2(s * (inv_cap * (2.f * kLog2e)));
  return fmaf(-2.f * cap, __builtin_amdgcn_rcpf(e + 1.f), cap);
}

// Scale of a partial result (m, l) under the common maximum.
__device__ __forceinline__ float join_factor(float m, float l, float top) {
  return l == 0.f ? 0.f : fast_exp2((m - top) * kLog2e);
}

// A sum in 32 bits of n terms alike may be off by n 2^-25 of itself, and stands still after 2^24: kernels that
// add one key at a time put their sums away every kKeyRun keys, in LDS (`at`, every 64th float the
// lane's; in registers rows of 512 elements took 15% longer), scaled to the maximum m of then.
constexpr int kKeyRun = 1 << 12;
template <int EPL> struct Runs {
  float* at;
  bool any = false;
  float m = -INFINITY, l = 0.f;
  __device__ __forceinline__ void add(float now, float& l_now, float (&o)[EPL]) {
    join(now, l_now, o);
    any = true, m = now, l = l_now, l_now = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) at[64 * i] = o[i], o[i] = 0.f;
  }
  // What has been put away, added to the sums since then, whose maximum is `now`.
  __device__ __forceinline__ void join(float now, float& l_now, float (&o)[EPL]) {
    if (!any) return;
    const float f = m == now ? 1.f : fast_exp2((m - now) * kLog2e);
    l_now = fmaf(l, f, l_now);
#pragma unroll
    for (int i = 0; i < EPL; ++i) o[i] = fmaf(at[64 * i], f, o[i]);
  }
};

constexpr int kAnyParts = 64;

// Joins the parts of one (request, query head).
template <int DT>
__global__ __launch_bounds__(kWaves * 64) void attn_any_join_kernel(AttnArgs a, int parts,
                                                                    const float* po,
                                                                    const float* pml) {
  const int64_t bh = blockIdx.x;
  const int D = (int)a.cache.dim;
  const float* ml = pml + bh * parts * 2;
  float top = -INFINITY, total = 0.f;
  for (int i = 0; i < parts; ++i) top = fmaxf(top, ml[2 * i]);
  for (int i = 0; i < parts; ++i)
    total = fmaf(join_factor(ml[2 * i], ml[2 * i + 1], top), ml[2 * i + 1], total);
  const bool any = total != 0.f;
  for (int e = threadIdx.x; e < D; e += kWaves * 64) {
    float t = 0.f;
    for (int i = 0; i < parts; ++i)
      t = fmaf(join_factor(ml[2 * i], ml[2 * i + 1], top), po[(bh * parts + i) * D + e], t);
    Val<DT>::put((typename Val<DT>::type*)a.out + bh * D + e, any ? t / total : 0.f);
  }
  if (a.lse && threadIdx.x == 0) a.lse[bh] = any ? top + logf(total) : -INFINITY;
}

// Parts of a request there: 2048 blocks over all, at most kAnyParts.
int64_t any_parts(int64_t B, int64_t Hq) {
  const int64_t n = B * Hq >= 2048 ? 1 : 2048 / (B * Hq > 0 ? B * Hq : 1);
  return n < kAnyParts ? n : kAnyParts;
}

// Keys of the longest request, at most: what the tables hold, or the caller's bound.
template <class Args> int64_t longest(const Args& a) {
  int64_t most = a.width * a.cache.page;
  if (most > 0x7FFFFFFF) most = 0x7FFFFFFF;
  return a.max_len > 0 && a.max_len < most ? a.max_len : most;
}

constexpr int kHeadTile = 16;
constexpr int kMaxCus = 256;

// A value that is the same in every lane, moved to scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Loads by address: the address space is stated, so that they are global loads
// and not generic ones, which the LDS counter would wait for too.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float floatx2_t __attribute__((ext_vector_type(2)));
typedef const __attribute__((address_space(1))) u32x4* gptr16;
typedef const __attribute__((address_space(1))) u32x2* gptr8;
typedef const __attribute__((address_space(1))) uint32_t* gptr4;
typedef const __attribute__((address_space(1))) int32_t* gptr_i32;
typedef const __attribute__((address_space(1))) float* gptr_f32;

__device__ __forceinline__ uint4 load16(uint64_t addr) {
  return __builtin_bit_cast(uint4, *(gptr16)addr);
}

// A load of n = 16, 8 or 4 bytes into the first words. STREAM: bytes that no one else
// reads are marked so and do not push out of L2 what others will read again (the 4.43 GB
// of 32 requests of 2048 to 65536 keys 815 -> 779 us); where waves share lines the mark makes them come twice (8 x 32768
// keys, 8 heads of 80: 200 us marked, 137 plain, 132 now).
template <int n, bool STREAM> __device__ __forceinline__ uint4 load_row(uint64_t addr) {
  if constexpr (n == 16) {
    return __builtin_bit_cast(uint4, STREAM ? __builtin_nontemporal_load((gptr16)addr) : *(gptr16)addr);
  } else if constexpr (n == 8) {
    const u32x2 h = STREAM ? __builtin_nontemporal_load((gptr8)addr) : *(gptr8)addr;
    return make_uint4(h.x, h.y, 0, 0);
  } else {
    return make_uint4(STREAM ? __builtin_nontemporal_load((gptr4)addr) : *(gptr4)addr, 0, 0, 0);
  }
}

// Keys that do not count are read from here: zeros, whatever the cache holds.
__device__ const uint4 zero_row[64] = {};

// How the work is shared. Request b costs its steps plus one step of each wave of its
// team (queries, first loads, joining, storing). The requests' costs are laid end to
// end and cut into equal parts, as many as the chip holds teams for each head, so that a
// batch of any lengths fills the chip evenly. A request inside one part is finished
// there; one that is cut leaves a partial result per part, at most two a part (one that
// started before, one that goes on), joined by attn_join_kernel. A larger share for a
// request's start was slower (one step 54.6, two 55.7, four 57.7 us for 32 requests
// of 0 to 16384 keys spread over the logarithm, 8 heads of 128).
struct Plan {
  int parts;            // blocks per (cache head, head tile); 0: a team per request
  int team, team_log;   // waves that share a request's steps: 8, 4, 2 or 1
  int heads, tiles;     // cache heads, head tiles per cache head
  int G, width, hr;     // query heads per cache head, per head tile, and per tile at most
  FastDiv page, by_tiles, by_heads;
  float* o;             // (parts, heads, tiles, 2, hr, D) partial sums
  float* ml;            // (parts, heads, tiles, 2, hr, 2) their maximum and sum
  int32_t* cover;       // (B, 2) first and last part of a request
};

__device__ __forceinline__ int len_of(const AttnArgs& a, int64_t b) {
  const int64_t cap = a.width * a.cache.page;
  const int n = a.lens[b];
  return n <= 0 ? 0 : (n < cap ? n : (int)cap);
}

// Steps of a request; a length may be 2^31 - 1, so the sum is unsigned.
template <int KEYS> __device__ __forceinline__ int steps_of(int len) {
  return (int)(((uint32_t)len + KEYS - 1) / KEYS);
}

template <int DT> struct Mfma16;
template <> struct Mfma16<FK_F16> {
  __device__ static __forceinline__ floatx4_t run(uint4 a, uint4 b, floatx4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a),
                                                  __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
  }
};
template <> struct Mfma16<FK_BF16> {
  __device__ static __forceinline__ floatx4_t run(uint4 a, uint4 b, floatx4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  }
};
// fp32: element j of the lanes' 16 bytes in turn, four k per product.
template <> struct Mfma16<FK_F32> {
  __device__ static __forceinline__ floatx4_t run(uint4 a, uint4 b, floatx4_t c) {
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, a.x),
                                             __builtin_bit_cast(float, b.x), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, a.y),
                                             __builtin_bit_cast(float, b.y), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, a.z),
                                             __builtin_bit_cast(float, b.z), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, a.w),
                                                __builtin_bit_cast(float, b.w), c, 0, 0, 0);
  }
};

// fp16 probabilities are scaled by 2^14, so that one 2^-38 of the largest is
// still a subnormal fp16 and a long tail of small ones is not lost.
template <int DT> constexpr float kProbShift = DT == FK_F16 ? 14.f : 0.f;

// e^x (x <= 0), scaled. 16-bit caches: x log2 e is rounded once, |x| 2^-24 of the result, less
// than a probability's own rounding. fp32: the whole part is taken off before that
// rounding, and the constant's own rest added.
template <int DT> __device__ __forceinline__ float prob(float x) {
  if constexpr (DT != FK_F32) return fast_exp2(fmaf(x, kLog2e, kProbShift<DT>));
  const float n = rintf(fmaxf(x, -200.f) * kLog2e);
  const float f = fmaf(x, kLog2eRest, fmaf(x, kLog2e, -n));
  return x < -200.f ? 0.f : __builtin_amdgcn_ldexpf(fast_exp2(f), (int)n);
}

// Eight numbers x >= 0 as hi + lo in 16 bits each: hi is x rounded down, lo the rest to
// nearest but at least the smallest number that a product does not flush, 2^-126 (bf16) or
// 2^-24 (fp16, 2^-38 of the largest probability); x = 0 gives 0 and 0.
template <int DT> struct Halves {
  typedef typename Val<DT>::arith T;
  typedef T T2 __attribute__((ext_vector_type(2)));
  static constexpr float tiny = DT == FK_F16 ? 0x1p-24f : 0x1p-126f;
  __device__ static __forceinline__ void split(const float (&x)[8], uint4& hi, uint4& lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      float ra, rb;
      if constexpr (DT == FK_F16) {
        const auto d = __builtin_amdgcn_cvt_pkrtz(a, b);
        h[i] = __builtin_bit_cast(uint32_t, d);
        ra = a - (float)d[0], rb = b - (float)d[1];
      } else {
        const uint32_t ua = __builtin_bit_cast(uint32_t, a), ub = __builtin_bit_cast(uint32_t, b);
        h[i] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
        ra = a - __builtin_bit_cast(float, ua & 0xFFFF0000u);
        rb = b - __builtin_bit_cast(float, ub & 0xFFFF0000u);
      }
      const T2 d = {(T)fmaxf(ra, a == 0.f ? 0.f : tiny), (T)fmaxf(rb, b == 0.f ? 0.f : tiny)};
      l[i] = __builtin_bit_cast(uint32_t, d);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]), lo = make_uint4(l[0], l[1], l[2], l[3]);
  }
};

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
}

// Where part `w` of the flattened costs starts: request and cost before it.
// Every block finds out by itself: thread i adds up requests [i n, (i + 1) n).
struct Start {
  int64_t lo, hi;            // this part's range of costs
  int64_t b, before;         // request that holds lo, cost of those before it
  // Part w of the parts in use: floor(total w / parts) on, in 32-bit divisions where the
  // total allows (a 64-bit one is some 150 instructions of a call's first microsecond).
  __device__ __forceinline__ void cut(int64_t total, const Plan& p, int w) {
    const int64_t most = total >> p.team_log;      // a part is a step of each wave at least
    const uint32_t parts = most < 1 ? 1 : (uint32_t)min(most, (int64_t)p.parts);
    if (w >= (int)parts) {
      lo = hi = total;
      return;
    }
    const int64_t q = total >> 32 ? total / parts : (int64_t)((uint32_t)total / parts);
    const uint32_t r = (uint32_t)(total - q * parts);
    lo = q * w + r * w / parts;
    hi = q * (w + 1) + r * (w + 1) / parts;
  }
};

template <int KEYS>
__device__ __forceinline__ int64_t cost_of(const AttnArgs& a, const Plan& p, int64_t b) {
  return p.team + steps_of<KEYS>(len_of(a, b));
}

template <int KEYS>
__device__ __forceinline__ Start find_start(const AttnArgs& a, const Plan& p, int w) {
  Start st;
  if (a.B <= 64 && a.width * a.cache.page <= (1 << 29)) {
    // a request a lane, every wave by itself, without barriers; 64 costs of at most
    // 2^29 / 16 + 4 fit 32 bits
    const int lane = threadIdx.x & 63;
    const uint32_t mine = lane < a.B ? (uint32_t)cost_of<KEYS>(a, p, lane) : 0;
    uint32_t incl = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t o = __shfl_up(incl, off, 64);
      if (lane >= off) incl += o;
    }
    st.cut((uint32_t)__builtin_amdgcn_readlane(incl, 63), p, w);
    const int b = __popcll(__ballot(incl <= st.lo));      // requests that end at or before lo
    st.b = b;
    st.before = b ? (uint32_t)__builtin_amdgcn_readlane(incl, b - 1) : 0;
    return st;
  }
  __shared__ int64_t wave_tot[kWaves];
  __shared__ int64_t found[2];
  const int64_t n = (a.B + kWaves * 64 - 1) / (kWaves * 64);
  const int64_t b0 = threadIdx.x * n, b1 = b0 + n < a.B ? b0 + n : a.B;
  int64_t mine = 0;
#pragma unroll 8
  for (int64_t b = b0; b < b1; ++b) mine += cost_of<KEYS>(a, p, b);
  int64_t incl = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t o = __shfl_up(incl, off, 64);
    if ((int)(threadIdx.x & 63) >= off) incl += o;
  }
  if ((threadIdx.x & 63) == 63) wave_tot[threadIdx.x >> 6] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i < (int)(threadIdx.x >> 6)) before += wave_tot[i];
    total += wave_tot[i];
  }
  st.cut(total, p, w);
  if (st.lo >= before && st.lo < before + mine) {
    int64_t b = b0, at = before;
    for (int64_t c = cost_of<KEYS>(a, p, b); at + c <= st.lo; c = cost_of<KEYS>(a, p, b)) at += c, ++b;
    found[0] = b;
    found[1] = at;
  }
  __syncthreads();
  st.b = found[0];
  st.before = found[1];
  return st;
}

template <int DT>
__device__ __forceinline__ void store4(void* out, int64_t at, const float* x) {
  if constexpr (DT == FK_F32) {
    *(float4*)((float*)out + at) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
    typedef typename Val<DT>::arith T;
    typedef T T4 __attribute__((ext_vector_type(4)));
    T4 v = {(T)x[0], (T)x[1], (T)x[2], (T)x[3]};
    *(T4*)((T*)out + at) = v;
  }
}

// Waves a SIMD holds (by their registers). The parts of a call are as many as the chip
// holds blocks at once.
constexpr int waves_per_simd(int64_t D) {
  return D <= 32 ? 4 : (D <= 64 ? 3 : (D <= 128 ? 2 : 1));
}
constexpr int kMaxParts = kMaxCus * 4;

// Rows narrower than the tile, rows that fill it, and rows that fill it and whole
// 128-byte lines that no other wave reads, by streaming loads.
enum { kNarrow, kWhole, kStream };

// State of one wave over a run of steps.
template <class S, int HT> struct Acc {
  float m[HT], l[HT];                  // of lane m's head of each tile; l: this lane's share
  floatx4_t o[HT][S::nu * S::ve];
};

// The kernel around an operator Op, which says how a wave attends to a run of steps (Op::attend)
// and in what shape (Op::S).
template <class Op, int KIND, int W>
__global__ __launch_bounds__(W * 64, W == kWaves ? waves_per_simd(Op::DP) : W / 4)
void attn_mfma_kernel(typename Op::Args a, Plan p) {
  using S = typename Op::S;
  constexpr int DT = Op::DT, DP = Op::DP, HT = Op::HT;
  __shared__ typename Op::Rows rows[W][2];
  __shared__ float so[W][kHeadTile][S::ldo];
  __shared__ float sm[W][kHeadTile], sl[W][kHeadTile];
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Waves k0 .. k1 - 1 of this block are one team; its teams take neighbouring heads.
  const int k0 = w >> p.team_log << p.team_log, k1 = k0 + p.team, teams = W >> p.team_log;
  const uint32_t unit =
      (uint32_t)xcd_remap(blockIdx.x, gridDim.x) * teams + (w >> p.team_log);
  const uint32_t rest = div_by(unit, p.by_tiles), at_head = div_by(rest, p.by_heads);
  const int ht = (int)(unit - rest * p.tiles), hk = (int)(rest - at_head * p.heads);
  const int64_t part = at_head;
  const int D = KIND == kNarrow ? (int)a.cache.dim : DP;

  Start st;
  const bool cut = W == kWaves && p.parts > 0;
  if (cut) {
    // the same for the block: held in scalar registers through the steps, which
    // have none to spare among the others
    st = find_start<S::keys>(a, p, (int)part);
    st.lo = uniform(st.lo), st.hi = uniform(st.hi);
    st.b = uniform(st.b), st.before = uniform(st.before);
    if (st.lo >= st.hi) return;
  } else {
    st.lo = 0, st.hi = 1, st.b = part, st.before = 0;
  }
  const bool idle = !cut && part >= a.B;     // a wave past the last request
  for (int64_t b = st.b, at = st.before; at < st.hi;) {
    const int len = idle ? 0 : __builtin_amdgcn_readfirstlane(len_of(a, b));
    const int steps = steps_of<S::keys>(len);
    int t0 = 0, t1 = steps;
    if (cut) {
      const int64_t first = at + p.team;
      t0 = (int)max((int64_t)0, min(st.lo - first, (int64_t)steps));
      t1 = (int)max((int64_t)0, min(st.hi - first, (int64_t)steps));
    }
    const bool starts = at >= st.lo;           // the request begins in this part
    if (t0 < t1 || (steps == 0 && starts)) {
      Acc<S, HT> acc;
      Op::template attend<KIND>(a, p, b, hk, ht, len, t0 + w - k0, p.team, t1, rows[w], acc);
      const bool whole = t0 == 0 && t1 == steps;
      const int slot = t0 == 0 ? 1 : 0;
      const int64_t ps = (((part * p.heads + hk) * p.tiles + ht) * 2 + slot) * p.hr;
#pragma unroll
      for (int h2 = 0; h2 < HT; ++h2) {
        const int h0 = (ht * HT + h2) * kHeadTile;        // first head of this tile
        const int nh = min(kHeadTile, p.G - h0);
        __syncthreads();                       // the last results are out
        if (m < nh) {
          if (g == 0) sm[w][m] = acc.m[h2], sl[w][m] = acc.l[h2];
#pragma unroll
          for (int u = 0; u < S::nu; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int t = 0; t < S::ve; ++t)
                so[w][m][u * 16 * S::ve + S::ve * (4 * g + i) + t] = acc.o[h2][u * S::ve + t][i];
        }
        __syncthreads();
        for (int i = threadIdx.x - k0 * 64; i < nh * (DP / 4) && !idle; i += p.team * 64) {
          const int h = i / (DP / 4), e = (i - h * (DP / 4)) * 4;
          float top = -INFINITY;
          for (int k = k0; k < k1; ++k) top = fmaxf(top, sm[k][h]);
          float x[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
          for (int k = k0; k < k1; ++k) {
            const float f = join_factor(sm[k][h], sl[k][h], top);
            l = fmaf(f, sl[k][h], l);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = fmaf(f, so[k][h][e + j], x[j]);
          }
          if (e >= D) continue;
          if (whole) {
            const int64_t row = b * a.Hq + hk * p.G + h0 + h;
            const float r = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] *= r;
            store4<DT>(a.out, row * D + e, x);
            if (e == 0 && a.lse)
              a.lse[row] = l == 0.f ? -INFINITY : top + (logf(l) - kProbShift<Op::PT> * kLn2);
          } else {
            const int64_t pr = ps + h2 * kHeadTile + h;
            *(float4*)(p.o + pr * D + e) = make_float4(x[0], x[1], x[2], x[3]);
            if (e == 0) p.ml[pr * 2] = top, p.ml[pr * 2 + 1] = l;
          }
        }
      }
      if (cut && hk == 0 && ht == 0 && threadIdx.x == 0) {
        if (t0 == 0) p.cover[2 * b] = (int32_t)part;
        if (t1 == steps) p.cover[2 * b + 1] = (int32_t)part;
      }
    }
    if (!cut) break;
    at += p.team + steps;
    ++b;
  }
}

constexpr int kJoin = 256;        // threads of a joining block

// Joins the partial results of a request that was cut: slot 1 of its first part,
// slot 0 of the others. R (request, query head) rows a block: one a wave, or one whose
// columns are dealt to `slices` blocks. Bound by latency: the parts' numbers, their
// maxima and sums, then the rows. Probabilities are scaled as those of type PT.
template <int DT, int PT, int R>
__global__ __launch_bounds__(kJoin) void attn_join_kernel(AttnArgs a, Plan p, int slices) {
  constexpr int threads = kJoin / R;
  __shared__ float fac[R][kMaxParts], part_l[R][kMaxParts];
  __shared__ float red[kJoin][4], redl[kJoin];
  const int me = R == 1 ? 0 : threadIdx.x / threads, tid = threadIdx.x - me * threads;
  const int slice = R == 1 ? blockIdx.x % slices : 0;
  const int64_t out_row = R == 1 ? blockIdx.x / slices : blockIdx.x * R + me;
  if (out_row >= a.B * a.Hq) return;
  const int64_t b = (uint32_t)out_row / (uint32_t)a.Hq;
  const int h = (int)(out_row - b * a.Hq);
  const int first = p.cover[2 * b], last = p.cover[2 * b + 1];
  if (first == last) return;
  const auto sync = [] {
    if constexpr (R == 1) __syncthreads();
    else __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");      // a row is one wave's
  };
  const int hk = h / p.G, ht = (h % p.G) / p.width, hr = (h % p.G) % p.width;
  const int D = (int)a.cache.dim, n = last - first + 1;
  auto row = [&](int i) {
    const int64_t part = first + i;
    return (((part * p.heads + hk) * p.tiles + ht) * 2 + (i == 0 ? 1 : 0)) * p.hr + hr;
  };
  // every thread: maximum over all parts; factors and the sum of the parts' sums
  float top = -INFINITY;
  for (int i = tid & 63; i < n; i += 64) top = fmaxf(top, p.ml[row(i) * 2]);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
  for (int i = tid; i < n; i += threads) {
    const float2 ml = *(const float2*)(p.ml + row(i) * 2);
    fac[me][i] = join_factor(ml.x, ml.y, top);
    part_l[me][i] = ml.y;
  }
  sync();
  // threads: the slice's columns, four each, by as many groups of partial results as fit
  const int cols = (D / 4 + slices - 1) / slices, groups = threads / cols;
  const int grp = tid / cols, e = (slice * cols + tid - grp * cols) * 4;
  float x[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
  if (grp < groups && e < D) {
#pragma unroll 4
    for (int i = grp; i < n; i += groups) {
      const float f = fac[me][i];
      const float4 v = *(const float4*)(p.o + row(i) * D + e);
      l = fmaf(f, part_l[me][i], l);
      x[0] = fmaf(f, v.x, x[0]);
      x[1] = fmaf(f, v.y, x[1]);
      x[2] = fmaf(f, v.z, x[2]);
      x[3] = fmaf(f, v.w, x[3]);
    }
  }
  for (int g = groups; g > 1;) {            // the upper half of the groups into the lower
    const int h = (g + 1) / 2;
    if (grp >= h && grp < g) {
#pragma unroll
      for (int j = 0; j < 4; ++j) red[threadIdx.x][j] = x[j];
      redl[threadIdx.x] = l;
    }
    sync();
    if (grp < g - h) {
      l += redl[threadIdx.x + h * cols];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] += red[threadIdx.x + h * cols][j];
    }
    g = h;                                  // (what was read is not written again)
  }
  if (tid >= cols || e >= D) return;
  const float r = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] *= r;
  store4<DT>(a.out, out_row * D + e, x);
  if (e == 0 && a.lse)
    a.lse[out_row] = l == 0.f ? -INFINITY : top + (logf(l) - kProbShift<PT> * kLn2);
}

// Query heads a wave serves at once: 32 where there are more than 16 and the registers
// hold both tiles (16-bit rows of at most 128; 8 requests of 32768 keys, 8 heads of 64 with
// 32 query heads each: 109 us, 4.9 TB/s; 4 heads of 128: 107 us, 5.0).
int64_t tile_width(int dt, int64_t D, int64_t G) {
  return G > kHeadTile && dt != FK_F32 && D <= 128 ? 2 * kHeadTile : kHeadTile;
}

// Parts per (cache head, head tile): `blocks` shared out.
int64_t parts_of(int64_t blocks, int64_t units) { return units >= blocks ? 1 : blocks / units; }

int64_t chip_blocks(int64_t cus, int64_t D) {
  return (cus < kMaxCus ? cus : kMaxCus) * waves_per_simd(D) * 4 / kWaves;
}

// Waves a head when requests are cut: the block's waves take as many neighbouring
// heads as divide them evenly.
int team_of(int64_t units) { return units % 4 == 0 ? 1 : (units % 2 == 0 ? 2 : 4); }

// How a call is run.
struct Choice {
  Plan p;
  bool cut, eight;      // requests cut into parts; blocks of 8 waves, else of kWaves
  int W;
  int64_t most, blocks; // (0 blocks: too many for a launch)
};

// keys: of a wave's step; HT head tiles a wave; DP: elements of a row's tile.
inline Choice choose(const AttnArgs& a, int keys, int HT, int DP, void* ws) {
  Choice c{};
  Plan& p = c.p;
  p.heads = (int)a.cache.heads;
  p.G = (int)(a.Hq / a.cache.heads);
  p.width = HT * kHeadTile;
  p.tiles = (p.G + p.width - 1) / p.width;
  p.hr = p.G < p.width ? p.G : p.width;
  p.page = fast_div((uint32_t)a.cache.page);
  const int64_t units = (int64_t)p.heads * p.tiles;
  const int64_t most = c.most = longest(a);
  // Cutting costs a second launch and a trip through memory. Up to 512 keys a request is
  // done faster whole (32 requests of 400 keys: 14.7 us, cut 21.4), unless there are
  // many, whose lengths may differ: one wave each is best up to 8 steps, and beyond that
  // cutting evens them out (256 requests up to 512 keys, spread over the logarithm: 35 us
  // cut, 50 whole; all alike: 91 and 87).
  const int64_t resident = chip_blocks(device_cus(), DP);
  const bool many = units * a.B >= 2 * resident;
  // Where every block has a CU to itself and half the CUs have one, 8 waves do up to 64 steps
  // whole (6 requests of 607 keys, 32 heads of 64: 12.6 us, cut 20.9; 16 of 1500, 8 heads of
  // 128: 23 and 27). With fewer blocks a CU's own rate is the bound, and more of them the
  // remedy (4 of 2000, 8 heads: 26, cut 17).
  const int64_t cus = device_cus(), rows = units * a.B;
  const bool eight = c.eight = DP <= 128 && most > 512 && most <= 64 * keys &&
                     rows <= cus && 2 * rows >= cus;
  const bool cut = c.cut = !eight && (most > 512 || (many && most > 8 * keys));
  if (cut) {
    // Where there are steps enough for every wave of the chip, a block's waves take
    // neighbouring heads, whose rows lie side by side in the cache, instead of one
    // head's steps in turn: the block reads 4 rows' length in one piece (the 4.43 GB
    // above: 774 us with 1 head a block, 697 with 2, 670 with 4). With fewer steps the
    // waves share them and join in LDS, not through memory.
    const double steps = (double)units * a.B * ((most + keys - 1) / keys);
    p.team = steps >= 4.0 * kWaves * resident ? team_of(units) : kWaves;
    const int64_t groups = units * p.team / kWaves;       // blocks that make one part
    p.parts = (int)parts_of(resident, groups);
    const int64_t slots = units * p.parts * 2 * p.hr;
    char* w = (char*)ws;
    p.o = (float*)w;
    p.ml = (float*)(w + slots * a.cache.dim * 4);
    p.cover = (int32_t*)(w + slots * a.cache.dim * 4 + slots * 8);
  } else {
    // One wave each where that alone fills the chip, or where a second wave would
    // find nothing to do (222 requests of 3 keys, 32 heads: 19 us, 40 with four waves).
    p.team = eight ? 8 : (many || most <= keys ? 1 : kWaves);
  }
  const int W = c.W = eight ? 8 : kWaves;
  p.team_log = p.team == 8 ? 3 : (p.team == 4 ? 2 : p.team - 1);
  p.by_tiles = fast_div((uint32_t)p.tiles);
  p.by_heads = fast_div((uint32_t)p.heads);
  const int64_t blocks = (units * (cut ? p.parts : a.B) * p.team + W - 1) / W;
  const bool joined = !cut || (a.B * a.Hq + 3) / 4 <= most_blocks(kWaves);      // (join_parts)
  if (units * a.B + W <= 0x7FFFFFFF && joined && blocks <= most_blocks(W)) c.blocks = blocks;
  return c;
}

// Joins what a call cut.
template <int DT, int PT> hipError_t join_parts(const AttnArgs& a, const Plan& p, hipStream_t s) {
  const int64_t cus = device_cus();
  // Many rows: most were not cut or have few parts, and a wave is enough for one.
  const int64_t outs = a.B * a.Hq;
  if (outs >= 8 * cus) {
    attn_join_kernel<DT, PT, 4><<<(unsigned)((outs + 3) / 4), kJoin, 0, s>>>(a, p, 1);
    return hipGetLastError();
  }
  // Few rows have many parts: as many blocks a row as there are CUs for, down to 64 bytes
  // of a partial result (one request of 131072 keys, 32 query heads: 95.9 -> 94.5 us).
  int slices = 1;
  while (2 * slices * outs <= cus && a.cache.dim / (2 * slices) >= 16) slices *= 2;
  attn_join_kernel<DT, PT, 1><<<(unsigned)(outs * slices), kJoin, 0, s>>>(a, p, slices);
  return hipGetLastError();
}

}  // namespace
}  // namespace fk

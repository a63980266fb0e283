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

// Scale of a partial result (m, l) under the common maximum.
__device__ __forceinline__ float join_factor(float m, float l, float top) {
  return l == 0.f ? 0.f : fast_exp2((m - top) * kLog2e);
}

// Any size, stride and alignment. One block per (request, query head, part of the
// request's keys); a wave takes every fourth key, a lane every 64th element of a row. With
// one part the result is final, else parts leave o (B,Hq,parts,D), ml (B,Hq,parts,2).
template <int DT, int EPL>
__global__ __launch_bounds__(kWaves * 64) void attn_any_kernel(AttnArgs a, int parts, float* po,
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

template <int DT>
hipError_t run_any(const AttnArgs& a, int64_t most, void* ws, hipStream_t s) {
  const int parts = most > 128 ? (int)any_parts(a.B, a.Hq) : 1;
  const int64_t heads = a.B * a.Hq, blocks = heads * parts;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const int64_t D = a.cache.dim;
  float* po = (float*)ws;
  float* pml = po + blocks * D;
  const auto kernel = D <= 64    ? attn_any_kernel<DT, 1>
                      : D <= 128 ? attn_any_kernel<DT, 2>
                      : D <= 256 ? attn_any_kernel<DT, 4>
                                 : attn_any_kernel<DT, 16>;
  kernel<<<(unsigned)blocks, kWaves * 64, 0, s>>>(a, parts, po, pml);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || parts == 1) return e;
  attn_any_join_kernel<DT><<<(unsigned)heads, kWaves * 64, 0, s>>>(a, parts, po, pml);
  return hipGetLastError();
}

// Keys of the longest request, at most: what the tables hold, or the caller's bound.
int64_t longest(const AttnArgs& a) {
  int64_t most = a.width * a.cache.page;
  if (most > 0x7FFFFFFF) most = 0x7FFFFFFF;
  return a.max_len > 0 && a.max_len < most ? a.max_len : most;
}

// ---------------------------------------------------------------------------
// Matrix-core kernel: rows of at most 256 elements in whole 16-byte units
// ---------------------------------------------------------------------------
// One block works for up to 16 query heads of one cache head, so a key is read
// once for all of them. With G query heads a key head, 16-bit caches give G
// operations a byte: HBM is the bound, and the 16 columns of the matrix product
// cost the same for any G up to 16.
//
// Lane 16 g + m of a wave. Scores are S^T = K Q^T with v_mfma 16x16: row =
// key, column = query head, so lane (m, g) holds query head m's scores of keys
// 4g..4g+3 of each 16-key tile. The values enter as O^T = V^T P^T, whose
// contraction index is the key: the same lane must hold head m's
// probabilities of some keys and, for row m of V^T, those keys' values. The
// order of keys within a contraction is free, so slot 8g + j stands for key 4g + j
// of the first (j < 4) or second (j >= 4) tile: the probabilities are used in the
// lane that computed them, and the lane loads rows 4g + j of V itself, elements
// VE m .. VE m + VE - 1 (16 lanes cover a row), picking tile t's element of
// each row with byte permutes. Nothing goes through LDS but row addresses.
//
// A wave's step is 32 keys (fp32: 16). The next step's keys are asked for as soon as the
// scores are out of the registers they sit in, the next values after the last product with
// these, so that one of the two is always on its way without a second set of
// registers: 64 to 128 KB in flight a CU for 8 waves of 128-element rows, 48 to 96 for 12
// of 64. A step of 16 KB costs about 280 VALU and 24 matrix instructions, a fifth of the
// time its bytes take.
// Measured: 32 requests of 2048 to 65536 keys, 8 heads of 128 bf16, 4.43 GB, 671 us or 6.6
// TB/s (a large copy reads and writes 4.8 on the same card).
constexpr int kHeadTile = 16;
constexpr int kMaxCus = 256;

template <int DT, int DP> struct Shape {
  static constexpr int tiles = DT == FK_F32 ? 1 : 2;        // 16-key tiles per step
  static constexpr int keys = 16 * tiles;                   // keys per wave and step
  static constexpr int unit = DT == FK_F32 ? 4 : 8;         // elements in 16 bytes
  static constexpr int nc = DP / (4 * unit);                // 16-byte key loads per row and lane
  static constexpr int ve = DP == 192 ? 4 : (DP / 16 < unit ? DP / 16 : unit);   // elements per value load
  static constexpr int nu = DP / (16 * ve);                 // value loads per row and lane
  static constexpr int rows = 4 * tiles;                    // value rows per lane
  static constexpr int ldo = DP + 4;                        // LDS row of merged results
  static constexpr int least = DP <= 32 ? 0 : (DP <= 64 ? 32 : (DP <= 192 ? DP - 64 : 192));  // D is above it
};

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
// above 815 -> 779 us); where waves share lines the mark makes them come twice (8 x 32768
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

// Rows narrower than the tile, rows that fill it, and rows that fill it and whole
// 128-byte lines that no other wave reads, by streaming loads.
enum { kNarrow, kWhole, kStream };

// State of one wave over a run of steps.
template <int DT, int DP, int HT> struct Acc {
  using S = Shape<DT, DP>;
  float m[HT], l[HT];                  // of lane m's head of each tile; l: this lane's share
  floatx4_t o[HT][S::nu * S::ve];
};

// Row addresses and bias of one step's keys, per wave and parity.
template <int DT, int DP> struct Rows {
  static constexpr int n = Shape<DT, DP>::keys;
  uint64_t k[n], v[n];
  float bias[n];
};

template <int DT, int DP, int HT, bool EXTRA, int KIND>
__device__ __forceinline__ void attend(const AttnArgs& a, const Plan& p, int64_t b, int hk, int ht,
                                       int len, int step, int stride, int end,
                                       Rows<DT, DP>* rows,
                                       Acc<DT, DP, HT>& acc) {
  using S = Shape<DT, DP>;
  const fk_kv_cache_t& c = a.cache;
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const int D = KIND == kNarrow ? (int)c.dim : DP;
  constexpr int eb = Val<DT>::bytes;
#pragma unroll
  for (int h = 0; h < HT; ++h) {
    acc.m[h] = -INFINITY;
    acc.l[h] = 0.f;
#pragma unroll
    for (int i = 0; i < S::nu * S::ve; ++i) acc.o[h][i] = floatx4_t{0.f, 0.f, 0.f, 0.f};
  }
  if (step >= end) return;

  // Query fragments; heads past G and elements past D are zero. Elements past D of a
  // key are read from the zeros too: an infinity of the row times a zero query is NaN.
  // A value's read the row's start again and are not stored.
  uint4 q[HT][S::nc];
  uint32_t koff[S::nc], voff[S::nu];
  const auto past = [&](int i) {            // unit i of this lane's part of a key is past D
    return (i + 1) * 4 * S::unit > S::least && i * 4 * S::unit + g * S::unit >= D;
  };
#pragma unroll
  for (int i = 0; i < S::nc; ++i) koff[i] = past(i) ? 0 : (i * 4 + g) * S::unit * eb;
#pragma unroll
  for (int h = 0; h < HT; ++h) {
    const int head = (ht * HT + h) * kHeadTile + m;
    const char* qp = (const char*)a.q + (b * a.q_stride[0] +
                                         (int64_t)(hk * p.G + min(head, p.G - 1)) * a.q_stride[1]) * eb;
#pragma unroll
    for (int i = 0; i < S::nc; ++i) {
      q[h][i] = load16((uint64_t)(qp + koff[i]));
      if (past(i) || head >= p.G) q[h][i] = make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < S::nu; ++i) {
    const int e = i * 16 * S::ve + m * S::ve;
    voff[i] = e < D ? e * eb : 0;
  }

  // Lane i < keys looks after key i of a step: table entry two steps ahead, bias
  // one step ahead, addresses to LDS just before the step's loads.
  const uint64_t table = (uint64_t)(a.table + b * a.ld_table);
  const int kl = lane & (S::keys - 1);
  const uint64_t kbase = (uint64_t)c.k + (uint64_t)hk * c.k_stride[2] * eb;
  const uint64_t vbase = (uint64_t)c.v + (uint64_t)hk * c.v_stride[2] * eb;
  const uint64_t zero = (uint64_t)zero_row;
  const bool cap = EXTRA && a.softcap > 0.f;
  const float inv_cap = cap ? 1.f / a.softcap : 0.f;
  const bool has_bias = EXTRA && c.key_bias && c.pages > 0;
  const uint64_t bbase = (uint64_t)c.key_bias + (uint64_t)hk * c.bias_stride[2] * 4;
  // (loads without branches: a key past the end reads the last one's entry)
  auto entry = [&](int st) -> int32_t {             // page of key kl of step st, -1: none
    const uint32_t key = (uint32_t)st * S::keys + kl;
    const uint32_t at = min(key, (uint32_t)len - 1);
    const int32_t pg = *(gptr_i32)(table + 4 * (uint64_t)div_by(at, p.page));
    return st < end && key == at ? pg : -1;
  };
  auto bias_of = [&](int st, int32_t pg) -> float {
    const bool live = (uint32_t)pg < (uint32_t)c.pages;
    float bias = 0.f;
    if (has_bias) {
      // (the last one's place for a key past the end: one past 2^31 would not divide)
      const uint32_t key = min((uint32_t)st * S::keys + kl, (uint32_t)len - 1);
      const uint32_t tok = key - div_by(key, p.page) * p.page.d;
      bias = *(gptr_f32)(bbase + (uint64_t)((live ? pg : 0) * c.bias_stride[0] + tok * c.bias_stride[1]) * 4);
    }
    return live ? bias : -INFINITY;
  };
  auto put_rows = [&](Rows<DT, DP>& r, int st, int32_t pg, float bias) {
    const uint32_t key = (uint32_t)st * S::keys + kl;
    const uint32_t tok = key - div_by(key, p.page) * p.page.d;
    const bool live = bias != -INFINITY;
    const uint64_t ka = kbase + (uint64_t)(pg * c.k_stride[0] + tok * c.k_stride[1]) * eb;
    const uint64_t va = vbase + (uint64_t)(pg * c.v_stride[0] + tok * c.v_stride[1]) * eb;
    // other lanes of the wave read these: keep the compiler's order
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    r.k[kl] = live ? ka : zero;
    r.v[kl] = live ? va : zero;
    r.bias[kl] = bias;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };
  uint4 kf[S::tiles][S::nc];
  auto load_k = [&](const Rows<DT, DP>& r) {
#pragma unroll
    for (int s = 0; s < S::tiles; ++s) {
      const uint64_t ad = r.k[16 * s + m];
#pragma unroll
      for (int i = 0; i < S::nc; ++i) kf[s][i] = load_row<16, KIND == kStream>((past(i) ? zero : ad) + koff[i]);
    }
  };
  uint4 vf[S::rows][S::nu];            // a load of fewer bytes fills the first words
  auto load_v = [&](const Rows<DT, DP>& r) {
#pragma unroll
    for (int j = 0; j < S::rows; ++j) {
      const uint64_t ad = r.v[16 * (j >> 2) + 4 * g + (j & 3)];
#pragma unroll
      for (int i = 0; i < S::nu; ++i) vf[j][i] = load_row<S::ve * eb, KIND == kStream>(ad + voff[i]);
    }
  };

  int32_t pg1 = entry(step), pg2 = entry(step + stride);
  put_rows(rows[0], step, pg1, bias_of(step, pg1));
  float bias1 = bias_of(step + stride, pg2);
  pg1 = pg2;
  pg2 = entry(step + 2 * stride);
  load_k(rows[0]);
  load_v(rows[0]);
  int par = 0;
  for (; step < end; step += stride, par ^= 1) {
    Rows<DT, DP>& now = rows[par];
    Rows<DT, DP>& next = rows[par ^ 1];
    put_rows(next, step + stride, pg1, bias1);
    float s[HT][S::tiles][4];
#pragma unroll
    for (int h = 0; h < HT; ++h)
#pragma unroll
      for (int u = 0; u < S::tiles; ++u) {
        // fp32: four sums, a quarter of the rounding steps each, as the products are not exact
        constexpr int sums = DT == FK_F32 && S::nc >= 4 ? 4 : 1;
        floatx4_t x[sums];
#pragma unroll
        for (int i = 0; i < sums; ++i) x[i] = floatx4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < S::nc; ++i) x[i % sums] = Mfma16<DT>::run(kf[u][i], q[h][i], x[i % sums]);
        if constexpr (sums == 4) x[0] = (x[0] + x[1]) + (x[2] + x[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[h][u][i] = x[0][i];
      }
    load_k(next);
    __builtin_amdgcn_sched_barrier(0);   // the next keys are on their way before the softmax
    bias1 = bias_of(step + 2 * stride, pg2);
    pg1 = pg2;
    pg2 = entry(step + 3 * stride);

#pragma unroll
    for (int h = 0; h < HT; ++h) {
      float top = acc.m[h];
#pragma unroll
      for (int u = 0; u < S::tiles; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // -inf where a key does not count: its score is 0 (a zero row), or NaN where
          // the query is not finite
          const float bias = now.bias[16 * u + 4 * g + i];
          float x = s[h][u][i] * a.scale;
          if (cap) x = capped(x, a.softcap, inv_cap);
          s[h][u][i] = bias == -INFINITY ? bias : (EXTRA ? x + bias : x);
          top = fmaxf(top, s[h][u][i]);
        }
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      // differences before the scaling by log2 e: a bias of the type's lowest
      // value must not overflow; with nothing but -inf so far, subtract nothing
      const float ref = top == -INFINITY ? 0.f : top;
      const float alpha = fast_exp2((acc.m[h] - ref) * kLog2e);
      acc.m[h] = top;
      float part = 0.f;
#pragma unroll
      for (int u = 0; u < S::tiles; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[h][u][i] = prob<DT>(s[h][u][i] - ref);
          part += s[h][u][i];
        }
      acc.l[h] = fmaf(acc.l[h], alpha, part);
#pragma unroll
      for (int i = 0; i < S::nu * S::ve; ++i) acc.o[h][i] *= alpha;
    }

    if constexpr (DT == FK_F32) {
#pragma unroll
      for (int y = 0; y < S::tiles; ++y)
#pragma unroll
        for (int u = 0; u < S::nu; ++u)
#pragma unroll
          for (int t = 0; t < S::ve; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              floatx4_t& o = acc.o[0][u * S::ve + t];
              o = __builtin_amdgcn_mfma_f32_16x16x4f32(
                  __builtin_bit_cast(float, word(vf[4 * y + j][u], t)), s[0][y][j], o, 0, 0, 0);
            }
    } else {
      // Probabilities as the sum of two 16-bit numbers: one alone would round
      // each to 8 (bf16) or 11 bits, an error as large as the result's own
      // rounding. The second product rides on matrix units that are idle anyway.
      // The first is rounded down and the second is above 0 where the probability is: an
      // infinite value times 0 or a negative rest would be NaN or take the infinity off.
#pragma unroll
      for (int y = 0; y < S::tiles / 2; ++y) {
        uint4 ph[HT], pl[HT];
#pragma unroll
        for (int h = 0; h < HT; ++h) {
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = s[h][2 * y + (j >> 2)][j & 3];
          Halves<DT>::split(x, ph[h], pl[h]);
        }
        auto pick = [&](int j, int u, int t) {       // element t of rows j (low half) and j + 1
          return __builtin_amdgcn_perm(word(vf[8 * y + j + 1][u], t >> 1),
                                       word(vf[8 * y + j][u], t >> 1),
                                       t & 1 ? 0x07060302u : 0x05040100u);
        };
#pragma unroll
        for (int u = 0; u < S::nu; ++u)
#pragma unroll
          for (int t = 0; t < S::ve; ++t) {
            const uint4 vt = make_uint4(pick(0, u, t), pick(2, u, t), pick(4, u, t), pick(6, u, t));
#pragma unroll
            for (int h = 0; h < HT; ++h) {
              floatx4_t& o = acc.o[h][u * S::ve + t];
              o = Mfma16<DT>::run(vt, ph[h], o);
              o = Mfma16<DT>::run(vt, pl[h], o);
            }
          }
      }
    }
    load_v(next);
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int h = 0; h < HT; ++h) {
    acc.l[h] += __shfl_xor(acc.l[h], 16, 64);
    acc.l[h] += __shfl_xor(acc.l[h], 32, 64);
  }
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

template <int DT, int DP, int HT, bool EXTRA, int KIND, int W>
__global__ __launch_bounds__(W * 64, W == kWaves ? waves_per_simd(DP) : W / 4) void attn_mfma_kernel(AttnArgs a, Plan p) {
  using S = Shape<DT, DP>;
  __shared__ Rows<DT, DP> rows[W][2];
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
      Acc<DT, DP, HT> acc;
      attend<DT, DP, HT, EXTRA, KIND>(a, p, b, hk, ht, len, t0 + w - k0, p.team, t1, rows[w], acc);
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
              a.lse[row] = l == 0.f ? -INFINITY : top + (logf(l) - kProbShift<DT> * kLn2);
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
// maxima and sums, then the rows.
template <int DT, int R>
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
    a.lse[out_row] = l == 0.f ? -INFINITY : top + (logf(l) - kProbShift<DT> * kLn2);
}

// Rows the matrix-core kernel can load: whole, aligned 16-byte units.
bool aligned16(const AttnArgs& a, int eb) {
  const fk_kv_cache_t& c = a.cache;
  const int64_t s[] = {a.q_stride[0], a.q_stride[1], c.k_stride[0], c.k_stride[1], c.k_stride[2],
                       c.v_stride[0], c.v_stride[1], c.v_stride[2], c.dim};
  for (int64_t v : s)
    if (v * eb % 16) return false;
  return !(((uintptr_t)a.q | (uintptr_t)c.k | (uintptr_t)c.v | (uintptr_t)a.out) & 15);
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

template <int DT, int DP, int HT>
hipError_t run_mfma(const AttnArgs& a, void* ws, hipStream_t s) {
  Plan p{};
  p.heads = (int)a.cache.heads;
  p.G = (int)(a.Hq / a.cache.heads);
  p.width = HT * kHeadTile;
  p.tiles = (p.G + p.width - 1) / p.width;
  p.hr = p.G < p.width ? p.G : p.width;
  p.page = fast_div((uint32_t)a.cache.page);
  const int64_t units = (int64_t)p.heads * p.tiles;
  const int64_t most = longest(a);
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
  const bool eight = DP <= 128 && most > 512 && most <= 64 * Shape<DT, DP>::keys &&
                     rows <= cus && 2 * rows >= cus;
  const bool cut = !eight && (most > 512 || (many && most > 8 * Shape<DT, DP>::keys));
  if (cut) {
    // Where there are steps enough for every wave of the chip, a block's waves take
    // neighbouring heads, whose rows lie side by side in the cache, instead of one
    // head's steps in turn: the block reads 4 rows' length in one piece (the 4.43 GB
    // above: 774 us with 1 head a block, 697 with 2, 670 with 4). With fewer steps the
    // waves share them and join in LDS, not through memory.
    const double steps = (double)units * a.B * ((most + Shape<DT, DP>::keys - 1) / Shape<DT, DP>::keys);
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
    p.team = eight ? 8 : (many || most <= Shape<DT, DP>::keys ? 1 : kWaves);
  }
  const int W = eight ? 8 : kWaves;
  p.team_log = p.team == 8 ? 3 : (p.team == 4 ? 2 : p.team - 1);
  p.by_tiles = fast_div((uint32_t)p.tiles);
  p.by_heads = fast_div((uint32_t)p.heads);
  const int64_t blocks = (units * (cut ? p.parts : a.B) * p.team + W - 1) / W;
  if (units * a.B + W > 0x7FFFFFFF || a.B * a.Hq > 0x7FFFFFFF - 4) return hipErrorInvalidConfiguration;
  const auto aligned = [](uintptr_t base, const int64_t* s) {
    return !((base | (uintptr_t)((s[0] | s[1] | s[2]) * Val<DT>::bytes)) & 127);
  };
  // Caches that the 256 MB last-level cache may still hold from the step before are read
  // without the mark (4 requests of 512 keys: 10.4 us, marked 13.3).
  const double bytes = 2.0 * a.B * most * a.cache.heads * DP * Val<DT>::bytes;
  const bool full = a.cache.dim == DP, extra = a.softcap > 0.f || a.cache.key_bias;
  auto kernel = full ? (extra ? attn_mfma_kernel<DT, DP, HT, true, kWhole, kWaves>
                              : attn_mfma_kernel<DT, DP, HT, false, kWhole, kWaves>)
                     : (extra ? attn_mfma_kernel<DT, DP, HT, true, kNarrow, kWaves>
                              : attn_mfma_kernel<DT, DP, HT, false, kNarrow, kWaves>);
  if constexpr (DP * Val<DT>::bytes % 128 == 0) {
    if (full && bytes >= (double)(128 << 20) && p.tiles == 1 &&
        aligned((uintptr_t)a.cache.k, a.cache.k_stride) && aligned((uintptr_t)a.cache.v, a.cache.v_stride))
      kernel = extra ? attn_mfma_kernel<DT, DP, HT, true, kStream, kWaves>
                     : attn_mfma_kernel<DT, DP, HT, false, kStream, kWaves>;
  }
  if constexpr (DP <= 128) {
    if (eight)
      kernel = full ? (extra ? attn_mfma_kernel<DT, DP, HT, true, kWhole, 8>
                             : attn_mfma_kernel<DT, DP, HT, false, kWhole, 8>)
                    : (extra ? attn_mfma_kernel<DT, DP, HT, true, kNarrow, 8>
                             : attn_mfma_kernel<DT, DP, HT, false, kNarrow, 8>);
  }
  kernel<<<(unsigned)blocks, W * 64, 0, s>>>(a, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !cut) return e;
  // Many rows: most were not cut or have few parts, and a wave is enough for one.
  const int64_t outs = a.B * a.Hq;
  if (outs >= 8 * cus) {
    attn_join_kernel<DT, 4><<<(unsigned)((outs + 3) / 4), kJoin, 0, s>>>(a, p, 1);
    return hipGetLastError();
  }
  // Few rows have many parts: as many blocks a row as there are CUs for, down to 64 bytes
  // of a partial result (one request of 131072 keys, 32 query heads: 95.9 -> 94.5 us).
  int slices = 1;
  while (2 * slices * outs <= cus && a.cache.dim / (2 * slices) >= 16) slices *= 2;
  attn_join_kernel<DT, 1><<<(unsigned)(outs * slices), kJoin, 0, s>>>(a, p, slices);
  return hipGetLastError();
}

template <int DT>
hipError_t run(const AttnArgs& a, void* ws, hipStream_t s) {
  const int64_t D = a.cache.dim;
  if (D > 256 || !aligned16(a, Val<DT>::bytes)) return run_any<DT>(a, longest(a), ws, s);
  if constexpr (DT != FK_F32) {
    if (tile_width(DT, D, a.Hq / a.cache.heads) > kHeadTile)
      return D <= 32   ? run_mfma<DT, 32, 2>(a, ws, s)
             : D <= 64 ? run_mfma<DT, 64, 2>(a, ws, s)
                       : run_mfma<DT, 128, 2>(a, ws, s);
  }
  return D <= 32    ? run_mfma<DT, 32, 1>(a, ws, s)
         : D <= 64  ? run_mfma<DT, 64, 1>(a, ws, s)
         : D <= 128 ? run_mfma<DT, 128, 1>(a, ws, s)
         : D <= 192 ? run_mfma<DT, 192, 1>(a, ws, s)
                    : run_mfma<DT, 256, 1>(a, ws, s);
}

}  // namespace

size_t attn_ws_bytes(int dt, int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  // either kernel may run: alignment is not known here
  const size_t any = (size_t)(B * Hq * any_parts(B, Hq)) * (D + 2) * 4;
  if (D > 256) return any;
  // sized for the largest chip: a pure function of the shape
  const int64_t G = Hq / Hkv, width = tile_width(dt, D, G), units = Hkv * ((G + width - 1) / width);
  const int64_t groups = units * team_of(units) / kWaves;
  const size_t slots = (size_t)units * parts_of(chip_blocks(kMaxCus, D), groups) * 2 * (G < width ? G : width);
  const size_t cut = slots * D * 4 + slots * 8 + (size_t)B * 8;
  return cut > any ? cut : any;
}

hipError_t launch_paged_attn(const AttnArgs& a, int dt, void* ws, hipStream_t s) {
  if (a.B == 0) return hipSuccess;
  return dt == FK_F32   ? run<FK_F32>(a, ws, s)
         : dt == FK_F16 ? run<FK_F16>(a, ws, s)
                        : run<FK_BF16>(a, ws, s);
}

}  // namespace fk

// Attention of a step's prompts over a paged key-value cache: every new token over
// its request's keys up to itself. The kernels; the other prompt units build them.
#pragma once

#include <type_traits>
#include <utility>

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

// One row (token t, query head h) of request b over keys j0 .. j1 - 1, any size, stride and
// alignment, by one wave: a lane holds every 64th element of the sums o.
template <int DT, int EPL>
__device__ __forceinline__ void row_sums(const PromptArgs& a, int64_t b, int64_t t, int64_t h, int64_t j0,
                                         int64_t j1, float& m, float& l, float (&o)[EPL]) {
  using E = typename Val<DT>::type;
  const int lane = threadIdx.x & 63;
  const fk_kv_cache_t& c = a.cache;
  const int D = (int)c.dim;
  const int64_t hk = h / (a.Hq / c.heads);
  const E* q = (const E*)a.q + t * a.q_stride[0] + h * a.q_stride[1];
  float qf[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    qf[i] = e < D ? Val<DT>::get(q + e) : 0.f;
    o[i] = 0.f;
  }
  m = -INFINITY, l = 0.f;
  // A sum in 32 bits stands still after 2^24 terms alike: sums over kRun keys are summed.
  constexpr int64_t kRun = 1 << 16;
  for (int64_t start = j0; start < j1; start += kRun) {
    float mr = -INFINITY, lr = 0.f, r[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) r[i] = 0.f;
    for (int64_t j = start; j < min(start + kRun, j1); ++j) {
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
      const float mn = fmaxf(mr, s);
      const float alpha = mr == -INFINITY ? 0.f : fast_exp2((mr - mn) * kLog2e);
      const float p = s == -INFINITY ? 0.f : fast_exp2((s - mn) * kLog2e);   // NaN stays NaN
      lr = lr * alpha + p;
      mr = mn;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + 64 * i;
        if (e < D) r[i] = fmaf(p, Val<DT>::get(v + e), r[i] * alpha);
      }
    }
    const float mn = fmaxf(m, mr);
    const float f = m == mn ? 1.f : fast_exp2((m - mn) * kLog2e), g = mr == mn ? 1.f : fast_exp2((mr - mn) * kLog2e);
    l = l * f + lr * g;
    m = mn;
#pragma unroll
    for (int i = 0; i < EPL; ++i) o[i] = start == j0 ? r[i] : fmaf(r[i], g, o[i] * f);
  }
}

// A row's result.
template <int DT, int EPL>
__device__ __forceinline__ void put_row(const PromptArgs& a, int64_t row, float m, float l,
                                        const float (&o)[EPL]) {
  const int lane = threadIdx.x & 63, D = (int)a.cache.dim;
  const bool any = l != 0.f;             // true for NaN: it has to reach the result
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    if (e < D) Val<DT>::put((typename Val<DT>::type*)a.out + row * D + e, any ? o[i] / l : 0.f);
  }
  if (a.lse && lane == 0) a.lse[row] = any ? m + logf(l) : -INFINITY;
}

// ---------------------------------------------------------------------------
// Matrix-core kernel: rows of at most 256 elements in whole 16-byte units
// ---------------------------------------------------------------------------
// The G query heads of a cache head see the same keys, so row r of a request is head r % G
// of token r / G, and a tile is 256 or 128 rows in a run. A block takes one tile of one cache head
// over a range of keys, a wave 32 of its rows, 64 keys a step (32 for wide fp32 rows).
//
// Lane (n = lane & 31, h = lane >> 5) of a wave. Scores are S^T = K Q^T with v_mfma 32x32x16:
// register i of the lane holds the score of query row n with key (i & 3) + 8 (i >> 2) + 4 h of
// 32. The values enter as O^T = V^T P^T: the contraction runs over keys, whose order is
// free, so the eight probabilities a lane gives to a product are those it holds, of keys 4 h +
// 0..3 and 8 + 4 h + 0..3 of 16, and V^T comes from LDS in that order by transposing reads
// (four keys of one element a lane each). fp32 products take two keys each, one a half of the
// wave: those a lane's two halves hold in the same register. Only keys and values go through LDS.
//
// Keys and values go from the cache's pages straight to LDS, 16 bytes a lane, two or three buffers in
// turn. Each wave brings its share of a step's rows; their addresses are found for as many
// steps at once as make up 64, and table entries and biases are asked for two such groups ahead.
//
// What bounds it: with 32 rows a wave a product of 32 cycles reads 1 KB of LDS, of which a CU
// gives four SIMDs 128 bytes a cycle, so products and reads would both fill their time at
// the peak; before that, power: half of the matrix units' cycles are used at a clock of
// 1.85 GHz (2.1 where the units wait more). Measured: 32768 tokens, 32 heads of 128 on 8, bf16, 8.45 to
// 8.7 ms, 1010 to 1040 TFLOP/s (a large library product on random numbers reaches 1142 on the
// same card); with probabilities and products in turn instead of together 9.6 ms, and
// with reads that wait for all loads on their way 9.8. Short prompts are bound by a block's start and
// end, 15 us of dependent loads and stores around a few steps of 2.
typedef const __attribute__((address_space(1))) uint32_t* gptr32;
typedef __attribute__((address_space(3))) uint32_t* lptr32;
typedef __attribute__((address_space(3))) char* lptr8;
typedef const __attribute__((address_space(3))) char* lptr8c;
typedef const __attribute__((address_space(3))) u32x4* lptr16c;
typedef const __attribute__((address_space(3))) uint32_t* lptr32c;

// W waves of a block, 8 or 4, share the keys of a step. Wide rows need the registers of 4, and
// fp32 products are an eighth as fast, so that smaller tiles, which more CUs share, cost
// nothing. Blocks of 4 have a CU to themselves where rows are wide, else two run on it.
constexpr bool only_four(int dt, int DC) { return dt == FK_F32 || DC > 128; }
constexpr int tile_blocks(int dt, int DC, int W) { return W == 4 && (dt == FK_F32 ? DC <= 64 : DC <= 128) ? 2 : 1; }

// fp16 probabilities are scaled by 2^13, and may pass the running maximum's by 2^2, bf16 by 2^8:
// the sums are scaled anew only when a maximum grows by more.
template <int DT> constexpr float prob_shift = DT == FK_F16 ? 13.f : 0.f;
template <int DT> constexpr float prob_slack = DT == FK_F16 ? 2.f : 8.f;

template <int DT, int DC, int W> struct Tile {
  static constexpr int eb = Val<DT>::bytes;
  static constexpr int pitch = DC <= 64 ? 64 : (DC <= 128 ? 128 : 256);    // elements of a row in LDS
  static constexpr int rb = pitch * eb;                   // and bytes
  static constexpr int rows = W * 32;
  static constexpr int step = eb == 4 && DC > 64 ? 32 : 64;      // keys a step: two buffers fit the LDS
  static constexpr int key_tiles = step / 32;
  static constexpr int unit = 16 / eb;                    // elements of 16 bytes
  static constexpr int units = pitch / unit;              // 16-byte units of a row
  static constexpr int per_load = 64 / units;             // rows a wave brings with one load
  static constexpr int share = step / W;                  // rows a wave brings a step
  static constexpr int loads = share / per_load;
  // Steps of keys and of values in LDS: as many as there is room for, up to three, so that a step's
  // rows have two steps' time to come.
  static constexpr int held = 3 * 2 * step * rb * tile_blocks(DT, DC, W) <= 144 * 1024 ? 3 : 2;
  static constexpr int group = 64 / share;                // steps whose rows a wave finds at once
  static constexpr int dt = DC / 32, kt = DC / (2 * unit);        // tiles of the output, units of a score
};

// Where unit u of row r lies in its LDS row. Scores read one unit of 32 rows at once: 16
// neighbouring rows are 16 different units. Transposing reads take two units of four
// rows, or four of them: the rows are put 2 and 4 units apart, mod 8 and mod 16. fp32 values are
// read 32 elements of two rows at once, four rows apart: one of them 8 units on.
template <class L> __device__ __forceinline__ int key_swizzle(int r) { return r & (L::units - 1) & 15; }
template <class L> __device__ __forceinline__ int value_swizzle(int r) {
  if constexpr (L::eb == 4) return (r & 4) << 1;
  if constexpr (L::units == 8) return (r & 1) << 1 | (r & 2) << 1;
  return (r & 1) << 2 | (r & 2) << 2 | (r & 2);
}

// Both halves' numbers of a wave, in every lane: (of lanes 0..31, of lanes 32..63).
__device__ __forceinline__ floatx2_t both_halves(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const u32x2 r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t lo = r.x, hi = r.y;       // (a bit cast of an element itself takes the first one's)
  return floatx2_t{__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi)};
}
__device__ __forceinline__ float max_halves(float x) {
  const floatx2_t r = both_halves(x);
  return fmaxf(r.x, r.y);
}
__device__ __forceinline__ float sum_halves(float x) {
  const floatx2_t r = both_halves(x);
  return r.x + r.y;
}

// Four keys of one element each, 16 lanes a 4 x 16 block that lies in LDS key by key.
__device__ __forceinline__ uint2 read_transposed(lptr8c at) {
  typedef short s4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s4* lp;
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)at));
}

// The tile of a block, from the last request's last tile on: the longest rows of a prompt come
// first and the chip does not wait for one at the end.
struct Where {
  int64_t b;          // request, -1: none
  int tile;           // tile of its rows
  int cu0, cu1, len;  // its tokens and keys
};
constexpr Where kNowhere = {-1, 0, 0, 0, 0};

// Of up to 64 requests: a lane counts one's tiles.
template <int ROWS> __device__ __forceinline__ Where count_tiles(const PromptArgs& a, int G, uint32_t order) {
  const int lane = threadIdx.x & 63, b = max((int)a.B - 1 - lane, 0);
  const int cu0 = a.cu[b], cu1 = a.cu[b + 1], len = a.lens[b];
  const int64_t n = (int64_t)cu1 - cu0;
  const uint32_t mine = lane < a.B && n > 0 ? (uint32_t)((n * G + ROWS - 1) / ROWS) : 0;
  uint32_t incl = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = __shfl_up(incl, off, 64);
    if (lane >= off) incl += o;
  }
  const int at = __popcll(__ballot(incl <= order));
  if (at == 64) return kNowhere;
  const uint32_t end = __builtin_amdgcn_readlane(incl, at);
  return {a.B - 1 - at, (int)(end - 1 - order), (int)__builtin_amdgcn_readlane(cu0, at),
          (int)__builtin_amdgcn_readlane(cu1, at), (int)__builtin_amdgcn_readlane(len, at)};
}

// Of more requests the tile is searched for, 64 ways a round: request b's tiles have the numbers
// floor(cu_tokens[b] G / ROWS) + b on, never more than there are up to the next request's. Numbers
// left over are blocks without work among the others, and as the chip hands blocks to its
// engines in turn, whatever they have left to do, few requests are better counted. (64
// requests of one token over 8192 keys: 234 us counted, 254 searched; 256 requests
// counted in four rounds take 1 to 3% longer, 1024 of 16 tokens 372 us and searched 291.)
template <int ROWS> __device__ __forceinline__ Where search_tile(const PromptArgs& a, int G, uint32_t order) {
  const int lane = threadIdx.x & 63;
  const auto first = [&](int64_t b, int cu) { return ((int64_t)cu * G) / ROWS + b; };
  const int64_t number = first(a.B, max(a.cu[a.B], 0)) - 1 - order;
  if (number < 0) return kNowhere;
  int64_t lo = 0, hi = a.B;
  for (;;) {
    const int64_t span = (hi - lo + 63) / 64, b = lo + lane * span, at = min(b, hi - 1);
    const int cu0 = max(a.cu[at], 0), cu1 = a.cu[at + 1], len = a.lens[at];
    const int before = __popcll(__ballot(b < hi && first(at, cu0) <= number));
    if (before == 0) return kNowhere;
    lo += (before - 1) * span;
    if (span == 1) {
      const int c0 = __builtin_amdgcn_readlane(cu0, before - 1), c1 = __builtin_amdgcn_readlane(cu1, before - 1);
      const int64_t tile = number - first(lo, c0);
      if (tile * ROWS >= ((int64_t)c1 - c0) * G) return kNowhere;
      return {lo, (int)tile, c0, c1, (int)__builtin_amdgcn_readlane(len, before - 1)};
    }
    hi = min(lo + span, hi);
  }
}

// Whether a lane's sums are all finite, and which of them are NaN, a bit each.
template <int N> struct NotFinite { uint32_t none, bits[(N + 1) / 2]; };
template <int N> __device__ __forceinline__ NotFinite<N> not_finite(const floatx16_t (&o)[N], bool none) {
  NotFinite<N> r = {none};
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) r.bits[i / 2] |= (o[i][j] == o[i][j] ? 0u : 1u) << ((i & 1) * 16 + j);
  return r;
}
template <int N> __device__ __forceinline__ bool all_finite(const floatx16_t (&o)[N]) {
  float x = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) x = fmaf(o[i][j], 0.f, x);
  return x == 0.f;
}
template <int N> __device__ __forceinline__ bool newly(const NotFinite<N>& now, const NotFinite<N>& before) {
  uint32_t r = before.none;
#pragma unroll
  for (int i = 0; i < (N + 1) / 2; ++i) r |= now.bits[i] & ~before.bits[i];
  return r != 0;
}

// 16 bytes a lane from its address straight to LDS, lane after lane from `to` on (the same in
// every lane). Written out, as the compiler would let every later read of LDS wait for
// the bytes, whatever it reads; what waits is an s_waitcnt vmcnt before the
// barrier after which they are read. No register is written, and the address is
// read when the instruction is issued. m0, which nothing else here uses, takes a wait
// state before it is read.
__device__ __forceinline__ void load_to_lds(uint64_t from, lptr8 to) {
  const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)to);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :: "s"(at), "v"(from) : "memory");
}

// f(0), ..., f(N - 1), each with its number as a type.
template <class F, int... I> __device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, const F& f) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, class F> __device__ __forceinline__ void each(const F& f) {
  each_of(std::make_integer_sequence<int, N>(), f);
}

struct PromptPlan {
  int heads, G, parts, chunk;     // cache heads, query heads of each, parts of a row's keys, steps of a part
  FastDiv page, by_heads, by_tiles, by_G;
  uint32_t turn, last;        // of a head's blocks: the first that comes in turned order, and the last
  float* o;                       // (parts, T, Hq, D) partial sums
  float* ml;                      // (parts, T, Hq, 2) their maximum and sum
};

// What a score takes part in: the scale alone; scale and bias; cap as well, by capped() or, for 16-bit
// types and caps of at most kNearCap, by cap_16bit().
enum { kPlainScore, kBiasScore, kCapScore, kNearCapScore };

template <int DT, int DC, int W, int SCORE>
__global__ __launch_bounds__(W * 64, W / 4 * tile_blocks(DT, DC, W))
void prompt_mfma_kernel(PromptArgs a, PromptPlan p) {
  using L = Tile<DT, DC, W>;
  constexpr bool EXTRA = SCORE != kPlainScore;
  constexpr int rb = L::rb, eb = L::eb, kStep = L::step, KT = L::key_tiles, GS = L::group, NB = L::held;
  __shared__ __attribute__((aligned(1024))) char lk[NB][kStep * rb], lv[NB][kStep * rb];
  __shared__ uint64_t row_k[W][64], row_v[2][W][64];   // (values are asked for two steps after their keys)
  __shared__ uint64_t valid[2][GS];                    // keys of a step that count, a bit each
  __shared__ float biases[EXTRA ? 2 : 1][EXTRA ? GS : 1][kStep];
  __shared__ NotFinite<L::dt> broken[W * 64];          // sums that were not finite before hidden keys came
  const fk_kv_cache_t& c = a.cache;
  const int lane = threadIdx.x & 63, n = lane & 31, h = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int D = (int)c.dim;

  const uint32_t rest = div_by(blockIdx.x, p.by_heads), hk = blockIdx.x - rest * p.heads;
  // Part after part, a part's tiles longest first: the chip hands blocks to its engines in turn,
  // so long and short ones that alternate would leave half of it idle (2048 tokens, fp32, cut
  // in two: 575 us tile after tile, 416 this way).
  const uint32_t at_order = rest < p.turn ? rest : p.last - (rest - p.turn);
  const uint32_t part = div_by(at_order, p.by_tiles), order = at_order - part * p.by_tiles.d;
  const Where at = a.B <= 64 ? count_tiles<L::rows>(a, p.G, order) : search_tile<L::rows>(a, p.G, order);
  if (at.b < 0) return;
  const int64_t b = uniform(at.b);
  const int64_t cu0 = at.cu0, cu1 = at.cu1, len = at.len;
  const int rows = (int)min((cu1 - cu0) * p.G - (int64_t)at.tile * L::rows, (int64_t)L::rows);
  const int64_t held = min(a.width * c.page, (int64_t)0x7FFFFFFF);
  // keys that row r of the tile sees
  const auto seen = [&](int r) {
    const int64_t t = div_by((uint32_t)(at.tile * L::rows + r), p.by_G);
    return (int)max((int64_t)0, min(len - (cu1 - cu0) + t + 1, held));
  };
  const int most = __builtin_amdgcn_readfirstlane(seen(rows - 1));      // of the tile's last row
  const int steps = (int)(((uint32_t)most + kStep - 1) / kStep);
  const int t0 = (int)part * p.chunk, t1 = (int)part == p.parts - 1 ? steps : min(steps, t0 + p.chunk);
  if (t0 >= t1 && part > 0) return;                    // (part 0 leaves the results of empty rows)

  // queries; rows past the tile's end are zero, see everything and are not stored
  const int r = w * 32 + n;
  const bool mine = r < rows;
  const uint32_t rr = at.tile * L::rows + min(r, rows - 1);
  const int64_t tok = div_by(rr, p.by_G);
  const int64_t t = cu0 + tok, qh = (int64_t)hk * p.G + (rr - tok * p.G);
  const int limit = mine ? seen(r) : 0x7FFFFFFF;
  const int wave_rows = min(rows - w * 32, 32);        // none or fewer: nothing to do
  const int low = wave_rows > 0 ? __builtin_amdgcn_readfirstlane(seen(w * 32)) : 0;
  const int high = wave_rows > 0 ? __builtin_amdgcn_readfirstlane(seen(w * 32 + wave_rows - 1)) : 0;
  uint4 q[L::kt];

  // rows of keys: lane (s, j) looks after row j of this wave's share in step s of a group
  constexpr int share = L::share;
  const int gs = lane / share, gj = w * share + lane % share;
  const uint64_t table = (uint64_t)(a.table + b * a.ld_table);
  const uint64_t kbase = (uint64_t)c.k + (uint64_t)hk * c.k_stride[2] * eb;
  const uint64_t vbase = (uint64_t)c.v + (uint64_t)hk * c.v_stride[2] * eb;
  const uint64_t bbase = (uint64_t)c.key_bias + (uint64_t)hk * c.bias_stride[2] * 4;
  const uint64_t zero = (uint64_t)zero_row;
  const bool has_bias = EXTRA && c.key_bias && c.pages > 0;
  const auto key_of = [&](int group) { return (uint32_t)(t0 + group * GS + gs) * kStep + gj; };
  const auto entry = [&](int group) -> int32_t {       // page of the lane's key, -1: none
    const uint32_t key = key_of(group), last = most > 0 ? most - 1 : 0;
    const uint32_t pos = min(key, last);
    const int32_t pg = most > 0 ? *(gptr_i32)(table + 4 * (uint64_t)div_by(pos, p.page)) : -1;
    return key == pos && (uint32_t)pg < (uint32_t)c.pages ? pg : -1;
  };
  const auto bias_of = [&](int group, int32_t pg) -> float {
    float x = 0.f;
    if (has_bias) {
      const uint32_t key = min(key_of(group), (uint32_t)most);
      const uint32_t tk = key - div_by(key, p.page) * p.page.d;
      x = *(gptr_f32)(bbase + (uint64_t)((pg < 0 ? 0 : pg) * c.bias_stride[0] + tk * c.bias_stride[1]) * 4);
    }
    return pg < 0 ? -INFINITY : x;
  };
  const auto put_rows = [&](int group, int32_t pg, float bias) {
    const uint32_t key = key_of(group);
    const uint32_t tk = key - div_by(key, p.page) * p.page.d;
    const bool live = bias != -INFINITY;
    const uint64_t ka = kbase + (uint64_t)(pg * c.k_stride[0] + tk * c.k_stride[1]) * eb;
    const uint64_t va = vbase + (uint64_t)(pg * c.v_stride[0] + tk * c.v_stride[1]) * eb;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    row_k[w][lane] = live ? ka : zero;
    row_v[group & 1][w][lane] = live ? va : zero;
    const uint64_t ok = __ballot(live);
    if (lane < GS) {
      char* to = (char*)&valid[group & 1][lane];
      if constexpr (share == 8) ((uint8_t*)to)[w] = (uint8_t)(ok >> (lane * 8));
      else ((uint16_t*)to)[w] = (uint16_t)(ok >> (lane * 16));
    }
    if constexpr (EXTRA) biases[group & 1][gs][gj] = bias;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };
  const int unit = lane % L::units, sub = lane / L::units;
  // Rows of step st to LDS. (Units past DC are never read.)
  const auto load_rows = [&](int st, const uint64_t* rows, auto swizzle, lptr8 to) {
    const int s = (st - t0) % GS;
    uint64_t ad[L::loads];
#pragma unroll
    for (int i = 0; i < L::loads; ++i) ad[i] = rows[s * share + i * L::per_load + sub];
#pragma unroll
    for (int i = 0; i < L::loads; ++i) {
      const int u = unit ^ swizzle(w * share + i * L::per_load + sub);
      if (DC == L::pitch || u * L::unit < DC)
        load_to_lds((u * L::unit < D ? ad[i] : zero) + u * 16, to + (w * share + i * L::per_load) * rb);
    }
  };
  const auto load_k = [&](int st, lptr8 to) { load_rows(st, row_k[w], key_swizzle<L>, to); };
  const auto load_v = [&](int st, lptr8 to) {
    load_rows(st, row_v[((st - t0) / GS) & 1][w], value_swizzle<L>, to);
  };

  floatx16_t o[L::dt];
#pragma unroll
  for (int i = 0; i < L::dt; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
  float m = -INFINITY, l = 0.f;
  bool looked = false, broken_before = false;
  const float unit_log2 = EXTRA ? kLog2e : a.scale * kLog2e;      // of a score as it is held
  const float cap = a.softcap, inv_cap = cap > 0.f ? 1.f / cap : 0.f;
  constexpr float shift = prob_shift<DT>, slack = prob_slack<DT>;

  // One step of the pipeline: the products of step st - 1's probabilities with its values and the
  // scores of step st + 1 keep the matrix units busy while the vector units make step st's
  // probabilities of its scores. A wave issues both in turn: after each product some of
  // the work on probabilities, which the product takes longer than; what the products read from LDS is
  // asked for two of them ahead. Loads for later steps go to the other buffers. masked: some key
  // of the step is hidden from some row.
  uint4 pr[DT == FK_F32 ? 1 : KT][2];                  // probabilities, 16 bits
  float pf[DT == FK_F32 ? KT : 1][16];                 // and fp32
  float grown = 1.f;                                   // what the sums have to be scaled by, and
  bool grew = false;                                   // whether any have

  constexpr int PV = DT == FK_F32 ? KT * 16 * L::dt : KT * 2 * L::dt, QK = KT * L::kt;
  const int l16 = lane & 15;
  // Lane's place in the rows of keys and values; other units lie at the place with bits flipped
  // (a row's length is a multiple of what is flipped).
  uint32_t key_place = n * rb + (h ^ key_swizzle<L>(n)) * 16;
  uint32_t value_place = DT == FK_F32
      ? 4 * h * rb + ((n >> 2) ^ value_swizzle<L>(4 * h)) * 16 + (n & 3) * 4
      : (4 * h + (l16 >> 2)) * rb + ((((lane >> 4) & 1) * 2 + ((l16 & 3) >> 1)) ^ value_swizzle<L>(l16 >> 2)) * 16 + (l16 & 1) * 8;
  const auto value_at = [&](lptr8c v_in, uint32_t place, int i) -> uint4 {        // of product i, tiles d within keys
    const int d = i % L::dt, ks = i / L::dt;
    if constexpr (DT == FK_F32) {
      const int row = (ks >> 4) * 32 + (ks & 3) + 8 * ((ks & 15) >> 2);
      return make_uint4(*(lptr32c)(v_in + row * rb + (place ^ (d * 128))), 0, 0, 0);
    } else {
      lptr8c at_v = v_in + ks * 16 * rb + (place ^ (d * 64));
      const uint2 lo = read_transposed(at_v), hi = read_transposed(at_v + 8 * rb);
      return make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  };
  const auto add_value = [&](const uint4& x, int i) {
    const int d = i % L::dt, ks = i / L::dt;
    if constexpr (DT == FK_F32)
      o[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(__builtin_bit_cast(float, x.x), pf[ks >> 4][ks & 15], o[d], 0, 0, 0);
    else
      o[d] = Mfma<DT>::run(x, pr[ks >> 1][ks & 1], o[d]);
  };
  const auto key_at = [&](lptr8c k_in, uint32_t place, int i) -> uint4 {          // of product i, halves of the keys in turn
    const int u = i % KT, k = i / KT;
    const u32x4 y = *(lptr16c)(k_in + u * 32 * rb + (place ^ (k * 32)));
    return __builtin_bit_cast(uint4, y);
  };
  const auto clear = [](floatx16_t (&x)[KT]) {
#pragma unroll
    for (int u = 0; u < KT; ++u)
#pragma unroll
      for (int j = 0; j < 16; ++j) x[u][j] = 0.f;
  };
  const auto advance = [&](int st, auto tag, floatx16_t (&s)[KT], floatx16_t (&next)[KT],
                           const lptr8c __restrict k_in, const lptr8c __restrict v_in,
                           const lptr8 __restrict k_out, const lptr8 __restrict v_out) {
    constexpr bool masked = decltype(tag)::value;
    const int i = st - t0, key0 = (int)((uint32_t)st * kStep);
    if (st + NB < t1) load_k(st + NB, k_out);
    if (st + NB - 2 < t1) load_v(st + NB - 2, v_out);
    if (grew) {
#pragma unroll
      for (int d = 0; d < L::dt; ++d)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[d][j] *= grown;
    }
    clear(next);
    // (as new numbers every step, so that the flipped places are not kept in registers)
    asm volatile("" : "+v"(key_place), "+v"(value_place));
    uint64_t ok = 0;
    if constexpr (masked && !EXTRA) ok = valid[(i / GS) & 1][i % GS];
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f}, ref = 0.f, off = 0.f, f = 1.f;
    bool grows = false;
    uint32_t made[KT][8];
    // the work on probabilities in pieces: scores four by four, the maximum, pairs
    constexpr int prep = KT * 4, pieces = prep + 1 + KT * 8;
    const auto piece = [&](auto number) {
      constexpr int at = decltype(number)::value;
      if constexpr (at < prep) {
        constexpr int u = at / 4, j4 = at % 4;
        float bb[4] = {0.f, 0.f, 0.f, 0.f};
        if constexpr (EXTRA) {
          const float4 bs = *(const float4*)&biases[(i / GS) & 1][i % GS][u * 32 + j4 * 8 + h * 4];
          bb[0] = bs.x, bb[1] = bs.y, bb[2] = bs.z, bb[3] = bs.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x = s[u][j4 * 4 + j];
          if constexpr (SCORE == kNearCapScore) {
            x = cap_16bit(x * a.scale, cap, inv_cap) + bb[j];
          } else if constexpr (SCORE == kCapScore) {
            x *= a.scale;
            if (DT != FK_F32 || cap > 0.f) x = capped(x, cap, inv_cap);
            x += bb[j];
          } else if constexpr (EXTRA) {
            x = fmaf(x, a.scale, bb[j]);
          }
          // (a key that is out has a score of 0, or NaN where the query is not finite:
          // then all steps are masked ones)
          if constexpr (EXTRA && masked) x = bb[j] == -INFINITY ? -INFINITY : x;
          if constexpr (masked) {
            const int key = u * 32 + j4 * 8 + h * 4 + j;
            x = key0 + key < limit && (EXTRA || ((ok >> key) & 1)) ? x : -INFINITY;
          }
          s[u][j4 * 4 + j] = x;
          top[j & 1] = fmaxf(top[j & 1], x);
        }
      } else if constexpr (at == prep) {
        const float t = max_halves(fmaxf(top[0], top[1]));
        grows = (t - m) * unit_log2 > slack;
        const float mn = grows ? fmaxf(m, t) : m;
        f = grows ? fast_exp2((m - mn) * unit_log2) : 1.f;
        m = mn;
        ref = m == -INFINITY ? 0.f : m;
        off = fmaf(-ref, unit_log2, shift);
      } else {
        constexpr int pair = at - prep - 1, u = pair / 8, j0 = pair % 8 * 2;
#pragma unroll
        for (int j = j0; j < j0 + 2; ++j) {
          float x;
          if constexpr (DT == FK_F32) x = prob<DT>(s[u][j] - ref);
          else if constexpr (EXTRA) x = fast_exp2(fmaf(s[u][j] - ref, kLog2e, shift));
          else x = fast_exp2(fmaf(s[u][j], unit_log2, off));
          s[u][j] = x;
          sum[j & 1] += x;
        }
        if constexpr (DT != FK_F32) {
          typedef typename Val<DT>::arith T;
          typedef T T2 __attribute__((ext_vector_type(2)));
          T2 two = {(T)s[u][j0], (T)s[u][j0 + 1]};
          // Rounded once; their sum is not. Next to the result's own rounding, which 64-bit results have too
          // (1.66e-3 of their size in bf16, 2.06e-4 in fp16), that makes 1.98e-3 and 2.22e-4. As sums of two numbers,
          // each multiplied, probabilities add nothing, and 32768 tokens take 13.0 ms instead of 8.6, 1024 53 us
          // instead of 35: the products with values are half of all.
          // (An infinite value times a probability that rounds to 0 would be NaN; in steps
          // that hide no key 2^-24, 2^-37 of the largest one, stands for those.)
          if constexpr (DT == FK_F16 && !masked) two = __builtin_elementwise_max(two, (T2)(T)0x1p-24f);
          uint32_t word = __builtin_bit_cast(uint32_t, two);
          asm volatile("" : "+v"(word));               // made here, not where it is used
          made[u][pair % 8] = word;
        }
      }
    };
    constexpr int products = PV + QK, ahead = DT == FK_F32 || DC > 128 ? 4 : 2;
    uint4 in[ahead + 1];
    const auto input = [&](int at) {
      return at < PV ? value_at(v_in, value_place, at) : key_at(k_in, key_place, at - PV);
    };
#pragma unroll
    for (int at = 0; at < ahead; ++at) in[at] = input(at);
    each<products>([&](auto number) {
      constexpr int at = decltype(number)::value;
      if constexpr (at + ahead < products) in[(at + ahead) % (ahead + 1)] = input(at + ahead);
      const uint4 x = in[at % (ahead + 1)];
      if constexpr (at < PV) add_value(x, at);
      else next[(at - PV) % KT] = Mfma<DT>::run(x, q[(at - PV) / KT], next[(at - PV) % KT]);
      constexpr int from = at * pieces / products, to = (at + 1) * pieces / products;
      each<to - from>([&](auto more) { piece(std::integral_constant<int, from + decltype(more)::value>()); });
      __builtin_amdgcn_sched_barrier(0);
    });
    l = fmaf(l, f, sum[0] + sum[1]);
    grown = f, grew = __any(grows);
#pragma unroll
    for (int u = 0; u < KT; ++u) {
      if constexpr (DT == FK_F32) {
#pragma unroll
        for (int j = 0; j < 16; ++j) pf[u][j] = s[u][j];
      } else {
#pragma unroll
        for (int sb = 0; sb < 2; ++sb)
          pr[u][sb] = make_uint4(made[u][sb * 4], made[u][sb * 4 + 1], made[u][sb * 4 + 2], made[u][sb * 4 + 3]);
      }
    }
  };
  const auto all_valid = [&](int st) {                 // every key of step st counts
    const int i = st - t0;
    const uint64_t ok = valid[(i / GS) & 1][i % GS];
    const uint32_t both = kStep == 32 ? (uint32_t)ok : (uint32_t)(ok & (ok >> 32));
    return __builtin_amdgcn_readfirstlane(both) == 0xFFFFFFFFu;
  };

  floatx16_t sa[KT], sb[KT];                           // scores of a step and of the next, in turn
  int32_t pg1 = -1, pg2 = -1;
  float bias1 = -INFINITY;
  const auto find_rows = [&](int st) {                 // before the keys of step st are asked for
    const int i = st - t0;
    if (i % GS != 0 || st >= t1) return;
    put_rows(i / GS, pg1, bias1);
    pg1 = pg2;
    bias1 = bias_of(i / GS + 1, pg1);
    pg2 = entry(i / GS + 2);
  };
  // Rows asked for are in, but for those of the last step where there are three buffers and it
  // asked for a whole one (loads come back in order); earlier steps are done with.
  const auto meet = [&](bool all) {
    constexpr int last = NB == 3 ? 2 * L::loads : 0;
    if (NB == 2 || all) __builtin_amdgcn_s_waitcnt(0x0F70);                              // vmcnt(0)
    else __builtin_amdgcn_s_waitcnt(0x0F70 | (last & 15) | (last >> 4) << 14);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  };
  // Buffer of step st's keys and values.
  int buf = 0;                                         // of the step that is at
  const auto after = [&](int k) { return NB == 2 ? buf ^ (k & 1) : (buf + k) % 3; };
  const auto keys_of = [&](int k) { return (lptr8)(lk[0]) + after(k) * (kStep * rb); };
  const auto values_of = [&](int k) { return (lptr8)(lv[0]) + after(k) * (kStep * rb); };
  // A sum in 32 bits of n terms alike may be off by n 2^-25 of itself, and fp32 products add two keys at a
  // time (16-bit ones 16): the sums over kRun steps, 2^15 terms, are added to the row's place in the
  // results or the workspace, where they are held scaled to `m_kept`. l has a term a step and stays in one
  // piece (held apart as well, in a register or in LDS, every fp32 call took 1 to 3% longer).
  constexpr int kRun = 1 << 10;
  bool kept = false;
  float m_kept = -INFINITY;
  const auto with_kept = [&](auto each_four) {         // the lane's sums and their place, four by four
    if (grew) {                                        // (what these sums wait for)
#pragma unroll
      for (int d = 0; d < L::dt; ++d)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[d][j] *= grown;
    }
    grew = false, grown = 1.f;
    const float f = m_kept == m ? 1.f : fast_exp2((m_kept - m) * unit_log2);
    const int64_t row = t * a.Hq + qh;
    float* to = p.parts > 1 && steps > p.chunk ? p.o + ((int64_t)part * a.T * a.Hq + row) * D : (float*)a.out + row * D;
    if (!mine || t < 0 || t >= a.T) return;
#pragma unroll
    for (int d = 0; d < L::dt; ++d)
#pragma unroll
      for (int j4 = 0; j4 < 4; ++j4) {
        const int e = d * 32 + j4 * 8 + h * 4;
        if (e < D) each_four((float4*)(to + e), f, d, j4 * 4);
      }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // (waits for keys and values count on no other accesses)
  };
  const auto keep = [&] {
    with_kept([&](float4* to, float f, int d, int j) {
      float4 x = kept ? *to : make_float4(0.f, 0.f, 0.f, 0.f);
      x = make_float4(fmaf(x.x, f, o[d][j]), fmaf(x.y, f, o[d][j + 1]), fmaf(x.z, f, o[d][j + 2]), fmaf(x.w, f, o[d][j + 3]));
      *to = x;
    });
#pragma unroll
    for (int d = 0; d < L::dt; ++d)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[d][j] = 0.f;
    kept = true, m_kept = m;
  };
  const auto take_back = [&] {
    with_kept([&](float4* to, float f, int d, int j) {
      const float4 x = *to;
      o[d][j] = fmaf(x.x, f, o[d][j]), o[d][j + 1] = fmaf(x.y, f, o[d][j + 1]);
      o[d][j + 2] = fmaf(x.z, f, o[d][j + 2]), o[d][j + 3] = fmaf(x.w, f, o[d][j + 3]);
    });
    kept = false;
  };
  bool finite = true;                                  // every query of the wave
  const int own_end = min(t1, (int)(((uint32_t)high + kStep - 1) / kStep));     // steps of this wave
  if (t0 < t1) {
    pg1 = entry(0), pg2 = entry(1);
    const uint64_t qp = (uint64_t)a.q + (uint64_t)(t * a.q_stride[0] + qh * a.q_stride[1]) * eb;
#pragma unroll
    for (int i = 0; i < L::kt; ++i) {
      const int e = (2 * i + h) * L::unit;
      q[i] = load16(e < D && mine && t >= 0 && t < a.T ? qp + e * eb : (uint64_t)zero_row);
    }
    bias1 = bias_of(0, pg1);
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      if (t0 + k >= t1) break;
      find_rows(t0 + k);
      load_k(t0 + k, keys_of(k));
    }
    if (NB == 3) load_v(t0, values_of(0));
    // the pipeline starts with no values and no probabilities
    for (int i = threadIdx.x; i < kStep * rb / 16; i += W * 64) ((uint4*)lv[NB - 1])[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < KT; ++u) {
      if constexpr (DT != FK_F32) pr[u][0] = pr[u][1] = make_uint4(0, 0, 0, 0);
      else
#pragma unroll
        for (int j = 0; j < 16; ++j) pf[u][j] = 0.f;
    }
    // (waited for here, or every step would wait for loads as if these were on their way)
#pragma unroll
    for (int i = 0; i < L::kt; ++i)
      asm volatile("" : "+v"(q[i].x), "+v"(q[i].y), "+v"(q[i].z), "+v"(q[i].w));
    if constexpr (EXTRA && DT != FK_F32) {
      uint32_t bad = 0;
#pragma unroll
      for (int i = 0; i < L::kt; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          constexpr uint32_t top = DT == FK_F16 ? 0x7C00u : 0x7F80u;      // of a number that is not finite
          const uint32_t x = word(q[i], j);
          bad |= (x & top) == top || ((x >> 16) & top) == top;
        }
      finite = !__any(bad);
    }
    meet(true);
    clear(sa);
#pragma unroll
    for (int at = 0; at < QK; ++at)
      sa[at % KT] = Mfma<DT>::run(key_at((lptr8c)lk[0], key_place, at), q[at / KT], sa[at % KT]);
  }
  // Steps that every row sees whole, then the others: every wave changes over in its own time
  // (a barrier counts waves, wherever they stand). fp32 products take longer than the
  // masks.
  int st = t0;
  bool here = false;                                   // step st has met already
  const auto few = [&] { return st + NB - 1 >= t1 || st == t0; };       // the last step asked for less than a whole one
  if constexpr (DT != FK_F32) {
    const int whole = finite ? min(t1, low / kStep) : t0;
    for (; st + 2 <= whole; st += 2) {                 // two at a time, so that scores change places
      meet(few());
      if (!EXTRA && !(all_valid(st) && all_valid(st + 1))) {
        here = true;
        break;
      }
      find_rows(st + NB);
      advance(st, std::false_type(), sa, sb, keys_of(1), values_of(NB - 1), keys_of(0), values_of(NB - 2));
      buf = after(1);
      meet(st + NB >= t1);
      find_rows(st + 1 + NB);
      advance(st + 1, std::false_type(), sb, sa, keys_of(1), values_of(NB - 1), keys_of(0), values_of(NB - 2));
      buf = after(1);
    }
  }
  for (; st < own_end; ++st, here = false) {
    if (!here) meet(few());
    find_rows(st + NB);
    advance(st, std::true_type(), sa, sb, keys_of(1), values_of(NB - 1), keys_of(0), values_of(NB - 2));
    buf = after(1);
#pragma unroll
    for (int u = 0; u < KT; ++u) sa[u] = sb[u];
    if constexpr (DT == FK_F32)
      if ((st - t0) % kRun == kRun - 1) keep();
    if (!looked && (uint32_t)(st + 1) * kStep > (uint32_t)low) {           // (its hidden values have not been added yet)
      looked = true;
      if (DT == FK_F32 && kept) take_back();
      const bool fine = all_finite<L::dt>(o);
      broken_before = __any(!fine);
      if (broken_before) broken[threadIdx.x] = not_finite<L::dt>(o, fine);
    }
  }
  for (; st <= t1 && t0 < t1; ++st, here = false) {    // the last values, and the other waves' steps
    if (!here) meet(few());
    if (st == own_end) {
#pragma unroll
      for (int d = 0; d < L::dt; ++d)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[d][j] *= grown;
      grew = false, grown = 1.f;                       // (done, for take_back() too)
      each<PV>([&](auto number) {
        constexpr int at = decltype(number)::value;
        add_value(value_at((lptr8c)values_of(NB - 1), value_place, at), at);
      });
    }
    find_rows(st + NB);
    if (st + NB < t1) load_k(st + NB, keys_of(0));
    if (st + NB - 2 < t1) load_v(st + NB - 2, values_of(NB - 2));
    buf = after(1);
  }
  if (DT == FK_F32 && kept) take_back();
  l = sum_halves(l);
  const int64_t row = t * a.Hq + qh;
  const float m_nat = EXTRA ? m : m * a.scale;
  const bool cut = p.parts > 1 && steps > p.chunk;
  const bool put = mine && t >= 0 && t < a.T;
  const int64_t at_o = (int64_t)part * a.T * a.Hq + row;
  if (put && cut) {
#pragma unroll
    for (int d = 0; d < L::dt; ++d)
#pragma unroll
      for (int j4 = 0; j4 < 4; ++j4) {
        const int e = d * 32 + j4 * 8 + h * 4;
        if (e < D) *(float4*)(p.o + at_o * D + e) = make_float4(o[d][j4 * 4], o[d][j4 * 4 + 1], o[d][j4 * 4 + 2], o[d][j4 * 4 + 3]);
      }
    if (h == 0) p.ml[at_o * 2] = l == 0.f ? -INFINITY : m_nat, p.ml[at_o * 2 + 1] = l;
  } else if (put) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int d = 0; d < L::dt; ++d)
#pragma unroll
      for (int j4 = 0; j4 < 4; ++j4) {
        const int e = d * 32 + j4 * 8 + h * 4;
        const float x[4] = {o[d][j4 * 4] * inv, o[d][j4 * 4 + 1] * inv, o[d][j4 * 4 + 2] * inv, o[d][j4 * 4 + 3] * inv};
        if (e < D) store4<DT>(a.out, row * D + e, x);
      }
    if (a.lse && h == 0) a.lse[row] = l == 0.f ? -INFINITY : m_nat + (logf(l) - shift * kLn2);
  }
  // A hidden key's probability is 0, but 0 times an infinity or NaN of its value is NaN. Rows whose
  // sums stopped being finite in steps that hide keys, or where some were not finite before and others became NaN,
  // are done again, key by key.
  bool again = looked && put && l - l == 0.f && !all_finite<L::dt>(o);
  if (broken_before && __any(again)) again = again && newly<L::dt>(not_finite<L::dt>(o, false), broken[threadIdx.x]);
  uint64_t todo = __ballot(again);
  todo = (todo | todo >> 32) & 0xFFFFFFFFu;
  constexpr int EPL = (DC + 63) / 64;
  while (todo) {
    const int i = __builtin_ctzll(todo);
    todo &= todo - 1;
    const int64_t t2 = __shfl(t, i, 64), h2 = __shfl(qh, i, 64), row2 = t2 * a.Hq + h2;
    const int64_t end = min((int64_t)__shfl(limit, i, 64), (int64_t)t1 * kStep);
    float m2, l2, o2[EPL];
    row_sums<DT, EPL>(a, b, t2, h2, (int64_t)t0 * kStep, end, m2, l2, o2);
    if (!cut) {
      put_row<DT, EPL>(a, row2, m2, l2, o2);
      continue;
    }
    const int64_t at2 = (int64_t)part * a.T * a.Hq + row2;
    const float f = 1 << (int)shift;
#pragma unroll
    for (int e = 0; e < EPL; ++e)
      if (lane + 64 * e < D) p.o[at2 * D + lane + 64 * e] = o2[e] * f;
    if (lane == 0) p.ml[at2 * 2] = m2, p.ml[at2 * 2 + 1] = l2 * f;
  }
}

// Joins the partial results of rows whose keys were cut, a row a wave.
template <int DT, int DC, int W>
__global__ __launch_bounds__(kWaves * 64) void prompt_join_kernel(PromptArgs a, PromptPlan p) {
  constexpr int EPL = (DC + 63) / 64, rows = Tile<DT, DC, W>::rows, kStep = Tile<DT, DC, W>::step;
  const int64_t r = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  const int64_t t = r / a.Hq, b = t < a.T ? request_of(a, t) : -1;
  if (b < 0) return;
  const int lane = threadIdx.x & 63, D = (int)a.cache.dim;
  // steps of the row's tile, by its last row
  const int64_t n = (a.cu[b + 1] - a.cu[b]) * (int64_t)p.G;
  const int64_t own = (t - a.cu[b]) * p.G + (r - t * a.Hq) % p.G;
  const int64_t last = min((own / rows + 1) * rows, n) - 1;
  const int64_t steps = (seen_by(a, b, a.cu[b] + last / p.G) + kStep - 1) / kStep;
  if (steps <= p.chunk) return;
  const int parts = (int)min((int64_t)p.parts, (steps + p.chunk - 1) / p.chunk);
  const int64_t every = a.T * a.Hq;
  // a part a lane (there are 64 at most), then eight parts' rows at a time
  const float2 ml = lane < parts ? *(const float2*)(p.ml + (lane * every + r) * 2) : make_float2(-INFINITY, 0.f);
  float m = ml.x;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  const float f = join_factor(ml.x, ml.y, m), l = wave_sum(f * ml.y);
  float o[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) o[e] = 0.f;
  for (int i0 = 0; i0 < parts; i0 += 8) {
    float x[8][EPL];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        const int64_t at = (min(i0 + i, parts - 1) * every + r) * D + lane + 64 * e;
        x[i][e] = lane + 64 * e < D ? p.o[at] : 0.f;
      }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float g = __shfl(f, min(i0 + i, 63), 64);          // (0 past the last part)
      // (a part without keys has left no row: what is there is not to be used)
#pragma unroll
      for (int e = 0; e < EPL; ++e) o[e] = g == 0.f ? o[e] : fmaf(g, x[i][e], o[e]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < EPL; ++e)
    if (lane + 64 * e < D)
      Val<DT>::put((typename Val<DT>::type*)a.out + r * D + lane + 64 * e, o[e] * inv);
  if (a.lse && lane == 0) a.lse[r] = l == 0.f ? -INFINITY : m + (logf(l) - prob_shift<DT> * kLn2);
}

// Numbers of a cache head's tiles: as many as there can be (count_tiles), or as are searched (search_tile).
int64_t tile_numbers(const PromptArgs& a, int64_t rows) {
  const int64_t all = a.T * (a.Hq / a.cache.heads);
  return a.B <= 64 ? (all + rows - 1) / rows + a.B - 1 : all / rows + a.B;
}

// Parts that a row's keys may be cut into: four blocks a CU at most. (Two of them keep the
// workspace half as large, and 4 requests of 250 to 999 tokens behind 1056 centres, fp32, take 117 us
// instead of 106, 1024 tokens of 64 elements 102 instead of 94.)
int64_t most_parts(int64_t T, int64_t G, int64_t heads, int64_t rows) {
  const int64_t units = (T * G + rows - 1) / rows * heads;
  const int64_t n = 4 * kMaxCus / (units < 1 ? 1 : units);
  return n < 1 ? 1 : (n > 64 ? 64 : n);
}

// What is known of a call without its lengths: tiles of so many rows at least, and the steps of a
// row, from the fewest to the most (all keys but the tokens behind it).
struct Outline {
  int64_t tiles, longest;
  double fewest, mean;
};
inline Outline outline(const PromptArgs& a, int64_t rows, int64_t step) {
  const int64_t G = a.Hq / a.cache.heads, full = (a.T * G + rows - 1) / rows, most = longest(a);
  const int64_t each = a.T / a.B < most ? a.T / a.B : most, longest = (most + step - 1) / step;
  const double fewest = (double)(most - each) / (double)step;
  return {full > a.B ? full : a.B, longest, fewest, 0.5 * (longest + fewest)};
}

// Microseconds of a call whose keys are cut into `parts`, from what was measured: products at
// 1000 TFLOP/s over the chip (16 bits; 700 for rows of 64 and less, 103 for fp32), 5% less for two
// blocks a CU; 15 us of a block before and after its steps, 3 more for a partial result; 6 us and
// 4 TB/s to join them. Blocks are taken longest first. A block of 4 waves alone on its
// CU is 1.6 times as fast as next to another, in fp32 1.95 times. Rows that see unlike numbers
// of keys leave CUs free for each other; where all are alike, a last round is as long as any.
inline double estimate(int dt, int DC, int W, int step, const PromptArgs& a, const Outline& o, int64_t parts) {
  const double cus = device_cus(), slots = cus * tile_blocks(dt, DC, W), rows = W * 32;
  const double rate = dt == FK_F32 ? 103e6 : DC <= 64 ? 700e6 : 1000e6;
  const double together = (slots > cus ? 1.05 : 1.) * 4. * rows * step * DC / (rate / slots);
  const double alone = slots > cus ? together / (dt == FK_F32 ? 1.95 : 1.6) : together;
  const double units = (double)o.tiles * a.cache.heads, fixed = parts > 1 ? 18. : 15.;
  const int64_t chunk = (o.longest + parts - 1) / parts;
  double blocks = 0.;                                  // with work: rows with few keys have few parts
  for (int64_t p = 0; p < parts && p * chunk < o.longest; ++p) {
    const double from = p * chunk > o.fewest ? (double)(p * chunk) : o.fewest;
    blocks += units * (p * chunk <= o.fewest ? 1. : (o.longest - from) / (o.longest - o.fewest));
  }
  double us;
  if (blocks <= slots) {
    // next to another block until that ends, a long one next to a short one
    const double first = chunk * alone + (parts == 1 && blocks > cus ? o.fewest * (together - alone) : 0.);
    const double mean = parts == 1 ? o.fewest : units * o.mean / blocks;         // beside the longest
    const double both = blocks > cus ? 0.5 * (chunk + mean) * together : 0.;
    us = (first > both ? first : both) + fixed;
  } else {
    const double alike = o.longest > 0 ? 2. * (o.mean / o.longest - 0.5) : 1.;
    const double one = chunk * together + fixed, all = (units * o.mean * together + blocks * fixed) / slots;
    const double uneven = (all > one ? all : one) + 0.2 * one, even = ceil(blocks / slots) * one;
    us = (1. - alike) * uneven + alike * even;
  }
  if (parts > 1) us += 6. + (double)(a.T * a.Hq) * parts * (a.cache.dim + 2) * 8. / 4e6;
  return us;
}

// The number of parts with the shortest estimate, of those that a launch can hold.
struct Best {
  double us;
  int parts;
};
inline Best best_parts(int dt, int DC, int W, int step, const PromptArgs& a) {
  const Outline o = outline(a, W * 32, step);
  const int64_t most = most_parts(a.T, a.Hq / a.cache.heads, a.cache.heads, W * 32);
  const int64_t blocks = tile_numbers(a, W * 32) * a.cache.heads;
  Best best{1e300, 1};
  for (int64_t n = 1; n <= most && (n == 1 || o.longest >= 4 * n) && blocks <= most_blocks(W) / n; ++n) {
    const double us = estimate(dt, DC, W, step, a, o, n);
    if (us < best.us) best = {us, (int)n};
  }
  return best;
}

template <int DT, int DC, int W> hipError_t run_tiles(const PromptArgs& a, int parts, void* ws, hipStream_t s) {
  using L = Tile<DT, DC, W>;
  PromptPlan p{};
  p.heads = (int)a.cache.heads;
  p.G = (int)(a.Hq / a.cache.heads);
  const Outline o = outline(a, L::rows, L::step);
  const int64_t tiles = tile_numbers(a, L::rows), blocks = tiles * p.heads * parts;
  if (blocks > most_blocks(W) || a.T * p.G > 0x7FFFFFFF - 512 ||
      (parts > 1 && (a.T * a.Hq + kWaves - 1) / kWaves > most_blocks(kWaves)))
    return hipErrorInvalidConfiguration;
  p.parts = parts;
  p.chunk = p.parts == 1 ? 0x7FFFFFFF / L::step : (int)((o.longest + p.parts - 1) / p.parts);
  p.o = (float*)ws;
  p.ml = p.o + (int64_t)p.parts * a.T * a.Hq * a.cache.dim;
  p.page = fast_div((uint32_t)a.cache.page);
  p.by_heads = fast_div((uint32_t)p.heads);
  p.by_tiles = fast_div((uint32_t)tiles);
  p.by_G = fast_div((uint32_t)p.G);
  // Where every block finds room at once, two to a CU, the second half comes in turned order: the
  // longest share a CU with the shortest. (2048 tokens, bf16: 70 us in one order, 61; fp32 rows of
  // 64: 253 and 205.)
  const int64_t each = device_cus() / p.heads;
  const bool pairs = tile_blocks(DT, DC, W) == 2 && p.parts == 1 && blocks <= 2 * device_cus() + p.heads * a.B;
  p.last = (uint32_t)(tiles * p.parts - 1);
  p.turn = pairs ? (uint32_t)each : 0xFFFFFFFFu;
  auto kernel = prompt_mfma_kernel<DT, DC, W, kCapScore>;
  if constexpr (DT != FK_F32) {
    if (a.softcap > 0.f && a.softcap <= kNearCap)
      kernel = prompt_mfma_kernel<DT, DC, W, kNearCapScore>;
    else if (a.softcap == 0.f)
      kernel = a.cache.key_bias || !(a.scale > 0.f) ? prompt_mfma_kernel<DT, DC, W, kBiasScore>
                                                    : prompt_mfma_kernel<DT, DC, W, kPlainScore>;
  }
  kernel<<<(unsigned)blocks, W * 64, 0, s>>>(a, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.parts == 1) return e;
  prompt_join_kernel<DT, DC, W><<<(unsigned)((a.T * a.Hq + kWaves - 1) / kWaves), kWaves * 64, 0, s>>>(a, p);
  return hipGetLastError();
}

// Tiles of 256 rows or of 128, of which two blocks share a CU. (16-bit, 32 heads of 128 on 8, 4096
// tokens: 163 us, 178 with 128 rows; 16384: 2340 and 2510; 512: 29 and 23; 8192 tokens of 8
// heads on 8: 236 and 193; 64 requests of one token over 8192 keys: 341 and 215.)
template <int DT, int DC> hipError_t run_mfma(const PromptArgs& a, void* ws, hipStream_t s) {
  const Best four = best_parts(DT, DC, 4, Tile<DT, DC, 4>::step, a);
  if constexpr (!only_four(DT, DC)) {
    const Best eight = best_parts(DT, DC, 8, Tile<DT, DC, 8>::step, a);
    if (eight.us < 0.97 * four.us) return run_tiles<DT, DC, 8>(a, eight.parts, ws, s);
  }
  return run_tiles<DT, DC, 4>(a, four.parts, ws, s);
}

}  // namespace
}  // namespace fk

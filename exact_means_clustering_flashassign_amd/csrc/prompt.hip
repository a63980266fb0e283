// Attention of a step's prompts: rows of any layout, and the choice of kernel.
#include "prompt.hpp"

#include <algorithm>

namespace fk {
namespace {

// Rows of any size, stride and alignment: all fp32 ones, 16-bit ones where they are few (few_rows). The
// rows of a request are laid out as for the matrix-core kernel (row r is head r % G of token
// r / G); a block takes R of one cache head, a wave every fourth step of 64 keys. For scores a lane has a key: 64 elements of every key go to LDS, an
// element a lane as they lie in memory, and are read back a key a lane, next to the R queries'
// elements. For sums a lane has every 64th element, and probabilities come back from LDS a key
// at a time. So a key or value is loaded once for R rows, and nothing is summed over lanes but a
// step's maxima. Bound by instructions: 1024 tokens, 32 heads of 65 on 8, 0.37 ms (a row a wave,
// each score summed over the lanes: 2.7 ms).
template <int DT, int EPL, int R>
__global__ __launch_bounds__(kWaves * 64) void prompt_any_kernel(PromptArgs a, PromptPlan p) {
  using E = typename Val<DT>::type;
  typedef float Row __attribute__((ext_vector_type(R)));
  constexpr int pitch = 65;                            // of 64 elements of a key: lanes meet in no bank
  __shared__ __attribute__((aligned(16))) float queries[EPL * 64][R], probs[kWaves][64][R];
  __shared__ float keys[kWaves][64 * pitch];
  __shared__ float tops[kWaves][R], totals[kWaves][R];
  const fk_kv_cache_t& c = a.cache;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int D = (int)c.dim;

  const uint32_t order = div_by(blockIdx.x, p.by_heads), hk = blockIdx.x - order * p.heads;
  const Where at = a.B <= 64 ? count_tiles<R>(a, p.G, order) : search_tile<R>(a, p.G, order);
  if (at.b < 0) return;
  const int64_t cu0 = at.cu0, cu1 = at.cu1, len = at.len;
  const int rows = (int)min((cu1 - cu0) * p.G - (int64_t)at.tile * R, (int64_t)R);
  const int64_t held = min(a.width * c.page, (int64_t)0x7FFFFFFF);
  // row r's token, query head and keys; past the last row its own again
  const auto token = [&](int r) { return cu0 + div_by((uint32_t)(at.tile * R + min(r, rows - 1)), p.by_G); };
  const auto head = [&](int r) {
    const uint32_t i = at.tile * R + min(r, rows - 1);
    return (int64_t)hk * p.G + (i - div_by(i, p.by_G) * p.G);
  };
  int limit[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
    limit[r] = (int)max((int64_t)0, min(len - cu1 + token(r) + 1, held));
  const int most = limit[R - 1], steps = (int)(((uint32_t)most + 63) / 64);

#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t t = token(r);
    const E* q = (const E*)a.q + t * a.q_stride[0] + head(r) * a.q_stride[1];
    for (int e = threadIdx.x; e < EPL * 64; e += kWaves * 64)
      queries[e][r] = e < D && t >= 0 && t < a.T ? Val<DT>::get(q + e) : 0.f;
  }
  __syncthreads();

  const int32_t* table = a.table + at.b * a.ld_table;
  // (a sum in 32 bits stands still after 2^24 terms alike: every kRun steps it joins `all`)
  constexpr int kRun = 1 << 10;
  Row m = -INFINITY, l = 0.f, l_all = 0.f;
  float o[R][EPL], all[R][EPL];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < EPL; ++i) o[r][i] = all[r][i] = 0.f;
  int el[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) el[i] = lane + 64 * i < D ? lane + 64 * i : 0;
  for (int st = w, n = 1; st < steps; st += kWaves, ++n) {
    const uint32_t key = (uint32_t)st * 64 + lane, pos = min(key, (uint32_t)most - 1);
    const uint32_t pg_at = div_by(pos, p.page), tok = pos - pg_at * p.page.d;
    const int64_t page = table[pg_at];
    bool live = key == pos && page >= 0 && page < c.pages;
    float bias = 0.f;
    if (c.key_bias && live) {
      bias = c.key_bias[page * c.bias_stride[0] + tok * c.bias_stride[1] + hk * c.bias_stride[2]];
      live = bias != -INFINITY;
    }
    const uint64_t counts = __ballot(live);
    if (counts == 0) continue;
    const int held_here = min(64, most - st * 64);
    // (in the place of a key that is out another one is read, and not used)
    const int64_t ko = page * c.k_stride[0] + tok * c.k_stride[1] + hk * c.k_stride[2];
    const int64_t vo = page * c.v_stride[0] + tok * c.v_stride[1] + hk * c.v_stride[2];
    const int first = __builtin_ctzll(counts);
    const auto of_lane = [](int64_t x, int i) {
      return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)x, i) |
                       (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), i) << 32);
    };
    const int64_t k_at = live ? ko : of_lane(ko, first), v_at = live ? vo : of_lane(vo, first);

    Row s = 0.f;
    float* const mine = keys[w];
    for (int e0 = 0; e0 < D; e0 += 64) {
      const int e = e0 + lane < D ? e0 + lane : 0;
#pragma unroll 1
      for (int j0 = 0; j0 < held_here; j0 += 32) {
        float x[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = Val<DT>::get((const E*)c.k + of_lane(k_at, j0 + j) + e);
#pragma unroll
        for (int j = 0; j < 32; ++j) mine[(j0 + j) * pitch + lane] = x[j];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const int count = min(64, D - e0);
#pragma unroll 4
      for (int i = 0; i < count; ++i) s += *(const Row*)queries[e0 + i] * mine[lane * pitch + i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    Row pr, alpha;
    const bool whole = counts == ~(uint64_t)0 && (uint32_t)st * 64 + 64 <= (uint32_t)limit[0];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float x = s[r] * a.scale;
      if (a.softcap > 0.f) x = capped(x, a.softcap, 1.f / a.softcap);
      x = live && key < (uint32_t)limit[r] ? x + bias : -INFINITY;
      float top = x;
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
      const float mr = m[r], mn = fmaxf(mr, top);
      alpha[r] = mr == -INFINITY ? 0.f : fast_exp2((mr - mn) * kLog2e);
      pr[r] = x == -INFINITY ? 0.f : fast_exp2((x - mn) * kLog2e);       // NaN stays NaN
      m[r] = mn;
    }
    l = l * alpha + pr;
    l_all *= alpha;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < EPL; ++i) o[r][i] *= alpha[r], all[r][i] *= alpha[r];
    *(Row*)probs[w][lane] = pr;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const auto sums = [&](auto tag) {
      constexpr bool masked = !decltype(tag)::value;
      constexpr int U = EPL <= 4 ? 8 : 32 / EPL;
#pragma unroll 1
      for (int j0 = 0; j0 < held_here; j0 += U) {
        float x[U][EPL];
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const E* v = (const E*)c.v + of_lane(v_at, j0 + j);
#pragma unroll
          for (int i = 0; i < EPL; ++i) x[j][i] = Val<DT>::get(v + el[i]);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const Row y = *(const Row*)probs[w][j0 + j];
          const bool out = masked && !((counts >> (j0 + j)) & 1);
#pragma unroll
          for (int i = 0; i < EPL; ++i) {
            const float v = out ? 0.f : x[j][i];
#pragma unroll
            for (int r = 0; r < R; ++r) {
              // (a value that is not finite does not reach the rows it is hidden from)
              const float sum = fmaf(y[r], v, o[r][i]);
              o[r][i] = !masked || (uint32_t)(st * 64u + j0 + j) < (uint32_t)limit[r] ? sum : o[r][i];
            }
          }
        }
      }
    };
    if (whole) sums(std::true_type());
    else sums(std::false_type());
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (n % kRun == 0) {
      l_all += l, l = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < EPL; ++i) all[r][i] += o[r][i], o[r][i] = 0.f;
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float total = wave_sum(l[r] + l_all[r]);
    if (lane == 0) tops[w][r] = m[r], totals[w][r] = total;
  }
  // the waves' sums, in the keys' place, as many elements at a time as it holds
  constexpr int G = R * EPL <= pitch ? EPL : pitch / R;
#pragma unroll
  for (int i0 = 0; i0 < EPL; i0 += G) {
    if (i0 > 0) __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = i0; i < i0 + G; ++i) keys[w][(r * G + i - i0) * 64 + lane] = o[r][i] + all[r][i];
    __syncthreads();
    for (int r = 0; r < rows; ++r) {
      const int64_t t = token(r), row = t * a.Hq + head(r);
      if (t < 0 || t >= a.T) continue;
      float top = tops[0][r];
      for (int k = 1; k < kWaves; ++k) top = fmaxf(top, tops[k][r]);
      float f[kWaves], total = 0.f;
      for (int k = 0; k < kWaves; ++k) {
        f[k] = join_factor(tops[k][r], totals[k][r], top);
        total += f[k] * totals[k][r];
      }
      const bool any = total != 0.f;     // true for NaN: it has to reach the result
      for (int e = threadIdx.x; e < G * 64 && i0 * 64 + e < D; e += kWaves * 64) {
        float x = 0.f;
        for (int k = 0; k < kWaves; ++k) x += f[k] * keys[k][r * G * 64 + e];
        Val<DT>::put((E*)a.out + row * D + i0 * 64 + e, any ? x / total : 0.f);
      }
      if (a.lse && i0 == 0 && threadIdx.x == 0) a.lse[row] = any ? top + logf(total) : -INFINITY;
    }
  }
}

template <int DT, int EPL, int R> hipError_t run_any_as(const PromptArgs& a, hipStream_t s) {
  PromptPlan p{};
  p.heads = (int)a.cache.heads;
  p.G = (int)(a.Hq / a.cache.heads);
  p.page = fast_div((uint32_t)a.cache.page);
  p.by_heads = fast_div((uint32_t)p.heads);
  p.by_G = fast_div((uint32_t)p.G);
  const int64_t blocks = tile_numbers(a, R) * p.heads;
  if (blocks > most_blocks(kWaves) || a.T * p.G > 0x7FFFFFFF - R) return hipErrorInvalidConfiguration;
  prompt_any_kernel<DT, EPL, R><<<(unsigned)blocks, kWaves * 64, 0, s>>>(a, p);
  return hipGetLastError();
}

template <int DT> hipError_t run_any(const PromptArgs& a, hipStream_t s) {
  const int64_t D = a.cache.dim;
  if (D <= 64) return run_any_as<DT, 1, 8>(a, s);
  if (D <= 128) return run_any_as<DT, 2, 8>(a, s);
  if constexpr (DT == FK_F32) {
    if (D > 512) return run_any_as<DT, 16, 8>(a, s);
    if (D > 256) return run_any_as<DT, 8, 8>(a, s);
  }
  return run_any_as<DT, 4, 8>(a, s);
}

// Whether 16-bit rows run there too: up to 256 elements, where the chip holds all blocks at once (two a CU
// up to 128 elements) and there are keys for the waves, of which each has its own. A block of
// prompt_split_kernel has all keys to itself. (One token of 32 heads on 8 over 8192 keys, 90 elements 446 us,
// there 1100; 33 284 and 862; 250 1430 and 1680; 512 8700 and 1070. 128 tokens behind 8192, 512 blocks, of 90
// 563 and 1102; 256 tokens 1099 and 1121, 512 2186 and 1327. 64 tokens alone 28 and 14.)
bool few_rows(const PromptArgs& a) {
  const Outline o = outline(a, 8, 64);
  return a.cache.dim <= 256 && longest(a) >= 256 &&
         o.tiles * a.cache.heads <= device_cus() * (a.cache.dim <= 128 ? 2 : 1);
}

// ---------------------------------------------------------------------------
// 16-bit rows that are not whole 16-byte units or have more than 256 elements
// ---------------------------------------------------------------------------
// The layout of the matrix-core kernel (prompt.hpp) with a tile of 32 rows a block, whose waves
// share the elements: a wave makes scores of its quarter of a row, and sums of its quarter of a
// value. The four parts of 32 x 32 scores meet in LDS, two buffers in turn, one barrier a step; all
// waves make the same probabilities of them. Keys and values are read by one wave each, straight
// into the lanes that multiply them: 8 elements of a key (one load where they are whole units), a value of
// 8 keys. Probabilities are scaled and rounded as there. Bound by those loads, which nothing
// hides but other blocks: 2048 tokens, 32 heads of 90 on 8, fp16, 0.63 ms (on the vector units, in the way
// of fp32 rows, 1.27); 1024 of 512 0.30 (3.4), 114 TFLOP/s; 300 of 1000 0.09 (0.74).

// Up to 8 elements from e on, zeros past D.
template <bool UNITS> __device__ __forceinline__ uint4 eight(const uint16_t* row, int e, int D) {
  if constexpr (UNITS) {
    const uint4 x = load16((uint64_t)(row + (e < D ? e : 0)));
    return e < D ? x : make_uint4(0, 0, 0, 0);
  }
  uint32_t x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = row[e + i < D ? e + i : 0];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = e + i < D ? x[i] : 0;
  return make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
}

template <int DT, int NT, bool UNITS>
__global__ __launch_bounds__(kWaves * 64) void prompt_split_kernel(PromptArgs a, PromptPlan p) {
  static_assert(kWaves == 4);
  constexpr float shift = prob_shift<DT>;
  __shared__ float4 parts[2][kWaves][4][64];           // scores of a wave's elements
  __shared__ uint64_t values[kWaves][32];              // where a step's values begin
  __shared__ float biases[kWaves][32];
  __shared__ uint32_t again[kWaves];
  const fk_kv_cache_t& c = a.cache;
  const int lane = threadIdx.x & 63, n = lane & 31, h = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int D = (int)c.dim, e0 = w * NT * 32;          // the wave's first element

  const uint32_t order = div_by(blockIdx.x, p.by_heads), hk = blockIdx.x - order * p.heads;
  const Where at = a.B <= 64 ? count_tiles<32>(a, p.G, order) : search_tile<32>(a, p.G, order);
  if (at.b < 0) return;
  const int64_t cu0 = at.cu0, cu1 = at.cu1, len = at.len;
  const int rows = (int)min((cu1 - cu0) * p.G - (int64_t)at.tile * 32, (int64_t)32);
  const int64_t held = min(a.width * c.page, (int64_t)0x7FFFFFFF);
  const auto seen = [&](int r) {
    const int64_t t = div_by((uint32_t)(at.tile * 32 + r), p.by_G);
    return (int)max((int64_t)0, min(len - (cu1 - cu0) + t + 1, held));
  };
  const int most = __builtin_amdgcn_readfirstlane(seen(rows - 1)), steps = (int)(((uint32_t)most + 31) / 32);
  const uint32_t rr = at.tile * 32 + min(n, rows - 1);
  const int64_t tok = div_by(rr, p.by_G), t = cu0 + tok, qh = (int64_t)hk * p.G + (rr - tok * p.G);
  const bool put = n < rows && t >= 0 && t < a.T;
  const uint32_t limit = n < rows ? seen(n) : 0;

  const uint16_t* qp = (const uint16_t*)a.q + (put ? t * a.q_stride[0] + qh * a.q_stride[1] : 0);
  uint4 q[2 * NT];
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) {
    const uint4 x = put ? eight<UNITS>(qp, e0 + 16 * i + 8 * h, D) : make_uint4(0, 0, 0, 0);
    q[i] = x;
  }
  floatx16_t o[NT];
#pragma unroll
  for (int d = 0; d < NT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = -INFINITY, l = 0.f;
  const int32_t* table = a.table + at.b * a.ld_table;
  const uint16_t* const kb = (const uint16_t*)c.k + hk * c.k_stride[2];
  const uint16_t* const vb = (const uint16_t*)c.v + hk * c.v_stride[2];
  int buf = 0;
  for (int st = 0; st < steps; ++st) {
    // every wave finds the same keys: a step without any is left out by all
    const uint32_t key = (uint32_t)st * 32 + n, pos = min(key, (uint32_t)most - 1);
    const uint32_t pg_at = div_by(pos, p.page), tk = pos - pg_at * p.page.d;
    const int64_t page = table[pg_at];
    bool live = key == pos && page >= 0 && page < c.pages;
    float bias = 0.f;
    if (c.key_bias && live) {
      bias = c.key_bias[page * c.bias_stride[0] + tk * c.bias_stride[1] + hk * c.bias_stride[2]];
      live = bias != -INFINITY;
    }
    const uint32_t counts = (uint32_t)__ballot(live);
    if (counts == 0) continue;
    // (in the place of a key that is out another one is read, and not used)
    int64_t ko = page * c.k_stride[0] + tk * c.k_stride[1], vo = page * c.v_stride[0] + tk * c.v_stride[1];
    const int first = __builtin_ctz(counts);
    const int64_t k1 = __shfl(ko, first, 64), v1 = __shfl(vo, first, 64);
    ko = live ? ko : k1, vo = live ? vo : v1;
    if (lane < 32) values[w][n] = (uint64_t)(vb + vo), biases[w][n] = bias;
    floatx16_t s;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.f;
    uint4 kf[2 * NT];
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) kf[i] = eight<UNITS>(kb + ko, e0 + 16 * i + 8 * h, D);
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) s = Mfma<DT>::run(kf[i], q[i], s);
#pragma unroll
    for (int i = 0; i < 4; ++i) parts[buf][w][i][lane] = make_float4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
    __syncthreads();
    float x[16], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float4 y[kWaves];
#pragma unroll
      for (int k = 0; k < kWaves; ++k) y[k] = parts[buf][k][i][lane];
      x[4 * i] = (y[0].x + y[1].x) + (y[2].x + y[3].x);
      x[4 * i + 1] = (y[0].y + y[1].y) + (y[2].y + y[3].y);
      x[4 * i + 2] = (y[0].z + y[1].z) + (y[2].z + y[3].z);
      x[4 * i + 3] = (y[0].w + y[1].w) + (y[2].w + y[3].w);
    }
    buf ^= 1;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int kk = (i & 3) + 8 * (i >> 2) + 4 * h;
      x[i] *= a.scale;
      if (a.softcap > 0.f) x[i] = capped(x[i], a.softcap, 1.f / a.softcap);
      x[i] += biases[w][kk];
      x[i] = ((counts >> kk) & 1) && (uint32_t)st * 32 + kk < limit ? x[i] : -INFINITY;
      top = fmaxf(top, x[i]);
    }
    const float mn = fmaxf(m, max_halves(top));
    const float f = m == mn ? 1.f : fast_exp2((m - mn) * kLog2e);
    m = mn;
    uint4 pr[2];
    float sum = 0.f;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      uint32_t word[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        typedef typename Val<DT>::arith T;
        typedef T T2 __attribute__((ext_vector_type(2)));
        float y[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float z = x[8 * ks + 2 * i + j];
          y[j] = z == -INFINITY ? 0.f : fast_exp2(fmaf(z - mn, kLog2e, shift));       // NaN stays NaN
          sum += y[j];
        }
        const T2 two = {(T)y[0], (T)y[1]};
        word[i] = __builtin_bit_cast(uint32_t, two);
      }
      pr[ks] = make_uint4(word[0], word[1], word[2], word[3]);
    }
    l = fmaf(l, f, sum);
    if (__any(f != 1.f)) {
#pragma unroll
      for (int d = 0; d < NT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= f;
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const uint16_t* v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (const uint16_t*)values[w][16 * ks + (j & 3) + 8 * (j >> 2) + 4 * h];
      uint32_t y[NT][8];
#pragma unroll
      for (int d = 0; d < NT; ++d) {
        const int e = e0 + d * 32 + n;
#pragma unroll
        for (int j = 0; j < 8; ++j) y[d][j] = v[j][e < D ? e : 0];
      }
#pragma unroll
      for (int d = 0; d < NT; ++d) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          y[d][j] = (counts >> (16 * ks + (j & 3) + 8 * (j >> 2) + 4 * h)) & 1 ? y[d][j] : 0;
        o[d] = Mfma<DT>::run(make_uint4(y[d][0] | y[d][1] << 16, y[d][2] | y[d][3] << 16, y[d][4] | y[d][5] << 16,
                                        y[d][6] | y[d][7] << 16), pr[ks], o[d]);
      }
    }
  }
  l = sum_halves(l);
  // rows whose sums are not finite while their weights are: a value may be one that is hidden from
  // the row (0 times infinity), so they are done again, key by key
  bool bad = false;
#pragma unroll
  for (int d = 0; d < NT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      bad |= e0 + d * 32 + (i & 3) + 8 * (i >> 2) + 4 * h < D && !(fabsf(o[d][i]) < INFINITY);
  const uint64_t votes = __ballot(bad && put && l - l == 0.f);
  if (lane == 0) again[w] = (uint32_t)(votes | votes >> 32);
  __syncthreads();
  uint32_t todo = again[0] | again[1] | again[2] | again[3];
  const int64_t row = t * a.Hq + qh;
  if (put && !((todo >> n) & 1)) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int d = 0; d < NT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int e = e0 + d * 32 + (i & 3) + 8 * (i >> 2) + 4 * h;
        if (e < D) Val<DT>::put((typename Val<DT>::type*)a.out + row * D + e, o[d][i] * inv);
      }
    if (a.lse && w == 0 && h == 0) a.lse[row] = l == 0.f ? -INFINITY : m + (logf(l) - shift * kLn2);
  }
  for (; todo; todo &= todo - 1) {
    const int i = __builtin_ctz(todo);
    if ((i & 3) != w) continue;
    const int64_t t2 = __shfl(t, i, 64), h2 = __shfl(qh, i, 64);
    float m2, l2, o2[2 * NT];
    row_sums<DT, 2 * NT>(a, at.b, t2, h2, 0, (int64_t)(uint32_t)__shfl((int)limit, i, 64), m2, l2, o2);
    put_row<DT, 2 * NT>(a, t2 * a.Hq + h2, m2, l2, o2);
  }
}

template <int DT, int NT> hipError_t run_split_as(const PromptArgs& a, bool units, hipStream_t s) {
  PromptPlan p{};
  p.heads = (int)a.cache.heads;
  p.G = (int)(a.Hq / a.cache.heads);
  p.page = fast_div((uint32_t)a.cache.page);
  p.by_heads = fast_div((uint32_t)p.heads);
  p.by_G = fast_div((uint32_t)p.G);
  const int64_t blocks = tile_numbers(a, 32) * p.heads;
  if (blocks > most_blocks(kWaves) || a.T * p.G > 0x7FFFFFFF - 32) return hipErrorInvalidConfiguration;
  (units ? prompt_split_kernel<DT, NT, true> : prompt_split_kernel<DT, NT, false>)
      <<<(unsigned)blocks, kWaves * 64, 0, s>>>(a, p);
  return hipGetLastError();
}

template <int DT> hipError_t run_split(const PromptArgs& a, bool units, hipStream_t s) {
  const int64_t D = a.cache.dim;
  return D <= 128   ? run_split_as<DT, 1>(a, units, s)
         : D <= 256 ? run_split_as<DT, 2>(a, units, s)
         : D <= 512 ? run_split_as<DT, 4>(a, units, s)
                    : run_split_as<DT, 8>(a, units, s);
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
  const bool units = aligned16(a, Val<DT>::bytes);
  if (D > 256 || !units) {
    if constexpr (DT == FK_F32) return run_any<DT>(a, s);
    else return few_rows(a) ? run_any<DT>(a, s) : run_split<DT>(a, units, s);
  }
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

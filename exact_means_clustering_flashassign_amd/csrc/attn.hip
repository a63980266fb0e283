// Attention of one new token per request over a paged key-value cache.
//
// Online softmax: a running maximum m, the sum l of e^(s - m) and the sums
// o = sum e^(s - m) v; a new maximum scales l and o by e^(m_old - m_new), and two
// partial results join the same way.
#include "attn_parts.hpp"

namespace fk {
namespace {

// Any size, stride and alignment. One block per (request, query head, part of the
// request's keys); a wave takes every fourth key, a lane every 64th element of a row. With
// one part the result is final, else parts leave o (B,Hq,parts,D), ml (B,Hq,parts,2).
template <int DT, int EPL>
__global__ __launch_bounds__(kWaves * 64) void attn_any_kernel(AttnArgs a, int parts, float* po,
                                                               float* pml) {
  using E = typename Val<DT>::type;
  __shared__ float sm[kWaves], sl[kWaves], so[kWaves][EPL * 64];
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
  Runs<EPL> runs{so[w] + lane};
  int n = 0;
  for (int64_t j = len * part / parts + w; j < last; j += kWaves) {
    if (n++ == kKeyRun) runs.add(m, l, o), n = 1;
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
  runs.join(m, l, o);
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
hipError_t run_any(const AttnArgs& a, int64_t most, void* ws, hipStream_t s) {
  const int parts = most > 128 ? (int)any_parts(a.B, a.Hq) : 1;
  const int64_t heads = a.B * a.Hq, blocks = heads * parts;
  if (blocks > most_blocks(kWaves)) return hipErrorInvalidConfiguration;
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
                                       Acc<Shape<DT, DP>, HT>& acc) {
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

// Rows the matrix-core kernel can load: whole, aligned 16-byte units.
bool aligned16(const AttnArgs& a, int eb) {
  const fk_kv_cache_t& c = a.cache;
  const int64_t s[] = {a.q_stride[0], a.q_stride[1], c.k_stride[0], c.k_stride[1], c.k_stride[2],
                       c.v_stride[0], c.v_stride[1], c.v_stride[2], c.dim};
  for (int64_t v : s)
    if (v * eb % 16) return false;
  return !(((uintptr_t)a.q | (uintptr_t)c.k | (uintptr_t)c.v | (uintptr_t)a.out) & 15);
}

template <int DT_, int DP_, int HT_, bool EXTRA> struct Op {
  static constexpr int DT = DT_, DP = DP_, HT = HT_, PT = DT_;
  using Args = AttnArgs;
  using S = Shape<DT, DP>;
  using Rows = fk::Rows<DT, DP>;
  template <int KIND, class... A> __device__ static __forceinline__ void attend(A&&... args) {
    fk::attend<DT, DP, HT, EXTRA, KIND>(args...);
  }
};

template <int DT, int DP, int HT>
hipError_t run_mfma(const AttnArgs& a, void* ws, hipStream_t s) {
  const Choice c = choose(a, Shape<DT, DP>::keys, HT, DP, ws);
  if (c.blocks == 0) return hipErrorInvalidConfiguration;
  const auto aligned = [](uintptr_t base, const int64_t* s) {
    return !((base | (uintptr_t)((s[0] | s[1] | s[2]) * Val<DT>::bytes)) & 127);
  };
  // Caches that the 256 MB last-level cache may still hold from the step before are read
  // without the mark (4 requests of 512 keys: 10.4 us, marked 13.3).
  const double bytes = 2.0 * a.B * c.most * a.cache.heads * DP * Val<DT>::bytes;
  const bool full = a.cache.dim == DP, extra = a.softcap > 0.f || a.cache.key_bias;
  auto kernel = full ? (extra ? attn_mfma_kernel<Op<DT, DP, HT, true>, kWhole, kWaves>
                              : attn_mfma_kernel<Op<DT, DP, HT, false>, kWhole, kWaves>)
                     : (extra ? attn_mfma_kernel<Op<DT, DP, HT, true>, kNarrow, kWaves>
                              : attn_mfma_kernel<Op<DT, DP, HT, false>, kNarrow, kWaves>);
  if constexpr (DP * Val<DT>::bytes % 128 == 0) {
    if (full && bytes >= (double)(128 << 20) && c.p.tiles == 1 &&
        aligned((uintptr_t)a.cache.k, a.cache.k_stride) && aligned((uintptr_t)a.cache.v, a.cache.v_stride))
      kernel = extra ? attn_mfma_kernel<Op<DT, DP, HT, true>, kStream, kWaves>
                     : attn_mfma_kernel<Op<DT, DP, HT, false>, kStream, kWaves>;
  }
  if constexpr (DP <= 128) {
    if (c.eight)
      kernel = full ? (extra ? attn_mfma_kernel<Op<DT, DP, HT, true>, kWhole, 8>
                             : attn_mfma_kernel<Op<DT, DP, HT, false>, kWhole, 8>)
                    : (extra ? attn_mfma_kernel<Op<DT, DP, HT, true>, kNarrow, 8>
                             : attn_mfma_kernel<Op<DT, DP, HT, false>, kNarrow, 8>);
  }
  kernel<<<(unsigned)c.blocks, c.W * 64, 0, s>>>(a, c.p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !c.cut) return e;
  return join_parts<DT, DT>(a, c.p, s);
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

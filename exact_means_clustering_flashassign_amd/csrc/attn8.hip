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
hipError_t run_any(const AttnArgs8& a, int64_t most, void* ws, hipStream_t s) {
  const int parts = most > 128 ? (int)any_parts(a.B, a.Hq) : 1;
  const int64_t heads = a.B * a.Hq, blocks = heads * parts;
  if (blocks > most_blocks(kWaves)) return hipErrorInvalidConfiguration;
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

// ---------------------------------------------------------------------------
// Matrix-core kernel: rows of at most 256 codes in whole 16-byte units
// ---------------------------------------------------------------------------
// The layout of the 16-bit caches' kernel (attn.hip) over codes: lane 16 g + m, scores S^T = K
// Q^T with row = key and column = query head, values as O^T = V^T P^T with the
// probabilities in the lanes that made them. What differs:
//   * a step is 64 keys, so that as many bytes are on their way;
//   * a code becomes a 16-bit number where it is used, two at a time (every e4m3 number is one
//     of fp16 and of bf16). 16 bytes of a key are two products' worth: the queries' elements are
//     taken in the same order. Of values, bytes of two rows are laid in turn first,
//     so that a conversion makes the pair that a product wants;
//   * a key's scale goes to its score, a value's to its probability;
//   * probabilities times scales have no bound, so they and the values are bf16 whatever the
//     queries are, as the sum of two numbers, or three for fp32. fp32 queries are
//     the sum of three bf16 numbers (24 bits); products of those with codes are exact.
// Bound by bytes where requests are long: 2.28 GB of codes and scales (32 requests of up to 65536
// keys, 8 heads of 128) in 391 us, 5.8 TB/s; the conversions' vector instructions keep it from
// the 6.6 that rows of 192 and 256 reach. Short requests are bound by the launch and
// the chain of dependent loads (lengths, table, scales, codes): one of 2048 keys takes 17 us.
template <int DT, int DP_> struct Shape8 {
  static constexpr int DP = DP_, keys = 64, tiles = 4;      // keys per wave and step, 16-key tiles
  static constexpr int nc = DP / 64;                        // 16-byte key loads per row and lane
  static constexpr int ve = DP == 192 ? 4 : DP / 16;        // codes per value load
  static constexpr int nu = DP / (16 * ve);                 // value loads per row and lane
  static constexpr int rows = 16;                           // value rows per lane
  static constexpr int ldo = DP + 4;                        // LDS row of merged results
  static constexpr int least = DP <= 64 ? 0 : DP - 64;      // D is above it
  static constexpr int qn = DT == FK_F32 ? 3 : 1;           // 16-bit numbers of a query's element
  static constexpr int pn = DT == FK_F32 ? 3 : 2;           // and of a probability
  static constexpr int qt = DT == FK_F16 ? FK_F16 : FK_BF16;
  static constexpr int pt = DT == FK_F32 ? FK_F32 : FK_BF16;       // (no factor: the largest scales' products overflow)
};

// Row addresses and numbers of one step's keys, per wave and parity.
struct Rows8 {
  uint64_t k[64], v[64];
  float bias[64], ks[64], vs[64];
};

// Two neighbouring codes of a word as 16-bit numbers.
template <int QT, bool HI> __device__ __forceinline__ uint32_t widen(uint32_t w) {
  if constexpr (QT == FK_F16) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, HI));
  else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, HI));
}
template <int QT> __device__ __forceinline__ uint4 widen8(uint32_t a, uint32_t b) {
  return make_uint4(widen<QT, false>(a), widen<QT, true>(a), widen<QT, false>(b), widen<QT, true>(b));
}

// x as a sum of N bf16 numbers, each the rest's upper 16 bits but the last, which is rounded.
// (Of an infinity or NaN the first holds all and the rest is taken as 0.)
template <int N> __device__ __forceinline__ void split_bf16(const float (&x)[8], uint4 (&out)[N]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (k + 1 < N) {
        const uint32_t a = __builtin_bit_cast(uint32_t, r[2 * i]), b = __builtin_bit_cast(uint32_t, r[2 * i + 1]);
        w[i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
        r[2 * i] -= __builtin_bit_cast(float, a & 0xFFFF0000u);
        r[2 * i + 1] -= __builtin_bit_cast(float, b & 0xFFFF0000u);
      } else {
        typedef __bf16 T2 __attribute__((ext_vector_type(2)));
        const T2 d = {(__bf16)r[2 * i], (__bf16)r[2 * i + 1]};
        w[i] = __builtin_bit_cast(uint32_t, d);
      }
    }
    out[k] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// What a score takes part in: the scales alone; a bias and a cap of at most kNearCap (16-bit types); a bias
// and any cap.
enum { kPlainScore, kNearCapScore, kCapScore };

template <int DT, int DP, int HT, int SCORE, int KIND>
__device__ __forceinline__ void attend8(const AttnArgs8& a, const Plan& p, int64_t b, int hk, int ht, int len,
                                        int step, int stride, int end, Rows8* rows,
                                        Acc<Shape8<DT, DP>, HT>& acc) {
  using S = Shape8<DT, DP>;
  constexpr int QT = S::qt;
  constexpr bool EXTRA = SCORE != kPlainScore;
  const fk_kv_cache_t& c = a.cache;
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const int D = KIND == kNarrow ? (int)c.dim : DP;
#pragma unroll
  for (int h = 0; h < HT; ++h) {
    acc.m[h] = -INFINITY;
    acc.l[h] = 0.f;
#pragma unroll
    for (int i = 0; i < S::nu * S::ve; ++i) acc.o[h][i] = floatx4_t{0.f, 0.f, 0.f, 0.f};
  }
  if (step >= end) return;

  // Query fragments; heads past G and elements past D are zero, and elements past D of a
  // key are read from the zeros too (a code there may be NaN).
  uint4 q[HT][S::nc][2][S::qn];
  uint32_t koff[S::nc], voff[S::nu];
  const auto past = [&](int i) {            // unit i of this lane's part of a key is past D
    return (i + 1) * 64 > S::least && (i * 4 + g) * 16 >= D;
  };
#pragma unroll
  for (int i = 0; i < S::nc; ++i) koff[i] = past(i) ? 0 : (i * 4 + g) * 16;
#pragma unroll
  for (int h = 0; h < HT; ++h) {
    const int head = (ht * HT + h) * kHeadTile + m;
    const uint64_t qp = (uint64_t)a.q + (uint64_t)(b * a.q_stride[0] +
                        (int64_t)(hk * p.G + min(head, p.G - 1)) * a.q_stride[1]) * Val<DT>::bytes;
#pragma unroll
    for (int i = 0; i < S::nc; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint64_t at = qp + (koff[i] + e * 8) * Val<DT>::bytes;
        const bool none = past(i) || head >= p.G;
        if constexpr (DT == FK_F32) {
          const uint4 lo = load16(at), hi = load16(at + 16);
          const uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = none ? 0.f : __builtin_bit_cast(float, u[j]);
          split_bf16<3>(x, q[h][i][e]);
          // of an infinity or NaN the rest is not a number
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (x[j] - x[j] == 0.f) continue;
#pragma unroll
            for (int k = 1; k < 3; ++k) {
              uint32_t* w = &q[h][i][e][k].x + (j >> 1);
              *w &= j & 1 ? 0x0000FFFFu : 0xFFFF0000u;
            }
          }
        } else {
          q[h][i][e][0] = load16(at);
          if (none) q[h][i][e][0] = make_uint4(0, 0, 0, 0);
        }
      }
  }
#pragma unroll
  for (int i = 0; i < S::nu; ++i) {
    const int e = i * 16 * S::ve + m * S::ve;
    voff[i] = e < D ? e : 0;
  }

  // Lane i looks after key i of a step: table entry two steps ahead, bias and scales
  // one step ahead, addresses to LDS just before the step's loads.
  const uint64_t table = (uint64_t)(a.table + b * a.ld_table);
  const uint64_t kbase = (uint64_t)c.k + (uint64_t)hk * c.k_stride[2];
  const uint64_t vbase = (uint64_t)c.v + (uint64_t)hk * c.v_stride[2];
  const uint64_t zero = (uint64_t)zero_row;
  const bool cap = EXTRA && a.softcap > 0.f;
  const float inv_cap = cap ? 1.f / a.softcap : 0.f;
  const bool has_bias = EXTRA && c.key_bias && c.pages > 0;
  const uint64_t bbase = (uint64_t)c.key_bias + (uint64_t)hk * c.bias_stride[2] * 4;
  const uint64_t ksbase = (uint64_t)a.k_scale + (uint64_t)hk * a.ks_stride[2] * 4;
  const uint64_t vsbase = (uint64_t)a.v_scale + (uint64_t)hk * a.vs_stride[2] * 4;
  struct Numbers { float bias, ks, vs; };
  auto entry = [&](int st) -> int32_t {             // page of key `lane` of step st, -1: none
    const uint32_t key = (uint32_t)st * S::keys + lane;
    const uint32_t at = min(key, (uint32_t)len - 1);
    const int32_t pg = *(gptr_i32)(table + 4 * (uint64_t)div_by(at, p.page));
    return st < end && key == at ? pg : -1;
  };
  auto numbers = [&](int st, int32_t pg) -> Numbers {
    const bool live = (uint32_t)pg < (uint32_t)c.pages;
    Numbers x = {-INFINITY, 0.f, 0.f};
    if (c.pages > 0) {
      // (the last one's place for a key past the end: one past 2^31 would not divide)
      const uint32_t key = min((uint32_t)st * S::keys + lane, (uint32_t)len - 1);
      const uint32_t tok = key - div_by(key, p.page) * p.page.d;
      const int64_t at = live ? pg : 0;
      x.ks = *(gptr_f32)(ksbase + (uint64_t)(at * a.ks_stride[0] + tok * a.ks_stride[1]) * 4);
      x.vs = *(gptr_f32)(vsbase + (uint64_t)(at * a.vs_stride[0] + tok * a.vs_stride[1]) * 4);
      x.bias = has_bias ? *(gptr_f32)(bbase + (uint64_t)(at * c.bias_stride[0] + tok * c.bias_stride[1]) * 4) : 0.f;
    }
    if (!live || x.bias == -INFINITY) x = {-INFINITY, 0.f, 0.f};
    return x;
  };
  auto put_rows = [&](Rows8& r, int st, int32_t pg, const Numbers& x) {
    const uint32_t key = (uint32_t)st * S::keys + lane;
    const uint32_t tok = key - div_by(key, p.page) * p.page.d;
    const bool live = x.bias != -INFINITY;
    const uint64_t ka = kbase + (uint64_t)(pg * c.k_stride[0] + tok * c.k_stride[1]);
    const uint64_t va = vbase + (uint64_t)(pg * c.v_stride[0] + tok * c.v_stride[1]);
    // other lanes of the wave read these: keep the compiler's order
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    r.k[lane] = live ? ka : zero;
    r.v[lane] = live ? va : zero;
    r.bias[lane] = x.bias;
    r.ks[lane] = x.ks;
    r.vs[lane] = x.vs;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };
  uint4 kf[S::tiles][S::nc];
  auto load_k = [&](const Rows8& r, int s) {
    const uint64_t ad = r.k[16 * s + m];
#pragma unroll
    for (int i = 0; i < S::nc; ++i) kf[s][i] = load_row<16, KIND == kStream>((past(i) ? zero : ad) + koff[i]);
  };
  uint4 vf[S::rows][S::nu];            // a load of fewer bytes fills the first words
  auto load_v = [&](const Rows8& r, int y) {             // of tiles 2 y and 2 y + 1
#pragma unroll
    for (int j = 8 * y; j < 8 * y + 8; ++j) {
      const uint64_t ad = r.v[16 * (j >> 2) + 4 * g + (j & 3)];
#pragma unroll
      for (int i = 0; i < S::nu; ++i) vf[j][i] = load_row<S::ve, KIND == kStream>(ad + voff[i]);
    }
  };

  int32_t pg1 = entry(step), pg2 = entry(step + stride);
  put_rows(rows[0], step, pg1, numbers(step, pg1));
  Numbers x1 = numbers(step + stride, pg2);
  pg1 = pg2;
  pg2 = entry(step + 2 * stride);
#pragma unroll
  for (int u = 0; u < S::tiles; ++u) load_k(rows[0], u);
#pragma unroll
  for (int y = 0; y < S::tiles / 2; ++y) load_v(rows[0], y);
  int par = 0;
  for (; step < end; step += stride, par ^= 1) {
    Rows8& now = rows[par];
    Rows8& next = rows[par ^ 1];
    put_rows(next, step + stride, pg1, x1);
    float s[HT][S::tiles][4];
#pragma unroll
    for (int u = 0; u < S::tiles; ++u) {
      floatx4_t x[HT];
#pragma unroll
      for (int h = 0; h < HT; ++h) x[h] = floatx4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < S::nc; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint4 k8 = widen8<QT>(word(kf[u][i], 2 * e), word(kf[u][i], 2 * e + 1));
#pragma unroll
          for (int h = 0; h < HT; ++h)
#pragma unroll
            for (int k = 0; k < S::qn; ++k) x[h] = Mfma16<QT>::run(k8, q[h][i][e][k], x[h]);
        }
#pragma unroll
      for (int h = 0; h < HT; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[h][u][i] = x[h][i];
      load_k(next, u);                   // the next keys are asked for as soon as these are out of
      __builtin_amdgcn_sched_barrier(0); // their registers
    }
    x1 = numbers(step + 2 * stride, pg2);
    pg1 = pg2;
    pg2 = entry(step + 3 * stride);

    uint4 ph[S::tiles / 2][HT][S::pn];
#pragma unroll
    for (int h = 0; h < HT; ++h) {
      float top = acc.m[h];
#pragma unroll
      for (int u = 0; u < S::tiles; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // -inf where a key does not count
          const int at = 16 * u + 4 * g + i;
          const float bias = now.bias[at];
          // (one after the other: the product of both scales may overflow where the score is 0)
          float x = s[h][u][i] * now.ks[at] * a.scale;
          if (cap) x = SCORE == kNearCapScore ? cap_16bit(x, a.softcap, inv_cap) : capped(x, a.softcap, inv_cap);
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
          const float x = prob<S::pt>(s[h][u][i] - ref);
          part += x;
          s[h][u][i] = x * now.vs[16 * u + 4 * g + i];
        }
      acc.l[h] = fmaf(acc.l[h], alpha, part);
#pragma unroll
      for (int i = 0; i < S::nu * S::ve; ++i) acc.o[h][i] *= alpha;
#pragma unroll
      for (int y = 0; y < S::tiles / 2; ++y) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = s[h][2 * y + (j >> 2)][j & 3];
        split_bf16<S::pn>(x, ph[y][h]);
      }
    }
#pragma unroll
    for (int y = 0; y < S::tiles / 2; ++y) {
#pragma unroll
      for (int u = 0; u < S::nu; ++u)
#pragma unroll
        for (int t4 = 0; t4 < S::ve; t4 += 2) {
          // codes t4 and t4 + 1 of rows j and j + 1, in turn
          uint32_t two[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            two[j] = __builtin_amdgcn_perm(word(vf[8 * y + 2 * j + 1][u], t4 >> 2), word(vf[8 * y + 2 * j][u], t4 >> 2),
                                           t4 & 2 ? 0x07030602u : 0x05010400u);
#pragma unroll
          for (int t = t4; t < t4 + 2; ++t) {
            const uint4 vt = t & 1 ? make_uint4(widen<FK_BF16, true>(two[0]), widen<FK_BF16, true>(two[1]),
                                                widen<FK_BF16, true>(two[2]), widen<FK_BF16, true>(two[3]))
                                   : make_uint4(widen<FK_BF16, false>(two[0]), widen<FK_BF16, false>(two[1]),
                                                widen<FK_BF16, false>(two[2]), widen<FK_BF16, false>(two[3]));
#pragma unroll
            for (int h = 0; h < HT; ++h) {
              floatx4_t& o = acc.o[h][u * S::ve + t];
#pragma unroll
              for (int k = 0; k < S::pn; ++k) o = Mfma16<FK_BF16>::run(vt, ph[y][h][k], o);
            }
          }
        }
      load_v(next, y);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int h = 0; h < HT; ++h) {
    acc.l[h] += __shfl_xor(acc.l[h], 16, 64);
    acc.l[h] += __shfl_xor(acc.l[h], 32, 64);
  }
}

template <int DT_, int DP_, int HT_, int SCORE> struct Op8 {
  static constexpr int DT = DT_, DP = DP_, HT = HT_;
  using Args = AttnArgs8;
  using S = Shape8<DT, DP>;
  static constexpr int PT = S::pt;
  using Rows = Rows8;
  template <int KIND, class... A> __device__ static __forceinline__ void attend(A&&... args) {
    attend8<DT, DP, HT, SCORE, KIND>(args...);
  }
};

// Rows the matrix-core kernel can load: whole, aligned 16-byte units.
bool aligned16(const AttnArgs8& a, int eb) {
  const fk_kv_cache_t& c = a.cache;
  const int64_t s[] = {a.q_stride[0] * eb, a.q_stride[1] * eb, c.k_stride[0], c.k_stride[1], c.k_stride[2],
                       c.v_stride[0], c.v_stride[1], c.v_stride[2], c.dim};
  for (int64_t v : s)
    if (v % 16) return false;
  return !(((uintptr_t)a.q | (uintptr_t)c.k | (uintptr_t)c.v | (uintptr_t)a.out) & 15);
}

template <int DT, int DP, int HT>
hipError_t run_mfma(const AttnArgs8& a, void* ws, hipStream_t s) {
  const Choice c = choose(a, Shape8<DT, DP>::keys, HT, DP, ws);
  if (c.blocks == 0) return hipErrorInvalidConfiguration;
  const auto aligned = [](uintptr_t base, const int64_t* s) { return !((base | (uintptr_t)(s[0] | s[1] | s[2])) & 127); };
  // Caches that the 256 MB last-level cache may still hold from the step before are read
  // without the mark.
  const double bytes = 2.0 * a.B * c.most * a.cache.heads * DP;
  const bool full = a.cache.dim == DP;
  const bool stream = DP % 128 == 0 && full && bytes >= (double)(128 << 20) && c.p.tiles == 1 &&
                      aligned((uintptr_t)a.cache.k, a.cache.k_stride) && aligned((uintptr_t)a.cache.v, a.cache.v_stride);
  const auto choose_kernel = [&](auto op) {
    using Op = decltype(op);
    auto kernel = full ? attn_mfma_kernel<Op, kWhole, kWaves> : attn_mfma_kernel<Op, kNarrow, kWaves>;
    if constexpr (DP % 128 == 0)
      if (stream) kernel = attn_mfma_kernel<Op, kStream, kWaves>;
    if constexpr (DP <= 128)
      if (c.eight) kernel = full ? attn_mfma_kernel<Op, kWhole, 8> : attn_mfma_kernel<Op, kNarrow, 8>;
    return kernel;
  };
  auto kernel = a.softcap > 0.f || a.cache.key_bias ? choose_kernel(Op8<DT, DP, HT, kCapScore>())
                                                    : choose_kernel(Op8<DT, DP, HT, kPlainScore>());
  if constexpr (DT != FK_F32)
    if ((a.softcap > 0.f || a.cache.key_bias) && a.softcap <= kNearCap) kernel = choose_kernel(Op8<DT, DP, HT, kNearCapScore>());
  kernel<<<(unsigned)c.blocks, c.W * 64, 0, s>>>(a, c.p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !c.cut) return e;
  return join_parts<DT, Shape8<DT, DP>::pt>(a, c.p, s);
}

template <int DT> hipError_t run(const AttnArgs8& a, void* ws, hipStream_t s) {
  const int64_t D = a.cache.dim;
  if (D > 256 || !aligned16(a, Val<DT>::bytes)) return run_any<DT>(a, longest(a), ws, s);
  if constexpr (DT != FK_F32) {
    if (tile_width(DT, D, a.Hq / a.cache.heads) > kHeadTile)
      return D <= 64 ? run_mfma<DT, 64, 2>(a, ws, s) : run_mfma<DT, 128, 2>(a, ws, s);
  }
  return D <= 64    ? run_mfma<DT, 64, 1>(a, ws, s)
         : D <= 128 ? run_mfma<DT, 128, 1>(a, ws, s)
         : D <= 192 ? run_mfma<DT, 192, 1>(a, ws, s)
                    : run_mfma<DT, 256, 1>(a, ws, s);
}

}  // namespace

size_t attn8_ws_bytes(int dt, int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  return attn_ws_bytes(dt, B, Hq, Hkv, D > 32 ? D : 33);       // (tiles of 64 codes at least)
}

hipError_t launch_paged_attn8(const AttnArgs8& a, int dt, void* ws, hipStream_t s) {
  return dt == FK_F32   ? run<FK_F32>(a, ws, s)
         : dt == FK_F16 ? run<FK_F16>(a, ws, s)
                        : run<FK_BF16>(a, ws, s);
}

}  // namespace fk

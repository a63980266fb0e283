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

// ---------------------------------------------------------------------------
// Rows in whole VE-element units (16 or 8 bytes)
// ---------------------------------------------------------------------------
// Memory-bound: each element is read and written once. A lane holds two units of
// a row, for pairs (i, i + rot/2) the two halves of VE pairs, so a pair is never
// split between lanes; L lanes make a row and the wave takes 64 / L rows a pass.
// A wave stays with one token: its cosines, sines and both weights are loaded
// once and serve all rows it takes. Measured: 75600 tokens of 32 + 8 + 8 heads of 128 fp16
// into a cache, 1.9 GB, 355 us or 5.3 TB/s (a large copy: 4.8); 32 tokens 4.5 us.
// A register cap for more waves a CU spills and costs half (355 -> 539 us).
struct RopePlan {
  int units, hp, rem;        // units a row; pairs of units that rotate; others, two by two
  int L, rp;                 // lanes a row (a power of two), rows a pass
  int rows, passes;          // rows a token, passes a token
  int ppw, wpt;              // passes a wave, waves a token
  FastDiv page, per, by_wpt; // tokens a page, rows a token, waves a token
};

enum { kApart, kSideBySide, kExchange };

template <int DT, int VE> struct Unit {
  typedef typename Val<DT>::arith T;
  typedef T vec __attribute__((ext_vector_type(VE)));
};

// MODE: pairs are half the rotated part apart and that half is whole units, so that one
// lane holds both of a pair; or pairs lie side by side; or neither, and the rotated
// elements of a row are exchanged through LDS.
// FLAT: rows of all tokens end to end, each lane with its own token. Takes the
// tokens whose rows would leave lanes of their own wave idle.
template <int DT, int VE, int MODE, bool FLAT>
__global__ __launch_bounds__(kWaves * 64) void rope_vec_kernel(RopeArgs a, RopePlan p,
                                                               int64_t waves) {
  typedef typename Unit<DT, VE>::T T;
  typedef typename Unit<DT, VE>::vec V;
  __shared__ float xch[MODE == kExchange ? kWaves : 1][MODE == kExchange ? 64 * 2 * VE : 1];
  const int lane = threadIdx.x & 63;
  const int64_t wave =
      (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave >= waves) return;

  // this lane's units of every row it meets
  const int j = lane & (p.L - 1), sub = lane / p.L;
  const bool turn = j < p.hp;
  const int ua = turn ? j : j + p.hp;
  const int ub = turn ? j + p.hp : ua + p.rem;
  const bool va = j < p.hp + p.rem, vb = va && ub < p.units;
  const int ea = va ? ua * VE : 0, eb = vb ? ub * VE : 0;

  // its token, and the passes over the token's rows
  int64_t t;
  int pass0 = 0, pass1 = 1, row0 = sub;
  bool live = va;
  if constexpr (FLAT) {
    const uint32_t row = (uint32_t)wave * p.rp + sub;     // T * rows < 2^31
    live = va && row < (uint32_t)a.T * p.rows;
    t = live ? div_by(row, p.per) : 0;
    row0 = live ? row - (uint32_t)t * p.rows : 0;
  } else {
    t = div_by((uint32_t)wave, p.by_wpt);
    pass0 = (int)(wave - t * p.wpt) * p.ppw;
    pass1 = min(pass0 + p.ppw, p.passes);
  }

  struct Row {
    V a, b;
    int kind, h;             // 0 query, 1 key, 2 value, 3 none
  };
  auto load = [&](int pass) {
    Row x;
    const int r = pass * p.rp + row0;
    x.kind = r < a.Hq ? 0 : (r < a.Hq + a.Hkv ? 1 : 2);
    x.h = r - (x.kind == 0 ? 0 : (x.kind == 1 ? (int)a.Hq : (int)(a.Hq + a.Hkv)));
    if (pass >= pass1 || r >= p.rows || !live) x.kind = 3;
    x.a = V{}, x.b = V{};
    if (x.kind == 3) return x;
    const T* src = x.kind == 0   ? (const T*)a.q + t * a.q_stride[0] + x.h * a.q_stride[1]
                   : x.kind == 1 ? (const T*)a.k + t * a.k_stride[0] + x.h * a.k_stride[1]
                                 : (const T*)a.v + t * a.v_stride[0] + x.h * a.v_stride[1];
    x.a = *(const V*)(src + ea);
    if (vb) x.b = *(const V*)(src + eb);
    return x;
  };
  Row next = load(pass0);      // on its way before anything is waited for

  // element i of a then b rotates with its own cosine and sine (kExchange), else pair i
  const int half = (int)(a.rot >> 1);
  constexpr int turns = MODE == kExchange ? 2 * VE : VE;
  float cs[turns] = {}, sn[turns] = {};
  bool on[turns];
#pragma unroll
  for (int i = 0; i < turns; ++i) on[i] = MODE == kApart && turn;
  if (half) {
    const int64_t pos = clamp_pos(a.positions[t], a.max_pos);
    const float* row = a.rope + pos * a.rot;
    if constexpr (MODE == kSideBySide) {
#pragma unroll
      for (int i = 0; i < VE; ++i) {         // first the pairs of unit a, then those of b
        const int pr = (i < VE / 2 ? ea / 2 + i : eb / 2 + i - VE / 2);
        on[i] = (i < VE / 2 ? va : vb) && pr < half;
        if (on[i]) cs[i] = row[pr], sn[i] = row[half + pr];
      }
    } else if constexpr (MODE == kExchange) {
#pragma unroll
      for (int i = 0; i < 2 * VE; ++i) {
        const int el = i < VE ? ea + i : eb + i - VE, pr = el < half ? el : el - half;
        on[i] = (i < VE ? va : vb) && el < 2 * half;
        if (on[i]) cs[i] = row[pr], sn[i] = el < half ? -row[half + pr] : row[half + pr];
      }
    } else if (turn) {
#pragma unroll
      for (int i = 0; i < VE; ++i) cs[i] = row[ea + i], sn[i] = row[half + ea + i];
    }
  }
  const bool norm = a.q_weight != nullptr;
  V wqa = {}, wqb = {}, wka = {}, wkb = {};
  if (norm) {
    const T *wq = (const T*)a.q_weight, *wk = (const T*)a.k_weight;
    wqa = *(const V*)(wq + ea), wqb = *(const V*)(wq + eb);
    wka = *(const V*)(wk + ea), wkb = *(const V*)(wk + eb);
  }
  bool slot_ok = false;
  int64_t kslot = 0, vslot = 0, bslot = 0;
  if (a.cache.k) {
    const int32_t slot = FLAT ? a.slots[t] : __builtin_amdgcn_readfirstlane(a.slots[t]);
    slot_ok = slot >= 0 && slot < a.cache.pages * a.cache.page;
    if (slot_ok) {
      const int64_t page = div_by(slot, p.page), tok = slot - page * p.page.d;
      kslot = page * a.cache.k_stride[0] + tok * a.cache.k_stride[1];
      vslot = page * a.cache.v_stride[0] + tok * a.cache.v_stride[1];
      bslot = page * a.cache.bias_stride[0] + tok * a.cache.bias_stride[1];
    }
  }

  for (int pass = pass0; pass < pass1; ++pass) {
    const Row x = next;
    next = load(pass + 1);
    float fa[VE], fb[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) fa[i] = (float)x.a[i], fb[i] = (float)x.b[i];
    if (norm) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < VE; ++i) ss = fmaf(fa[i], fa[i], fmaf(fb[i], fb[i], ss));
      for (int off = p.L >> 1; off >= 1; off >>= 1) ss += __shfl_xor(ss, off, 64);
      const float r = 1.f / sqrtf(ss / (float)a.D + a.eps);
      const V wa = x.kind == 0 ? wqa : wka, wb = x.kind == 0 ? wqb : wkb;
#pragma unroll
      for (int i = 0; i < VE; ++i) fa[i] = fa[i] * r * (float)wa[i], fb[i] = fb[i] * r * (float)wb[i];
    }
    if constexpr (MODE == kExchange) {
      float* mine = xch[threadIdx.x >> 6] + sub * 2 * VE * p.L;
      // (only this wave's lanes read it: the compiler's order is enough)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int i = 0; i < 2 * VE; ++i)
        if (on[i]) mine[i < VE ? ea + i : eb + i - VE] = i < VE ? fa[i] : fb[i - VE];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int i = 0; i < 2 * VE; ++i) {
        const int el = i < VE ? ea + i : eb + i - VE;
        float& f = i < VE ? fa[i] : fb[i - VE];
        if (on[i]) f = f * cs[i] + mine[el < half ? el + half : el - half] * sn[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        // pair i: elements 2i, 2i+1 of a then b, or element i of both
        float* e0 = MODE == kApart ? &fa[i] : (i < VE / 2 ? &fa[2 * i] : &fb[2 * i - VE]);
        float* e1 = MODE == kApart ? &fb[i] : e0 + 1;
        const float u = *e0, w = *e1;
        *e0 = on[i] ? u * cs[i] - w * sn[i] : u;
        *e1 = on[i] ? w * cs[i] + u * sn[i] : w;
      }
    }
    if (x.kind == 3) continue;
    V ya, yb;
#pragma unroll
    for (int i = 0; i < VE; ++i) ya[i] = (T)fa[i], yb[i] = (T)fb[i];
    T *y0 = nullptr, *y1 = nullptr;
    if (x.kind == 0) {
      y0 = (T*)a.q_out + (t * a.Hq + x.h) * a.D;
    } else if (x.kind == 1) {
      if (a.k_out) y0 = (T*)a.k_out + (t * a.Hkv + x.h) * a.D;
      if (slot_ok) y1 = (T*)a.cache.k + kslot + x.h * a.cache.k_stride[2];
      if (slot_ok && a.cache.key_bias && j == 0)
        a.cache.key_bias[bslot + x.h * a.cache.bias_stride[2]] = 0.f;
    } else {
      ya = x.a, yb = x.b;                    // values as they are
      if (slot_ok) y1 = (T*)a.cache.v + vslot + x.h * a.cache.v_stride[2];
    }
    if (y0) {
      *(V*)(y0 + ea) = ya;
      if (vb) *(V*)(y0 + eb) = yb;
    }
    if (y1) {
      *(V*)(y1 + ea) = ya;
      if (vb) *(V*)(y1 + eb) = yb;
    }
  }
}

// Whether every row starts at a multiple of `bytes` and holds whole units of it.
bool in_units(const RopeArgs& a, int eb, int bytes) {
  const fk_kv_cache_t& c = a.cache;
  int64_t s = a.D | a.q_stride[0] | a.q_stride[1] | a.k_stride[0] | a.k_stride[1];
  uintptr_t p = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.q_out | (uintptr_t)a.k_out |
                (uintptr_t)a.q_weight | (uintptr_t)a.k_weight;
  if (c.k) {
    s |= a.v_stride[0] | a.v_stride[1];
    for (int i = 0; i < 3; ++i) s |= c.k_stride[i] | c.v_stride[i];
    p |= (uintptr_t)a.v | (uintptr_t)c.k | (uintptr_t)c.v;
  }
  return s * eb % bytes == 0 && p % bytes == 0;     // powers of two: a bit below shows in the or
}

template <int DT, int VE, int MODE>
hipError_t run_mode(const RopeArgs& a, hipStream_t s) {
  RopePlan p{};
  p.units = (int)(a.D / VE);
  p.hp = MODE == kApart ? (int)(a.rot / 2 / VE) : 0;
  p.rem = (p.units - 2 * p.hp + 1) / 2;
  p.L = 1;
  while (p.L < p.hp + p.rem) p.L *= 2;
  p.rp = 64 / p.L;
  const int64_t rows = a.Hq + a.Hkv * (a.cache.k ? 2 : 1);
  if (rows > 1 << 30) return hipErrorInvalidConfiguration;
  p.rows = (int)rows;
  p.passes = (p.rows + p.rp - 1) / p.rp;
  // A wave takes several passes once there are waves enough for every CU's slots.
  const int64_t all = a.T * p.passes;
  const int64_t want = device_cus() > 0 ? (int64_t)device_cus() * 32 : 1;
  p.ppw = (int)(all / want < 1 ? 1 : (all / want < p.passes ? all / want : p.passes));
  p.wpt = (p.passes + p.ppw - 1) / p.ppw;
  p.page = fast_div(a.cache.k ? (uint32_t)a.cache.page : 1);
  p.per = fast_div((uint32_t)p.rows);
  p.by_wpt = fast_div((uint32_t)p.wpt);
  // Tokens of one pass, or that leave a quarter of their passes' lanes idle, go end to
  // end (60000 tokens of 3 rows: 51 -> 26 us; of 10 rows in two passes: 47 -> 41); with more
  // rows the wave that stays with its token is faster (48 rows: 356 us, end to end 406).
  const bool flat = (p.passes == 1 || 4 * p.rows < 3 * p.passes * p.rp) &&
                    a.T * p.rows < 0x7FFFFFFF - 64;
  const int64_t waves = flat ? (a.T * p.rows + p.rp - 1) / p.rp : a.T * p.wpt;
  const int64_t blocks = (waves + kWaves - 1) / kWaves;
  if (waves > 0x7FFFFFFF - kWaves) return hipErrorInvalidConfiguration;
  const auto kernel =
      flat ? rope_vec_kernel<DT, VE, MODE, true> : rope_vec_kernel<DT, VE, MODE, false>;
  kernel<<<(unsigned)blocks, kWaves * 64, 0, s>>>(a, p, waves);
  return hipGetLastError();
}

template <int DT, int VE>
hipError_t run_vec(const RopeArgs& a, hipStream_t s) {
  if (a.interleaved) return run_mode<DT, VE, kSideBySide>(a, s);
  return a.rot / 2 % VE ? run_mode<DT, VE, kExchange>(a, s) : run_mode<DT, VE, kApart>(a, s);
}

}  // namespace

hipError_t launch_qk_norm_rope(const RopeArgs& a, int dt, hipStream_t s) {
  const int64_t rows = a.T * (a.Hq + a.Hkv * (a.cache.k ? 2 : 1));
  if (rows == 0) return hipSuccess;
  // 64 lanes of two units are the longest row
  if (dt == FK_F32) {
    if (a.D <= 512 && in_units(a, 4, 16)) return run_vec<FK_F32, 4>(a, s);
  } else {
    const bool f16 = dt == FK_F16;
    // A half of whole 8-byte units takes those rather than an exchange (20000 tokens of 24
    // heads of 128, 72 rotated: 61 us, exchanged 93; with a half of 6 the exchange is left, 74).
    const bool narrow = !a.interleaved && a.rot / 2 % 8 == 4 && a.D <= 512;
    if (a.D <= 1024 && !narrow && in_units(a, 2, 16))
      return f16 ? run_vec<FK_F16, 8>(a, s) : run_vec<FK_BF16, 8>(a, s);
    if (a.D <= 512 && in_units(a, 2, 8))
      return f16 ? run_vec<FK_F16, 4>(a, s) : run_vec<FK_BF16, 4>(a, s);
  }
  const int64_t blocks = (rows + kWaves - 1) / kWaves;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const auto kernel = dt == FK_F32   ? rope_any_kernel<FK_F32>
                      : dt == FK_F16 ? rope_any_kernel<FK_F16>
                                     : rope_any_kernel<FK_BF16>;
  kernel<<<(unsigned)blocks, kWaves * 64, 0, s>>>(a, rows);
  return hipGetLastError();
}

}  // namespace fk

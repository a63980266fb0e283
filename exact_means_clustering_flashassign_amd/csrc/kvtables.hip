// Block tables, token slots and positions from request lengths (integers only).
//
// Two running sums over the requests carry everything: new tokens (which
// request a token of the step belongs to) and pages taken from the free list
// (which free page an entry gets). With them every table entry and every token is
// independent. Up to kOwnScan requests, every block forms both sums for itself
// in LDS (8 bytes a request from L2) and one launch does it all: the call is a
// few microseconds of latency, and a second launch would add as much again.
// Beyond that one block writes the sums first and the others read them. Measured: 32
// requests with one new token and 4726 entries each 4.4 us, 1024 requests with 0.84 million
// new tokens 11 us in one launch (13.8 in two), 3723 requests in two 10.6 us.
#include "fk_kv.hpp"

namespace fk {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kOwnScan = 2048;
constexpr int kRun = 256, kTokens = 64;       // entries and tokens a wave takes at a time

struct Geometry {
  FastDiv page, by_row;
  int32_t cap;            // tokens that a row of pages holds, at most 2^31 - 1
  int64_t row_items, items;
  int32_t token_items;
};

struct Need {
  int32_t old, fresh;     // tokens held and new
  int32_t held, need;     // pages of the old tokens and of all, at most a row
};

__device__ __forceinline__ int32_t to_i32(int64_t v) {
  return (int32_t)(v < 0x7FFFFFFF ? v : 0x7FFFFFFF);
}
__device__ __forceinline__ int32_t pages_of(int32_t tokens, const Geometry& g) {
  const int32_t n = min(tokens, g.cap);
  return n > 0 ? (int32_t)div_by(n - 1, g.page) + 1 : 0;
}
__device__ __forceinline__ Need need_of(const TablesArgs& a, const Geometry& g, int64_t b) {
  Need n;
  n.old = max(a.len_old[b], 0);
  n.fresh = max(a.len_new[b], 0);
  n.held = pages_of(n.old, g);
  n.need = pages_of(to_i32((int64_t)n.old + n.fresh), g);
  return n;
}

// Running sums of up to `room` requests from b0 on, on top of `base`, in LDS:
// cu_t[i], cu_p[i] = sums before request b0 + i. 32-bit sums that stay at 2^32 - 1 once they
// get there (such an addition is associative) and are stored as at most 2^31 - 1.
struct Sums {
  uint32_t t, p;
};
__device__ __forceinline__ Sums operator+(Sums a, Sums b) {
  return Sums{__builtin_elementwise_add_sat(a.t, b.t), __builtin_elementwise_add_sat(a.p, b.p)};
}
__device__ __forceinline__ int32_t stored(uint32_t v) { return (int32_t)min(v, 0x7FFFFFFFu); }

__device__ __forceinline__ Sums wave_scan(Sums v) {       // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const Sums u{__shfl_up(v.t, off, 64), __shfl_up(v.p, off, 64)};
    if (lane >= off) v = v + u;
  }
  return v;
}
// kN threads, of which thread i sums requests b0 + i n .. b0 + (i + 1) n - 1.
template <int kN>
__device__ __forceinline__ Sums scan_requests(const TablesArgs& a, const Geometry& g, int64_t b0,
                                              Sums base, int room, int32_t* cu_t, int32_t* cu_p) {
  __shared__ Sums tot[kN / 64];
  const int count = (int)min((int64_t)room, a.B - b0);
#pragma unroll 4
  for (int i = threadIdx.x; i < count; i += kN) {
    const Need r = need_of(a, g, b0 + i);
    cu_t[i] = r.fresh, cu_p[i] = r.need - r.held;
  }
  __syncthreads();
  const int n = (count + kN - 1) / kN, first = min((int)threadIdx.x * n, count);
  const int past = min(first + n, count);
  Sums mine{0, 0};
  for (int i = first; i < past; ++i) mine = mine + Sums{(uint32_t)cu_t[i], (uint32_t)cu_p[i]};
  const Sums incl = wave_scan(mine);
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (lane == 63) tot[w] = incl;
  Sums before{__shfl_up(incl.t, 1, 64), __shfl_up(incl.p, 1, 64)};
  if (lane == 0) before = Sums{0, 0};
  __syncthreads();
  Sums at = base, end = base;
#pragma unroll
  for (int i = 0; i < kN / 64; ++i) {
    if (i < w) at = at + tot[i];
    end = end + tot[i];
  }
  at = at + before;
  for (int i = first; i < past; ++i) {
    const Sums own{(uint32_t)cu_t[i], (uint32_t)cu_p[i]};
    cu_t[i] = stored(at.t), cu_p[i] = stored(at.p);
    at = at + own;
  }
  __syncthreads();
  return end;
}

// The last request whose sum before it is <= t, found by the whole wave: 64 probes at a
// time, so that 4096 requests take two dependent reads.
__device__ __forceinline__ int64_t request_of(const int32_t* cu, int64_t B, int64_t t) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, hi = B;                       // cu[lo] <= t, and cu[hi] > t or hi == B
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 63) / 64, at = lo + (lane + 1) * step;
    const int below = __popcll(__ballot(at < hi && cu[at] <= t));
    lo += below * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The same for each lane's own t, where request b is lane 0's and t does not fall from
// lane to lane: among the next 64 requests by their sums in registers, else by halving.
__device__ __forceinline__ int64_t lane_request_of(const int32_t* cu, int64_t B, int64_t b,
                                                   int64_t t) {
  const int lane = threadIdx.x & 63;
  const int32_t c = b + lane < B ? cu[b + lane] : 0x7FFFFFFF;
  const int32_t past = b + 64 < B ? cu[b + 64] : 0x7FFFFFFF;
  int i = 0;                                  // the last of the 64 that is <= t
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    if (__shfl(c, i + off, 64) <= t) i += off;
  }
  int64_t lo = b + i;
  if (b + 64 < B && past <= t) {
    lo = b + 64;
    for (int64_t hi = B; hi - lo > 1;) {
      const int64_t mid = (lo + hi) >> 1;
      if (cu[mid] <= t) lo = mid; else hi = mid;
    }
  }
  return lo;
}

// Page of entry j of a request: kept, from the free list at `taken`, or -1.
__device__ __forceinline__ int32_t entry_of(const TablesArgs& a, int64_t b, const Need& n,
                                            int32_t taken, int32_t j) {
  if (j < n.held) return j < a.width_in ? a.table_in[b * a.width_in + j] : -1;
  if (j >= n.need) return -1;
  const int64_t f = (int64_t)taken + (j - n.held);
  return f < a.n_free ? a.free_pages[f] : -1;
}

constexpr int kScanThreads = 1024, kScanRoom = 4096;

__global__ __launch_bounds__(kScanThreads) void tables_scan_kernel(TablesArgs a, Geometry g) {
  __shared__ int32_t lds_t[kScanRoom], lds_p[kScanRoom];
  Sums base{0, 0};
  for (int64_t b0 = 0; b0 < a.B; b0 += kScanRoom) {
    base = scan_requests<kScanThreads>(a, g, b0, base, kScanRoom, lds_t, lds_p);
    for (int i = threadIdx.x; i < kScanRoom && b0 + i < a.B; i += kScanThreads)
      a.cu_tokens[b0 + i] = lds_t[i], a.cu_pages[b0 + i] = lds_p[i];
    __syncthreads();
  }
  if (threadIdx.x == 0) a.cu_tokens[a.B] = stored(base.t), a.cu_pages[a.B] = stored(base.p);
}

// A wave takes kRun entries of one row, or kTokens tokens, at a time.
template <bool OWN>
__global__ __launch_bounds__(kThreads) void tables_fill_kernel(TablesArgs a, Geometry g) {
  __shared__ int32_t lds_t[OWN ? kOwnScan : 1], lds_p[OWN ? kOwnScan : 1];
  const int32_t *cu_t = a.cu_tokens, *cu_p = a.cu_pages;
  int32_t total;
  if (OWN) {
    const Sums end = scan_requests<kThreads>(a, g, 0, Sums{0, 0}, kOwnScan, lds_t, lds_p);
    cu_t = lds_t, cu_p = lds_p;
    total = stored(end.t);
    if (blockIdx.x == 0) {
      for (int b = threadIdx.x; b < a.B; b += kThreads) a.cu_tokens[b] = lds_t[b], a.cu_pages[b] = lds_p[b];
      if (threadIdx.x == 0) a.cu_tokens[a.B] = total, a.cu_pages[a.B] = stored(end.p);
    }
  } else {
    total = a.cu_tokens[a.B];
  }
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t it = wave; it < g.items; it += (int64_t)gridDim.x * kWaves) {
    if (it >= g.token_items) {
      const uint32_t r = (uint32_t)(it - g.token_items);
      const int64_t b = div_by(r, g.by_row), c = r - b * g.row_items;
      const Need n = need_of(a, g, b);
      const int32_t taken = cu_p[b];
      if (c == 0 && lane == 0) a.lens[b] = to_i32((int64_t)n.old + n.fresh);
#pragma unroll
      for (int k = 0; k < kRun / 64; ++k) {
        const int64_t j = c * kRun + k * 64 + lane;
        if (j < a.width) a.table[b * a.width + j] = entry_of(a, b, n, taken, (int32_t)j);
      }
      continue;
    }
    const int64_t t0 = it * kTokens, t = t0 + lane;
    int32_t slot = -1, pos = 0;
    if (t0 < total) {                         // the same for the wave
      const int64_t b = lane_request_of(cu_t, a.B, request_of(cu_t, a.B, t0), min(t, (int64_t)total - 1));
      const Need n = need_of(a, g, b);
      if (t < total) {
        pos = to_i32((int64_t)n.old + (t - cu_t[b]));
        const int32_t j = (int32_t)div_by(pos, g.page);
        if (j < n.need) {
          const int32_t pg = entry_of(a, b, n, cu_p[b], j);
          if (pg >= 0) slot = to_i32((int64_t)pg * a.page + (pos - j * (int32_t)a.page));
        }
      }
    }
    if (t < a.tokens) {
      a.slots[t] = slot;
      a.positions[t] = pos;
    }
  }
}

}  // namespace

hipError_t launch_page_tables(const TablesArgs& a, hipStream_t s) {
  Geometry g;
  g.page = fast_div((uint32_t)a.page);
  const int64_t cap = a.page * a.width;
  g.cap = (int32_t)(cap < 0x7FFFFFFF ? cap : 0x7FFFFFFF);
  g.token_items = (int32_t)((a.tokens + kTokens - 1) / kTokens);
  g.row_items = (a.width + kRun - 1) / kRun;
  g.items = g.token_items + a.B * g.row_items;
  if (g.items > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  g.by_row = fast_div((uint32_t)g.row_items);
  const int64_t need = (g.items + kWaves - 1) / kWaves, most = device_cus() > 0 ? (int64_t)device_cus() * 4 : 1;
  const unsigned blocks = (unsigned)(need < 1 ? 1 : (need < most ? need : most));
  if (a.B <= kOwnScan) {
    tables_fill_kernel<true><<<blocks, kThreads, 0, s>>>(a, g);
    return hipGetLastError();
  }
  tables_scan_kernel<<<1, kScanThreads, 0, s>>>(a, g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  tables_fill_kernel<false><<<blocks, kThreads, 0, s>>>(a, g);
  return hipGetLastError();
}

}  // namespace fk

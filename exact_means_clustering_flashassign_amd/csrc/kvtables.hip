// Block tables, token slots and positions from request lengths (integers only).
//
// Two running sums over the requests carry everything: new tokens (which
// request a token of the step belongs to) and pages taken from the free list
// (which free page an entry gets). tables_scan_kernel writes both; in
// tables_fill_kernel every table entry and every token is then independent.
#include "fk_kv.hpp"

namespace fk {
namespace {

constexpr int kThreads = 256;

struct Need {
  int64_t old, len, held, need;   // held and need in pages
};

__device__ __forceinline__ Need need_of(const TablesArgs& a, int64_t b) {
  Need n;
  const int32_t o = a.len_old[b], w = a.len_new[b];
  n.old = o > 0 ? o : 0;
  n.len = n.old + (w > 0 ? w : 0);
  n.held = min((n.old + a.page - 1) / a.page, a.width);
  n.need = min((n.len + a.page - 1) / a.page, a.width);
  return n;
}

__device__ __forceinline__ int32_t to_i32(int64_t v) {
  return (int32_t)(v < 0x7FFFFFFF ? v : 0x7FFFFFFF);
}

// One block: running sums over the requests, kThreads at a time.
__global__ __launch_bounds__(kThreads) void tables_scan_kernel(TablesArgs a) {
  __shared__ int64_t part[2][kThreads];
  int64_t base_t = 0, base_p = 0;
  if (threadIdx.x == 0) a.cu_tokens[0] = a.cu_pages[0] = 0;
  for (int64_t b0 = 0; b0 < a.B; b0 += kThreads) {
    const int64_t b = b0 + threadIdx.x;
    int64_t t = 0, p = 0;
    if (b < a.B) {
      const Need n = need_of(a, b);
      t = n.len - n.old;
      p = n.need - n.held;
      a.lens[b] = to_i32(n.len);
    }
    part[0][threadIdx.x] = t;
    part[1][threadIdx.x] = p;
    for (int off = 1; off < kThreads; off <<= 1) {
      __syncthreads();
      int64_t ut = 0, up = 0;
      if ((int)threadIdx.x >= off) {
        ut = part[0][threadIdx.x - off];
        up = part[1][threadIdx.x - off];
      }
      __syncthreads();
      part[0][threadIdx.x] += ut;
      part[1][threadIdx.x] += up;
    }
    __syncthreads();
    if (b < a.B) {
      a.cu_tokens[b + 1] = to_i32(base_t + part[0][threadIdx.x]);
      a.cu_pages[b + 1] = to_i32(base_p + part[1][threadIdx.x]);
    }
    base_t += part[0][kThreads - 1];
    base_p += part[1][kThreads - 1];
    __syncthreads();
  }
}

// Physical page of entry j of request b: kept, from the free list, or -1.
__device__ __forceinline__ int32_t entry_of(const TablesArgs& a, int64_t b, const Need& n,
                                            int64_t j) {
  if (j < n.held) return j < a.width_in ? a.table_in[b * a.width_in + j] : -1;
  if (j >= n.need) return -1;
  const int64_t f = (int64_t)a.cu_pages[b] + (j - n.held);
  return f < a.n_free ? a.free_pages[f] : -1;
}

__global__ __launch_bounds__(kThreads) void tables_fill_kernel(TablesArgs a) {
  const int64_t entries = a.B * a.width, all = entries + a.tokens;
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += step) {
    if (i < entries) {
      const int64_t b = i / a.width, j = i - b * a.width;
      a.table[i] = entry_of(a, b, need_of(a, b), j);
      continue;
    }
    const int64_t t = i - entries;
    int32_t slot = -1;
    int64_t pos = 0;
    if (a.B > 0 && t < a.cu_tokens[a.B]) {
      int64_t lo = 0, hi = a.B;             // the request with cu[lo] <= t < cu[lo + 1]
      while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (a.cu_tokens[mid] <= t) lo = mid; else hi = mid;
      }
      const Need n = need_of(a, lo);
      pos = n.old + (t - a.cu_tokens[lo]);
      const int64_t j = pos / a.page;
      if (j < n.need) {
        const int32_t pg = entry_of(a, lo, n, j);
        if (pg >= 0) slot = to_i32((int64_t)pg * a.page + pos % a.page);
      }
    }
    a.slots[t] = slot;
    a.positions[t] = to_i32(pos);
  }
}

}  // namespace

hipError_t launch_page_tables(const TablesArgs& a, hipStream_t s) {
  tables_scan_kernel<<<1, kThreads, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t all = a.B * a.width + a.tokens;
  if (all == 0) return hipSuccess;
  const int64_t blocks = (all + kThreads - 1) / kThreads;
  tables_fill_kernel<<<(unsigned)(blocks < 4096 ? blocks : 4096), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace fk

// worklist.cuh -- work lists over a batch's requests, built by each block from
// the tree index: no list is kept between calls and no kernel prepares one.
#pragma once

#include "common.cuh"

namespace flide {

constexpr int kMaxListR = 2048;  // requests of a work list

// pref[r * step] = sum of count(0 .. r-1), pref[R * step] = the total; 64 bits,
// because a long history's units times its heads pass 2^31.  `part` holds the
// warps' sums (32 entries); ends with a barrier.
template <typename F>
__device__ __forceinline__ void request_prefix(int R, F count, long long *pref, long long *part,
                                               int step = 1) {
  const int nt = blockDim.x, per = (R + nt - 1) / nt, tid = threadIdx.x;
  const int lo = min(R, tid * per), hi = min(R, lo + per);
  long long sum = 0;
  for (int r = lo; r < hi; ++r) {
    const long long c = count(r);
    pref[(size_t)r * step] = c;
    sum += c;
  }
  const int lane = tid & 31, warp = tid >> 5;
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  long long base = incl - sum;
  for (int w = 0; w < warp; ++w) base += part[w];
  for (int r = lo; r < hi; ++r) {
    const long long c = pref[(size_t)r * step];
    pref[(size_t)r * step] = base;
    base += c;
  }
  if (tid == nt - 1) pref[(size_t)R * step] = base;
  __syncthreads();
}

// the request r with pref[r] <= u < pref[r + 1]
__device__ __forceinline__ int request_of(const long long *pref, int R, long long u) {
  int lo = 0, hi = R;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pref[mid + 1] > u) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// A history's rows are counted in 32 bits, tile ends past the last row included.
constexpr int kMaxHistory = 1 << 30;

// A request's history rows: packed rows [base, base + len), or rows of pool
// slot `slot` through its block table.
struct HistoryView {
  const int32_t *block_table, *req_slot;  // NULL table: packed
  int max_blocks, block_rows, n_blocks, n_slots;
  long long rows;  // rows of the packed arrays
};

// Rows that can be read of a history of `len` rows, packed from row p0 or in pool
// slot `slot`: 0 and a status code where the slot or the lengths are bad.  *base:
// its first packed row, or its slot.
__device__ __forceinline__ int history_length(const HistoryView &h, int p0, int len, int slot, int *base,
                                              int *code) {
  *base = h.block_table ? slot : p0;
  if (len <= 0) return 0;
  if (len > kMaxHistory) {
    *code = FLIDE_ERR_CAPACITY;
    return 0;
  }
  if (h.block_table) {
    if (slot < 0 || slot >= h.n_slots || len > (long long)h.max_blocks * h.block_rows) {
      *code = FLIDE_ERR_INVALID;
      return 0;
    }
  } else if (p0 < 0 || (long long)p0 + len > h.rows) {
    *code = h.rows ? FLIDE_ERR_CAPACITY : FLIDE_ERR_SHAPE;
    return 0;
  }
  return len;
}

// The same of request r, with the status set where `report`.
__device__ __forceinline__ int history_rows(const flide_tree_index &x, const HistoryView &h, int r,
                                            bool report, int *base) {
  int code = 0;
  const int p0 = x.past_start[r];
  const int len = history_length(h, p0, x.past_start[r + 1] - p0, h.block_table ? h.req_slot[r] : 0, base, &code);
  if (code && report) set_status(x.status, code);
  return len;
}

// Row of the K/V arrays that holds history row i, or -1 (status set) where the
// table has no valid block.
__device__ __forceinline__ long long history_row(const flide_tree_index &x, const HistoryView &h,
                                                 long long base, int i) {
  if (!h.block_table) return base + i;
  const int b = i / h.block_rows;
  const int blk = h.block_table[base * h.max_blocks + b];
  if (blk < 0 || blk >= h.n_blocks) {
    set_status(x.status, FLIDE_ERR_INVALID);
    return -1;
  }
  return (long long)blk * h.block_rows + (i - b * h.block_rows);
}

}  // namespace flide

// draft.cuh -- what the draft attention kernels share: their parameters and the
// division of a batch's (request, row tile, kv head, key unit) list over workers.
// A run of a worker inside one item costs what `extra` units cost (its queries,
// its partial's store, an emptied pipeline), so each item begins with that many
// units without keys: a worker with many short histories gets fewer keys.
#pragma once

#include "common.cuh"
#include "worklist.cuh"

namespace flide {

constexpr float kLog2eD = 1.4426950408889634f;

// A request in the work list: its first unit and item, the units of one item, its
// stream tokens from t0, its history rows and (history_rows) their base.  Entry R
// holds the totals.
struct __align__(16) DraftReq {
  long long unit0;
  int item0, units, t0, tokens, hist, base;
};

struct DraftParams {
  flide_tree_index x;
  HistoryView hist;
  const void *q, *k, *v, *past_k, *past_v;
  const float *descale;
  int Hq, Hkv, G, d;
  float scale;
  // row tiles of tile_rows query rows (tokens x heads of the group), key units of
  // `unit` history rows; a run's slot holds 2^parts_log partials of a tile's rows
  int workers, tile_rows, parts_log, unit, extra;
  void *out;
  float *lse;
  // workspace: the work list, partial rows and their (max, sum)
  DraftReq *list;
  float *part_o, *part_ml;
};

__device__ __forceinline__ int tiles_of(const DraftParams &p, int tokens) {
  return (int)(((long long)tokens * p.G + p.tile_rows - 1) / p.tile_rows);
}

// workers that get a unit (none of them an empty run: the join reads the slot
// of every worker between an item's first and last)
__device__ __forceinline__ int workers_of(long long U, int W) { return (int)min((long long)W, U); }
// first unit of worker w
__device__ __forceinline__ long long worker_start(long long U, int W, int w) { return w * U / W; }
// the worker whose units contain u
__device__ __forceinline__ int worker_of(long long U, int W, long long u) {
  // a 64-bit quotient by way of a double's, put right by one where that rounded
  const long long num = (u + 1) * W - 1;
  int w = (int)((double)num / (double)U);
  if ((long long)w * U > num) --w;
  else if ((long long)(w + 1) * U <= num) ++w;
  return w;
}

// The batch's work list, in shared memory and, for the join kernel, in the
// workspace; false (and no list) where the status word says that the batch failed:
// one thread's reading, since it may change while the grid runs.  part: 64 entries.
// Ends with a barrier.  What a request's number alone addresses is loaded before
// anything is waited for: after a long history nothing of it is left in L2, and
// every dependent load takes a microsecond.
__device__ __forceinline__ bool draft_list(const DraftParams &p, DraftReq *list, long long *part) {
  const flide_tree_index &x = p.x;
  const int R = x.R, nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (R + nt - 1) / nt, lo = min(R, tid * per), hi = min(R, lo + per);
  const int stop = tid == 0 ? failed(x.status) : 0;
  int n0 = 0, n1 = 0, p0 = 0, p1 = 0, slot = 0;
  auto first = [&](int r) {
    n0 = x.req_node[r];
    n1 = x.req_node[r + 1];
    p0 = x.past_start[r];
    p1 = x.past_start[r + 1];
    if (p.hist.block_table) slot = p.hist.req_slot[r];
  };
  if (lo < hi) first(lo);
  if (__syncthreads_or(stop)) return false;
  long long units = 0, items = 0;
  for (int r = lo; r < hi; ++r) {
    if (r > lo) first(r);
    DraftReq q;
    // debug build: the request's nodes lie among the tree's, its tokens in the stream
    const int N = x.counts[FLIDE_CNT_N];
    if (!in_bounds(x.status, x.counts, n0, N + 1, 802) || !in_bounds(x.status, x.counts, n1, N + 1, 802)) n0 = n1 = 0;
    q.t0 = n1 > n0 ? x.node_start[n0] : 0;
    q.tokens = n1 > n0 ? x.node_start[n1] - q.t0 : 0;
    if (!in_bounds(x.status, x.counts, (long long)q.t0 + q.tokens, x.counts[FLIDE_CNT_T] + 1ll, 803)) q.tokens = 0;
    int code = 0;
    q.hist = history_length(p.hist, p0, p1 - p0, slot, &q.base, &code);
    if (code && blockIdx.x == 0) set_status(x.status, code);
    q.unit0 = units;
    q.item0 = (int)items;
    q.units = q.hist > 0 ? (q.hist + p.unit - 1) / p.unit + p.extra : 0;
    const long long n = (long long)tiles_of(p, q.tokens) * p.Hkv;
    items += n;
    units += n * q.units;
    list[r] = q;
  }
  long long iu = units, ii = items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long yu = __shfl_up_sync(0xffffffffu, iu, o), yi = __shfl_up_sync(0xffffffffu, ii, o);
    if (lane >= o) {
      iu += yu;
      ii += yi;
    }
  }
  if (lane == 31) {
    part[warp] = iu;
    part[32 + warp] = ii;
  }
  __syncthreads();
  long long bu = iu - units, bi = ii - items;
  for (int w = 0; w < warp; ++w) {
    bu += part[w];
    bi += part[32 + w];
  }
  for (int r = lo; r < hi; ++r) {
    list[r].unit0 += bu;
    list[r].item0 += (int)bi;
    if (blockIdx.x == 0) p.list[r] = list[r];
  }
  if (tid == nt - 1) {
    const DraftReq end{bu + units, (int)(bi + items), 0, 0, 0, 0, 0};
    list[R] = end;
    if (blockIdx.x == 0) p.list[R] = end;
  }
  __syncthreads();
  return true;
}

// A worker's run: history rows [k0, k1) of one item (row tile `tile`, kv head
// hk of a request of `tokens` tokens from t0); base: history_rows.
struct Run {
  int tile, hk, t0, tokens, k0, k1, base;
  long long slot;
};

// The next run of worker w from unit u on, which moves past it; false at the end.
__device__ __forceinline__ bool draft_run(const DraftParams &p, const DraftReq *list, long long &u,
                                          long long u_end, int w, Run &run) {
  while (u < u_end) {
    int lo = 0, hi = p.x.R;  // the request with unit0 <= u < the next one's
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (list[mid + 1].unit0 > u) hi = mid; else lo = mid + 1;
    }
    const DraftReq q = list[lo];
    const long long at = u - q.unit0;
    const int li = at >> 31 ? (int)(at / q.units) : (int)at / q.units;  // (a 64-bit quotient is slow)
    const int c0 = (int)(at - (long long)li * q.units);
    const int c1 = (int)min((long long)q.units, c0 + (u_end - u));
    u += c1 - c0;
    run.tile = li / p.Hkv;
    run.hk = li - run.tile * p.Hkv;
    run.t0 = q.t0;
    run.tokens = q.tokens;
    run.base = q.base;
    run.k0 = max(c0 - p.extra, 0) * p.unit;
    run.k1 = min(q.hist, (c1 - p.extra) * p.unit);
    run.slot = (long long)w + q.item0 + li;
    if (run.k1 > run.k0) return true;
  }
  return false;
}

// draft_wide.cu (sets p's unit and extra): operands of 32, 64, 128 (bf16, e4m3) or 256 rows (bf16) on tcgen05,
// of which whole tokens fill p.tile_rows; d of 128, or 64 (bf16, no 32-row operand)
// whether a call of R requests leaves such a tile its shared memory
bool draft_wide_fits(int operand, int d, bool f8, long long R);
int draft_wide_launch(DraftParams &p, int operand, int past_rows, bool f8, int dev, cudaStream_t s);

}  // namespace flide

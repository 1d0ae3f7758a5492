// draft.cuh -- what the draft attention kernels share: their parameters and the
// division of a batch's (request, row tile, kv head, key unit) list over workers.
#pragma once

#include "common.cuh"
#include "worklist.cuh"

namespace flide {

constexpr float kLog2eD = 1.4426950408889634f;

struct DraftParams {
  flide_tree_index x;
  HistoryView hist;
  const void *q, *k, *v, *past_k, *past_v;
  const float *descale;
  int Hq, Hkv, G, d;
  float scale;
  // row tiles of tile_rows query rows (tokens x heads of the group), key units of
  // `unit` history rows; a run's slot holds 2^parts_log partials of a tile's rows
  int workers, tile_rows, parts_log, unit;
  void *out;
  float *lse;
  // workspace: prefix sums of units and items, partial rows and their (max, sum)
  long long *unit0, *item0;
  float *part_o, *part_ml;
};

// tokens of request r's stream region
__device__ __forceinline__ int request_tokens(const flide_tree_index &x, int r, int *t0) {
  const int n0 = x.req_node[r], n1 = x.req_node[r + 1];
  *t0 = n1 > n0 ? x.node_start[n0] : 0;
  return n1 > n0 ? x.node_start[n1] - *t0 : 0;
}

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

// A worker's run: history rows [k0, k1) of one item (row tile `tile`, kv head
// hk of a request of `tokens` tokens from t0); base: history_rows.
struct Run {
  int tile, hk, t0, tokens, k0, k1;
  long long base, slot;
};

// Prefix sums over the requests of their units and items, in
// shared memory, and for the join kernel in the workspace.
__device__ __forceinline__ void draft_lists(const DraftParams &p, long long *unit0, long long *item0,
                                            long long *part) {
  const flide_tree_index &x = p.x;
  const int unit = p.unit;
  request_prefix(x.R, [&](int r) -> long long {
    int t0;
    return (long long)tiles_of(p, request_tokens(x, r, &t0)) * p.Hkv;
  }, item0, part);
  request_prefix(x.R, [&](int r) -> long long {
    long long base;
    const long long n = history_rows(x, p.hist, r, blockIdx.x == 0, &base);
    return (item0[r + 1] - item0[r]) * ((n + unit - 1) / unit);
  }, unit0, part);
  if (blockIdx.x == 0)
    for (int r = threadIdx.x; r <= x.R; r += blockDim.x) {
      p.unit0[r] = unit0[r];
      p.item0[r] = item0[r];
    }
}

// The run that starts at unit u of worker w; returns its units.
__device__ __forceinline__ int draft_run(const DraftParams &p, const long long *unit0,
                                         const long long *item0, long long u, long long u_end,
                                         int w, Run &run) {
  const int unit = p.unit;
  const int r = request_of(unit0, p.x.R, u);
  run.tokens = request_tokens(p.x, r, &run.t0);
  const int n = history_rows(p.x, p.hist, r, false, &run.base);
  const int units = (n + unit - 1) / unit;
  const long long li = (u - unit0[r]) / units;
  const int c0 = (int)(u - unit0[r] - li * units);
  const int c1 = (int)min((long long)units, c0 + (u_end - u));
  run.tile = (int)(li / p.Hkv);
  run.hk = (int)(li % p.Hkv);
  run.k0 = c0 * unit;
  run.k1 = min(n, c1 * unit);
  run.slot = w + item0[r] + li;
  return c1 - c0;
}

// draft_wide.cu: tiles of 32, 64, 128 (bf16, e4m3) or 256 rows (bf16) on tcgen05, d == 128
int draft_wide_launch(const DraftParams &p, int past_rows, bool f8, int dev, cudaStream_t s);

}  // namespace flide

// draft_attn.cu -- attention of a few query tokens per request (a root and the
// tree drafted below it) over a long history.
//
//   o_t = sum_j w_tj v_j / sum_j w_tj,  w_tj = exp(scale q_t . k_j),
//   lse_t = log sum_j w_tj
// over the request's history rows and the tokens on t's path (its ancestors'
// tokens, its own node up to itself).  Fork attention gives a query tile's
// whole key range to one block; here a request has one tile or two, so the
// history is cut along the keys instead:
//   - the batch's work is the list of (request, row tile, kv head, key unit),
//     request major; worker w of W takes units [w U / W, (w + 1) U / W): every
//     worker streams the same number of keys, however ragged the histories;
//   - a worker's run inside one (request, row tile, kv head) item leaves a
//     partial (O, max, sum) in slot w + item, which no other run shares, as
//     every next run raises w, item or both;
//   - the join kernel adds the tokens on the row's path, a few, with plain
//     fused multiply-adds: a masked key is never multiplied, so what stands in
//     a sibling branch cannot reach a row, NaN and infinity included.
// History rows need no mask but their number, and rows past it are not read.
#include <cuda_fp8.h>
#include <math.h>

#include "common.cuh"
#include "sm100.cuh"
#include "worklist.cuh"

namespace flide {
namespace {

using sm100::ex2_approx;

constexpr float kLog2eD = 1.4426950408889634f;
constexpr float kLn2D = 0.6931471805599453f;
constexpr int kRows = 16;         // query rows of a tile (tokens x heads of the group)
constexpr int kMaxWorkers = 1024; // what the workspace allows for

struct DraftParams {
  flide_tree_index x;
  HistoryView hist;
  const void *q, *k, *v, *past_k, *past_v;
  const float *descale;
  int Hq, Hkv, G, d;
  float scale;
  int workers;
  void *out;
  float *lse;
  // workspace: prefix sums of units and items, partial rows and their (max, sum)
  long long *unit0, *item0;
  float *part_o, *part_ml;
};

template <typename T>
__device__ __forceinline__ float value_of(const T *p) { return load_f(p); }
template <>
__device__ __forceinline__ float value_of<uint8_t>(const uint8_t *p) {
  __nv_fp8_e4m3 c;
  c.__x = *p;
  return (float)c;
}

// tokens of request r's stream region
__device__ __forceinline__ int request_tokens(const flide_tree_index &x, int r, int *t0) {
  const int n0 = x.req_node[r], n1 = x.req_node[r + 1];
  *t0 = n1 > n0 ? x.node_start[n0] : 0;
  return n1 > n0 ? x.node_start[n1] - *t0 : 0;
}

__device__ __forceinline__ int tiles_of(int tokens, int G) {
  return (int)(((long long)tokens * G + kRows - 1) / kRows);
}

// workers that get a unit (none of them an empty run: the join reads the slot
// of every worker between an item's first and last)
__device__ __forceinline__ int workers_of(long long U, int W) { return (int)min((long long)W, U); }
// first unit of worker w
__device__ __forceinline__ long long worker_start(long long U, int W, int w) { return w * U / W; }
// the worker whose units contain u
__device__ __forceinline__ int worker_of(long long U, int W, long long u) {
  return (int)(((u + 1) * W - 1) / U);
}

// A worker's run: key units [c0, c1) of one item.
struct Run {
  int r, tile, hk, t0, tokens, hist, k0, k1;
  long long base, slot;
};

// Any element type and head size: CUDA cores, 32 keys a step.
constexpr int kPT = 128;   // threads
constexpr int kPKeys = 32; // keys of a unit

template <typename T>
__global__ void __launch_bounds__(kPT) draft_part_portable(const DraftParams p) {
  extern __shared__ float smem[];
  __shared__ long long part[32];
  const flide_tree_index &x = p.x;
  if (failed(x.status)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int d = p.d, ld = d + 4, R = x.R;
  long long *unit0 = reinterpret_cast<long long *>(smem), *item0 = unit0 + (R + 1);
  float *sq = smem + 4 * (R + 1) + (4 - (4 * (R + 1)) % 4) % 4, *sk = sq + kRows * ld, *sv = sk + kPKeys * ld;
  float *sp = sv + kPKeys * ld;
  request_prefix(R, [&](int r) -> long long {
    int t0;
    return (long long)tiles_of(request_tokens(x, r, &t0), p.G) * p.Hkv;
  }, item0, part);
  request_prefix(R, [&](int r) -> long long {
    long long base;
    const long long n = history_rows(x, p.hist, r, blockIdx.x == 0, &base);
    return (item0[r + 1] - item0[r]) * ((n + kPKeys - 1) / kPKeys);
  }, unit0, part);
  if (blockIdx.x == 0)
    for (int r = tid; r <= R; r += kPT) {
      p.unit0[r] = unit0[r];
      p.item0[r] = item0[r];
    }
  const long long U = unit0[R];
  const int w = blockIdx.x, W = workers_of(U, p.workers);
  if (w >= W) return;
  long long u = worker_start(U, W, w);
  const long long u_end = worker_start(U, W, w + 1);
  const T *Q = static_cast<const T *>(p.q), *K = static_cast<const T *>(p.past_k),
          *Vp = static_cast<const T *>(p.past_v);
  const float qk_scale = p.scale * kLog2eD * (p.descale ? p.descale[0] * p.descale[1] : 1.f);
  const int nd = d / 32;
  while (u < u_end) {
    const int r = request_of(unit0, R, u);
    int t0;
    const int tokens = request_tokens(x, r, &t0);
    long long base;
    const int n = history_rows(x, p.hist, r, false, &base);
    const int units = (n + kPKeys - 1) / kPKeys;
    const long long li = (u - unit0[r]) / units;
    const int c0 = (int)(u - unit0[r] - li * units);
    const int c1 = (int)min((long long)units, c0 + (u_end - u));
    const int tile = (int)(li / p.Hkv), hk = (int)(li % p.Hkv);
    const long long slot = w + item0[r] + li;
    u += c1 - c0;
    __syncthreads();
    for (int e = tid; e < kRows * d; e += kPT) {
      const int row = e / d, i = e - row * d, g = tile * kRows + row;
      sq[row * ld + i] = g < tokens * p.G
          ? value_of(Q + ((size_t)(t0 + g / p.G) * p.Hq + hk * p.G + g % p.G) * d + i) : 0.f;
    }
    float m[4], l[4], acc[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    }
    for (int c = c0; c < c1; ++c) {
      __syncthreads();
      const int left = min(kPKeys, n - c * kPKeys);
      for (int kr = warp; kr < kPKeys; kr += kPT / 32) {
        const long long row = kr < left ? history_row(x, p.hist, base, c * kPKeys + kr) : -1;
        for (int i = lane; i < d; i += 32) {
          const size_t at = ((size_t)max(row, 0ll) * p.Hkv + hk) * d + i;
          sk[kr * ld + i] = row >= 0 ? value_of(K + at) : 0.f;
          sv[kr * ld + i] = row >= 0 ? value_of(Vp + at) : 0.f;
        }
      }
      __syncthreads();
      // rows 4 warp .. 4 warp + 3, key = lane
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      for (int i = 0; i < d; i += 4) {
        const float4 b = *reinterpret_cast<const float4 *>(sk + lane * ld + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 a = *reinterpret_cast<const float4 *>(sq + (4 * warp + j) * ld + i);
          s[j] = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s[j]))));
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = lane < left ? s[j] * qk_scale : -INFINITY;
        const float mn = fmaxf(m[j], warp_max(v));
        const float base_m = mn == -INFINITY ? 0.f : mn;
        const float e = exp2f(v - base_m), f = exp2f(m[j] - base_m);
        l[j] = l[j] * f + warp_sum(e);
        m[j] = mn;
        for (int i = 0; i < 8; ++i) acc[j][i] *= f;
        sp[(4 * warp + j) * kPKeys + lane] = e;
      }
      __syncwarp();
      for (int kr = 0; kr < left; ++kr) {
        float pr[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) pr[j] = sp[(4 * warp + j) * kPKeys + kr];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < nd) {
            const float b = sv[kr * ld + lane + 32 * i];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j][i] = fmaf(pr[j], b, acc[j][i]);
          }
      }
      __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const size_t row = slot * kRows + 4 * warp + j;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < nd) p.part_o[row * d + lane + 32 * i] = acc[j][i];
      if (lane == 0) {
        p.part_ml[2 * row] = m[j];
        p.part_ml[2 * row + 1] = l[j];
      }
    }
  }
}

// One warp per (token, query head): the tokens on its path, then the partial
// results of its history, then the output row and its log-sum-exp.
template <typename T, typename TOut>
__global__ void __launch_bounds__(256) draft_join_kernel(const DraftParams p) {
  const flide_tree_index &x = p.x;
  if (failed(x.status)) return;
  const int lane = threadIdx.x & 31;
  const long long job = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int t = (int)(job / p.Hq), h = (int)(job % p.Hq);
  if (t >= x.counts[FLIDE_CNT_T]) return;
  const int hk = h / p.G, d = p.d, nd = d / 32;
  const int n = (int)checked(x.status, x.counts, x.token_node[t], x.counts[FLIDE_CNT_N], 801);
  const T *Q = static_cast<const T *>(p.q), *K = static_cast<const T *>(p.k), *Vs = static_cast<const T *>(p.v);
  const float sv = p.descale ? p.descale[2] : 1.f;
  const float qk_scale = p.scale * kLog2eD * (p.descale ? p.descale[0] * p.descale[1] : 1.f);
  float qv[8], acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    qv[i] = i < nd ? value_of(Q + ((size_t)t * p.Hq + h) * d + lane + 32 * i) * qk_scale : 0.f;
    acc[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int a = x.anc_ptr[n]; a < x.anc_ptr[n + 1]; ++a) {
    const int node = x.anc_node[a];
    const int e = node == n ? t + 1 : x.node_start[node + 1];
    for (int j = x.node_start[node]; j < e; ++j) {
      const size_t at = ((size_t)j * p.Hkv + hk) * d + lane;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < nd) s = fmaf(qv[i], value_of(K + at + 32 * i), s);
      s = warp_sum(s);
      const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m - ref), w = exp2f(s - ref);
      l = l * f + w;
      m = mn;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < nd) acc[i] = fmaf(w, value_of(Vs + at + 32 * i), acc[i] * f);
    }
  }
  const int r = x.node_req[n];
  const long long U = p.unit0[x.R], ua = p.unit0[r];
  const long long items = p.item0[r + 1] - p.item0[r];
  const long long per = items > 0 ? (p.unit0[r + 1] - ua) / items : 0;  // units of one item
  if (per > 0) {
    const int row = (t - x.node_start[x.req_node[r]]) * p.G + h % p.G;
    const long long li = (long long)(row / kRows) * p.Hkv + hk;
    const long long u0 = ua + li * per;
    const int W = workers_of(U, p.workers);
    const int w0 = worker_of(U, W, u0), w1 = worker_of(U, W, u0 + per - 1);
    for (int w = w0; w <= w1; ++w) {
      const size_t pr = (size_t)(w + p.item0[r] + li) * kRows + row % kRows;
      const float pm = p.part_ml[2 * pr], pl = p.part_ml[2 * pr + 1];
      const float mn = fmaxf(m, pm), ref = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m - ref), g = exp2f(pm - ref);
      l = l * f + pl * g;
      m = mn;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < nd) acc[i] = fmaf(g, p.part_o[pr * d + lane + 32 * i], acc[i] * f);
    }
  }
  const float inv = sv / l;
  TOut *O = static_cast<TOut *>(p.out) + ((size_t)t * p.Hq + h) * d + lane;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < nd) store_f(O + 32 * i, acc[i] * inv);
  if (p.lse && lane == 0) p.lse[(size_t)t * p.Hq + h] = (m + log2f(l)) * kLn2D;
}

struct DraftSpace {
  size_t unit0, item0, ml, o, total;
};

// Bytes of the workspace's parts: a slot for every worker and item.
DraftSpace draft_space(long long R, long long T, long long Hq, long long Hkv, long long d) {
  const long long G = Hq / Hkv;
  const long long slots = kMaxWorkers + ((T * G + kRows - 1) / kRows + R) * Hkv;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  DraftSpace s;
  s.unit0 = 0;
  s.item0 = up((R + 1) * sizeof(long long));
  s.ml = s.item0 + up((R + 1) * sizeof(long long));
  s.o = s.ml + up((size_t)slots * kRows * 2 * sizeof(float));
  s.total = s.o + up((size_t)slots * kRows * d * sizeof(float));
  return s;
}

template <typename T, typename TOut>
int draft_launch(DraftParams &p, cudaStream_t s) {
  const size_t smem = (size_t)(p.x.R + 1) * 16 + 16 +
                      sizeof(float) * ((size_t)(kRows + 2 * kPKeys) * (p.d + 4) + kRows * kPKeys);
  if (cudaFuncSetAttribute(draft_part_portable<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)smem) != cudaSuccess)
    return FLIDE_ERR_CUDA;
  draft_part_portable<T><<<p.workers, kPT, smem, s>>>(p);
  FLIDE_LAUNCH_CHECK();
  const long long warps = (long long)p.x.T * p.Hq;
  draft_join_kernel<T, TOut><<<(unsigned)((warps + 7) / 8), 256, 0, s>>>(p);
  FLIDE_LAUNCH_CHECK();
  return FLIDE_OK;
}

int draft_attn(const void *q, const void *k, const void *v, const void *past_k, const void *past_v,
               const HistoryView &hist, const flide_tree_index *idx, int Hq, int Hkv, int d, int dtype,
               const float *descale, float scale, void *out, float *lse, void *workspace,
               size_t workspace_bytes, cudaStream_t s) {
  if (!idx || !q || !k || !v || !out || !workspace) return FLIDE_ERR_SHAPE;
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv || d < 32 || d % 32 || d > 256) return FLIDE_ERR_SHAPE;
  if (dtype != FLIDE_F32 && dtype != FLIDE_BF16 && dtype != FLIDE_E4M3) return FLIDE_ERR_SHAPE;
  if (dtype == FLIDE_E4M3 && (!descale || d != 128)) return FLIDE_ERR_SHAPE;
  if (idx->R < 0 || idx->T < 0) return FLIDE_ERR_SHAPE;
  if ((uintptr_t)workspace % 256) return FLIDE_ERR_SHAPE;
  if (idx->R > kMaxListR || (long long)idx->T * Hq > 0x3fffffffLL) return FLIDE_ERR_CAPACITY;
  if (idx->R == 0 || idx->T == 0) return FLIDE_OK;
  const DraftSpace sp = draft_space(idx->R, idx->T, Hq, Hkv, d);
  if (workspace_bytes < sp.total) return FLIDE_ERR_CAPACITY;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FLIDE_ERR_CUDA;
  char *ws = static_cast<char *>(workspace);
  DraftParams p;
  p.x = *idx;
  p.hist = hist;
  p.q = q;
  p.k = k;
  p.v = v;
  p.past_k = past_k;
  p.past_v = past_v;
  p.descale = dtype == FLIDE_E4M3 ? descale : nullptr;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.d = d;
  p.scale = scale;
  p.workers = min(kMaxWorkers, 4 * sms);
  p.out = out;
  p.lse = lse;
  p.unit0 = reinterpret_cast<long long *>(ws + sp.unit0);
  p.item0 = reinterpret_cast<long long *>(ws + sp.item0);
  p.part_ml = reinterpret_cast<float *>(ws + sp.ml);
  p.part_o = reinterpret_cast<float *>(ws + sp.o);
  if (dtype == FLIDE_F32) return draft_launch<float, float>(p, s);
  if (dtype == FLIDE_BF16) return draft_launch<__nv_bfloat16, __nv_bfloat16>(p, s);
  return draft_launch<uint8_t, __nv_bfloat16>(p, s);
}

}  // namespace
}  // namespace flide

extern "C" {

size_t flide_draft_attn_workspace_bytes(int32_t R, int32_t T, int32_t Hq, int32_t Hkv, int32_t d) {
  if (R < 0 || T < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || d <= 0) return 0;
  return flide::draft_space(R, T, Hq, Hkv, d).total;
}

int flide_draft_attn(const void *q, const void *k, const void *v, const void *past_k,
                     const void *past_v, int32_t past_rows, const flide_tree_index *idx, int32_t Hq,
                     int32_t Hkv, int32_t d, int32_t dtype, const float *descale, float scale,
                     void *out, float *lse, void *workspace, size_t workspace_bytes,
                     flide_stream stream) {
  if (past_rows < 0 || (past_k == nullptr) != (past_v == nullptr)) return FLIDE_ERR_SHAPE;
  const flide::HistoryView h{nullptr, nullptr, 0, 0, 0, 0, past_k ? past_rows : 0};
  return flide::draft_attn(q, k, v, past_k, past_v, h, idx, Hq, Hkv, d, dtype, descale, scale, out,
                           lse, workspace, workspace_bytes, (cudaStream_t)stream);
}

int flide_draft_attn_paged(const void *q, const void *k, const void *v, const void *pool_k,
                           const void *pool_v, int32_t n_blocks, int32_t block_rows,
                           const int32_t *block_table, int32_t max_blocks, const int32_t *req_slot,
                           int32_t n_slots, const flide_tree_index *idx, int32_t Hq, int32_t Hkv,
                           int32_t d, int32_t dtype, const float *descale, float scale, void *out,
                           float *lse, void *workspace, size_t workspace_bytes, flide_stream stream) {
  if (!pool_k || !pool_v || !block_table || !req_slot) return FLIDE_ERR_SHAPE;
  if (n_blocks <= 0 || max_blocks <= 0 || n_slots <= 0 || block_rows <= 0 || block_rows % 16)
    return FLIDE_ERR_SHAPE;
  const flide::HistoryView h{block_table, req_slot, max_blocks, block_rows, n_blocks, n_slots, 0};
  return flide::draft_attn(q, k, v, pool_k, pool_v, h, idx, Hq, Hkv, d, dtype, descale, scale, out,
                           lse, workspace, workspace_bytes, (cudaStream_t)stream);
}

}  // extern "C"

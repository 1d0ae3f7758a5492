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
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>
#include <cmath>

#include "draft.cuh"
#include "launch.cuh"
#include "sm100.cuh"

namespace flide {
namespace {

using namespace sm100;

constexpr float kLn2D = 0.6931471805599453f;

// float32, and bf16 head sizes of no tensor-core kernel: CUDA cores, 32 keys a step.
constexpr int kPT = 128;   // threads
constexpr int kPRows = 16; // rows of a tile
constexpr int kPKeys = 32; // keys of a unit

template <typename T>
__global__ void __launch_bounds__(kPT) draft_part_portable(const DraftParams p) {
  extern __shared__ float smem[];
  __shared__ long long part[64];
  const flide_tree_index &x = p.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int d = p.d, ld = d + 4, R = x.R;
  DraftReq *list = reinterpret_cast<DraftReq *>(smem);
  float *sq = smem + 8 * (R + 1), *sk = sq + kPRows * ld, *sv = sk + kPKeys * ld;
  float *sp = sv + kPKeys * ld;
  if (!draft_list(p, list, part)) return;
  const long long U = list[R].unit0;
  const int w = blockIdx.x, W = workers_of(U, p.workers);
  if (w >= W) return;
  long long u = worker_start(U, W, w);
  const long long u_end = worker_start(U, W, w + 1);
  const T *Q = static_cast<const T *>(p.q), *K = static_cast<const T *>(p.past_k),
          *Vp = static_cast<const T *>(p.past_v);
  const float qk_scale = p.scale * kLog2eD;
  const int nd = d / 32;
  Run run;
  while (draft_run(p, list, u, u_end, w, run)) {
    __syncthreads();
    for (int e = tid; e < kPRows * d; e += kPT) {
      const int row = e / d, i = e - row * d, g = run.tile * kPRows + row;
      sq[row * ld + i] = g < run.tokens * p.G
          ? load_f(Q + ((size_t)(run.t0 + g / p.G) * p.Hq + run.hk * p.G + g % p.G) * d + i) : 0.f;
    }
    float m[4], l[4], acc[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    }
    for (int k0 = run.k0; k0 < run.k1; k0 += kPKeys) {
      __syncthreads();
      const int left = min(kPKeys, run.k1 - k0);
      for (int kr = warp; kr < kPKeys; kr += kPT / 32) {
        const long long row = kr < left ? history_row(x, p.hist, run.base, k0 + kr) : -1;
        for (int i = lane; i < d; i += 32) {
          const size_t at = ((size_t)max(row, 0ll) * p.Hkv + run.hk) * d + i;
          sk[kr * ld + i] = row >= 0 ? load_f(K + at) : 0.f;
          sv[kr * ld + i] = row >= 0 ? load_f(Vp + at) : 0.f;
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
      const size_t row = run.slot * kPRows + 4 * warp + j;
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

// ---- tensor-core kernel for few rows -------------------------------------------
//
// A tile's 16 rows (or 32: two operands that share a warp's keys) are one
// m16n8k16 operand, so a warp needs no tile of keys in
// shared memory: it streams 16 keys at a time from global memory straight into
// operand registers and keeps its own running maximum, sum and O.
//   - S = Q K^T sums over d in any order as long as both operands agree, so a
//     lane's B operand is what it gets from 16-byte loads of its key row
//     (lane 4 g + c: key g, bytes 16 c + 64 j): the k index of the instruction
//     stands for the element that the load puts there, and Q's fragments,
//     laid out once per run in shared memory, follow it.
//   - O^T = V^T P^T takes V as the A operand: lane (g, c) loads bytes 16 g of
//     keys 2c, 2c+1, 2c+8, 2c+9 (a row's 128 bytes by 8 lanes) and byte
//     permutes pair two keys' elements; row g of tile m is element m of the
//     lane's own bytes.  P^T is then exactly the accumulator layout of S: the
//     weights go from one product to the other without leaving their lane.
// e4m3 codes become half pairs on the way (exact), bf16 stays as it is; the
// weights are rounded to that type (2^-8 bf16, 2^-11 half, relative) and summed
// unrounded in 32 bits.  O is rescaled only when a row's maximum grows by more
// than 2^8.
//
// Bound by the history's bytes.

template <int D, bool F8, int kMT>
struct MmaShape {
  static constexpr int kRows = 16 * kMT;         // query rows of a tile
  static constexpr int kMW = kMT == 1 ? 6 : 8;   // warps of a block
  static constexpr int kBlocks = kMT == 1 ? 2 : 1;  // blocks to an SM
  static constexpr int kRow = D * (F8 ? 1 : 2);  // bytes of a key row
  static constexpr int kSub = 256 / kRow;        // 16-key groups of a step: 4 KB of K and of V each
  static constexpr int kCj = kRow / 64;          // a lane's 16-byte loads of a K row
  static constexpr int kCv = kRow / 128;         // ... of a V row
  static constexpr int kSteps = D / 16;          // k steps of S, m tiles of O^T
  static constexpr int kStepKeys = 16 * kSub;
  static constexpr int kUnit = kMW * kStepKeys;  // one step of every warp
  static constexpr int kSmem = kRows * D * 4 * kMW + 2 * kMW * kRows * 4;  // O and (max, sum) per warp
};

template <int D, bool F8, int kMT>
__global__ void __launch_bounds__(MmaShape<D, F8, kMT>::kMW * 32, MmaShape<D, F8, kMT>::kBlocks)
draft_part_mma(const DraftParams p) {
  using S = MmaShape<D, F8, kMT>;
  constexpr int kMW = S::kMW, kRows = S::kRows;
  extern __shared__ float smem[];
  __shared__ long long part[64];
  __shared__ uint4 qfrag[kMT * S::kSteps * 32];
  const flide_tree_index &x = p.x;
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int R = x.R;
  // O [warp][rows][D], then max and sum [warp][rows]; the work list after them
  float *so = smem, *sm = smem + kMW * kRows * D, *sl = sm + kMW * kRows;
  DraftReq *list = reinterpret_cast<DraftReq *>(sl + kMW * kRows);
  if (!draft_list(p, list, part)) return;
  const long long U = list[R].unit0;
  const int w = blockIdx.x, W = workers_of(U, p.workers);
  if (w >= W) return;
  long long u = worker_start(U, W, w);
  const long long u_end = worker_start(U, W, w + 1);
  const float qk_scale = p.scale * kLog2eD * (F8 ? p.descale[0] * p.descale[1] : 1.f);
  const char *Kp = static_cast<const char *>(p.past_k), *Vp = static_cast<const char *>(p.past_v);
  const size_t stride = (size_t)p.Hkv * S::kRow;
  Run run;
  while (draft_run(p, list, u, u_end, w, run)) {
    __syncthreads();  // the last run's shared memory is free
    // Q fragments: lane (g, c) of step s holds rows g, g + 8 at the elements its K loads give
    for (int e = tid; e < kMT * S::kCj * 32; e += kMW * 32) {
      const int mt = e / (S::kCj * 32), j = (e >> 5) % S::kCj, eg = (e & 31) >> 2, ec = e & 3;
      uint4 *frag = qfrag + mt * S::kSteps * 32 + (e & 31);
      uint4 row[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int qr = run.tile * kRows + 16 * mt + eg + 8 * h;
        row[h] = make_uint4(0u, 0u, 0u, 0u);
        if (qr < run.tokens * p.G)
          row[h] = *reinterpret_cast<const uint4 *>(
              static_cast<const char *>(p.q) +
              ((size_t)(run.t0 + qr / p.G) * p.Hq + run.hk * p.G + qr % p.G) * S::kRow + 64 * j + 16 * ec);
      }
      if (F8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a = word_of(row[0], i), b = word_of(row[1], i);
          frag[(4 * j + i) * 32] = make_uint4(e4m3x2_to_half2(a), e4m3x2_to_half2(b),
                                                          e4m3x2_to_half2(a >> 16), e4m3x2_to_half2(b >> 16));
        }
      } else {
        frag[(2 * j) * 32] = make_uint4(row[0].x, row[1].x, row[0].y, row[1].y);
        frag[(2 * j + 1) * 32] = make_uint4(row[0].z, row[1].z, row[0].w, row[1].w);
      }
    }
    __syncthreads();

    float o[2 * kMT][S::kSteps][4];
#pragma unroll
    for (int n = 0; n < 2 * kMT; ++n)
#pragma unroll
      for (int m = 0; m < S::kSteps; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][m][i] = 0.f;
    float mx[2 * kMT], sum[2 * kMT];  // rows g + 8 n
#pragma unroll
    for (int n = 0; n < 2 * kMT; ++n) {
      mx[n] = -INFINITY;
      sum[n] = 0.f;
    }

    const char *kbase = Kp + (size_t)run.hk * S::kRow + 16 * c, *vbase = Vp + (size_t)run.hk * S::kRow + 16 * g;
    uint4 kr[S::kSub][2][S::kCj], vr[S::kSub][4][S::kCv];
    // first row of the 16-key group at history row k (a multiple of 16, as the blocks' sizes)
    auto row_at = [&](int k) -> long long { return k < run.k1 ? history_row(x, p.hist, run.base, k) : -1; };
    auto load_k = [&](const long long (&row)[S::kSub], int k0) {
#pragma unroll
      for (int s = 0; s < S::kSub; ++s)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int k = 16 * s + 8 * t + g;
          const bool ok = row[s] >= 0 && k0 + k < run.k1;
          const char *src = kbase + (row[s] + 8 * t + g) * stride;
#pragma unroll
          for (int j = 0; j < S::kCj; ++j)
            kr[s][t][j] = ok ? ld_stream(src + 64 * j) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    auto load_v = [&](const long long (&row)[S::kSub], int k0) {
#pragma unroll
      for (int s = 0; s < S::kSub; ++s)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int k = 2 * c + (t & 1) + 8 * (t >> 1);
          const bool ok = row[s] >= 0 && k0 + 16 * s + k < run.k1;
          const char *src = vbase + (row[s] + k) * stride;
#pragma unroll
          for (int j = 0; j < S::kCv; ++j)
            vr[s][t][j] = ok ? ld_stream(src + 128 * j) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    int k0 = run.k0 + warp * S::kStepKeys;
    long long row[S::kSub];
#pragma unroll
    for (int s = 0; s < S::kSub; ++s) row[s] = row_at(k0 + 16 * s);
    load_k(row, k0);
    load_v(row, k0);
#pragma unroll
    for (int s = 0; s < S::kSub; ++s) row[s] = row_at(k0 + S::kUnit + 16 * s);
    for (; k0 < run.k1; k0 += S::kUnit) {
      float sc[kMT][S::kSub][2][4];
#pragma unroll
      for (int q = 0; q < kMT; ++q)
#pragma unroll
        for (int s = 0; s < S::kSub; ++s)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[q][s][t][i] = 0.f;
#pragma unroll
      for (int st = 0; st < S::kSteps; ++st) {
        uint4 a[kMT];
#pragma unroll
        for (int q = 0; q < kMT; ++q) a[q] = qfrag[(q * S::kSteps + st) * 32 + lane];
#pragma unroll
        for (int s = 0; s < S::kSub; ++s)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            uint32_t b0, b1;
            if (F8) {
              const uint32_t v = word_of(kr[s][t][st / 4], st % 4);
              b0 = e4m3x2_to_half2(v);
              b1 = e4m3x2_to_half2(v >> 16);
            } else {
              b0 = word_of(kr[s][t][st / 2], 2 * (st % 2));
              b1 = word_of(kr[s][t][st / 2], 2 * (st % 2) + 1);
            }
#pragma unroll
            for (int q = 0; q < kMT; ++q) mma16816<F8>(sc[q][s][t], a[q].x, a[q].y, a[q].z, a[q].w, b0, b1);
          }
      }
      load_k(row, k0 + S::kUnit);
      // scores in log2 units, keys past the end out
      float top[2 * kMT];
#pragma unroll
      for (int n = 0; n < 2 * kMT; ++n) top[n] = -INFINITY;
#pragma unroll
      for (int s = 0; s < S::kSub; ++s)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool in = k0 + 16 * s + 8 * t + 2 * c + (i & 1) < run.k1;
#pragma unroll
            for (int q = 0; q < kMT; ++q) {
              const float v = in ? sc[q][s][t][i] * qk_scale : -INFINITY;
              sc[q][s][t][i] = v;
              top[2 * q + (i >> 1)] = fmaxf(top[2 * q + (i >> 1)], v);
            }
          }
      bool grown = false;
#pragma unroll
      for (int n = 0; n < 2 * kMT; ++n) {
        top[n] = fmaxf(top[n], __shfl_xor_sync(0xffffffffu, top[n], 1));
        top[n] = fmaxf(top[n], __shfl_xor_sync(0xffffffffu, top[n], 2));
        grown |= top[n] > mx[n] + 8.f;
      }
      if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
        for (int n = 0; n < 2 * kMT; ++n) {
          const float mn = fmaxf(mx[n], top[n]);
          const float f = mx[n] == -INFINITY ? 0.f : ex2_approx(mx[n] - mn);
          mx[n] = mn;
          sum[n] *= f;
          const float f0 = __shfl_sync(0xffffffffu, f, 8 * c), f1 = __shfl_sync(0xffffffffu, f, 8 * c + 4);
#pragma unroll
          for (int m = 0; m < S::kSteps; ++m) {
            o[n][m][0] *= f0;
            o[n][m][1] *= f1;
            o[n][m][2] *= f0;
            o[n][m][3] *= f1;
          }
        }
      }
#pragma unroll
      for (int s = 0; s < S::kSub; ++s) {
        uint32_t b[2 * kMT][2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int n = 0; n < 2 * kMT; ++n) {
            const float ref = mx[n] == -INFINITY ? 0.f : mx[n];
            const float e0 = ex2_approx(sc[n >> 1][s][t][2 * (n & 1)] - ref);
            const float e1 = ex2_approx(sc[n >> 1][s][t][2 * (n & 1) + 1] - ref);
            sum[n] += e0 + e1;
            b[n][t] = F8 ? pack_half2(e0, e1) : pack_bf16x2(e0, e1);
          }
#pragma unroll
        for (int m = 0; m < S::kSteps; ++m) {
          uint32_t a[4];  // (element m, keys 2c..), (the upper element, keys 2c..), the same of keys 2c + 8..
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int lo = 2 * (i >> 1);                       // keys 2c, 2c+1 or 2c+8, 2c+9
            const int el = F8 ? m + 8 * (i & 1) : D == 64 ? m + 4 * (i & 1) : m;
            const int ch = (!F8 && D == 128) ? (i & 1) : 0;
            if (F8) {
              const uint32_t v = __byte_perm(word_of(vr[s][lo][ch], el / 4), word_of(vr[s][lo + 1][ch], el / 4),
                                             (el & 2) ? 0x7362 : 0x5140);
              a[i] = e4m3x2_to_half2((el & 1) ? v >> 16 : v);
            } else {
              a[i] = __byte_perm(word_of(vr[s][lo][ch], el / 2), word_of(vr[s][lo + 1][ch], el / 2),
                                 (el & 1) ? 0x7632 : 0x5410);
            }
          }
#pragma unroll
          for (int n = 0; n < 2 * kMT; ++n) mma16816<F8>(o[n][m], a[0], a[1], a[2], a[3], b[n][0], b[n][1]);
        }
      }
      load_v(row, k0 + S::kUnit);
#pragma unroll
      for (int s = 0; s < S::kSub; ++s) row[s] = row_at(k0 + 2 * S::kUnit + 16 * s);
    }
    // the warps' results, joined into the run's partial rows
#pragma unroll
    for (int n = 0; n < 2 * kMT; ++n) {
      sum[n] += __shfl_xor_sync(0xffffffffu, sum[n], 1);
      sum[n] += __shfl_xor_sync(0xffffffffu, sum[n], 2);
      if (c == 0) {
        sm[warp * kRows + g + 8 * n] = mx[n];
        sl[warp * kRows + g + 8 * n] = sum[n];
      }
    }
    // lane (g, c) holds rows 2c, 2c + 1 (+ 8 n) at elements 8 g + m (and the upper half's)
    constexpr int kRun = F8 ? 16 : 8;                         // contiguous elements of a lane
    constexpr int kUp = F8 ? 8 : D == 64 ? 4 : 64;            // from a tile's row g to its row g + 8
#pragma unroll
    for (int n = 0; n < 2 * kMT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float *dst = so + (warp * kRows + 8 * n + 2 * c + i) * D + kRun * g;
#pragma unroll
        for (int m = 0; m < S::kSteps; ++m) {
          dst[m] = o[n][m][i];
          dst[m + kUp] = o[n][m][2 + i];
        }
      }
    __syncthreads();
    for (int e = tid; e < kRows * D / 4; e += kMW * 32) {
      const int r = e / (D / 4), i = e - r * (D / 4);
      float m = sm[r];
#pragma unroll
      for (int k = 1; k < kMW; ++k) m = fmaxf(m, sm[k * kRows + r]);
      const float ref = m == -INFINITY ? 0.f : m;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.f;
#pragma unroll
      for (int k = 0; k < kMW; ++k) {
        const float f = ex2_approx(sm[k * kRows + r] - ref);
        const float4 v = *reinterpret_cast<const float4 *>(so + (k * kRows + r) * D + 4 * i);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
        l = fmaf(f, sl[k * kRows + r], l);
      }
      const size_t at = run.slot * kRows + r;
      *reinterpret_cast<float4 *>(p.part_o + at * D + 4 * i) = acc;
      if (i == 0) {
        p.part_ml[2 * at] = m;
        p.part_ml[2 * at + 1] = l;
      }
    }
  }
}

// float32, and bf16 head sizes of no tensor-core kernel: one warp per (token, query
// head): the tokens on its path, then the partial results of its history, then the
// output row and its log-sum-exp.
template <typename T>
__global__ void __launch_bounds__(256) draft_join_portable(const DraftParams p) {
  const flide_tree_index &x = p.x;
  if (failed(x.status)) return;
  const int lane = threadIdx.x & 31;
  const long long job = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int t = (int)(job / p.Hq), h = (int)(job % p.Hq);
  if (t >= x.counts[FLIDE_CNT_T]) return;
  const int hk = h / p.G, d = p.d, nd = d / 32;
  const int n = (int)checked(x.status, x.counts, x.token_node[t], x.counts[FLIDE_CNT_N], 801);
  const T *Q = static_cast<const T *>(p.q), *K = static_cast<const T *>(p.k), *Vs = static_cast<const T *>(p.v);
  const float qk_scale = p.scale * kLog2eD;
  float qv[8], acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    qv[i] = i < nd ? load_f(Q + ((size_t)t * p.Hq + h) * d + lane + 32 * i) * qk_scale : 0.f;
    acc[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int a = x.anc_ptr[n]; a < x.anc_ptr[n + 1]; ++a) {
    const int node = (int)checked(x.status, x.counts, x.anc_node[a], x.counts[FLIDE_CNT_N], 804);
    const int e = node == n ? t + 1 : x.node_start[node + 1];
    for (int j = x.node_start[node]; j < e; ++j) {
      const size_t at = ((size_t)j * p.Hkv + hk) * d + lane;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < nd) s = fmaf(qv[i], load_f(K + at + 32 * i), s);
      s = warp_sum(s);
      const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m - ref), w = exp2f(s - ref);
      l = l * f + w;
      m = mn;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < nd) acc[i] = fmaf(w, load_f(Vs + at + 32 * i), acc[i] * f);
    }
  }
  const DraftReq q = p.list[x.node_req[n]];
  if (q.units > 0) {
    const long long U = p.list[x.R].unit0;
    const int row = (t - q.t0) * p.G + h % p.G;
    const int li = row / p.tile_rows * p.Hkv + hk;
    const long long u0 = q.unit0 + (long long)li * q.units;
    const int W = workers_of(U, p.workers);
    const int w0 = worker_of(U, W, u0 + p.extra), w1 = worker_of(U, W, u0 + q.units - 1);
    for (int w = w0; w <= w1; ++w) {
      const size_t pr = (size_t)(w + q.item0 + li) * p.tile_rows + row % p.tile_rows;
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
  const float inv = 1.f / l;
  T *O = static_cast<T *>(p.out) + ((size_t)t * p.Hq + h) * d + lane;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < nd) store_f(O + 32 * i, acc[i] * inv);
  if (p.lse && lane == 0) p.lse[(size_t)t * p.Hq + h] = (m + log2f(l)) * kLn2D;
}

// D elements of type T as they lie for an 8-lane group: a lane's are kWords words
// of 16 bytes, word i at byte (8 i + lane) 16, so that a group reads whole rows.
template <typename T, int D>
struct Row8 {
  static constexpr int kE = D / 8;
  static constexpr int kW = 16 / sizeof(T);
  static constexpr int kWords = kE / kW;
  static __device__ __forceinline__ void load(const T *p, int l, uint4 (&w)[kWords]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = *reinterpret_cast<const uint4 *>(p + (8 * i + l) * kW);
  }
  static __device__ __forceinline__ void unpack(const uint4 (&w)[kWords], float (&v)[kE]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t u = word_of(w[i], j);
        float *o = v + i * kW + j * (kW / 4);
        if constexpr (sizeof(T) == 2) {
          o[0] = __uint_as_float(u << 16);
          o[1] = __uint_as_float(u & 0xffff0000u);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t pair = e4m3x2_to_half2(h ? u >> 16 : u);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&pair));
            o[2 * h] = f.x;
            o[2 * h + 1] = f.y;
          }
        }
      }
  }
  // element of v[e]
  static __device__ __forceinline__ int at(int e, int l) { return (8 * (e / kW) + l) * kW + e % kW; }
};

// bf16 and e4m3, d of 64 or 128: a warp is four groups of eight lanes, each with
// its own running (max, sum, O).  Few rows: a warp to a (token, query head), each
// group takes every fourth key of the token's path and every fourth partial of its
// history, joined by shuffles at the end.  Many rows: two or four heads of a
// group's K/V head to a warp, which list the path once and load its keys once.
// Bound by latency: five dependent loads stand before the path's first product and
// two before the first partial.  Starts beside the part kernel (programmatic
// launch) and waits for its results only where it needs them, so what counts is
// that all warps run at once.  1, 2, 4 heads to a warp, whole call: 80 rows of 16
// partials 14, 16, 18 us; 10240 rows 72, 64, 61; 16384 rows 312, 297, 291.  Half the
// registers and 32 warps to an SM spill (10240 rows: 68 us with four heads).
constexpr int kJoinWarps = 8;
constexpr int kPath = 64;  // keys of a path listed at a time

template <typename T, int D, int kHeads>
__global__ void __launch_bounds__(kJoinWarps * 32, 2) draft_join_kernel(const DraftParams p) {
  constexpr int kKeys = 4 / kHeads;  // groups that share a head's keys and partials
  using Row = Row8<T, D>;
  constexpr int kE = Row::kE;
  __shared__ int path_rows[kJoinWarps][kPath];
  const flide_tree_index &x = p.x;
  const int lane = threadIdx.x & 31, grp = (lane >> 3) / kHeads, l8 = lane & 7;
  int *path = path_rows[threadIdx.x >> 5];
  const unsigned job = blockIdx.x * kJoinWarps + (threadIdx.x >> 5), sets = (unsigned)p.Hq / kHeads;
  const int t = (int)(job / sets), h = (int)(job - t * sets) * kHeads + (lane >> 3) % kHeads, hk = h / p.G;
  const size_t head = (size_t)t * p.Hq + h;
  // what t alone addresses is loaded at once (the last block's rows past the capacity
  // take its last token's); a token past the stream's has no node
  const int tc = min(t, x.T - 1), node_of_t = x.token_node[tc];
  uint4 qw[Row::kWords];
  Row::load(static_cast<const T *>(p.q) + ((size_t)tc * p.Hq + h) * D, l8, qw);
  const int n_tokens = x.counts[FLIDE_CNT_T];
  const bool live = !failed(x.status) && t < n_tokens;
  float m = -INFINITY, l = 0.f, acc[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) acc[e] = 0.f;
  int r = 0;
  if (live) {
    const T *K = static_cast<const T *>(p.k), *Vs = static_cast<const T *>(p.v);
    const float qk_scale = p.scale * kLog2eD * (p.descale ? p.descale[0] * p.descale[1] : 1.f);
    const int n = (int)checked(x.status, x.counts, node_of_t, x.counts[FLIDE_CNT_N], 801);
    r = x.node_req[n];
    const int a1 = x.anc_ptr[n + 1];
    for (int a0 = x.anc_ptr[n]; a0 < a1; a0 += 32) {
      int first = 0, len = 0;  // this lane's ancestor: its keys
      if (a0 + lane < a1) {
        const int node = (int)checked(x.status, x.counts, x.anc_node[a0 + lane], x.counts[FLIDE_CNT_N], 804);
        first = x.node_start[node];
        len = (node == n ? t + 1 : x.node_start[node + 1]) - first;
      }
      const int end = warp_incl_scan(len), total = __shfl_sync(0xffffffffu, end, 31);
      for (int b0 = 0; b0 < total; b0 += kPath) {
        __syncwarp();
        for (int i = max(b0, end - len); i < min(b0 + kPath, end); ++i) path[i - b0] = first + i - (end - len);
        __syncwarp();
        const int cnt = min(kPath, total - b0);
        uint4 kw[Row::kWords], vw[Row::kWords];
        auto key_at = [&](int i, uint4 (&kn)[Row::kWords], uint4 (&vn)[Row::kWords]) {
          const int key = (int)checked(x.status, x.counts, path[i < cnt ? i : 0], x.counts[FLIDE_CNT_T], 805);
          const size_t at = ((size_t)key * p.Hkv + hk) * D;
          Row::load(K + at, l8, kn);
          Row::load(Vs + at, l8, vn);
        };
        if (kHeads > 1) key_at(grp, kw, vw);
        for (int k0 = 0; k0 < cnt; k0 += kKeys) {
          const bool on = k0 + grp < cnt;
          uint4 kn[Row::kWords], vn[Row::kWords];  // several heads: the next key's, a step ahead
          if (kHeads == 1) key_at(k0 + grp, kw, vw);
          else if (k0 + kKeys < cnt) key_at(k0 + kKeys + grp, kn, vn);
          float f[kE], s = 0.f;
          {
            float qv[kE];
            Row::unpack(qw, qv);
            Row::unpack(kw, f);
#pragma unroll
            for (int e = 0; e < kE; ++e) s = fmaf(qv[e], f[e], s);
          }
          s += __shfl_xor_sync(0xffffffffu, s, 1);
          s += __shfl_xor_sync(0xffffffffu, s, 2);
          s += __shfl_xor_sync(0xffffffffu, s, 4);
          if (on) {
            s *= qk_scale;
            const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
            const float o = ex2_approx(m - ref), w = ex2_approx(s - ref);
            l = l * o + w;
            m = mn;
            Row::unpack(vw, f);
#pragma unroll
            for (int e = 0; e < kE; ++e) acc[e] = fmaf(w, f[e], acc[e] * o);
          }
          if (kHeads > 1) {
#pragma unroll
            for (int i = 0; i < Row::kWords; ++i) {
              kw[i] = kn[i];
              vw[i] = vn[i];
            }
          }
        }
      }
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the part kernel's results
  const DraftReq q = p.list[r];  // (loaded beside the status word: a failed call's is not used)
  const long long U = p.list[x.R].unit0;
  if (!live || failed(x.status)) return;
  if (q.units > 0) {
    const int row = (t - q.t0) * p.G + h - hk * p.G;
    const int tile = row / p.tile_rows, li = tile * p.Hkv + hk;
    const long long u0 = q.unit0 + (long long)li * q.units;
    const int W = workers_of(U, p.workers);
    // the workers of the item's units with keys
    const int w0 = worker_of(U, W, u0 + p.extra), w1 = worker_of(U, W, u0 + q.units - 1);
    const int parts = (w1 - w0 + 1) << p.parts_log;
    const size_t pr0 = ((size_t)(w0 + q.item0 + li) << p.parts_log) * p.tile_rows + row - tile * p.tile_rows;
    auto partial = [&](int i, float2 &ml, float4 (&v)[kE / 4]) {
      const size_t pr = pr0 + (size_t)i * p.tile_rows;
      ml = *reinterpret_cast<const float2 *>(p.part_ml + 2 * pr);
#pragma unroll
      for (int e = 0; e < kE / 4; ++e)
        v[e] = *reinterpret_cast<const float4 *>(p.part_o + pr * D + Row::at(4 * e, l8));
    };
    float2 ml;
    float4 v[kE / 4];
    if (grp < parts) partial(grp, ml, v);
    for (int i = grp; i < parts; i += kKeys) {
      const float2 ml0 = ml;
      float4 v0[kE / 4];
#pragma unroll
      for (int e = 0; e < kE / 4; ++e) v0[e] = v[e];
      if (i + kKeys < parts) partial(i + kKeys, ml, v);
      if (ml0.x == -INFINITY && ml0.y == 0.f) continue;  // an empty partial (of NaN scores: not 0)
      const float mn = fmaxf(m, ml0.x);
      const float f = ex2_approx(m - mn), g = ex2_approx(ml0.x - mn);
      l = l * f + ml0.y * g;
      m = mn;
#pragma unroll
      for (int e = 0; e < kE / 4; ++e) {
        acc[4 * e] = fmaf(g, v0[e].x, acc[4 * e] * f);
        acc[4 * e + 1] = fmaf(g, v0[e].y, acc[4 * e + 1] * f);
        acc[4 * e + 2] = fmaf(g, v0[e].z, acc[4 * e + 2] * f);
        acc[4 * e + 3] = fmaf(g, v0[e].w, acc[4 * e + 3] * f);
      }
    }
  }
  // the results of a head's groups
  float mt = m;
#pragma unroll
  for (int o = 8 * kHeads; o < 32; o *= 2) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
  const float f = m == -INFINITY ? 0.f : ex2_approx(m - mt);
  l *= f;
#pragma unroll
  for (int o = 8 * kHeads; o < 32; o *= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = (p.descale ? p.descale[2] : 1.f) / l;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    acc[e] *= f;
#pragma unroll
    for (int o = 8 * kHeads; o < 32; o *= 2) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
    acc[e] *= inv;
  }
  // a group stores its share of its lanes' elements, four at a time
  __nv_bfloat16 *O = static_cast<__nv_bfloat16 *>(p.out) + head * D;
#pragma unroll
  for (int e = 0; e < kE; e += 4)
    if (e / 4 % kKeys == grp)
      *reinterpret_cast<uint2 *>(O + Row::at(e, l8)) =
          make_uint2(pack_bf16x2(acc[e], acc[e + 1]), pack_bf16x2(acc[e + 2], acc[e + 3]));
  if (p.lse && grp == 0 && l8 == 0) p.lse[head] = (mt + log2f(l)) * kLn2D;
}

// ---- host ----------------------------------------------------------------------

// Which part kernel.  The tcgen05 kernel, where it takes the type and head layout,
// with its smallest tile that holds a request's query rows on average (the
// capacities: the host sees no more; bf16 up to 256 rows, e4m3 128); elsewhere
// 16-row tiles or 32-row tiles, each a pass over the keys, on mma.sync.  One
// request's decoding, 4 rows a K/V head: 65536 rows of history 55 us in a 32-row
// tile, 74 in the 16-row kernel; 64 requests of 4096 rows 111 and 167; 512 rows 13
// and 11 (e4m3 65536: 44 and 49; 16 requests of 512: 18 and 15).  8 requests over
// 32768 rows, 64 rows to a head: 167 us in a 64-row tile, 187 in a 128-row tile, 272
// in a 256-row tile, 407 in 32-row tiles on mma.sync; 128 rows: 190 in a 128-row
// tile, 277 in a 256-row tile; 64 requests of 512 rows, 4 rows: 39 us in a 32-row
// tile, 42 in a 64-row tile.  Groups that do not divide the tile leave rows of it
// empty: 5 heads to a group, 24 tokens, 8 requests over 32768 rows 199 us, 804 in
// 32-row tiles on mma.sync.  Heads of 64: half the bytes of a key row, so up to 32
// rows the loads in registers win (8 requests over 32768 rows: 16 rows 105 us, 134 in
// a 64-row tile; 32 rows 117 and 134), beyond them the tile (64 rows 214 and 134, 256
// rows 820 and 251).  The tiles leave room for 1024 list entries, but for the 64-row
// one of 128-wide bf16 heads, whose merge buffer takes 34 KB of it: from 968 requests
// on the 128-row tile takes its rows.
enum Kernel { kPortable, kMma, kWide };
struct Variant {
  Kernel kernel;
  int tile_rows, parts_log;
  int operand = 0;  // kWide: rows of the operand, whole tokens of which are the tile's
};

Variant variant_of(long long R, long long T, int G, int d, int dtype) {
  if (dtype == FLIDE_F32 || (d != 64 && d != 128)) return {kPortable, 16, 0};
  const long long rows = (T * G + R - 1) / (R > 0 ? R : 1);
  if (G > 128 || R > 1024 || (d == 64 && rows <= 32)) return {kMma, rows <= 16 ? 16 : 32, 0};
  auto tile_of = [&](int operand) { return operand / G * G; };
  for (int operand : {32, 64, 128})
    if (G <= operand && (operand > 32 || d == 128) && (rows <= tile_of(operand) || (operand == 128 && dtype == FLIDE_E4M3)) &&
        draft_wide_fits(operand, d, dtype == FLIDE_E4M3, R))
      return {kWide, tile_of(operand), operand == 128, operand};
  return {kWide, 2 * tile_of(128), 0, 256};
}

constexpr int kMaxWorkers = 640;  // of any variant: what the workspace allows for
constexpr int kWideWorkers = 160; // of the wide ones, one to an SM

struct DraftSpace {
  size_t list, ml, o, total;
};

// Bytes of the workspace's parts: a slot for every worker and item.
DraftSpace draft_space(long long R, long long T, int Hkv, int G, int d, const Variant &v) {
  const long long slots = (v.kernel == kWide ? kWideWorkers : kMaxWorkers) +
                          ((T * G + v.tile_rows - 1) / v.tile_rows + R) * Hkv;
  const long long rows = (slots << v.parts_log) * v.tile_rows;
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  DraftSpace s;
  s.list = 0;
  s.ml = up((R + 1) * sizeof(DraftReq));
  s.o = s.ml + up((size_t)rows * 2 * sizeof(float));
  s.total = s.o + up((size_t)rows * d * sizeof(float));
  return s;
}

// Launches a part kernel on the workers with `smem` bytes of dynamic shared memory.
template <auto kKernel>
int part_launch(const DraftParams &p, int dev, int threads, size_t smem, cudaStream_t s) {
  if (!allow_smem<kKernel>(dev)) return FLIDE_ERR_CUDA;
  kKernel<<<p.workers, threads, smem, s>>>(p);
  FLIDE_LAUNCH_CHECK();
  return FLIDE_OK;
}

template <typename T>
int portable_launch(DraftParams &p, int dev, int sms, cudaStream_t s) {
  p.workers = min(kMaxWorkers, 4 * sms);
  p.unit = kPKeys;
  p.extra = 0;
  return part_launch<draft_part_portable<T>>(
      p, dev, kPT, (size_t)(p.x.R + 1) * sizeof(DraftReq) +
                       sizeof(float) * ((size_t)(kPRows + 2 * kPKeys) * (p.d + 4) + kPRows * kPKeys), s);
}

template <int D, bool F8, int kMT>
int mma_launch(DraftParams &p, int dev, int sms, cudaStream_t s) {
  using S = MmaShape<D, F8, kMT>;
  p.workers = min(kMaxWorkers, S::kBlocks * sms);
  p.unit = S::kUnit;
  p.extra = 0;
  return part_launch<draft_part_mma<D, F8, kMT>>(p, dev, S::kMW * 32, S::kSmem + (size_t)(p.x.R + 1) * sizeof(DraftReq), s);
}

template <typename T>
int join_portable_launch(const DraftParams &p, cudaStream_t s) {
  const long long warps = (long long)p.x.T * p.Hq;
  draft_join_portable<T><<<(unsigned)((warps + 7) / 8), 256, 0, s>>>(p);
  FLIDE_LAUNCH_CHECK();
  return FLIDE_OK;
}

template <typename T, int D, int kHeads>
int join_of(const DraftParams &p, cudaStream_t s) {
  const long long warps = (long long)p.x.T * (p.Hq / kHeads);
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((warps + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return launched(cudaLaunchKernelEx(&cfg, draft_join_kernel<T, D, kHeads>, p));
}

template <typename T, int D>
int join_launch(const DraftParams &p, int sms, cudaStream_t s) {
  const long long rows = (long long)p.x.T * p.Hq, at_once = 2ll * kJoinWarps * sms;
  // as many heads to a warp as it takes for all warps to run at once (16 to an SM); a
  // wave of them that starts after the part kernel repeats the path's loads behind it
  if (rows <= at_once || p.G % 2) return join_of<T, D, 1>(p, s);
  if (rows <= 2 * at_once || p.G % 4) return join_of<T, D, 2>(p, s);
  return join_of<T, D, 4>(p, s);
}

int draft_attn(const void *q, const void *k, const void *v, const void *past_k, const void *past_v,
               const HistoryView &hist, int past_rows, const flide_tree_index *idx, int Hq, int Hkv, int d, int dtype,
               const float *descale, float scale, void *out, float *lse, void *workspace,
               size_t workspace_bytes, cudaStream_t s) {
  if (!idx || !q || !k || !v || !out || !workspace) return FLIDE_ERR_SHAPE;
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv || d < 32 || d % 32 || d > 256) return FLIDE_ERR_SHAPE;
  if (dtype != FLIDE_F32 && dtype != FLIDE_BF16 && dtype != FLIDE_E4M3) return FLIDE_ERR_SHAPE;
  if (dtype == FLIDE_E4M3 && (!descale || d != 128)) return FLIDE_ERR_SHAPE;
  if (idx->R < 0 || idx->T < 0) return FLIDE_ERR_SHAPE;
  if ((uintptr_t)workspace % 256) return FLIDE_ERR_SHAPE;
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)past_k | (uintptr_t)past_v | (uintptr_t)out) % 16)
    return FLIDE_ERR_SHAPE;
  // a tile's largest score is scale times the largest product
  if (!(scale >= 0.f) || std::isinf(scale)) return FLIDE_ERR_INVALID;
  if (idx->R > kMaxListR || (long long)idx->T * Hq > 0x3fffffffLL) return FLIDE_ERR_CAPACITY;
  if (idx->R == 0 || idx->T == 0) return FLIDE_OK;
  const Variant var = variant_of(idx->R, idx->T, Hq / Hkv, d, dtype);
  const DraftSpace sp = draft_space(idx->R, idx->T, Hkv, Hq / Hkv, d, var);
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
  p.tile_rows = var.tile_rows;
  p.parts_log = var.parts_log;
  p.out = out;
  p.lse = lse;
  p.list = reinterpret_cast<DraftReq *>(ws + sp.list);
  p.part_ml = reinterpret_cast<float *>(ws + sp.ml);
  p.part_o = reinterpret_cast<float *>(ws + sp.o);
  int rc;
  if (var.kernel == kPortable) {
    rc = dtype == FLIDE_F32 ? portable_launch<float>(p, dev, sms, s) : portable_launch<__nv_bfloat16>(p, dev, sms, s);
    if (rc != FLIDE_OK) return rc;
    return dtype == FLIDE_F32 ? join_portable_launch<float>(p, s) : join_portable_launch<__nv_bfloat16>(p, s);
  }
  if (var.kernel == kWide) {
    p.workers = min(kWideWorkers, sms);
    rc = draft_wide_launch(p, var.operand, past_rows, dtype == FLIDE_E4M3, dev, s);
  } else if (var.tile_rows == 16) {
    rc = dtype == FLIDE_E4M3 ? mma_launch<128, true, 1>(p, dev, sms, s)
         : d == 128          ? mma_launch<128, false, 1>(p, dev, sms, s)
                             : mma_launch<64, false, 1>(p, dev, sms, s);
  } else {
    rc = dtype == FLIDE_E4M3 ? mma_launch<128, true, 2>(p, dev, sms, s)
         : d == 128          ? mma_launch<128, false, 2>(p, dev, sms, s)
                             : mma_launch<64, false, 2>(p, dev, sms, s);
  }
  if (rc != FLIDE_OK) return rc;
  if (dtype == FLIDE_E4M3) return join_launch<uint8_t, 128>(p, sms, s);
  return d == 128 ? join_launch<__nv_bfloat16, 128>(p, sms, s) : join_launch<__nv_bfloat16, 64>(p, sms, s);
}

}  // namespace
}  // namespace flide

extern "C" {

size_t flide_draft_attn_workspace_bytes(int32_t R, int32_t T, int32_t Hq, int32_t Hkv, int32_t d) {
  if (R < 0 || T < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || d <= 0) return 0;
  size_t most = 0;  // the element type, which chooses the kernel too, is not known here
  for (int dtype : {FLIDE_F32, FLIDE_BF16, FLIDE_E4M3})
    most = std::max(most, flide::draft_space(R, T, Hkv, Hq / Hkv, d,
                                             flide::variant_of(R, T, Hq / Hkv, d, dtype)).total);
  return most;
}

int flide_draft_attn(const void *q, const void *k, const void *v, const void *past_k,
                     const void *past_v, int32_t past_rows, const flide_tree_index *idx, int32_t Hq,
                     int32_t Hkv, int32_t d, int32_t dtype, const float *descale, float scale,
                     void *out, float *lse, void *workspace, size_t workspace_bytes,
                     flide_stream stream) {
  if (past_rows < 0 || (past_k == nullptr) != (past_v == nullptr)) return FLIDE_ERR_SHAPE;
  const flide::HistoryView h{nullptr, nullptr, 0, 0, 0, 0, past_k ? past_rows : 0};
  return flide::draft_attn(q, k, v, past_k, past_v, h, past_k ? past_rows : 0, idx, Hq, Hkv, d, dtype, descale, scale, out,
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
  if ((long long)n_blocks * block_rows > 0x7fffffffLL) return FLIDE_ERR_CAPACITY;
  const flide::HistoryView h{block_table, req_slot, max_blocks, block_rows, n_blocks, n_slots, 0};
  return flide::draft_attn(q, k, v, pool_k, pool_v, h, n_blocks * block_rows, idx, Hq, Hkv, d, dtype, descale, scale, out,
                           lse, workspace, workspace_bytes, (cudaStream_t)stream);
}

}  // extern "C"

// evict.cu -- which history rows were looked at, and dropping those that were
// not.
//
// flide_history_mass adds, for every history row i of a request, the attention
// weight that the step's root tokens (the tokens the step commits; drafted
// ones may still be rejected) gave it over all query heads:
//   mass_i += sum_{t in root} sum_h exp(scale q_th . k_i - lse_th),
// with lse as the step's attention wrote it, so the weights are final and no
// second softmax is needed.  The root's own rows, which enter the history with
// this step, start from what they received in it.  A block takes whole rows
// (all heads), so each sum has one writer and one order.
//
// flide_history_evict keeps `budget` rows of each longer history: the first
// `sinks`, the last `recent`, and the rows of largest mass between them (of
// equal ones the lowest index).  The kept rows stay in order and move to the
// front of the destination's blocks, in place if they are the source's.
#include <cmath>

#include "common.cuh"
#include "launch.cuh"
#include "sm100.cuh"
#include "worklist.cuh"

namespace flide {
namespace {

using namespace sm100;

constexpr float kLog2eM = 1.4426950408889634f;

struct MassParams {
  flide_tree_index x;
  HistoryView hist;
  const void *q, *k, *pool_k;
  const float *lse, *mass, *descale;
  float *mass_out;
  int Hq, Hkv, G, d;
  float scale;
  int held;  // query tiles in shared memory at a time (tensor-core kernel)
};

// Units of a request: its history rows and its root's rows, `unit` at a time
// each.  Requests without a slot have no history and take no part.
constexpr int kMKeys = 32;
constexpr int kMThreads = 128;

__device__ __forceinline__ int root_tokens(const flide_tree_index &x, int r, int *t0) {
  const int n0 = x.req_node[r], n1 = x.req_node[r + 1], N = x.counts[FLIDE_CNT_N];
  *t0 = 0;
  // debug build: the root lies among the tree's nodes, its tokens in the stream
  if (n1 <= n0 || !in_bounds(x.status, x.counts, n0, N, 811)) return 0;
  const int end = x.node_start[n0 + 1];
  if (!in_bounds(x.status, x.counts, end, x.counts[FLIDE_CNT_T] + 1ll, 812)) return 0;
  *t0 = x.node_start[n0];
  return end - *t0;
}

__device__ __forceinline__ long long mass_units(const MassParams &p, int r, int unit, bool report) {
  const flide_tree_index &x = p.x;
  const int slot = p.hist.req_slot[r];
  if (slot < 0) return 0;
  int t0;
  const int root = root_tokens(x, r, &t0), n = x.past_start[r + 1] - x.past_start[r];
  if (root == 0) return 0;
  if (slot >= p.hist.n_slots || n > kMaxHistory ||
      n + (long long)root > (long long)p.hist.max_blocks * p.hist.block_rows) {
    if (report) set_status(x.status, slot >= p.hist.n_slots ? FLIDE_ERR_INVALID : FLIDE_ERR_CAPACITY);
    return 0;
  }
  return (n + unit - 1) / unit + (root + unit - 1) / unit;
}

// float32, and head sizes of no tensor-core kernel: a lane per key, the heads and tokens split
// over the warps.
template <typename T>
__global__ void __launch_bounds__(kMThreads) mass_kernel_portable(const MassParams p) {
  extern __shared__ float smem[];
  __shared__ long long part[32];
  __shared__ float sums[kMThreads / 32][kMKeys];
  const flide_tree_index &x = p.x;
  if (failed(x.status)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = x.R, d = p.d, ld = d + 1;
  long long *unit0 = reinterpret_cast<long long *>(smem);
  float *sk = smem + 2 * (R + 1);
  request_prefix(R, [&](int r) { return mass_units(p, r, kMKeys, blockIdx.x == 0); }, unit0, part);
  const T *Q = static_cast<const T *>(p.q), *K = static_cast<const T *>(p.k),
          *Pk = static_cast<const T *>(p.pool_k);
  for (long long u = blockIdx.x; u < unit0[R]; u += gridDim.x) {
    const int r = request_of(unit0, R, u);
    int t0, slot;
    const int root = root_tokens(x, r, &t0);
    const int n = history_rows(x, p.hist, r, false, &slot);
    slot = p.hist.req_slot[r];
    const int past_units = (n + kMKeys - 1) / kMKeys;
    const int c = (int)(u - unit0[r]);
    const bool fresh = c >= past_units;
    const int k0 = (fresh ? c - past_units : c) * kMKeys;
    const int left = min(kMKeys, (fresh ? root : n) - k0);
    float acc = 0.f;
    for (int hk = 0; hk < p.Hkv; ++hk) {
      __syncthreads();
      for (int kr = warp; kr < left; kr += kMThreads / 32) {
        const long long row = fresh ? t0 + k0 + kr : history_row(x, p.hist, slot, k0 + kr);
        const T *src = (fresh ? K : Pk) + ((size_t)max(row, 0ll) * p.Hkv + hk) * d;
        for (int i = lane; i < d; i += 32) sk[kr * ld + i] = row >= 0 ? load_f(src + i) : 0.f;
      }
      __syncthreads();
      for (int j = warp; j < root * p.G; j += kMThreads / 32) {
        const int t = t0 + j / p.G, h = hk * p.G + j % p.G;
        const T *qr = Q + ((size_t)t * p.Hq + h) * d;
        float s = 0.f;
        if (lane < left)
          for (int i = 0; i < d; ++i) s = fmaf(load_f(qr + i), sk[lane * ld + i], s);
        if (lane < left && (!fresh || t0 + k0 + lane <= t))
          acc += exp2f((s * p.scale - p.lse[(size_t)t * p.Hq + h]) * kLog2eM);
      }
    }
    sums[warp][lane] = acc;
    __syncthreads();
    if (tid < left) {
      float all = 0.f;
#pragma unroll
      for (int w = 0; w < kMThreads / 32; ++w) all += sums[w][tid];
      const size_t at = (size_t)slot * p.hist.max_blocks * p.hist.block_rows + (fresh ? n : 0) + k0 + tid;
      p.mass_out[at] = fresh ? all : p.mass[at] + all;
    }
  }
}

// bf16 rows of 64 or 128 elements and e4m3 rows of 128, on the tensor cores.  A
// warp takes 16 history rows over all heads, so a row's sum over heads and
// tokens stays in one lane quad's registers: S^T = K Q^T with the 16 rows as the
// m16 operand and 8 query rows (tokens x heads of the group) as the n8 one, kept
// in shared memory as the raw 16-byte words that the lanes' k order asks for (see
// draft_attn.cu).
//
// Bound by K's bytes, and so by what is on its way: each lane copies the very
// words it will need to its own places in shared memory (8 KB a warp), a head or
// more ahead and past the end of a group of rows; no lane reads another's words,
// so nothing but the copies is waited for.  K leaves L2 before other lines: it is
// read once.  Blocks share the batch's groups of 16 rows evenly, a block's warps
// the (group, head) steps of its share; parts of a group are added in order at the
// end.  16 histories of 1024 to 16384 rows, 4 root tokens of 32 heads (238 MB):
// 48 us, 5.0 TB/s, of which 6 before the first product and 34 in the loop at 7
// TB/s.  8 warps an SM instead of 16: 14 us more; whole groups to a warp (four
// rounds where 3.1 would do) 5 more; the queries behind the ring's copies 5 more.
constexpr int kMassWarps = 16;
constexpr int kRing = 8192;  // bytes of a warp's ring
constexpr int kMassExtra = 5;  // groups that a block's start on a request costs beside its own (3 us of 0.7)

template <int D, bool F8>
struct MassShape {
  static constexpr int kRow = D * (F8 ? 1 : 2);
  static constexpr int kCj = kRow / 64;                     // a lane's 16-byte loads of a row
  static constexpr int kStages = kRing / (2 * kCj * 512);   // steps (16 rows of a head) of the ring
  static constexpr int kWords = kCj * (F8 ? 2 : 1);         // a lane's 16-byte words of an 8-row query tile
  static constexpr int kTileBytes = kWords * 32 * 16 + 32;  // and the tile's 8 lse
};

// A request in the list: its first group, its root's tokens, its history.
struct __align__(16) MassReq {
  long long group0;
  int t0, root, hist, slot;
};

__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src, bool on, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
               "r"(on ? 16 : 0), "l"(policy)
               : "memory");
}

__device__ __forceinline__ void copy_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <int D, bool F8>
__global__ void __launch_bounds__(kMassWarps * 32, 1) mass_kernel_mma(const MassParams p) {
  using S = MassShape<D, F8>;
  extern __shared__ uint4 qs[];  // [held][kWords][32], lse [held][8], the warps' rings, the list
  __shared__ long long part[32];
  __shared__ float edge[kMassWarps][2][16];  // sums of a warp's first and last group, where it has a part of it
  float *ls = reinterpret_cast<float *>(qs + p.held * S::kWords * 32);
  uint4 *rings = reinterpret_cast<uint4 *>(ls + p.held * 8);
  MassReq *list = reinterpret_cast<MassReq *>(rings + kMassWarps * (kRing / 16));
  const flide_tree_index &x = p.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3, R = x.R;
  if (__syncthreads_or(tid == 0 && failed(x.status))) return;
  {
    long long *group0 = &list[0].group0;  // every fourth 8-byte word of the list
    request_prefix(R, [&](int r) -> long long {
      MassReq &q = list[r];
      long long n = mass_units(p, r, 16, blockIdx.x == 0);
      if (n > 0) n += kMassExtra;
      q.root = root_tokens(x, r, &q.t0);
      int base;
      q.hist = history_rows(x, p.hist, r, false, &base);
      q.slot = p.hist.req_slot[r];
      return n;
    }, group0, part, sizeof(MassReq) / sizeof(long long));
  }
  const long long N = list[R].group0;
  const float qk_scale = p.scale * (F8 ? p.descale[0] * p.descale[1] : 1.f) * kLog2eM;
  uint4 *ring = rings + warp * (kRing / 16) + lane;
  const uint64_t once = policy_evict_first(), again = policy_evict_normal();
  long long u = blockIdx.x * N / gridDim.x;
  const long long u_end = (blockIdx.x + 1) * N / gridDim.x;
  while (u < u_end) {
    int r = 0;
    for (int hi = R; r < hi;) {
      const int mid = (r + hi) >> 1;
      if (list[mid + 1].group0 > u) hi = mid; else r = mid + 1;
    }
    const MassReq q = list[r];
    const int ua = (int)(u - q.group0), ub = (int)min(list[r + 1].group0 - q.group0, ua + (u_end - u));
    u += ub - ua;
    const int ga = max(ua - kMassExtra, 0), gb = ub - kMassExtra;
    if (gb <= ga) continue;
    const int past_groups = (q.hist + 15) / 16;
    const int rows = q.root * p.G, per = (rows + 7) / 8, tiles = p.Hkv * per;  // tile = head * per + row tile
    const uint64_t policy = tiles > p.held ? again : once;
    float *out = p.mass_out + (size_t)q.slot * p.hist.max_blocks * p.hist.block_rows;
    const float *in = p.mass + (size_t)q.slot * p.hist.max_blocks * p.hist.block_rows;
    for (int b0 = 0; b0 < tiles; b0 += p.held) {
      const int b1 = min(tiles, b0 + p.held), h0 = b0 / per, heads = (b1 - 1) / per - h0 + 1;
      // the pass's steps (group, head) are cut evenly over the warps; warp w takes
      // [step0(w), step0(w + 1)), and they go into its ring in order
      const long long steps = (long long)(gb - ga) * heads;
      auto step0 = [&](int w) -> long long { return steps * w / kMassWarps; };
      const long long s0 = step0(warp), s1 = step0(warp + 1);
      const int grp0 = ga + (int)(s0 / heads), hh0 = (int)(s0 % heads);
      // row of a group's first history row, or its first stream row; -1: no group
      auto row_of = [&](int grp) -> long long {
        if (grp >= gb) return -1;
        return grp < past_groups ? history_row(x, p.hist, q.slot, 16 * grp) : q.t0 + 16 * (grp - past_groups);
      };
      int ig = grp0, ih = hh0;  // the next step to copy: group, head (from h0)
      long long to_copy = s1 - s0;
      long long inext = row_of(ig);
      const char *src[2];          // its rows g and g + 8 (on: history or root has them)
      bool on[2];
      auto group = [&]() {
        const bool fresh = ig >= past_groups;
        const int left = (fresh ? q.root : q.hist) - 16 * (fresh ? ig - past_groups : ig);
        const char *base = static_cast<const char *>(fresh ? p.k : p.pool_k) + 16 * c + (size_t)h0 * S::kRow;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          on[t] = inext >= 0 && g + 8 * t < left;
          src[t] = base + (size_t)(on[t] ? inext + g + 8 * t : 0) * p.Hkv * S::kRow;
        }
        inext = row_of(ig + 1);  // looked up a group ahead
      };
      group();
      src[0] += (size_t)ih * S::kRow;
      src[1] += (size_t)ih * S::kRow;
      const uint32_t ring0 = smem_u32(ring);
      uint32_t to = ring0;         // the next stage
      auto copy = [&]() {
        if (to_copy > 0) {
          --to_copy;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < S::kCj; ++j)
              copy_async16(to + (t * S::kCj + j) * 512, src[t] + 64 * j, on[t], policy);
          src[0] += S::kRow;
          src[1] += S::kRow;
          to += 2 * S::kCj * 512;
          if (to == ring0 + S::kStages * 2 * S::kCj * 512) to = ring0;
          if (++ih == heads) {
            ih = 0;
            ++ig;
            group();
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      // the query tiles before the ring's first copies, which would keep them waiting
      // (the tiles held before are done with: the last pass ended in a barrier)
      auto tiles_words = [&](auto &&f) {
        for (int e = tid; e < (b1 - b0) * S::kCj * 32; e += kMassWarps * 32) {
          const int t = e / (S::kCj * 32), j = e / 32 % S::kCj, l = e & 31;
          const int h = (b0 + t) / per, qr = (b0 + t) % per * 8 + (l >> 2);
          const size_t at = (size_t)(q.t0 + qr / p.G) * p.Hq + h * p.G + qr % p.G;
          f(qs + (t * S::kWords + (F8 ? 2 : 1) * j) * 32 + l, j, l, qr < rows, qr < rows ? at : 0, ls + t * 8 + (l >> 2));
        }
      };
      tiles_words([&](uint4 *to, int j, int l, bool row, size_t at, float *lse_to) {
        copy_async16(smem_u32(to), static_cast<const char *>(p.q) + at * S::kRow + 64 * j + 16 * (l & 3), row, again);
        if (j == 0 && (l & 3) == 0) copy_async4(smem_u32(lse_to), p.lse + at);
      });
      asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll 1
      for (int k = 0; k < S::kStages - 1; ++k) copy();
      asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 1) : "memory");
      // what this thread copied, in its final form
      tiles_words([&](uint4 *to, int j, int l, bool row, size_t, float *lse_to) {
        if (F8) {
          const uint4 v = *to;
          to[0] = make_uint4(e4m3x2_to_half2(v.x), e4m3x2_to_half2(v.x >> 16), e4m3x2_to_half2(v.y),
                             e4m3x2_to_half2(v.y >> 16));
          to[32] = make_uint4(e4m3x2_to_half2(v.z), e4m3x2_to_half2(v.z >> 16), e4m3x2_to_half2(v.w),
                              e4m3x2_to_half2(v.w >> 16));
        }
        if (j == 0 && (l & 3) == 0) *lse_to *= kLog2eM;  // (a padding row's is not used)
      });
      __syncthreads();
      // place of row i of a group's 16 in the weights, -1: no such row
      auto place = [&](int grp, int i) -> int {
        const bool fresh = grp >= past_groups;
        i += 16 * (fresh ? grp - past_groups : grp);
        return i >= (fresh ? q.root : q.hist) ? -1 : (fresh ? q.hist : 0) + i;
      };
      // what this pass's sum is added to (a later batch of query tiles adds to the first
      // one's sum); loaded well before it is needed
      auto prior = [&](int grp, int at) -> float {
        return at < 0 ? 0.f : b0 > 0 ? out[at] : grp < past_groups ? in[at] : 0.f;
      };
      // the warp's last group, where other warps have parts of it and this one its first head
      const int cut = ga + (int)((s1 - 1) / heads);
      const long long end = (long long)(cut + 1 - ga) * heads;
      const bool owner = s1 > s0 && end > s1 && end - heads >= s0;
      const int cut_at = owner && lane < 16 ? place(cut, lane) : -1;
      const float cut_prior = prior(cut, cut_at);
      int st = 0, grp = grp0, first = hh0;
      for (long long s = s0; s < s1; ++grp, first = 0) {
        const bool fresh = grp >= past_groups;
        const int i0 = 16 * (fresh ? grp - past_groups : grp);
        const int last = (int)min((long long)heads, first + (s1 - s));
        s += last - first;
        float acc[2] = {0.f, 0.f};  // rows i0 + g, i0 + g + 8
        const bool whole = last - first == heads;
        int at[2];
        float was[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          at[t] = whole && c == 0 ? place(grp, g + 8 * t) : -1;
          was[t] = prior(grp, at[t]);
        }
        for (int hh = first; hh < last; ++hh) {
          asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 2) : "memory");
          uint4 kr[2][S::kCj];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < S::kCj; ++j) kr[t][j] = ring[((st * 2 + t) * S::kCj + j) * 32];
          if (++st == S::kStages) st = 0;
          copy();  // into the stage taken one step ago
          const int h = h0 + hh;
          // query tiles two at a time: two chains of products over the same rows
          const int t1 = min(b1, (h + 1) * per);
          for (int t = max(b0, h * per); t < t1; t += 2) {
            float s[2][4] = {};
            const uint4 *qt = qs + (t - b0) * S::kWords * 32 + lane;
            const int two = t + 1 < t1 ? S::kWords * 32 : 0;  // (a last odd tile twice, its second sum unused)
#pragma unroll
            for (int j = 0; j < S::kWords; ++j) {
              const uint4 q0 = qt[j * 32], q1 = qt[j * 32 + two];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                uint32_t a[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if (F8) {  // word 2 (j % 2) + i of load j / 2: its low and high code pairs
                    const uint32_t v = word_of(kr[k & 1][j / 2], 2 * (j % 2) + i);
                    a[k] = e4m3x2_to_half2(k >> 1 ? v >> 16 : v);
                  } else {
                    a[k] = word_of(kr[k & 1][j], 2 * i + (k >> 1));
                  }
                }
                mma16816<F8>(s[0], a[0], a[1], a[2], a[3], i ? q0.z : q0.x, i ? q0.w : q0.y);
                mma16816<F8>(s[1], a[0], a[1], a[2], a[3], i ? q1.z : q1.x, i ? q1.w : q1.y);
              }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              if (k && !two) break;
              const int r0 = (t + k - h * per) * 8 + 2 * c;
              const float2 l2 = *reinterpret_cast<const float2 *>(ls + (t + k - b0) * 8 + 2 * c);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float e = ex2_approx(fmaf(s[k][i], qk_scale, -(i & 1 ? l2.y : l2.x)));
                // a root row is seen by its own token and later ones; a padding row's score
                // is 0, or NaN with an infinite key
                if (r0 + (i & 1) >= rows || (fresh && (r0 + (i & 1)) / p.G < i0 + g + 8 * (i >> 1))) e = 0.f;
                acc[i >> 1] += e;
              }
            }
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], 1);
          acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], 2);
          if (at[t] >= 0) out[at[t]] = was[t] + acc[t];
          if (!whole && c == 0) edge[warp][first == 0][g + 8 * t] = acc[t];
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      // a group that several warps share: the warp with its first head adds their
      // sums, in order
      __syncthreads();
      if (cut_at >= 0) {
        float sum = edge[warp][1][lane];
        for (int w = warp + 1; w < kMassWarps && step0(w) < end; ++w)
          if (step0(w + 1) > step0(w)) sum += edge[w][0][lane];
        out[cut_at] = cut_prior + sum;
      }
    }
  }
}

template <int D, bool F8>
int mass_mma_launch(MassParams &p, int dev, int sms, cudaStream_t s) {
  using S = MassShape<D, F8>;
  if (!allow_smem<mass_kernel_mma<D, F8>>(dev)) return FLIDE_ERR_CUDA;
  // what the rings and the list (2048 requests: 64 KB) leave, for all query tiles
  // that a request may have if they fit
  const int fixed = kMassWarps * kRing + (p.x.R + 1) * (int)sizeof(MassReq);
  p.held = min((230000 - fixed) / S::kTileBytes, p.Hkv * (((int)min((long long)p.x.T * p.G, 1ll << 20) + 7) / 8));
  mass_kernel_mma<D, F8><<<sms, kMassWarps * 32, (size_t)fixed + p.held * S::kTileBytes, s>>>(p);
  FLIDE_LAUNCH_CHECK();
  return FLIDE_OK;
}

template <typename T>
int mass_launch(const MassParams &p, int dev, int sms, cudaStream_t s) {
  const size_t smem = (size_t)(p.x.R + 1) * 8 + sizeof(float) * kMKeys * (p.d + 1);
  if (!allow_smem<mass_kernel_portable<T>>(dev)) return FLIDE_ERR_CUDA;
  mass_kernel_portable<T><<<8 * sms, kMThreads, smem, s>>>(p);
  FLIDE_LAUNCH_CHECK();
  return FLIDE_OK;
}

// ---- eviction ------------------------------------------------------------------

struct EvictParams {
  int R, n_slots, n_blocks, dst_blocks, max_blocks, block_rows, budget, sinks, recent;
  const int32_t *req_slot, *hist_len, *table, *dst_table;
  const char *pool_k, *pool_v;
  char *dst_k, *dst_v;
  const float *mass;
  float *mass_out;
  int32_t *kept, *status;
  int row_bytes;
};

// Order-preserving code of a mass: NaN counts as the lowest, -0 as 0.
__device__ __forceinline__ uint32_t mass_code(float v) {
  if (!(v == v)) return 0u;
  const uint32_t b = __float_as_uint(v + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Rows of the history that request r has to be cut from, or -1 where the
// request is skipped (no slot) or refused (status set).
__device__ __forceinline__ int evict_length(const EvictParams &p, int r, bool report) {
  const int slot = p.req_slot[r];
  if (slot < 0) return -1;
  const int len = slot < p.n_slots ? p.hist_len[slot] : -1;
  if (len < 0 || len > (long long)p.max_blocks * p.block_rows) {
    if (report) set_status(p.status, FLIDE_ERR_INVALID);
    return -1;
  }
  return len;
}

constexpr int kMaxEvictR = 4096;  // each request looks through the others' slots
constexpr int kSelThreads = 1024;
constexpr int kBits = 11;  // 3 passes over 32-bit codes
constexpr int kBins = 1 << kBits;

// One block per request: the code of the smallest kept mass by radix selection
// over the rows between sinks and recent, then the kept rows in order.  A thread
// has kEach neighbouring rows of a chunk, so one scan places a whole chunk; the
// first chunk is read once and stays in registers for all passes (longer histories
// read the others again).  The kept rows are gathered in shared memory and stored
// from there: a thread's own stores lie kEach rows apart, a line each, and took
// most of 21 us for 16384 rows.
template <int kEach>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  constexpr int kChunk = kEach * kSelThreads;
  extern __shared__ int kept_s[];  // [kChunk], then their masses
  float *mass_s = reinterpret_cast<float *>(kept_s + kChunk);
  __shared__ int hist[kBins];
  __shared__ int scratch[40];
  __shared__ int s_dup, s_bin, s_left;
  const int r = blockIdx.x, tid = threadIdx.x;
  const int len = evict_length(p, r, tid == 0);
  int32_t *kept = p.kept + (size_t)r * p.budget;
  if (tid == 0) s_dup = 0;
  __syncthreads();
  if (len >= 0) {  // a slot twice in one call would be moved twice
    for (int i = tid; i < p.R; i += kSelThreads)
      if (i != r && p.req_slot[i] == p.req_slot[r]) s_dup = 1;
  }
  __syncthreads();
  if (len < 0 || s_dup) {
    if (s_dup && tid == 0) set_status(p.status, FLIDE_ERR_INVALID);
    for (int j = tid; j < p.budget; j += kSelThreads) kept[j] = -1;
    return;
  }
  const size_t at = (size_t)p.req_slot[r] * p.max_blocks * p.block_rows;
  const float *mass = p.mass + at;
  float *mass_out = p.mass_out + at;
  float v[kEach];
  auto load = [&](int base) {
    const int i0 = base + kEach * tid;
    if (i0 + kEach <= len && (at & 3) == 0 && ((uintptr_t)p.mass & 15) == 0) {
#pragma unroll
      for (int k = 0; k < kEach; k += 4) *reinterpret_cast<float4 *>(v + k) = *reinterpret_cast<const float4 *>(mass + i0 + k);
    } else {
#pragma unroll
      for (int k = 0; k < kEach; ++k) v[k] = i0 + k < len ? mass[i0 + k] : 0.f;
    }
  };
  load(0);
  const bool one = len <= kChunk, all = len <= p.budget;
  const int lo = all ? 0 : p.sinks, hi = all ? 0 : len - p.recent;  // candidates
  int want = all ? 0 : p.budget - p.sinks - p.recent;
  const bool any = want > 0;
  uint32_t prefix = 0, mask = 0;  // codes still in question: (code & mask) == prefix
  if (any) {
    for (int shift = 32 - kBits; ; shift = max(0, shift - kBits)) {
      const uint32_t bins = mask == 0 || shift > 0 ? kBins : 1u << (32 - 2 * kBits);
      for (int b = tid; b < kBins; b += kSelThreads) hist[b] = 0;
      __syncthreads();
      for (int base = 0; base < len; base += kChunk) {
        if (!one) load(base);
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
          const int i = base + kEach * tid + k;
          const uint32_t c = mass_code(v[k]);
          if (i >= lo && i < hi && (c & mask) == prefix) atomicAdd(&hist[(c >> shift) & (bins - 1)], 1);
        }
      }
      __syncthreads();
      // bins from the top: thread b holds bins kBins-1-2b and kBins-2-2b
      const int b0 = kBins - 1 - 2 * tid, h0 = hist[b0], h1 = hist[b0 - 1];
      int tot;
      const int before = block_excl_scan(h0 + h1, scratch, &tot);
      if (before < want && before + h0 >= want) {
        s_bin = b0;
        s_left = want - before;
      } else if (before + h0 < want && before + h0 + h1 >= want) {
        s_bin = b0 - 1;
        s_left = want - before - h0;
      }
      __syncthreads();
      want = s_left;  // of the chosen bin's rows
      prefix |= (uint32_t)s_bin << shift;
      mask |= (bins - 1) << shift;
      if (shift == 0) break;
    }
  }
  // rows above the threshold, the first `want` at it, and the fixed ones: row i
  // goes to (sure rows before it) + min(ties before it, want), so one scan of
  // both counts places a chunk.  A chunk's masses are read before its scan and
  // written after it, to places not past them: in place works.
  int out = 0, ties = 0;
  for (int base = 0; base < len; base += kChunk) {
    if (!one) load(base);
    const int i0 = base + kEach * tid;
    uint32_t sure = 0, tie = 0;  // bit k: row i0 + k
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int i = i0 + k;
      if (i >= len) continue;
      const uint32_t c = mass_code(v[k]);
      if (all || i < lo || i >= hi || (any && c > prefix)) sure |= 1u << k;
      else if (any && c == prefix) tie |= 1u << k;
    }
    int tot;
    const int before = block_excl_scan(__popc(sure) | __popc(tie) << 16, scratch, &tot);
    const int first = out + min(ties, want);  // the chunk's first place
    int s = out + (before & 0xffff), e = ties + (before >> 16);
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const bool even = tie >> k & 1;
      if ((sure >> k & 1) || (even && e < want)) {
        const int j = s + min(e, want) - first;
        kept_s[j] = i0 + k;
        mass_s[j] = v[k];
      }
      s += sure >> k & 1;
      e += even;
    }
    out += tot & 0xffff;
    ties += tot >> 16;
    const int n = out + min(ties, want) - first;
    __syncthreads();
    for (int j = tid; j < n; j += kSelThreads) {
      kept[first + j] = kept_s[j];
      mass_out[first + j] = mass_s[j];
    }
    __syncthreads();
  }
  out += min(ties, want);
  for (int j = out + tid; j < p.budget; j += kSelThreads) kept[j] = -1;
}

constexpr int kMoveThreads = 256;
constexpr int kUnroll = 8;  // 16-byte words in flight per thread

// Pool rows that history row i is at (in block sb) and row j goes to (in block
// db); false (status set, *to -1) without blocks.
__device__ __forceinline__ bool move_rows(const EvictParams &p, int sb, int db, int i, int j, int *from, int *to) {
  *from = *to = -1;
  if (sb < 0 || sb >= p.n_blocks || db < 0 || db >= p.dst_blocks) {
    set_status(p.status, FLIDE_ERR_INVALID);
    return false;
  }
  *from = sb * p.block_rows + i % p.block_rows;
  *to = db * p.block_rows + j % p.block_rows;
  return true;
}

// Within a pool.  Block (slice, request) moves `slice` bytes of every kept row,
// front to back: a row never moves past one that is still to be read (kept is
// ascending and kept[j] >= j), so in one block order is all that in-place
// movement needs.  A chunk of rows is stored after the barrier that follows its
// loads; the next chunk's loads, which no earlier store can touch, and the rows of
// the one after it are on their way meanwhile.  16 histories cut from 16384 to
// 8192 rows of 4 KB: 281 us, 3.8 TB/s; in turn, with a row found by each of its
// lanes, 529 us.  One history of 131072 rows cut to half: 1.4 TB/s, all that 128
// blocks have on their way.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p, int slice) {
  extern __shared__ int row_from[];
  const int r = blockIdx.y, tid = threadIdx.x;
  const int len = evict_length(p, r, false);
  if (len < 0) return;
  const int32_t *kept = p.kept + (size_t)r * p.budget;
  const int n = min(len, p.budget);
  const int slices = (p.row_bytes + slice - 1) / slice, lanes = slice / 16, rows = kMoveThreads / lanes;
  const bool is_v = (int)blockIdx.x >= slices;
  const int off = (is_v ? blockIdx.x - slices : blockIdx.x) * slice + (tid % lanes) * 16;
  const char *src = (is_v ? p.pool_v : p.pool_k) + off;
  char *dst = (is_v ? p.dst_v : p.dst_k) + off;
  const bool same = (is_v ? p.pool_v : p.pool_k) == (is_v ? p.dst_v : p.dst_k);
  const size_t slot = p.req_slot[r];
  const int32_t *st = p.table + slot * p.max_blocks, *dt = p.dst_table + slot * p.max_blocks;
  if (n == 0 || kept[0] < 0) return;  // (refused by the selection: a slot twice)
  const int mine = tid / lanes, step = rows * kUnroll;
  int *row_to = row_from + 4 * step;
  // a chunk's rows, found once for all lanes: where they are and where they go
  // (-1: nothing to move), for the chunks c to c + 3 at (c % 4) step
  auto find = [&](int c) {
    // (four rows a thread at most, their loads together)
    int i[4], sb[4], db[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = tid + k * kMoveThreads, j = c * step + e;
      i[k] = e < step && j < n ? kept[j] : -1;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i[k] < 0) continue;
      sb[k] = st[i[k] / p.block_rows];
      db[k] = dt[(c * step + tid + k * kMoveThreads) / p.block_rows];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = tid + k * kMoveThreads;
      if (e >= step) continue;
      int a = -1, b = -1;
      if (i[k] >= 0 && move_rows(p, sb[k], db[k], i[k], c * step + e, &a, &b) && same && a == b) b = -1;
      row_from[(c & 3) * step + e] = a;
      row_to[(c & 3) * step + e] = b;
    }
  };
  uint4 v[2][kUnroll];
  const bool live = off < p.row_bytes;
  auto load = [&](int c, uint4 (&w)[kUnroll]) {
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int e = (c & 3) * step + k * rows + mine;
      if (live && row_to[e] >= 0) w[k] = *reinterpret_cast<const uint4 *>(src + (size_t)row_from[e] * p.row_bytes);
    }
  };
  find(0);
  find(1);
  __syncthreads();
  load(0, v[0]);
  for (int c = 0; c * step < n; c += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load(c + h + 1, v[h ^ 1]);
      find(c + h + 2);
      __syncthreads();  // every thread's loads of chunk c + h are done
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int e = ((c + h) & 3) * step + k * rows + mine;
        if (live && row_to[e] >= 0) *reinterpret_cast<uint4 *>(dst + (size_t)row_to[e] * p.row_bytes) = v[h][k];
      }
    }
  }
}

// Between pools nothing is overwritten: warps copy whole rows in any order.
__global__ void __launch_bounds__(kMoveThreads) evict_copy_kernel(const EvictParams p) {
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.y;
  const int len = evict_length(p, r, false);
  if (len < 0) return;
  const int32_t *kept = p.kept + (size_t)r * p.budget;
  const int n = min(len, p.budget);
  if (n > 0 && kept[0] < 0) return;
  const size_t slot = p.req_slot[r];
  const int32_t *st = p.table + slot * p.max_blocks, *dt = p.dst_table + slot * p.max_blocks;
  const int warps = gridDim.x * (kMoveThreads / 32);
  const int words = p.row_bytes / 16;  // of a K row; its V row's follow
  for (int j = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); j < n; j += warps) {
    int from, to;
    const int i = kept[j];
    if (!move_rows(p, st[i / p.block_rows], dt[j / p.block_rows], i, j, &from, &to)) continue;
    const size_t a = (size_t)from * p.row_bytes, b = (size_t)to * p.row_bytes;
    for (int w0 = lane; w0 < 2 * words; w0 += 32 * kUnroll) {
      uint4 v[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int w = w0 + 32 * k;
        if (w < 2 * words)
          v[k] = ld_stream((w < words ? p.pool_k : p.pool_v) + a + 16 * (size_t)(w < words ? w : w - words));
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int w = w0 + 32 * k;
        if (w < 2 * words)
          *reinterpret_cast<uint4 *>((w < words ? p.dst_k : p.dst_v) + b + 16 * (size_t)(w < words ? w : w - words)) = v[k];
      }
    }
  }
}

}  // namespace
}  // namespace flide

extern "C" {

int flide_history_mass(const void *q, const void *k, const float *lse, const void *pool_k,
                       int32_t n_blocks, int32_t block_rows, const int32_t *block_table,
                       int32_t max_blocks, const int32_t *req_slot, int32_t n_slots,
                       const flide_tree_index *idx, int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype,
                       const float *descale, float scale, const float *mass, float *mass_out,
                       flide_stream stream) {
  using namespace flide;
  if (!idx || !q || !k || !lse || !pool_k || !block_table || !req_slot || !mass || !mass_out)
    return FLIDE_ERR_SHAPE;
  if (n_blocks <= 0 || max_blocks <= 0 || n_slots <= 0 || block_rows <= 0 || block_rows % 16)
    return FLIDE_ERR_SHAPE;
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv || d < 32 || d % 32 || d > 256) return FLIDE_ERR_SHAPE;
  if (dtype != FLIDE_F32 && dtype != FLIDE_BF16 && dtype != FLIDE_E4M3) return FLIDE_ERR_SHAPE;
  if (dtype == FLIDE_E4M3 && (!descale || d != 128)) return FLIDE_ERR_SHAPE;
  if (idx->R < 0 || idx->T < 0) return FLIDE_ERR_SHAPE;
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)pool_k) % 16) return FLIDE_ERR_SHAPE;
  // (in place, a weight of NaN would stay)
  if (!(scale >= 0.f) || std::isinf(scale)) return FLIDE_ERR_INVALID;
  if (idx->R > kMaxListR || (long long)idx->T * Hq > 0x3fffffffLL || (long long)n_blocks * block_rows > 0x7fffffffLL)
    return FLIDE_ERR_CAPACITY;
  if (idx->R == 0 || idx->T == 0) return FLIDE_OK;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FLIDE_ERR_CUDA;
  MassParams p;
  p.x = *idx;
  p.hist = HistoryView{block_table, req_slot, max_blocks, block_rows, n_blocks, n_slots, 0};
  p.q = q;
  p.k = k;
  p.pool_k = pool_k;
  p.lse = lse;
  p.mass = mass;
  p.mass_out = mass_out;
  p.descale = dtype == FLIDE_E4M3 ? descale : nullptr;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.d = d;
  p.scale = scale;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == FLIDE_F32) return mass_launch<float>(p, dev, sms, s);
  if (dtype == FLIDE_E4M3) return mass_mma_launch<128, true>(p, dev, sms, s);
  if (d == 128) return mass_mma_launch<128, false>(p, dev, sms, s);
  if (d == 64) return mass_mma_launch<64, false>(p, dev, sms, s);
  return mass_launch<__nv_bfloat16>(p, dev, sms, s);
}

int flide_history_evict(int32_t R, const int32_t *req_slot, int32_t n_slots, const int32_t *hist_len,
                        const int32_t *block_table, int32_t max_blocks, int32_t block_rows,
                        const void *pool_k, const void *pool_v, int32_t n_blocks, int32_t Hkv,
                        int32_t d, int32_t dtype, const float *mass, int32_t budget, int32_t sinks,
                        int32_t recent, void *dst_k, void *dst_v, const int32_t *dst_table,
                        int32_t dst_blocks, float *mass_out, int32_t *kept, int32_t *status,
                        flide_stream stream) {
  using namespace flide;
  if (!req_slot || !hist_len || !block_table || !pool_k || !pool_v || !mass || !dst_k || !dst_v ||
      !dst_table || !mass_out || !kept || !status)
    return FLIDE_ERR_SHAPE;
  if (R < 0 || n_slots <= 0 || max_blocks <= 0 || block_rows <= 0 || n_blocks <= 0 || dst_blocks <= 0 ||
      Hkv <= 0 || d <= 0)
    return FLIDE_ERR_SHAPE;
  if (budget <= 0 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget) return FLIDE_ERR_SHAPE;
  const int es = dtype == FLIDE_BF16 ? 2 : dtype == FLIDE_F32 ? 4 : dtype == FLIDE_E4M3 ? 1 : 0;
  if (!es) return FLIDE_ERR_SHAPE;
  const int64_t row_bytes = (int64_t)Hkv * d * es;
  if (row_bytes % 16 || row_bytes > (1 << 20)) return FLIDE_ERR_SHAPE;
  if (((uintptr_t)pool_k | (uintptr_t)pool_v | (uintptr_t)dst_k | (uintptr_t)dst_v) % 16) return FLIDE_ERR_SHAPE;
  if (R > kMaxEvictR || (int64_t)max_blocks * block_rows > kMaxHistory ||
      (int64_t)n_blocks * block_rows > INT32_MAX || (int64_t)dst_blocks * block_rows > INT32_MAX)
    return FLIDE_ERR_CAPACITY;
  if (R == 0) return FLIDE_OK;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FLIDE_ERR_CUDA;
  EvictParams p;
  p.R = R;
  p.n_slots = n_slots;
  p.n_blocks = n_blocks;
  p.dst_blocks = dst_blocks;
  p.max_blocks = max_blocks;
  p.block_rows = block_rows;
  p.budget = budget;
  p.sinks = sinks;
  p.recent = recent;
  p.req_slot = req_slot;
  p.hist_len = hist_len;
  p.table = block_table;
  p.dst_table = dst_table;
  p.pool_k = static_cast<const char *>(pool_k);
  p.pool_v = static_cast<const char *>(pool_v);
  p.dst_k = static_cast<char *>(dst_k);
  p.dst_v = static_cast<char *>(dst_v);
  p.mass = mass;
  p.mass_out = mass_out;
  p.kept = kept;
  p.status = status;
  p.row_bytes = (int)row_bytes;
  cudaStream_t s = (cudaStream_t)stream;
  // few rows a thread for short histories: 4 of 4096 (2304 rows: 8 us, with 16 of
  // 16384 13 us)
  if ((int64_t)max_blocks * block_rows <= 4 * kSelThreads) {
    evict_select_kernel<4><<<R, kSelThreads, 8 * 4 * kSelThreads, s>>>(p);
  } else {
    if (!allow_smem<evict_select_kernel<16>>(dev)) return FLIDE_ERR_CUDA;
    evict_select_kernel<16><<<R, kSelThreads, 8 * 16 * kSelThreads, s>>>(p);
  }
  FLIDE_LAUNCH_CHECK();
  if (dst_k != pool_k && dst_v != pool_v) {
    const unsigned blocks = (unsigned)min(((int64_t)budget + 7) / 8, max((int64_t)1, (int64_t)16 * sms / R));
    evict_copy_kernel<<<dim3(blocks, R), kMoveThreads, 0, s>>>(p);
  } else {
    // wide slices read and write DRAM in longer runs, narrow ones give a small
    // batch enough blocks
    int slice = 256;
    while (slice > 32 && 2 * ((row_bytes + slice - 1) / slice) * R < 2 * sms) slice /= 2;
    const unsigned slices = (unsigned)((row_bytes + slice - 1) / slice);
    const size_t smem = 2 * 4 * sizeof(int) * kUnroll * (kMoveThreads / (slice / 16));
    if (!allow_smem<evict_move_kernel>(dev)) return FLIDE_ERR_CUDA;
    evict_move_kernel<<<dim3(2 * slices, R), kMoveThreads, smem, s>>>(p, slice);
  }
  FLIDE_LAUNCH_CHECK();
  return FLIDE_OK;
}

}  // extern "C"

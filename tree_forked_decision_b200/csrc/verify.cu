// verify.cu -- verification of a drafted tree against the target's
// probabilities, with the random numbers given.
//
// The walk starts at a request's last root token.  At a token with target row
// p and, where the drafted tokens were sampled, draft row q, its drafted
// continuations (the next token of its node, or the first tokens of its
// node's children in stream order) are tried in turn.  After i rejections the
// target's distribution is the residual
//   r_0 = p,  r_i = (r_{i-1} - q)+ / sum (r_{i-1} - q)+,
// and x, with its random number u, is accepted when u < r_i(x) / q(x).  Every
// r_i has the form (p - c_i q)+ / D_i:
//   c_0 = 0, D_0 = 1;  c_i = c_{i-1} + D_{i-1},  D_i = sum_v (p - c_i q)+ ,
// so a rejection costs one pass over the two rows and no row is written.
// Without q the drafted tokens are point masses: x is accepted when
// u D < p(x) with D = 1 - (the rejected tokens' p), and a rejected token's p
// becomes 0.  Where no continuation is left, the next token is drawn from the
// residual by inverse CDF.  All of this is in 64 bits, so a decision does not
// hang on the order of a sum.
//
// A cluster of 8 (or 16) blocks walks one request: every block takes its part of
// the vocabulary in each pass and repeats the walk's decisions from the same
// numbers (sums are exchanged through distributed shared memory in a fixed
// order).  Bound by latency: of the walk's dependent loads for one tree (8192
// point masses: 9 us), of the passes of the tree that rejects most for a batch
// (64 sampled trees, 131072 entries: 43 us; every tree's first pass ends after 11 to
// 18 us, the last trees take 6 to 7 for each further one).
#include <cooperative_groups.h>

#include "common.cuh"
#include "launch.cuh"

namespace cg = cooperative_groups;

namespace flide {
namespace {

constexpr int kVThreads = 256;  // four blocks to an SM: 74 trees at a time
constexpr int kVWarps = kVThreads / 32;
constexpr int kMaxNodes = 4096;  // nodes of one request
constexpr int kMaxKids = 1024;   // continuations of one token
constexpr int kMaxSegs = 1024;   // inverse-CDF segments of a block's slice

struct VerifyParams {
  flide_tree_index x;
  const int32_t *tokens;
  const void *target, *draft;
  const float *u, *u_next;
  int V;
  int32_t *n_accept, *next_token, *path;
};

// entries of a probability row as non-negative 64-bit values; what is not a
// positive number counts as 0
__device__ __forceinline__ double prob_of(float v) { return v > 0.f ? (double)v : 0.; }

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// prob_of(v) 2^-896: the float's bits moved to where a double has them, subnormal
// numbers too.  A pass converts two entries of every kind of token, and the
// conversion instruction has a sixteenth of the shifts' rate.
__device__ __forceinline__ double small_prob(float v) {
  const uint32_t b = __float_as_uint(fmaxf(v, 0.f));  // (of NaN and 0: 0; of -0 and 0: 0)
  return __hiloint2double((int)(b >> 3), (int)(b << 29));
}
// x where it is positive, else 0; x is a number
__device__ __forceinline__ double positive_part(double x) {
  const int keep = ~(__double2hiint(x) >> 31);
  return __hiloint2double(__double2hiint(x) & keep, __double2loint(x) & keep);
}

template <int k>
struct Kind {
  static constexpr int value = k;
};

constexpr int kHeld = 512;  // branch tokens whose candidates are looked up beforehand

struct VerifyShared {
  int start[kMaxNodes + 1];     // first stream row of each node (and the end)
  int16_t parent[kMaxNodes];    // request-local parent of each node
  int tok[kHeld];               // a drafted token, its random number and its
  float u[kHeld], px[kHeld], qx[kHeld];  // probabilities at the token before it
  int kid_token[kMaxKids];
  double seg[kMaxSegs];
  double warp[kVWarps];
  double total[2][16];    // the blocks' parts of a sum, by parity of the exchange
  int stop;
};

// Entries v .. v + 3 of a row (0 past `end`); kVec: rows are whole 4-entry words.
template <typename T, bool kVec>
__device__ __forceinline__ float4 load4(const T *row, int v, int end) {
  if constexpr (kVec && sizeof(T) == 4) {
    return v < end ? __ldg(reinterpret_cast<const float4 *>(row + v)) : make_float4(0.f, 0.f, 0.f, 0.f);
  } else if constexpr (kVec) {
    const uint2 w = v < end ? __ldg(reinterpret_cast<const uint2 *>(row + v)) : make_uint2(0u, 0u);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
  } else {
    return make_float4(v < end ? load_f(row + v) : 0.f, v + 1 < end ? load_f(row + v + 1) : 0.f,
                       v + 2 < end ? load_f(row + v + 2) : 0.f, v + 3 < end ? load_f(row + v + 3) : 0.f);
  }
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kVThreads, 4)
verify_kernel(const VerifyParams p) {
  __shared__ VerifyShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const flide_tree_index &x = p.x;
  const int rank = (int)cluster.block_rank(), blocks = (int)cluster.num_blocks();
  const int r = blockIdx.x / blocks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the status word may change while this kernel runs (another cluster's bad
  // token), so one block's reading decides for its whole cluster
  if (tid == 0) sh.stop = failed(x.status);
  cluster.sync();
  bool stop = *cluster.map_shared_rank(&sh.stop, 0) != 0;
  // debug build: the request's nodes lie among the tree's (the same finding in every block)
  const int N = stop ? 0 : x.counts[FLIDE_CNT_N];
  int n0 = stop ? 0 : x.req_node[r], n1 = stop ? 0 : x.req_node[r + 1];
  if (!in_bounds(x.status, x.counts, n0, N + 1, 901) || !in_bounds(x.status, x.counts, n1, N + 1, 901)) n0 = n1 = 0;
  const int first = n1 > n0 ? x.node_start[n0] : 0, end = n1 > n0 ? x.node_start[n1] : 0;
  const int nn = n1 - n0;
  if (rank == 0 && !stop)
    for (int t = first + tid; t < end; t += kVThreads) p.path[t] = -1;
  if (stop || nn <= 0 || x.node_start[n0 + 1] == first || nn > kMaxNodes) {
    if (!stop && rank == 0 && tid == 0) {
      if (nn > kMaxNodes) set_status(x.status, FLIDE_ERR_CAPACITY);
      p.n_accept[r] = 0;
      p.next_token[r] = -1;
    }
    cluster.sync();  // block 0's flag has been read
    return;
  }
  for (int i = tid; i <= nn; i += kVThreads) {
    sh.start[i] = x.node_start[n0 + i];
    if (i < nn)
      sh.parent[i] = (int16_t)(i == 0 ? -1 : checked(x.status, x.counts, x.anc_node[x.anc_ptr[n0 + i + 1] - 2] - n0, i, 902));
  }
  __syncthreads();

  const T *P = static_cast<const T *>(p.target), *Q = static_cast<const T *>(p.draft);
  const bool sampled = Q != nullptr;
  const int V = p.V;
  // this block's slice and its segments (contiguous, at most kMaxSegs)
  const int slice = ((V + blocks - 1) / blocks + 127) / 128 * 128;
  const int v_lo = min(V, rank * slice), v_hi = min(V, v_lo + slice);
  const int seg_len = max(128, ((slice + kMaxSegs - 1) / kMaxSegs + 127) / 128 * 128);
  const int n_seg = (v_hi - v_lo + seg_len - 1) / seg_len;

  // what a walk can ask of the drafted tokens, all at once: a walk that loads it
  // token by token waits for three loads in a row at every level
  const int branch = sh.start[1];
  struct Candidate {
    int tok;
    float u, px, qx;
  };
  auto look_up = [&](int row, int before) -> Candidate {
    Candidate k{p.tokens[row], p.u[row], 0.f, 0.f};
    if (k.tok >= 0 && k.tok < V) {
      k.px = load_f(P + (size_t)before * V + k.tok);
      if (sampled) k.qx = load_f(Q + (size_t)before * V + k.tok);
    }
    return k;
  };
  for (int i = tid; i < min(kHeld, end - branch); i += kVThreads) {
    const int row = branch + i, m = (int)checked(x.status, x.counts, x.token_node[row] - n0, nn, 903);
    const Candidate k = look_up(row, row > sh.start[m] ? row - 1 : sh.start[sh.parent[m] + 1] - 1);
    sh.tok[i] = k.tok;
    sh.u[i] = k.u;
    sh.px[i] = k.px;
    sh.qx[i] = k.qx;
  }
  __syncthreads();

  int cur = branch - 1, node = 0, taken = 0;
  int flip = 0;
  double c = 0., D = 1.;
  int n_out = 0;  // point masses rejected at this token

  // weight of entry v in the residual of the current token
  auto weight = [&](int v, float pv, float qv) -> double {
    double w = prob_of(pv);
    if (sampled) {
      if (c > 0.) w = fma(-c, prob_of(qv), w);
      return w > 0. ? w : 0.;
    }
    for (int i = 0; i < n_out; ++i)
      if (sh.kid_token[i] == v) return 0.;
    return w;
  };
  // this block's segment sums, kind: 0 the row p, 1 (p - c q)+, 2 p without the
  // rejected tokens (kept apart: the test for each entry cost more than its sum)
  auto sum_segments = [&](const T *prow, const T *qrow, auto kind) {
    constexpr int kKind = decltype(kind)::value;
    constexpr int kAhead = 4;  // segments on their way per warp
    for (int s0 = warp; s0 < n_seg; s0 += kAhead * kVWarps) {
      double acc[kAhead] = {};
      for (int o = 4 * lane; o < seg_len; o += 128) {
        float4 a[kAhead], b[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int v = v_lo + (s0 + k * kVWarps) * seg_len + o;
          a[k] = load4<T, kVec>(prow, v, v_hi);
          if (kKind == 1) b[k] = load4<T, kVec>(qrow, v, v_hi);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float pv[4] = {a[k].x, a[k].y, a[k].z, a[k].w}, qv[4] = {b[k].x, b[k].y, b[k].z, b[k].w};
          double w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (kKind == 1) w[i] = positive_part(fma(-c, small_prob(qv[i]), small_prob(pv[i])));
            else if (kKind == 0) w[i] = small_prob(pv[i]);
            else w[i] = weight(v_lo + (s0 + k * kVWarps) * seg_len + o + i, pv[i], 0.f);
          }
          acc[k] += (w[0] + w[1]) + (w[2] + w[3]);
        }
      }
      // the four segments' sums over the lanes: halves of the warp take two of them
      // each, quarters one, so six exchanges stand for twenty
      static_assert(kAhead == 4, "a segment to a quarter of the warp");
      const bool up = lane & 16, right = lane & 8;
      double x = up ? acc[2] : acc[0], y = up ? acc[3] : acc[1];
      x += __shfl_xor_sync(0xffffffffu, up ? acc[0] : acc[2], 16);
      y += __shfl_xor_sync(0xffffffffu, up ? acc[1] : acc[3], 16);
      double t = right ? y : x;
      t += __shfl_xor_sync(0xffffffffu, right ? x : y, 8);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (kKind != 2) t *= 0x1p896;
      if (kKind != 2 && t >= 0x1p128) t = INFINITY;  // an infinite entry
      const int k = lane >> 3;
      if ((lane & 7) == 0 && s0 + k * kVWarps < n_seg) sh.seg[s0 + k * kVWarps] = t;
    }
  };
  // sum of the weights over the vocabulary, the same bits in every block;
  // leaves each segment's sum in sh.seg and the blocks' in sh.total
  auto sum_weights = [&](const T *prow, const T *qrow) -> double {
    __syncthreads();
    if (sampled && c > 0.) sum_segments(prow, qrow, Kind<1>{});
    else if (sampled || n_out == 0) sum_segments(prow, qrow, Kind<0>{});
    else sum_segments(prow, qrow, Kind<2>{});
    __syncthreads();
    if (warp == 0) {
      double acc = 0.;
      for (int s = lane; s < n_seg; s += 32) acc += sh.seg[s];
      acc = warp_sum_d(acc);
      // every block gets a copy: nothing remote is read after the barrier
      if (lane < blocks) cluster.map_shared_rank(&sh.total[flip][0], lane)[rank] = acc;
    }
    cluster.sync();
    double all = 0.;
    for (int b = 0; b < blocks; ++b) all += sh.total[flip][b];
    flip ^= 1;
    return all;
  };
  // the next child of `node` after child m, or nn
  auto next_kid = [&](int m) -> int {
    for (int b = m + 1; b < nn; b += 32) {
      const unsigned hit = __ballot_sync(0xffffffffu, b + lane < nn && sh.parent[b + lane] == node);
      if (hit) return b + __ffs(hit) - 1;
    }
    return nn;
  };

  const T *prow, *qrow;
  double all = -1.;  // sum of the residual at the current token, if a pass has formed it
  for (;;) {
    prow = P + (size_t)cur * V;
    qrow = sampled ? Q + (size_t)cur * V : prow;
    c = 0.;
    D = 1.;
    all = -1.;
    n_out = 0;
    const bool inside = cur + 1 < sh.start[node + 1];  // the node goes on
    int m = inside ? node : next_kid(node);
    int down = -1, tried = 0;
    while (m < nn && down < 0) {
      // up to 32 continuations at a time, a lane each (every warp alike)
      int mine = -1, kids = 0;
      for (; kids < 32 && m < nn; ++kids) {
        if (lane == kids) mine = m;
        m = inside ? nn : next_kid(m);
      }
      int row = -1;
      Candidate own{-1, 0.f, 0.f, 0.f};
      if (mine >= 0) {
        row = inside ? cur + 1 : sh.start[mine];
        const int i = row - branch;
        own = i < kHeld ? Candidate{sh.tok[i], sh.u[i], sh.px[i], sh.qx[i]} : look_up(row, cur);
      }
      for (int k = 0; k < kids && down < 0; ++k) {
        const int k_row = __shfl_sync(0xffffffffu, row, k), k_tok = __shfl_sync(0xffffffffu, own.tok, k);
        const double k_u = __shfl_sync(0xffffffffu, own.u, k), k_p = prob_of(__shfl_sync(0xffffffffu, own.px, k));
        const double k_q = prob_of(__shfl_sync(0xffffffffu, own.qx, k));
        if (++tried > kMaxKids) {
          if (rank == 0 && tid == 0) set_status(x.status, FLIDE_ERR_CAPACITY);
          m = nn;
          break;
        }
        if (k_tok < 0 || k_tok >= V) {
          if (rank == 0 && tid == 0) set_status(x.status, FLIDE_ERR_INVALID);  // never accepted
        } else if (sampled) {
          if (k_u * k_q * D < fma(-c, k_q, k_p)) {
            down = k_row;
          } else {
            c += D;
            all = D = sum_weights(prow, qrow);
          }
        } else {
          bool gone = false;
          for (int i = 0; i < n_out; ++i) gone |= sh.kid_token[i] == k_tok;
          if (!gone && k_u * D < k_p) {
            down = k_row;
          } else if (!gone) {
            D -= k_p;
            __syncthreads();
            if (tid == 0) sh.kid_token[n_out] = k_tok;
            __syncthreads();
            ++n_out;
          }
        }
        if (down >= 0) node = __shfl_sync(0xffffffffu, mine, k);
      }
    }
    if (down < 0) break;
    if (rank == 0 && tid == 0) p.path[first + taken] = down;
    ++taken;
    cur = down;
  }

  // the next token: first entry whose cumulative weight passes u * sum
  if (all < 0.) all = sum_weights(prow, qrow);
  if (!(all > 0.)) {  // nothing left (rounding): the target row itself
    c = 0.;
    n_out = 0;
    all = sum_weights(prow, qrow);
  }
  flip ^= 1;  // the totals of the last exchange
  const double aim = (double)p.u_next[r] * all;
  double before = 0.;
  int owner = -1, last = -1;
  for (int b = 0; b < blocks; ++b) {
    const double t = sh.total[flip][b];
    if (t > 0.) last = b;
    if (owner < 0) {
      if (before + t > aim) owner = b;
      else before += t;
    }
  }
  const bool fell = owner < 0;  // rounding put the aim past the end
  if (fell) owner = last;
  if (rank == 0 && tid == 0) {
    p.n_accept[r] = taken;
    if (owner < 0 || !isfinite(all)) p.next_token[r] = -1;
  }
  if (owner < 0 || !isfinite(all) || rank != owner || warp != 0) return;
  // the segment: lanes sum runs of segments, then the run that holds the aim is
  // looked through
  const int per = (n_seg + 31) / 32;
  double run = 0.;
  int s_last = -1;
  for (int s = lane * per; s < min(n_seg, (lane + 1) * per); ++s) {
    run += sh.seg[s];
    if (sh.seg[s] > 0.) s_last = s;
  }
  double upto = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  s_last = __reduce_max_sync(0xffffffffu, s_last);
  const unsigned held = __ballot_sync(0xffffffffu, !fell && run > 0. && before + upto > aim);
  int s_hit = -1;
  double acc = before;
  if (held) {
    const int at = __ffs(held) - 1;
    acc += __shfl_sync(0xffffffffu, upto - run, at);
    for (int s = at * per; s < min(n_seg, (at + 1) * per) && s_hit < 0; ++s) {
      if (acc + sh.seg[s] > aim) s_hit = s;
      else acc += sh.seg[s];
    }
  }
  const bool to_end = s_hit < 0;
  const int s = to_end ? s_last : s_hit;
  const int a = v_lo + s * seg_len, b = min(v_hi, a + seg_len);
  int pick = -1, positive = -1;
  for (int v0 = a; v0 < b; v0 += 128) {  // four entries to a lane
    const int v = v0 + 4 * lane;
    const float4 pv = load4<T, kVec>(prow, v, b), qv = load4<T, kVec>(qrow, v, b);
    const double w[4] = {weight(v, pv.x, qv.x), weight(v + 1, pv.y, qv.y), weight(v + 2, pv.z, qv.z),
                         weight(v + 3, pv.w, qv.w)};
    double upto4 = (w[0] + w[1]) + (w[2] + w[3]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, upto4, o);
      if (lane >= o) upto4 += y;
    }
    // the sums before each of the lane's entries
    double at = __shfl_up_sync(0xffffffffu, upto4, 1);
    at = acc + (lane ? at : 0.);
    int mine = -1, some = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      at += w[i];
      if (w[i] > 0.) some = v + i;
      if (!to_end && mine < 0 && w[i] > 0. && at > aim) mine = v + i;
    }
    positive = max(positive, __reduce_max_sync(0xffffffffu, some));
    const unsigned hit = __ballot_sync(0xffffffffu, mine >= 0);
    if (hit) {
      pick = __shfl_sync(0xffffffffu, mine, __ffs(hit) - 1);
      break;
    }
    acc += __shfl_sync(0xffffffffu, upto4, 31);
  }
  if (lane == 0) p.next_token[r] = pick >= 0 ? pick : positive;
}

template <typename T, bool kVec>
int verify_launch(const VerifyParams &p, bool wide, int dev, cudaStream_t s) {
  static std::atomic<bool> allowed[64];  // zero-initialised: false
  if (wide && (dev < 0 || dev >= 64 || !allowed[dev].load(std::memory_order_acquire))) {
    if (cudaFuncSetAttribute(verify_kernel<T, kVec>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
        cudaSuccess)
      return FLIDE_ERR_CUDA;
    if (dev >= 0 && dev < 64) allowed[dev].store(true, std::memory_order_release);
  }
  const unsigned blocks = wide ? 16 : 8;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = blocks;
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.x.R * blocks);
  cfg.blockDim = dim3(kVThreads);
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return launched(cudaLaunchKernelEx(&cfg, verify_kernel<T, kVec>, p));
}

}  // namespace
}  // namespace flide

extern "C" int flide_verify_draft(const flide_tree_index *idx, const int32_t *tokens,
                                  const void *target, const void *draft, const float *u,
                                  const float *u_next, int32_t V, int32_t dtype, int32_t *n_accept,
                                  int32_t *next_token, int32_t *path, flide_stream stream) {
  using namespace flide;
  if (!idx || !tokens || !target || !u || !u_next || !n_accept || !next_token || !path)
    return FLIDE_ERR_SHAPE;
  if (V <= 0 || V > (1 << 26) || idx->R < 0) return FLIDE_ERR_SHAPE;
  if (dtype != FLIDE_F32 && dtype != FLIDE_BF16) return FLIDE_ERR_SHAPE;
  if (idx->R > (1 << 24)) return FLIDE_ERR_CAPACITY;
  if (idx->R == 0) return FLIDE_OK;
  const VerifyParams p{*idx, tokens, target, draft, u, u_next, V, n_accept, next_token, path};
  cudaStream_t s = (cudaStream_t)stream;
    // rows of whole 16-byte (bf16: 8-byte) words are read as such
  const bool vec = V % 4 == 0 && ((uintptr_t)target | (uintptr_t)draft) % 16 == 0;
  // 16 blocks to a cluster where every tree has its 16 at once and its rows are
  // long: a pass over 131072 entries takes 3.5 us instead of 6, the wider
  // exchange costs 2 us a call (8192 entries: 11 instead of 9 us)
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FLIDE_ERR_CUDA;
  const bool wide = V >= 32768 && idx->R * 16 <= 4 * sms;
  if (dtype == FLIDE_F32)
    return vec ? verify_launch<float, true>(p, wide, dev, s) : verify_launch<float, false>(p, wide, dev, s);
  return vec ? verify_launch<__nv_bfloat16, true>(p, wide, dev, s)
             : verify_launch<__nv_bfloat16, false>(p, wide, dev, s);
}

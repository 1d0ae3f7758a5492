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
// A cluster of 8 blocks walks one request: every block takes an eighth of the
// vocabulary in each pass and repeats the walk's decisions from the same
// numbers (sums are exchanged through distributed shared memory in a fixed
// order).  Bound by the latency of the walk's dependent loads for one tree,
// by the rows' bytes for a batch.
#include <cooperative_groups.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace flide {
namespace {

constexpr int kCluster = 8;
constexpr int kVThreads = 512;
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

struct VerifyShared {
  int parent[kMaxNodes];  // request-local parent of each node
  int kid_token[kMaxKids];
  double seg[kMaxSegs];
  double warp[kVWarps];
  double total[2];        // this block's part of a sum, by parity of the exchange
  int stop;
};

template <typename T>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kVThreads)
verify_kernel(const VerifyParams p) {
  __shared__ VerifyShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const flide_tree_index &x = p.x;
  const int rank = (int)cluster.block_rank();
  const int r = blockIdx.x / kCluster;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the status word may change while this kernel runs (another cluster's bad
  // token), so one block's reading decides for its whole cluster
  if (tid == 0) sh.stop = failed(x.status);
  cluster.sync();
  const bool stop = *cluster.map_shared_rank(&sh.stop, 0) != 0;
  const int n0 = x.req_node[r], n1 = x.req_node[r + 1];
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
  for (int i = tid; i < nn; i += kVThreads)
    sh.parent[i] = i == 0 ? -1 : x.anc_node[x.anc_ptr[n0 + i + 1] - 2] - n0;
  __syncthreads();

  const T *P = static_cast<const T *>(p.target), *Q = static_cast<const T *>(p.draft);
  const bool sampled = Q != nullptr;
  const int V = p.V;
  // this block's slice and its segments (contiguous, at most kMaxSegs)
  const int slice = ((V + kCluster - 1) / kCluster + 127) / 128 * 128;
  const int v_lo = min(V, rank * slice), v_hi = min(V, v_lo + slice);
  const int seg_len = max(128, ((slice + kMaxSegs - 1) / kMaxSegs + 127) / 128 * 128);
  const int n_seg = (v_hi - v_lo + seg_len - 1) / seg_len;

  int cur = x.node_start[n0 + 1] - 1, node = 0, taken = 0;
  int flip = 0;
  double c = 0., D = 1.;
  int n_out = 0;  // point masses rejected at this token

  // weight of entry v in the residual of the current token
  auto weight = [&](const T *prow, const T *qrow, int v) -> double {
    double w = prob_of(load_f(prow + v));
    if (sampled) {
      if (c > 0.) w = w - c * prob_of(load_f(qrow + v));
      return w > 0. ? w : 0.;
    }
    for (int i = 0; i < n_out; ++i)
      if (sh.kid_token[i] == v) return 0.;
    return w;
  };
  // sum of the weights over the vocabulary, the same bits in every block;
  // leaves each segment's sum in sh.seg and each block's in its sh.total
  auto sum_weights = [&](const T *prow, const T *qrow) -> double {
    __syncthreads();
    for (int s = warp; s < n_seg; s += kVWarps) {
      const int a = v_lo + s * seg_len, b = min(v_hi, a + seg_len);
      double acc = 0.;
      for (int v = a + lane; v < b; v += 32) acc += weight(prow, qrow, v);
      acc = warp_sum_d(acc);
      if (lane == 0) sh.seg[s] = acc;
    }
    __syncthreads();
    if (warp == 0) {
      double acc = 0.;
      for (int s = lane; s < n_seg; s += 32) acc += sh.seg[s];
      acc = warp_sum_d(acc);
      if (lane == 0) sh.total[flip] = acc;
    }
    cluster.sync();
    double all = 0.;
    for (int b = 0; b < kCluster; ++b) all += cluster.map_shared_rank(sh.total, b)[flip];
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
  for (;;) {
    prow = P + (size_t)cur * V;
    qrow = sampled ? Q + (size_t)cur * V : nullptr;
    c = 0.;
    D = 1.;
    n_out = 0;
    const bool inside = cur + 1 < x.node_start[n0 + node + 1];  // the node goes on
    int m = inside ? node : next_kid(node);
    int down = -1, tried = 0;
    while (m < nn) {
      const int row = inside ? cur + 1 : x.node_start[n0 + m];
      const int tok = p.tokens[row];
      if (++tried > kMaxKids) {
        if (rank == 0 && tid == 0) set_status(x.status, FLIDE_ERR_CAPACITY);
        break;
      }
      if (tok < 0 || tok >= V) {
        if (rank == 0 && tid == 0) set_status(x.status, FLIDE_ERR_INVALID);  // never accepted
      } else {
        const double u = (double)p.u[row], px = prob_of(load_f(prow + tok));
        if (sampled) {
          const double qx = prob_of(load_f(qrow + tok));
          const double left = c > 0. ? px - c * qx : px;
          if (u * qx * D < left) {
            down = row;
          } else {
            c += D;
            D = sum_weights(prow, qrow);
          }
        } else {
          bool gone = false;
          for (int i = 0; i < n_out; ++i) gone |= sh.kid_token[i] == tok;
          if (!gone && u * D < px) {
            down = row;
          } else if (!gone) {
            D -= px;
            __syncthreads();
            if (tid == 0) sh.kid_token[n_out] = tok;
            __syncthreads();
            ++n_out;
          }
        }
      }
      if (down >= 0 || inside) break;
      m = next_kid(m);
    }
    if (down < 0) break;
    if (rank == 0 && tid == 0) p.path[first + taken] = down;
    ++taken;
    cur = down;
    node = m;
  }

  // the next token: first entry whose cumulative weight passes u * sum
  double all = sum_weights(prow, qrow);
  if (!(all > 0.)) {  // nothing left (rounding): the target row itself
    c = 0.;
    n_out = 0;
    all = sum_weights(prow, qrow);
  }
  flip ^= 1;  // the totals of the last exchange
  const double aim = (double)p.u_next[r] * all;
  double before = 0.;
  int owner = -1, last = -1;
  for (int b = 0; b < kCluster; ++b) {
    const double t = cluster.map_shared_rank(sh.total, b)[flip];
    if (t > 0.) last = b;
    if (owner < 0) {
      if (before + t > aim) owner = b;
      else before += t;
    }
  }
  cluster.sync();  // every block has read the totals
  const bool fell = owner < 0;  // rounding put the aim past the end
  if (fell) owner = last;
  if (rank == 0 && tid == 0) {
    p.n_accept[r] = taken;
    if (owner < 0 || !isfinite(all)) p.next_token[r] = -1;
  }
  if (owner < 0 || !isfinite(all) || rank != owner || warp != 0) return;
  int s_hit = -1, s_last = -1;
  double acc = before;
  for (int s = 0; s < n_seg; ++s) {
    const double t = sh.seg[s];
    if (t > 0.) s_last = s;
    if (s_hit < 0) {
      if (!fell && acc + t > aim) s_hit = s;
      else acc += t;
    }
  }
  bool to_end = fell || s_hit < 0;
  const int s = s_hit >= 0 ? s_hit : s_last;
  const int a = v_lo + s * seg_len, b = min(v_hi, a + seg_len);
  int pick = -1, positive = -1;
  for (int v0 = a; v0 < b; v0 += 32) {
    const int v = v0 + lane;
    const double w = v < b ? weight(prow, qrow, v) : 0.;
    double incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned pos = __ballot_sync(0xffffffffu, w > 0.);
    if (pos) positive = v0 + 31 - __clz(pos);
    const unsigned hit = __ballot_sync(0xffffffffu, !to_end && w > 0. && acc + incl > aim);
    if (hit) {
      pick = v0 + __ffs(hit) - 1;
      break;
    }
    acc += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) p.next_token[r] = pick >= 0 ? pick : positive;
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
  const unsigned grid = (unsigned)idx->R * kCluster;
  if (dtype == FLIDE_F32) verify_kernel<float><<<grid, kVThreads, 0, s>>>(p);
  else verify_kernel<__nv_bfloat16><<<grid, kVThreads, 0, s>>>(p);
  FLIDE_LAUNCH_CHECK();
  return FLIDE_OK;
}

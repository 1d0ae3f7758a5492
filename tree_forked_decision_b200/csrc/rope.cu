// rope.cu -- rotary positions of a request tree's tokens.
//
// A token at isolated position p (token_pos of the tree index plus the
// request's offset) turns pair i of the first rot_dim elements of every head
// by the angle p * freqs[i]:
//   a' = m (a cos - b sin),  b' = m (a sin + b cos),
// with (a, b) = elements (i, i + rot_dim/2) in the half layout, (2i, 2i + 1)
// in the interleaved one, and m the long-context factor; the transposed
// rotation (sin -> -sin) is the gradient of the rotation, and undoes it for
// m = 1.  Elements from rot_dim on are copied.
//
// Angles are formed in 64 bits: a position of 10^6 leaves a 32-bit angle 20
// bits short of its fraction of a turn.  p f / 2pi is reduced to a fraction
// of a turn there, and only that goes to the 32-bit sincospi.
//
// Bound by bandwidth: q and k once in, once out.
#include <cmath>

#include "common.cuh"

namespace flide {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxRot = 1024;

struct RopeParams {
  flide_tree_index x;
  const int32_t *pos_offset;
  const double *freqs;
  const void *in[2];
  void *out[2];
  int heads[2];
  int d, rot, interleaved;
  float mscale, sign;
};

// One block per token: the token's cos and sin once, then every head.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  __shared__ float2 cs[kMaxRot / 2];
  const flide_tree_index &x = p.x;
  const int t = blockIdx.x;
  if (failed(x.status) || t >= x.counts[FLIDE_CNT_T]) return;
  const int half = p.rot >> 1;
  const int n = (int)checked(x.status, x.counts, x.token_node[t], x.counts[FLIDE_CNT_N], 701);
  const long long pos = (long long)x.token_pos[t] + (p.pos_offset ? p.pos_offset[x.node_req[n]] : 0);
  for (int i = threadIdx.x; i < half; i += blockDim.x) {
    const double turns = (double)pos * p.freqs[i] * 0.15915494309189535;  // 1 / 2 pi
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    cs[i] = make_float2(p.mscale * c, p.sign * p.mscale * s);
  }
  __syncthreads();
  const int rest = p.d - p.rot;  // copied elements of a head
  const int per = half + rest;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if (!p.in[w]) continue;
    const size_t row = (size_t)t * p.heads[w] * p.d;
    const T *in = static_cast<const T *>(p.in[w]) + row;
    T *out = static_cast<T *>(p.out[w]) + row;
    for (int e = threadIdx.x; e < p.heads[w] * per; e += blockDim.x) {
      const int h = e / per, i = e - h * per;
      const int base = h * p.d;
      if (i < half) {
        const int ia = base + (p.interleaved ? 2 * i : i), ib = p.interleaved ? ia + 1 : ia + half;
        const float a = load_f(in + ia), b = load_f(in + ib);
        const float2 r = cs[i];
        store_f(out + ia, a * r.x - b * r.y);
        store_f(out + ib, a * r.y + b * r.x);
      } else {
        const int ic = base + p.rot + i - half;
        out[ic] = in[ic];
      }
    }
  }
}

}  // namespace
}  // namespace flide

extern "C" int flide_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor,
                                double orig_len, double fast, double slow, double *freqs,
                                float *mscale) {
  using namespace flide;
  if (!freqs || !mscale || rot_dim < 2 || rot_dim > kMaxRot || rot_dim % 2) return FLIDE_ERR_SHAPE;
  if (!(base > 0.) || !std::isfinite(base)) return FLIDE_ERR_INVALID;
  if (scaling != FLIDE_ROPE_NONE && (!(factor >= 1.) || !std::isfinite(factor))) return FLIDE_ERR_INVALID;
  *mscale = 1.f;
  switch (scaling) {
    case FLIDE_ROPE_NONE: break;
    case FLIDE_ROPE_LINEAR: break;
    case FLIDE_ROPE_NTK:
      if (rot_dim > 2) base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
      break;
    case FLIDE_ROPE_YARN:
      if (!(orig_len > 0.) || !std::isfinite(orig_len) || !(fast > slow) || !(slow >= 0.) ||
          !std::isfinite(fast))
        return FLIDE_ERR_INVALID;
      *mscale = (float)(0.1 * std::log(factor) + 1.);
      break;
    default: return FLIDE_ERR_SHAPE;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2. * i / rot_dim);
    if (scaling == FLIDE_ROPE_LINEAR) f /= factor;
    if (scaling == FLIDE_ROPE_YARN) {
      const double turns = orig_len * f / 6.283185307179586;  // over the trained length
      const double keep = std::fmin(std::fmax((turns - slow) / (fast - slow), 0.), 1.);
      f *= keep + (1. - keep) / factor;
    }
    freqs[i] = f;
  }
  return FLIDE_OK;
}

extern "C" int flide_rope(const flide_tree_index *idx, const int32_t *pos_offset, const double *freqs,
                          const void *q, const void *k, void *q_out, void *k_out, int32_t Hq,
                          int32_t Hkv, int32_t d, int32_t rot_dim, int32_t interleaved,
                          int32_t transpose, float mscale, int32_t dtype, flide_stream stream) {
  using namespace flide;
  if (!idx || !freqs || (!q && !k) || (q != nullptr) != (q_out != nullptr) ||
      (k != nullptr) != (k_out != nullptr))
    return FLIDE_ERR_SHAPE;
  if ((q && Hq <= 0) || (k && Hkv <= 0) || d <= 0 || rot_dim < 2 || rot_dim % 2 || rot_dim > d ||
      rot_dim > kMaxRot)
    return FLIDE_ERR_SHAPE;
  if ((long long)d * ((q ? Hq : 0) + (long long)(k ? Hkv : 0)) > 0x3fffffffLL) return FLIDE_ERR_CAPACITY;
  if (dtype != FLIDE_F32 && dtype != FLIDE_BF16) return FLIDE_ERR_SHAPE;
  if (idx->T < 0) return FLIDE_ERR_SHAPE;
  if (idx->T == 0) return FLIDE_OK;
  RopeParams p;
  p.x = *idx;
  p.pos_offset = pos_offset;
  p.freqs = freqs;
  p.in[0] = q;
  p.in[1] = k;
  p.out[0] = q_out;
  p.out[1] = k_out;
  p.heads[0] = Hq;
  p.heads[1] = Hkv;
  p.d = d;
  p.rot = rot_dim;
  p.interleaved = interleaved != 0;
  p.mscale = mscale;
  p.sign = transpose ? -1.f : 1.f;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == FLIDE_F32) rope_kernel<float><<<idx->T, kRopeThreads, 0, s>>>(p);
  else rope_kernel<__nv_bfloat16><<<idx->T, kRopeThreads, 0, s>>>(p);
  FLIDE_LAUNCH_CHECK();
  return FLIDE_OK;
}

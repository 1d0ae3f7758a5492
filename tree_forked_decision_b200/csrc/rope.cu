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
#include "sm100.cuh"

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

// What a thread loads at once, and its values: a 16-byte word, or one element.
template <typename T, bool kVec>
struct Unit {
  static constexpr int kN = 16 / sizeof(T);
  using Word = uint4;
  static __device__ __forceinline__ void unpack(const uint4 &w, float (&v)[kN]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      } else {
        v[i] = __uint_as_float(u[i]);
      }
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[kN]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) u[i] = sm100::pack_bf16x2(v[2 * i], v[2 * i + 1]);
      else u[i] = __float_as_uint(v[i]);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <typename T>
struct Unit<T, false> {
  static constexpr int kN = 1;
  using Word = T;
  static __device__ __forceinline__ void unpack(const T &w, float (&v)[1]) { v[0] = load_f(&w); }
  static __device__ __forceinline__ T pack(const float (&v)[1]) {
    T w;
    store_f(&w, v[0]);
    return w;
  }
};

// Blocks of `tok` tokens.  Their angles come first, all at once: the loads behind
// a position and the 64-bit turn take about 5 us in a row, which a block per token
// waited for with 3 blocks to an SM (326 us for 839 MB, whatever came after).  A
// unit of a head is what a thread turns between a load and a store: with kVec a
// 16-byte word of pairs (interleaved), one word of each half (half layout) or one
// copied word; else one pair or one copied element.  A thread keeps its unit and
// goes over the block's (token, head) rows, some of them loaded ahead (as raw
// words: unpacking at the load waits for each in turn, 199 us).  8 requests of
// 4096 + 64 x 16 tokens, 32 + 8 heads of 128, bf16: 138 us replayed from a graph, 6.1
// TB/s; 144 called back to back.
template <typename T, bool kVec, bool kInter>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, int tok) {
  extern __shared__ __align__(16) float cs[];  // cos [tok][half], sin [tok][half]
  const flide_tree_index &x = p.x;
  const int t0 = blockIdx.x * tok, tid = threadIdx.x;
  const int T_act = x.counts[FLIDE_CNT_T];
  if (failed(x.status) || t0 >= T_act) return;
  const int nt = min(tok, T_act - t0);
  const int half = p.rot >> 1;
  float *cosv = cs, *sinv = cs + tok * half;
  for (int e = tid; e < nt * half; e += kRopeThreads) {
    const int tt = e / half, t = t0 + tt;
    const int n = (int)checked(x.status, x.counts, x.token_node[t], x.counts[FLIDE_CNT_N], 701);
    const long long pos = (long long)x.token_pos[t] + (p.pos_offset ? p.pos_offset[x.node_req[n]] : 0);
    const double turns = (double)pos * p.freqs[e - tt * half] * 0.15915494309189535;  // 1 / 2 pi
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    cosv[e] = p.mscale * c;
    sinv[e] = p.sign * p.mscale * s;
  }
  __syncthreads();
  using U = Unit<T, kVec>;
  using Word = typename U::Word;
  constexpr int kN = U::kN;
  constexpr int kPairs = kVec && kInter ? kN / 2 : kN;  // pairs of a unit
  constexpr bool kTwo = !(kVec && kInter);              // its second elements lie elsewhere
  constexpr int kAhead = kTwo && kVec ? 2 : 4;          // heads loaded before the first is turned
  const int turned = half / kPairs;
  const int per = turned + (p.d - p.rot) / kN;
  const int pw = min(per, kRopeThreads), rows = kRopeThreads / pw;
  const int heads = p.heads[0] + p.heads[1];
  const int h0 = tid / pw;
  if (h0 >= rows) return;
  for (int i = tid - h0 * pw; i < per; i += pw) {
    const bool turn = i < turned;
    const int first = turn ? (kInter ? i * 2 * kPairs : i * kN) : p.rot + (i - turned) * kN;
    const int off = kInter ? 1 : half;
    // the block's (token, head) rows h0, h0 + rows, ...
    int tt = h0 / heads, h = h0 - tt * heads;
    while (tt < nt) {
      Word wa[kAhead], wb[kAhead];
      T *dst[kAhead];
      const float *ang[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        dst[k] = nullptr;
        if (tt < nt) {
          const int w = h >= p.heads[0];
          const size_t at = ((size_t)(t0 + tt) * p.heads[w] + h - (w ? p.heads[0] : 0)) * p.d + first;
          const T *src = static_cast<const T *>(w ? p.in[1] : p.in[0]) + at;
          dst[k] = static_cast<T *>(w ? p.out[1] : p.out[0]) + at;
          ang[k] = cosv + tt * half + i * kPairs;
          wa[k] = *reinterpret_cast<const Word *>(src);
          if (kTwo && turn) wb[k] = *reinterpret_cast<const Word *>(src + off);
        }
        for (h += rows; h >= heads; h -= heads) ++tt;
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (!dst[k]) continue;
        if (turn) {
          float co[kPairs], si[kPairs], a[kN], b[kN];
          U::unpack(wa[k], a);
          if (kTwo) U::unpack(wb[k], b);
          if constexpr (kPairs % 4 == 0) {
#pragma unroll
            for (int j = 0; j < kPairs; j += 4) {
              *reinterpret_cast<float4 *>(co + j) = *reinterpret_cast<const float4 *>(ang[k] + j);
              *reinterpret_cast<float4 *>(si + j) = *reinterpret_cast<const float4 *>(ang[k] + tok * half + j);
            }
          } else {
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
              co[j] = ang[k][j];
              si[j] = ang[k][tok * half + j];
            }
          }
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
            float &u = kTwo ? a[j] : a[(2 * j) % kN], &v = kTwo ? b[j] : a[(2 * j + 1) % kN];
            const float u0 = u, v0 = v;
            u = u0 * co[j] - v0 * si[j];
            v = u0 * si[j] + v0 * co[j];
          }
          wa[k] = U::pack(a);
          if (kTwo) wb[k] = U::pack(b);
        }
        *reinterpret_cast<Word *>(dst[k]) = wa[k];
        if (kTwo && turn) *reinterpret_cast<Word *>(dst[k] + off) = wb[k];
      }
    }
  }
}

// 16-byte words where rows, the turned part and (half layout) its halves are
// whole words; more tokens to a block where that leaves at least 1024 blocks.
template <typename T>
int rope_launch(const RopeParams &p, bool aligned, cudaStream_t s) {
  constexpr int kN = Unit<T, true>::kN;
  const bool vec = aligned && p.d % kN == 0 && (p.interleaved ? p.rot : p.rot / 2) % kN == 0;
  int tok = 1;
  while (tok < 16 && p.x.T >= 2048 * tok && tok * p.rot * sizeof(float) <= 16384) tok *= 2;
  const size_t smem = (size_t)tok * p.rot * sizeof(float);
  const unsigned grid = (unsigned)((p.x.T + tok - 1) / tok);
  if (vec && p.interleaved) rope_kernel<T, true, true><<<grid, kRopeThreads, smem, s>>>(p, tok);
  else if (vec) rope_kernel<T, true, false><<<grid, kRopeThreads, smem, s>>>(p, tok);
  else if (p.interleaved) rope_kernel<T, false, true><<<grid, kRopeThreads, smem, s>>>(p, tok);
  else rope_kernel<T, false, false><<<grid, kRopeThreads, smem, s>>>(p, tok);
  FLIDE_LAUNCH_CHECK();
  return FLIDE_OK;
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
  p.heads[0] = q ? Hq : 0;
  p.heads[1] = k ? Hkv : 0;
  p.d = d;
  p.rot = rot_dim;
  p.interleaved = interleaved != 0;
  p.mscale = mscale;
  p.sign = transpose ? -1.f : 1.f;
  const bool aligned = ((uintptr_t)q | (uintptr_t)k | (uintptr_t)q_out | (uintptr_t)k_out) % 16 == 0;
  return dtype == FLIDE_F32 ? rope_launch<float>(p, aligned, (cudaStream_t)stream)
                            : rope_launch<__nv_bfloat16>(p, aligned, (cudaStream_t)stream);
}

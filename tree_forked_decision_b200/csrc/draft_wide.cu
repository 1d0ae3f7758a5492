// draft_wide.cu -- draft attention's part kernel for wide trees, on tcgen05.
//
// A tile of query rows (whole tokens x heads of the group, as many as fit) is one or
// two 128-row operands.  Keys come in tiles of 128 by TMA, K and V each through a ring of
// stages; S = Q K^T and O += P V accumulate in TMEM, the softmax reads S and
// writes P there, one row a thread.  Two softmax warpgroups work on two S
// buffers, so the tensor core always has the other one's products to do:
//   - 256 rows: each warpgroup has its own 128 rows, both see every key tile;
//   - 128 rows: both have the same rows and take every second key tile; their
//     (O, max, sum) are two partials for the join.  One operand's softmax alone
//     would leave the tensor core and the memory idle half the time;
//   - 64 or 32 rows: the operand holds them two or four times, and each copy's
//     threads take a half or quarter of the tile's keys (their weights for the
//     others are 0): a half or quarter of the softmax in each thread's chain, which
//     is what bounds a tile.  The four or eight results are joined in the block.
// A block (one to an SM) takes its share of the batch's key tiles as runs
// inside one (request, row tile, kv head) item (draft.cuh); barriers count over
// the block's life, so the next run's loads are in flight while the last tiles
// of a run are computed.  V rows behind the history's end are zeroed in shared
// memory before they are multiplied: their weight is 0, but what stands there
// may be NaN.
//
// e4m3: S and O come from the codes (kind::f8f6f4, exact products).  A weight in
// e4m3 would be 2^-4 off, so it goes in as two codes, its own and its remainder's:
// two products at twice the rate.  The remainder is in e5m2: half a step of either
// type is 2^-8 of the weight (3 + 1 + 3 bits and a sign), but e5m2 reaches from 2^-16
// up, where e4m3's least step, 2^-9, would lose every key below 2^-16 of a row's
// dominant one, however many there are (16384 keys of 2^-17 of a first one, a ninth of
// the sum together: results up to half short).  Scaled by 2^6, a weight is off by 2^-8
// of itself or 2^-20 of the row's largest, and below 2^-16 of it by an eighth of itself.
// A row's reference is raised once a score passes it by 2.75 (2^8.75 < 448, the
// format's largest; raised at 2, some warp of a tile had to rescale O in most of a
// history's first tiles: 82 us instead of 78).  (Widening V to half in the softmax
// warps instead: 13 us more of 110.)
//
// 256 rows are bound by the two warpgroups' softmax and the MMA issue (see
// attn_tc.cu): 2.35 us a key tile where its bytes would take 1.5; 8 requests of 64
// tokens over 32768 rows, 32 + 8 heads, 296 us a call, 930 TFLOP/s, while the clock
// holds; back to back the power limit makes it 353 (1.49 GHz, 780 TFLOP/s).  128 rows
// and fewer by the history's bytes and the ends of runs: a tile takes 1.25 us (bytes
// 1.5, part of them from L2), a block's first scores come after 8 us, a run's
// end takes 4 to 5; 16 histories of 512 to 8192 rows, 20 tokens each, 61 us a call,
// 4.2 TB/s (back to back 67 to 71).  e4m3, 32 rows: 0.93 us a tile (bytes 0.75), bound
// by its twelve products (1.75K cycles); a run's end 3 us; 16 histories of 1024 to
// 16391 rows, 8 tokens each, 79 us a call, 3.9 TB/s (back to back 92 to 97).  The tiles
// of 128 and 256 rows spill 170 to 200 bytes a thread at the 168 registers that 352
// threads leave.  Histories that one tile reads leave L2
// before other lines (16 x 8192 rows: 75 -> 68 us; blocks that many requests share
// through their tables pay for it: 64 requests over the same 16384 rows 476 -> 499).
// Loading the next run's Q in a warp of its own, or as soon as the last scores are
// out, changed nothing.  Every wait is bounded (2 s);
// on expiry the block records FLIDE_ERR_TIMEOUT, waits for its own copies and
// MMAs, frees TMEM and ends.
#include <cstddef>
#include <cuda.h>
#include <cuda_fp16.h>

#include "draft.cuh"
#include "launch.cuh"
#include "sm100.cuh"

namespace flide {
namespace {

using namespace sm100;

constexpr int kBM = 128, kBN = 128;
constexpr int kWThreads = 352;  // two softmax warpgroups, K and Q loads, MMA, V loads
constexpr uint64_t kWaitNs = 2000000000ull;

// Shared memory: Q's operands, the stages of K and of V (32 KB a tile, 16 KB of
// codes), then the barriers and the block's work list (32 bytes a request).  As many
// stages as fit.
constexpr int kMaxStages = 4;
constexpr int kMinStages = 4;  // of K and V together: two each
constexpr int kSmemMax = 232448;
enum {
  bQ = 0,
  bQFree = 1,
  bK = 2,                     // [stages]
  bKFree = bK + kMaxStages,   // [stages]
  bV = bKFree + kMaxStages,   // [stages]
  bVFree = bV + kMaxStages,   // [stages]
  bS = bVFree + kMaxStages,   // [2 S buffers]
  bP = bS + 2,                // [2], 4 warps
  bOFree = bP + 2,            // [2], the 4 warps of an S buffer, or (copies) all 8
  bO = bOFree + 2,
  bMerge = bO + 1,            // 8 warps
  bDrain = bMerge + 1,
  kBars = bDrain + 1
};
constexpr int kBarBytes = (8 * kBars + 15) / 16 * 16;
struct __align__(16) Misc {
  uint32_t tmem;
  int abort;
  long long part[64];
};
// Where copies' results are joined: their rows (132 floats: eight lanes' words in
// 32 banks), and a warp's (max, sum) for each of its rows.
constexpr int merge_bytes(int d, int rep) { return rep > 1 ? kBM / rep * (d + 4) * 4 + 2 * 8 * 32 * 4 : 0; }
constexpr size_t wide_smem(int tile_bytes, int d, int halves, int rep, int tiles, long long R) {
  return (size_t)(halves + tiles) * tile_bytes + merge_bytes(d, rep) + kBarBytes + sizeof(Misc) +
         (size_t)(R + 1) * sizeof(DraftReq) + 1024;
}

// A key tile's stage and how often the ring has been round (its parity is that of
// the stage's barriers); a division per tile would stand between two products.
struct Ring {
  int st = 0;
  uint32_t turn = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++st == stages) {
      st = 0;
      turn ^= 1;
    }
  }
};

struct WideMaps {
  CUtensorMap q, k, v;
};

template <int kD, int kHalves, int kRep, bool F8>
__global__ void __launch_bounds__(kWThreads, 1)
draft_part_wide(const __grid_constant__ WideMaps maps, const DraftParams p, int mtok, int box_rows,
                int stages_k, int stages_v) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sb = smem_u32(smem);
  static_assert(kHalves == 1 || kRep == 1, "copies are of a tile of one operand");
  constexpr int kCopy = kBM / kRep, kCols = kBN / kRep;  // rows of a copy, keys of its threads
  constexpr int kSlabs = kD * (F8 ? 1 : 2) / 128, kTile = kSlabs * 16384;  // 128-byte slabs of a row; bytes
  const int s_k = kHalves * kTile, s_v = s_k + stages_k * kTile, s_m = s_v + stages_v * kTile;
  const int s_bar = s_m + merge_bytes(kD, kRep);
  Misc &ms = *reinterpret_cast<Misc *>(smem + s_bar + kBarBytes);
  volatile int *abort_flag = &ms.abort;
  DraftReq *list = reinterpret_cast<DraftReq *>(&ms + 1);
  const flide_tree_index &x = p.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](int i) -> uint32_t { return sb + s_bar + 8 * i; };
  asm volatile("griddepcontrol.launch_dependents;");
  if (tid == 0) {
    for (int i = 0; i < kBars; ++i)
      mbar_init(bar(i), i >= bP && i < bP + 2 ? 4u
                        : i >= bOFree && i < bOFree + 2 ? (kRep > 1 ? 8u : 4u) : i == bMerge ? 8u : 1u);
    fence_mbar_init();
    ms.abort = 0;
  }
  // rows of an operand, or of a copy, that hold queries: whole tokens.  The rows behind
  // them stay 0 (no copy writes them), so their softmax is quiet.
  const int real = mtok * p.G;
  if (real != kCopy) {
    for (int e = tid; e < kHalves * kTile / 16; e += kWThreads)
      reinterpret_cast<uint4 *>(smem)[e] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  if (!draft_list(p, list, ms.part)) return;
  const long long U = list[x.R].unit0;
  const int w = blockIdx.x, W = workers_of(U, p.workers);
  if (w >= W) return;
  if (warp == 9) {
    tmem_alloc(sb + s_bar + kBarBytes + (uint32_t)offsetof(Misc, tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem;
  long long u = worker_start(U, W, w);
  const long long u_end = worker_start(U, W, w + 1);
  // step i of a run: S buffer i & 1, key tile i (128 rows) or i / 2 (256 rows)
  auto tile_of = [](int i) { return kHalves == 2 ? i >> 1 : i; };
  // first step that a key tile is used by
  auto opens = [](int i) { return kHalves == 1 || !(i & 1); };

  if (warp == 8 || warp == 10) {
    // -------------------------------------------------------------- producers
    // warp 8 loads Q and K, warp 10 V: K's next tile does not wait behind V's
    const bool is_v = warp == 10;
    const CUtensorMap *map = is_v ? &maps.v : &maps.k;
    const int stages = is_v ? stages_v : stages_k;
    const int b_full = is_v ? bV : bK, b_free = is_v ? bVFree : bKFree, s_at = is_v ? s_v : s_k;
    if (lane == 0) {
      if (!is_v) prefetch_tmap(&maps.q);
      prefetch_tmap(map);
    }
    const int boxes = kBN / box_rows;
    auto wait = [&](int b, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, abort_flag, kWaitNs));
    };
    bool ok = true;
    int rc = 0, kt = 0;  // runs, key tiles so far
    Ring ring;
    Run run;
    const uint64_t once = policy_evict_first(), again = policy_evict_normal();
    for (; ok && draft_run(p, list, u, u_end, w, run); ++rc) {
      const uint64_t policy = tiles_of(p, run.tokens) > 1 ? again : once;
      // boxes that hold history rows, a lane each (the rest of the last tile keeps
      // what the stage held, and is masked); looked up a tile ahead
      auto row_at = [&](int k0) -> long long {
        const int k = k0 + lane * box_rows;
        if (lane >= boxes || k >= run.k1) return -1;
        return max(history_row(x, p.hist, run.base, k), 0ll);  // no block: row 0, the call is flagged
      };
      long long next = row_at(run.k0);
      if (!is_v) {
        if (rc > 0 && !(ok = wait(bQFree, (rc - 1) & 1))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(bQ), kHalves * kSlabs * kRep * real * 128);
          for (int h = 0; h < kHalves; ++h)
            for (int s = 0; s < kSlabs; ++s)
              for (int c = 0; c < kRep; ++c)
                tma_load_3d(sb + h * kTile + s * 16384 + c * kCopy * 128, &maps.q, bar(bQ), 64 * s, run.hk * p.G,
                            run.t0 + (run.tile * kHalves + h) * mtok);
        }
      }
      for (int k0 = run.k0; k0 < run.k1; k0 += kBN, ++kt) {
        const int st = ring.st;
        const int used = min(boxes, (run.k1 - k0 + box_rows - 1) / box_rows);
        const long long row = next;
        next = row_at(k0 + kBN);
        if (kt >= stages && !(ok = wait(b_free + st, ring.turn ^ 1))) break;
        if (lane == 0) mbar_arrive_expect_tx(bar(b_full + st), used * box_rows * 128 * kSlabs);
        __syncwarp();
        if (lane < used)
          for (int s = 0; s < kSlabs; ++s)
            tma_load_3d(sb + s_at + st * kTile + s * 16384 + lane * box_rows * 128, map, bar(b_full + st), 64 * s,
                        run.hk, (int)row, policy);
        ring.next(stages);
      }
    }
    // no copy may be in flight when the block ends
    if (!is_v && rc > 0) mbar_wait(bar(bQ), (rc - 1) & 1, abort_flag, kWaitNs, false);
    for (int t = max(0, kt - stages); t < kt; ++t)
      mbar_wait(bar(b_full + t % stages), (t / stages) & 1, abort_flag, kWaitNs, false);
  } else if (warp == 9) {
    // -------------------------------------------------------------- MMA
    if (lane == 0) {
      constexpr uint32_t id_s = F8 ? idesc_e4m3(kBM, kBN, false) : idesc_bf16(kBM, kBN, false);
      constexpr uint32_t id_pv = F8 ? idesc_e4m3(kBM, kD, true) : idesc_bf16(kBM, kD, true);
      constexpr uint32_t id_rem = idesc_e5m2_e4m3(kBM, kD, true);
      auto wait = [&](int b, uint32_t parity) { return mbar_wait(bar(b), parity, abort_flag, kWaitNs); };
      bool ok = true;
      int rc = 0;
      uint32_t np[2] = {0, 0};  // weights taken per S buffer, mod 2
      Ring rs, rv;              // key tiles of the scores and of the products with V
      Run run;
      for (; ok && draft_run(p, list, u, u_end, w, run); ++rc) {
        const int steps = (run.k1 - run.k0 + kBN - 1) / kBN * kHalves;
        // S of the next step, in S buffer h
        auto scores = [&](int h) -> bool {
          if ((kHalves == 1 || h == 0) && !wait(bK + rs.st, rs.turn)) return false;
          tc_fence_after();
          const uint32_t k_at = sb + s_k + rs.st * kTile;
#pragma unroll
          for (int kk = 0; kk < 4 * kSlabs; ++kk) {  // 32 bytes of a row each
            const uint32_t o = (kk >> 2) * 16384 + (kk & 3) * 32;
            const uint64_t a = sdesc_sw128(sb + (kHalves == 2 ? h : 0) * kTile + o, 16, 1024);
            const uint64_t b = sdesc_sw128(k_at + o, 16, 1024);
            if (F8) mma_f8(tmem + h * 256, a, b, id_s, kk > 0 ? 1u : 0u);
            else mma_bf16(tmem + h * 256, a, b, id_s, kk > 0 ? 1u : 0u);
          }
          mma_commit(bar(bS + h));
          if (kHalves == 1 || h == 1) {
            mma_commit(bar(bKFree + rs.st));
            rs.next(stages_k);
          }
          return true;
        };
        // O += P V of step i, in S buffer h = i & 1
        auto products = [&](int i, int h) -> bool {
          if (!wait(bP + h, np[h])) return false;
          np[h] ^= 1;
          if ((kHalves == 1 || h == 0) && !wait(bV + rv.st, rv.turn)) return false;
          if (i < 2 && rc > 0 && !wait(bOFree + h, (rc - 1) & 1)) return false;
          tc_fence_after();
          const uint32_t v_at = sb + s_v + rv.st * kTile;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            // bf16: 16 keys each; codes: 32 keys each, the weights and then their remainders
            const uint32_t acc = (i >= 2 || kk > 0) ? 1u : 0u;
            const uint64_t b = sdesc_sw128(v_at + (F8 ? (kk & 3) * 4096 : kk * 2048), 16384, 1024);
            if (F8) mma_f8_ts(tmem + h * 256 + 128, tmem + h * 256 + kk * 8, b, kk < 4 ? id_pv : id_rem, acc);
            else mma_bf16_ts(tmem + h * 256 + 128, tmem + h * 256 + kk * 8, b, id_pv, acc);
          }
          if (kHalves == 1 || h == 1) {
            mma_commit(bar(bVFree + rv.st));
            rv.next(stages_v);
          }
          return true;
        };
        if (!(ok = wait(bQ, rc & 1))) break;
        ok = scores(0) && (steps < 2 || scores(1));
        for (int i = 0; i < steps && ok; i += 2) {
          ok = products(i, 0) && (i + 2 >= steps || scores(0));
          if (ok && i + 1 < steps) ok = products(i + 1, 1) && (i + 3 >= steps || scores(1));
        }
        if (!ok) break;
        // the second half had no step: its phase is waited for all the same
        if (steps == 1 && rc > 0 && !(ok = wait(bOFree + 1, (rc - 1) & 1))) break;
        mma_commit(bar(bQFree));
        mma_commit(bar(bO));
      }
      // every MMA issued here is complete before TMEM is freed
      mma_commit(bar(bDrain));
      mbar_wait(bar(bDrain), 0, abort_flag, kWaitNs, false);
    }
  } else {
    // -------------------------------------------------------------- softmax
    const int h = warp >> 2, row = (warp & 3) * 32 + lane;  // S buffer; its row = TMEM lane
    const int col0 = (warp & 3) * 32 / kCopy * kCols;       // the first key of this warp's copy
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_s = tl + h * 256, t_o = tl + h * 256 + 128;
    // keys behind the history are -inf before they are scaled, and -inf times 0 would be
    // NaN: a factor of 0 becomes 2^-140, which moves a score below 2^100 by less than 2^-40
    const float factor = p.scale * kLog2eD * (F8 ? p.descale[0] * p.descale[1] : 1.f);
    const float c = factor == 0.f ? 0x1p-140f : factor;
    auto wait = [&](int b, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, abort_flag, kWaitNs));
    };
    constexpr float kShift = F8 ? 6.f : 0.f;  // weights carry 2^kShift
    bool ok = true;
    uint32_t met = 0;
    auto meet = [&]() -> bool {  // all softmax warps
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bMerge));
      const uint32_t phase = met;
      met ^= 1;
      return wait(bMerge, phase);
    };
    uint32_t ns = 0;  // score tiles taken, mod 2
    int rc = 0, kt0 = 0;
    Run run;
    for (; ok && draft_run(p, list, u, u_end, w, run); ++rc) {
      const int tiles = (run.k1 - run.k0 + kBN - 1) / kBN, steps = tiles * kHalves;
      float m = -INFINITY, l = 0.f;
      for (int i = h; i < steps; i += 2) {
        const int kt = tile_of(i), left = run.k1 - run.k0 - kt * kBN;
        if (!(ok = wait(bS + h, ns))) break;
        ns ^= 1;
        tc_fence_after();
        uint32_t sr[kCols];
        if constexpr (kCols == 128) tmem_ld128(t_s, sr);
        else if constexpr (kCols == 64) tmem_ld64(t_s + col0, sr);
        else tmem_ld32(t_s + col0, sr);
        if (left < kBN) {
#pragma unroll
          for (int j = 0; j < kCols; ++j)
            if (col0 + j >= left) sr[j] = 0xff800000u;  // -inf
          if (opens(i)) {
            // V rows behind the history: zero, whatever was there
            const int st = (kt0 + kt) % stages_v;
            if (!(ok = wait(bV + st, ((kt0 + kt) / stages_v) & 1))) break;
            for (int e = left * 8 + (tid & 127); e < kBN * 8; e += 128) {
              uint4 *z = reinterpret_cast<uint4 *>(smem + s_v + st * kTile) + e;
              z[0] = make_uint4(0u, 0u, 0u, 0u);
              if (kSlabs == 2) z[1024] = make_uint4(0u, 0u, 0u, 0u);  // the upper 64 elements
            }
            fence_proxy_async_smem();
          }
        }
        // row max: 8 chains of three-input max
        float mx[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mx[k] = __uint_as_float(sr[k]);
#pragma unroll
        for (int j = 8; j < kCols; j += 8) {
#pragma unroll
          for (int k = 0; k < 8; k += 2) {
            const int o = (j / 8 & 1) * 4 + k / 2;
            mx[o] = fmax3f(mx[o], __uint_as_float(sr[j + k]), __uint_as_float(sr[j + k + 1]));
          }
        }
        const float mt = c * fmaxf(fmax3f(mx[0], mx[1], mx[2]), fmax3f(fmax3f(mx[3], mx[4], mx[5]), mx[6], mx[7]));
        if (i < 2) {
          m = mt;
        } else if (__any_sync(0xffffffffu, mt > m + (F8 ? 2.75f : 8.f))) {
          // this buffer's last PV is complete: it was issued before this S
          const float mn = fmaxf(m, mt), f = mn == -INFINITY ? 1.f : exp2f(m - mn);
#pragma unroll 1
          for (int c4 = 0; c4 < kD / 32; ++c4) {
            uint32_t r32[32];
            tmem_ld32(t_o + 32 * c4, r32);
#pragma unroll
            for (int j = 0; j < 32; ++j) r32[j] = __float_as_uint(__uint_as_float(r32[j]) * f);
            tmem_st32(t_o + 32 * c4, r32);
          }
          l *= f;
          m = mn;
        }
        const float ref = (m == -INFINITY ? 0.f : m) - kShift;
        const uint64_t c2 = f2_pack(c, c), nm2 = f2_pack(-ref, -ref);
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
        uint32_t rem[F8 ? kCols / 4 : 1];
        constexpr int kWords = F8 ? kCols / 4 : kCols / 2;  // of packed weights (codes: and as many of remainders)
        if constexpr (F8) {
#pragma unroll
          for (int j = 0; j < kCols; j += 4) {
            float e[4];
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[j + k]), __uint_as_float(sr[j + k + 1])), c2, nm2), e[k],
                        e[k + 1]);
              e[k] = ex2_approx(e[k]);
              e[k + 1] = ex2_approx(e[k + 1]);
              acc[(j + k) / 2 & 3] = f2_add(acc[(j + k) / 2 & 3], f2_pack(e[k], e[k + 1]));
            }
            const uint32_t code = pack_e4m3x4(e[0], e[1], e[2], e[3]);
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const uint32_t pair = e4m3x2_to_half2(k ? code >> 16 : code);
              const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&pair));
              e[k] -= f.x;
              e[k + 1] -= f.y;
            }
            // words of codes take the places of scores that were read: j / 4 < j
            const uint32_t rest = pack_e5m2x4(e[0], e[1], e[2], e[3]);
            sr[j / 4] = code;
            rem[j / 4] = rest;
          }
        } else {
#pragma unroll
          for (int j = 0; j < kCols; j += 2) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[j]), __uint_as_float(sr[j + 1])), c2, nm2), x0, x1);
            const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
            acc[(j >> 1) & 3] = f2_add(acc[(j >> 1) & 3], f2_pack(e0, e1));
            sr[j >> 1] = pack_bf16x2(e0, e1);
          }
        }
        {
          float a0, a1, b0, b1;
          f2_unpack(f2_add(acc[0], acc[1]), a0, a1);
          f2_unpack(f2_add(acc[2], acc[3]), b0, b1);
          l += (a0 + a1) + (b0 + b1);
        }
        if constexpr (kCols == 128 && !F8) {
          tmem_st64(t_s, *reinterpret_cast<uint32_t(*)[64]>(sr));
        } else {  // the other copies' keys: weight 0
          uint32_t all[64];
          const int mine = col0 / kCols;
#pragma unroll
          for (int j = 0; j < 64; ++j) {
            const int k = F8 ? j % 32 : j;
            const uint32_t v = F8 && j >= 32 ? rem[k % kWords] : sr[k % kWords];
            all[j] = k / kWords == mine ? v : 0u;
          }
          tmem_st64(t_s, all);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bP + h));
      }
      if (!ok || !(ok = wait(bO, rc & 1))) break;
      tc_fence_after();
      // the rows with tokens of the request
      const int limit = min(real, run.tokens * p.G - run.tile * p.tile_rows - (kHalves == 2 ? h * real : 0));
      if constexpr (kRep == 1) {
        // the partial's rows, 128 bytes of four rows a store: eight lanes exchange
        // their rows' 16-byte words (lane j takes word j of each), because a lane
        // writing its own row touches 32 lines a store (6.4K cycles a run)
        const size_t at = (size_t)(2 * run.slot + h) * real;
        const int l8 = lane & 7;
#pragma unroll 1
        for (int c4 = 0; c4 < kD / 32 && h < steps; ++c4) {
          uint32_t r32[32];
          tmem_ld32(t_o + 32 * c4, r32);
#pragma unroll
          for (int s = 4; s > 0; s >>= 1) {
            const bool up = l8 & s;
#pragma unroll
            for (int a = 0; a < 8; ++a) {
              if (a & s) continue;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t &lo = r32[4 * a + k], &hi = r32[4 * (a | s) + k];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, s);
                if (up) lo = got; else hi = got;
              }
            }
          }
#pragma unroll
          for (int a = 0; a < 8; ++a) {
            const int r = row - l8 + a;
            if (r % kCopy < limit)
              *reinterpret_cast<uint4 *>(p.part_o + (at + r) * kD + 32 * c4 + 4 * l8) =
                  make_uint4(r32[4 * a], r32[4 * a + 1], r32[4 * a + 2], r32[4 * a + 3]);
          }
        }
        if (row % kCopy < limit) *reinterpret_cast<float2 *>(p.part_ml + 2 * (at + row)) = make_float2(m - kShift, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bOFree + h));
      } else {
        // The copies' results become one.  A warp adds the two S buffers' (both are its
        // TMEM lanes), in one half of the columns; the kRep warps that share a row
        // there then add a chunk of columns each to the buffer in shared memory and
        // move on to the next, so every sum has one order.
        constexpr int kChunk = kD / 2 / kRep, kLine = kD + 4;
        static_assert(kChunk == 16 || kChunk == 32, "columns of a TMEM load");
        const int mine = row / kCopy, r = row % kCopy, wid = warp;
        float *buf = reinterpret_cast<float *>(smem + s_m), *st_m = buf + kCopy * kLine, *st_l = st_m + 256;
        if (h >= steps) m = -INFINITY;
        st_m[wid * 32 + lane] = m - kShift;
        st_l[wid * 32 + lane] = l;
        if (!(ok = meet())) break;
        float top = -INFINITY, all = 0.f;
#pragma unroll
        for (int k = 0; k < 2 * kRep; ++k) {  // S buffer k / kRep, this row's quadrant of copy k % kRep
          const int wk = (k / kRep) * 4 + (k % kRep) * (4 / kRep) + (warp & 3) % (4 / kRep);
          top = fmaxf(top, st_m[wk * 32 + lane]);
        }
#pragma unroll
        for (int k = 0; k < 2 * kRep; ++k) {
          const int wk = (k / kRep) * 4 + (k % kRep) * (4 / kRep) + (warp & 3) % (4 / kRep);
          all += st_l[wk * 32 + lane] * (top == -INFINITY ? 0.f : ex2_approx(st_m[wk * 32 + lane] - top));
        }
        float f[2];  // of this copy's O in each S buffer
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float mk = st_m[((warp & 3) + 4 * k) * 32 + lane];
          f[k] = mk == -INFINITY ? 0.f : ex2_approx(mk - top);
        }
#pragma unroll 1
        for (int k = 0; k < kRep && ok; ++k) {
          const int c0 = kD / 2 * h + (mine + k) % kRep * kChunk;
          uint32_t v[2][kChunk];
          if constexpr (kChunk == 16) {
            tmem_ld16(tl + 128 + c0, v[0]);
            tmem_ld16(tl + 384 + c0, v[1]);
          } else {
            tmem_ld32(tl + 128 + c0, v[0]);
            tmem_ld32(tl + 384 + c0, v[1]);
          }
          float4 *to = reinterpret_cast<float4 *>(buf + r * kLine + c0);
#pragma unroll
          for (int j = 0; j < kChunk / 4; ++j) {
            float o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              o[i] = f[0] * __uint_as_float(v[0][4 * j + i]);
              if (steps > 1) o[i] = fmaf(f[1], __uint_as_float(v[1][4 * j + i]), o[i]);  // (else never written)
            }
            const float4 was = k > 0 ? to[j] : make_float4(0.f, 0.f, 0.f, 0.f);
            to[j] = make_float4(was.x + o[0], was.y + o[1], was.z + o[2], was.w + o[3]);
          }
          ok = meet();
        }
        if (!ok) break;
        tc_fence_before();
        __syncwarp();
        if (lane < 2) mbar_arrive(bar(bOFree + lane));
        const size_t at = (size_t)run.slot * real;
        constexpr int kQuads = kD / 4;
        bool nan = false;
        for (int e = tid; e < kCopy * kQuads; e += 256)
          if (e / kQuads < limit) {
            const float4 o = *reinterpret_cast<const float4 *>(buf + e / kQuads * kLine + 4 * (e % kQuads));
            *reinterpret_cast<float4 *>(p.part_o + (at + e / kQuads) * kD + 4 * (e % kQuads)) = o;
            nan |= isnan(o.x) | isnan(o.y) | isnan(o.z) | isnan(o.w);
          }
        if (!F8 && __any_sync(0xffffffffu, nan)) {  // (codes have no infinity)
          // An infinite value times the weight 0 that other copies have for its key is NaN.
          // Where a column of the run's values holds infinities of one sign and no NaN,
          // that infinity is its sum.
          uint32_t seen = 0;  // the thread's columns: +inf bits 0 to 3, -inf 4 to 7, NaN 8 to 11
          const __nv_bfloat16 *col = static_cast<const __nv_bfloat16 *>(p.past_v) + run.hk * kD + 4 * (tid % kQuads);
#pragma unroll 1
          for (int key = run.k0; key < run.k1; key += 16) {  // (rows of a block come in sixteens)
            const long long from = history_row(x, p.hist, run.base, key);
            if (from < 0) continue;
            uint2 w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              w[j] = key + j < run.k1 ? *reinterpret_cast<const uint2 *>(col + (size_t)(from + j) * p.Hkv * kD)
                                      : make_uint2(0u, 0u);
#pragma unroll
            for (int j = 0; j < 16; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t v = (i < 2 ? w[j].x : w[j].y) >> 16 * (i & 1) & 0xffffu;
                if ((v & 0x7fffu) >= 0x7f80u) seen |= (v == 0x7f80u ? 1u : v == 0xff80u ? 16u : 256u) << i;
              }
          }
          for (int e = tid; e < kCopy * kQuads; e += 256)
            if (e / kQuads < limit)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t kind = seen >> i & 0x111u;
                if ((kind == 1u || kind == 16u) && isnan(buf[e / kQuads * kLine + 4 * (e % kQuads) + i]))
                  p.part_o[(at + e / kQuads) * kD + 4 * (e % kQuads) + i] = kind == 1u ? INFINITY : -INFINITY;
              }
        }
        if (h == 0 && mine == 0 && r < limit) *reinterpret_cast<float2 *>(p.part_ml + 2 * (at + r)) = make_float2(top, all);
      }
      kt0 += tiles;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (ms.abort && tid == 0) set_status(x.status, FLIDE_ERR_TIMEOUT);
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

EncodeFn encode_tiled() {
  static std::atomic<EncodeFn> cached{nullptr};  // host threads may race on a first call
  EncodeFn fn = cached.load(std::memory_order_acquire);
  if (!fn) {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      fn = (EncodeFn)ptr;
      cached.store(fn, std::memory_order_release);
    }
  }
  return fn;
}

// [rows, heads, d] bf16 or codes as (element, head, row); box of 128 swizzled
// bytes x box_heads x box_rows
bool wide_map(CUtensorMap *m, const void *base, int d, int esz, int heads, long rows, int box_heads, int box_rows) {
  EncodeFn enc = encode_tiled();
  if (!enc || rows <= 0) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * esz, (cuuint64_t)heads * d * esz};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / esz), (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t step[3] = {1, 1, 1};
  return enc(m, esz == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
             const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kD, int kHalves, int kRep, bool F8>
int wide_launch(const DraftParams &p, const WideMaps &maps, int mtok, int box_rows, int dev, cudaStream_t s) {
  constexpr int kTileBytes = kBN * kD * (F8 ? 1 : 2);
  int k = kMaxStages, v = kMaxStages;  // as many as fit, K's first
  while (k + v > kMinStages && wide_smem(kTileBytes, kD, kHalves, kRep, k + v, p.x.R) > kSmemMax) (k > v ? k : v)--;
  const size_t smem = wide_smem(kTileBytes, kD, kHalves, kRep, k + v, p.x.R);
  if (!allow_smem<draft_part_wide<kD, kHalves, kRep, F8>>(dev)) return FLIDE_ERR_CUDA;
  draft_part_wide<kD, kHalves, kRep, F8><<<p.workers, kWThreads, smem, s>>>(maps, p, mtok, box_rows, k, v);
  FLIDE_LAUNCH_CHECK();
  return FLIDE_OK;
}

}  // namespace

bool draft_wide_fits(int operand, int d, bool f8, long long R) {
  return wide_smem(kBN * d * (f8 ? 1 : 2), d, operand == 2 * kBM ? 2 : 1, operand < kBM ? kBM / operand : 1, kMinStages,
                   R) <= kSmemMax;
}

int draft_wide_launch(DraftParams &p, int operand, int past_rows, bool f8, int dev, cudaStream_t s) {
  p.unit = kBN;
  // key tiles that a run costs beside its own: about 11K cycles of 1.5K (codes),
  // 2.2K and (256 rows) 3.9K a tile
  p.extra = f8 ? 6 : operand == 2 * kBM ? 3 : 5;
  const int rep = operand < kBM ? kBM / operand : 1;
  const int mtok = kBM / rep / p.G, esz = f8 ? 1 : 2, d = p.d;
  // rows of a box: a tile's, or the most that divides both it and a block
  int box_rows = kBN;
  if (p.hist.block_table)
    while (p.hist.block_rows % box_rows) box_rows /= 2;
  WideMaps maps;
  const bool past = p.past_k != nullptr && past_rows > 0;  // without: no unit, no load
  if (!wide_map(&maps.q, p.q, d, esz, p.Hq, p.x.T, p.G, mtok) ||
      !wide_map(&maps.k, past ? p.past_k : p.k, d, esz, p.Hkv, past ? past_rows : p.x.T, 1, box_rows) ||
      !wide_map(&maps.v, past ? p.past_v : p.v, d, esz, p.Hkv, past ? past_rows : p.x.T, 1, box_rows))
    return FLIDE_ERR_CUDA;
  if (d == 64) {
    if (operand == 2 * kBM) return wide_launch<64, 2, 1, false>(p, maps, mtok, box_rows, dev, s);
    return rep == 2 ? wide_launch<64, 1, 2, false>(p, maps, mtok, box_rows, dev, s)
                    : wide_launch<64, 1, 1, false>(p, maps, mtok, box_rows, dev, s);
  }
  if (operand == 2 * kBM) return wide_launch<128, 2, 1, false>(p, maps, mtok, box_rows, dev, s);
  switch (rep) {
    case 4:
      return f8 ? wide_launch<128, 1, 4, true>(p, maps, mtok, box_rows, dev, s)
                : wide_launch<128, 1, 4, false>(p, maps, mtok, box_rows, dev, s);
    case 2:
      return f8 ? wide_launch<128, 1, 2, true>(p, maps, mtok, box_rows, dev, s)
                : wide_launch<128, 1, 2, false>(p, maps, mtok, box_rows, dev, s);
    default:
      return f8 ? wide_launch<128, 1, 1, true>(p, maps, mtok, box_rows, dev, s)
                : wide_launch<128, 1, 1, false>(p, maps, mtok, box_rows, dev, s);
  }
}

}  // namespace flide

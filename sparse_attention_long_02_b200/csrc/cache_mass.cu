// cache_mass.cu -- the attention weight each cached token receives, sm_100a.
//
// With lse[b,j,h] the natural log normaliser of query j, head h (as the
// attention returns it), key s of sequence b receives
//   w[b,s] = sum_{j,h: s <= pos_j} exp(sm_scale q[b,j,h] . kv[s] - lse[b,j,h])
// from the nq new tokens, pos_j = seq_len[b] - nq + j, and its running total
// becomes mass + w (w alone for the new tokens, which have no total yet).
//
// Keys sit on the MMA's M and queries x heads on N, so that the sum over them
// runs inside a thread: S^T = K Q^T (M = 128 keys, N = up to 128 rows, K = 576),
// thread = key. Every total belongs to one thread: no atomics, one order of
// addition. Q (one row tile, 144 KB) stays in shared memory for a CTA's piece of
// a sequence; K chunks (128 keys x 64 dims) stream through a ring of TMA loads
// into one of two TMEM buffers that two groups of four warps empty in turn. The
// tiles of all sequences are cut into equal shares, one a CTA; sequences with
// more than 128 rows of queries walk their piece once a row tile.
//
// Bound by HBM: 1152 bytes and 8 of the total a key; the tensor cores take 36
// MMAs of 64 cycles a 128-key tile, the exponentials 1024 cycles, an SM's share
// of the copy bandwidth about 6000. 64 x 32768 tokens take 423 to 435 us in 20 calls
// in a row (5.7 TB/s, 87% of the copy rate), and 475 us in a loop of seconds, which
// the board's 1000 W hold at 1.4 GHz (5.1 TB/s, 79%). (Asking L2 for tiles ahead of
// their loads made it slower, whatever the instruction: 413 us without when that was
// tried, 559 us one tile ahead, 700 us three ahead.)
//
// Precision. Products are exact and sums fp32, but the tensor core's additions cut
// where they do not round: a logit from a sum of about 100 comes out some 3e-6 too
// small, and so does its weight (relative; 2e-7 with products in fp32). Rounding lse
// to log2 units before the difference costs next to nothing beside that (scaled
// after it: 2.40e-6 instead of 2.43e-6, 1.86e-6 instead of 1.90e-6).
#include <algorithm>

#include "common.cuh"
#include "dsa_internal.h"
#include "split.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 384;
constexpr int kChunk = 128 * 128;               // 128 keys (or rows) x 64 dims
constexpr int kUnit = 64 * 128;
// Even, so that each of the two loading warps has its own places.
constexpr int kRing = 4;
constexpr int kCtas = 148;                      // one an SM

struct MassSmem {
  uint8_t q[9][kChunk];
  uint8_t k[kRing][kChunk];
  // each warp's own copy, so that none waits for another
  float lse2[8][128];                           // the rows' normalisers in log2 units
  int pos[8][128];                              // the rows' positions, -1: gives nothing
  Share share;
  long long sums[2 * (kThreads / 32)];
  unsigned long long q_full, q_free;
  unsigned long long k_full[kRing], k_empty[kRing];
  unsigned long long s_full[2], s_empty[2];
  unsigned long long done;                      // completes only in the give-up path
  uint32_t tmem_base;
  int abort_flag[2];                            // (no wait is for more than a tile: [1] stays 0)
};
static_assert(sizeof(MassSmem) + 1024 <= 232448, "fits the 227 KB of shared memory a CTA may use");

__device__ __forceinline__ int seq_tokens(const MassArgs& A, int b) {
  return max(0, min(A.seq_len[b], A.max_blocks * 64));
}

// A CTA's share, a piece (128-key tiles [t0, t1) of a sequence) after another.
struct MassWalk {
  int item, off;
  long long left;
  int b, len, t0, t1;                           // the piece
  __device__ __forceinline__ explicit MassWalk(const Share& s)
      : item(s.item), off(s.off), left(s.left) {}
  __device__ __forceinline__ bool next(const MassArgs& A) {
    while (left > 0 && item < A.B) {
      len = seq_tokens(A, item);
      const int tiles = (len + 127) >> 7;
      const int take = static_cast<int>(min(static_cast<long long>(tiles - off), left));
      b = item++;
      t0 = off;
      t1 = off + take;
      left -= take;
      off = 0;
      if (take > 0) return true;
    }
    return false;
  }
};

__global__ void __launch_bounds__(kThreads, 1)
mass_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ MassArgs A) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  MassSmem& sm = *reinterpret_cast<MassSmem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned* err = A.err;
  const int warp = warp_id(), lane = lane_id();
  find_share<kThreads>(sm.share, sm.sums, A.B, static_cast<int>(blockIdx.x),
                       static_cast<int>(gridDim.x), 0, [&](int b) {
                         const int len = A.seq_len[b];
                         if (blockIdx.x == 0 && (len < 0 || len > A.max_blocks * 64))
                           raise_error(err, kErrBounds);
                         return (seq_tokens(A, b) + 127) >> 7;
                       });
  if (threadIdx.x == 0) {
    auto init = [](unsigned long long& b, int count) { mbar_init(smem_u32(&b), count); };
    init(sm.q_full, 1);
    init(sm.q_free, 1);
    init(sm.done, 1);
    for (int i = 0; i < kRing; ++i) {
      init(sm.k_full[i], 1);
      init(sm.k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      init(sm.s_full[i], 1);
      init(sm.s_empty[i], 4);
    }
    sm.abort_flag[0] = launch_aborted(err) ? 1 : 0;
    sm.abort_flag[1] = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sm.tmem_base), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = sm.abort_flag;
  MassWalk walk(sm.share);
  bool ok = *abort_flag == 0;

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------ Q and K loads
    const int par = warp >> 1;
    if (lane == 0) {
      int ent = 0, passes = 0, q_loads = 0;
      const uint32_t q_bytes = 9u * static_cast<uint32_t>(A.box_rows) * 128u;
      while (ok && walk.next(A)) {
        const int* table = A.block_table + static_cast<long long>(walk.b) * A.max_blocks;
        const int units = (walk.len + 63) >> 6;
        auto entry = [&](int u) { return u < units ? __ldg(table + u) : -1; };
        auto row_of = [&](int e) { return e < 0 || e >= A.nblk ? A.kv_rows : e * 64; };
        for (int rt = 0; ok && rt < A.per_seq; ++rt, ++passes) {
          if (par == 0) {
            if (passes > 0 && !(ok = wait1(sm.q_free, (passes - 1) & 1, abort_flag, err))) break;
            const int q_row = (walk.b * A.nq + rt * A.G) * A.H;
            mbar_expect_tx(smem_u32(&sm.q_full), q_bytes);
            for (int a = 0; a < 9; ++a)
              tma_load_2d(smem_u32(sm.q[a]), &tm_q, smem_u32(&sm.q_full), 64 * a, q_row);
            ++q_loads;
          }
          int e0 = entry(2 * walk.t0), e1 = entry(2 * walk.t0 + 1);
          for (int t = walk.t0; ok && t < walk.t1; ++t) {
            // table entries are loaded a tile before they are used
            const int c0 = row_of(e0), c1 = row_of(e1);
            e0 = entry(2 * t + 2);
            e1 = entry(2 * t + 3);
#pragma unroll 1
            for (int ch = 0; ch < 9; ++ch, ++ent) {
              if ((ent & 1) != par) continue;
              const int st = ent & (kRing - 1);
              if (ent >= kRing &&
                  !(ok = wait1(sm.k_empty[st], (ent / kRing + 1) & 1, abort_flag, err)))
                break;
              const uint32_t full = smem_u32(&sm.k_full[st]);
              mbar_expect_tx(full, kChunk);
              tma_load_3d(smem_u32(sm.k[st]), &tm_k, full, 0, c0, ch);
              tma_load_3d(smem_u32(sm.k[st] + kUnit), &tm_k, full, 0, c1, ch);
            }
          }
        }
      }
      if (!ok) {             // let the loads in flight land before this CTA leaves
        for (int c = max(0, ent - kRing); c < ent; ++c)
          if ((c & 1) == par) mbar_drain(smem_u32(&sm.k_full[c & (kRing - 1)]), (c / kRing) & 1);
        if (q_loads > 0) mbar_drain(smem_u32(&sm.q_full), (q_loads - 1) & 1);
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------------------- MMAs
    // N: the rows of a full row tile, in sixteens (rows past a tile's own are
    // other queries' or zeros, and their columns are not read)
    const uint32_t id = idesc_bf16(128, (A.G * A.H + 15) / 16 * 16, false);
    const uint64_t q_d = sdesc_sw128(smem_u32(sm.q[0]), 0, 1024);
    const uint64_t k_d = sdesc_sw128(smem_u32(sm.k[0]), 0, 1024);
    int ent = 0, passes = 0;
    unsigned uses = 0;                            // parity of each buffer's uses
    unsigned used = 0;                            // buffers used at all
    while (ok && walk.next(A)) {
      for (int rt = 0; ok && rt < A.per_seq; ++rt, ++passes) {
        if (!(ok = wait32(sm.q_full, passes & 1, abort_flag, err))) break;
        for (int t = walk.t0; ok && t < walk.t1; ++t) {
          const int g = t & 1;
          if (((used >> g) & 1) &&
              !(ok = wait32(sm.s_empty[g], ((uses >> g) & 1) ^ 1, abort_flag, err)))
            break;
          used |= 1u << g;
          uses ^= 1u << g;
          tc_fence_after();
          const uint32_t d = tmem + 128 * g;
          bool there = mbar_try_wait(smem_u32(&sm.k_full[ent & (kRing - 1)]), (ent / kRing) & 1);
#pragma unroll 1
          for (int ch = 0; ch < 9; ++ch, ++ent) {
            const int st = ent & (kRing - 1);
            if (!__all_sync(0xffffffffu, there) &&
                !(ok = wait32(sm.k_full[st], (ent / kRing) & 1, abort_flag, err)))
              break;
            there = mbar_try_wait(smem_u32(&sm.k_full[(ent + 1) & (kRing - 1)]),
                                  ((ent + 1) / kRing) & 1);
            const uint64_t kd = k_d + st * (kChunk >> 4), qd = q_d + ch * (kChunk >> 4);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_bf16(d, kd + 2 * kk, qd + 2 * kk, id, (ch > 0 || kk > 0) ? 1u : 0u);
              mma_commit(smem_u32(&sm.k_empty[st]));
              if (ch == 8) {
                mma_commit(smem_u32(&sm.s_full[g]));
                if (t + 1 == walk.t1) mma_commit(smem_u32(&sm.q_free));
              }
            }
            __syncwarp();
          }
        }
      }
    }
    if (!ok) {               // MMAs in flight read shared memory: wait for them
      if (elect_one()) {
        mma_commit(smem_u32(&sm.done));
        mbar_drain(smem_u32(&sm.done), 0);
      }
      __syncwarp();
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------- the weights
    const int g = (warp - 4) >> 2;                // takes the tiles of its parity
    const int key = 32 * (warp & 3) + lane;       // of a tile = TMEM lane
    const uint32_t s_cols = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + 128 * g;
    float* lse2 = sm.lse2[warp - 4];
    int* pos = sm.pos[warp - 4];
    unsigned uses = 0;
    while (ok && walk.next(A)) {
      const int* table = A.block_table + static_cast<long long>(walk.b) * A.max_blocks;
      float* mass = A.mass + walk.b * A.ld;
      for (int rt = 0; ok && rt < A.per_seq; ++rt) {
        // The rows' normalisers and positions. Columns past the rows hold
        // other queries or nothing, and a row without a normaliser gives
        // nothing; `whole` marks the 32s that have neither.
        const int nrows = min(A.G, A.nq - rt * A.G) * A.H;
        const int pos0 = walk.len - A.nq + rt * A.G;
        const long long row0 = (static_cast<long long>(walk.b) * A.nq + rt * A.G) * A.H;
        unsigned whole = 0;
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = 32 * k + lane;
          const float l = c < nrows ? A.lse[row0 + c] : -INFINITY;
          lse2[c] = l * 1.4426950408889634f;
          pos[c] = l == -INFINITY ? -1 : pos0 + c / A.H;
          if (__all_sync(0xffffffffu, l != -INFINITY)) whole |= 1u << k;
        }
        __syncwarp();
        for (int t = walk.t0; ok && t < walk.t1; ++t) {
          if ((t & 1) != g) continue;
          const int s = 128 * t + key;
          bool good = s < walk.len;
          if (good) {
            const int pb = __ldg(table + (s >> 6));
            if (pb < 0 || pb >= A.nblk) {
              good = false;
              raise_error(err, kErrBounds);
            }
          }
          float total = 0.f;
          if (good && (rt > 0 || s < walk.len - A.nq)) total = mass[s];
          if (!(ok = wait32(sm.s_full[g], uses, abort_flag, err))) break;
          uses ^= 1u;
          tc_fence_after();
          float w[4] = {0.f, 0.f, 0.f, 0.f};
          const bool all = 128 * t + 127 <= pos0;   // every row's query sees the tile
#pragma unroll 1
          for (int c = 0; c < nrows; c += 32) {
            float z[32];
            tmem_ld32(s_cols + c, z);
            if (all && ((whole >> (c >> 5)) & 1u)) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                w[e & 3] += fast_exp2(fmaf(z[e], A.sm_scale_log2, -lse2[c + e]));
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (s <= pos[c + e])
                  w[e & 3] += fast_exp2(fmaf(z[e], A.sm_scale_log2, -lse2[c + e]));
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.s_empty[g]));
          if (good) mass[s] = total + ((w[0] + w[1]) + (w[2] + w[3]));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

}  // namespace

cudaError_t launch_attention_mass(const MassArgs& a_in, cudaStream_t st) {
  MassArgs a = a_in;
  a.G = std::max(1, std::min(a.nq, 128 / a.H));
  a.per_seq = (a.nq + a.G - 1) / a.G;
  a.kv_rows = a.nblk * 64;
  a.box_rows = (a.G * a.H + 15) / 16 * 16;
  CUtensorMap tq, tk;
  cudaError_t e = make_tmap_2d(&tq, a.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 576,
                               static_cast<uint64_t>(a.B) * a.nq * a.H, 576 * 2, 64, a.box_rows,
                               CU_TENSOR_MAP_SWIZZLE_128B);
  if (e == cudaSuccess) e = make_tmap_chunks(&tk, a.kv, a.kv_rows, 64, 1);
  if (e != cudaSuccess) return e;
  const size_t smem = sizeof(MassSmem) + 1024;
  e = cudaFuncSetAttribute(mass_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>(a.B) * ((a.max_blocks + 1) / 2);
  mass_kernel<<<static_cast<int>(std::min<long long>(kCtas, tiles)), kThreads, smem, st>>>(tq, tk,
                                                                                           a);
  return cudaGetLastError();
}

}  // namespace dsa

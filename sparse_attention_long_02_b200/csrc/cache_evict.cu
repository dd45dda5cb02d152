// cache_evict.cu -- eviction from the paged cache by accumulated attention
// weight, sm_100a.
//
// A sequence of n > budget tokens keeps its first `sinks` tokens, its last
// `recent` ones and, of the rest, the budget - sinks - recent of the largest
// running totals (ties to the smaller slot). The kept rows move, in order, to
// the sequence's slots 0 .. budget-1, in place.
//
// evict_select_kernel, one CTA per sequence: a radix select (four 8-bit
// digits) of the threshold total, then one ordered pass that writes the kept
// slots. evict_move_kernel: a row's destination is never behind its source
// slot, so a CTA that walks the kept rows in order, reading a chunk of rows
// before it writes them, never overwrites a row it has still to read. The
// bytes of a row are split over CTAs by column, each CTA moving its columns of
// every row: no CTA reads what another one writes.
#include "common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 512;

// Order-preserving key of a total; NaN below everything, -0 equal to +0.
__device__ __forceinline__ unsigned total_key(float v) {
  if (!(v == v)) return 0u;
  const unsigned u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of v over the block, total in *sum.
__device__ __forceinline__ int block_prefix(int v, int* warp_sums, int* sum) {
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane_id() >= o) x += y;
  }
  if (lane_id() == 31) warp_sums[warp_id()] = x;
  __syncthreads();
  if (warp_id() == 0) {
    int w = warp_sums[lane_id()];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane_id() >= o) w += y;
    }
    warp_sums[lane_id()] = w;
  }
  __syncthreads();
  const int before = warp_id() ? warp_sums[warp_id() - 1] : 0;
  *sum = warp_sums[31];
  __syncthreads();
  return before + x - v;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs A) {
  __shared__ unsigned hist[256];
  __shared__ unsigned s_prefix, s_want;
  __shared__ int warp_sums[32];
  const int b = static_cast<int>(blockIdx.x);
  const int tid = static_cast<int>(threadIdx.x);
  const int raw = A.seq_len[b];
  if (tid == 0 && (raw < 0 || raw > A.max_blocks * 64)) raise_error(A.err, kErrBounds);
  const int n = max(0, min(raw, A.max_blocks * 64));
  int* idx = A.idx + static_cast<long long>(b) * A.budget;
  __syncthreads();
  if (tid == 0) A.seq_len_out[b] = min(n, A.budget);
  if (n <= A.budget) {
    for (int i = tid; i < A.budget; i += kSelThreads) idx[i] = i < n ? i : -1;
    return;
  }
  const float* mass = A.mass + b * A.ld;
  const int lo = A.sinks, hi = n - A.recent;      // candidates
  const int want = A.budget - A.sinks - A.recent;
  // threshold: the want-th largest key; `ties` of the keys equal to it are kept
  unsigned thr = 0xffffffffu;
  int ties = 0;
  if (want > 0) {
    unsigned prefix = 0, left = want;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int i = lo + tid; i < hi; i += kSelThreads) {
        const unsigned k = total_key(mass[i]);
        if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        unsigned w = left;
        int d = 255;
        for (; d > 0 && hist[d] < w; --d) w -= hist[d];
        s_prefix = (prefix << 8) | static_cast<unsigned>(d);
        s_want = w;
      }
      __syncthreads();
      prefix = s_prefix;
      left = s_want;
      __syncthreads();
    }
    thr = prefix;
    ties = static_cast<int>(left);
  }
  int out = 0, eq_before = 0;
  for (int i0 = 0; i0 < n; i0 += kSelThreads) {
    const int i = i0 + tid;
    bool above = false, eq = false;
    if (i < n) {
      if (i < lo || i >= hi) {
        above = true;
      } else if (want > 0) {
        const unsigned k = total_key(mass[i]);
        above = k > thr;
        eq = k == thr;
      }
    }
    int neq, nkeep;
    const int rank = eq_before + block_prefix(eq, warp_sums, &neq);
    const bool keep = above || (eq && rank < ties);
    const int at = out + block_prefix(keep, warp_sums, &nkeep);
    if (keep) idx[at] = i;
    out += nkeep;
    eq_before += neq;
  }
}

// One column slice of one sequence: `width` bytes of every row of a pool
// (rows of `pitch` bytes), kMoveThreads / (width / 4) rows a step.
template <typename V>
__device__ __forceinline__ void move_columns(const EvictArgs& A, int b, int count, V* pool,
                                             int pitch_v, int cols_v, int first_v) {
  const int rows = kMoveThreads / cols_v;
  const int col = static_cast<int>(threadIdx.x) % cols_v, sub = static_cast<int>(threadIdx.x) / cols_v;
  const int* idx = A.idx + static_cast<long long>(b) * A.budget;
  const int* table = A.block_table + static_cast<long long>(b) * A.max_blocks;
  auto row = [&](int s) -> long long {
    const int pb = table[s >> 6];
    return pb < 0 || pb >= A.nblk ? -1 : static_cast<long long>(pb) * 64 + (s & 63);
  };
  for (int j0 = 0; j0 < count; j0 += rows) {
    const int j = j0 + sub;
    V v = {};
    long long to = -1;
    if (sub < rows && j < count && idx[j] != j) {
      const long long from = row(idx[j]);
      to = row(j);
      if (from < 0 || to < 0) {
        raise_error(A.err, kErrBounds);
        to = -1;
      } else {
        v = pool[from * pitch_v + first_v + col];
      }
    }
    __syncthreads();
    if (to >= 0) pool[to * pitch_v + first_v + col] = v;
  }
}

constexpr int kKvSlices = 9;       // 128 bytes of the latent row each

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs A) {
  const int b = static_cast<int>(blockIdx.y);
  const int slice = static_cast<int>(blockIdx.x);
  const int count = A.seq_len_out[b];
  if (slice < kKvSlices) {
    move_columns(A, b, count, static_cast<uint4*>(A.kv_pool), 72, 8, 8 * slice);
  } else if (slice == kKvSlices) {
    if (A.k8_pool) move_columns(A, b, count, static_cast<uint4*>(A.k8_pool), 8, 8, 0);
  } else if (slice == kKvSlices + 1) {
    if (A.k_scale_pool) move_columns(A, b, count, A.k_scale_pool, 1, 1, 0);
  } else if (A.mass_out) {
    const int* idx = A.idx + static_cast<long long>(b) * A.budget;
    for (int j0 = 0; j0 < count; j0 += kMoveThreads) {
      const int j = j0 + static_cast<int>(threadIdx.x);
      const float v = j < count ? A.mass[b * A.ld + idx[j]] : 0.f;
      __syncthreads();
      if (j < count) A.mass_out[b * A.ld_out + j] = v;
    }
  }
}

}  // namespace

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t st) {
  evict_select_kernel<<<a.B, kSelThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  evict_move_kernel<<<dim3(kKvSlices + 3, a.B), kMoveThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace dsa

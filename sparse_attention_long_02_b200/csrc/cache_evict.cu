// cache_evict.cu -- eviction from the paged cache by accumulated attention
// weight, sm_100a.
//
// A sequence of n > budget tokens keeps its first `sinks` tokens, its last
// `recent` ones and, of the rest, the budget - sinks - recent of the largest
// running totals (ties to the smaller slot). The kept rows move, in order, to
// the sequence's slots 0 .. budget-1, in place.
//
// evict_select_kernel, a cluster of 1 to 8 CTAs per sequence: a radix select
// (11 + 11 + 10 bits) of the threshold total over the CTAs' histograms, of which
// one warp reads, through distributed shared memory, first the sums of 64 bins
// and then the 64 bins that matter. It runs each of its instructions a few times
// only and is bound by latency, that of its own code among them: loops are kept
// short and rolled (with the keys in registers and the loops over them unrolled 16
// times a call over one sequence of 131072 tokens, move included, took 74 us where
// it took 66 then; it takes 60 now). With `ties` the number of totals equal to the
// threshold that are kept, slot i's place is
//   (kept for certain before i) + min(ties, equal before i),
// so one counting pass and one writing pass over each warp's own run of slots
// give the kept slots in order without a scan per step.
//
// evict_move_kernel: a row's destination is never behind its source slot, so a
// walk over the kept rows in order that reads a step's rows before it writes them
// never overwrites a row it has still to read, nor one of later steps, which it
// may read ahead. A cluster of up to 8 CTAs walks a sequence, its rows split over
// them, with the cluster's barrier between a step's reads and its writes. Where
// there are few sequences the bytes of a row are split by column too, each slice
// moved by a cluster of its own: none reads what another slice's write. Bound by
// HBM, each moved byte read and written once (64 x 32768 -> 16384 tokens: 481 us
// with the selection, 5.6 TB/s), and for few sequences by the latency of a step's
// chain (read, barrier, write).
//
// A pending timeout (of this or another stream) leaves a sequence as it is. The
// selection alone looks at the error word, which other streams may set and clear
// at any time, and leaves a verdict for each sequence that all CTAs of the move
// obey: a sequence is evicted as a whole or not at all.
#include <atomic>

#include "common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelKeys = 40960;                 // keys a CTA keeps in shared memory
constexpr int kBins = 2048;
// Two CTAs of 1024 threads fit an SM. (64 x 32768 -> 16384 took 519 us with 512
// threads, two rows a thread and four steps, 556 us with 1024, two and three.)
constexpr int kMoveThreads = 1024;
constexpr int kDepth = 3;                       // steps of a move in shared memory
constexpr int kMoveWant = 256, kMoveMost = 296; // CTAs that move latent rows, at least and at most

// A call's verdicts, a byte a sequence: its place in the list of eager calls or of
// captured ones, which are launched again later. Two calls share a place only with
// a million sequences between them, and then must run at the same time, with a
// timeout set or cleared between their selections, for one to read the other's.
constexpr unsigned kVerdicts = 1u << 20;
__device__ unsigned char g_verdict[2][kVerdicts];
struct Verdicts {
  unsigned list, first;
  __device__ __forceinline__ unsigned char& of(int b) const {
    return g_verdict[list][(first + static_cast<unsigned>(b)) & (kVerdicts - 1)];
  }
};

// Order-preserving key of a total; NaN below everything, -0 equal to +0.
__device__ __forceinline__ unsigned total_key(float v) {
  if (!(v == v)) return 0u;
  const unsigned u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct SelSmem {
  unsigned hist[4][kBins];                      // by lane % 4
  unsigned bins[2][kBins];                      // the CTA's sums, by pass parity
  unsigned coarse[2][kSelWarps];                // and those of 64 bins
  int warp_above[kSelWarps], warp_eq[kSelWarps];
  int above, eq;                                // the CTA's counts
  unsigned digit, left;
  unsigned skip;                                // a timeout is recorded: do nothing
};

__device__ __forceinline__ unsigned cluster_size() {
  unsigned n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
__device__ __forceinline__ unsigned ld_cluster(uint32_t addr) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Inclusive sum over the lanes from this one up.
__device__ __forceinline__ unsigned sum_from_lane(unsigned x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_down_sync(0xffffffffu, x, o);
    if (lane_id() + o < 32) x += y;
  }
  return x;
}

__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const EvictArgs A, const Verdicts verdicts) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SelSmem& sm = *reinterpret_cast<SelSmem*>(smem_raw);
  unsigned* kept_keys = reinterpret_cast<unsigned*>(smem_raw + sizeof(SelSmem));
  const int cl = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int b = static_cast<int>(blockIdx.x) / cl;
  const int tid = static_cast<int>(threadIdx.x), warp = warp_id(), lane = lane_id();
  const int raw = A.seq_len[b];
  const int n = max(0, min(raw, A.max_blocks * 64));
  int* idx = A.idx + static_cast<long long>(b) * A.budget;
  if (tid == 0) sm.skip = launch_aborted(A.err);
  cluster_sync();                               // also: seq_len_out may be seq_len
  const bool skip = ld_cluster(mapa(smem_u32(&sm.skip), 0)) != 0;
  if (rank == 0 && tid == 0) verdicts.of(b) = !skip;
  if (skip) {
    cluster_sync();
    return;
  }
  if (rank == 0 && tid == 0) {
    if (raw != n) raise_error(A.err, kErrBounds);
    A.seq_len_out[b] = min(n, A.budget);
  }
  if (n <= A.budget) {
    // (unsigned: a budget of no limit is near 2^31)
    for (unsigned i = rank * kSelThreads + tid; i < static_cast<unsigned>(A.budget);
         i += cl * kSelThreads)
      idx[i] = i < static_cast<unsigned>(n) ? static_cast<int>(i) : -1;
    cluster_sync();                             // the others may still read sm.skip
    return;
  }
  const float* mass = A.mass + b * A.ld;
  const int lo = A.sinks, hi = n - A.recent;    // candidates
  const int want = A.budget - A.sinks - A.recent;
  // each warp of the cluster has a run of `seg` slots, each CTA 32 such runs
  const int warps = cl * kSelWarps;
  const int seg = ((n + warps - 1) / warps + 31) / 32 * 32;
  const int base = min(n, rank * kSelWarps * seg), end = min(n, base + kSelWarps * seg);
  const int s0 = min(n, base + warp * seg), s1 = min(n, s0 + seg);      // the warp's run
  const bool in_smem = kSelWarps * seg <= kSelKeys;
  auto key = [&](int i) { return in_smem ? kept_keys[i - base] : total_key(__ldg(mass + i)); };
  if (in_smem) {
#pragma unroll 8
    for (int i = base + tid; i < end; i += kSelThreads)
      kept_keys[i - base] = total_key(__ldg(mass + i));
  }
  // threshold: the want-th largest key of the candidates; `ties` of the keys
  // equal to it are kept
  unsigned thr = 0xffffffffu;
  int ties = 0;
  if (want > 0) {
    for (int i = tid; i < 4 * kBins; i += kSelThreads) (&sm.hist[0][0])[i] = 0;
    __syncthreads();
    unsigned prefix = 0, left = static_cast<unsigned>(want);
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      const unsigned mask = (1u << bits) - 1;
      unsigned* hist = sm.hist[lane & 3];
#pragma unroll 1
      for (int i = max(s0, lo) + lane; i < min(s1, hi); i += 32) {
        const unsigned x = key(i);
        if (pass == 0 || (x >> (shift + bits)) == prefix)
          atomicAdd(hist + ((x >> shift) & mask), 1u);
      }
      __syncthreads();
      // this thread's two bins: added up, and empty again for the next pass
      unsigned two[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        two[e] = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          two[e] += sm.hist[c][2 * tid + e];
          sm.hist[c][2 * tid + e] = 0;
        }
        sm.bins[pass & 1][2 * tid + e] = two[e];
      }
      const unsigned all = __reduce_add_sync(0xffffffffu, two[0] + two[1]);
      if (lane == 0) sm.coarse[pass & 1][warp] = all;
      cluster_sync();                           // (every CTA has read the pass before's, too)
      if (warp == 0) {
        // the 64 bins that hold the left-th largest, then the bin
        unsigned x = 0;
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < cl) x += ld_cluster(mapa(smem_u32(&sm.coarse[pass & 1][lane]), r));
        unsigned from = sum_from_lane(x);
        const int group = 31 - __clz(__ballot_sync(0xffffffffu, from >= left));
        unsigned rest = left - __shfl_sync(0xffffffffu, from - x, group);
        unsigned c0 = 0, c1 = 0;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          if (r >= cl) continue;
          const uint32_t at = mapa(smem_u32(&sm.bins[pass & 1][64 * group + 2 * lane]), r);
          uint32_t v0, v1;
          asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
                       : "=r"(v0), "=r"(v1)
                       : "r"(at)
                       : "memory");
          c0 += v0;
          c1 += v1;
        }
        from = sum_from_lane(c0 + c1);
        const int pair = 31 - __clz(__ballot_sync(0xffffffffu, from >= rest));
        rest -= __shfl_sync(0xffffffffu, from - c0 - c1, pair);
        if (lane == pair) {
          const bool upper = rest <= c1;
          sm.digit = static_cast<unsigned>(64 * group + 2 * pair + (upper ? 1 : 0));
          sm.left = rest - (upper ? 0 : c1);
        }
      }
      __syncthreads();
      prefix = (prefix << bits) | sm.digit;
      left = sm.left;
    }
    thr = prefix;
    ties = static_cast<int>(left);
  }
  // counts of the warp's run, then of everything before it
  auto classify = [&](int i, unsigned& above, unsigned& eq) {
    bool a = false, e = false;
    if (i < s1) {
      if (i < lo || i >= hi) {
        a = true;
      } else if (want > 0) {
        const unsigned x = key(i);
        a = x > thr;
        e = x == thr;
      }
    }
    above = __ballot_sync(0xffffffffu, a);
    eq = __ballot_sync(0xffffffffu, e);
  };
  int n_above = 0, n_eq = 0;
#pragma unroll 1
  for (int i = s0; i < s1; i += 32) {
    unsigned a, e;
    classify(i + lane, a, e);
    n_above += __popc(a);
    n_eq += __popc(e);
  }
  if (lane == 0) {
    sm.warp_above[warp] = n_above;
    sm.warp_eq[warp] = n_eq;
  }
  __syncthreads();
  const int w_above = sm.warp_above[lane], w_eq = sm.warp_eq[lane];     // (32 warps)
  int above_before = __reduce_add_sync(0xffffffffu, lane < warp ? w_above : 0);
  int eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? w_eq : 0);
  if (warp == 0) {
    const int a = __reduce_add_sync(0xffffffffu, w_above), e = __reduce_add_sync(0xffffffffu, w_eq);
    if (lane == 0) {
      sm.above = a;
      sm.eq = e;
    }
  }
  cluster_sync();
  for (int r = 0; r < rank; ++r) {
    above_before += static_cast<int>(ld_cluster(mapa(smem_u32(&sm.above), r)));
    eq_before += static_cast<int>(ld_cluster(mapa(smem_u32(&sm.eq), r)));
  }
  const unsigned below = (1u << lane) - 1;
#pragma unroll 1
  for (int i = s0; i < s1; i += 32) {
    unsigned a, e;
    classify(i + lane, a, e);
    const int ra = above_before + __popc(a & below), re = eq_before + __popc(e & below);
    if (((a >> lane) & 1u) || (((e >> lane) & 1u) && re < ties))
      idx[ra + min(ties, re)] = i + lane;
    above_before += __popc(a);
    eq_before += __popc(e);
  }
  cluster_sync();                               // the others may still read this CTA's counts
}

struct MoveSmem {                               // places by step and thread
  uint4 row[kDepth][kMoveThreads];
  int dst[kDepth][kMoveThreads];                // the row it goes to, -1: nowhere
};
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes)
                 : "memory");
}

// One column slice of one sequence: `cols` elements from element `first` of
// every row (rows of `pitch` elements), threads / cols rows a CTA and step.
// Rows pass through shared memory, each thread's in places of its own, with
// kDepth - 1 steps' reads on their way; a step's table entries are loaded a step
// before its reads, and its slots a step before that.
//
// Between a step's reads and its writes stands a barrier that orders nothing
// else: no thread reads what another has written, and a read is over once it
// has landed. So the arrival is relaxed (one that releases waits for all reads
// and writes in flight, the next steps' too: 8 x 32768 -> 16384 took 161 us).
template <typename V>
__device__ __forceinline__ void move_columns(const EvictArgs& A, MoveSmem& sm, int b, int count,
                                             const V* from, V* to, bool paged, int pitch, int cols,
                                             int first) {
  const int cl = static_cast<int>(cluster_size()), tid = static_cast<int>(threadIdx.x);
  const int rows = kMoveThreads / cols, col = first + tid % cols;
  const int step = rows * cl, sub = rows * static_cast<int>(cluster_rank()) + tid / cols;
  const int end = tid < rows * cols ? count : 0;                // (threads past the last row are idle)
  const int* idx = A.idx + static_cast<long long>(b) * A.budget;
  const int* table = A.block_table + static_cast<long long>(b) * A.max_blocks;
  // (the last kept row in its place: so are all before it)
  if (count <= 0 || (from == to && __ldg(idx + count - 1) == count - 1)) return;
  int src, slot, src_block, dst_block;
  auto slots = [&](int j) { src = j < end ? __ldg(idx + j) : -1; };
  auto blocks = [&](int j) {
    const bool moves = src >= 0 && src < A.max_blocks * 64 && !(src == j && from == to);
    slot = moves ? src : -1;
    src_block = moves && paged ? __ldg(table + (src >> 6)) : 0;
    dst_block = moves && paged ? __ldg(table + (j >> 6)) : 0;
  };
  auto read = [&](int j, int d) {
    int dst = -1;
    if (slot >= 0) {
      if (paged && (src_block < 0 || src_block >= A.nblk || dst_block < 0 || dst_block >= A.nblk)) {
        raise_error(A.err, kErrBounds);
      } else {
        const int r = paged ? src_block * 64 + (slot & 63) : slot;
        dst = paged ? dst_block * 64 + (j & 63) : j;
        copy_async<sizeof(V)>(smem_u32(&sm.row[d][tid]),
                              from + static_cast<long long>(r) * pitch + col);
      }
    }
    sm.dst[d][tid] = dst;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int next = sub;                               // this thread's row of the step read next
  slots(next);
  blocks(next);
  slots(next + step);
#pragma unroll 1
  for (int d = 0; d + 1 < kDepth; ++d, next += step) {
    read(next, d);
    blocks(next + step);
    slots(next + 2 * step);
  }
  int d = 0;
#pragma unroll 1
  for (int j0 = 0; j0 < count; j0 += step, next += step) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
    if (cl > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    read(next, d == 0 ? kDepth - 1 : d - 1);
    blocks(next + step);
    slots(next + 2 * step);
    if (cl > 1)
      cluster_wait();
    else
      __syncthreads();
    const int dst = sm.dst[d][tid];
    if (dst >= 0)
      to[static_cast<long long>(dst) * pitch + col] = *reinterpret_cast<V*>(&sm.row[d][tid]);
    d = d + 1 == kDepth ? 0 : d + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Job y of a sequence: a slice of the latent rows' 72 16-byte columns, then the
// indexer's keys, their scales and the totals.
__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(const EvictArgs A, const Verdicts verdicts, int slices) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  MoveSmem& sm = *reinterpret_cast<MoveSmem*>(smem_raw);
  const int b = static_cast<int>(blockIdx.x / cluster_size());
  const int count = min(A.seq_len_out[b], min(A.budget, A.max_blocks * 64));
  if (!verdicts.of(b)) return;                  // (the same for all CTAs of the sequence)
  const int job = static_cast<int>(blockIdx.y);
  if (job < slices) {
    uint4* p = static_cast<uint4*>(A.kv_pool);
    const int cols = 72 / slices;
    move_columns<uint4>(A, sm, b, count, p, p, true, 72, cols, cols * job);
  } else if (job == slices) {
    uint4* p = static_cast<uint4*>(A.k8_pool);
    if (p) move_columns<uint4>(A, sm, b, count, p, p, true, 8, 8, 0);
  } else if (job == slices + 1) {
    if (A.k_scale_pool)
      move_columns<float>(A, sm, b, count, A.k_scale_pool, A.k_scale_pool, true, 1, 1, 0);
  } else if (A.mass_out) {
    move_columns<float>(A, sm, b, count, A.mass + b * A.ld, A.mass_out + b * A.ld_out, false, 1,
                        1, 0);
  }
}

}  // namespace

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t st) {
  // CTAs per sequence: more while they leave SMs idle and have 4096 slots each
  int cl = 1;
  while (cl < 8 && a.B * cl * 2 <= 148 && a.max_blocks * 64 > 4096 * cl) cl *= 2;
  const size_t smem = sizeof(SelSmem) + kSelKeys * sizeof(unsigned);
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * cl);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(cl);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  static std::atomic<unsigned> next[2];
  cudaStreamCaptureStatus capture;
  e = cudaStreamIsCapturing(st, &capture);
  if (e != cudaSuccess) return e;
  Verdicts verdicts;
  verdicts.list = capture == cudaStreamCaptureStatusNone ? 0 : 1;
  verdicts.first = next[verdicts.list].fetch_add(static_cast<unsigned>(a.B));
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, verdicts);
  if (e != cudaSuccess) return e;
  // Whole rows where the sequences' clusters fill the GPU, else as few slices of
  // them as do, of 384, 128 or 64 bytes (measured with 512 threads a CTA, 64 x
  // 32768 -> 16384: 515 us in whole rows, 613 us in three slices and 626 us in
  // nine; 16 x 32768: 214 us in whole rows, 194 us in three slices)
  int slices = 1;
  while (slices < 18 && a.B * slices * 8 < kMoveWant) slices = slices == 9 ? 18 : 3 * slices;
  cl = 1;
  while (cl < 8 && a.B * slices * cl * 2 <= kMoveMost) cl *= 2;
  cfg.gridDim = dim3(static_cast<unsigned>(a.B * cl), static_cast<unsigned>(slices + 3));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = sizeof(MoveSmem);
  at.val.clusterDim.x = static_cast<unsigned>(cl);
  e = cudaFuncSetAttribute(evict_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(cfg.dynamicSmemBytes));
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel, a, verdicts, slices);
}

}  // namespace dsa

// split.cuh -- equal shares of a list of work over CTAs, and bounded waits whose
// slow path is out of line; shared by the kernels that walk the paged cache.
#pragma once

#include "common.cuh"

namespace dsa {

// The bounded waits of common.cuh with the slow path out of line: these kernels
// have some thirty of them in warps that run different code, and their short
// loops have to fit the instruction caches.
//
// The slow path suspends the warp in the barrier unit, at most a millisecond at
// a time, and spends no issue slots that the SM's other warps could use.
//
// A wait may be for the whole of a row tile that another role works on, which for
// a very long cache takes over a second: the limit counts from the CTA's last
// progress, a number that one of its roles changes with each tile (abort_flag[1];
// a tile takes microseconds).
static __device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity,
                                              volatile int* abort_flag, unsigned* err) {
  unsigned long long t0 = globaltimer();
  int tiles = abort_flag[1];
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(1000000u)
        : "memory");
    if (ok) return true;
    if (*abort_flag) return false;
    if (globaltimer() - t0 > kWaitLimitNs) {
      const int now = abort_flag[1];
      if (now != tiles) {
        tiles = now;
        t0 = globaltimer();
        continue;
      }
      *abort_flag = 1;
      raise_error(err, kErrTimeout);
      return false;
    }
  }
}
template <bool kCluster = false>
__device__ __forceinline__ bool wait1(unsigned long long& b, uint32_t parity,
                                      volatile int* abort_flag, unsigned* err) {
  const uint32_t bar = smem_u32(&b);
  if (kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, abort_flag, err);
}
// By every lane of a warp, which agrees on the result.
template <bool kCluster = false>
__device__ __forceinline__ bool wait32(unsigned long long& b, uint32_t parity,
                                       volatile int* abort_flag, unsigned* err) {
  return __all_sync(0xffffffffu, wait1<kCluster>(b, parity, abort_flag, err));
}

// One CTA's (or cluster's) share of a list of weighted items: the weights are
// laid end to end and cut into equal parts.
struct Share {
  long long total, start;                       // all weight; the weight before the first item
  long long left;                               // weight of the share
  int item, off, parts;                         // first item, offset into it
  int whole;                                    // items c, c + parts_max, ... whole instead
};

// Where part c of `parts` begins. Totals that fit 32 bits, the usual ones, spare
// the 64-bit division.
__device__ __forceinline__ long long share_begin(long long total, int parts, int c) {
  if (total < (1ll << 24))
    return static_cast<unsigned>(total) * static_cast<unsigned>(c) /
           static_cast<unsigned>(parts);
  return total * c / parts;
}

// Finds share `c` of at most `parts_max`, each of one unit of weight at least.
// Where items taken whole, in turn, are as fast as equal shares and `cut_cost`
// (weight that a cut costs; 0: always cut), the share says so instead. Called
// by all kThreads threads; `sums` is scratch for two numbers a warp; weight(i)
// is item i's. Ends with sh written by one thread: the caller synchronises.
// Shares past the last part get item = items.
template <int kThreads, typename Weight>
__device__ __forceinline__ void find_share(Share& sh, long long* sums, int items, int c,
                                           int parts_max, int cut_cost, Weight weight) {
  const int tid = static_cast<int>(threadIdx.x);
  const int per = (items + kThreads - 1) / kThreads;
  const int i0 = min(items, tid * per), i1 = min(items, i0 + per);
  long long sum = 0;
  int w_first = 0, w_max = 0;
  for (int i = i0; i < i1; ++i) {
    const int w = weight(i);
    if (i == i0) w_first = w;
    w_max = max(w_max, w);
    sum += w;
  }
  // exclusive prefix over the block: within warps, then over the warps' sums
  long long before = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, before, o);
    if (lane_id() >= o) before += y;
  }
  w_max = __reduce_max_sync(0xffffffffu, w_max);
  if (lane_id() == 31) {
    sums[warp_id()] = before;
    sums[kThreads / 32 + warp_id()] = w_max;
  }
  before -= sum;
  if (tid == 0) {
    sh.item = items;
    sh.off = sh.whole = 0;
    sh.left = sh.start = 0;
  }
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp_id()) before += total;
    total += sums[w];
    w_max = max(w_max, static_cast<int>(sums[kThreads / 32 + w]));
  }
  const int parts = static_cast<int>(
      max(1ll, min(static_cast<long long>(parts_max), total)));
  if (tid == 0) {
    sh.total = total;
    sh.parts = parts;
  }
  if (static_cast<long long>((items + parts_max - 1) / parts_max) * w_max <=
      total / parts + cut_cost && cut_cost > 0) {
    if (tid == 0) {
      sh.item = c;
      sh.whole = 1;
    }
    return;
  }
  if (c >= parts) return;
  const long long w0 = share_begin(total, parts, c), w1 = share_begin(total, parts, c + 1);
  if (before <= w0 && w0 < before + sum) {
    long long at = before;
    for (int i = i0; i < i1; ++i) {
      const int w = i == i0 ? w_first : weight(i);
      if (w0 < at + w) {
        sh.item = i;
        sh.off = static_cast<int>(w0 - at);
        sh.left = w1 - w0;
        sh.start = at;
        break;
      }
      at += w;
    }
  }
}

}  // namespace dsa

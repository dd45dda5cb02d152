// cache_mass.cu -- the attention weight each cached token receives, sm_100a.
//
// With lse[b,j,h] the natural log normaliser of query j, head h (as the
// attention returns it), key s of sequence b receives
//   w[b,s] = sum_{j,h: s <= pos_j} exp(sm_scale q[b,j,h] . kv[s] - lse[b,j,h])
// from the nq new tokens, pos_j = seq_len[b] - nq + j, and its running total
// becomes mass + w (w alone for the new tokens, which have no total yet).
// Every total belongs to one thread, so no atomics and one order of addition.
//
// One thread per key: the row's dot product with every query in fp32.
#include "common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kThreads = 64;

__global__ void __launch_bounds__(kThreads) mass_kernel(const MassArgs A) {
  __shared__ float qs[576];
  const int b = static_cast<int>(blockIdx.y);
  const int cap = A.max_blocks * 64;
  int len = A.seq_len[b];
  if (threadIdx.x == 0 && blockIdx.x == 0 && (len < 0 || len > cap)) raise_error(A.err, kErrBounds);
  len = max(0, min(len, cap));
  const int s0 = static_cast<int>(blockIdx.x) * 64, s = s0 + static_cast<int>(threadIdx.x);
  if (s0 >= len) return;
  const int pb = A.block_table[static_cast<long long>(b) * A.max_blocks + blockIdx.x];
  if (pb < 0 || pb >= A.nblk) {
    if (threadIdx.x == 0) raise_error(A.err, kErrBounds);
    return;
  }
  const __nv_bfloat16* k = A.kv + (static_cast<long long>(pb) * 64 + threadIdx.x) * 576;
  float w = 0.f;
  for (int i = 0; i < A.nq * A.H; ++i) {
    const long long r = static_cast<long long>(b) * A.nq * A.H + i;
    __syncthreads();
    for (int d = threadIdx.x; d < 576; d += kThreads) qs[d] = __bfloat162float(A.q[r * 576 + d]);
    __syncthreads();
    if (s >= len || s > len - A.nq + i / A.H || A.lse[r] == -INFINITY) continue;
    float z = 0.f;
    for (int d = 0; d < 576; ++d) z += qs[d] * __bfloat162float(k[d]);
    w += exp2f(z * A.sm_scale_log2 - A.lse[r] * 1.4426950408889634f);
  }
  if (s < len) {
    float* m = A.mass + b * A.ld + s;
    *m = (s < len - A.nq ? *m : 0.f) + w;
  }
}

}  // namespace

cudaError_t launch_attention_mass(const MassArgs& a, cudaStream_t st) {
  mass_kernel<<<dim3(a.max_blocks, a.B), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace dsa

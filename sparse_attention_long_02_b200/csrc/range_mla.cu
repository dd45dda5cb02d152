// range_mla.cu -- MLA attention over ranges of the latent cache, sm_100a: every
// earlier key (dense), or a sliding window and the first few keys (sinks).
//
// Row t of a contiguous cache sits at position p = q_pos0 + t; query j of
// sequence b of a paged cache at p = seq_len[b] - nq + j. It sees the keys s
// with s <= min(p, last key) and, with a window w, s > p - w or s < sinks:
//   out = sum_s exp(z_s - lse) kv[s, :512],  z_s = sm_scale q . kv[s],
//   lse = log sum_s exp(z_s).
// A row that sees no key gets out = 0 and lse = -inf.
//
// One CTA per (query, head): the running maximum and sum of the softmax over
// blocks of 128 keys, everything in fp32.
#include "common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kThreads = 128;

// Physical row of key `s`, or -1 when its block id is out of range.
__device__ __forceinline__ long long key_row(const RangeArgs& A, int b, int s) {
  if (!A.block_table) return s;
  const int pb = A.block_table[static_cast<long long>(b) * A.max_blocks + (s >> 6)];
  if (pb < 0 || pb >= A.nblk) return -1;
  return static_cast<long long>(pb) * 64 + (s & 63);
}

__global__ void __launch_bounds__(kThreads) range_mla_kernel(const RangeArgs A) {
  __shared__ float qs[576], ps[kThreads];
  __shared__ long long rows[kThreads];
  __shared__ float red[kThreads / 32];
  const long long qr = static_cast<long long>(blockIdx.x) / A.H;          // query row
  const int h = static_cast<int>(blockIdx.x % A.H);
  const int b = A.block_table ? static_cast<int>(qr / A.nq) : 0;
  int pos, last;
  if (A.block_table) {
    const int len = A.seq_len[b], cap = A.max_blocks * 64;
    if (threadIdx.x == 0 && (len < 0 || len > cap)) raise_error(A.err, kErrBounds);
    last = max(0, min(len, cap)) - 1;
    pos = last + 1 - A.nq + static_cast<int>(qr % A.nq);
  } else {
    last = A.S - 1;
    pos = A.q_pos0 + static_cast<int>(qr);
  }
  const int hi = min(pos, last);
  const int lo = A.window ? max(0, pos - A.window + 1) : 0;
  const int ns = A.window ? min(min(A.sinks, lo), hi + 1) : 0;            // sinks before the window
  const int n = max(0, ns) + max(0, hi - lo + 1);
  const __nv_bfloat16* q = A.q + (qr * A.H + h) * 576;
  for (int i = threadIdx.x; i < 576; i += kThreads) qs[i] = __bfloat162float(q[i]);
  __syncthreads();
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < n; k0 += kThreads) {
    const int i = k0 + threadIdx.x;
    float z = -INFINITY;
    long long r = -1;
    if (i < n) {
      r = key_row(A, b, i < ns ? i : lo + i - ns);
      if (r < 0) {
        raise_error(A.err, kErrBounds);
      } else {
        const __nv_bfloat16* k = A.kv + r * 576;
        float s = 0.f;
        for (int d = 0; d < 576; ++d) s += qs[d] * __bfloat162float(k[d]);
        z = s * A.sm_scale_log2;
      }
    }
    float t = z;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, w));
    if (lane_id() == 0) red[warp_id()] = t;
    __syncthreads();
    t = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float mn = fmaxf(m, t);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float alpha = exp2f(m - base);
    const float p = r < 0 ? 0.f : exp2f(z - base);
    rows[threadIdx.x] = r;
    ps[threadIdx.x] = p;
    __syncthreads();
    l *= alpha;
    for (int e = 0; e < 4; ++e) o[e] *= alpha;
    for (int j = 0; j < min(kThreads, n - k0); ++j) {
      l += ps[j];
      if (rows[j] < 0) continue;
      const __nv_bfloat16* v = A.kv + rows[j] * 576 + 4 * threadIdx.x;
      for (int e = 0; e < 4; ++e) o[e] += ps[j] * __bfloat162float(v[e]);
    }
    m = mn;
    __syncthreads();
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __nv_bfloat16* out = A.out + (qr * A.H + h) * 512 + 4 * threadIdx.x;
  for (int e = 0; e < 4; ++e) out[e] = __float2bfloat16(o[e] * inv);
  if (threadIdx.x == 0 && A.lse)
    A.lse[qr * A.H + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

cudaError_t launch_range_mla(const RangeArgs& a, cudaStream_t st) {
  const long long rows = a.block_table ? static_cast<long long>(a.B) * a.nq : a.T;
  range_mla_kernel<<<static_cast<unsigned>(rows * a.H), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace dsa

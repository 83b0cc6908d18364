// smqa_paged_fwd.cu -- sparse MQA over the 8-bit paged cache on sm_103a.
//
// Per token t and head h, over the valid slots j (an index list, or every
// position up to the token's own), with k_j = s_j c_j the cache row (s_j its
// page's scale, c_j its e4m3 codes):
//   x_j = sm_scale log2(e) q.k_j,  l = sum_j 2^x_j + 2^(sink log2(e)),
//   O = sum_j 2^x_j k_j / l,  lse = log2 l.
#include <cuda_runtime.h>

#include <cmath>

#include "smqa_internal.h"
#include "smqa_ptx.cuh"

namespace smqa {

namespace {

constexpr int kWarps = 8;

// One CTA per (token, head); its warps take slots in turn, each with a running
// maximum and sum of its own, joined at the end.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) smqa_paged_fwd_kernel(const PagedFwdParams p) {
  constexpr int E = D / 32;  // elements per lane
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  const int t = blockIdx.x / p.H, h = blockIdx.x % p.H;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = static_cast<int64_t>(t) * p.H + h;
  const int req = p.token_req[t];
  if (static_cast<unsigned>(req) >= static_cast<unsigned>(p.R)) {
    if (p.zero_padding) {
      for (int d = threadIdx.x; d < D; d += kWarps * 32) p.o[row * D + d] = __float2bfloat16(0.f);
      if (threadIdx.x == 0) p.lse[row] = -INFINITY;
    }
    return;
  }
  const int len = p.seq_lens[req];
  const int n = p.idx ? p.topk : min(len, p.positions[t] + 1);
  float q[E], o[E] = {};
  for (int k = 0; k < E; ++k) q[k] = __bfloat162float(p.q[row * D + lane * E + k]) * p.scale_log2;
  float m = -INFINITY, l = 0.f;
  for (int j = warp; j < n; j += kWarps) {
    const int i = p.idx ? p.idx[static_cast<int64_t>(t) * p.topk + j] : j;
    if (i < 0 || i >= len) continue;
    const int col = i >> p.page_shift;
    const int pg = col < p.max_pages ? p.table[static_cast<int64_t>(req) * p.max_pages + col] : -1;
    if (static_cast<unsigned>(pg) >= static_cast<unsigned>(p.n_pages)) continue;
    const float s = p.scales[pg];
    const uint8_t* c = p.cache + ((static_cast<int64_t>(pg) << p.page_shift) +
                                  (i & ((1 << p.page_shift) - 1))) * D + lane * E;
    float k[E];
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      uint32_t f;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(*reinterpret_cast<const uint16_t*>(c + e)));
      const float2 v = __half22float2(*reinterpret_cast<__half2*>(&f));
      k[e] = v.x * s;
      k[e + 1] = v.y * s;
    }
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) x = fmaf(q[e], k[e], x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    const float mn = x != x ? x : fmaxf(m, x);  // a NaN stays
    const float a = m == -INFINITY ? 0.f : exp2f(m - mn), b = exp2f(x - mn);
    m = mn;
    l = l * a + b;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], a, b * k[e]);
  }
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
  __syncthreads();
  const float sink = p.sink[h] * 1.4426950408889634f;
  float top = sink;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  float total = sink == -INFINITY ? 0.f : exp2f(sink - top);
  for (int w = 0; w < kWarps; ++w) total += s_m[w] == -INFINITY ? 0.f : s_l[w] * exp2f(s_m[w] - top);
  for (int d = threadIdx.x; d < D; d += kWarps * 32) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w) v += s_m[w] == -INFINITY ? 0.f : s_o[w][d] * exp2f(s_m[w] - top);
    p.o[row * D + d] = __float2bfloat16(total > 0.f || total != total ? v / total : 0.f);
  }
  if (threadIdx.x == 0) p.lse[row] = top == -INFINITY ? -INFINITY : log2f(total) + top;
}

}  // namespace

cudaError_t launch_paged_fwd(const PagedFwdParams& p, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.T) * p.H;
  if (p.D == 512)
    smqa_paged_fwd_kernel<512><<<grid, kWarps * 32, 0, stream>>>(p);
  else
    smqa_paged_fwd_kernel<64><<<grid, kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace smqa

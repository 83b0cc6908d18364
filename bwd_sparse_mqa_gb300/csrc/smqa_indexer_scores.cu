// smqa_indexer_scores.cu -- the lightning indexer's scores at given positions on
// sm_103a, and their gradients with respect to queries, weights and keys.
//
//   x[h,j] = q[t,h] . k[idx[t,j]],   score[t,j] = sum_h w[t,h] ReLU(x[h,j])
// and, for a gradient g[t,j] of the scores, over the valid slots j (index in
// [0, S_kv); a slot listed twice counts twice; the ReLU's slope at 0 is 0):
//   dq[t,h] = sum_j w[t,h] g[t,j] [x > 0] k_j
//   dw[t,h] = sum_j g[t,j] ReLU(x[h,j])
//   dk[i]   = sum over (t, j) with idx[t,j] = i of sum_h w[t,h] g[t,j] [x > 0] q[t,h]
// (tilelang_indexer_bwd of the DeepSeek-V4 kernel pages of NeMo AutoModel gives dq
// only, and no forward; smqa_indexer.cu is that.)
//
// Forward, one CTA per token, two per SM.  Per block of 128 slots: gather (warps 4-7)
// copies the key rows by 16-byte cp.async into a 128-byte-swizzled tile (two in a ring);
// the tensor core (warp 8) forms x with M = 128 slots, N = heads, K = D, two
// accumulators; epilogue (warps 0-3) has a slot per thread and sums over its heads, no
// exchange between threads.
//
// Backward, one CTA per token, two per SM.  Per block of 64 slots: gather (warps 4-5);
// tensor core (warp 6): L = Q.K^T (M = 128 head rows, N = 64, K = D), and once the gate
// operand G[h,j] = [L > 0] w[h] g[j] is written in bf16 (the type of the products' other
// factors, and the one rounding on the way to dq and dk: 2^-8 of each term at most),
// dq += G.K into an accumulator that lives for the token,
// and dk^T = Q^T.G (M = D, N = 64, K = 128 heads; both operands read MN-major from where
// they lie); gate (warps 0-3): thread = head row, which also sums dw in fp32; drain
// (warps 8-11): thread = element of D, adds dk^T to the fp32 accumulator in global
// memory, 32 consecutive elements per warp instruction.
#include <cuda_runtime.h>

#include "smqa_internal.h"
#include "smqa_paged.cuh"

namespace smqa {

namespace {

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
template <int D>
struct FwdLayout {
  static constexpr int kBI = 128;
  static constexpr int kChunks = D / 64;
  static constexpr int kStages = 2;
  static constexpr uint32_t kQChunkBytes = 128 * 128;
  static constexpr uint32_t kChunkBytes = kBI * 128;
  static constexpr uint32_t kStageBytes = kChunks * kChunkBytes;
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffK = kChunks * kQChunkBytes;
  static constexpr uint32_t kOffW = kOffK + kStages * kStageBytes;  // float [128]
  static constexpr uint32_t kOffBar = kOffW + 512;
  static constexpr int kBarFull = 0, kBarEmpty = 2, kBarAccFull = 4, kBarAccEmpty = 6, kBarQ = 8, kBarDrain = 9;
  static constexpr int kNumBars = 10;
  static constexpr uint32_t kOffCtl = kOffBar + 8 * kNumBars;  // TMEM base, abort flag
  static constexpr uint32_t kOffLast = kOffCtl + 8;            // int [9]
  static constexpr uint32_t kSmem = kOffLast + 40 + 1024;
  static_assert(2 * (kSmem + 1024) <= 233472, "two CTAs per SM");
  static constexpr int kThreads = 288;
};

template <int D>
__global__ void __launch_bounds__(288, 2) smqa_indexer_scores_kernel(const IdxParams p, const __nv_bfloat16* q, float* scores) {
  using L = FwdLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint32_t base = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (base & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  base += pad;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int64_t t = blockIdx.x, b = t / p.S;             // token of all batch elements
  const int32_t* idx_row = p.idx + t * p.topk;
  const int heads = (p.H + 31) & ~31;                    // N: whole groups of 32 columns
  auto bar = [&](int i) -> uint32_t { return base + L::kOffBar + 8u * static_cast<uint32_t>(i); };
  volatile uint32_t* tmem_holder = reinterpret_cast<volatile uint32_t*>(smem + L::kOffCtl);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffCtl + 4);
  const WaitCtl ctl{abort_flag, p.status, p.limit_ns};
  float* ws = reinterpret_cast<float*>(smem + L::kOffW);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(L::kBarFull + i), 128);
      mbar_init(bar(L::kBarEmpty + i), 1);
      mbar_init(bar(L::kBarAccFull + i), 1);
      mbar_init(bar(L::kBarAccEmpty + i), 4);
    }
    mbar_init(bar(L::kBarQ), 128);
    mbar_init(bar(L::kBarDrain), 1);
    *abort_flag = *reinterpret_cast<volatile int*>(p.status) != 0 ? 1 : 0;
    fence_mbar_init();
  }
  if (warp == 8) tmem_alloc(base + L::kOffCtl, 256);
  if (tid < 128) ws[tid] = tid < p.H ? __ldg(p.w + t * p.H + tid) : 0.f;
  volatile int* warp_last = reinterpret_cast<volatile int*>(smem + L::kOffLast);
  scan_last_valid(idx_row, p.topk, p.S_kv, warp_last);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int nblk = live_blocks(warp_last, L::kBI);

  if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ gather
    const int gt = tid - 128, gw = warp - 4;
    constexpr int kPer = D / 8;                          // 16-byte pieces of a row
    const __nv_bfloat16* q0 = q + t * p.H * D;
    for (int i = gt; i < heads * kPer; i += 128) {
      const int h = i / kPer, c = i % kPer;
      const bool there = h < p.H;
      cp_async_16_or_zero(base + L::kOffQ + (c >> 3) * L::kQChunkBytes + h * 128 + (((c & 7) ^ (h & 7)) << 4),
                          q0 + (there ? h : 0) * D + c * 8, there);
    }
    cp_async_arrive_noinc(bar(L::kBarQ));
    constexpr int kRpi = 32 / kPer;                      // rows per warp instruction
    const int rsub = lane / kPer, cc = lane % kPer;
    const __nv_bfloat16* k_col = p.k + b * p.k_b_stride + cc * 8;
    const uint32_t lane_off = static_cast<uint32_t>(cc >> 3) * L::kChunkBytes;
    for (int i = 0; i < nblk; ++i) {
      const int st = i & 1, j = i * L::kBI + gt;
      const int r = j < p.topk ? __ldg(idx_row + j) : -1;
      const bool ok_row = static_cast<unsigned>(r) < static_cast<unsigned>(p.S_kv);
      const unsigned mask = __ballot_sync(0xffffffffu, ok_row);
      if (i >= 2) {
        if (!__all_sync(0xffffffffu, mbar_wait_soon(bar(L::kBarEmpty + st), ((i >> 1) - 1) & 1, ctl))) break;
      } else if (*abort_flag) {
        break;
      }
      const uint32_t stage = base + L::kOffK + st * L::kStageBytes + lane_off;
#pragma unroll
      for (int k = 0; k < 32 / kRpi; ++k) {
        const int rw = k * kRpi + rsub;
        const int rr = __shfl_sync(0xffffffffu, ok_row ? r : 0, rw);
        const uint32_t srow = static_cast<uint32_t>(32 * gw + rw);
        cp_async_16_or_zero(stage + srow * 128u + ((static_cast<uint32_t>(cc & 7) ^ (srow & 7u)) << 4),
                            k_col + static_cast<size_t>(rr) * p.k_row_stride, (mask >> rw) & 1u);
      }
      cp_async_arrive_noinc(bar(L::kBarFull + st));
    }
    cp_async_wait_all();
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t idesc = (idesc_bf16_f32(128, 16, false, false) & ~(0x3fu << 17)) | (static_cast<uint32_t>(heads >> 3) << 17);
      const uint64_t d_q = smem_desc(base + L::kOffQ, 16u, 1024u, kSwizzle128B);
      const uint64_t d_k = smem_desc(base + L::kOffK, 16u, 1024u, kSwizzle128B);
      bool ok = mbar_wait_soon(bar(L::kBarQ), 0, ctl);
      for (int i = 0; ok && i < nblk; ++i) {
        const int st = i & 1;
        ok = (i < 2 || mbar_wait_soon(bar(L::kBarAccEmpty + st), ((i >> 1) - 1) & 1, ctl)) &&
             mbar_wait_soon(bar(L::kBarFull + st), (i >> 1) & 1, ctl);
        if (!ok) break;
        fence_proxy_async_smem();                        // rows written by cp.async -> tensor core
        tc_fence_after();
        const uint64_t kd = d_k + ((static_cast<uint32_t>(st) * L::kStageBytes) >> 4);
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(tmem + st * 128, kd + ((c * L::kChunkBytes + k * 32u) >> 4), d_q + ((c * L::kQChunkBytes + k * 32u) >> 4), idesc,
                   (c | k) != 0 ? 1u : 0u);
        mma_commit(bar(L::kBarEmpty + st));
        mma_commit(bar(L::kBarAccFull + st));
        if (i == 0 && static_cast<int>(blockIdx.x) == p.stall_cta) ok = stall_until_limit(ctl);  // test hook only
      }
      mma_commit(bar(L::kBarDrain));
      mbar_wait_drain(bar(L::kBarDrain), 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    float* out = scores + t * p.topk;
    bool ok = *abort_flag == 0;
    for (int i = 0; ok && i < nblk; ++i) {
      const int st = i & 1, j = i * L::kBI + tid;
      const int r = j < p.topk ? __ldg(idx_row + j) : -1;
      ok = __all_sync(0xffffffffu, mbar_wait_soon(bar(L::kBarAccFull + st), (i >> 1) & 1, ctl));
      if (!ok) break;
      tc_fence_after();
      auto relu = [](float v) {                          // (a NaN stays one)
        float y;
        asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(v));
        return y;
      };
      float2 a0 = {}, a1 = {};
      for (int c = 0; c < heads; c += 32) {
        float x[32];
        tmem_ld32(tmem + lanes + st * 128 + c, x);
        const float4* w4 = reinterpret_cast<const float4*>(ws + c);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float4 w = w4[k];
          a0 = fma2(make_float2(w.x, w.y), make_float2(relu(x[4 * k]), relu(x[4 * k + 1])), a0);
          a1 = fma2(make_float2(w.z, w.w), make_float2(relu(x[4 * k + 2]), relu(x[4 * k + 3])), a1);
        }
      }
      float s = (a0.x + a0.y) + (a1.x + a1.y);
      if (heads != p.H && __any_sync(0xffffffffu, s != s)) {
        // Without the heads behind H (0 times an infinity is no number), in four chains as above.
        float a[4] = {};
#pragma unroll 1
        for (int c = 0; c < p.H; c += 32) {
          float x[32];
          tmem_ld32(tmem + lanes + st * 128 + c, x);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (c + k < p.H) a[k & 3] = fmaf(ws[c + k], relu(x[k]), a[k & 3]);
        }
        s = (a[0] + a[1]) + (a[2] + a[3]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kBarAccEmpty + st));
      if (j < p.topk)
        out[j] = static_cast<unsigned>(r) < static_cast<unsigned>(p.S_kv) ? s : -INFINITY;
    }
    if (ok)
      for (int j = nblk * L::kBI + tid; j < p.topk; j += 128) out[j] = -INFINITY;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
template <int D>
struct BwdLayout {
  static constexpr int kHPad = 128;
  static constexpr int kBI = 64;
  static constexpr int kChunks = D / 64;
  static constexpr int kStages = 3;
  static constexpr int kInfo = 8;                        // blocks whose rows and gradients are kept
  static constexpr uint32_t kQChunkBytes = kHPad * 128;
  static constexpr uint32_t kChunkBytes = kBI * 128;
  static constexpr uint32_t kStageBytes = kChunks * kChunkBytes;
  static constexpr uint32_t kGateBytes = kHPad * kBI * 2;
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffKv = kOffQ + kChunks * kQChunkBytes;
  static constexpr uint32_t kOffGate = kOffKv + kStages * kStageBytes;
  static constexpr uint32_t kOffG = kOffGate + kGateBytes;         // float [kInfo][64]
  static constexpr uint32_t kOffRow = kOffG + kInfo * kBI * 4;     // int [kInfo][64] (-1: masked)
  static constexpr uint32_t kOffBar = kOffRow + kInfo * kBI * 4;
  static constexpr int kBarKvFull = 0, kBarKvEmpty = 3, kBarLFull = 6, kBarLFree = 7, kBarGFull = 8, kBarGFree = 9;
  static constexpr int kBarDkFull = 10, kBarDkFree = 11, kBarQ = 12, kBarDone = 13, kBarDrain = 14, kBarStaged = 15;
  static constexpr int kNumBars = 16;
  static constexpr uint32_t kOffCtl = kOffBar + 8 * kNumBars;
  static constexpr uint32_t kOffLast = kOffCtl + 8;                // int [12]
  static constexpr uint32_t kSmem = kOffLast + 56 + 1024;
  static_assert(2 * (kSmem + 1024) <= 233472, "two CTAs per SM");
  static_assert(kChunks * kQChunkBytes <= kStages * kStageBytes, "dq staging fits the ring");
  static constexpr uint32_t kTmemL = 0, kTmemDk = 64, kTmemDq = 128;
  static constexpr int kThreads = 384;
};

template <int D>
__global__ void __launch_bounds__(384, 2)
    smqa_indexer_scores_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_dq, const IdxParams p,
                                   float* dw, float* dk) {
  using L = BwdLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint32_t base = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (base & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  base += pad;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int64_t t = blockIdx.x, b = t / p.S, row0 = t * p.H;
  const int32_t* idx_row = p.idx + t * p.topk;
  const float* g_row = p.g + t * p.topk;
  auto bar = [&](int i) -> uint32_t { return base + L::kOffBar + 8u * static_cast<uint32_t>(i); };
  volatile uint32_t* tmem_holder = reinterpret_cast<volatile uint32_t*>(smem + L::kOffCtl);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffCtl + 4);
  const WaitCtl ctl{abort_flag, p.status, p.limit_ns};

  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(bar(L::kBarKvFull + i), 128);            // 64 copies landed, 64 rows and gradients written
      mbar_init(bar(L::kBarKvEmpty + i), 1);
    }
    mbar_init(bar(L::kBarLFull), 1);
    mbar_init(bar(L::kBarLFree), 128);
    mbar_init(bar(L::kBarGFull), 128);
    mbar_init(bar(L::kBarGFree), 1);
    mbar_init(bar(L::kBarDkFull), 1);
    mbar_init(bar(L::kBarDkFree), 4);
    mbar_init(bar(L::kBarQ), 1);
    mbar_init(bar(L::kBarDone), 1);
    mbar_init(bar(L::kBarDrain), 1);
    mbar_init(bar(L::kBarStaged), 128);
    *abort_flag = *reinterpret_cast<volatile int*>(p.status) != 0 ? 1 : 0;
    fence_mbar_init();
    mbar_arrive_expect_tx(bar(L::kBarQ), static_cast<uint32_t>(p.H) * 128u * L::kChunks);
    for (int c = 0; c < L::kChunks; ++c)
      tma_load_2d(base + L::kOffQ + c * L::kQChunkBytes, &tm_q, c * 64, static_cast<int>(row0), bar(L::kBarQ));
  }
  if (warp == 6) tmem_alloc(base + L::kOffCtl, 256);
  if (tid < L::kHPad && tid >= p.H) {
#pragma unroll
    for (int c = 0; c < L::kChunks; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) st_shared_v4(base + L::kOffQ + c * L::kQChunkBytes + tid * 128u + k * 16u, 0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  volatile int* warp_last = reinterpret_cast<volatile int*>(smem + L::kOffLast);
  scan_last_valid(idx_row, p.topk, p.S_kv, warp_last);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int nblk = live_blocks(warp_last, L::kBI);
  volatile float* g_of = reinterpret_cast<volatile float*>(smem + L::kOffG);
  volatile int* row_of = reinterpret_cast<volatile int*>(smem + L::kOffRow);

  if (warp == 4 || warp == 5) {
    // ------------------------------------------------------------ gather
    const int gw = warp - 4, gt = tid - 128;             // slot within a block
    constexpr int kPer = D / 8, kRpi = 32 / kPer;
    const int rsub = lane / kPer, cc = lane % kPer;
    const uint32_t lane_off = static_cast<uint32_t>(cc >> 3) * L::kChunkBytes;
    const __nv_bfloat16* k_col = p.k + b * p.k_b_stride + cc * 8;
    for (int i = 0; i < nblk; ++i) {
      const int st = i % L::kStages;
      const int j = i * L::kBI + gt;
      const int r = j < p.topk ? __ldg(idx_row + j) : -1;
      const bool there = static_cast<unsigned>(r) < static_cast<unsigned>(p.S_kv);
      const float gj = there ? __ldg(g_row + j) : 0.f;
      const unsigned mask = __ballot_sync(0xffffffffu, there);
      if (i >= L::kStages) {
        if (!__all_sync(0xffffffffu, mbar_wait_soon(bar(L::kBarKvEmpty + st), ((i / L::kStages) - 1) & 1, ctl))) break;
      } else if (*abort_flag) {
        break;
      }
      g_of[(i % L::kInfo) * L::kBI + gt] = gj;
      row_of[(i % L::kInfo) * L::kBI + gt] = there ? r : -1;
      const uint32_t stage = base + L::kOffKv + st * L::kStageBytes + lane_off;
#pragma unroll
      for (int k = 0; k < 32 / kRpi; ++k) {
        const int rw = k * kRpi + rsub;
        const int rr = __shfl_sync(0xffffffffu, there ? r : 0, rw);
        const uint32_t srow = static_cast<uint32_t>(32 * gw + rw);
        cp_async_16_or_zero(stage + srow * 128u + ((static_cast<uint32_t>(cc & 7) ^ (srow & 7u)) << 4),
                            k_col + static_cast<size_t>(rr) * p.k_row_stride, (mask >> rw) & 1u);
      }
      cp_async_arrive_noinc(bar(L::kBarKvFull + st));
      mbar_arrive(bar(L::kBarKvFull + st));              // (releases the row and gradient)
    }
    cp_async_wait_all();
    if (warp == 4 && lane == 0) mbar_wait_drain(bar(L::kBarQ), 0);
  } else if (warp == 6) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_l = idesc_bf16_f32(128, L::kBI, false, false);
      constexpr uint32_t idesc_dq = idesc_bf16_f32(128, D, false, true);
      constexpr uint32_t idesc_dk = idesc_bf16_f32(128, L::kBI, true, true);
      const uint64_t d_q = smem_desc(base + L::kOffQ, 16u, 1024u, kSwizzle128B);
      const uint64_t d_qt = smem_desc(base + L::kOffQ, L::kQChunkBytes, 1024u, kSwizzle128B);
      const uint64_t d_kv = smem_desc(base + L::kOffKv, 16u, 1024u, kSwizzle128B);
      const uint64_t d_kvt = smem_desc(base + L::kOffKv, L::kChunkBytes, 1024u, kSwizzle128B);
      const uint64_t d_g = smem_desc(base + L::kOffGate, 16u, 1024u, kSwizzle128B);
      const uint64_t d_gt = smem_desc(base + L::kOffGate, L::kGateBytes, 1024u, kSwizzle128B);
      auto issue_l = [&](int i) {
        const int st = i % L::kStages;
        const uint64_t k0 = d_kv + ((static_cast<uint32_t>(st) * L::kStageBytes) >> 4);
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(tmem + L::kTmemL, d_q + ((c * L::kQChunkBytes + k * 32u) >> 4), k0 + ((c * L::kChunkBytes + k * 32u) >> 4), idesc_l,
                   (c | k) != 0 ? 1u : 0u);
        mma_commit(bar(L::kBarLFull));
      };
      auto issue_grad = [&](int j) {
        const int st = j % L::kStages;
        const uint64_t k0 = d_kvt + ((static_cast<uint32_t>(st) * L::kStageBytes) >> 4);
        // dk^T first: the drain of it takes longest.  (D = 64: the upper 64 rows of M are of
        // what lies behind Q, and never looked at.)
#pragma unroll
        for (int k = 0; k < L::kHPad / 16; ++k)
          mma_ss(tmem + L::kTmemDk, d_qt + (k * 2048u >> 4), d_gt + (k * 2048u >> 4), idesc_dk, k != 0 ? 1u : 0u);
        mma_commit(bar(L::kBarDkFull));
#pragma unroll
        for (int k = 0; k < L::kBI / 16; ++k)
          mma_ss(tmem + L::kTmemDq, d_g + (k * 32u >> 4), k0 + (k * 2048u >> 4), idesc_dq, (j > 0 || k > 0) ? 1u : 0u);
        mma_commit(bar(L::kBarKvEmpty + st));
        mma_commit(bar(L::kBarGFree));
      };
      // Oldest work first: the gradients of block n2 once its gate operand is written and the
      // dk before has been read; L of block n1 once its rows are there and the L before has
      // been read.
      bool ok = mbar_wait_soon(bar(L::kBarQ), 0, ctl);
      int n1 = 0, n2 = 0;
      PollState ps = poll_start();
      uint32_t spins = 0;
      while (ok && n2 < nblk) {
        if (n2 < n1 && mbar_probe(bar(L::kBarGFull), n2 & 1) && (n2 == 0 || mbar_probe(bar(L::kBarDkFree), (n2 - 1) & 1))) {
          tc_fence_after();
          issue_grad(n2);
          ++n2;
        } else if (n1 < nblk && n1 - n2 < 2 && mbar_probe(bar(L::kBarKvFull + n1 % L::kStages), (n1 / L::kStages) & 1) &&
                   (n1 == 0 || mbar_probe(bar(L::kBarLFree), (n1 - 1) & 1))) {
          fence_proxy_async_smem();
          tc_fence_after();
          issue_l(n1);
          ++n1;
          if (static_cast<int>(blockIdx.x) == p.stall_cta) {  // test hook only
            ok = stall_until_limit(ctl);
            break;
          }
        } else {
          if ((++spins & 63u) == 0u && !poll_check(ctl, ps)) {
            ok = false;
            break;
          }
          continue;
        }
        ps.t0 = globaltimer_ns();
      }
      mma_commit(bar(L::kBarDone));
      mma_commit(bar(L::kBarDrain));
      mbar_wait_drain(bar(L::kBarDrain), 0);
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ------------------------------------------------------------ drain of dk
    const int d = tid - 256, quarter = warp - 8;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    float* dk0 = dk + b * p.S_kv * static_cast<int64_t>(D) + d;
    bool ok = *abort_flag == 0;
    for (int i = 0; ok && i < nblk; ++i) {
      ok = __all_sync(0xffffffffu, mbar_wait_soon(bar(L::kBarDkFull), i & 1, ctl));
      if (!ok) break;
      tc_fence_after();
      // (The block's rows were written before its L was formed, long before this.)
      if (quarter * 32 < D) {
        const int4* rows = reinterpret_cast<const int4*>(smem + L::kOffRow) + (i % L::kInfo) * (L::kBI / 4);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x[32];
          tmem_ld32(tmem + lanes + L::kTmemDk + c * 32, x);
          if (c == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kBarDkFree));
          }
          // (Four rows per load, the same in all lanes: with a shuffle per row the adds of a
          // warp came one latency apart.)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int4 r = rows[8 * c + k];
            if (r.x >= 0) red_add_f32(dk0 + static_cast<int64_t>(r.x) * D, x[4 * k]);
            if (r.y >= 0) red_add_f32(dk0 + static_cast<int64_t>(r.y) * D, x[4 * k + 1]);
            if (r.z >= 0) red_add_f32(dk0 + static_cast<int64_t>(r.z) * D, x[4 * k + 2]);
            if (r.w >= 0) red_add_f32(dk0 + static_cast<int64_t>(r.w) * D, x[4 * k + 3]);
          }
        }
      } else {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kBarDkFree));
      }
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ gate
    const int h = tid;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t row128 = static_cast<uint32_t>(h) * 128u;
    const float wh = h < p.H ? __ldg(p.w + row0 + h) : 0.f;
    float2 s0 = {}, s1 = {};
    bool ok = *abort_flag == 0;
    for (int i = 0; ok && i < nblk; ++i) {
      ok = __all_sync(0xffffffffu, mbar_wait_soon(bar(L::kBarLFull), i & 1, ctl));
      if (!ok) break;
      tc_fence_after();
      float x[64];
      tmem_ld32x2(tmem + lanes + L::kTmemL, tmem + lanes + L::kTmemL + 32, *reinterpret_cast<float(*)[32]>(x),
                  *reinterpret_cast<float(*)[32]>(x + 32));
      tc_fence_before();
      mbar_arrive(bar(L::kBarLFree));
      // (This wait has completed, as the block's L needed its rows; it orders the reads.)
      ok = __all_sync(0xffffffffu, mbar_wait_soon(bar(L::kBarKvFull + i % L::kStages), (i / L::kStages) & 1, ctl));
      if (ok && i > 0) ok = __all_sync(0xffffffffu, mbar_wait_soon(bar(L::kBarGFree), (i - 1) & 1, ctl));
      if (!ok) break;
      const float4* gq = reinterpret_cast<const float4*>(smem + L::kOffG) + (i % L::kInfo) * (L::kBI / 4);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t w4[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 gv = gq[2 * c + k];
          const float* xs = x + 8 * c + 4 * k;
          // (A NaN's product with the gradient is one; its gate is 0.)
          auto relu = [](float v) {
            float y;
            asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(v));
            return y;
          };
          s0 = fma2(make_float2(gv.x, gv.y), make_float2(relu(xs[0]), relu(xs[1])), s0);
          s1 = fma2(make_float2(gv.z, gv.w), make_float2(relu(xs[2]), relu(xs[3])), s1);
          const float2 a = mul2(make_float2(gv.x, gv.y), make_float2(wh, wh)), e = mul2(make_float2(gv.z, gv.w), make_float2(wh, wh));
          w4[2 * k] = pack_bf16x2(xs[0] > 0.f ? a.x : 0.f, xs[1] > 0.f ? a.y : 0.f);
          w4[2 * k + 1] = pack_bf16x2(xs[2] > 0.f ? e.x : 0.f, xs[3] > 0.f ? e.y : 0.f);
        }
        st_shared_v4(base + L::kOffGate + row128 + ((static_cast<uint32_t>(c) ^ static_cast<uint32_t>(h & 7)) << 4), w4[0], w4[1], w4[2],
                     w4[3]);
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(L::kBarGFull));
    }
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait_soon(bar(L::kBarDone), 0, ctl));
    if (ok) {
      tc_fence_after();
      if (h < p.H) dw[row0 + h] = (s0.x + s0.y) + (s1.x + s1.y);
      // dq, bf16, as 64-column tiles in dq's swizzled layout (the ring is free: every MMA has
      // completed).
#pragma unroll 1
      for (int cc = 0; cc < L::kChunks; ++cc) {
#pragma unroll 1
        for (int u = 0; u < 2; ++u) {
          float v[32];
          if (nblk > 0) {
            tmem_ld32(tmem + lanes + L::kTmemDq + cc * 64 + u * 32, v);
          } else {                                       // no valid slot: the gradient is 0
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = 0.f;
          }
          const uint32_t row = base + L::kOffKv + static_cast<uint32_t>(cc) * L::kQChunkBytes + row128;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t piece = static_cast<uint32_t>(4 * u + k);
            st_shared_v4(row + ((piece ^ (static_cast<uint32_t>(h) & 7u)) << 4), pack_bf16x2(v[8 * k], v[8 * k + 1]),
                         pack_bf16x2(v[8 * k + 2], v[8 * k + 3]), pack_bf16x2(v[8 * k + 4], v[8 * k + 5]),
                         pack_bf16x2(v[8 * k + 6], v[8 * k + 7]));
          }
        }
      }
    }
    // Every gate thread arrives (also after a failed wait); one ships the tiles.
    fence_proxy_async_smem();
    mbar_arrive(bar(L::kBarStaged));
    if (tid == 0) {
      if (mbar_wait_soon(bar(L::kBarStaged), 0, ctl) && *abort_flag == 0) {
        for (int cc = 0; cc < L::kChunks; ++cc)
          tma_store_2d(&tm_dq, base + L::kOffKv + static_cast<uint32_t>(cc) * L::kQChunkBytes, cc * 64, static_cast<int>(row0));
        bulk_commit_group();
        bulk_wait_group0();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 6) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

template <int D>
cudaError_t launch_fwd_impl(const IdxParams& p, const __nv_bfloat16* q, float* scores, cudaStream_t stream) {
  using L = FwdLayout<D>;
  const auto kern = smqa_indexer_scores_kernel<D>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), L::kSmem, allowed);
  if (e != cudaSuccess) return e;
  kern<<<p.B * p.S, L::kThreads, L::kSmem, stream>>>(p, q, scores);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_bwd_impl(const CUtensorMap& tq, const CUtensorMap& tdq, const IdxParams& p, float* dw, float* dk, cudaStream_t stream) {
  using L = BwdLayout<D>;
  const auto kern = smqa_indexer_scores_bwd_kernel<D>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), L::kSmem, allowed);
  if (e != cudaSuccess) return e;
  kern<<<p.B * p.S, L::kThreads, L::kSmem, stream>>>(tq, tdq, p, dw, dk);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_indexer_scores(const IdxParams& p, const __nv_bfloat16* q, float* scores, cudaStream_t stream) {
  return p.D == 64 ? launch_fwd_impl<64>(p, q, scores, stream) : launch_fwd_impl<128>(p, q, scores, stream);
}
cudaError_t launch_indexer_scores_bwd(const CUtensorMap& tq, const CUtensorMap& tdq, const IdxParams& p, float* dw, float* dk,
                                      cudaStream_t stream) {
  return p.D == 64 ? launch_bwd_impl<64>(tq, tdq, p, dw, dk, stream) : launch_bwd_impl<128>(tq, tdq, p, dw, dk, stream);
}

}  // namespace smqa

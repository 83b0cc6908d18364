// smqa_paged.cu -- the 8-bit paged kv cache on sm_103a: the step's block
// table and slots from request lengths, the release of pages, the quantising
// write of new rows, and the argument checks of the attention that reads it.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdio>

#include "smqa_internal.h"
#include "smqa_paged.cuh"

namespace smqa {

namespace {

// ---------------------------------------------------------------------------
// Plan: block table, offsets, positions and slots
// ---------------------------------------------------------------------------
struct PlanParams {
  const int32_t *ctx, *qry, *table, *free_pages, *free_count;
  int R, W, page_shift, n_pages, pool, N;
  int32_t *table_out, *free_count_out, *seq, *cu, *req, *pos, *slot;
};

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxR = 16384;

__device__ __forceinline__ int clamp_int(int64_t v) {
  return static_cast<int>(v > 0x7fffffff ? 0x7fffffff : v);
}

// Every CTA scans the lengths of all R requests (tokens and pages needed, two
// sums at once) into shared memory, then fills its share of the table and of
// the tokens: the scan is cheaper than a second launch.  kInPlace: the CTAs
// are one cluster, and nothing is written before all have read the lengths
// and free_count, which the outputs may overwrite.
template <bool kInPlace>
__global__ void __launch_bounds__(kPlanThreads) smqa_paged_plan_kernel(const PlanParams p) {
  extern __shared__ int32_t sm[];
  int32_t* s_cu = sm;                // [R + 1] first token of each request
  int32_t* s_pg = sm + p.R + 1;      // [R]     first new page of each request
  __shared__ int64_t warp_tok[32], warp_pg[32];
  __shared__ int64_t carry[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int page = 1 << p.page_shift;
  if (tid == 0) carry[0] = carry[1] = 0;
  __syncthreads();
  // (Launched beside the kernel before, whose results are read from here on; the
  // next one may be launched beside this.)
  grid_dependency_wait();
  grid_dependents_launch();
  for (int r0 = 0; r0 < p.R; r0 += kPlanThreads) {
    const int r = r0 + tid;
    int64_t tok = 0, pg = 0;
    if (r < p.R) {
      const int64_t c = max(p.ctx[r], 0), q = max(p.qry[r], 0);
      const int64_t have = (c + page - 1) >> p.page_shift, full = (c + q + page - 1) >> p.page_shift;
      tok = q;
      pg = min(full, static_cast<int64_t>(p.W)) - min(have, static_cast<int64_t>(p.W));
    }
    int64_t a = tok, b = pg;  // inclusive sums over the warp
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, a, off), y = __shfl_up_sync(0xffffffffu, b, off);
      if (lane >= off) { a += x; b += y; }
    }
    if (lane == 31) { warp_tok[warp] = a; warp_pg[warp] = b; }
    __syncthreads();
    if (warp == 0) {
      int64_t x = warp_tok[lane], y = warp_pg[lane];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, x, off), v = __shfl_up_sync(0xffffffffu, y, off);
        if (lane >= off) { x += u; y += v; }
      }
      warp_tok[lane] = x;
      warp_pg[lane] = y;
    }
    __syncthreads();
    const int64_t tb = carry[0] + (warp ? warp_tok[warp - 1] : 0);
    const int64_t pb = carry[1] + (warp ? warp_pg[warp - 1] : 0);
    if (r < p.R) {
      s_cu[r] = clamp_int(tb + a - tok);
      s_pg[r] = clamp_int(pb + b - pg);
    }
    __syncthreads();
    if (tid == kPlanThreads - 1) {
      carry[0] = tb + a;
      carry[1] = pb + b;
    }
    __syncthreads();
  }
  if (tid == 0) s_cu[p.R] = clamp_int(carry[0]);
  const int need = clamp_int(carry[1]);
  const int count = min(max(*p.free_count, 0), p.pool);
  __syncthreads();

  const int gthreads = gridDim.x * kPlanThreads;
  const int gid = blockIdx.x * kPlanThreads + tid;
  auto stack = [&](int64_t nth) {  // the nth page taken in this step
    const int64_t at = count - 1 - nth;
    return at >= 0 ? load(p.free_pages + at) : -1;
  };
  // Tokens.  (Before the barrier of the in-place form: they read ctx.)
  const int total = s_cu[p.R];
  for (int64_t i = gid; i < p.N; i += gthreads) {
    const int t = static_cast<int>(i);
    int r = -1, ps = -1, sl = -1;
    if (t < total) {
      int lo = 0, hi = p.R;  // the last r with s_cu[r] <= t (it has tokens)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= t) lo = mid; else hi = mid;
      }
      r = lo;
      const int c = max(p.ctx[r], 0);
      ps = c + (t - s_cu[r]);
      const int col = ps >> p.page_shift;
      if (col < p.W) {
        const int have = (c + page - 1) >> p.page_shift;
        const int pg = col < have ? p.table[static_cast<int64_t>(r) * p.W + col]
                                  : stack(static_cast<int64_t>(s_pg[r]) + col - have);
        if (static_cast<unsigned>(pg) < static_cast<unsigned>(p.n_pages))
          sl = (pg << p.page_shift) + (ps & (page - 1));
      }
    }
    p.req[t] = r;
    p.pos[t] = ps;
    p.slot[t] = sl;
  }
  // The table: all of it, or only the new entries when it is updated in place.
  if (p.table_out != p.table) {
    const int64_t n = static_cast<int64_t>(p.R) * p.W;
    for (int64_t e = gid; e < n; e += gthreads) {
      const int r = static_cast<int>(e / p.W), col = static_cast<int>(e - static_cast<int64_t>(r) * p.W);
      const int64_t c = max(p.ctx[r], 0), q = max(p.qry[r], 0);
      const int64_t have = (c + page - 1) >> p.page_shift, full = (c + q + page - 1) >> p.page_shift;
      p.table_out[e] = (col >= have && col < full) ? stack(static_cast<int64_t>(s_pg[r]) + col - have) : p.table[e];
    }
  } else {
    for (int r = gid >> 5; r < p.R; r += gthreads >> 5) {
      const int64_t c = max(p.ctx[r], 0), q = max(p.qry[r], 0);
      const int64_t have = (c + page - 1) >> p.page_shift;
      const int64_t full = min((c + q + page - 1) >> p.page_shift, static_cast<int64_t>(p.W));
      for (int64_t col = have + lane; col < full; col += 32)
        p.table_out[static_cast<int64_t>(r) * p.W + col] = stack(s_pg[r] + col - have);
    }
  }
  if constexpr (kInPlace) {
    __syncthreads();
    cluster_sync();
  }
  for (int r = gid; r < p.R; r += gthreads)
    p.seq[r] = clamp_int(static_cast<int64_t>(max(p.ctx[r], 0)) + max(p.qry[r], 0));
  for (int r = gid; r <= p.R; r += gthreads) p.cu[r] = s_cu[r];
  if (gid == 0) *p.free_count_out = count - need;
}

// ---------------------------------------------------------------------------
// Release: pages of finished requests back on the stack
// ---------------------------------------------------------------------------
// One CTA: the stack's order must not depend on timing.  A warp takes a row;
// rows are numbered by a scan over their counts.
__global__ void __launch_bounds__(1024)
    smqa_paged_release_kernel(int32_t* table, int32_t* seq, const uint8_t* release, int R, int W,
                              int n_pages, int32_t* free_pages, int32_t* free_count, int pool) {
  __shared__ int32_t cnt[32];
  __shared__ int64_t base;                               // (pages counted, fitting or not)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) base = min(max(*free_count, 0), pool);
  __syncthreads();
  for (int64_t r0 = 0; r0 < R; r0 += 32) {
    const int64_t r = r0 + warp;
    const bool mine = r < R && release[r] != 0;
    int32_t* row = table + r * W;
    int n = 0;
    if (mine)
      for (int64_t c0 = 0; c0 < W; c0 += 32) {
        const int pg = c0 + lane < W ? row[c0 + lane] : -1;
        n += __popc(__ballot_sync(0xffffffffu,
                                  static_cast<unsigned>(pg) < static_cast<unsigned>(n_pages)));
      }
    if (lane == 0) cnt[warp] = n;
    __syncthreads();
    int64_t at = base;
    for (int w = 0; w < warp; ++w) at += cnt[w];
    if (mine) {
      for (int64_t c0 = 0; c0 < W; c0 += 32) {
        const bool in = c0 + lane < W;
        const int pg = in ? row[c0 + lane] : -1;
        const bool ok = static_cast<unsigned>(pg) < static_cast<unsigned>(n_pages);
        const unsigned m = __ballot_sync(0xffffffffu, ok);
        const int64_t k = at + __popc(m & ((1u << lane) - 1));
        if (ok && k < pool) free_pages[k] = pg;
        if (in) row[c0 + lane] = -1;
        at += __popc(m);
      }
      if (lane == 0 && seq) seq[r] = 0;
    }
    __syncthreads();
    if (threadIdx.x == 0)
      for (int w = 0; w < 32; ++w) base += cnt[w];
    __syncthreads();
  }
  if (threadIdx.x == 0) *free_count = static_cast<int>(min(base, static_cast<int64_t>(pool)));
}

// ---------------------------------------------------------------------------
// Append: new rows into the cache, one power-of-two scale per page
// ---------------------------------------------------------------------------
// The least k >= -60 with amax <= 448 * 2^k, from amax's exponent and
// mantissa (448 = 1.75 * 2^8): amax = m 2^e with 1 <= m < 2.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127;
  const int k = e - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(k, -60);
}

// 16 rows per CTA, a warp each.  The warp of a run's first row (a run:
// consecutive rows with ascending slots in one page) does the whole run if it is
// short; a longer one, and the earlier rows of a page whose scale has grown, are
// left to the whole CTA.  A run's rows are one flat range in kv_new and in the
// cache, read twice, the second time from L1.  Bound by latency: 8192 rows
// (D=512, pages of 64: 130 runs) took 11.9 us with a CTA per row, most of which
// left at once, and take 7.0 us so; 128 single rows 2.5 us.
constexpr int kAppendWarps = 16, kAppendThreads = 32 * kAppendWarps;
constexpr int kShortRun = 8;                             // rows (512 runs of 6: 4.4 us by warps, 6.1 by CTAs)

// The largest finite magnitude of uint4 i, i + step, ... below n, as bf16 bits
// (which order like values).
__device__ __forceinline__ uint32_t largest(const uint4* src, int i, int step, int n) {
  uint32_t top = 0;
#pragma unroll 8
  for (; i < n; i += step) {
    const uint4 v = load(src + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t lo = w[k] & 0x7fffu, hi = (w[k] >> 16) & 0x7fffu;
      top = max(top, lo < 0x7f80u ? lo : 0u);
      top = max(top, hi < 0x7f80u ? hi : 0u);
    }
  }
  return top;
}
// Their codes under a scale of 1 / inv.
__device__ __forceinline__ void encode(const uint4* src, uint2* dst, int i, int step, int n, float inv) {
  auto code = [&](uint32_t w) {  // two bf16 -> two codes; an infinity becomes NaN
    float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xffff0000u);
    lo = (w & 0x7fffu) >= 0x7f80u ? __uint_as_float(0x7fffffffu) : lo * inv;
    hi = ((w >> 16) & 0x7fffu) >= 0x7f80u ? __uint_as_float(0x7fffffffu) : hi * inv;
    return static_cast<uint32_t>(e4m3x2(lo, hi));
  };
#pragma unroll 8
  for (; i < n; i += step) {
    const uint4 v = load(src + i);
    dst[i] = make_uint2(code(v.x) | (code(v.y) << 16), code(v.z) | (code(v.w) << 16));
  }
}
// Codes times f = 2^-k.
__device__ __forceinline__ void rescale(uint4* row, int i, int step, int n, float f) {
#pragma unroll 8
  for (; i < n; i += step) {
    uint4 v = row[i];
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 a = e4m3x2_value(static_cast<uint16_t>(w[k])), b = e4m3x2_value(static_cast<uint16_t>(w[k] >> 16));
      w[k] = e4m3x2(a.x * f, a.y * f) | (static_cast<uint32_t>(e4m3x2(b.x * f, b.y * f)) << 16);
    }
    row[i] = v;
  }
}

__global__ void __launch_bounds__(kAppendThreads, 2)
    smqa_paged_append_kernel(const __nv_bfloat16* kv_new, const int32_t* slots, int T, int D,
                             int page_shift, int n_slots, uint8_t* cache, float* scales) {
  __shared__ int runs, grown;                            // long runs: first row, number of rows;
  __shared__ int run_at[kAppendWarps], run_rows[kAppendWarps];
  __shared__ int grown_to[kAppendWarps];                 // pages whose scale has grown: up to this
  __shared__ float grown_by[kAppendWarps];               // slot, by 1 / f
  __shared__ uint32_t warp_top[2][kAppendWarps];         // (of even and odd runs)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int page = 1 << page_shift;
  if (tid == 0) runs = grown = 0;
  __syncthreads();
  grid_dependency_wait();                                // (launched beside the kernel before,
  grid_dependents_launch();                              // the next one beside this)
  {
    // The slots of the row before, of the warp's row and of those behind it that
    // can be in its page.
    const int t = blockIdx.x * kAppendWarps + warp;
    const int before = t > 0 && t <= T ? load(slots + t - 1) : -2;
    int x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = 32 * k + lane;
      x[k] = i < page && i < T - t ? load(slots + t + i) : -2;
    }
    const int s0 = __shfl_sync(0xffffffffu, x[0], 0);
    const int off = s0 & (page - 1);
    if (static_cast<unsigned>(s0) < static_cast<unsigned>(n_slots) && (off == 0 || before != s0 - 1)) {
      int rows = 0;                                      // the first that does not go on ends the run
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = 32 * k + lane;
        const unsigned same = __ballot_sync(0xffffffffu, i < page - off && x[k] == s0 + i);
        if (rows == 32 * k) rows += same == 0xffffffffu ? 32 : __ffs(~same) - 1;
      }
      if (rows <= kShortRun) {
        const int64_t pg = s0 >> page_shift;
        const float had = __shfl_sync(0xffffffffu, off && lane == 0 ? scales[pg] : 0.f, 0);  // (which lane 0 writes)
        const int n = rows * D / 8;
        const uint4* src = reinterpret_cast<const uint4*>(kv_new + static_cast<int64_t>(t) * D);
        const uint32_t top = __reduce_max_sync(0xffffffffu, largest(src, lane, 32, n));
        const float s = fmaxf(pow2f(scale_exponent(__uint_as_float(top << 16))), had);
        encode(src, reinterpret_cast<uint2*>(cache + static_cast<int64_t>(s0) * D), lane, 32, n, 1.f / s);
        if (lane == 0) {
          scales[pg] = s;
          if (off && s > had) {
            const int i = atomicAdd(&grown, 1);
            grown_to[i] = s0;
            grown_by[i] = had / s;
          }
        }
      } else if (lane == 0) {
        const int i = atomicAdd(&runs, 1);
        run_at[i] = t;
        run_rows[i] = rows;
      }
    }
  }
  __syncthreads();
  const int n_grown = grown, n_runs = runs;
  for (int i = 0; i < n_grown; ++i) {
    const int off = grown_to[i] & (page - 1);
    rescale(reinterpret_cast<uint4*>(cache + static_cast<int64_t>(grown_to[i] - off) * D), tid, kAppendThreads, off * D / 16,
            grown_by[i]);
  }
  for (int i = 0; i < n_runs; ++i) {
    const int t = run_at[i], s0 = load(slots + t), off = s0 & (page - 1);
    const int64_t pg = s0 >> page_shift;
    const float had = off ? scales[pg] : 0.f;            // (written behind a barrier)
    const int n = run_rows[i] * D / 8;
    const uint4* src = reinterpret_cast<const uint4*>(kv_new + static_cast<int64_t>(t) * D);
    uint32_t top = __reduce_max_sync(0xffffffffu, largest(src, tid, kAppendThreads, n));
    if (lane == 0) warp_top[i & 1][warp] = top;
    __syncthreads();
    for (int w = 0; w < kAppendWarps; ++w) top = max(top, warp_top[i & 1][w]);
    const float s = fmaxf(pow2f(scale_exponent(__uint_as_float(top << 16))), had);
    if (off && s > had) rescale(reinterpret_cast<uint4*>(cache + (pg << page_shift) * D), tid, kAppendThreads, off * D / 16, had / s);
    encode(src, reinterpret_cast<uint2*>(cache + static_cast<int64_t>(s0) * D), tid, kAppendThreads, n, 1.f / s);
    if (tid == 0) scales[pg] = s;
  }
}

int page_shift_of(int page_size) {
  switch (page_size) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
  }
  return -1;
}

smqa_status refuse(smqa_status st, const char* why) {
  set_last_error(why);
  return st;
}

constexpr int64_t kLim = int64_t{1} << 31;
// Slots of a token: the attention rounds them up to blocks of 128 in 32 bits.
constexpr int64_t kMaxSlots = kLim - 128;

smqa_status check_paged(const smqa_paged_shape& s) {
  if (s.T < 0 || s.R <= 0 || s.H <= 0 || s.D <= 0 || s.topk < 0 || s.page_size <= 0 ||
      s.max_pages <= 0 || s.n_pages <= 0)
    return refuse(SMQA_ERR_INVALID_ARG, "non-positive size in paged shape");
  if (s.H > 128 || (s.D != 64 && s.D != 512) || page_shift_of(s.page_size) < 0 ||
      static_cast<int64_t>(s.n_pages) * s.page_size >= kLim ||
      static_cast<int64_t>(s.max_pages) * s.page_size > kMaxSlots || s.topk > kMaxSlots ||
      static_cast<int64_t>(s.T) * std::max(s.H, s.topk) >= kLim)
    return refuse(SMQA_ERR_UNSUPPORTED,
                  "unsupported paged shape (need 1<=H<=128, D in {64,512}, page_size in "
                  "{16,32,64,128}, topk and max_pages * page_size <= 2^31 - 128, sizes < 2^31)");
  return SMQA_OK;
}

}  // namespace

}  // namespace smqa

using namespace smqa;

extern "C" {

smqa_status smqa_paged_plan(const int32_t* context_lens, const int32_t* query_lens,
                            const int32_t* block_table, const int32_t* free_pages,
                            const int32_t* free_count, int32_t R, int32_t max_pages,
                            int32_t page_size, int32_t n_pages, int32_t pool,
                            int32_t max_tokens, int32_t* block_table_out,
                            int32_t* free_count_out, int32_t* seq_lens, int32_t* cu_query,
                            int32_t* token_req, int32_t* positions, int32_t* slot_mapping,
                            cudaStream_t stream) {
  if (R <= 0 || max_pages <= 0 || page_size <= 0 || n_pages <= 0 || pool < 0 || max_tokens < 0)
    return refuse(SMQA_ERR_INVALID_ARG, "non-positive size in paged plan");
  const int shift = page_shift_of(page_size);
  if (R > kPlanMaxR || shift < 0 || static_cast<int64_t>(n_pages) * page_size >= kLim ||
      static_cast<int64_t>(max_pages) * page_size >= kLim)
    return refuse(SMQA_ERR_UNSUPPORTED,
                  "unsupported paged plan (need R<=16384, page_size in {16,32,64,128}, "
                  "sizes < 2^31)");
  const void* need[] = {context_lens, query_lens,     block_table, free_count, block_table_out,
                        free_count_out, seq_lens, cu_query};
  for (const void* q : need)
    if (!q || !is_aligned(q, 4)) return refuse(SMQA_ERR_INVALID_ARG, "null or misaligned pointer");
  const void* maybe[] = {token_req, positions, slot_mapping};
  for (const void* q : maybe)
    if ((max_tokens > 0 && !q) || !is_aligned(q, 4))
      return refuse(SMQA_ERR_INVALID_ARG, "null or misaligned pointer");
  if ((pool > 0 && !free_pages) || !is_aligned(free_pages, 4))
    return refuse(SMQA_ERR_INVALID_ARG, "null or misaligned pointer");
  const bool in_place = free_count_out == free_count;
  if (seq_lens == context_lens && !in_place)
    return refuse(SMQA_ERR_INVALID_ARG,
                  "seq_lens may be context_lens only when free_count_out is free_count");
  PlanParams p{context_lens, query_lens, block_table, free_pages, free_count, R, max_pages, shift,
               n_pages, pool, max_tokens, block_table_out, free_count_out, seq_lens, cu_query,
               token_req, positions, slot_mapping};
  const size_t smem = (static_cast<size_t>(R) * 2 + 1) * sizeof(int32_t);
  const auto kern = in_place ? smqa_paged_plan_kernel<true> : smqa_paged_plan_kernel<false>;
  static std::atomic<uint64_t> allowed[2];
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), (2 * kPlanMaxR + 1) * 4, allowed[in_place]);
  if (e != cudaSuccess) return cuda_failure(e, "paged plan launch");
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (in_place) {
    cfg.gridDim = dim3(8);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 8;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  } else {
    const int64_t work = std::max<int64_t>(static_cast<int64_t>(R) * max_pages, max_tokens);
    cfg.gridDim = dim3(static_cast<unsigned>(
        std::min<int64_t>(kSMs, std::max<int64_t>(1, (work + kPlanThreads - 1) / kPlanThreads))));
  }
  e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) return cuda_failure(e, "paged plan launch");
  return SMQA_OK;
}

smqa_status smqa_paged_release(int32_t* block_table, int32_t* seq_lens, const uint8_t* release,
                               int32_t R, int32_t max_pages, int32_t n_pages,
                               int32_t* free_pages, int32_t* free_count, int32_t pool,
                               cudaStream_t stream) {
  if (R <= 0 || max_pages <= 0 || n_pages <= 0 || pool <= 0)
    return refuse(SMQA_ERR_INVALID_ARG, "non-positive size in paged release");
  if (!block_table || !release || !free_pages || !free_count || !is_aligned(block_table, 4) ||
      !is_aligned(free_pages, 4) || !is_aligned(free_count, 4) || !is_aligned(seq_lens, 4))
    return refuse(SMQA_ERR_INVALID_ARG, "null or misaligned pointer");
  smqa_paged_release_kernel<<<1, 1024, 0, stream>>>(block_table, seq_lens, release, R, max_pages,
                                                    n_pages, free_pages, free_count, pool);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_failure(e, "paged release launch");
  return SMQA_OK;
}

smqa_status smqa_paged_append(const void* kv_new, const int32_t* slot_mapping, int32_t T,
                              int32_t D, int32_t page_size, int32_t n_pages, void* kv_cache,
                              float* kv_scales, cudaStream_t stream) {
  if (T < 0 || D <= 0 || page_size <= 0 || n_pages <= 0)
    return refuse(SMQA_ERR_INVALID_ARG, "non-positive size in paged append");
  const int shift = page_shift_of(page_size);
  if ((D != 64 && D != 512) || shift < 0 || static_cast<int64_t>(n_pages) * page_size >= kLim)
    return refuse(SMQA_ERR_UNSUPPORTED,
                  "unsupported paged append (need D in {64,512}, page_size in {16,32,64,128}, "
                  "sizes < 2^31)");
  if (T == 0) return SMQA_OK;
  if (!kv_new || !slot_mapping || !kv_cache || !kv_scales || !is_aligned(kv_new, 16) ||
      !is_aligned(kv_cache, 16) || !is_aligned(slot_mapping, 4) || !is_aligned(kv_scales, 4))
    return refuse(SMQA_ERR_INVALID_ARG, "null or misaligned pointer");
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((T - 1) / kAppendWarps + 1));
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, smqa_paged_append_kernel, static_cast<const __nv_bfloat16*>(kv_new), slot_mapping, T, D,
      shift, n_pages * page_size, static_cast<uint8_t*>(kv_cache), kv_scales);
  if (e != cudaSuccess) return cuda_failure(e, "paged append launch");
  return SMQA_OK;
}

size_t smqa_paged_fwd_workspace_bytes(smqa_paged_shape shape) {
  return check_paged(shape) == SMQA_OK && shape.T > 0 ? paged_fwd_workspace(shape) : 0;
}

smqa_status smqa_paged_fwd(const void* q, const void* kv_cache, const float* kv_scales,
                           const float* attn_sink, const int32_t* block_table,
                           const int32_t* seq_lens, const int32_t* token_req,
                           const int32_t* positions, const int32_t* topk_idxs,
                           smqa_paged_shape shape, float sm_scale, void* o, float* lse,
                           void* workspace, size_t workspace_bytes, unsigned flags,
                           cudaStream_t stream) {
  const smqa_status sc = check_paged(shape);
  if (sc != SMQA_OK) return sc;
  if (flags & ~SMQA_FLAG_ZERO_PADDING) return refuse(SMQA_ERR_INVALID_ARG, "bad flags");
  if (shape.T == 0) return SMQA_OK;
  const size_t need = smqa_paged_fwd_workspace_bytes(shape);
  if (!q || !kv_cache || !kv_scales || !attn_sink || !block_table || !seq_lens || !token_req ||
      !o || !lse || (shape.topk > 0 ? !topk_idxs : !positions) || (need != 0 && !workspace) ||
      !is_aligned(q, 16) || !is_aligned(kv_cache, 16) || !is_aligned(o, 16) ||
      !is_aligned(kv_scales, 4) || !is_aligned(attn_sink, 4) || !is_aligned(block_table, 4) ||
      !is_aligned(seq_lens, 4) || !is_aligned(token_req, 4) || !is_aligned(positions, 4) ||
      !is_aligned(topk_idxs, 4) || !is_aligned(lse, 4) || !is_aligned(workspace, 256))
    return refuse(SMQA_ERR_INVALID_ARG, "null or misaligned pointer");
  if (workspace_bytes < need) {
    char msg[128];
    std::snprintf(msg, sizeof msg, "workspace too small (%zu < %zu bytes)", workspace_bytes, need);
    return refuse(SMQA_ERR_UNSUPPORTED, msg);
  }
  PagedFwdParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.cache = static_cast<const uint8_t*>(kv_cache);
  p.scales = kv_scales;
  p.sink = attn_sink;
  p.table = block_table;
  p.seq_lens = seq_lens;
  p.token_req = token_req;
  p.positions = positions;
  p.idx = shape.topk > 0 ? topk_idxs : nullptr;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.T = shape.T;
  p.R = shape.R;
  p.H = shape.H;
  p.D = shape.D;
  p.topk = shape.topk;
  p.max_pages = shape.max_pages;
  p.n_pages = shape.n_pages;
  p.page_shift = page_shift_of(shape.page_size);
  p.scale_log2 = effective_scale(sm_scale, shape.D) * 1.4426950408889634f;
  p.zero_padding = (flags & SMQA_FLAG_ZERO_PADDING) ? 1 : 0;
  p.ws = static_cast<uint8_t*>(workspace);
  cudaError_t e;
  p.status = device_status_word(&e);
  if (!p.status) return cuda_failure(e, "status word");
  p.limit_ns = current_wait_limit_ns();
  p.stall_cta = current_stall_cta();
  e = launch_paged_fwd(p, shape, stream);
  if (e != cudaSuccess) return cuda_failure(e, "paged fwd launch");
  return SMQA_OK;
}

}  // extern "C"

// smqa_paged_fwd.cu -- sparse MQA over the 8-bit paged cache on sm_103a.
//
// Per token t and head h, over the valid slots j (an index list, or every
// position up to the token's own), with k_j = s_j c_j the cache row (s_j its
// page's scale, c_j its e4m3 codes):
//   x_j = sm_scale log2(e) q.k_j,  l = sum_j 2^x_j + 2^(sink log2(e)),
//   O = sum_j 2^x_j k_j / l,  lse = log2 l.
//
// The codes feed the tensor core as they lie in the cache (kind::f8f6f4): a
// conversion to bf16 would double the shared memory a row takes and its
// traffic.  What multiplies them is split in two e4m3 pieces instead, which
// costs as much tensor time as one bf16 operand (e4m3 runs at twice the rate):
//   q  = 2^-k (hi + lo / 32), k per row so that the largest value of 2^k q
//        lies in [128, 256): bf16's 8 bits fit the two pieces exactly down to
//        2^-22 of the row's largest value;
//   w' = 2^(6 + y_j - m), y_j = x_j + log2 s_j the weight that multiplies the
//        codes, m the running maximum of y, w' = hi + lo: a relative error of
//        2^-8 + 2^-11 at most, down to 2^-16 of the largest weight.  m may lag
//        behind the true maximum by 2.75 (w' <= 2^8.75 < 448, e4m3's largest),
//        so that O is seldom rescaled.  l adds w' / s_j in fp32.
//
// Work: the tokens' blocks of 128 slots form one sequence, cut into equal
// ranges; a CTA takes one range for one group of up to 64 heads, so a lone
// token's slots and an uneven batch are spread over the whole GPU alike.  A
// token whose blocks lie in one range is finished there; otherwise each CTA
// leaves its O (unnormalised), m and l in the workspace, at most two per CTA,
// and a second kernel joins them.  The two head groups of a token run side by
// side in neighbouring CTAs, so its rows come from HBM once.
//
// Per block (D = 512), 288 threads, one CTA per SM:
//   gather (warps 5-8)   slot -> page -> row, and the rows by 16-byte cp.async
//                        into a 128-byte-swizzled tile [D/128][128 slots][128],
//                        three tiles in a ring, a warp's 32 rows freed and
//                        refilled on their own; the slots' scale factors;
//   MMA (warp 4)         S = Q.K^T: M = 128 (64 heads x 2 pieces, A in TMEM),
//                        N = 128 slots; O^T += V^T.P^T: M = 128 of D (A: the
//                        same tile read MN-major), N = 64 heads, K = 128 slots,
//                        for both pieces of P;
//   softmax (warps 0-3)  two lanes per head (piece hi / lo of its row of S,
//                        then slots 0-63 / 64-127): weights, their two pieces
//                        to shared memory, Q's pieces into TMEM at the start of
//                        a token and O^T out of it at the end.
// TMEM: S 128 columns, O^T D/2, Q D/4.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "smqa_internal.h"
#include "smqa_paged.cuh"

namespace smqa {

namespace {

constexpr int kBlk = 128;                 // slots per block
constexpr int kHeads = 64;                // heads per CTA
constexpr int kThreads = 288;
constexpr int kSoftmaxThreads = 128;
constexpr int kMmaWarp = 4, kGatherWarp0 = 5;
constexpr float kShift = 6.f;             // weights are 2^6 at the running maximum
constexpr float kLag = 2.75f;             // how far the maximum may lag behind

template <int D>
struct PagedLayout {
  static constexpr int kChunks = D < 128 ? 1 : D / 128;      // 128-byte pieces of a row
  static constexpr uint32_t kChunkBytes = kBlk * 128;
  static constexpr uint32_t kStageBytes = kChunks * kChunkBytes;
  static constexpr int kStages = D == 512 ? 3 : 6;
  static constexpr uint32_t kPieceBytes = kHeads * 128;      // one piece of P^T: 64 heads x 128 slots
  static constexpr uint32_t kQStage = 32 * 64;               // per warp: 32 rows x 64 bytes
  static constexpr int kMeta = 132;                          // floats per array (halves 16 bytes apart)
  static constexpr uint32_t kOffP = kStages * kStageBytes;
  static constexpr uint32_t kOffQ = kOffP + 2 * kPieceBytes;
  static constexpr uint32_t kOffA = kOffQ + 4 * kQStage;     // [kStages][3][kMeta]: a, c, r
  static constexpr uint32_t kOffFlags = kOffA + kStages * 3 * kMeta * 4;  // [kStages]
  static constexpr uint32_t kOffHead = (kOffFlags + kStages * 4 + 15) & ~15u;  // float [64]
  static constexpr uint32_t kOffBar = kOffHead + kHeads * 4;
  static constexpr int kBarFull = 0;                         // [kStages]
  static constexpr int kBarEmpty = kBarFull + kStages;       // [kStages][4], a gather warp's rows
  static constexpr int kBarSFull = kBarEmpty + 4 * kStages;
  static constexpr int kBarSFree = kBarSFull + 1;
  static constexpr int kBarPFull = kBarSFree + 1;
  static constexpr int kBarPDone = kBarPFull + 1;            // P and its tile used, O up to date
  static constexpr int kBarQFull = kBarPDone + 1;
  static constexpr int kBarDrain = kBarQFull + 1;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr uint32_t kOffCtl = kOffBar + 8 * kNumBars;  // TMEM base, abort flag
  static constexpr uint32_t kOffRange = kOffCtl + 8;         // range of the CTA, scan space
  static constexpr uint32_t kSmem = kOffRange + 160 + 1024;  // + alignment
  static_assert(kSmem <= 232448, "shared memory budget");
  static constexpr uint32_t kTmemS = 0, kTmemO = 128;
  static constexpr uint32_t kTmemQ = kTmemO + kChunks * kHeads;
  static constexpr uint32_t kTmemCols = D == 512 ? 512 : 256;
  static_assert(kTmemQ + D / 4 <= kTmemCols, "TMEM budget");
};

// The range of blocks of a CTA: from block `off` of token `tok`, `count` blocks.
struct Range {
  int tok, off;
  int64_t count;
};

// Flags of a ring entry.
enum : int { kFirst = 1, kLast = 2, kFinal = 4 };

// What a CTA leaves in the workspace: the token its range starts inside of
// (-1: none) and whether that token goes on behind the range, and the token
// that starts in the range and goes on behind it (-1: none).
struct Leftover {
  int head_tok, head_more, tail_tok, pad;
};
constexpr size_t kLeftoverBytes = 4096;
constexpr int kMaxCtas = static_cast<int>(kLeftoverBytes / sizeof(Leftover));
__host__ __device__ constexpr size_t part_floats(int D) { return static_cast<size_t>(kHeads) * D + 2 * kHeads; }

__device__ __forceinline__ bool live_token(const PagedFwdParams& p, int req) {
  return static_cast<unsigned>(req) < static_cast<unsigned>(p.R);
}
// Slots to look at for token t of request req.
__device__ __forceinline__ int slots_of(const PagedFwdParams& p, int t, int req, int len) {
  if (p.idx) return p.topk;
  const int64_t cap = static_cast<int64_t>(p.max_pages) << p.page_shift;
  const int64_t n = min(min(static_cast<int64_t>(len), static_cast<int64_t>(__ldg(p.positions + t)) + 1), cap);
  return n > 0 ? static_cast<int>(n) : 0;
}
// Blocks of token t: at least one (it writes O = 0), none for padding.
__device__ __forceinline__ int blocks_of(const PagedFwdParams& p, int t) {
  const int req = __ldg(p.token_req + t);
  if (!live_token(p, req)) return 0;
  if (p.idx) return (p.topk + kBlk - 1) / kBlk;
  return max(1, (slots_of(p, t, req, __ldg(p.seq_lens + req)) + kBlk - 1) / kBlk);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) smqa_paged_fwd_kernel(const PagedFwdParams p) {
  using L = PagedLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint32_t base = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (base & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  base += pad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int groups = (p.H + kHeads - 1) / kHeads;
  const int part = blockIdx.x / groups, parts = gridDim.x / groups;
  const int h0 = (blockIdx.x % groups) * kHeads;
  const int heads = min(kHeads, p.H - h0);
  auto bar = [&](int i) -> uint32_t { return base + L::kOffBar + 8u * static_cast<uint32_t>(i); };
  volatile uint32_t* tmem_holder = reinterpret_cast<volatile uint32_t*>(smem + L::kOffCtl);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffCtl + 4);
  const WaitCtl ctl{abort_flag, p.status, p.limit_ns};
  Range* range = reinterpret_cast<Range*>(smem + L::kOffRange);
  int64_t* warp_sum = reinterpret_cast<int64_t*>(smem + L::kOffRange + 16);  // [9]
  int* end_tok = reinterpret_cast<int*>(smem + L::kOffRange + 16 + 72);      // token, its end inside

  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i) mbar_init(bar(L::kBarFull + i), 256);
    for (int i = 0; i < 4 * L::kStages; ++i) mbar_init(bar(L::kBarEmpty + i), 1);
    mbar_init(bar(L::kBarSFull), 1);
    mbar_init(bar(L::kBarSFree), kSoftmaxThreads);
    mbar_init(bar(L::kBarPFull), kSoftmaxThreads);
    mbar_init(bar(L::kBarPDone), 1);
    mbar_init(bar(L::kBarQFull), kSoftmaxThreads);
    mbar_init(bar(L::kBarDrain), 1);
    *abort_flag = *reinterpret_cast<volatile int*>(p.status) != 0 ? 1 : 0;
    range->count = 0;
    end_tok[0] = -1;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(base + L::kOffCtl, L::kTmemCols);
  // Padding tokens belong to no range.
  if (p.zero_padding)
    for (int t = blockIdx.x; t < p.T; t += gridDim.x)
      if (!live_token(p, __ldg(p.token_req + t))) {
        uint4* o = reinterpret_cast<uint4*>(p.o + static_cast<int64_t>(t) * p.H * D);
        for (int i = tid; i < p.H * D / 8; i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
        for (int h = tid; h < p.H; h += kThreads) p.lse[static_cast<int64_t>(t) * p.H + h] = -INFINITY;
      }
  // The CTA's range: the total number of blocks, and the tokens in which the
  // range begins and ends (each thread sums a run of tokens).
  {
    const int per = (p.T + kThreads - 1) / kThreads;
    const int t0 = min(tid * per, p.T), t1 = min(t0 + per, p.T);
    int64_t mine = 0;
    for (int t = t0; t < t1; ++t) mine += blocks_of(p, t);
    int64_t incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += x;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += warp_sum[w];
      total += warp_sum[w];
    }
    const int64_t begin = total * part / parts, end = total * (part + 1) / parts;
    if (begin < end) {
      if (before <= begin && begin < before + mine) {
        int64_t at = before;
        int t = t0, nb = blocks_of(p, t);
        while (at + nb <= begin) {
          at += nb;
          nb = blocks_of(p, ++t);
        }
        range->tok = t;
        range->off = static_cast<int>(begin - at);
        range->count = end - begin;
      }
      if (before < end && end <= before + mine) {
        int64_t at = before;
        int t = t0, nb = blocks_of(p, t);
        while (at + nb < end) {
          at += nb;
          nb = blocks_of(p, ++t);
        }
        end_tok[0] = t;
        end_tok[1] = at + nb == end;   // the token ends with the range
        end_tok[2] = at >= begin;      // and begins in it
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Range rg = *range;
  const uint32_t tmem = *tmem_holder;
  if (tid == 0) {
    Leftover l{-1, 0, -1, 0};
    if (rg.count > 0) {
      if (rg.off > 0) {
        l.head_tok = rg.tok;
        l.head_more = end_tok[0] == rg.tok && !end_tok[1];
      }
      if (!end_tok[1] && end_tok[2]) l.tail_tok = end_tok[0];
    }
    reinterpret_cast<Leftover*>(p.ws)[blockIdx.x] = l;
  }

  if (rg.count > 0 && warp >= kGatherWarp0) {
    // ------------------------------------------------------------ gather
    const int pw = warp - kGatherWarp0;
    const int my = 32 * pw + lane;                       // this thread's slot of the block
    const int meta = my + (my >= 64 ? 4 : 0);
    int64_t left = rg.count;
    int e = 0;                                           // ring entries so far
    bool ok = *abort_flag == 0;
    for (int t = rg.tok, b = rg.off; ok && left > 0; ++t, b = 0) {
      const int nb = blocks_of(p, t);
      if (nb == 0) continue;
      const int req = __ldg(p.token_req + t);
      const int len = __ldg(p.seq_lens + req);
      const int n = slots_of(p, t, req, len);
      const int32_t* idx_row = p.idx ? p.idx + static_cast<int64_t>(t) * p.topk : nullptr;
      const int32_t* tab = p.table + static_cast<int64_t>(req) * p.max_pages;
      const int stop = static_cast<int>(min(static_cast<int64_t>(nb), b + left));
      left -= stop - b;
      int flags = kFirst;
      for (; ok && b < stop; ++b) {
        const bool last = b + 1 == stop;
        int pos = -1;                                    // this slot's position, -1: masked
        if (idx_row) {
          // Every warp looks at all 128 slots: a block with none left is
          // skipped (but for the last, which carries the token's end).
          unsigned any = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int j = b * kBlk + 32 * k + lane;
            const int i = j < n ? __ldg(idx_row + j) : -1;
            const bool in = i >= 0 && i < len;
            any |= __ballot_sync(0xffffffffu, in);
            if (k == pw && in) pos = i;
          }
          if (any == 0 && !last) continue;
        } else {
          const int j = b * kBlk + my;
          if (j < n) pos = j;
        }
        int row = -1;
        float s = 1.f;
        if (pos >= 0) {
          const int col = pos >> p.page_shift;
          const int pg = col < p.max_pages ? __ldg(tab + col) : -1;
          if (static_cast<unsigned>(pg) < static_cast<unsigned>(p.n_pages)) {
            row = (pg << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
            s = __ldg(p.scales + pg);
          }
        }
        const int st = e % L::kStages;
        if (e >= L::kStages) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarEmpty + 4 * st + pw), ((e / L::kStages) - 1) & 1, ctl));
          if (!ok) break;
        }
        // y = S a + c, l += w r: a masked slot's row is zero, its c -inf.
        float* m = reinterpret_cast<float*>(smem + L::kOffA) + st * 3 * L::kMeta + meta;
        m[0] = row >= 0 ? s * p.scale_log2 : 0.f;
        m[L::kMeta] = row >= 0 ? log2f(s) : -INFINITY;
        m[2 * L::kMeta] = row >= 0 ? 1.f / s : 0.f;
        if (my == 0)
          reinterpret_cast<int*>(smem + L::kOffFlags)[st] =
              flags | (last ? kLast : 0) | (last && left == 0 ? kFinal : 0);
        flags = 0;
        const uint32_t tile = base + static_cast<uint32_t>(st) * L::kStageBytes;
        constexpr int kLpr = D / 16;                     // lanes per row
        constexpr int kRpi = 32 / kLpr;                  // rows per warp instruction
        const int sub = lane / kLpr, cc = lane % kLpr;
        const uint32_t col = static_cast<uint32_t>(cc / 8) * L::kChunkBytes;
#pragma unroll 8
        for (int k = 0; k < 32 / kRpi; ++k) {
          const int rw = k * kRpi + sub;
          const int rr = __shfl_sync(0xffffffffu, row, rw);
          const uint32_t at = static_cast<uint32_t>(32 * pw + rw);
          cp_async_16_or_zero(tile + col + at * 128u + ((static_cast<uint32_t>(cc % 8) ^ (at & 7u)) << 4),
                              p.cache + static_cast<int64_t>(max(rr, 0)) * D + cc * 16, rr >= 0);
        }
        cp_async_arrive_noinc(bar(L::kBarFull + st));    // once the copies have landed
        mbar_arrive(bar(L::kBarFull + st));              // releases the factors
        ++e;
      }
    }
    cp_async_wait_all();
  } else if (rg.count > 0 && warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_e4m3_f32(128, kBlk, false);
      constexpr uint32_t idesc_o = idesc_e4m3_f32(128, kHeads, true);
      const uint64_t d_k = smem_desc(base, 16u, 1024u, kSwizzle128B);
      const uint64_t d_v = smem_desc(base, L::kChunkBytes, 1024u, kSwizzle128B);
      const uint64_t d_p = smem_desc(base + L::kOffP, 16u, 1024u, kSwizzle128B);
      const volatile int* flags_of = reinterpret_cast<const volatile int*>(smem + L::kOffFlags);
      auto issue_s = [&](int st) {
        const uint64_t k = d_k + ((static_cast<uint32_t>(st) * L::kStageBytes) >> 4);
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
          mma8_ts(tmem + L::kTmemS, tmem + L::kTmemQ + c * 8,
                  k + (((c / 4) * L::kChunkBytes + (c % 4) * 32u) >> 4), idesc_s, c != 0 ? 1u : 0u);
        mma_commit(bar(L::kBarSFull));
      };
      auto issue_o = [&](int st, bool first) {
        const uint64_t v = d_v + ((static_cast<uint32_t>(st) * L::kStageBytes) >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
          for (int c = 0; c < L::kChunks; ++c)
#pragma unroll
            for (int piece = 0; piece < 2; ++piece)
              mma8_ss(tmem + L::kTmemO + c * kHeads, v + ((c * L::kChunkBytes + k * 4096u) >> 4),
                      d_p + ((piece * L::kPieceBytes + k * 32u) >> 4), idesc_o,
                      (!first || k > 0 || piece > 0) ? 1u : 0u);
          mma_commit(bar(L::kBarEmpty + 4 * st + k));
        }
        mma_commit(bar(L::kBarPDone));
      };
      bool ok = *abort_flag == 0;
      int seg = 0, before = 0;                           // tokens so far, the previous entry's flags
      // O of entry e, once its P is written.
      auto do_o = [&](int e, int flags) {
        ok = mbar_wait(bar(L::kBarPFull), e & 1, ctl);
        if (!ok) return;
        tc_fence_after();
        issue_o(e % L::kStages, (flags & kFirst) != 0);
      };
      for (int e = 0; ok; ++e) {
        const int st = e % L::kStages;
        ok = mbar_wait(bar(L::kBarFull + st), (e / L::kStages) & 1, ctl);
        if (!ok) break;
        const int flags = flags_of[st];
        const bool first = (flags & kFirst) != 0;
        // A token's first S needs its Q, which the softmax warps bring once
        // the token before is finished: that one's last O goes first.
        if (first) {
          if (e > 0) do_o(e - 1, before);
          if (ok) ok = mbar_wait(bar(L::kBarQFull), seg & 1, ctl);
          ++seg;
        }
        if (ok && e > 0) ok = mbar_wait(bar(L::kBarSFree), (e - 1) & 1, ctl);
        if (!ok) break;
        fence_proxy_async_smem();                        // rows written by cp.async -> tensor core
        tc_fence_after();
        issue_s(st);
        if (e == 0 && static_cast<int>(blockIdx.x) == p.stall_cta) {  // test hook only
          ok = stall_until_limit(ctl);
          break;
        }
        if (!first) do_o(e - 1, before);
        before = flags;
        if (flags & kFinal) {
          if (ok) do_o(e, flags);
          break;
        }
      }
      mma_commit(bar(L::kBarDrain));
      mbar_wait_drain(bar(L::kBarDrain), 0);
    }
    __syncwarp();
  } else if (rg.count > 0) {
    // ------------------------------------------------------------ softmax
    // A failed wait sets `bad`; the four warps leave together at the next
    // vote, so that none waits at a barrier that another has left.
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const int hl = 16 * warp + (lane >> 1);              // this lane's head within the CTA
    const bool odd = lane & 1;
    float* head_f = reinterpret_cast<float*>(smem + L::kOffHead);
    const volatile int* flags_of = reinterpret_cast<const volatile int*>(smem + L::kOffFlags);
    bool bad = *abort_flag != 0;
    int64_t left = rg.count;
    int e = 0;
    bool run = true;
    for (int t = rg.tok, b = rg.off; run && left > 0; ++t, b = 0) {
      const int nb = blocks_of(p, t);
      if (nb == 0) continue;
      const int stop = static_cast<int>(min(static_cast<int64_t>(nb), b + left));
      const bool whole = b == 0 && stop == nb;
      const int slot = b == 0 ? 1 : 0;                   // of the CTA's two workspace parts
      left -= stop - b;

      // Q: half-warps take heads in turn, 4 elements per lane of each
      // 64-column piece; then both pieces of every row through shared memory
      // into the row's TMEM lane (row 2h: hi, row 2h + 1: lo).
      float rs;                                          // 2^-k of this lane's head
      {
        constexpr int kC = D / 64;
        uint2 v[8][kC];
        const int half = lane >> 4, l16 = lane & 15;
        const __nv_bfloat16* q0 = p.q + (static_cast<int64_t>(t) * p.H + h0) * D + l16 * 4;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int h = 16 * warp + 2 * i + half;
#pragma unroll
          for (int c = 0; c < kC; ++c)
            v[i][c] = h < heads ? __ldg(reinterpret_cast<const uint2*>(q0 + static_cast<int64_t>(h) * D + c * 64))
                                : make_uint2(0, 0);
        }
        uint32_t top[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t m = 0;
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            m = max(m, max(v[i][c].x & 0x7fffu, (v[i][c].x >> 16) & 0x7fffu));
            m = max(m, max(v[i][c].y & 0x7fffu, (v[i][c].y >> 16) & 0x7fffu));
          }
#pragma unroll
          for (int off = 8; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
          top[i] = m;
        }
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t x = __shfl_sync(0xffffffffu, top[i], ((lane >> 1) & 1) * 16);
          if ((lane >> 2) == i) mine = x;
        }
        // floor(log2) of the largest magnitude (bf16 bits), not below -100.
        auto exponent = [](uint32_t m) { return max(static_cast<int>(m >> 7) - 127, -100); };
        rs = mine >= 0x7f80u ? __uint_as_float(0x7fffffffu) : pow2f(exponent(mine) - 7);
        const uint32_t stage = base + L::kOffQ + static_cast<uint32_t>(warp) * L::kQStage;
        // The previous token's last S is done (its block was read above), so
        // Q's columns are free.
#pragma unroll
        for (int c = 0; c < kC; ++c) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float f = pow2f(7 - exponent(min(top[i], 0x7f7fu)));
            const float x0 = __uint_as_float(v[i][c].x << 16) * f, x1 = __uint_as_float(v[i][c].x & 0xffff0000u) * f;
            const float x2 = __uint_as_float(v[i][c].y << 16) * f, x3 = __uint_as_float(v[i][c].y & 0xffff0000u) * f;
            const uint16_t a = e4m3x2(x0, x1), d = e4m3x2(x2, x3);
            const float2 ra = e4m3x2_value(a), rd = e4m3x2_value(d);
            const uint32_t hi = a | (static_cast<uint32_t>(d) << 16);
            const uint32_t lo = e4m3x2((x0 - ra.x) * 32.f, (x1 - ra.y) * 32.f) |
                                (static_cast<uint32_t>(e4m3x2((x2 - rd.x) * 32.f, (x3 - rd.y) * 32.f)) << 16);
            const uint32_t r = static_cast<uint32_t>(2 * (2 * i + half));  // rows r, r + 1
            const uint32_t at = stage + r * 64u + ((static_cast<uint32_t>(l16 >> 2) ^ ((r >> 1) & 3u)) << 4) + (l16 & 3) * 4;
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(hi) : "memory");
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 64u), "r"(lo) : "memory");
          }
          __syncwarp();
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 x = *reinterpret_cast<const uint4*>(
                smem + L::kOffQ + warp * L::kQStage + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4));
            w[4 * k] = x.x;
            w[4 * k + 1] = x.y;
            w[4 * k + 2] = x.z;
            w[4 * k + 3] = x.w;
          }
          tmem_st16u(tmem + lanes + L::kTmemQ + c * 16, w);
          __syncwarp();
        }
        tc_fence_before();
        mbar_arrive(bar(L::kBarQFull));
      }

      const float f_own = odd ? rs * 0.03125f : rs, f_peer = odd ? rs : rs * 0.03125f;
      float m = -INFINITY, l = 0.f;
      for (bool last = false; run && !last; ++e) {
        const int st = e % L::kStages;
        if (!mbar_wait(bar(L::kBarSFull), e & 1, ctl)) bad = true;
        // (Completed before S was formed; orders the reads of the factors.)
        if (!mbar_wait(bar(L::kBarFull + st), (e / L::kStages) & 1, ctl)) bad = true;
        __syncwarp();
        tc_fence_after();
        const int flags = flags_of[st];
        last = (flags & kLast) != 0;
        const float* a = reinterpret_cast<const float*>(smem + L::kOffA) + st * 3 * L::kMeta + (odd ? 68 : 0);
        float y[64];
        float mx = -INFINITY;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float x0[32], x1[32];
          const uint32_t s0 = tmem + lanes + L::kTmemS + g * 32;
          tmem_ld32x2(s0, s0 + 64, x0, x1);
          if (g == 1) {
            tc_fence_before();
            mbar_arrive(bar(L::kBarSFree));
          }
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 aj = *reinterpret_cast<const float4*>(a + g * 32 + i);
            const float4 cj = *reinterpret_cast<const float4*>(a + L::kMeta + g * 32 + i);
            const float as[4] = {aj.x, aj.y, aj.z, aj.w}, cs[4] = {cj.x, cj.y, cj.z, cj.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float own = odd ? x1[i + k] : x0[i + k], send = odd ? x0[i + k] : x1[i + k];
              const float peer = __shfl_xor_sync(0xffffffffu, send, 1);
              y[g * 32 + i + k] = fmaf(fmaf(own, f_own, peer * f_peer), as[k], cs[k]);
              mx = fmaxf(mx, y[g * 32 + i + k]);
            }
          }
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        const bool first = (flags & kFirst) != 0;
        const bool grow = !first && mx > m + kLag;
        const bool any = bar_any(1, kSoftmaxThreads, grow || bad);
        if (any && bar_any(1, kSoftmaxThreads, bad)) {
          run = false;
          break;
        }
        // P and O are this thread's once the previous block's products are done.
        if (e > 0 && !mbar_wait(bar(L::kBarPDone), (e - 1) & 1, ctl)) bad = true;
        __syncwarp();
        if (any) {                                       // some head's O has to be rescaled
          tc_fence_after();
          const float f = grow ? fast_exp2(m - mx) : 1.f;
          if (grow) {
            m = mx;
            l *= f;
          }
          if (!odd) head_f[hl] = f;
          bar_sync(1, kSoftmaxThreads);
#pragma unroll 1
          for (int c = 0; c < 2 * L::kChunks; ++c) {
            float o[32];
            const uint32_t at = tmem + lanes + L::kTmemO + c * 32;
            tmem_ld32(at, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= head_f[(c & 1) * 32 + i];
            tmem_st32(at, o);
          }
          bar_sync(1, kSoftmaxThreads);                  // head_f is read
        }
        if (first) m = mx;
        const float shift = (m == -INFINITY ? 0.f : m) - kShift;
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {                 // 16 slots: 16 bytes of each piece
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 rj = *reinterpret_cast<const float4*>(a + 2 * L::kMeta + q4 * 16 + i * 4);
            const float* yy = y + q4 * 16 + i * 4;
            const float w0 = fast_exp2(yy[0] - shift), w1 = fast_exp2(yy[1] - shift);
            const float w2 = fast_exp2(yy[2] - shift), w3 = fast_exp2(yy[3] - shift);
            l = fmaf(w0, rj.x, l);
            l = fmaf(w1, rj.y, l);
            l = fmaf(w2, rj.z, l);
            l = fmaf(w3, rj.w, l);
            const __half2 u = __floats2half2_rn(w0, w1), v = __floats2half2_rn(w2, w3);
            const uint16_t uh = e4m3x2(u), vh = e4m3x2(v);
            hi[i] = uh | (static_cast<uint32_t>(vh) << 16);
            lo[i] = e4m3x2(__hsub2(u, e4m3x2_half2(uh))) |
                    (static_cast<uint32_t>(e4m3x2(__hsub2(v, e4m3x2_half2(vh)))) << 16);
          }
          const uint32_t piece = static_cast<uint32_t>((odd ? 4 : 0) + q4) ^ static_cast<uint32_t>(hl & 7);
          const uint32_t at = base + L::kOffP + static_cast<uint32_t>(hl) * 128u + (piece << 4);
          st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
          st_shared_v4(at + L::kPieceBytes, lo[0], lo[1], lo[2], lo[3]);
        }
        tc_fence_before();
        fence_proxy_async_smem();
        mbar_arrive(bar(L::kBarPFull));
      }
      if (!run) break;

      // The token's (or its part's) result, once its last products are done.
      if (!mbar_wait(bar(L::kBarPDone), (e - 1) & 1, ctl)) bad = true;
      __syncwarp();
      tc_fence_after();
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      float* ws = reinterpret_cast<float*>(p.ws + kLeftoverBytes) +
                  (static_cast<int64_t>(blockIdx.x) * 2 + slot) * part_floats(D);
      if (whole) {
        const float sink = hl < heads ? __ldg(p.sink + h0 + hl) * 1.4426950408889634f : 0.f;
        const float top = fmaxf(m, sink);
        float inv, lse;
        if (top == -INFINITY) {                          // nothing at all (or only NaN)
          inv = l * 0.f;
          lse = l != l ? l : -INFINITY;
        } else {
          const float f = 0.015625f * exp2f(m - top);    // 2^-6: the weights' shift
          const float total = l * f + exp2f(sink - top);
          inv = f / total;
          lse = log2f(total) + top;
        }
        if (!odd) {
          head_f[hl] = inv;
          if (hl < heads) p.lse[static_cast<int64_t>(t) * p.H + h0 + hl] = lse;
        }
      } else if (!odd) {
        ws[kHeads * D + hl] = m;
        ws[kHeads * D + kHeads + hl] = l;
      }
      bar_sync(1, kSoftmaxThreads);
#pragma unroll 1
      for (int c = 0; c < 2 * L::kChunks; ++c) {         // 128 of D, 32 heads at a time
        float o[32];
        tmem_ld32(tmem + lanes + L::kTmemO + c * 32, o);
        const int d = (c >> 1) * 128 + tid;
        const int hb = (c & 1) * 32;
        if (D < 128 && warp >= D / 32) continue;         // rows that the tile does not have
        if (whole) {
          // Lane pairs trade, so that each stores two columns of one head.
          __nv_bfloat16* dst = p.o + (static_cast<int64_t>(t) * p.H + h0) * D + (d & ~1);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float u = o[i] * head_f[hb + i], v = o[i + 1] * head_f[hb + i + 1];
            const float got = __shfl_xor_sync(0xffffffffu, odd ? u : v, 1);
            const int h = hb + i + (odd ? 1 : 0);
            if (h < heads)
              *reinterpret_cast<uint32_t*>(dst + static_cast<int64_t>(h) * D) =
                  odd ? pack_bf16x2(got, v) : pack_bf16x2(u, got);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) ws[static_cast<int64_t>(hb + i) * D + d] = o[i];
        }
      }
      tc_fence_before();
      bar_sync(1, kSoftmaxThreads);                      // head_f and O are read
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// Joins the parts of a token that several CTAs hold.  One block per (CTA whose
// range a token starts in and leaves, 4 heads): part i of n weighs
// 2^(m_i - top).
constexpr int kJoinHeads = 4, kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) smqa_paged_join_kernel(const PagedFwdParams p, int ctas) {
  grid_dependency_wait();
  const int groups = (p.H + kHeads - 1) / kHeads;
  const int cta = blockIdx.x / (kHeads / kJoinHeads);
  const int hb = (blockIdx.x % (kHeads / kJoinHeads)) * kJoinHeads;
  const int h0 = (cta % groups) * kHeads;
  const Leftover* left = reinterpret_cast<const Leftover*>(p.ws);
  const int tok = left[cta].tail_tok;
  if (tok < 0 || h0 + hb >= p.H) return;
  // The CTAs behind it that hold the rest: up to the first whose range the
  // token does not leave.
  const int lane = threadIdx.x & 31;
  int lastc = cta;
  for (int c0 = cta + groups; c0 < ctas; c0 += 32 * groups) {
    const int c = c0 + lane * groups;
    const bool end = c < ctas && left[c].head_tok == tok && !left[c].head_more;
    const unsigned b = __ballot_sync(0xffffffffu, end);
    if (b) {
      lastc = c0 + (__ffs(b) - 1) * groups;
      break;
    }
  }
  constexpr int kPer = kJoinHeads * D / kJoinThreads;    // consecutive columns per thread
  const int hl = hb + static_cast<int>(threadIdx.x) / (kJoinThreads / kJoinHeads);
  const int d = (static_cast<int>(threadIdx.x) % (kJoinThreads / kJoinHeads)) * kPer;
  const float* parts = reinterpret_cast<const float*>(p.ws + kLeftoverBytes);
  auto part = [&](int c) { return parts + (static_cast<int64_t>(c) * 2 + (c == cta ? 1 : 0)) * part_floats(D); };
  if (h0 + hl >= p.H) return;
  const float sink = __ldg(p.sink + h0 + hl) * 1.4426950408889634f;
  float top = sink;
  for (int c = cta; c <= lastc; c += groups)
    if (c == cta || left[c].head_tok == tok) top = fmaxf(top, part(c)[kHeads * D + hl]);
  float total = top == -INFINITY ? 0.f : 64.f * exp2f(sink - top);
  float o[kPer] = {};
  for (int c = cta; c <= lastc; c += groups) {
    if (c != cta && left[c].head_tok != tok) continue;   // an empty range
    const float* w = part(c);
    const float f = top == -INFINITY ? 0.f : exp2f(w[kHeads * D + hl] - top);
    total = fmaf(w[kHeads * D + kHeads + hl], f, total);
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = fmaf(w[static_cast<int64_t>(hl) * D + d + i], f, o[i]);
  }
  const int64_t row = static_cast<int64_t>(tok) * p.H + h0 + hl;
  const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
  for (int i = 0; i < kPer; ++i) p.o[row * D + d + i] = __float2bfloat16(o[i] * inv);
  if (d == 0) p.lse[row] = total == 0.f ? -INFINITY : log2f(total) - kShift + top;
}

// CTAs of a call: per head group, as many ranges as SMs (or as the tokens can
// have blocks).
int ranges_of(const smqa_paged_shape& s) {
  const int groups = (s.H + kHeads - 1) / kHeads;
  const int64_t slots = s.topk > 0 ? s.topk : static_cast<int64_t>(s.max_pages) * s.page_size;
  const int64_t blocks = static_cast<int64_t>(s.T) * ((slots + kBlk - 1) / kBlk);
  return static_cast<int>(std::min<int64_t>(152 / groups, std::max<int64_t>(blocks, 1)));
}

template <int D>
cudaError_t launch(const PagedFwdParams& p, int ctas, cudaStream_t stream) {
  using L = PagedLayout<D>;
  cudaError_t e = cudaFuncSetAttribute(smqa_paged_fwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  smqa_paged_fwd_kernel<D><<<ctas, kThreads, L::kSmem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas) * (kHeads / kJoinHeads));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, smqa_paged_join_kernel<D>, p, ctas);
}

}  // namespace

size_t paged_fwd_workspace(const smqa_paged_shape& s) {
  const int groups = (s.H + kHeads - 1) / kHeads;
  static_assert(152 <= kMaxCtas, "a leftover per CTA");
  return kLeftoverBytes + static_cast<size_t>(ranges_of(s)) * groups * 2 * part_floats(s.D) * sizeof(float);
}

cudaError_t launch_paged_fwd(const PagedFwdParams& p, const smqa_paged_shape& s, cudaStream_t stream) {
  const int ctas = ranges_of(s) * ((s.H + kHeads - 1) / kHeads);
  return p.D == 512 ? launch<512>(p, ctas, stream) : launch<64>(p, ctas, stream);
}

}  // namespace smqa

// smqa_topk_score.cu -- scores of the indexer's selection on sm_103a.
//
// For token t and the key rows j it sees,
//   score[t, j] = sum_h w[t, h] ReLU(q[t, h] . k_j),
// rows of up to 32 positions (a block) by their largest, as ordered integers in
// the workspace; smqa_topk.cu chooses from them.
//
// A tile is 128 key rows (A, M = 128) against the heads of a group of up to
// 256 / Hp tokens (B, N = Hp per token; Hp: H rounded up to 16, 32, 64 or 128,
// with zero rows behind H), K = D: a thread of the epilogue has one key row in its TMEM lane, the
// heads in columns, so the sum over heads needs no exchange between threads and
// a warp writes 32 consecutive scores.  bf16 keys: kind::f16.  e4m3 keys (the
// paged cache): kind::f8f6f4, the codes as they lie in the cache, the queries as
// two e4m3 pieces added into one accumulator.
//
// The groups' tiles form one sequence, cut into equal ranges, one per CTA: a
// lone token's context and the triangle of a causal prompt are spread over the
// GPU alike.  A group's tiles share its queries, which stay in shared memory (two
// buffers); key tiles come by TMA through a ring of 128-byte pieces.  Tokens that
// see no more rows than they choose need no scores and are left out.
//
// Warps: the epilogue's; one that issues the key tiles' copies; one that feeds the tensor
// core; two that walk through the groups, a group ahead of the tensor core, and bring its
// queries and weights; and with paged keys four that bound the key rows' lengths as the
// tiles pass (which the choice's error bound needs; contiguous rows are bounded once, by
// the two).  Described and fetched only behind a group's own copies, as it was, queries
// came late: a part of 16 tiles waited 12000 clocks for them.
//
// What bounds it is the epilogue, more than the tensor core (1024 clocks a tile of 256
// columns; without half of the products 1000 queries over 32768 positions took 310 us of
// 322, 2 x 4096 tokens 184 of 211): a thread's chain of barrier, loads, sums and stores.  With contiguous keys and up to 64 heads four warpgroups
// share a tile's columns, 64 each, and hide each other's latencies (1000 queries over 32768
// positions of 64 heads: 404 us with two of 128 columns, 325 with four; S = 8192 in four
// chunks 401 and 323).  More than 64 heads need a thread that sums 128 columns; paged keys,
// the two warpgroups' registers for the four warps that bound the rows.  Narrower tiles go
// to the warpgroups in turn.  A thread keeps the weights of its columns in registers for a
// whole group: read from shared memory for every tile, 4 bytes a lane, they took as long as
// the tensor core from the bandwidth that it needs for its operands.  The accumulator is
// given back before the sums are made into keys and written.  Half of the ReLUs are x + |x|
// with the weight halved: an addition, where a maximum takes twice as long and waits for
// the unit of the integer operations.
#include <cuda_runtime.h>

#include <type_traits>

#include "smqa_topk.cuh"

namespace smqa {

namespace {

constexpr int kCols = 256;                               // accumulator columns

// The warps' roles.
template <bool kPaged, int Hp>
struct Roles {
  static constexpr int kGroups = kPaged || Hp == 128 ? 2 : 4;  // epilogue warpgroups
  static constexpr int kMine = kCols / kGroups;          // columns of one of them
  static constexpr int kEpilogueWarps = 4 * kGroups;
  static constexpr int kLoadWarp = kEpilogueWarps, kMmaWarp = kLoadWarp + 1;
  static constexpr int kHelpWarp0 = kLoadWarp + 2, kHelpers = 2;
  static constexpr int kBoundWarp0 = kLoadWarp + 4, kBounders = kPaged ? 4 : 0;
  static constexpr int kThreads = 32 * (kBoundWarp0 + kBounders);
  // Registers of the epilogue's warpgroups and of the others: their sum is what the block
  // is launched with.
  static constexpr int kEpilogueRegs = kGroups == 2 ? 192 : 104, kOtherRegs = 64;
  static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
  static_assert(kThreads % 128 == 0 && (kThreads / 128 - kGroups) * kOtherRegs + kGroups * kEpilogueRegs <= kThreads / 128 * kLaunchRegs,
                "registers of the launch, roles by warpgroup");
};
constexpr int kMaxWarps = 20;
constexpr int kMaxGroup = 16;                            // tokens of a group

// What the CTA does for one group (or the part of one that its range holds).
struct Work {
  int64_t tok;                                           // its first token
  int ntok, tile0, ntiles, req;                          // (ntiles = 0: no more work)
  int n[kMaxGroup];                                      // rows that each token sees (0: needs no scores)
};

template <int D, bool kPaged>
struct ScoreLayout {
  static constexpr int kRowBytes = kPaged ? D : 2 * D;
  static constexpr int kPieces = kRowBytes > 128 ? kRowBytes / 128 : 1;  // of a key row
  static constexpr int kPitch = kRowBytes > 128 ? 128 : kRowBytes;       // bytes of a row in a piece
  static constexpr uint32_t kPieceBytes = kTile * kPitch;
  static constexpr int kQParts = kPaged ? 2 : kPieces;   // (hi and lo, or 64 columns each)
  static constexpr uint32_t kQPartBytes = kCols * kPitch;
  static constexpr uint32_t kQBytes = kQParts * kQPartBytes;
  static constexpr int kStages = kQBytes == 65536 ? 5 : 8;
  static constexpr int kShared = kStages & 1 ? kStages - 1 : -1;  // paged: the stage of all warps that bound the rows
  static constexpr uint32_t kSwizzle = kPitch == 128 ? kSwizzle128B : kSwizzle64B;
  static constexpr uint32_t kAtom = 8 * kPitch;          // 8 rows
  static constexpr int kMeta = 16;                       // tiles whose page scales are kept
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffK = 2 * kQBytes;
  static constexpr uint32_t kOffW = kOffK + kStages * kPieceBytes;      // float [2][256]
  static constexpr uint32_t kOffMeta = kOffW + 2 * kCols * 4;           // float [kMeta][8]
  static constexpr uint32_t kOffWork = kOffMeta + kMeta * 8 * 4;        // Work [2]
  static constexpr uint32_t kOffSum = kOffWork + 2 * sizeof(Work);      // int64 [kMaxWarps], then the range's start
  static constexpr uint32_t kOffBar = kOffSum + kMaxWarps * 8 + 32;
  static constexpr int kBarKFull = 0;
  static constexpr int kBarKEmpty = kBarKFull + kStages;
  static constexpr int kBarAccFull = kBarKEmpty + kStages;  // [2]
  static constexpr int kBarAccEmpty = kBarAccFull + 2;      // [2]
  static constexpr int kBarWork = kBarAccEmpty + 2;         // [2] work described
  static constexpr int kBarQFull = kBarWork + 2;            // [2] queries and weights there
  static constexpr int kBarQEmpty = kBarQFull + 2;          // [2]
  static constexpr int kBarQFirst = kBarQEmpty + 2;         // paged: those of the first part
  static constexpr int kBarDrain = kBarQFirst + 1;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr uint32_t kOffCtl = kOffBar + 8 * kNumBars;  // TMEM base, abort flag
  static constexpr uint32_t kSmem = kOffCtl + 16 + 1024;
  static_assert(kOffBar % 8 == 0 && kOffWork % 8 == 0 && kOffSum % 8 == 0 && kOffK % 1024 == 0, "alignment");
  static_assert(kSmem <= 232448, "shared memory budget");
  // Tiles between the copies of one and the epilogue of another: the ring, and the two
  // accumulators.
  static_assert(kMeta >= kStages + 4, "page scales are read before they are replaced");
};

// One lane of a converged warp issues; bf16 operands.
__device__ __forceinline__ void mma16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// 16 consecutive columns of the warp's lanes at t, and (kBoth) 16 at t + 64; one wait.
template <bool kBoth>
__device__ __forceinline__ void tmem_ld16_and_64(uint32_t t, float (&v)[32]) {
  uint32_t r[32] = {};
  if constexpr (kBoth)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(t), "r"(t + 64)
        : "memory");
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t)
        : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ float relu(float x) {         // (a NaN stays one)
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float twice_relu(float x) { return x + fabsf(x); }  // (of -infinity: NaN)

// A token's sum of a key row that holds infinities: real ReLUs (not x + |x|), and of real heads
// only (those behind H are zeros, and 0 times an infinity is no number); four chains, as the
// epilogue's.  (A function of its own: inlined among the epilogue's instructions, S = 8192 took
// 679 us and not 663.)
__device__ __noinline__ float sum_of_real_heads(uint32_t t, uint32_t w, int H) {
  float a[4] = {};
#pragma unroll 1
  for (int h = 0; h < H; h += 16) {
    float x[32];
    tmem_ld16_and_64<false>(t + h, x);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float wi;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(wi) : "r"(w + (h + i) * 4));
      if (h + i < H) a[i & 3] = fmaf(wi, relu(x[i]), a[i & 3]);
    }
  }
  return (a[0] + a[1]) + (a[2] + a[3]);
}

__device__ __forceinline__ int tiles_for(const TopkParams& p, int n) { return n > p.topk ? (n + kTile - 1) / kTile : 0; }

// The tokens of unit u (a group of consecutive tokens; contiguous: of one batch
// element), as [first, first + count).
template <bool kPaged>
__device__ __forceinline__ int unit_tokens(const TopkParams& p, int64_t u, int group, int64_t& first) {
  if constexpr (kPaged) {
    first = u * group;
    return static_cast<int>(min(static_cast<int64_t>(group), p.T - first));
  } else {
    const int per = (p.S + group - 1) / group;
    const int64_t b = u / per;
    const int s = static_cast<int>(u - b * per) * group;
    first = b * p.S + s;
    return min(group, p.S - s);
  }
}

// Tiles of the part of a unit that starts at token i, and its end (tokens of one
// request).
template <bool kPaged>
__device__ __forceinline__ int part_tiles(const TopkParams& p, int64_t first, int count, int i, int& end, int& req) {
  if constexpr (kPaged) {
    int tiles = tiles_for(p, visible<true>(p, first + i, req));
    for (end = i + 1; end < count; ++end) {
      int r;
      const int n = visible<true>(p, first + end, r);
      if (r != req) break;
      tiles = max(tiles, tiles_for(p, n));
    }
    return req < 0 ? 0 : tiles;
  } else {
    end = count;                                         // (the last token sees most)
    return tiles_for(p, visible<false>(p, first + count - 1, req));
  }
}
template <bool kPaged>
__device__ __forceinline__ int64_t unit_tiles(const TopkParams& p, int64_t u, int group) {
  int64_t first, tiles = 0;
  const int count = unit_tokens<kPaged>(p, u, group, first);
  for (int i = 0, end, req; i < count; i = end) tiles += part_tiles<kPaged>(p, first, count, i, end, req);
  return tiles;
}

template <int D, bool kPaged, int Hp>
__global__ void __launch_bounds__(Roles<kPaged, Hp>::kThreads, 1)
    smqa_topk_score_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q, const TopkParams p) {
  using L = ScoreLayout<D, kPaged>;
  using Ro = Roles<kPaged, Hp>;
  constexpr int kThreads = Ro::kThreads, kMine = Ro::kMine;
  static_assert(kThreads <= 32 * kMaxWarps, "room for the warps' sums");
  constexpr int kGroup = kCols / Hp;
  extern __shared__ uint8_t smem_raw[];
  uint32_t base = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (base & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  base += pad;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  auto bar = [&](int i) -> uint32_t { return base + L::kOffBar + 8u * static_cast<uint32_t>(i); };
  volatile uint32_t* tmem_holder = reinterpret_cast<volatile uint32_t*>(smem + L::kOffCtl);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffCtl + 4);
  const WaitCtl ctl{abort_flag, p.status, p.limit_ns};
  int64_t* warp_sum = reinterpret_cast<int64_t*>(smem + L::kOffSum);
  int64_t* start = warp_sum + kMaxWarps;                        // unit, tiles of it before the range, tiles of the range
  Work* works = reinterpret_cast<Work*>(smem + L::kOffWork);

  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(bar(L::kBarKFull + i), 1);
      // Tensor core (and the two or four warps that bound the rows' lengths).
      mbar_init(bar(L::kBarKEmpty + i), !kPaged ? 1 : i == L::kShared ? 5 : 3);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(L::kBarAccFull + i), 1);
      mbar_init(bar(L::kBarAccEmpty + i), Ro::kEpilogueWarps);
      mbar_init(bar(L::kBarWork + i), 1);
      mbar_init(bar(L::kBarQFull + i), Ro::kHelpers + (kPaged ? 0 : 1));  // (1: the copy)
      mbar_init(bar(L::kBarQEmpty + i), 1 + Ro::kEpilogueWarps + Ro::kBounders);  // (1: tensor core)
    }
    mbar_init(bar(L::kBarQFirst), Ro::kHelpers + Ro::kBounders);
    mbar_init(bar(L::kBarDrain), 1);
    start[2] = 0;
    fence_mbar_init();
  }
  if (warp == Ro::kMmaWarp) tmem_alloc(base + L::kOffCtl, 2 * kCols);
  // (So far beside the kernel before, whose results are read from here on.)
  grid_dependency_wait();
  grid_dependents_launch();
  if (tid == 0) *abort_flag = *reinterpret_cast<volatile int*>(p.status) != 0 ? 1 : 0;
  // The CTA's range of tiles, and the unit it starts in (each thread sums a run of
  // units).
  {
    const int64_t per = (p.units + kThreads - 1) / kThreads;
    const int64_t u0 = min(tid * per, p.units), u1 = min(u0 + per, p.units);
    int64_t mine = 0;
    for (int64_t u = u0; u < u1; ++u) mine += unit_tiles<kPaged>(p, p.unit0 + u, kGroup);
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
    // Equal ranges, the first total mod grid of them one tile longer.
    const int64_t parts = gridDim.x, part = blockIdx.x;
    const int64_t each = (total >> 32) != 0 ? total / parts : static_cast<uint32_t>(total) / static_cast<uint32_t>(parts);
    const int64_t extra = total - each * parts;
    const int64_t begin = each * part + min(part, extra), end = begin + each + (part < extra ? 1 : 0);
    if (begin < end && before <= begin && begin < before + mine) {
      int64_t at = before, u = u0, n;
      while (at + (n = unit_tiles<kPaged>(p, p.unit0 + u, kGroup)) <= begin) {
        at += n;
        ++u;
      }
      start[0] = p.unit0 + u;
      start[1] = begin - at;
      start[2] = end - begin;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int64_t count_all = start[2];
  // The barrier that a part's queries and weights arrive on, and its phase.
  auto q_bar = [&](int seg) { return kPaged && seg == 0 ? L::kBarQFirst : L::kBarQFull + (seg & 1); };
  auto q_phase = [&](int seg) { return !kPaged ? seg >> 1 : seg == 0 ? 0 : (seg - 1) >> 1; };
  // Paged: two e4m3 pieces of each query row times 2^k, which its weight takes back, by
  // warp `me` of n; four lanes share a row.  (A row with a NaN or an infinity becomes NaN.)
  // The next rows are asked for before these are written.
  auto bring = [&](int me, int n, int qb, int64_t tok, int ntok) {
    float* ws = reinterpret_cast<float*>(smem + L::kOffW) + qb * kCols;
    const uint32_t to = base + L::kOffQ + static_cast<uint32_t>(qb) * L::kQBytes;
    constexpr int kSeg = D / 4;                          // elements per lane
    const int part = lane & 3;
    uint4 v[kSeg / 8], next[kSeg / 8];
    float w = 0.f, next_w = 0.f;
    auto ask = [&](int r0, uint4 (&x)[kSeg / 8], float& xw) {
      const int r = r0 + (lane >> 2), h = r % Hp;
      const bool there = r0 < ntok * Hp && h < p.H;
#pragma unroll
      for (int c = 0; c < kSeg / 8; ++c)
        x[c] = there ? load(reinterpret_cast<const uint4*>(p.q + ((tok + r / Hp) * p.H + h) * D + part * kSeg) + c)
                     : make_uint4(0, 0, 0, 0);
      xw = there ? load(p.w + (tok + r / Hp) * p.H + h) : 0.f;
    };
    ask(me * 8, v, w);
    for (int r0 = me * 8; r0 < ntok * Hp; r0 += 8 * n) {
      ask(r0 + 8 * n, next, next_w);
      const int r = r0 + (lane >> 2);
      uint32_t m = 0;
#pragma unroll
      for (int c = 0; c < kSeg / 8; ++c)
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(v[c].x & 0x7fff7fffu, v[c].y & 0x7fff7fffu),
                                 __vmaxu2(v[c].z & 0x7fff7fffu, v[c].w & 0x7fff7fffu)));
      m = max(m & 0xffffu, m >> 16);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int k = query_exponent(m);
      const float f = m >= 0x7f80u ? __uint_as_float(0x7fffffffu) : pow2f(k);
      if (part == 0) ws[r] = w * pow2f(-k);
#pragma unroll
      for (int c = 0; c < kSeg / 16; ++c) {              // 16 elements: 16 bytes of each piece
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k2 = 0; k2 < 4; ++k2) {
          const uint4& x = v[2 * c + (k2 >> 1)];
          const uint32_t a = (k2 & 1) ? x.z : x.x, b = (k2 & 1) ? x.w : x.y;
          uint16_t h0, l0, h1, l1;
          split_query(make_float2(__uint_as_float(a << 16) * f, __uint_as_float(a & 0xffff0000u) * f), h0, l0);
          split_query(make_float2(__uint_as_float(b << 16) * f, __uint_as_float(b & 0xffff0000u) * f), h1, l1);
          hi[k2] = h0 | (static_cast<uint32_t>(h1) << 16);
          lo[k2] = l0 | (static_cast<uint32_t>(l1) << 16);
        }
        const int piece = part * (kSeg / 16) + c;
        const uint32_t at = to + r * L::kPitch +
                            ((L::kPitch == 128 ? piece ^ (r & 7) : piece ^ ((r >> 1) & 3)) << 4);
        st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
        st_shared_v4(at + L::kQPartBytes, lo[0], lo[1], lo[2], lo[3]);
      }
#pragma unroll
      for (int c = 0; c < kSeg / 8; ++c) v[c] = next[c];
      w = next_w;
    }
    fence_proxy_async_smem();
  };

  if (count_all == 0 && (kPaged || warp < Ro::kLoadWarp)) {
    // nothing to do
  } else if (warp >= Ro::kLoadWarp) {
    reg_dealloc<Ro::kOtherRegs>();
    auto wait = [&](int i, int phase) { return __all_sync(0xffffffffu, mbar_wait_soon(bar(i), phase & 1, ctl)); };
    if (warp == Ro::kLoadWarp && count_all > 0) {
      // ------------------------------------------------------------ copies of key tiles
      bool ok = *abort_flag == 0;
      int e = 0, tile_no = 0;                              // pieces and tiles so far
      for (int seg = 0; ok; ++seg) {
        ok = wait(L::kBarWork + (seg & 1), seg >> 1);
        if (!ok) break;
        const Work& wk = works[seg & 1];
        const int ntiles = wk.ntiles, tile0 = wk.tile0, req = wk.req;
        if (ntiles == 0) break;
        // Paged: lane = page of a tile.  The pages of the tile after next and the scales of the
        // next one are asked for before a tile's copies are issued (one after another, the
        // loads took 1200 cycles a tile).
        auto page_of = [&](int i) {
          const int col = ((tile0 + i) * kTile >> p.page_shift) + lane;
          const bool in = i < ntiles && lane < (kTile >> p.page_shift) && col < p.max_pages;
          return in ? load(p.table + static_cast<int64_t>(req) * p.max_pages + col) : -1;
        };
        auto is_page = [&](int page) { return static_cast<unsigned>(page) < static_cast<unsigned>(p.n_pages); };
        auto scale_of = [&](int page) { return is_page(page) ? load(p.scales + page) : -1.f; };
        int page = -1, next_page = -1;
        float scale = -1.f;
        if constexpr (kPaged) {
          page = page_of(0);
          next_page = page_of(1);
          scale = scale_of(page);
        }
        for (int i = 0; ok && i < ntiles; ++i, ++tile_no) {
          const int j0 = (tile0 + i) * kTile;
          const bool live = !kPaged || is_page(page);
          int later_page = -1;
          float next_scale = -1.f;
          if constexpr (kPaged) {
            later_page = page_of(i + 2);
            next_scale = scale_of(next_page);
          }
          const unsigned pages_there = __ballot_sync(0xffffffffu, live);
  #pragma unroll
          for (int c = 0; c < L::kPieces; ++c, ++e) {
            const int st = e % L::kStages;
            if (e >= L::kStages)
              ok = ok && __all_sync(0xffffffffu, mbar_wait_soon(bar(L::kBarKEmpty + st), ((e / L::kStages) - 1) & 1, ctl));
            if (!ok) break;
            const uint32_t to = base + L::kOffK + static_cast<uint32_t>(st) * L::kPieceBytes;
            if constexpr (kPaged) {
              const uint32_t bytes = static_cast<uint32_t>(D) << p.page_shift;
              // (-1 for a page that is not there: its rows get no copy, what lies in
              // their place is never used.)
              if (lane < 8)
                reinterpret_cast<float*>(smem + L::kOffMeta)[(tile_no % L::kMeta) * 8 + lane] = scale;
              __syncwarp();
              if (lane == 0) mbar_arrive_expect_tx(bar(L::kBarKFull + st), bytes * __popc(pages_there));
              __syncwarp();
              if (live) tma_load_2d(to + lane * bytes, &tm_k, 0, page << p.page_shift, bar(L::kBarKFull + st));
            } else if (lane == 0) {
              mbar_arrive_expect_tx(bar(L::kBarKFull + st), L::kPieceBytes);
              tma_load_2d(to, &tm_k, c * 64, req * p.S_kv + j0, bar(L::kBarKFull + st));
            }
          }
          page = next_page;
          next_page = later_page;
          scale = next_scale;
        }
        if (!ok) break;
      }
      // Copies in flight land before the CTA ends.
      if (lane == 0)
        for (int i = max(0, e - L::kStages); i < e; ++i)
          mbar_wait_drain(bar(L::kBarKFull + i % L::kStages), (i / L::kStages) & 1);
      __syncwarp();
    } else if (warp == Ro::kMmaWarp && count_all > 0) {
      // ------------------------------------------------------------ MMA issuer
      const uint64_t d_k = smem_desc(base + L::kOffK, 16u, L::kAtom, L::kSwizzle);
      const uint64_t d_q = smem_desc(base + L::kOffQ, 16u, L::kAtom, L::kSwizzle);
      bool ok = *abort_flag == 0;
      int e = 0, tile_no = 0;
      for (int seg = 0; ok; ++seg) {
        const int qb = seg & 1;
        ok = wait(L::kBarWork + qb, seg >> 1);
        if (!ok) break;
        const int ntiles = works[qb].ntiles, ntok = works[qb].ntok;
        if (ntiles == 0) break;
        ok = wait(q_bar(seg), q_phase(seg));
        const uint64_t qd = d_q + ((static_cast<uint32_t>(qb) * L::kQBytes) >> 4);
        const uint32_t idesc = kPaged ? idesc_e4m3_f32(128, 16, false) : idesc_bf16_f32(128, 16, false, false);
        const uint32_t id = (idesc & ~(0x3fu << 17)) | (static_cast<uint32_t>(ntok * Hp >> 3) << 17);
        for (int i = 0; ok && i < ntiles; ++i, ++tile_no) {
          const int acc = tile_no & 1;
          if (tile_no >= 2) ok = wait(L::kBarAccEmpty + acc, (tile_no >> 1) - 1);
          const uint32_t d = tmem + static_cast<uint32_t>(acc) * kCols;
  #pragma unroll
          for (int c = 0; c < L::kPieces; ++c, ++e) {
            const int st = e % L::kStages;
            ok = ok && wait(L::kBarKFull + st, e / L::kStages);
            if (!ok) break;
            tc_fence_after();
            const uint64_t kd = d_k + ((static_cast<uint32_t>(st) * L::kPieceBytes) >> 4);
            if constexpr (kPaged) {
  #pragma unroll
              for (int part = 1; part >= 0; --part)        // (the small pieces first: see the error bound)
  #pragma unroll
                for (int k = 0; k < D / 32; ++k)
                  mma8_ss(d, kd + (k * 32u >> 4), qd + ((part * L::kQPartBytes + k * 32u) >> 4), id, part == 0 || k != 0);
            } else {
  #pragma unroll
              for (int k = 0; k < 4; ++k)
                mma16_ss(d, kd + (k * 32u >> 4), qd + ((c * L::kQPartBytes + k * 32u) >> 4), id, (c | k) != 0);
            }
            mma_commit_elect(bar(L::kBarKEmpty + st));
          }
          if (!ok) break;
          mma_commit_elect(bar(L::kBarAccFull + acc));
          if (static_cast<int>(blockIdx.x) == p.stall_cta && tile_no == 0) {  // test hook only
            ok = __any_sync(0xffffffffu, stall_until_limit(ctl));
            break;
          }
        }
        if (ok) mma_commit_elect(bar(L::kBarQEmpty + qb));
      }
      mma_commit_elect(bar(L::kBarDrain));
      mbar_wait_drain(bar(L::kBarDrain), 0);
      __syncwarp();
    } else if (warp >= Ro::kHelpWarp0 && warp < Ro::kBoundWarp0) {
      // ------------------------------------------------------------ walk, queries, weights
      // (A part is described as soon as its buffers are free, a part ahead of the tensor core.)
      const int hw = warp - Ro::kHelpWarp0;
      if constexpr (!kPaged) {
        // Bounds of the key rows' lengths, 32 rows a warp, over all CTAs.
        const int64_t all = p.B * p.norm_ld, step = static_cast<int64_t>(gridDim.x) * Ro::kHelpers;
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * Ro::kHelpers + hw; i < all; i += step) {
          const int64_t b = i / p.norm_ld;
          const int j = static_cast<int>(i - b * p.norm_ld) * 32 + lane;
          float s = 0.f;
          if (j < p.S_kv) {
            const uint4* row = reinterpret_cast<const uint4*>(p.k + (b * p.S_kv + j) * D);
  #pragma unroll 8
            for (int c = 0; c < D / 8; ++c) {
              const uint4 v = load(row + c);
              const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
  #pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float a = __uint_as_float(w4[k] << 16), d = __uint_as_float(w4[k] & 0xffff0000u);
                s = fmaf(a, a, fmaf(d, d, s));
              }
            }
            if (s >= 0x1p-90f && s < INFINITY) {
              s = sqrtf(s) * 1.0001f;
            } else {
              // Squares that leave fp32's range: once more, the row times 2^70 or 2^-70.  (A row of
              // infinities has scores that are infinite, NaN or 0, and needs no bound.)
              const float f = s < 1.f ? 0x1p70f : 0x1p-70f;
              s = 0.f;
  #pragma unroll 1
              for (int c = 0; c < D / 8; ++c) {
                const uint4 v = load(row + c);
                const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
                for (int k = 0; k < 4; ++k) {
                  const float a = __uint_as_float(w4[k] << 16) * f, d = __uint_as_float(w4[k] & 0xffff0000u) * f;
                  s = fmaf(a, a, fmaf(d, d, s));
                }
              }
              s = s < INFINITY ? __fmul_ru(sqrtf(s) * 1.0001f, 1.f / f) : 0.f;
            }
          }
          const float m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(s)));
          if (lane == 0) p.norms[i] = m;
        }
      }
      bool ok = count_all > 0 && *abort_flag == 0;
      int64_t u = start[0], skip = start[1], left = count_all, first = 0;
      int issued = 0;                                      // copies of queries
      int part = 0, count = ok ? unit_tokens<kPaged>(p, u, kGroup, first) : 0;
      for (int seg = 0; ok; ++seg) {
        const int qb = seg & 1;
        if (hw == 0) {
          // The next part with tiles in the range.
          int end = 0, req = 0, tiles = 0;
          if (left > 0) {
            while (true) {
              if (part >= count) {
                count = unit_tokens<kPaged>(p, ++u, kGroup, first);
                part = 0;
              }
              tiles = part_tiles<kPaged>(p, first, count, part, end, req);
              if (skip < tiles) break;
              skip -= tiles;
              part = end;
            }
          }
          int n = 0, r;
          if (left > 0 && lane < end - part) n = visible<kPaged>(p, first + part + lane, r);
          if (seg >= 2) ok = wait(L::kBarQEmpty + qb, (seg >> 1) - 1);
          if (!ok) break;
          Work* wk = works + qb;
          const int64_t ntiles = min(left, static_cast<int64_t>(tiles) - skip);
          if (lane < kMaxGroup) wk->n[lane] = n > p.topk ? n : 0;
          if (lane == 0) {
            wk->tok = first + part;
            wk->ntok = end - part;
            wk->tile0 = static_cast<int>(skip);
            wk->ntiles = left > 0 ? static_cast<int>(ntiles) : 0;
            wk->req = req;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kBarWork + qb));
          if (left <= 0) break;
          left -= ntiles;
          skip = 0;
          part = end;
        }
        ok = wait(L::kBarWork + qb, seg >> 1);
        if (!ok) break;
        const Work& wk = works[qb];
        const int ntok = wk.ntok;
        const int64_t tok = wk.tok;
        if (wk.ntiles == 0) break;
        if constexpr (!kPaged) {
          // One copy of the group's rows for each 64 elements (zeros behind H; a group that is
          // not full brings rows that no column takes), and the weights.
          if (hw == 0 && lane == 0) {
            mbar_arrive_expect_tx(bar(L::kBarQFull + qb), L::kQBytes);
#pragma unroll
            for (int c = 0; c < L::kQParts; ++c)
              tma_load_3d(base + L::kOffQ + static_cast<uint32_t>(qb) * L::kQBytes + c * L::kQPartBytes, &tm_q, c * 64, 0,
                          static_cast<int>(tok), bar(L::kBarQFull + qb));
          }
          __syncwarp();
          issued = seg + 1;
          float w[kCols / 64];
#pragma unroll
          for (int i = 0; i < kCols / 64; ++i) {
            const int col = i * 64 + hw * 32 + lane, h = col % Hp;
            w[i] = col < ntok * Hp && h < p.H ? load(p.w + (tok + col / Hp) * p.H + h) : 0.f;
          }
          float* ws = reinterpret_cast<float*>(smem + L::kOffW) + qb * kCols + hw * 32 + lane;
#pragma unroll
          for (int i = 0; i < kCols / 64; ++i) ws[i * 64] = w[i];
        } else {
          bring(hw, seg == 0 ? Ro::kHelpers + Ro::kBounders : Ro::kHelpers, qb, tok, ntok);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(q_bar(seg)));
      }
      // Copies in flight land before the CTA ends.
      if (hw == 0 && lane == 0)
        for (int i = max(0, issued - 2); i < issued; ++i) mbar_wait_drain(bar(L::kBarQFull + (i & 1)), (i >> 1) & 1);
      __syncwarp();
    } else if (kPaged && warp >= Ro::kBoundWarp0) {
      const int hw = warp - Ro::kBoundWarp0;
      bool ok = *abort_flag == 0;
      int e = 0;
      for (int seg = 0; ok; ++seg) {
        const int qb = seg & 1;
        ok = wait(L::kBarWork + qb, seg >> 1);
        if (!ok) break;
        const Work& wk = works[qb];
        const int ntok = wk.ntok, ntiles = wk.ntiles, tile0 = wk.tile0;
        const int64_t tok = wk.tok;
        if (ntiles == 0) break;
        if (seg == 0) {
          bring(Ro::kHelpers + hw, Ro::kHelpers + Ro::kBounders, 0, tok, ntok);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kBarQFirst));
        }
        // Bounds of the key rows' lengths, from the tiles as they pass: two warps have the ring's
        // even stages, two the odd ones, a thread two rows; the last of an odd number of stages
        // is shared by all four.  (All four at every tile took 1250 cycles a tile, half of it
        // the wait.  128 tokens over 32768 positions: 97 us with three stages to two, 98 with
        // a stage per warp, which held it longer.)  A stage's warps come to it at every round
        // of the ring: with the tiles in turn to the pairs they came at every other one, and
        // a barrier's one parity bit cannot tell a round from the one before the last.
        // |code| 2^-8 is the fp16 number with the code's seven bits at 7-13; squares and
        // sums of 16 of them in fp16 are off by 2^-11 each step, and lose 2^-25 each
        // where they are subnormal.
        for (int i = 0; ok && i < ntiles; ++i, ++e) {
          const int st = e % L::kStages;
          const bool shared = st == L::kShared;
          if (!shared && (st & 1) != (hw >> 1)) continue;
          ok = wait(L::kBarKFull + st, e / L::kStages);
          if (!ok) break;
          float top = 0.f;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (half == 1 && shared) break;
            const int r = (shared ? hw * 32 : (hw & 1) * 64 + half * 32) + lane;
            const uint8_t* row = smem + L::kOffK + st * L::kPieceBytes + r * L::kPitch;
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              const int at = L::kPitch == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
              const uint4 v = *reinterpret_cast<const uint4*>(row + at * 16);
              const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
              __half2 a = __float2half2_rn(0.f);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t x = (w4[k] & 0x007f007fu) << 7, y = (w4[k] & 0x7f007f00u) >> 1;
                a = __hfma2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&x), a);
                a = __hfma2(*reinterpret_cast<const __half2*>(&y), *reinterpret_cast<const __half2*>(&y), a);
              }
              const float2 f = __half22float2(a);
              s += f.x + f.y;
            }
            const float scale = reinterpret_cast<const float*>(smem + L::kOffMeta)[(e % L::kMeta) * 8 + (r >> p.page_shift)];
            top = fmaxf(top, sqrtf(s * 1.02f + 0x1p-16f) * 256.f * fmaxf(scale, 0.f));
          }
          top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
          if (lane == 0) mbar_arrive(bar(L::kBarKEmpty + st));
          if (lane < ntok) {
            float* to = p.norms + (tok + lane - p.tok0) * p.norm_ld + (tile0 + i) * 4;
            if (shared)
              to[hw] = top;
            else
              *reinterpret_cast<float2*>(to + (hw & 1) * 2) = make_float2(top, top);
          }
        }
        if (lane == 0) mbar_arrive(bar(L::kBarQEmpty + qb));
      }
    }
  } else {
    reg_alloc<Ro::kEpilogueRegs>();
    // ------------------------------------------------------------ epilogue
    const int group = warp >> 2, quarter = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int my = quarter * 32 + lane;                  // this thread's row of a tile
    const int eshift = entry_shift(p.block_shift);
    const int64_t ld = p.ld;
    const int recent = p.recent, page_shift = p.page_shift;
    bool ok = *abort_flag == 0;
    int tile_no = 0;
    for (int seg = 0; ok; ++seg) {
      const int qb = seg & 1;
      ok = __all_sync(0xffffffffu, mbar_wait_soon(bar(L::kBarWork + qb), (seg >> 1) & 1, ctl));
      if (!ok) break;
      const Work& wk = works[qb];
      const int ntiles = wk.ntiles, ntok = wk.ntok, tile0 = wk.tile0;
      if (ntiles == 0) break;
      ok = __all_sync(0xffffffffu, mbar_wait_soon(bar(q_bar(seg)), q_phase(seg) & 1, ctl));
      if (!ok) break;
      // A tile's columns are shared by as many warpgroups, and so many sets of them take tiles
      // in turn.
      const int cols = ntok * Hp;
      const int share = cols <= kMine ? 1 : cols <= 2 * kMine ? 2 : 4;
      const int sets = Ro::kGroups / share, set = group / share;
      const int col0 = (group - set * share) * kMine;
      constexpr int kTok = kMine / Hp;                   // tokens of its columns
      const int tok0 = col0 / Hp;
      float w[kMine];
      const float4* ws = reinterpret_cast<const float4*>(smem + L::kOffW + (qb * kCols + col0) * 4);
#pragma unroll
      for (int c = 0; c < kMine / 4; ++c) {
        const float4 v = ws[c];
        w[4 * c] = v.x;
        w[4 * c + 1] = v.y;
        w[4 * c + 2] = 0.5f * v.z;                       // (for twice the ReLU)
        w[4 * c + 3] = 0.5f * v.w;
      }
      int seen[kTok];                                    // rows that its tokens see
#pragma unroll
      for (int i = 0; i < kTok; ++i) seen[i] = tok0 + i < ntok ? wk.n[tok0 + i] : 0;
      int32_t* out = p.rows + (wk.tok + tok0 - p.tok0) * ld;
      for (int i = 0; ok && i < ntiles; ++i, ++tile_no) {
        const int acc = tile_no & 1;
        ok = __all_sync(0xffffffffu, mbar_wait_soon(bar(L::kBarAccFull + acc), (tile_no >> 1) & 1, ctl));
        if (!ok) break;
        if ((tile_no & (sets - 1)) == set && col0 < cols) {
          tc_fence_after();
          const int j = (tile0 + i) * kTile + my;
          float scale = 1.f;
          if constexpr (kPaged) scale = reinterpret_cast<const float*>(smem + L::kOffMeta)[(tile_no % L::kMeta) * 8 + (my >> page_shift)];
          const uint32_t t_acc = tmem + lanes + static_cast<uint32_t>(acc) * kCols + static_cast<uint32_t>(col0);
          // The sums of its tokens, 16 columns of the first 64 beside 16 of the last (four
          // chains of additions in a load's shadow, not two).
          float sum[kTok] = {};
          auto sums = [&](auto both_tag) {
            constexpr bool kBoth = decltype(both_tag)::value;
            float2 a[4];
            auto four = [&](int at, const float* x, float2& u, float2& v) {
              u = fma2(make_float2(w[at], w[at + 1]), make_float2(relu(x[0]), relu(x[1])), u);
              v = fma2(make_float2(w[at + 2], w[at + 3]), make_float2(twice_relu(x[2]), twice_relu(x[3])), v);
            };
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              float x[32];
              tmem_ld16_and_64<kBoth>(t_acc + u * 16, x);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int at = u * 16 + 4 * c;
                if (at % Hp == 0) a[0] = a[1] = a[2] = a[3] = make_float2(0.f, 0.f);
                four(at, x + 4 * c, a[0], a[1]);
                if constexpr (kBoth) four(64 + at, x + 16 + 4 * c, a[2], a[3]);
                if ((at + 4) % (Hp < 64 ? Hp : 64) == 0) {
                  const float first = (a[0].x + a[0].y) + (a[1].x + a[1].y), second = (a[2].x + a[2].y) + (a[3].x + a[3].y);
                  if constexpr (Hp == 128) {
                    sum[0] = first + second;
                  } else {
                    sum[at / Hp] = first;
                    if constexpr (kBoth) sum[kTok / 2 + at / Hp] = second;
                  }
                }
              }
            }
          };
          using Wide = std::bool_constant<kMine == 128>;
          if (kMine == 128 && cols - col0 > 64)
            sums(Wide{});
          else
            sums(std::false_type{});
          if constexpr (!kPaged) {
            // (A key row that holds infinities, with logits of -infinity and NaN: e4m3 has none.)
            bool again = false;
#pragma unroll
            for (int k = 0; k < kTok; ++k) again = again || (tok0 + k < ntok && sum[k] != sum[k]);
            if (__any_sync(0xffffffffu, again)) {
#pragma unroll
              for (int k = 0; k < kTok; ++k)
                sum[k] = sum_of_real_heads(t_acc + k * Hp, base + L::kOffW + (qb * kCols + col0 + k * Hp) * 4, p.H);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kBarAccEmpty + acc));
          // The tokens' scores of this row, written as their blocks'.  (All tokens side by
          // side: one after another they took a latency each, more than the sums.)
          int32_t key[kTok];
#pragma unroll
          for (int k = 0; k < kTok; ++k) {
            key[k] = key_of(kPaged ? sum[k] * scale : sum[k]);
            if (j >= seen[k] - recent) key[k] = kKeyAlways;
            if (j >= seen[k] || (kPaged && scale < 0.f)) key[k] = kKeyNever;
          }
          for (int off = 1; off < (1 << eshift); off <<= 1)
#pragma unroll
            for (int k = 0; k < kTok; ++k) key[k] = max(key[k], __shfl_xor_sync(0xffffffffu, key[k], off));
          int32_t* to = out + (j >> eshift);
          const bool first = (lane & ((1 << eshift) - 1)) == 0;
#pragma unroll
          for (int k = 0; k < kTok; ++k)
            if (first && j < seen[k]) to[k * ld] = key[k];  // (seen[k] = 0: no such token)
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kBarAccEmpty + acc));
        }
      }
      if (lane == 0) mbar_arrive(bar(L::kBarQEmpty + qb));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == Ro::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kCols);
  }
}

template <int D, bool kPaged, int Hp>
cudaError_t launch(const CUtensorMap& tm_k, const CUtensorMap& tm_q, const TopkParams& p, cudaStream_t stream) {
  using L = ScoreLayout<D, kPaged>;
  const auto kern = smqa_topk_score_kernel<D, kPaged, Hp>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), L::kSmem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kSMs);
  cfg.blockDim = dim3(Roles<kPaged, Hp>::kThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tm_k, tm_q, p);
}
template <int D, bool kPaged>
cudaError_t launch(const CUtensorMap& tm_k, const CUtensorMap& tm_q, const TopkParams& p, cudaStream_t stream) {
  switch (padded_heads(p.H)) {
    case 16: return launch<D, kPaged, 16>(tm_k, tm_q, p, stream);
    case 32: return launch<D, kPaged, 32>(tm_k, tm_q, p, stream);
    case 64: return launch<D, kPaged, 64>(tm_k, tm_q, p, stream);
    default: return launch<D, kPaged, 128>(tm_k, tm_q, p, stream);
  }
}

}  // namespace

cudaError_t launch_topk_score(const CUtensorMap& tm_k, const CUtensorMap& tm_q, const TopkParams& p, int D, bool paged, cudaStream_t stream) {
  if (paged) return D == 64 ? launch<64, true>(tm_k, tm_q, p, stream) : launch<128, true>(tm_k, tm_q, p, stream);
  return D == 64 ? launch<64, false>(tm_k, tm_q, p, stream) : launch<128, false>(tm_k, tm_q, p, stream);
}

}  // namespace smqa

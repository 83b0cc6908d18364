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
//        2^-22 of the row's largest value (or of 2^-119);
//   w  = 2^(y_j - u), y_j = x_j + log2 s_j: the weight that multiplies the
//        codes, 2^8 w = hi + lo / 32.  u is an integer for each head and group of
//        32 slots, the least at or above the group's largest y, so that its
//        largest w lies in (1/2, 1]: a weight has a relative error of 2^-8 + 2^-11
//        at most down to 2^-14 of its group's largest, and one of 2^-22 of that
//        below.  The sums' unit is 2^m; the block-scaled MMA (kind::mxf8f6f4)
//        multiplies each group's products by 2^(u - m), and hi's and lo's by their
//        own factor.  One unit for all of a token's slots, as two e4m3 pieces
//        could hold it, ends 2^14 below the largest weight: a long flat rest
//        beside one heavy position would be lost from O, whatever its sum.
//        m is set by the token's first block and raised, O being rescaled, where
//        later ones exceed it by more than 2^32.  l adds w / s_j in fp32.
//        An fp16 number below 2 holds an e4m3 code of its 2^8-fold in bits
//        7-13 (and the sign), subnormals included, so both pieces come from
//        integer operations on pairs of fp16: the conversion instructions
//        share the unit that exp2 needs (a block took 2300 cycles with them).
//
// Work: the tokens' blocks of 128 slots form one sequence, cut into equal
// ranges; a CTA takes one range for one group of up to 64 heads, so a lone
// token's slots and an uneven batch are spread over the whole GPU alike.  A
// token whose blocks lie in one range is finished there; otherwise each CTA
// leaves its O (unnormalised), m and l in the workspace, at most two per CTA,
// and a second kernel joins them.  The two head groups of a token run side by
// side in neighbouring CTAs, so its rows come from HBM once.
//
// Per block (D = 512), 512 threads, one CTA per SM:
//   gather (warps 12-15) slot -> page -> row, and the rows by 16-byte cp.async
//                        into a 128-byte-swizzled tile [D/128][128 slots][128],
//                        three tiles in a ring, a warp's 32 rows freed and
//                        refilled on their own; the slots' scale factors;
//   MMA (warp 8)         S = Q.K^T: M = 128 (64 heads x 2 pieces, A in TMEM,
//                        its last 32 of D in shared memory), N = 128 slots; O^T += V^T.P^T: M = 128 of D (A: the
//                        same tile read MN-major, kept in the collector for
//                        the second piece), N = 64 heads, K = 128 slots, for
//                        both pieces of P;
//   softmax (warps 0-7)  two warpgroups take alternate blocks; a warp reads 16
//                        heads of S, four lanes per head, both pieces of a row
//                        in one lane; weights, their two pieces to shared
//                        memory, Q's pieces into TMEM at the start of a token
//                        and O^T out of it at the end.
// TMEM: S 128 columns, O^T D/2, Q D/4 (D = 512: 8 less), factors 8.
//
// Bound by shared memory: a block writes 64 KB of rows into it and reads them
// for S, again for O (once, by the collector) and P four times (once per 128 of
// D), 2050 cycles at 128 bytes a clock; the tensor core takes 2700 for it (N of
// 64 and 128 fill it by two thirds; the factors make an instruction of O 7 cycles
// longer, eight in a row 704 instead of 645) and a block 3700 in all.  A token's
// end and the next one's start take some 20000 more (the next Q's loads 4000,
// placing it 4000 to 10000, the read-out of O 6000).  Tried and slower, before the
// factors (128 tokens H=128 topk=2048, 80 us then): O's pieces without the
// collector, S and O issued by two warps, 93; P in a ring of three halves, written
// and multiplied by halves, 90; blocks of 64 slots, 84.  128 tokens take 78 us,
// 1024 tokens 501 (H=128, topk=2048), a lone one 17.3, its join included; with one
// unit per token instead of the groups' (which loses flat rests) 74, 480 and 17.2.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "smqa_internal.h"
#include "smqa_paged.cuh"

namespace smqa {

namespace {

constexpr int kBlk = 128;                 // slots per block
constexpr int kHeads = 64;                // heads per CTA
constexpr int kThreads = 512;
constexpr int kSoftmaxThreads = 256;
constexpr int kMmaWarp = 8, kGatherWarp0 = 12;
// Registers per thread of the softmax warpgroups and of the other two: their
// sum is what the block is launched with (128 a thread).
constexpr int kSoftmaxRegs = 192, kOtherRegs = 64;
static_assert(2 * kSoftmaxRegs + 2 * kOtherRegs <= 512, "registers of the launch");
// Warps 0-7 take more registers, 8-15 give some back: a warpgroup does one of
// the two as a whole, or none of its warps would go on.
static_assert(kSoftmaxThreads == 256 && kMmaWarp == 8 && kGatherWarp0 == 12 && kThreads == 512, "roles by warpgroup");
// How far the running maximum may exceed m (in log2), and how far below m a group's
// unit may lie: with 448 2^8 per slot both leave fp32's range alone, and what lies
// further below is lost beside the slot that set m.
constexpr float kLag = 32.f, kDepth = 120.f;
constexpr float kCodeUnit = 0x1p-8f;      // what the tensor core's P counts
constexpr float kFine = 32.f;             // P's lo counts as much less,
constexpr uint32_t kFineSteps = 0x05050505u;  // in four factors' exponents

// What the warpgroup that takes a block tells the other about it: whether it is
// its token's last, and the heads whose m it has raised, to `to`, O and l being
// multiplied by f (of a token's first block, `to` has every head's).  `units` is
// for its own warps: the exponents of 2^(u - m) of each head's four groups of
// slots, as ue8m0 bytes.
struct Note {
  unsigned heads[2];
  int last, failed;
  float to[kHeads], f[kHeads];
  uint32_t units[kHeads];
};
static_assert(sizeof(Note) % 8 == 0, "alignment of what follows");
// A note is cleared four blocks before it is written (by the same warpgroup:
// the vote of its block lies between) and four blocks after it was last read.
constexpr int kNotes = 8;

template <int D>
struct PagedLayout {
  static constexpr int kChunks = D < 128 ? 1 : D / 128;      // 128-byte pieces of a row
  static constexpr uint32_t kChunkBytes = kBlk * 128;
  static constexpr uint32_t kStageBytes = kChunks * kChunkBytes;
  static constexpr int kStages = D == 512 ? 3 : 6;
  static constexpr uint32_t kPieceBytes = kHeads * 128;      // one piece of P^T: 64 heads x 128 slots
  static constexpr uint32_t kQStage = 32 * 64;               // per softmax warp, in P's place: 32 rows x 64 bytes
  static_assert(8 * kQStage <= 2 * kPieceBytes, "Q staging fits P");
  // Per stage and slot pair (a0, a1, c0, c1), then the r of all slots, two
  // pairs of one lane together (meta_at, rec_at).
  static constexpr int kMeta = 4 * kBlk / 2 + kBlk;          // floats
  static constexpr uint32_t kOffP = kStages * kStageBytes;
  // The last 32 elements of Q's rows, where TMEM has no room for them: as 8 x 16-byte
  // matrices, [16 groups of 8 rows][2][8][16].
  static constexpr bool kQTail = D == 512;
  static constexpr uint32_t kOffQ = kOffP + 2 * kPieceBytes;
  static constexpr uint32_t kOffA = kOffQ + (kQTail ? 4096 : 0);  // [kStages][kMeta]: a, c, r
  static constexpr uint32_t kOffFlags = kOffA + kStages * kMeta * 4;  // [kStages]
  static constexpr uint32_t kOffHead = (kOffFlags + kStages * 4 + 15) & ~15u;  // float [64]
  static constexpr uint32_t kOffMax = kOffHead + kHeads * 4;   // uint32 [2][64] (QLoader)
  static constexpr uint32_t kOffSum = kOffMax + 2 * kHeads * 4;  // float [2][64]
  static constexpr uint32_t kOffEnd = kOffSum + 2 * kHeads * 4;  // float [64]
  static constexpr uint32_t kOffNotes = kOffEnd + kHeads * 4;  // Note [kNotes]
  static constexpr uint32_t kOffBar = kOffNotes + kNotes * sizeof(Note);
  static constexpr int kBarFull = 0;                         // [kStages]
  static constexpr int kBarEmpty = kBarFull + kStages;       // [kStages][4], a gather warp's rows
  static constexpr int kBarSFull = kBarEmpty + 4 * kStages;
  static constexpr int kBarSFree = kBarSFull + 1;
  static constexpr int kBarPFull = kBarSFree + 1;
  // P and its tile used, O up to date.  [2], of even and odd entries: a
  // warpgroup waits for every other one, which in one barrier's two parities
  // could not be told from the one before.
  static constexpr int kBarPDone = kBarPFull + 1;
  static constexpr int kBarNote = kBarPDone + 2;             // [2] a warpgroup's note is written
  static constexpr int kBarQFull = kBarNote + 2;
  static constexpr int kBarDrain = kBarQFull + 1;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr uint32_t kOffCtl = kOffBar + 8 * kNumBars;  // TMEM base, abort flag
  static constexpr uint32_t kOffRange = kOffCtl + 8;         // range of the CTA, scan space
  static constexpr uint32_t kSmem = kOffRange + 192 + 1024;  // + alignment
  static_assert(kOffRange % 8 == 0, "alignment");
  static_assert(kSmem <= 232448, "shared memory budget");
  static constexpr uint32_t kTmemS = 0, kTmemO = 128;
  static constexpr uint32_t kTmemQ = kTmemO + kChunks * kHeads;
  static constexpr uint32_t kTmemCols = D == 512 ? 512 : 256;
  // The block-scaled MMA's factors: of V's 128 rows (all 1) and of the 64 heads, for
  // P's hi and lo.
  static constexpr uint32_t kTmemFV = kTmemCols - 8, kTmemFHi = kTmemFV + 4, kTmemFLo = kTmemFHi + 2;
  static_assert(kTmemQ + (D - (kQTail ? 32 : 0)) / 4 <= kTmemFV, "TMEM budget");
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
// A part: O as [D / 128][16 groups of 4 heads][128 columns][4 heads] (D = 64:
// half of the columns unused), then m and l of the heads.
__host__ __device__ constexpr int part_o(int D) { return kHeads * (D < 128 ? 128 : D); }
__host__ __device__ constexpr size_t part_floats(int D) { return static_cast<size_t>(part_o(D)) + 2 * kHeads; }

__device__ __forceinline__ bool live_token(const PagedFwdParams& p, int req) {
  return static_cast<unsigned>(req) < static_cast<unsigned>(p.R);
}
// Slots to look at for token t of request req.
__device__ __forceinline__ int slots_of(const PagedFwdParams& p, int t, int req, int len) {
  if (p.idx) return p.topk;
  const int64_t cap = static_cast<int64_t>(p.max_pages) << p.page_shift;
  const int64_t n = min(min(static_cast<int64_t>(len), static_cast<int64_t>(load(p.positions + t)) + 1), cap);
  return n > 0 ? static_cast<int>(n) : 0;
}
// Blocks of token t: at least one (it writes O = 0), none for padding.
__device__ __forceinline__ int blocks_of(const PagedFwdParams& p, int t, int req) {
  if (!live_token(p, req)) return 0;
  if (p.idx) return (p.topk + kBlk - 1) / kBlk;
  return max(1, (slots_of(p, t, req, load(p.seq_lens + req)) + kBlk - 1) / kBlk);
}

__device__ __forceinline__ int blocks_of(const PagedFwdParams& p, int t) { return blocks_of(p, t, load(p.token_req + t)); }

// The two e4m3 pieces of 2^8 w for four weights 0 <= w <= 1: hi the nearest code
// (halves up), lo that of 32 times the rest (which is 2^-5 at most).
__device__ __forceinline__ void split_e4m3x4(float2 w01, float2 w23, uint32_t& hi, uint32_t& lo) {
  const __half2 a = __floats2half2_rn(w01.x, w01.y), b = __floats2half2_rn(w23.x, w23.y);
  const uint32_t ra = *reinterpret_cast<const uint32_t*>(&a) + 0x00400040u;
  const uint32_t rb = *reinterpret_cast<const uint32_t*>(&b) + 0x00400040u;
  hi = __byte_perm(ra << 1, rb << 1, 0x7531);
  const uint32_t ka = ra & 0xff80ff80u, kb = rb & 0xff80ff80u;
  const __half2 fine = __float2half2_rn(kFine);
  const __half2 da = __hmul2(__hsub2(a, *reinterpret_cast<const __half2*>(&ka)), fine);
  const __half2 db = __hmul2(__hsub2(b, *reinterpret_cast<const __half2*>(&kb)), fine);
  const uint32_t sa = *reinterpret_cast<const uint32_t*>(&da) + 0x00400040u;
  const uint32_t sb = *reinterpret_cast<const uint32_t*>(&db) + 0x00400040u;
  // The sign next to the code (bit 14 is free: the values are below 2).
  lo = __byte_perm((sa | ((sa >> 1) & 0x40004000u)) << 1, (sb | ((sb >> 1) & 0x40004000u)) << 1, 0x7531);
}

// Where slot n's factors a and c (+ 2) lie among a stage's floats, and its r:
// the softmax lane q of a quad takes the slot pairs 8j + 2q, two j at a time.
__device__ __forceinline__ int meta_at(int n) { return (n >> 1) * 4 + (n & 1); }
__device__ __forceinline__ int rec_at(int n) {
  return 2 * kBlk + (n >> 4) * 16 + ((n >> 1) & 3) * 4 + ((n >> 3) & 1) * 2 + (n & 1);
}

// The e4m3 codes of 2^8 x for four fp16 values |x| <= 1.6875 (nearest, halves
// away from 0), and the rounded values.
__device__ __forceinline__ uint32_t round_e4m3x4(__half2 a, __half2 b, __half2& ra, __half2& rb) {
  const uint32_t sa = *reinterpret_cast<const uint32_t*>(&a) + 0x00400040u;
  const uint32_t sb = *reinterpret_cast<const uint32_t*>(&b) + 0x00400040u;
  const uint32_t ka = sa & 0xff80ff80u, kb = sb & 0xff80ff80u;
  ra = *reinterpret_cast<const __half2*>(&ka);
  rb = *reinterpret_cast<const __half2*>(&kb);
  // The sign next to the code (bit 14 is free: the values are below 2).
  return __byte_perm((sa | ((sa >> 1) & 0x40004000u)) << 1, (sb | ((sb >> 1) & 0x40004000u)) << 1, 0x7531);
}

// Q of a token, heads h0.. (`heads` of them, zeros behind), by the eight softmax
// warps: a warp takes 16 heads and half of D, two heads at a time (four columns
// per lane of each 64-column piece).  fetch() loads it into registers; place()
// writes both pieces of every row into TMEM lanes (of 16 lanes, 0-7 the hi
// pieces of eight heads, 8-15 their lo pieces) once the MMAs that read the Q and
// the P before are done, and returns 2^-k of the two heads whose S the lane
// reads (NaN where a row is not finite).
template <int D>
struct QLoader {
  using L = PagedLayout<D>;
  static constexpr int kC = D < 128 ? 1 : D / 128;       // 64-column pieces per warp
  uint2 v[8][kC];

  __device__ __forceinline__ void fetch(const PagedFwdParams& p, int t, int h0, int heads, int quarter, int half,
                                        int lane) {
    const bool mine = D >= 128 || half == 0;             // (D = 64 is one piece)
    const __nv_bfloat16* q0 = p.q + (static_cast<int64_t>(t) * p.H + h0) * D + half * kC * 64 + (lane & 15) * 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int h = 16 * quarter + 2 * i + (lane >> 4);
#pragma unroll
      for (int c = 0; c < kC; ++c)
        v[i][c] = mine && h < heads ? load(reinterpret_cast<const uint2*>(q0 + static_cast<int64_t>(h) * D + c * 64))
                                    : make_uint2(0, 0);
    }
  }

  __device__ __forceinline__ float2 place(uint32_t base, uint8_t* smem, uint32_t tmem, int quarter, int half,
                                         int lane) {
    const int sub = lane >> 4, l16 = lane & 15;
    uint32_t* head_top = reinterpret_cast<uint32_t*>(smem + L::kOffMax);  // [2][64] largest magnitudes
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = 0;                                    // bf16 bit patterns order like values
#pragma unroll
      for (int c = 0; c < kC; ++c) m = __vmaxu2(m, __vmaxu2(v[i][c].x & 0x7fff7fffu, v[i][c].y & 0x7fff7fffu));
      m = max(m & 0xffffu, m >> 16);
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
      if (l16 == 0) head_top[half * kHeads + 16 * quarter + 2 * i + sub] = m;
    }
    bar_sync(4 + quarter, 64);
    auto top_of = [&](int h) { return max(head_top[h], head_top[kHeads + h]); };
    // floor(log2) of the largest magnitude, not below -119 (whose 2^-k is the
    // smallest normal number).
    auto exponent = [](uint32_t m) { return max(static_cast<int>(m >> 7) - 127, -119); };
    const uint32_t stage = base + L::kOffP + static_cast<uint32_t>(4 * half + quarter) * L::kQStage;
    if (D >= 128 || half == 0) {
      // In fp16, scaled so that the row's largest value lies in [1/2, 1): exact
      // but for values below 2^-13 of it (then off by 2^-25 at most).
      float2 f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = -1 - exponent(min(top_of(16 * quarter + 2 * i + sub), 0x7f7fu));
        const float x = k > -127 ? pow2f(k) : k == -127 ? 0x1p-127f : 0x1p-128f;  // (pow2f is of normal numbers)
        f[i] = make_float2(x, x);
      }
#pragma unroll
      for (int c = 0; c < kC; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 x01 = mul2(make_float2(__uint_as_float(v[i][c].x << 16), __uint_as_float(v[i][c].x & 0xffff0000u)), f[i]);
          const float2 x23 = mul2(make_float2(__uint_as_float(v[i][c].y << 16), __uint_as_float(v[i][c].y & 0xffff0000u)), f[i]);
          const __half2 a = __floats2half2_rn(x01.x, x01.y), d = __floats2half2_rn(x23.x, x23.y);
          __half2 ra, rd;
          const uint32_t hi = round_e4m3x4(a, d, ra, rd);
          const __half2 times = __float2half2_rn(32.f);
          const uint32_t lo = round_e4m3x4(__hmul2(__hsub2(a, ra), times), __hmul2(__hsub2(d, rd), times), ra, rd);
          const int hh = 2 * i + sub;                    // of the warp's 16 heads
          const uint32_t r = static_cast<uint32_t>(hh + (hh & 8));  // rows r, r + 8
          const uint32_t at = stage + r * 64u + ((static_cast<uint32_t>(l16 >> 2) ^ ((r >> 1) & 3u)) << 4) + (l16 & 3) * 4;
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(hi) : "memory");
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 512u), "r"(lo) : "memory");
        }
        __syncwarp();
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 x = *reinterpret_cast<const uint4*>(smem + (stage - base) + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4));
          w[4 * k] = x.x;
          w[4 * k + 1] = x.y;
          w[4 * k + 2] = x.z;
          w[4 * k + 3] = x.w;
        }
        const uint32_t to = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + L::kTmemQ + (half * kC + c) * 16;
        if (L::kQTail && half == 1 && c == kC - 1) {     // 32 of the 64 elements to shared memory
          tmem_st8u(to, w);
          uint4* tail = reinterpret_cast<uint4*>(smem + L::kOffQ + quarter * 1024 + (lane >> 3) * 256 + (lane & 7) * 16);
          tail[0] = make_uint4(w[8], w[9], w[10], w[11]);
          tail[8] = make_uint4(w[12], w[13], w[14], w[15]);
          tmem_wait_st();
        } else {
          tmem_st16u(to, w);
        }
        __syncwarp();
      }
    }
    const uint32_t t0 = top_of(16 * quarter + (lane >> 2)), t1 = top_of(16 * quarter + 8 + (lane >> 2));
    auto scale = [&](uint32_t m) { return m >= 0x7f80u ? __uint_as_float(0x7fffffffu) : pow2f(exponent(m) - 7); };
    return make_float2(scale(t0), scale(t1));
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) smqa_paged_fwd_kernel(const PagedFwdParams p) {
  using L = PagedLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint32_t base = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (base & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  base += pad;
  // (The warp's number as a value the compiler knows to be the same in all
  // lanes: without it the instructions that feed the tensor core take 15 %
  // longer to issue.)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int groups = (p.H + kHeads - 1) / kHeads;
  const int part = blockIdx.x / groups, parts = gridDim.x / groups;
  const int h0 = (blockIdx.x % groups) * kHeads;
  const int heads = min(kHeads, p.H - h0);
  auto bar = [&](int i) -> uint32_t { return base + L::kOffBar + 8u * static_cast<uint32_t>(i); };
  volatile uint32_t* tmem_holder = reinterpret_cast<volatile uint32_t*>(smem + L::kOffCtl);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffCtl + 4);
  const WaitCtl ctl{abort_flag, p.status, p.limit_ns};
  Range* range = reinterpret_cast<Range*>(smem + L::kOffRange);
  int64_t* warp_sum = reinterpret_cast<int64_t*>(smem + L::kOffRange + 16);  // [16]
  int* end_tok = reinterpret_cast<int*>(smem + L::kOffRange + 16 + 128);     // token, its end, its begin

  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i) mbar_init(bar(L::kBarFull + i), 128 + 4);  // copies landed, factors written
    for (int i = 0; i < 4 * L::kStages; ++i) mbar_init(bar(L::kBarEmpty + i), 1);
    mbar_init(bar(L::kBarSFull), 1);
    mbar_init(bar(L::kBarSFree), kSoftmaxThreads / 64);  // (one arrival per warp)
    mbar_init(bar(L::kBarPFull), kSoftmaxThreads / 64);
    for (int i = 0; i < 2; ++i) mbar_init(bar(L::kBarPDone + i), 1);
    mbar_init(bar(L::kBarNote), kSoftmaxThreads / 64);
    mbar_init(bar(L::kBarNote + 1), kSoftmaxThreads / 64);
    mbar_init(bar(L::kBarQFull), kSoftmaxThreads / 32);
    mbar_init(bar(L::kBarDrain), 1);
    range->count = 0;
    end_tok[0] = -1;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(base + L::kOffCtl, L::kTmemCols);
  // So far beside the kernel before, whose results are read (or whose workspace
  // is written) from here on.
  grid_dependency_wait();
  grid_dependents_launch();
  if (tid == 0) *abort_flag = *reinterpret_cast<volatile int*>(p.status) != 0 ? 1 : 0;
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
    // Equal ranges, the first total mod parts of them one block (or token)
    // longer.
    const int unit = p.whole_tokens && p.idx ? (p.topk + kBlk - 1) / kBlk : 1;
    total = static_cast<uint32_t>(total >> 32) != 0 ? total / unit : static_cast<uint32_t>(total) / static_cast<uint32_t>(unit);
    const int64_t each = (total >> 32) != 0 ? total / parts : static_cast<uint32_t>(total) / static_cast<uint32_t>(parts);
    const int extra = static_cast<int>(total - each * parts);
    const int64_t begin = (each * part + min(part, extra)) * unit, end = begin + (each + (part < extra ? 1 : 0)) * unit;
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
    if (!p.whole_tokens) reinterpret_cast<Leftover*>(p.ws)[blockIdx.x] = l;
  }

  // Padding tokens belong to no range; warps without another role see to them.
  if (p.zero_padding && warp > kMmaWarp && warp < kGatherWarp0)
    for (int t = blockIdx.x + (warp - kMmaWarp - 1) * gridDim.x; t < p.T; t += gridDim.x * (kGatherWarp0 - kMmaWarp - 1))
      if (!live_token(p, load(p.token_req + t))) {
        uint4* o = reinterpret_cast<uint4*>(p.o + static_cast<int64_t>(t) * p.H * D);
        for (int i = lane; i < p.H * D / 8; i += 32) o[i] = make_uint4(0, 0, 0, 0);
        for (int h = lane; h < p.H; h += 32) p.lse[static_cast<int64_t>(t) * p.H + h] = -INFINITY;
      }

  if (rg.count > 0 && warp >= kGatherWarp0) {
    reg_dealloc<kOtherRegs>();
    // ------------------------------------------------------------ gather
    // Looking a slot up takes three loads, one after another: while the rows
    // of one block are copied, the next block's indices and then its pages
    // arrive.
    const int pw = warp - kGatherWarp0;
    const int my = 32 * pw + lane;                       // this thread's slot of a block
    int64_t left = rg.count;                             // blocks behind the current token's
    int t = rg.tok - 1, b = 0, stop = 0, n = 0, len = 0;
    const int32_t *idx_row = nullptr, *tab = nullptr;
    bool fresh = true;                                   // no block of this token yet
    int idx[4];                                          // of slots 32 k + lane
    // Goes to the next block and asks for its indices.
    auto ask = [&] {
      if (++b >= stop) {
        int nb;
        do nb = blocks_of(p, ++t);
        while (nb == 0);
        const int req = load(p.token_req + t);
        b = t == rg.tok ? rg.off : 0;
        stop = static_cast<int>(min(static_cast<int64_t>(nb), b + left));
        left -= stop - b;
        len = load(p.seq_lens + req);
        n = slots_of(p, t, req, len);
        tab = p.table + static_cast<int64_t>(req) * p.max_pages;
        idx_row = p.idx ? p.idx + static_cast<int64_t>(t) * p.topk : nullptr;
        fresh = true;
      }
      if (idx_row)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int j = b * kBlk + 32 * k + lane;
          idx[k] = j < n ? load(idx_row + j) : -1;
        }
    };
    // This slot's position in its page and its page (-1: masked); the block's
    // flags.  A block without any slot left is passed over, but for the last,
    // which carries the token's end.
    int in_page = 0, page = -1, flags = 0;
    auto look = [&] {
      int pos = -1;
      while (true) {
        if (!idx_row) {
          if (b * kBlk + my < n) pos = b * kBlk + my;
          break;
        }
        unsigned any = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool in = idx[k] >= 0 && idx[k] < len;
          any |= __ballot_sync(0xffffffffu, in);
          if (k == pw && in) pos = idx[k];
        }
        if (any != 0 || b + 1 == stop) break;
        ask();
      }
      const bool last = b + 1 == stop;
      flags = (fresh ? kFirst : 0) | (last ? kLast : 0) | (last && left == 0 ? kFinal : 0);
      fresh = false;
      const int col = pos >> p.page_shift;
      in_page = pos & ((1 << p.page_shift) - 1);
      page = pos >= 0 && col < p.max_pages ? load(tab + col) : -1;
    };
    // This slot's row on its way to L2: the tile it will be copied to may be in
    // use for longer than HBM takes.
    auto prefetch = [&] {
      if (static_cast<unsigned>(page) < static_cast<unsigned>(p.n_pages)) {
        const uint8_t* r = p.cache + ((static_cast<int64_t>(page) << p.page_shift) + in_page) * D;
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c) asm volatile("prefetch.global.L2 [%0];" ::"l"(r + c * 128));
      }
    };
    ask();
    look();
    for (int e = 0;; ++e) {
      const bool live = static_cast<unsigned>(page) < static_cast<unsigned>(p.n_pages);
      const int row = live ? (page << p.page_shift) + in_page : 0;
      const float s = live ? load(p.scales + page) : 1.f;
      const unsigned mask = __ballot_sync(0xffffffffu, live);
      const int now = flags;
      if (!(now & kFinal)) ask();
      const int st = e % L::kStages;
      if (e >= L::kStages) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar(L::kBarEmpty + 4 * st + pw), ((e / L::kStages) - 1) & 1, ctl))) break;
      } else if (!__all_sync(0xffffffffu, *abort_flag == 0)) {
        break;
      }
      const uint32_t tile = base + static_cast<uint32_t>(st) * L::kStageBytes;
      // An instruction copies 128 bytes (D = 64: 64) of each of several rows:
      // a row's address is fetched from its lane once, its further pieces are
      // at fixed distances (4 warps: 52 bytes a clock from L2, against 38 with
      // one whole row per instruction).
      constexpr int kLanes = D < 128 ? D / 16 : 8;       // lanes per row
      constexpr int kRows = 32 / kLanes;                 // rows per instruction
      const int sub = lane / kLanes, cc = lane % kLanes;
      const uint8_t* src = p.cache + cc * 16;
      auto copy = [&](int g) {                           // rows g kRows + sub of the warp's 32
        const int rw = g * kRows + sub;
        const uint8_t* from = src + static_cast<int64_t>(__shfl_sync(0xffffffffu, row, rw)) * D;
        const bool on = (mask >> rw) & 1u;
        const uint32_t to = tile + static_cast<uint32_t>(32 * pw + rw) * 128u + ((static_cast<uint32_t>(cc) ^ (static_cast<uint32_t>(rw) & 7u)) << 4);
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c) cp_async_16_or_zero(to + c * L::kChunkBytes, from + c * 128, on);
      };
#pragma unroll
      for (int g = 0; g < 16 / kRows; ++g) copy(g);
      if (!(now & kFinal)) look();
#pragma unroll
      for (int g = 16 / kRows; g < 32 / kRows; ++g) copy(g);
      // y = S a + c, l += w r: a masked slot's row is zero, its c -inf.
      float* m = reinterpret_cast<float*>(smem + L::kOffA) + st * L::kMeta;
      m[meta_at(my)] = live ? s * p.scale_log2 : 0.f;
      m[meta_at(my) + 2] = live ? log2f(s) : -INFINITY;
      m[rec_at(my)] = live ? 1.f / s : 0.f;
      if (my == 0) reinterpret_cast<int*>(smem + L::kOffFlags)[st] = now;
      if (!(now & kFinal) && e >= L::kStages - 1) prefetch();
      cp_async_arrive_noinc(bar(L::kBarFull + st));      // once the copies have landed
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kBarFull + st)); // releases the factors
      if (now & kFinal) break;
    }
    cp_async_wait_all();
  } else if (rg.count > 0 && warp >= kMmaWarp) {
    reg_dealloc<kOtherRegs>();                           // (the warpgroup's other warps have no role)
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs this, one lane of it issues.
    if (warp == kMmaWarp) {
      constexpr uint32_t idesc_s = idesc_e4m3_f32(128, kBlk, false);
      const uint64_t d_k = smem_desc(base, 16u, 1024u, kSwizzle128B);
      const uint64_t d_v = smem_desc(base, L::kChunkBytes, 1024u, kSwizzle128B);
      const uint64_t d_p = smem_desc(base + L::kOffP, 16u, 1024u, kSwizzle128B);
      const uint64_t d_q = smem_desc(base + L::kOffQ, 128u, 256u, 0u);
      const volatile int* flags_of = reinterpret_cast<const volatile int*>(smem + L::kOffFlags);
      auto issue_s = [&](int st) {
        const uint64_t k = d_k + ((static_cast<uint32_t>(st) * L::kStageBytes) >> 4);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const uint64_t kd = k + (((c / 4) * L::kChunkBytes + (c % 4) * 32u) >> 4);
          if (L::kQTail && c == D / 32 - 1)
            mma8_ss(tmem + L::kTmemS, d_q, kd, idesc_s, 1u);
          else
            mma8_ts(tmem + L::kTmemS, tmem + L::kTmemQ + c * 8, kd, idesc_s, c != 0 ? 1u : 0u);
        }
        mma_commit_elect(bar(L::kBarSFull));
      };
      auto issue_o = [&](int e, int st, bool first) {
        const uint64_t v = d_v + ((static_cast<uint32_t>(st) * L::kStageBytes) >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
          for (int c = 0; c < L::kChunks; ++c) {
            const uint64_t ad = v + ((c * L::kChunkBytes + k * 4096u) >> 4);
            const uint64_t bd = d_p + ((k * 32u) >> 4);
            const uint32_t idesc_o = idesc_mx_e4m3_f32(128, kHeads, true, k);
            mma_mx_ss_keep(tmem + L::kTmemO + c * kHeads, ad, bd, idesc_o, tmem + L::kTmemFV, tmem + L::kTmemFHi,
                           (!first || k > 0) ? 1u : 0u);
            mma_mx_ss_again(tmem + L::kTmemO + c * kHeads, ad, bd + (L::kPieceBytes >> 4), idesc_o, tmem + L::kTmemFV,
                            tmem + L::kTmemFLo, 1u);
          }
          mma_commit_elect(bar(L::kBarEmpty + 4 * st + k));
        }
        mma_commit_elect(bar(L::kBarPDone + (e & 1)));
      };
      // S of an entry before O of the one before, so that the softmax works on the
      // former's while the latter is formed; but O first if the rows come late.
      // A test of a barrier takes some 280 cycles beside the other warps' copies
      // and stores: what has been seen done is not asked again.
      auto wait = [&](int i, int phase) { return __all_sync(0xffffffffu, mbar_wait(bar(i), phase & 1, ctl)); };
      auto ready = [&](int i, int phase) { return __all_sync(0xffffffffu, mbar_probe(bar(i), phase & 1)); };
      bool ok = *abort_flag == 0, more = true, rows = false;  // (more S to come; the next one's rows are there)
      int ns = 0, no = 0, seg = 0, st_s = 0, turn = 0, st_o = 0, flags = 0;
      unsigned begins = 0;                               // bit i: entry no + i is its token's first
      PollState ps = poll_start();
      for (uint32_t spins = 0; ok && (more || no < ns);) {
        const bool only_o = !more || ns - no >= 2;       // (S after next: its softmax waits for O)
        bool s_next = false;
        if (!only_o) {
          if (!rows && (rows = ready(L::kBarFull + st_s, turn))) flags = flags_of[st_s];
          s_next = rows && (ns == 0 || ready(L::kBarSFree, ns - 1));
          // A token's first S needs its Q, brought once the token before is finished.
          if (s_next && (flags & kFirst)) s_next = no == ns && ready(L::kBarQFull, seg);
        }
        if (s_next) {
          if (flags & kFirst) {
            ++seg;
            begins |= 1u << (ns - no);
          }
          fence_proxy_async_smem();                      // rows written by cp.async -> tensor core
          tc_fence_after();
          issue_s(st_s);
          more = (flags & kFinal) == 0;
          if (ns == 0 && static_cast<int>(blockIdx.x) == p.stall_cta) {  // test hook only
            ok = __any_sync(0xffffffffu, stall_until_limit(ctl));
            break;
          }
          rows = false;
          ++ns;
          if (++st_s == L::kStages) {
            st_s = 0;
            ++turn;
          }
        } else if (only_o ? (ok = wait(L::kBarPFull, no)) : no < ns && ready(L::kBarPFull, no)) {
          tc_fence_after();
          issue_o(no, st_o, begins & 1u);
          begins >>= 1;
          ++no;
          if (++st_o == L::kStages) st_o = 0;
        } else {
          if ((++spins & 63u) == 0u) ok = ok && __all_sync(0xffffffffu, poll_check(ctl, ps));
          continue;
        }
        ps.t0 = globaltimer_ns();                        // progress: the limit counts from here
      }
      mma_commit_elect(bar(L::kBarDrain));
      mbar_wait_drain(bar(L::kBarDrain), 0);
    }
    __syncwarp();
  } else if (rg.count > 0) {
    reg_alloc<kSoftmaxRegs>();
    // ------------------------------------------------------------ softmax
    // A warpgroup takes every other ring entry.  Its warp w owns the TMEM lanes
    // of quarter w, 16 heads.  A thread whose wait failed keeps taking the same
    // steps as the others and says so in its next note, which all read before
    // they leave: none waits at a barrier that another has left.
    const int quarter = warp & 3, half = warp >> 2;      // half: the warpgroup
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int hq = 16 * quarter + (lane >> 2);           // this lane's heads: hq, hq + 8
    const int quad = lane & 3;                           // its slots: pairs 8 j + 2 quad
    const bool lead = quad == 0;
    // Byte selectors of the exchange between lanes of a pair (below).
    const uint32_t sel_send = (lane & 1) ? 0x5410u : 0x7632u;
    const uint32_t sel_hi = (lane & 1) ? 0x3254u : 0x5410u, sel_lo = (lane & 1) ? 0x3276u : 0x7610u;
    float* head_f = reinterpret_cast<float*>(smem + L::kOffHead);
    float* head_sum = reinterpret_cast<float*>(smem + L::kOffSum);  // at a token's end: l of each
    float* head_end = reinterpret_cast<float*>(smem + L::kOffEnd);  // warpgroup, and m
    Note* notes = reinterpret_cast<Note*>(smem + L::kOffNotes);
    const volatile int* flags_of = reinterpret_cast<const volatile int*>(smem + L::kOffFlags);
    auto done_with = [&](int e) { return mbar_wait(bar(L::kBarPDone + (e & 1)), (e >> 1) & 1, ctl); };
    int64_t left = rg.count;
    int e = 0;
    bool run = true;
    bool bad = *abort_flag != 0;                         // a wait of this thread has failed
    const float sink = tid < heads ? load(p.sink + h0 + tid) * 1.4426950408889634f : 0.f;  // (thread = head)
    if (tid < kNotes) notes[tid].heads[0] = notes[tid].heads[1] = notes[tid].failed = 0;
    if (half == 0) {                                     // V's factors (seen by the tensor core as Q is)
      tmem_st4u(tmem + lanes + L::kTmemFV, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
      tmem_wait_st();
    }
    bar_sync(1, kSoftmaxThreads);
    // The CTA's tokens, or parts of tokens, one after another.
    int t = rg.tok, b = rg.off, nb = blocks_of(p, t);
    QLoader<D> q;
    q.fetch(p, t, h0, heads, quarter, half, lane);
    float2 rs = make_float2(0.f, 0.f);
    int done = -1, slot = 0;                             // the token before (-1: none yet), its part
    bool whole = false;
    // (One copy of the code that places Q and of the one that reads O out: the
    // first time through a piece of code is slow.)
    while (true) {
      // The next token's Q, whose S then runs beside what is left of the one before.
      const bool more = done < 0 || left > 0;
      if (more) {
        rs = q.place(base, smem, tmem, quarter, half, lane);
        tc_fence_before();
        if (L::kQTail) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kBarQFull));
      }
      // The token's (or its part's) result.
      if (done >= 0) {
        float* ws = reinterpret_cast<float*>(p.ws + kLeftoverBytes) +
                    (static_cast<int64_t>(blockIdx.x) * 2 + slot) * part_floats(D);
        if (tid < kHeads) {                                // thread = head
          const int hl = tid;
          const float m_end = head_end[hl], l_end = head_sum[hl] + head_sum[kHeads + hl];
          if (whole) {
            const float top = fmaxf(m_end, sink);
            float inv, lse;
            if (top == -INFINITY && sink == -INFINITY) {   // nothing at all (or only NaN)
              inv = l_end * 0.f;
              lse = l_end != l_end ? l_end : -INFINITY;
            } else {
              const float f = exp2f(m_end - top);
              const float total = fmaf(l_end, f, exp2f(sink - top));
              inv = kCodeUnit * f / total;
              lse = log2f(total) + top;
            }
            head_f[hl] = inv;
            if (hl < heads) p.lse[static_cast<int64_t>(done) * p.H + h0 + hl] = lse;
          } else {
            ws[part_o(D) + hl] = m_end;
            ws[part_o(D) + kHeads + hl] = l_end;
          }
        }
        if (whole) {
          bar_sync(1, kSoftmaxThreads);
          // 32 heads x 32 columns a time through the warp's part of P's place
          // (free now) to 64-byte rows: [head][4 pieces of 8 columns].
          uint8_t* tile = smem + L::kOffP + warp * 2048;
          const uint32_t tile_at = base + L::kOffP + warp * 2048;
          float2 f[4];                                     // of heads 8 j + 2 quad, + 1
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = *reinterpret_cast<const float2*>(head_f + half * 32 + 8 * j + 2 * quad);
          if (D >= 128 || quarter < D / 32) {
#pragma unroll 1
            for (int c = 0; c < L::kChunks; ++c) {
              float v[2][16];                              // columns 0-15, 16-31 of the quarter's 32
              tmem_ld16x32x2(tmem + lanes + L::kTmemO + c * kHeads + half * 32, v[0], v[1]);
#pragma unroll
              for (int j = 0; j < 4; ++j) {                // 8 heads: four 8-column matrices
                uint32_t w[4];
#pragma unroll
                for (int o = 0; o < 4; ++o)
                  w[o] = pack_bf16x2(v[o >> 1][4 * j + 2 * (o & 1)] * f[j].x, v[o >> 1][4 * j + 2 * (o & 1) + 1] * f[j].y);
                const uint32_t h = static_cast<uint32_t>(8 * j + (lane & 7));
                stmatrix_trans_x4(tile_at + h * 64u + ((static_cast<uint32_t>(lane >> 3) ^ ((h >> 1) & 3u)) << 4), w[0], w[1], w[2], w[3]);
              }
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int h = 8 * i + (lane >> 2);
                const uint4 x = *reinterpret_cast<const uint4*>(tile + h * 64 + ((quad ^ ((h >> 1) & 3)) << 4));
                if (half * 32 + h < heads)
                  *reinterpret_cast<uint4*>(p.o + (static_cast<int64_t>(done) * p.H + h0 + half * 32 + h) * D + c * 128 + 32 * quarter + quad * 8) = x;
              }
              __syncwarp();
            }
          }
        } else if (D >= 128 || quarter < D / 32) {
          float4* part = reinterpret_cast<float4*>(ws) + half * 8 * 128 + 32 * quarter + lane;
#pragma unroll 1
          for (int c = 0; c < L::kChunks; ++c) {           // 128 of D, 32 heads per warpgroup
            float o[32];
            tmem_ld32(tmem + lanes + L::kTmemO + c * kHeads + half * 32, o);
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              __stcg(part + (c * (kHeads / 4) + i / 4) * 128, make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]));
          }
        }
        tc_fence_before();
        if (!more) break;
        // Both have read O and P's place before either brings the next token's.
        bar_sync(1, kSoftmaxThreads);
      }
      const int stop = static_cast<int>(min(static_cast<int64_t>(nb), b + left));
      whole = b == 0 && stop == nb;
      slot = b == 0 ? 1 : 0;                             // of the CTA's two workspace parts
      left -= stop - b;
      // (Asked for here: its answer takes 1600 cycles at the token's end.)
      int next_req = left > 0 ? load(p.token_req + t + 1) : -1;

      float m[2] = {-INFINITY, -INFINITY};
      float2 l[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};  // (even and odd slots apart)
      for (bool first = true, last = false; !last; first = false, ++e) {
        Note* note = notes + e % kNotes;
        // Every softmax warp comes here for every block, failed or not.
        auto wait_note = [&] {
          if (!mbar_test(bar(L::kBarNote + (e & 1)), (e >> 1) & 1))
            mbar_wait_drain(bar(L::kBarNote + (e & 1)), (e >> 1) & 1, 2 * p.limit_ns + 1000000000ull);
          __syncwarp();
        };
        if ((e & 1) != half) {                           // the other warpgroup's block
          wait_note();
          if (*reinterpret_cast<volatile int*>(&note->failed) != 0) {
            run = false;
            break;
          }
          last = note->last != 0;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int h = hq + 8 * g;
            if (first) {
              m[g] = note->to[h];
            } else if ((note->heads[h >> 5] >> (h & 31)) & 1u) {
              m[g] = note->to[h];
              l[g] = mul2(l[g], make_float2(note->f[h], note->f[h]));
            }
          }
          continue;
        }
        const int st = e % L::kStages;
        if (!mbar_wait(bar(L::kBarFull + st), (e / L::kStages) & 1, ctl)) bad = true;  // the factors
        if (!mbar_wait(bar(L::kBarSFull), e & 1, ctl)) bad = true;
        __syncwarp();
        tc_fence_after();
        const float* meta = reinterpret_cast<const float*>(smem + L::kOffA) + st * L::kMeta;
        float2 y[2][16];                                 // per head, of its slot pairs
        const float2 fh[2] = {make_float2(rs.x, rs.x), make_float2(rs.y, rs.y)};
        const float2 fl[2] = {make_float2(rs.x * 0.03125f, rs.x * 0.03125f), make_float2(rs.y * 0.03125f, rs.y * 0.03125f)};
        {
          float x[2][64];
          tmem_ld16x128x2(tmem + lanes + L::kTmemS, x[0], x[1]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kBarSFree));
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float4 ac = *reinterpret_cast<const float4*>(meta + (4 * j + quad) * 4);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const float2 hi = make_float2(x[g][4 * j], x[g][4 * j + 1]), lo = make_float2(x[g][4 * j + 2], x[g][4 * j + 3]);
              y[g][j] = fma2(fma2(hi, fh[g], mul2(lo, fl[g])), make_float2(ac.x, ac.y), make_float2(ac.z, ac.w));
            }
          }
        }
        // The groups' maxima.  m is set by a token's first block, raised where this
        // block's outran it.
        float u[2][4];                                   // u of the groups
        uint32_t unit_of[2];                             // the exponents of 2^(u - m)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int h = hq + 8 * g;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float t = fmaxf(y[g][4 * k].x, y[g][4 * k].y);
#pragma unroll
            for (int j = 4 * k + 1; j < 4 * k + 4; ++j) t = fmax3f(t, y[g][j].x, y[g][j].y);
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
            u[g][k] = ceilf(fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2)));
          }
          const float top = fmaxf(fmaxf(u[g][0], u[g][1]), fmaxf(u[g][2], u[g][3]));
          if (first) {
            if (lead) note->to[h] = top;
            m[g] = top;
          } else if (top > m[g] + kLag) {
            const float f = fast_exp2(m[g] - top);
            l[g] = mul2(l[g], make_float2(f, f));
            m[g] = top;
            if (lead) {
              note->to[h] = top;
              note->f[h] = f;
              atomicOr(&note->heads[h >> 5], 1u << (h & 31));
            }
          }
          // (Nothing yet: any unit will do.  A NaN becomes a factor of 1; its weight is NaN.)
          const float m0 = m[g] == -INFINITY ? 0.f : m[g];
          uint32_t units = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            u[g][k] = fmaxf(u[g][k], m0 - kDepth);
            units |= static_cast<uint32_t>(127 + static_cast<int>(u[g][k] - m0)) << (8 * k);
          }
          if (lead) note->units[h] = units;
          unit_of[g] = units;
        }
        if (bad) note->failed = 1;
        if (lane == 0 && quarter == 0) {
          note->last = flags_of[st] & kLast;
          Note* next = notes + (e + 4) % kNotes;
          next->heads[0] = next->heads[1] = next->failed = 0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kBarNote + (e & 1)));
        // The weights, their part of l, and their two pieces.
        uint32_t out_hi[2][8], out_lo[2][8];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 shift2 = make_float2(-u[g][k], -u[g][k]);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 4 * k; j < 4 * k + 4; j += 2) {
              const float4 r = *reinterpret_cast<const float4*>(meta + 2 * kBlk + (j / 2) * 16 + quad * 4);
              const float2 d01 = add2(y[g][j], shift2), d23 = add2(y[g][j + 1], shift2);
              const float2 w01 = make_float2(fast_exp2(d01.x), fast_exp2(d01.y));
              const float2 w23 = make_float2(fast_exp2(d23.x), fast_exp2(d23.y));
              sum = fma2(w01, make_float2(r.x, r.y), sum);
              sum = fma2(w23, make_float2(r.z, r.w), sum);
              uint32_t hi, lo;                           // codes of slots 8j + 2 quad, + 1; + 8, + 9
              split_e4m3x4(w01, w23, hi, lo);
              // Lanes of a pair trade, the even one for four slots in a row at
              // 8j, the odd one at 8j + 8.
              const uint32_t got = __shfl_xor_sync(0xffffffffu, __byte_perm(hi, lo, sel_send), 1);
              out_hi[g][j / 2] = __byte_perm(hi, got, sel_hi);
              out_lo[g][j / 2] = __byte_perm(lo, got, sel_lo);
            }
            const float f = __uint_as_float(((unit_of[g] >> (8 * k)) & 0xffu) << 23);
            l[g] = fma2(sum, make_float2(f, f), l[g]);
          }
        }
        wait_note();
        if (*reinterpret_cast<volatile int*>(&note->failed) != 0) {
          run = false;
          break;
        }
        last = note->last != 0;
        const unsigned raised[2] = {*reinterpret_cast<volatile unsigned*>(&note->heads[0]),
                                    *reinterpret_cast<volatile unsigned*>(&note->heads[1])};
        // P and O are this thread's once the previous block's products are done.
        if (e > 0 && !done_with(e - 1)) bad = true;
        __syncwarp();
        tc_fence_after();
        {                                                // the heads' factors, in every lane quarter
          const uint32_t f0 = note->units[lane], f1 = note->units[32 + lane];
          tmem_st4u(tmem + lanes + L::kTmemFHi, f0, f1, f0 - kFineSteps, f1 - kFineSteps);
        }
        if (raised[0] | raised[1]) {                     // O of these heads, rescaled
          const uint32_t o = tmem + lanes + L::kTmemO;
          // A column at a time, few as they mostly are: a second form for many heads at
          // once cost every call 1 to 2 % by its size alone.
#pragma unroll
          for (int u = 0; u < 2; ++u)
            for (unsigned some = raised[u]; some != 0; some &= some - 1) {
              const int h = 32 * u + __ffs(some) - 1;
              const float f = note->f[h];
              float v[L::kChunks];
              tmem_ld1xn<L::kChunks, kHeads>(o + h, v);
#pragma unroll
              for (int c = 0; c < L::kChunks; ++c) tmem_st1(o + c * kHeads + h, v[c] * f);
            }
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int h = hq + 8 * g;
          const uint32_t row = base + L::kOffP + static_cast<uint32_t>(h) * 128u + (lane & 1) * 8u + (quad >> 1) * 4u;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t at = row + ((static_cast<uint32_t>(j) ^ static_cast<uint32_t>(h & 7)) << 4);
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(out_hi[g][j]) : "memory");
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + L::kPieceBytes), "r"(out_lo[g][j]) : "memory");
          }
        }
        tmem_wait_st();
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kBarPFull));
      }
      if (!run) break;

      // On to the next token, once the last products are done.
      done = t;
      if (left > 0) {
        for (++t; !live_token(p, next_req); next_req = load(p.token_req + t)) ++t;
        nb = blocks_of(p, t, next_req);
        b = 0;
        q.fetch(p, t, h0, heads, quarter, half, lane);
      }
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float sum = l[g].x + l[g].y;
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (lead) {
          head_sum[half * kHeads + hq + 8 * g] = sum;
          if (half == 0) head_end[hq + 8 * g] = m[g];
        }
      }
      if (!done_with(e - 1)) bad = true;
      __syncwarp();
      bar_sync(1, kSoftmaxThreads);
      tc_fence_after();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// Joins the parts of a token that several CTAs hold: a block per CTA whose range
// a token starts in and leaves and per 4 heads; a thread takes one column of
// every 128 for the four heads, lane i of every warp also m and l of part i,
// which weighs 2^(m_i - top).  Bound by latency: whose token and how many parts
// is one trip to L2, m, l and the first kAhead parts of O together the second.
// Small blocks with many loads each: with four times larger ones, each warp with
// all the reductions for a quarter of the columns, a call whose 152 CTAs all leave
// parts took 16 us longer.  It adds 5.6 us to a lone token's 12 (H=128 D=512
// topk=2048), 10 to 93 where all 152 CTAs leave parts (16 dense tokens of up to
// 32768 positions).
constexpr int kJoinHeads = 4;

template <int D, int kAhead>
__global__ void __launch_bounds__(D < 128 ? D : 128) smqa_paged_join_kernel(const PagedFwdParams p, int ctas) {
  constexpr int kChunks = D < 128 ? 1 : D / 128;
  grid_dependency_wait();
  const int groups = (p.H + kHeads - 1) / kHeads;
  const int cta = blockIdx.x / (kHeads / kJoinHeads), hg = blockIdx.x % (kHeads / kJoinHeads);
  const int h0 = (cta % groups) * kHeads;
  const int lane = threadIdx.x & 31;
  const int4* left = reinterpret_cast<const int4*>(p.ws);  // Leftover
  const float* parts = reinterpret_cast<const float*>(p.ws + kLeftoverBytes);
  auto part = [&](int c) { return parts + (static_cast<int64_t>(c) * 2 + (c == cta ? 1 : 0)) * part_floats(D); };
  // 32 CTAs at a time: this one and those behind it that hold the rest, up to
  // the first whose range the token does not leave.  An empty range in between
  // holds nothing.
  int tok = -1;
  auto chain = [&](int c0, bool& more) -> unsigned {
    const int c = c0 + lane * groups;
    const int4 x = c < ctas ? __ldcg(left + c) : make_int4(-1, 0, -1, 0);
    if (c0 == cta) tok = __shfl_sync(0xffffffffu, x.z, 0);
    const bool head = c != cta && x.x == tok;
    const unsigned ends = __ballot_sync(0xffffffffu, head && !x.y);
    more = ends == 0 && c0 + 32 * groups < ctas;
    return __ballot_sync(0xffffffffu, head || c == cta) & (ends == 0 ? 0xffffffffu : (2u << (__ffs(ends) - 1)) - 1u);
  };
  const int hb = hg * kJoinHeads;
  const int heads = min(kJoinHeads, p.H - h0 - hb);
  if (heads <= 0) return;
  bool more;
  unsigned held = chain(cta, more);
  if (tok < 0) return;
  float top[kJoinHeads], total[kJoinHeads], o[kChunks][kJoinHeads] = {};
#pragma unroll
  for (int h = 0; h < kJoinHeads; ++h) {
    top[h] = h < heads ? load(p.sink + h0 + hb + h) * 1.4426950408889634f : 0.f;
    total[h] = top[h] == -INFINITY ? 0.f : 1.f;
  }
  for (int c0 = cta;;) {
    const int c = c0 + lane * groups;
    float4 m = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY), l = make_float4(0.f, 0.f, 0.f, 0.f);
    if ((held >> lane) & 1u) {
      m = __ldcg(reinterpret_cast<const float4*>(part(c) + part_o(D) + hb));
      l = __ldcg(reinterpret_cast<const float4*>(part(c) + part_o(D) + kHeads + hb));
    }
    float4 v[kAhead][kChunks];
    int who[kAhead];
    auto load = [&] {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        who[i] = held != 0 ? __ffs(held) - 1 : -1;
        held &= held - 1;
        if (who[i] >= 0) {
          const float4* src = reinterpret_cast<const float4*>(part(c0 + who[i] * groups)) + hg * 128 + threadIdx.x;
#pragma unroll
          for (int k = 0; k < kChunks; ++k) v[i][k] = __ldcg(src + k * (kHeads / kJoinHeads) * 128);
        }
      }
    };
    load();
    const float ms[kJoinHeads] = {m.x, m.y, m.z, m.w}, ls[kJoinHeads] = {l.x, l.y, l.z, l.w};
    float f[kJoinHeads];
#pragma unroll
    for (int h = 0; h < kJoinHeads; ++h) {
      float t = ms[h];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off));
      t = fmaxf(t, top[h]);
      const float back = top[h] == -INFINITY ? 0.f : exp2f(top[h] - t);  // what came before, under the new maximum
      f[h] = t == -INFINITY ? 0.f : exp2f(ms[h] - t);
      top[h] = t;
      float u = ls[h] * f[h];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) u += __shfl_xor_sync(0xffffffffu, u, off);
      total[h] = fmaf(total[h], back, u);
#pragma unroll
      for (int k = 0; k < kChunks; ++k) o[k][h] *= back;
    }
    while (true) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (who[i] < 0) break;
        float w[kJoinHeads];
#pragma unroll
        for (int h = 0; h < kJoinHeads; ++h) w[h] = __shfl_sync(0xffffffffu, f[h], who[i]);
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          o[k][0] = fmaf(v[i][k].x, w[0], o[k][0]);
          o[k][1] = fmaf(v[i][k].y, w[1], o[k][1]);
          o[k][2] = fmaf(v[i][k].z, w[2], o[k][2]);
          o[k][3] = fmaf(v[i][k].w, w[3], o[k][3]);
        }
      }
      if (held == 0) break;
      load();
    }
    if (!more) break;
    c0 += 32 * groups;
    held = chain(c0, more);
  }
#pragma unroll
  for (int h = 0; h < kJoinHeads; ++h) {
    if (h >= heads) break;
    const int64_t row = static_cast<int64_t>(tok) * p.H + h0 + hb + h;
    const float inv = total[h] == 0.f ? 0.f : kCodeUnit / total[h];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) p.o[row * D + k * 128 + threadIdx.x] = __float2bfloat16(o[k][h] * inv);
    if (threadIdx.x == 0) p.lse[row] = total[h] == 0.f ? -INFINITY : log2f(total[h]) + top[h];
  }
}

// The most blocks a token can have (one: no token is ever split).
int64_t blocks_per_token(const smqa_paged_shape& s) {
  const int64_t slots = s.topk > 0 ? s.topk : static_cast<int64_t>(s.max_pages) * s.page_size;
  return (slots + kBlk - 1) / kBlk;
}
// Whether ranges are whole tokens (index lists: all tokens have the same number
// of blocks).  Splitting tokens evens the ranges out but costs the joining kernel,
// two blocks' time for a lone token, and a read-out and a Q more for the ranges
// that hold parts of two tokens, the more the nearer the tokens are to the ranges
// in number: up to 12 blocks' time (D = 64: 7).  GPU times, whole and split, in us:
//   T=1   H=128 D=512: topk=256 12.4 15.3, 512 16.2 15.9, 1024 22.8 16.7, 1536 29.5 17.4
//   T=8   H=128 D=512: topk=512 16.3 18.5, 1024 22.8 22.1, 1536 29.7 24.3
//   T=32  H=128 D=512: topk=1024 23.2 32.2, 1536 30.1 36.1, 2048 37.0 40.6
//   T=32  H=64  D=512: topk=1024 22.9 23.7, 1536 29.7 25.5
//   T=32  H=128 D=64:  topk=1024 17.1 19.5, 1536 22.6 22.1, 2048 28.2 24.9
//   T=100 H=128 D=512: topk=1024 44.6 55.1, 2048 73.5 75.2
//   T=128 H=128 D=64:  topk=2048 54.0 56.4, 4096 98.7 93.8
bool whole_tokens(const smqa_paged_shape& s) {
  if (s.topk == 0) return blocks_per_token(s) <= 1;
  const int groups = (s.H + kHeads - 1) / kHeads;
  const int64_t parts = kSMs / groups, T = s.T, nb = blocks_per_token(s);
  const int64_t spare = std::min<int64_t>(2 + 24 * T / parts, s.D == 512 ? 12 : 7);
  return (T + parts - 1) / parts * nb <= std::max<int64_t>(T * nb / parts, 1) + spare;
}
// CTAs of a call: per head group, as many ranges as SMs (or as the tokens can
// have blocks).
int ranges_of(const smqa_paged_shape& s) {
  const int groups = (s.H + kHeads - 1) / kHeads;
  const int64_t most = whole_tokens(s) ? s.T : s.T * blocks_per_token(s);
  return static_cast<int>(std::min<int64_t>(kSMs / groups, std::max<int64_t>(most, 1)));
}

template <int D>
cudaError_t launch(const PagedFwdParams& p, int ctas, cudaStream_t stream) {
  using L = PagedLayout<D>;
  // A split of registers above what the block is launched with would wait for
  // ever: refuse to launch a kernel that was not built with 128 a thread.  (Asked
  // until it has been answered.)
  static std::atomic<bool> built{false};
  cudaError_t e;
  if (!built.load(std::memory_order_relaxed)) {
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, smqa_paged_fwd_kernel<D>);
    if (e != cudaSuccess) return e;
    if (a.numRegs * kThreads < 2 * 128 * (kSoftmaxRegs + kOtherRegs)) return cudaErrorInvalidConfiguration;
    built.store(true, std::memory_order_relaxed);
  }
  static std::atomic<uint64_t> allowed{0};
  e = allow_smem(reinterpret_cast<const void*>(smqa_paged_fwd_kernel<D>), L::kSmem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, smqa_paged_fwd_kernel<D>, p);
  if (e != cudaSuccess || p.whole_tokens) return e;  // nothing to join
  // How many parts a thread asks for at once: a lone token's are many (32: 8 ahead
  // 19.4 us, 2 ahead 22.3, H=64 topk=4096; 16: 17.3 and 18.5); where all CTAs leave
  // parts a token has few, and more blocks fit an SM with fewer registers each (8
  // tokens of topk=1024, 128 CTAs: 24.7 and 23.0 us; 16 dense ones, 152: 105.6, 102.4).
  const bool few = ctas <= 64;
  cfg.gridDim = dim3(static_cast<unsigned>(ctas) * (kHeads / kJoinHeads));
  cfg.blockDim = dim3(D < 128 ? D : 128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, few ? smqa_paged_join_kernel<D, 8> : smqa_paged_join_kernel<D, 2>, p, ctas);
}

}  // namespace

size_t paged_fwd_workspace(const smqa_paged_shape& s) {
  const int groups = (s.H + kHeads - 1) / kHeads;
  static_assert(kSMs <= kMaxCtas, "a leftover per CTA");
  if (whole_tokens(s)) return 0;
  return kLeftoverBytes + static_cast<size_t>(ranges_of(s)) * groups * 2 * part_floats(s.D) * sizeof(float);
}

cudaError_t launch_paged_fwd(const PagedFwdParams& p, const smqa_paged_shape& s, cudaStream_t stream) {
  const int ctas = ranges_of(s) * ((s.H + kHeads - 1) / kHeads);
  PagedFwdParams q = p;
  q.whole_tokens = whole_tokens(s) ? 1 : 0;
  return p.D == 512 ? launch<512>(q, ctas, stream) : launch<64>(q, ctas, stream);
}

}  // namespace smqa

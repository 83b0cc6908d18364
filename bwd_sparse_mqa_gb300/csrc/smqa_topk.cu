// smqa_topk.cu -- the indexer's selection on sm_103a: which blocks of positions a
// token attends to, and the argument checks of its two forms (contiguous keys, and
// the 8-bit paged cache).
//
// The choice is that of the scores in real numbers, ties to the lowest position, so
// that it does not depend on how a batch is cut or summed.  The score kernel's values
// are off by E at most; with T the k-th largest of them, a block above T + 2E is
// chosen and one below T - 2E is not.  The few between are scored again by sums of 16
// products, added in pairs of fp32 numbers, whose error is a fraction of E, and those
// that are still open with each product (exact in fp32, as those of bf16 and e4m3
// numbers are) added with its rounding error kept in a second sum (two-sum).  That sum is
// fp32, of eight errors of 2^-24 of their chain each: the last values are off by 2^-41 of
// sum_h |w_h||q_h||k| at most.
//
// E = K sum_h |w_h| (c |q_h| + rho_h), K the largest length of a key row that the
// token sees.  The tensor core drops from every product what lies 2^24 below the
// largest term of its step, and no term or partial sum exceeds |q||k|: D products and
// 16 step sums, c = (D + 16) 2^-24 (measured: up to 2^-18.5 |q||k| at D = 128, one large
// product beside 127 small ones).  With two e4m3 pieces of q the sums of the small
// pieces, up to 2^-4 |q||k|, come first: D / 16 more.  The sum
// over heads adds (H/4 + 4) 2^-24; rho_h is what two e4m3 pieces leave of a query row
// (0 with bf16 keys).
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdio>
#include <type_traits>

#include "smqa_topk.cuh"

namespace smqa {

namespace {

constexpr int kBins = 2048;
constexpr int kList = 512;                               // (of which 509 are used: nth_of)
constexpr int32_t kKeyNegInf = -kKeyInf - 1;            // (key_of(-infinity): the bits 0xff800000 but for the sign flipped)

// A CTA of NT threads takes a token; of up to kCap candidates it keeps the bins of their
// scores in shared memory.
template <int D, int NT>
struct SelLayout {
  static constexpr int kWarps = NT / 32;
  static constexpr int kCap = NT == 1024 ? 65536 : 16384;
  static constexpr int kBatch = NT == 1024 ? 32 : 16;    // key rows that are scored again together, at most
  static constexpr int kPitch = D * 2 + 16;              // of a staged key row, bf16 (eight rows: other banks)
  static constexpr uint32_t kPartBytes = NT == 1024 ? 16384 : 8192;
  static constexpr uint32_t kOffHist = 0;                // int [kBins]; in its place the parts of scores
  static constexpr uint32_t kOffVal = kPartBytes;        // int64 [kList], or two int [kList]
  static constexpr uint32_t kOffIdx = kOffVal + kList * 8;    // int [kList]: candidates of a border
  static constexpr uint32_t kOffOpen = kOffIdx + kList * 4;   // int [kList]: places in idx
  static constexpr uint32_t kOffMark = kOffOpen + kList * 4;  // int [kList]: whether idx[i] is chosen
  static constexpr uint32_t kOffRow = kOffMark + kList * 4;   // bf16 [kBatch][D], padded
  static constexpr uint32_t kOffScale = kOffRow + kBatch * kPitch;  // float [kBatch]
  static constexpr uint32_t kOffW = kOffScale + kBatch * 4;   // float [128]
  static constexpr uint32_t kOffLen = kOffW + 128 * 4;        // float [128]: lengths of the query rows
  static constexpr uint32_t kOffRed = kOffLen + 128 * 4;      // int [8][kWarps]
  static constexpr uint32_t kOffMore = kOffRed + 8 * kWarps * 4;  // int [kWarps]
  static constexpr uint32_t kOffMisc = kOffMore + kWarps * 4;
  static constexpr uint32_t kOffBins = kOffMisc + 64;    // uint16 [kCap]
  static constexpr uint32_t kOffQ = kOffBins + kCap * 2;  // bf16 [H][D], 16-byte pieces c at c ^ (h mod 8)
  static constexpr uint32_t bytes(int H) { return kOffQ + static_cast<uint32_t>(H) * D * 2; }
};
static_assert(SelLayout<128, 1024>::bytes(128) <= 232448, "shared memory budget");
static_assert(3 * (SelLayout<128, 256>::bytes(64) + 1024) <= 233472, "three CTAs per SM");

__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, make_float2(-1.f, -1.f), a); }

// A value as two fp32 numbers, hi its nearest one and lo the rest (some 48 bits; fp64
// would take 20 times as long here).
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair sum_of(float a, float b) {  // exactly
  const float s = __fadd_rn(a, b), back = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, back)), __fsub_rn(b, back))};
}
__device__ __forceinline__ Pair normal(float a, float b) {  // |a| >= |b|, or a = 0
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = sum_of(a.hi, b.hi);
  return normal(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Pair times(Pair a, float f) {
  const float x = __fmul_rn(a.hi, f);
  return normal(x, fmaf(a.lo, f, fmaf(a.hi, f, -x)));
}
// Pairs as integers that order like them (not of a NaN).
__device__ __forceinline__ long long key64_of(Pair x) {
  return (static_cast<long long>(key_of(x.hi)) << 32) |
         (static_cast<uint32_t>(key_of(x.lo)) ^ 0x80000000u);
}
__device__ __forceinline__ double value64_of(long long k) {
  return static_cast<double>(value_of(static_cast<int32_t>(k >> 32))) +
         value_of(static_cast<int32_t>(static_cast<uint32_t>(k) ^ 0x80000000u));
}

// (By name where a function of its own needs it: through a pointer that it was given, the
// compiler could not tell that this is shared memory.)
__device__ __forceinline__ uint8_t* dynamic_smem() {
  extern __shared__ __align__(16) uint8_t select_smem[];
  return select_smem;
}

// What a CTA knows of its token.
template <int D, bool kPaged, int NT>
struct Token {
  using L = SelLayout<D, NT>;
  const TopkParams& p;
  uint8_t* smem;
  int64_t t;
  int n, req;
  int tid, warp, lane;
  float e_score, e_plain;                                // error bounds of the score kernel's values, of plain ones
  float longest;                                         // bound of the key rows' lengths

  template <typename T>
  __device__ __forceinline__ T* at(uint32_t off) const {
    return reinterpret_cast<T*>(smem + off);
  }
  // Over the CTA, the same in all threads: with kEnds the least of v[0] and the largest
  // of v[1], and the sums of the others.
  template <int N, bool kEnds>
  __device__ __forceinline__ void reduce(int (&v)[N]) {
    static_assert(N <= 8, "room for eight values");
    int* red = at<int>(L::kOffRed);
    auto over_warp = [](int i, int x) {
      return kEnds && i == 0   ? __reduce_min_sync(0xffffffffu, x)
             : kEnds && i == 1 ? __reduce_max_sync(0xffffffffu, x)
                               : __reduce_add_sync(0xffffffffu, x);
    };
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = over_warp(i, v[i]);
      if (lane == 0) red[i * L::kWarps + warp] = x;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = lane < L::kWarps ? red[i * L::kWarps + lane] : kEnds && i == 0 ? INT32_MAX : kEnds && i == 1 ? INT32_MIN : 0;
      v[i] = over_warp(i, x);
    }
    __syncthreads();
  }

  __device__ __forceinline__ int page_of(int j) const {  // (-1: none)
    const int pg = load(p.table + static_cast<int64_t>(req) * p.max_pages + (j >> p.page_shift));
    return static_cast<unsigned>(pg) < static_cast<unsigned>(p.n_pages) ? pg : -1;
  }
  // Starts the copies of the queries into shared memory.
  __device__ __forceinline__ void start_queries() const {
    constexpr int kPer = D / 8;
    const __nv_bfloat16* q = p.q + t * p.H * D;
    const uint32_t to = smem_u32(smem) + L::kOffQ;
    for (int i = tid; i < p.H * kPer; i += NT) {
      const int h = i / kPer, c = i % kPer;
      cp_async_16(to + (h * kPer + (c ^ (h & 7))) * 16, q + static_cast<int64_t>(i) * 8);
    }
    if (tid < p.H) at<float>(L::kOffW)[tid] = load(p.w + t * p.H + tid);
  }
  // Once they are there: the error bounds.  D / 8 threads share a head.
  __device__ __forceinline__ void bounds() {
    cp_async_wait_all();
    __syncthreads();
    constexpr int kPer = D / 8, kHeads = NT / kPer;
    const int c = tid % kPer;
    float len = 0.f, rest = 0.f;
#pragma unroll 2
    for (int h0 = 0; h0 < p.H; h0 += kHeads) {
      const int h = h0 + tid / kPer;
      const bool there = h < p.H;
      const uint4 v = there ? at<uint4>(L::kOffQ)[h * kPer + (c ^ (h & 7))] : make_uint4(0, 0, 0, 0);
      const float w = there ? at<float>(L::kOffW)[h] : 0.f;
      // In units that make a row's largest value 2^7 to 2^8, as the score kernel has them.
      uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
      m = max(m & 0xffffu, m >> 16);
#pragma unroll
      for (int off = 1; off < kPer; off <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
      const int k = query_exponent(m);
      const float f = pow2f(k);
      const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
      float sq = 0.f, sr = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = make_float2(__uint_as_float(w4[i] << 16) * f, __uint_as_float(w4[i] & 0xffff0000u) * f);
        sq = fmaf(y.x, y.x, fmaf(y.y, y.y, sq));
        if constexpr (kPaged) {
          uint16_t hi, lo;
          split_query(y, hi, lo);
          const float2 a = e4m3x2_value(hi), b = e4m3x2_value(lo);
          const float dx = y.x - a.x - b.x, dy = y.y - a.y - b.y;
          sr = fmaf(dx, dx, fmaf(dy, dy, sr));
        }
      }
#pragma unroll
      for (int off = 1; off < kPer; off <<= 1) {
        sq += __shfl_xor_sync(0xffffffffu, sq, off);
        if constexpr (kPaged) sr += __shfl_xor_sync(0xffffffffu, sr, off);
      }
      // (What fp32 or the tensor core may lose of a weight below 2^-126 or of a query element below
      // that: the weight counts as 2^-126 at least, the row's length as 2^-88 more, and a sum over
      // heads that are not 0 is not 0.)
      const float wa = c == 0 && w != 0.f && m != 0 ? fmaxf(fabsf(w), 0x1p-126f) : 0.f, wh = wa * pow2f(-k);
      if (there && c == 0) at<float>(L::kOffLen)[h] = 1.01f * sqrtf(sq) * pow2f(-k);
      len = fmaf(wh, sqrtf(sq), fmaf(wa, 0x1p-88f, wa > 0.f ? len + 0x1p-126f : len));
      rest = kPaged ? fmaf(wh, sqrtf(sr), rest) : rest + wa;
    }
    // The longest row of the tiles that the token sees.
    const int tiles = 4 * ((n + kTile - 1) / kTile);     // (a bound per 32 rows)
    const float* norms = p.norms + (kPaged ? t - p.tok0 : static_cast<int64_t>(req)) * p.norm_ld;
    float top = 0.f;
    for (int i = tid; i < tiles; i += NT) top = fmaxf(top, load(norms + i));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      len += __shfl_xor_sync(0xffffffffu, len, off);
      rest += __shfl_xor_sync(0xffffffffu, rest, off);
    }
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    float* red = at<float>(L::kOffRed);
    if (lane == 0) {
      red[warp] = len;
      red[L::kWarps + warp] = rest;
      red[2 * L::kWarps + warp] = top;
    }
    __syncthreads();
    len = lane < L::kWarps ? red[lane] : 0.f;
    rest = lane < L::kWarps ? red[L::kWarps + lane] : 0.f;
    top = lane < L::kWarps ? red[2 * L::kWarps + lane] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      len += __shfl_xor_sync(0xffffffffu, len, off);
      rest += __shfl_xor_sync(0xffffffffu, rest, off);
    }
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    __syncthreads();
    // (1.01 for the rounding of these sums.  What underflows, with bf16 keys: D products, of which the
    // tensor core may take those below 2^-126 for 0, and key elements, as 2^-100 more of length; with
    // e4m3 keys: 2^-150 of a head's weight, times 2^12 |k|.  Only where all weights and queries or
    // all key rows are 0, all scores are exactly 0.)
    const float c_score = (static_cast<float>(kPaged ? D + D / 16 + 17 : D + 16) + static_cast<float>(p.H) * 0.25f + 4.f) * 0x1p-24f;
    const float tiny = (kPaged ? top * 0x1p-110f : rest * 0x1p-116f) + 0x1p-140f;
    const bool zero = len == 0.f || top == 0.f;
    longest = kPaged ? top : top + 0x1p-100f;
    e_score = zero ? 0.f : 1.01f * longest * (kPaged ? len * c_score + rest : len * c_score) + tiny;
    if (!(e_score < INFINITY)) e_score = INFINITY;
    // Plain values: 16 products and their sum (2^-23 of it), and a rounding of the score.
    e_plain = zero ? 0.f : 1.01f * longest * len * (20.f * 0x1p-24f) + tiny;
    if (!(e_plain < INFINITY)) e_plain = INFINITY;
  }

  // Whether position j's score is exactly 0: its key row is 0, or every logit lies below 0
  // by more than the error of its fp32 sum (D / 8 products in a row, then four adds).  By
  // one thread: the row's bytes from the caches, the queries the same for all lanes.
  __device__ __forceinline__ bool surely_zero(int j) const {
    uint4 k[kPaged ? D / 16 : D / 8];
    if constexpr (kPaged) {
      const int pg = page_of(j);
      if (pg < 0) return false;
      const uint4* src = reinterpret_cast<const uint4*>(p.codes + ((static_cast<int64_t>(pg) << p.page_shift) + (j & ((1 << p.page_shift) - 1))) * D);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) k[c] = load(src + c);
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(p.k + (static_cast<int64_t>(req) * p.S_kv + j) * D);
#pragma unroll
      for (int c = 0; c < D / 8; ++c) k[c] = load(src + c);
    }
    constexpr uint32_t kMagnitudes = kPaged ? 0x7f7f7f7fu : 0x7fff7fffu;
    uint32_t any = 0;
#pragma unroll
    for (int c = 0; c < (kPaged ? D / 16 : D / 8); ++c) any |= (k[c].x | k[c].y | k[c].z | k[c].w) & kMagnitudes;
    if (any == 0) return true;
    // (Paged: the bound's lengths are scaled, the codes are not.)
    float scale = 1.f;
    if constexpr (kPaged) scale = load(p.scales + page_of(j));
    for (int h = 0; h < p.H; ++h) {
      const uint4* q = at<uint4>(L::kOffQ) + h * (D / 8);
      float2 s[4] = {};
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint4 v = q[c ^ (h & 7)];
        const uint32_t q4[4] = {v.x, v.y, v.z, v.w};
        float2 kk[4];
        if constexpr (kPaged) {
          const uint32_t lo = (c & 1) ? k[c / 2].z : k[c / 2].x, hi = (c & 1) ? k[c / 2].w : k[c / 2].y;
          kk[0] = e4m3x2_value(static_cast<uint16_t>(lo));
          kk[1] = e4m3x2_value(static_cast<uint16_t>(lo >> 16));
          kk[2] = e4m3x2_value(static_cast<uint16_t>(hi));
          kk[3] = e4m3x2_value(static_cast<uint16_t>(hi >> 16));
        } else {
          const uint32_t w4[4] = {k[c].x, k[c].y, k[c].z, k[c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) kk[i] = make_float2(__uint_as_float(w4[i] << 16), __uint_as_float(w4[i] & 0xffff0000u));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = fma2(make_float2(__uint_as_float(q4[i] << 16), __uint_as_float(q4[i] & 0xffff0000u)), kk[i], s[i]);
      }
      const float2 sum = add2(add2(s[0], s[1]), add2(s[2], s[3]));
      const float bound = longest * (at<float>(L::kOffLen)[h] + 0x1p-126f) * (static_cast<float>(D / 8 + 4) * 0x1p-24f) + 0x1p-140f;
      if (!((sum.x + sum.y) * scale < -bound)) return false;
    }
    return true;
  }

  // Scores of the rows of candidates (blocks) cand(0 .. m - 1) once more, plain or exact:
  // put(i, value) for every row that is there, by one lane each.  A batch of rows is
  // staged as bf16 (which holds an e4m3 number).  Of larger blocks, exact scores only of
  // rows whose plain one is `floor` or more.
  template <bool kExact, typename Cand, typename Put>
  __device__ __forceinline__ void score(Cand cand, int m, float floor, Put put) {
    // (Copies: a call's parameters behind a pointer would be loaded again after every store.)
    const int H = p.H, shift = p.block_shift, page_shift = p.page_shift, n_pages = p.n_pages, seen = n;
    const int32_t* table = kPaged ? p.table + static_cast<int64_t>(req) * p.max_pages : nullptr;
    const uint8_t* codes = p.codes;
    const float* page_scales = p.scales;
    const __nv_bfloat16* keys = kPaged ? nullptr : p.k + static_cast<int64_t>(req) * p.S_kv * D;
    const int bs = 1 << shift, total = m << shift;
    float* scale = at<float>(L::kOffScale);
    // Exact: a warp has 32 elements of a row, its lanes 32 heads (or, with few heads, the
    // heads of several rows).
    constexpr int kParts = D / 32;
    int nh = 1;
    while (nh < H && nh < 32) nh <<= 1;
    const int groups = (H + 31) / 32, heads = groups > 1 ? 32 * groups : nh, together = 32 / nh;
    const int units = groups * kParts, slots = max(1, L::kWarps / units), slot = warp / units;
    const int batch = kExact ? min(L::kBatch, static_cast<int>(L::kPartBytes / 8) / (kParts * heads)) : L::kBatch;
    for (int b0 = 0; b0 < total; b0 += batch) {
      const int rows = min(batch, total - b0);
      for (int r = warp; r < rows; r += L::kWarps) {
        const int j = (cand((b0 + r) >> shift) << shift) + ((b0 + r) & (bs - 1));
        uint32_t* to = reinterpret_cast<uint32_t*>(smem + L::kOffRow + r * L::kPitch);
        float s = -1.f;
        if (j < seen) {
          if constexpr (kPaged) {
            const int pg = load(table + (j >> page_shift));
            if (static_cast<unsigned>(pg) < static_cast<unsigned>(n_pages)) {
              const uint8_t* src = codes + ((static_cast<int64_t>(pg) << page_shift) + (j & ((1 << page_shift) - 1))) * D;
              s = load(page_scales + pg);
#pragma unroll
              for (int i = 0; i < D / 64; ++i) {
                uint16_t v;
                asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(src + (i * 32 + lane) * 2));
                const float2 x = e4m3x2_value(v);
                to[i * 32 + lane] = pack_bf16x2(x.x, x.y);
              }
            }
          } else {
            const int* src = reinterpret_cast<const int*>(keys + static_cast<int64_t>(j) * D);
            s = 1.f;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) to[i * 32 + lane] = static_cast<uint32_t>(load(src + i * 32 + lane));
          }
        }
        if (lane == 0) scale[r] = s;
      }
      __syncthreads();
      if (!kExact || shift > 0) {
        // Plain: 16 heads x 8 rows by a warp, 16 elements at a time into fresh sums of the
        // tensor core (a running sum would lose bits at every step); what follows is in pairs.
        const int mt = (H + 15) / 16, nt = (rows + 7) / 8;
        float2* part = at<float2>(L::kOffHist);          // [mt][kBatch]
        for (int u = warp; u < mt * nt; u += L::kWarps) {
          const int h0 = u % mt * 16, r0 = u / mt * 8;
          const int hl = min(h0 + (lane & 15), H - 1);
          const uint32_t qa = smem_u32(smem) + L::kOffQ + hl * (D * 2);
          const uint32_t* kr = reinterpret_cast<const uint32_t*>(smem + L::kOffRow + (r0 + (lane >> 2)) * L::kPitch) + (lane & 3);
          Pair sum[4] = {};
#pragma unroll 2
          for (int c = 0; c < D / 16; ++c) {
            uint32_t a0, a1, a2, a3;
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                         : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3)
                         : "r"(qa + (((2 * c + (lane >> 4)) ^ (hl & 7)) << 4))
                         : "memory");
            float d[4];
            asm volatile(
                "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                "{%10, %10, %10, %10};"
                : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(kr[8 * c]), "r"(kr[8 * c + 4]), "f"(0.f));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const Pair s = sum_of(sum[i].hi, d[i]);
              sum[i] = Pair{s.hi, sum[i].lo + s.lo};
            }
          }
          // Heads h0 + lane / 4 and 8 more, rows r0 + 2 (lane mod 4) and the next.
          const int ha = h0 + (lane >> 2), hb = ha + 8;
          // (A logit that is NaN or +infinity makes its row's sum one that is no number, which put leaves
          // out: such a row ranks below its block's others, or above, and its block is not here.)
          auto weighted = [&](Pair x, int h) {
            const Pair y = normal(x.hi, x.lo);
            return h < H && x.hi != -INFINITY && !(y.hi <= 0.f) ? times(y, at<float>(L::kOffW)[h]) : Pair{0.f, 0.f};
          };
          Pair x = add(weighted(sum[0], ha), weighted(sum[2], hb)), y = add(weighted(sum[1], ha), weighted(sum[3], hb));
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            x = add(x, Pair{__shfl_xor_sync(0xffffffffu, x.hi, off), __shfl_xor_sync(0xffffffffu, x.lo, off)});
            y = add(y, Pair{__shfl_xor_sync(0xffffffffu, y.hi, off), __shfl_xor_sync(0xffffffffu, y.lo, off)});
          }
          if (lane < 4) *reinterpret_cast<float4*>(part + u % mt * L::kBatch + r0 + 2 * lane) = make_float4(x.hi, x.lo, y.hi, y.lo);
        }
        __syncthreads();
        if (tid < rows && scale[tid] >= 0.f) {
          Pair sum{0.f, 0.f};
          for (int i = 0; i < mt; ++i) {
            const float2 x = part[i * L::kBatch + tid];
            sum = add(sum, Pair{x.x, x.y});
          }
          const float x = sum.hi * scale[tid];
          if constexpr (kExact) {
            if (x < floor) scale[tid] = -1.f;
          } else {
            put((b0 + tid) >> shift, x);
          }
        }
        __syncthreads();
      }
      if constexpr (kExact) {
        for (int u = warp % units; u < units && slot < slots; u += L::kWarps) {
          const int part = u % kParts, h = u / kParts * 32 + lane % nh, hq = min(h, H - 1);
          const uint4* qr = at<uint4>(L::kOffQ) + hq * (D / 8);
          for (int r0 = slot * together; r0 < rows; r0 += slots * together) {
            const int r = r0 + lane / nh;
            if (r >= rows || scale[r] < 0.f) continue;
            const uint4* kr = reinterpret_cast<const uint4*>(smem + L::kOffRow + r * L::kPitch) + part * 4;
            float2 s0 = {}, s1 = {}, e0 = {}, e1 = {};
            auto two_sum = [](float2& s, float2& err, float2 x) {
              const float2 sum = add2(s, x), back = sub2(sum, s);
              err = add2(err, add2(sub2(s, sub2(sum, back)), sub2(x, back)));
              s = sum;
            };
            auto pair = [](uint32_t v) { return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)); };
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              const uint4 q = qr[(part * 4 + i) ^ (hq & 7)], k = kr[i];
              two_sum(s0, e0, mul2(pair(q.x), pair(k.x)));
              two_sum(s1, e1, mul2(pair(q.y), pair(k.y)));
              two_sum(s0, e0, mul2(pair(q.z), pair(k.z)));
              two_sum(s1, e1, mul2(pair(q.w), pair(k.w)));
            }
            two_sum(s0, e0, s1);
            const Pair d = sum_of(s0.x, s0.y);
            const float2 e = add2(e0, e1);
            // (An infinity's error is no number.)
            at<float2>(L::kOffHist)[(r * kParts + part) * heads + h] =
                fabsf(d.hi) < INFINITY ? make_float2(d.hi, d.lo + (e.x + e.y)) : make_float2(d.hi, 0.f);
          }
        }
        __syncthreads();
        for (int r = warp; r < rows; r += L::kWarps) {
          if (scale[r] < 0.f) continue;
          Pair sum{0.f, 0.f};
          for (int h = lane; h < H; h += 32) {
            Pair d{0.f, 0.f};
            float all = 0.f;                             // (where it is -infinity, d is no number)
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
              const float2 x = at<float2>(L::kOffHist)[(r * kParts + i) * heads + h];
              d = add(d, Pair{x.x, x.y});
              all += x.x;
            }
            if (all != -INFINITY && !(d.hi <= 0.f)) sum = add(sum, times(d, at<float>(L::kOffW)[h]));
          }
#pragma unroll
          for (int off = 16; off > 0; off >>= 1)
            sum = add(sum, Pair{__shfl_xor_sync(0xffffffffu, sum.hi, off), __shfl_xor_sync(0xffffffffu, sum.lo, off)});
          if (lane == 0) put((b0 + r) >> shift, times(sum, scale[r]));
        }
        __syncthreads();
      }
    }
  }
};

// val[i] = the exact score of block idx[open[i]] (kOpen) or idx[i], as an ordered
// integer.  (A function of its own: one copy of the code.)
template <int D, bool kPaged, int NT, bool kOpen>
__device__ __noinline__ void exact_scores(Token<D, kPaged, NT> tk, int m, float floor) {
  using L = SelLayout<D, NT>;
  tk.smem = dynamic_smem();
  const int *idx = tk.template at<int>(L::kOffIdx), *open = tk.template at<int>(L::kOffOpen);
  long long* val = tk.template at<long long>(L::kOffVal);
  for (int i = tk.tid; i < m; i += NT) val[i] = key64_of(Pair{-INFINITY, 0.f});
  __syncthreads();
  tk.template score<true>([&](int i) { return idx[kOpen ? open[i] : i]; }, m, floor, [&](int i, Pair x) {
    if (x.hi == x.hi) atomicMax(val + i, key64_of(fabsf(x.hi) < INFINITY ? x : Pair{x.hi, 0.f}));
  });
}

// The candidates (blocks) of a token: their keys, in the token's row.  A warp has a run
// of them, lane by lane, in `steps` steps.
template <int D, bool kPaged, int NT>
struct Keys {
  using L = SelLayout<D, NT>;
  int32_t* row;
  int nb, per, entries, steps, c0, lane;

  __device__ __forceinline__ Keys(const Token<D, kPaged, NT>& tk) {
    const TopkParams& p = tk.p;
    const int eshift = entry_shift(p.block_shift);
    row = p.rows + (tk.t - p.tok0) * p.ld;
    nb = (tk.n + (1 << p.block_shift) - 1) >> p.block_shift;
    per = 1 << (p.block_shift - eshift);
    entries = (tk.n + (1 << eshift) - 1) >> eshift;
    const int run = ((nb + L::kWarps - 1) / L::kWarps + 63) & ~63;
    steps = run / 32;
    c0 = tk.warp * run;
    lane = tk.lane;
  }
  __device__ __forceinline__ int fetch(int c) const {    // (every load made, where it is not needed of another)
    int key = kKeyNever;
    for (int i = 0; i < per; ++i) key = max(key, load(row + min(c * per + i, entries - 1)));
    return c < nb ? key : kKeyNever;
  }
  __device__ __forceinline__ void store(int c, int key) const {  // (all of a block in its first entry)
    row[c * per] = key;
    for (int i = 1; i < per; ++i)
      if (c * per + i < entries) row[c * per + i] = kKeyNever;
  }
  // f(candidate, key) for all of the thread's, in order (the warp's lanes together).
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    constexpr int kAhead = 8;
    for (int i0 = 0; i0 < steps; i0 += kAhead) {
      int key[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) key[i] = per == 1 ? load(row + min(c0 + (i0 + i) * 32 + lane, nb - 1)) : 0;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int c = c0 + (i0 + i) * 32 + lane;
        if (i0 + i < steps) f(c, per != 1 ? fetch(c) : c < nb ? key[i] : kKeyNever);
      }
    }
  }
};

// What is chosen: keys above khi, and the first r candidates of [klo, khi].
struct Cut {
  int klo, khi, r;
};

// The keys of x - 2 e and x + 2 e, rounded outwards.
__device__ __forceinline__ void window(float x, float e, int& klo, int& khi) {
  const float lo = __fadd_rd(x, -2.f * e), hi = __fadd_ru(x, 2.f * e);
  klo = lo == lo ? key_of(lo) : kKeyNegInf;              // (infinities of opposite signs: everything)
  khi = hi == hi ? key_of(hi) : kKeyInf;
}

// The bin that holds number r from the top, how many lie above it, and in it, into
// misc[0..2]; 0 into misc[3].
template <int D, bool kPaged, int NT>
__device__ __forceinline__ void find_bin(Token<D, kPaged, NT>& tk, int r) {
  using L = SelLayout<D, NT>;
  const int* hist = tk.template at<int>(L::kOffHist);
  int *misc = tk.template at<int>(L::kOffMisc), *red = tk.template at<int>(L::kOffRed);
  constexpr int kPer = kBins / NT;                       // thread i: bins kBins - 1 - kPer i and those below
  int mine[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) sum += mine[i] = hist[kBins - 1 - kPer * tk.tid - i];
  int incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, off);
    if (tk.lane >= off) incl += x;
  }
  if (tk.lane == 31) red[tk.warp] = incl;
  if (tk.tid == 0) misc[3] = 0;
  __syncthreads();
  int above = incl - sum + __reduce_add_sync(0xffffffffu, tk.lane < tk.warp ? red[tk.lane] : 0);
  if (above < r && r <= above + sum) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (above < r && r <= above + mine[i]) {
        misc[0] = kBins - 1 - kPer * tk.tid - i;
        misc[1] = above;
        misc[2] = mine[i];
      }
      above += mine[i];
    }
  }
  __syncthreads();
}

// Of keys[0 .. m): number r from the largest.  (Room for three more.)
template <int D, bool kPaged, int NT>
__device__ __forceinline__ int nth_of(Token<D, kPaged, NT>& tk, int* keys, int m, int r) {
  int* misc = tk.template at<int>(SelLayout<D, NT>::kOffMisc);
  if (tk.tid < 3) keys[m + tk.tid] = INT32_MIN;          // (below every finite value's)
  __syncthreads();
  const int4* k4 = reinterpret_cast<const int4*>(keys);
  for (int i = tk.tid; i < m; i += NT) {
    const int v = keys[i];
    int more = 0, same = 0;
#pragma unroll 4
    for (int k = 0; k < (m + 3) / 4; ++k) {
      const int4 x = k4[k];
      more += (x.x > v) + (x.y > v) + (x.z > v) + (x.w > v);
      same += (x.x == v) + (x.y == v) + (x.z == v) + (x.w == v);
    }
    if (more < r && r <= more + same) misc[0] = v;
  }
  __syncthreads();
  const int found = misc[0];
  __syncthreads();
  return found;
}

// Of idx[0 .. m), r are to be chosen: mark[i] = 1 for those with the best exact scores,
// ties by number.  (Behind a barrier that all have passed since they last looked at misc[3]
// and at the lists.)
template <int D, bool kPaged, int NT>
__device__ __noinline__ void settle(Token<D, kPaged, NT> tk, int m, int r) {
  using L = SelLayout<D, NT>;
  tk.smem = dynamic_smem();
  int *misc = tk.template at<int>(L::kOffMisc), *idx = tk.template at<int>(L::kOffIdx), *open = tk.template at<int>(L::kOffOpen);
  int* mark = tk.template at<int>(L::kOffMark);
  long long* val = tk.template at<long long>(L::kOffVal);
  int* pk = reinterpret_cast<int*>(val);
  // By plain scores first.
  for (int i = tk.tid; i < m; i += NT) pk[i] = kKeyNegInf;
  if (tk.tid == 0) misc[3] = 0;
  __syncthreads();
  tk.template score<false>([&](int i) { return idx[i]; }, m, 0.f, [&](int i, float x) { if (x == x) atomicMax(pk + i, key_of(x)); });
  int klo, khi;
  const float at = value_of(nth_of(tk, pk, m, r));
  window(at, tk.e_plain, klo, khi);
  int cnt[1] = {0};
  for (int i = tk.tid; i < m; i += NT) {
    const int key = pk[i];
    mark[i] = key > khi;
    cnt[0] += key > khi;
    if (key >= klo && key <= khi) open[atomicAdd(misc + 3, 1)] = i;
  }
  tk.template reduce<1, false>(cnt);
  m = misc[3];
  r -= cnt[0];
  if (m == r) {
    for (int i = tk.tid; i < m; i += NT) mark[open[i]] = 1;
  } else {
    // (Their best rows' plain scores are at - 2 e_plain or more.)
    exact_scores<D, kPaged, NT, true>(tk, m, at - 4.f * tk.e_plain);
    for (int i = tk.tid; i < m; i += NT) {
      const long long x = val[i];
      const int c = idx[open[i]];
      int before = 0;
      for (int k = 0; k < m; ++k) before += val[k] > x || (val[k] == x && idx[open[k]] < c);
      mark[open[i]] = before < r;
    }
  }
  __syncthreads();
}

// The cut of any scores.  `level` 0: the score kernel's values.  Where more
// candidates than the list holds lie in the window, their exact scores less T take the
// values' place, off by a rounding of what is left (level 1), and so again (level 2:
// what is still equal ties).
template <int D, bool kPaged, int NT>
__device__ __forceinline__ Cut any_cut(Token<D, kPaged, NT>& tk, const Keys<D, kPaged, NT>& keys, int want) {
  using L = SelLayout<D, NT>;
  int *hist = tk.template at<int>(L::kOffHist), *misc = tk.template at<int>(L::kOffMisc), *idx = tk.template at<int>(L::kOffIdx);
  long long* val = tk.template at<long long>(L::kOffVal);
  double base = 0.;
  for (int level = 0;; ++level) {
    __syncthreads();
    int v[7] = {INT32_MAX, INT32_MIN, 0, 0, 0, 0, 0};    // finite: least, largest, number; >= inf; always; NaN; never
    keys.each([&](int c, int key) {
      if (key > kKeyNegInf && key < kKeyInf) {
        v[0] = min(v[0], key);
        v[1] = max(v[1], key);
        ++v[2];
      }
      v[3] += key >= kKeyInf;
      v[4] += key == kKeyAlways;
      v[5] += key == kKeyNan;
      v[6] += c < keys.nb && key == kKeyNever;
    });
    tk.template reduce<7, true>(v);
    if (keys.nb - v[6] <= want) return Cut{kKeyNever, kKeyNever, 0};  // all there are
    if (want <= v[4]) return Cut{kKeyAlways, kKeyAlways, want};
    if (want <= v[3]) return Cut{kKeyInf, kKeyInf, want - v[4]};
    if (want > v[3] + v[2]) {
      const int neg = keys.nb - v[6] - v[5] - v[3] - v[2], r = want - v[3] - v[2];
      return r <= neg ? Cut{kKeyNegInf, kKeyNegInf, r} : Cut{kKeyNan, kKeyNan, r - neg};
    }
    // Number r of the finite keys in [lo, hi].
    int lo = v[0], hi = v[1], r = want - v[3], at = lo;
    while (lo < hi) {
      // Linear in the value, or (a range that fp32 cannot hold) in the key.
      const float half = 0.5f * value_of(lo), range = 0.5f * value_of(hi) - half;
      const bool linear = range > 1e-30f && range < 1e38f;
      const float per = (kBins - 0.5f) / range;
      const int shift = max(0, 21 - __clz(static_cast<unsigned>(hi) - static_cast<unsigned>(lo)));
      auto bin_of = [&](int key) {
        return linear ? min(kBins - 1, static_cast<int>((0.5f * value_of(key) - half) * per))
                      : static_cast<int>((static_cast<unsigned>(key) - static_cast<unsigned>(lo)) >> shift);
      };
      for (int i = tk.tid; i < kBins; i += NT) hist[i] = 0;
      __syncthreads();
      keys.each([&](int, int key) {
        if (key >= lo && key <= hi) atomicAdd(hist + bin_of(key), 1);
      });
      __syncthreads();
      find_bin(tk, r);
      const int bin = misc[0], members = misc[2];
      r -= misc[1];
      if (members <= kList - 3) {
        keys.each([&](int, int key) {
          if (key >= lo && key <= hi && bin_of(key) == bin) idx[atomicAdd(misc + 3, 1)] = key;
        });
        __syncthreads();
        lo = hi = nth_of(tk, idx, members, r);
      } else {
        int ends[2] = {INT32_MAX, INT32_MIN};
        keys.each([&](int, int key) {
          if (key >= lo && key <= hi && bin_of(key) == bin) {
            ends[0] = min(ends[0], key);
            ends[1] = max(ends[1], key);
          }
        });
        tk.template reduce<2, true>(ends);
        lo = ends[0];
        hi = ends[1];
      }
      at = lo;
    }
    const float mid = value_of(at);
    const float e = level == 0 ? tk.e_score : level == 1 ? fmaxf(fabsf(value_of(v[0])), fabsf(value_of(v[1]))) * 0x1p-23f : 0.f;
    int klo, khi;
    window(mid, e, klo, khi);
    klo = max(klo, kKeyNegInf + 1);
    khi = min(khi, kKeyInf - 1);
    if (tk.tid == 0) misc[3] = 0;
    __syncthreads();
    int cnt[2] = {0, 0};
    keys.each([&](int c, int key) {
      cnt[0] += key > khi;
      if (key >= klo && key <= khi) {
        ++cnt[1];
        const int i = atomicAdd(misc + 3, 1);
        if (i < kList) idx[i] = c;
      }
    });
    tk.template reduce<2, false>(cnt);
    const int m = cnt[1];
    r = want - cnt[0];
    if (m == r || klo == khi) return Cut{klo, khi, r};
    if (m <= kList - 3) {
      settle(tk, m, r);
      const int* mark = tk.template at<int>(L::kOffMark);
      for (int i = tk.tid; i < m; i += NT) keys.store(idx[i], mark[i] ? kKeyAlways : kKeyNever);
      return Cut{khi, khi, 0};
    }
    // Many scores of exactly 0 (few heads, key rows of 0): those are settled without the
    // exact sums, and the few others of the window against them.
    if (level == 0 && tk.p.block_shift == 0) {
      __syncthreads();
      if (tk.tid == 0) misc[3] = 0;
      __syncthreads();
      int zeros = 0;
      for (int c = tk.tid; c < keys.nb; c += NT) {
        const int key = keys.fetch(c);
        if (key < klo || key > khi) {
          keys.store(c, key > khi ? kKeyAlways : kKeyNever);
        } else if (tk.surely_zero(c)) {
          ++zeros;
          keys.store(c, 0);
        } else {
          const int i = atomicAdd(misc + 3, 1);
          if (i < kList) idx[i] = c;
          if (key == 0) keys.store(c, khi != 0 ? khi : klo);  // (not a sure one; within the window)
        }
      }
      int n0[1] = {zeros};
      tk.template reduce<1, false>(n0);
      const int some = misc[3];
      if (n0[0] > 0 && some <= kList) {
        exact_scores<D, kPaged, NT, false>(tk, some, -INFINITY);
        const long long zero = key64_of(Pair{0.f, 0.f});
        int by[2] = {0, 0};                              // above 0, equal
        for (int i = tk.tid; i < some; i += NT) {
          by[0] += val[i] > zero;
          by[1] += val[i] == zero;
        }
        tk.template reduce<2, false>(by);
        const int ties = n0[0] + by[1];
        // Above 0 first, the zeros by number, below 0 last.
        for (int i = tk.tid; i < some; i += NT) {
          const long long x = val[i];
          const int c = idx[i];
          int before = x < zero ? ties : 0;
          for (int k = 0; k < some; ++k) before += val[k] != zero && (val[k] > x || (val[k] == x && idx[k] < c));
          keys.store(c, x == zero ? 0 : before < r ? kKeyAlways : kKeyNever);
        }
        return Cut{0, 0, max(0, min(r - by[0], ties))};
      }
    }
    // (base: of the values so far; the new ones' is T.)  As many candidates as the list
    // holds at a time.
    base += static_cast<double>(mid);
    for (int x0 = 0; x0 < keys.nb; x0 += kList) {
      __syncthreads();
      if (tk.tid == 0) misc[3] = 0;
      __syncthreads();
      for (int c = x0 + tk.tid; c < min(x0 + kList, keys.nb); c += NT) {
        const int key = keys.fetch(c);
        if (key >= klo && key <= khi) idx[atomicAdd(misc + 3, 1)] = c;
        else keys.store(c, key > khi ? kKeyAlways : kKeyNever);
      }
      __syncthreads();
      const int some = misc[3];
      exact_scores<D, kPaged, NT, false>(tk, some, -INFINITY);
      for (int i = tk.tid; i < some; i += NT) keys.store(idx[i], key_of(static_cast<float>(value64_of(val[i]) - base)));
    }
  }
}

// Rows of block c: those the token sees, on pages that are there; and their positions
// into out, by the warp.
template <int D, bool kPaged, int NT>
__device__ __forceinline__ int rows_of(const Token<D, kPaged, NT>& tk, int c) {
  const TopkParams& p = tk.p;
  const int j0 = c << p.block_shift, j1 = min(j0 + (1 << p.block_shift), tk.n);
  int sum = j1 - j0;
  if constexpr (kPaged)
    if (p.block_shift > p.page_shift)
      for (int j = j0; j < j1; j += 1 << p.page_shift)
        if (tk.page_of(j) < 0) sum -= min(1 << p.page_shift, j1 - j);
  return sum;
}
template <int D, bool kPaged, int NT>
__device__ __forceinline__ int write_block(const Token<D, kPaged, NT>& tk, int32_t* out, int at, int c) {
  const TopkParams& p = tk.p;
  const int j0 = c << p.block_shift, j1 = min(j0 + (1 << p.block_shift), tk.n);
  const unsigned below = (1u << tk.lane) - 1;
  for (int j = j0; j < j1; j += 32) {
    bool there = j + tk.lane < j1;
    if constexpr (kPaged) there = there && tk.page_of(j + tk.lane) >= 0;
    const unsigned m = __ballot_sync(0xffffffffu, there);
    if (there && at + __popc(m & below) < p.topk) out[at + __popc(m & below)] = j + tk.lane;
    at += __popc(m);
  }
  return at;
}
// Sum of `mine` (a warp's number) over the warps before this one.
template <int D, bool kPaged, int NT>
__device__ __forceinline__ int before_warp(Token<D, kPaged, NT>& tk, int mine) {
  int* red = tk.template at<int>(SelLayout<D, NT>::kOffRed);
  __syncthreads();
  if (tk.lane == 0) red[tk.warp] = mine;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, tk.lane < tk.warp ? red[tk.lane] : 0);
}
// Nothing behind the last position (after before_warp).
template <int D, bool kPaged, int NT>
__device__ __forceinline__ void fill_rest(Token<D, kPaged, NT>& tk, int32_t* out) {
  using L = SelLayout<D, NT>;
  const int* red = tk.template at<int>(L::kOffRed);
  const int total = __reduce_add_sync(0xffffffffu, tk.lane < L::kWarps ? red[tk.lane] : 0);
  for (int i = total + tk.tid; i < tk.p.topk; i += NT) out[i] = -1;
}

// The token's choice whatever its scores and their number: every pass reads the keys
// again.
template <int D, bool kPaged, int NT>
__device__ __noinline__ void choose_any(Token<D, kPaged, NT> tk) {
  tk.smem = dynamic_smem();
  const TopkParams& p = tk.p;
  const Keys<D, kPaged, NT> keys(tk);
  const Cut cut = any_cut(tk, keys, p.topk >> p.block_shift);
  __syncthreads();
  int tie0 = 0;
  if (cut.r > 0) {
    int ties = 0;
    keys.each([&](int, int key) { ties += key >= cut.klo && key <= cut.khi; });
    tie0 = before_warp(tk, __reduce_add_sync(0xffffffffu, ties));
  }
  const unsigned below = (1u << tk.lane) - 1;
  auto chosen = [&](int key, int& tie) {                 // (a warp's candidates in order; tie: ties so far)
    bool in = key > cut.khi;
    if (cut.r > 0) {
      const bool is_tie = !in && key >= cut.klo;
      const unsigned m = __ballot_sync(0xffffffffu, is_tie);
      in = in || (is_tie && tie + __popc(m & below) < cut.r);
      tie += __popc(m);
    }
    return in;
  };
  int32_t* out = p.out + tk.t * p.topk;
  int rows = 0, tie = tie0;
  keys.each([&](int c, int key) {
    if (chosen(key, tie)) rows += p.block_shift == 0 ? 1 : rows_of(tk, c);
  });
  int at = before_warp(tk, __reduce_add_sync(0xffffffffu, rows));
  tie = tie0;
  keys.each([&](int c, int key) {
    const bool in = chosen(key, tie);
    unsigned m = __ballot_sync(0xffffffffu, in);
    if (p.block_shift == 0) {
      const int to = at + __popc(m & below);
      if (in && to < p.topk) out[to] = c;
      at += __popc(m);
    } else {
      for (; m != 0; m &= m - 1) at = write_block(tk, out, at, __shfl_sync(0xffffffffu, c, __ffs(m) - 1));
    }
  });
  fill_rest(tk, out);
}

// The choice among ordinary scores: bins over the range that a sample of them suggests,
// kept for every candidate (16 bits each: the scores are read once); what lies in and
// next to the bin of number `want` is looked at one by one, and its bin becomes all
// ones or 0.  False where that will not do (scores that are not numbers, a border in the
// ends, many ties).
// kOne: a candidate has one entry in the row.
template <int D, bool kPaged, int NT, bool kOne>
__device__ __forceinline__ bool choose_ordinary(Token<D, kPaged, NT>& tk) {
  using L = SelLayout<D, NT>;
  const TopkParams& p = tk.p;
  const Keys<D, kPaged, NT> keys(tk);
  int *hist = tk.template at<int>(L::kOffHist), *misc = tk.template at<int>(L::kOffMisc), *idx = tk.template at<int>(L::kOffIdx);
  int *more = tk.template at<int>(L::kOffMore), *mark = tk.template at<int>(L::kOffMark), *list = tk.template at<int>(L::kOffVal);
  uint32_t* bins = tk.template at<uint32_t>(L::kOffBins);  // two candidates a word
  const int want = p.topk >> p.block_shift, words = keys.steps / 2, w0 = keys.c0 / 2 + tk.lane;
  // A lane's candidates c, c + 1 of word i: c = c0 + 64 i + 2 lane.  Loads without a
  // branch, and nothing made of them before the next are on their way; what lies behind the
  // last candidate (a row is padded to whole words of four) is seen to where it is used.
  constexpr int kAhead = 8;
  uint2 key[kAhead];
  const uint2* pairs = reinterpret_cast<const uint2*>(keys.row);
  const int last_pair = (keys.nb - 1) / 2;
  auto ask = [&](int i) {
    const int c = keys.c0 + i * 64 + 2 * tk.lane;
    if constexpr (kOne) return load(pairs + min(c / 2, last_pair));
    return make_uint2(keys.fetch(c), keys.fetch(c + 1));
  };
  auto of = [&](uint32_t k, int c) { return c < keys.nb ? static_cast<int>(k) : kKeyNever; };
  tk.start_queries();
#pragma unroll
  for (int i = 0; i < kAhead; ++i) key[i] = ask(i);
  for (int i = tk.tid; i < kBins / 4; i += NT) reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
  if (tk.tid < L::kWarps) more[tk.tid] = 0;
  tk.bounds();
  const int first = of(key[0].x, keys.c0 + 2 * tk.lane);
  const bool fin = first > kKeyNegInf && first < kKeyInf;
  int ends[2] = {fin ? first : INT32_MAX, fin ? first : INT32_MIN};
  tk.template reduce<2, true>(ends);
  if (ends[0] >= ends[1]) return false;
  const float a = value_of(ends[0]), b = value_of(ends[1]), range = b - a;
  const float lo = a - 0.5f * range, per = (0.5f * kBins) / range;  // (twice the range)
  // (fp32 has to resolve the bins.)
  if (!(range > 1e-30f && range < 1e30f && range > 0x1p-11f * fmaxf(fabsf(a), fabsf(b)) && tk.e_score < range)) return false;
  auto bin_of_value = [&](float x) { return max(0, min(kBins - 1, static_cast<int>((x - lo) * per))); };
  auto bin_of = [&](int k) { return k >= kKeyInf ? kBins - 1 : bin_of_value(value_of(k)); };  // (a NaN: 0)
  for (int i0 = 0; i0 < words; i0 += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= words) break;
      const int c = keys.c0 + (i0 + i) * 64 + 2 * tk.lane;
      const int x = bin_of(of(key[i].x, c)), y = bin_of(of(key[i].y, c + 1));
      key[i] = ask(i0 + i + kAhead);
      if (c < keys.nb) atomicAdd(hist + x, 1);
      if (c + 1 < keys.nb) atomicAdd(hist + y, 1);
      bins[w0 + (i0 + i) * 32] = static_cast<uint32_t>(x) | (static_cast<uint32_t>(y) << 16);
    }
  }
  __syncthreads();
  find_bin(tk, want);
  const int bin = misc[0];
  // The bins that T +- 2E can reach, and one more on either side for the roundings.
  const float w = 1.f / per, e2 = 2.f * tk.e_score;
  const int bl = bin_of_value(lo + static_cast<float>(bin) * w - e2) - 1, bh = bin_of_value(lo + static_cast<float>(bin + 1) * w + e2) + 1;
  if (bl < 1 || bh > kBins - 2 || bh - bl > 31) return false;
  const int here = tk.lane <= bh - bl ? hist[bl + tk.lane] : 0;
  const int above = misc[1] - __reduce_add_sync(0xffffffffu, bl + tk.lane > bin ? here : 0);
  const int near = __reduce_add_sync(0xffffffffu, here);
  if (near > kList - 3) return false;
  int sure = 0;
  for (int i0 = 0; i0 < words; i0 += kAhead) {
    uint32_t v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) v[i] = i0 + i < words ? bins[w0 + (i0 + i) * 32] : 0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int x = v[i] & 0xffff, y = v[i] >> 16;
      sure += (x > bh) + (y > bh);
      const bool nx = x >= bl && x <= bh, ny = y >= bl && y <= bh;
      if (nx || ny) {
        const int c = keys.c0 + (i0 + i) * 64 + 2 * tk.lane;
        if (nx) list[kList + atomicAdd(misc + 3, 1)] = c;
        if (ny) list[kList + atomicAdd(misc + 3, 1)] = c + 1;
      }
    }
  }
  __syncthreads();
  for (int i = tk.tid; i < near; i += NT) list[i] = keys.fetch(list[kList + i]);
  __syncthreads();
  int klo, khi;
  const float mid = value_of(nth_of(tk, list, near, want - above));
  window(mid, tk.e_score, klo, khi);
  // Of the list: those above the window, and those in it.
  uint16_t* bin16 = reinterpret_cast<uint16_t*>(bins);
  const int run = keys.steps * 32;
  auto decide = [&](int c, bool in) {
    bin16[c] = in ? 0xffff : 0;
    if (in) atomicAdd(more + c / run, 1);
  };
  if (tk.tid == 0) misc[3] = 0;
  __syncthreads();
  int cnt[2] = {0, 0};
  for (int i = tk.tid; i < near; i += NT) {
    const int k = list[i], c = list[kList + i];
    cnt[0] += k > khi;
    if (k >= klo && k <= khi) {
      ++cnt[1];
      idx[atomicAdd(misc + 3, 1)] = c;
    } else {
      decide(c, k > khi);
    }
  }
  tk.template reduce<2, false>(cnt);
  // (Not from misc[3], which settle sets back before its first barrier.)
  const int m = cnt[1], r = want - above - cnt[0];
  if (m == r) {
    for (int i = tk.tid; i < m; i += NT) decide(idx[i], true);
  } else if (klo == khi) {                               // (exact scores that tie)
    for (int i = tk.tid; i < m; i += NT) {
      int before = 0;
      for (int k = 0; k < m; ++k) before += idx[k] < idx[i];
      decide(idx[i], before < r);
    }
  } else {
    settle(tk, m, r);
    for (int i = tk.tid; i < m; i += NT) decide(idx[i], mark[i] != 0);
  }
  __syncthreads();

  // Positions in order.
  int32_t* out = p.out + tk.t * p.topk;
  const unsigned below = (1u << tk.lane) - 1;
  if (p.block_shift == 0) {
    int at = before_warp(tk, __reduce_add_sync(0xffffffffu, sure) + more[tk.warp]);
#pragma unroll 4
    for (int i = 0; i < words; ++i) {
      const uint32_t v = bins[w0 + i * 32];
      const bool x = static_cast<int>(v & 0xffff) > bh, y = static_cast<int>(v >> 16) > bh;
      const unsigned mx = __ballot_sync(0xffffffffu, x), my = __ballot_sync(0xffffffffu, y);
      const int c = keys.c0 + i * 64 + 2 * tk.lane, to = at + __popc(mx & below) + __popc(my & below);
      if (x && to < p.topk) out[to] = c;
      if (y && to + x < p.topk) out[to + x] = c + 1;
      at += __popc(mx) + __popc(my);
    }
  } else {
    int rows = 0;
    for (int i = 0; i < words; ++i) {
      const uint32_t v = bins[w0 + i * 32];
      const int c = keys.c0 + i * 64 + 2 * tk.lane;
      if (static_cast<int>(v & 0xffff) > bh) rows += rows_of(tk, c);
      if (static_cast<int>(v >> 16) > bh) rows += rows_of(tk, c + 1);
    }
    int at = before_warp(tk, __reduce_add_sync(0xffffffffu, rows));
    for (int i = 0; i < words; ++i) {
      const uint32_t v = bins[w0 + i * 32];
      const unsigned mx = __ballot_sync(0xffffffffu, static_cast<int>(v & 0xffff) > bh);
      const unsigned my = __ballot_sync(0xffffffffu, static_cast<int>(v >> 16) > bh);
      for (unsigned todo = mx | my; todo != 0; todo &= todo - 1) {
        const int from = __ffs(todo) - 1, c = keys.c0 + i * 64 + 2 * from;
        if ((mx >> from) & 1u) at = write_block(tk, out, at, c);
        if ((my >> from) & 1u) at = write_block(tk, out, at, c + 1);
      }
    }
  }
  fill_rest(tk, out);
  return true;
}

template <int D, bool kPaged, int NT>
__global__ void __launch_bounds__(NT, NT == 1024 ? 1 : 3) smqa_topk_select_kernel(const __grid_constant__ TopkParams p) {
  using L = SelLayout<D, NT>;
  uint8_t* smem = dynamic_smem();
  const int tid = threadIdx.x;
  const int64_t t = p.tok0 + blockIdx.x;
  grid_dependency_wait();
  grid_dependents_launch();
  // Scores are missing where a wait ran out.  (Of all threads together: another stream's kernel
  // may set the word between two threads' looks at it, and the others would go on without them.)
  if (__syncthreads_or(*reinterpret_cast<volatile int*>(p.status)) != 0) return;
  int req;
  const int n = visible<kPaged>(p, t, req);
  int32_t* out = p.out + t * p.topk;
  if (req < 0) {
    if (p.zero_padding)
      for (int i = tid; i < p.topk; i += NT) out[i] = -1;
    return;
  }
  Token<D, kPaged, NT> tk{p, smem, t, n, req, tid, tid >> 5, tid & 31, 0.f, 0.f, 0.f};
  if (n <= p.topk) {
    // All that the token sees.
    if constexpr (kPaged) {
      int* red = tk.template at<int>(L::kOffRed);
      int at = 0;
      for (int j0 = 0; j0 < p.topk; j0 += NT) {
        const int j = j0 + tid;
        const bool there = j < n && tk.page_of(j) >= 0;
        const unsigned m = __ballot_sync(0xffffffffu, there);
        if (tk.lane == 0) red[tk.warp] = __popc(m);
        __syncthreads();
        const int mine = tk.lane < L::kWarps ? red[tk.lane] : 0;
        const int before = at + __reduce_add_sync(0xffffffffu, tk.lane < tk.warp ? mine : 0);
        at += __reduce_add_sync(0xffffffffu, mine);
        if (there) out[before + __popc(m & ((1u << tk.lane) - 1))] = j;
        __syncthreads();
      }
      for (int i = at + tid; i < p.topk; i += NT) out[i] = -1;
    } else {
      for (int i = tid; i < p.topk; i += NT) out[i] = i < n ? i : -1;
    }
    return;
  }
  if ((n + (1 << p.block_shift) - 1) >> p.block_shift <= L::kCap) {
    if (p.block_shift <= 5 ? choose_ordinary<D, kPaged, NT, true>(tk) : choose_ordinary<D, kPaged, NT, false>(tk)) return;
  } else {
    tk.start_queries();
    tk.bounds();
  }
  __syncthreads();
  choose_any(tk);
}

template <int D, bool kPaged, int NT>
cudaError_t launch_select(const TopkParams& p, cudaStream_t stream) {
  using L = SelLayout<D, NT>;
  const auto kern = smqa_topk_select_kernel<D, kPaged, NT>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), L::bytes(128), allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.toks));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = L::bytes(p.H);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}
// Long rows, or few tokens with more than short ones: 1024 threads and one CTA per SM;
// else 256 and three.  H = 64, D = 128, topk = 2048, us a call with 256 and with 1024 (nothing
// in L2): 16 paged tokens over 8192 positions 58 and 52, 150 over 12000 103 and 95; 300 over
// 12000 140 and 161, S = 8192 673 and 1101.  (A row's pitch is the table's width with paged
// keys: the host does not know the lengths.)
template <int D, bool kPaged>
cudaError_t launch_select(const TopkParams& p, cudaStream_t stream) {
  return p.ld > SelLayout<D, 256>::kCap || (p.toks <= kSMs && p.ld > 4096) ? launch_select<D, kPaged, 1024>(p, stream)
                                                                          : launch_select<D, kPaged, 256>(p, stream);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
constexpr int64_t kLim = int64_t{1} << 31;
// Entries of a list, and positions that a token may see: the kernels' loops over them step by
// up to 1024 threads, in 32 bits.
constexpr int64_t kMaxCount = kLim - 2048;
// Bytes of scores that a chunk of tokens may take: half of L2, from which the choice reads
// them, or one group's.  (S = 8192, H = 64, topk = 2048: 902 us with 16 MB, 673 with 64, 640 with
// 256, whose workspace a caller would have to hold.)
constexpr int64_t kChunkBytes = int64_t{64} << 20;

smqa_status refuse(smqa_status st, const char* why) {
  set_last_error(why);
  return st;
}
int shift_of(int x) {                                    // (-1: not a power of two up to 128)
  for (int s = 0; s <= 7; ++s)
    if (x == 1 << s) return s;
  return -1;
}
int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Rows that a token may see at most, tokens, units per chunk and the workspace's parts.
struct TopkPlan {
  int64_t ld, norm_ld, units, chunk_units, chunk_toks, norm_bytes, bytes;
};
TopkPlan plan_topk(int64_t rows, int block_shift, int H, bool paged, int64_t B, int64_t S) {
  TopkPlan pl{};
  pl.ld = round_up((rows + (1 << entry_shift(block_shift)) - 1) >> entry_shift(block_shift), 4);
  pl.norm_ld = 4 * ((rows + kTile - 1) / kTile);
  const int group = group_tokens(H);
  pl.units = B * ((S + group - 1) / group);              // (paged: B = 1, S = T)
  pl.chunk_units = std::min(pl.units, std::max<int64_t>(1, kChunkBytes / (pl.ld * 4) / group));
  pl.chunk_toks = std::min(pl.chunk_units * group, B * S);
  pl.norm_bytes = round_up((paged ? pl.chunk_toks : B) * pl.norm_ld * 4, 256);
  pl.bytes = pl.norm_bytes + round_up(pl.chunk_toks * pl.ld * 4, 256);
  return pl;
}

// The choice's own arguments.
smqa_status check_choice(int topk, int block_size, int recent) {
  if (topk <= 0 || block_size <= 0 || recent < 0) return refuse(SMQA_ERR_INVALID_ARG, "non-positive size in topk");
  const int bs = shift_of(block_size);
  if (bs < 0 || topk % block_size != 0 || topk > kMaxCount)
    return refuse(SMQA_ERR_UNSUPPORTED,
                  "unsupported topk (need block_size a power of two up to 128, topk a multiple of it, up to 2^31 - 2048)");
  // (The last `recent` positions touch this many blocks at most.)
  if (recent > 0 && (static_cast<int64_t>(recent) - 2 + block_size) / block_size + 1 > topk / block_size)
    return refuse(SMQA_ERR_INVALID_ARG, "recent positions take more blocks than topk has");
  return SMQA_OK;
}
smqa_status check_flat(const smqa_shape& s) {
  if (s.B <= 0 || s.S <= 0 || s.S_kv <= 0 || s.H <= 0 || s.D <= 0)
    return refuse(SMQA_ERR_INVALID_ARG, "non-positive size in shape");
  if (s.H > 128 || (s.D != 64 && s.D != 128) || s.S_kv > kMaxCount || static_cast<int64_t>(s.B) * s.S_kv >= kLim ||
      static_cast<int64_t>(s.B) * s.S >= kLim)
    return refuse(SMQA_ERR_UNSUPPORTED,
                  "unsupported indexer shape (need 1<=H<=128, D in {64,128}, B*S, B*S_kv < 2^31, S_kv <= 2^31 - 2048)");
  return SMQA_OK;
}
smqa_status check_paged_topk(const smqa_paged_shape& s) {
  if (s.T < 0 || s.R <= 0 || s.H <= 0 || s.D <= 0 || s.page_size <= 0 || s.max_pages <= 0 || s.n_pages <= 0)
    return refuse(SMQA_ERR_INVALID_ARG, "non-positive size in paged shape");
  if (s.H > 128 || (s.D != 64 && s.D != 128) || shift_of(s.page_size) < 4 ||
      static_cast<int64_t>(s.n_pages) * s.page_size >= kLim ||
      static_cast<int64_t>(s.max_pages) * s.page_size > kMaxCount)
    return refuse(SMQA_ERR_UNSUPPORTED,
                  "unsupported paged indexer shape (need 1<=H<=128, D in {64,128}, page_size in {16,32,64,128}, "
                  "n_pages * page_size < 2^31, max_pages * page_size <= 2^31 - 2048)");
  return SMQA_OK;
}

// Boxes of 64 bf16 elements or D codes, swizzled as the tensor core reads them.
bool encode(CUtensorMap* m, const void* ptr, bool codes, int D, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  const auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!fn) {
    set_last_error("cuTensorMapEncodeTiled unavailable");
    return false;
  }
  const cuuint32_t estr[3] = {1, 1, 1};
  auto call = [&] {
    return fn(m, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(ptr), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, codes && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = call();
  if (r == CUDA_ERROR_INVALID_CONTEXT && make_context_current()) r = call();
  if (r != CUDA_SUCCESS) set_last_error("cuTensorMapEncodeTiled failed");
  return r == CUDA_SUCCESS;
}
// Key rows, `box_rows` at a time.
bool encode_keys(CUtensorMap* m, const void* ptr, bool codes, int D, uint64_t rows, uint32_t box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), rows};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * (codes ? 1 : 2)};
  const cuuint32_t box[2] = {codes ? static_cast<cuuint32_t>(D) : 64u, box_rows};
  return encode(m, ptr, codes, D, 2, dims, strides, box);
}
// The queries [T, H, D], a group of tokens at a time, their heads padded with zeros.
bool encode_queries(CUtensorMap* m, const void* ptr, int H, int D, uint64_t T) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), T};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(H) * D * 2};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(padded_heads(H)), static_cast<cuuint32_t>(group_tokens(H))};
  return encode(m, ptr, false, D, 3, dims, strides, box);
}

// The chunks of one call, one after another.
smqa_status run_topk(TopkParams p, const TopkPlan& pl, const CUtensorMap& tm_k, const CUtensorMap& tm_q, int D, bool paged, int64_t per_batch_units,
                     void* workspace, cudaStream_t stream) {
  cudaError_t e;
  p.status = device_status_word(&e);
  if (!p.status) return cuda_failure(e, "status word");
  p.limit_ns = current_wait_limit_ns();
  p.stall_cta = current_stall_cta();
  p.ld = pl.ld;
  p.norm_ld = pl.norm_ld;
  p.norms = static_cast<float*>(workspace);
  p.rows = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + pl.norm_bytes);
  const int group = group_tokens(p.H);
  // First token of a unit.
  auto first_of = [&](int64_t u) {
    if (u >= pl.units) return static_cast<int64_t>(p.T);
    return paged ? u * group : u / per_batch_units * p.S + u % per_batch_units * group;
  };
  for (int64_t u = 0; u < pl.units; u += pl.chunk_units) {
    p.unit0 = u;
    p.units = std::min(pl.chunk_units, pl.units - u);
    p.tok0 = first_of(u);
    p.toks = first_of(u + p.units) - p.tok0;
    e = launch_topk_score(tm_k, tm_q, p, D, paged, stream);
    if (e != cudaSuccess) return cuda_failure(e, "topk score launch");
    e = launch_topk_select(p, D, paged, stream);
    if (e != cudaSuccess) return cuda_failure(e, "topk select launch");
  }
  return SMQA_OK;
}

smqa_status check_workspace(const void* workspace, size_t have, int64_t need) {
  if (!workspace || !is_aligned(workspace, 256)) return refuse(SMQA_ERR_INVALID_ARG, "null or misaligned pointer");
  if (have < static_cast<size_t>(need)) {
    char msg[128];
    std::snprintf(msg, sizeof msg, "workspace too small (%zu < %zu bytes)", have, static_cast<size_t>(need));
    return refuse(SMQA_ERR_UNSUPPORTED, msg);
  }
  return SMQA_OK;
}

}  // namespace

cudaError_t launch_topk_select(const TopkParams& p, int D, bool paged, cudaStream_t stream) {
  if (paged) return D == 64 ? launch_select<64, true>(p, stream) : launch_select<128, true>(p, stream);
  return D == 64 ? launch_select<64, false>(p, stream) : launch_select<128, false>(p, stream);
}

}  // namespace smqa

using namespace smqa;

extern "C" {

size_t smqa_indexer_topk_workspace_bytes(smqa_shape s, int32_t block_size) {
  if (check_flat(s) != SMQA_OK || check_choice(s.topk, block_size, 0) != SMQA_OK) return 0;
  return static_cast<size_t>(plan_topk(s.S_kv, shift_of(block_size), s.H, false, s.B, s.S).bytes);
}

smqa_status smqa_indexer_topk(const void* index_q, const float* weights, const void* index_k, smqa_shape s,
                              int32_t block_size, int32_t recent, int64_t first_position, int32_t* topk_idxs,
                              void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  smqa_status st = check_flat(s);
  if (st == SMQA_OK) st = check_choice(s.topk, block_size, recent);
  if (st != SMQA_OK) return st;
  if (!index_q || !weights || !index_k || !topk_idxs || !is_aligned(index_q, 16) || !is_aligned(index_k, 16) ||
      !is_aligned(weights, 4) || !is_aligned(topk_idxs, 4))
    return refuse(SMQA_ERR_INVALID_ARG, "null or misaligned pointer");
  const TopkPlan pl = plan_topk(s.S_kv, shift_of(block_size), s.H, false, s.B, s.S);
  st = check_workspace(workspace, workspace_bytes, pl.bytes);
  if (st != SMQA_OK) return st;
  CUtensorMap tm, tm_q;
  if (!encode_keys(&tm, index_k, false, s.D, static_cast<uint64_t>(s.B) * s.S_kv, kTile) ||
      !encode_queries(&tm_q, index_q, s.H, s.D, static_cast<uint64_t>(s.B) * s.S))
    return SMQA_ERR_CUDA;
  TopkParams p{};
  p.q = static_cast<const __nv_bfloat16*>(index_q);
  p.w = weights;
  p.k = static_cast<const __nv_bfloat16*>(index_k);
  p.T = s.B * s.S;
  p.H = s.H;
  p.S = s.S;
  p.S_kv = s.S_kv;
  p.B = s.B;
  // (Beyond these a token sees nothing, or everything.)
  p.first = std::max<int64_t>(-kLim, std::min<int64_t>(first_position, kLim));
  p.topk = s.topk;
  p.block_shift = shift_of(block_size);
  p.recent = recent;
  p.out = topk_idxs;
  return run_topk(p, pl, tm, tm_q, s.D, false, (s.S + group_tokens(s.H) - 1) / group_tokens(s.H), workspace, stream);
}

size_t smqa_paged_indexer_topk_workspace_bytes(smqa_paged_shape s, int32_t block_size) {
  if (check_paged_topk(s) != SMQA_OK || check_choice(s.topk, block_size, 0) != SMQA_OK || s.T == 0) return 0;
  return static_cast<size_t>(
      plan_topk(static_cast<int64_t>(s.max_pages) * s.page_size, shift_of(block_size), s.H, true, 1, s.T).bytes);
}

smqa_status smqa_paged_indexer_topk(const void* index_q, const float* weights, const void* k_cache, const float* k_scales,
                                    const int32_t* block_table, const int32_t* seq_lens, const int32_t* token_req,
                                    const int32_t* positions, smqa_paged_shape s, int32_t block_size, int32_t recent,
                                    int32_t* topk_idxs, void* workspace, size_t workspace_bytes, unsigned flags,
                                    cudaStream_t stream) {
  smqa_status st = check_paged_topk(s);
  if (st == SMQA_OK) st = check_choice(s.topk, block_size, recent);
  if (st != SMQA_OK) return st;
  if (flags & ~SMQA_FLAG_ZERO_PADDING) return refuse(SMQA_ERR_INVALID_ARG, "bad flags");
  if (s.T == 0) return SMQA_OK;
  if (!index_q || !weights || !k_cache || !k_scales || !block_table || !seq_lens || !token_req || !topk_idxs ||
      !is_aligned(index_q, 16) || !is_aligned(k_cache, 16) || !is_aligned(weights, 4) || !is_aligned(k_scales, 4) ||
      !is_aligned(block_table, 4) || !is_aligned(seq_lens, 4) || !is_aligned(token_req, 4) || !is_aligned(positions, 4) ||
      !is_aligned(topk_idxs, 4))
    return refuse(SMQA_ERR_INVALID_ARG, "null or misaligned pointer");
  const TopkPlan pl = plan_topk(static_cast<int64_t>(s.max_pages) * s.page_size, shift_of(block_size), s.H, true, 1, s.T);
  st = check_workspace(workspace, workspace_bytes, pl.bytes);
  if (st != SMQA_OK) return st;
  CUtensorMap tm;
  if (!encode_keys(&tm, k_cache, true, s.D, static_cast<uint64_t>(s.n_pages) * s.page_size, s.page_size)) return SMQA_ERR_CUDA;
  TopkParams p{};
  p.q = static_cast<const __nv_bfloat16*>(index_q);
  p.w = weights;
  p.codes = static_cast<const uint8_t*>(k_cache);
  p.scales = k_scales;
  p.table = block_table;
  p.seq_lens = seq_lens;
  p.token_req = token_req;
  p.positions = positions;
  p.T = s.T;
  p.H = s.H;
  p.S = s.T;
  p.B = 1;
  p.R = s.R;
  p.max_pages = s.max_pages;
  p.n_pages = s.n_pages;
  p.page_shift = shift_of(s.page_size);
  p.topk = s.topk;
  p.block_shift = shift_of(block_size);
  p.recent = recent;
  p.out = topk_idxs;
  p.zero_padding = (flags & SMQA_FLAG_ZERO_PADDING) ? 1 : 0;
  return run_topk(p, pl, tm, tm, s.D, true, pl.units, workspace, stream);
}

}  // extern "C"

// smqa_topk.cu -- the indexer's selection on sm_103a: which blocks of positions a
// token attends to, and the argument checks of its two forms (contiguous keys, and
// the 8-bit paged cache).
//
// The choice is that of the scores in real numbers, ties to the lowest position, so
// that it does not depend on how a batch is cut or summed.  The score kernel's values
// are off by E at most (below); with T the k-th largest of them, a block above T + 2E
// is chosen and one below T - 2E is not.  The few between are scored again: products
// of bf16 and of e4m3 numbers are exact in fp32, and each is added with its rounding
// error kept in a second fp32 sum (two-sum), heads in fp64.
//
// E = K sum_h |w_h| (c |q_h| + rho_h), K the largest length of a key row that the
// token sees: an fp32 accumulation of D products loses at most kDotError |q||k| (a
// step is off by 2^-24 of a partial sum of at most |q||k|, D/16 or D/32 x 2 steps,
// each with some 2^-21 for the sum inside the step), the sum over heads (H/4 + 4)
// 2^-24, and rho_h is what two e4m3 pieces leave of a query row (0 with bf16 keys).
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdio>

#include "smqa_topk.cuh"

namespace smqa {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kItems = 16;                               // candidates of a thread that stay in registers
constexpr int kBins = 2048;
constexpr int kList = 1024;
constexpr float kDotError = 0x1p-19f;
constexpr int32_t kKeyNegInf = -kKeyInf - 1;            // (key_of(-infinity): the bits 0xff800000 but for the sign flipped)

template <int D, bool kPaged>
struct SelLayout {
  static constexpr uint32_t kOffQ = 0;                   // bf16 [128][D], 16-byte pieces c at c ^ (h mod 8)
  static constexpr uint32_t kOffHist = 128 * D * 2;      // int [kBins]
  static constexpr uint32_t kOffVal = kOffHist + kBins * 4;   // double [kList]
  static constexpr uint32_t kOffIdx = kOffVal + kList * 8;    // int [kList]
  static constexpr uint32_t kOffRow = kOffIdx + kList * 4;    // float [kWarps][D]
  static constexpr uint32_t kOffW = kOffRow + kWarps * D * 4;  // float [128]
  static constexpr uint32_t kOffRed = kOffW + 128 * 4;        // int [8][kWarps]
  static constexpr uint32_t kOffMisc = kOffRed + 8 * kWarps * 4;
  static constexpr uint32_t kSmem = kOffMisc + 64;
};

__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, make_float2(-1.f, -1.f), a); }

// What a CTA knows of its token.
template <int D, bool kPaged>
struct Token {
  using L = SelLayout<D, kPaged>;
  const TopkParams& p;
  uint8_t* smem;
  int64_t t;
  int n, req;
  int tid, warp, lane;

  // Over the CTA, the same in all threads: with kEnds the least of v[0] and the largest
  // of v[1], and the sums of the others.
  template <int N, bool kEnds>
  __device__ __forceinline__ void reduce(int (&v)[N]) {
    static_assert(N <= 8, "room for eight values");
    int* red = reinterpret_cast<int*>(smem + L::kOffRed);
    auto over_warp = [](int i, int x) {
      return kEnds && i == 0   ? __reduce_min_sync(0xffffffffu, x)
             : kEnds && i == 1 ? __reduce_max_sync(0xffffffffu, x)
                               : __reduce_add_sync(0xffffffffu, x);
    };
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = over_warp(i, v[i]);
      if (lane == 0) red[i * kWarps + warp] = x;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = lane < kWarps ? red[i * kWarps + lane] : kEnds && i == 0 ? INT32_MAX : kEnds && i == 1 ? INT32_MIN : 0;
      v[i] = over_warp(i, x);
    }
    __syncthreads();
  }

  __device__ __forceinline__ int page_of(int j) const {  // (-1: none)
    const int pg = load(p.table + static_cast<int64_t>(req) * p.max_pages + (j >> p.page_shift));
    return static_cast<unsigned>(pg) < static_cast<unsigned>(p.n_pages) ? pg : -1;
  }
  // Key row j's values, D/32 per lane, into the warp's row buffer, and its scale (-1: no such row).
  __device__ __forceinline__ float bring(int j) {
    float* buf = reinterpret_cast<float*>(smem + L::kOffRow) + warp * D;
    __syncwarp();
    float scale = 1.f;
    if constexpr (kPaged) {
      const int pg = page_of(j);
      if (pg < 0) return -1.f;
      const uint8_t* src = p.codes + ((static_cast<int64_t>(pg) << p.page_shift) + (j & ((1 << p.page_shift) - 1))) * D;
      scale = load(p.scales + pg);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        uint16_t v;
        asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(src + (i * 32 + lane) * 2));
        reinterpret_cast<float2*>(buf)[i * 32 + lane] = e4m3x2_value(v);
      }
    } else {
      const __nv_bfloat16* src = p.k + (static_cast<int64_t>(req) * p.S_kv + j) * D;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint32_t v = static_cast<uint32_t>(load(reinterpret_cast<const int*>(src) + i * 32 + lane));
        reinterpret_cast<float2*>(buf)[i * 32 + lane] = make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
      }
    }
    __syncwarp();
    return scale;
  }
  // The score of the row in the buffer: lane = head.  kExact: products and sums with
  // their errors kept; else plain fp32, off by kPlainError K sum |w||q| at most.
  template <bool kExact>
  __device__ __forceinline__ double dot_heads() {
    const float4* kb = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + L::kOffRow) + warp * D);
    const float* w = reinterpret_cast<const float*>(smem + L::kOffW);
    double total = 0.;
    for (int h = lane; h < p.H; h += 32) {
      const uint4* qr = reinterpret_cast<const uint4*>(smem + L::kOffQ) + h * (D / 8);
      float2 s = make_float2(0.f, 0.f), err = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        const uint4 v = qr[c ^ (h & 7)];
        const float4 ka = kb[2 * c], kc = kb[2 * c + 1];
        const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
        const float2 k4[4] = {make_float2(ka.x, ka.y), make_float2(ka.z, ka.w), make_float2(kc.x, kc.y), make_float2(kc.z, kc.w)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 q = make_float2(__uint_as_float(w4[i] << 16), __uint_as_float(w4[i] & 0xffff0000u));
          if constexpr (kExact) {
            const float2 x = mul2(q, k4[i]);
            const float2 sum = add2(s, x), back = sub2(sum, s);
            err = add2(err, add2(sub2(s, sub2(sum, back)), sub2(x, back)));
            s = sum;
          } else {
            s = fma2(q, k4[i], s);
          }
        }
      }
      double d = static_cast<double>(s.x) + s.y;
      if (kExact && fabs(d) < static_cast<double>(INFINITY)) d += static_cast<double>(err.x) + err.y;
      total += static_cast<double>(w[h]) * (d > 0. ? d : d == d ? 0. : d);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    return total;
  }
  // The exact score of block c (a NaN as -infinity), by the whole warp: of a larger
  // block only the rows whose plain score may exceed the best so far.
  __device__ __forceinline__ double exact(int c, float margin) {
    const int j0 = c << p.block_shift, j1 = min(j0 + (1 << p.block_shift), n);
    double best = -static_cast<double>(INFINITY);
    for (int j = j0; j < j1; ++j) {
      const float scale = bring(j);
      if (scale < 0.f) continue;
      if (p.block_shift > 0 && dot_heads<false>() * scale < best - margin) continue;
      const double x = dot_heads<true>() * scale;
      if (x > best) best = x;
    }
    return best;
  }
};

// Of candidates with keys: the one whose number r (1-based, from the largest) is
// asked for among those that are finite, between keys lo and hi; by histograms over
// values, then by ranks.  get(f): f(candidate, key) for all candidates of the thread.
template <int D, bool kPaged, typename Get>
__device__ __forceinline__ int32_t find(Token<D, kPaged>& tk, int lo, int hi, int r, Get get) {
  using L = SelLayout<D, kPaged>;
  int* hist = reinterpret_cast<int*>(tk.smem + L::kOffHist);
  int* list = reinterpret_cast<int*>(tk.smem + L::kOffIdx);
  int* misc = reinterpret_cast<int*>(tk.smem + L::kOffMisc);
  int* red = reinterpret_cast<int*>(tk.smem + L::kOffRed);
  while (lo < hi) {
    // Linear in the value, or (a range that fp32 cannot hold) in the key.
    const float half = 0.5f * value_of(lo), range = 0.5f * value_of(hi) - half;
    const bool linear = range > 1e-30f && range < 1e38f;
    const float per = (kBins - 0.5f) / range;
    const int shift = max(0, 22 - __clz(static_cast<unsigned>(hi) - static_cast<unsigned>(lo)));
    auto bin_of = [&](int key) {
      return linear ? min(kBins - 1, static_cast<int>((0.5f * value_of(key) - half) * per))
                    : static_cast<int>((static_cast<unsigned>(key) - static_cast<unsigned>(lo)) >> shift);
    };
    for (int i = tk.tid; i < kBins; i += kThreads) hist[i] = 0;
    __syncthreads();
    get([&](int, int key) {
      if (key >= lo && key <= hi) atomicAdd(hist + bin_of(key), 1);
    });
    __syncthreads();
    // From the top: thread i has bins kBins - 1 - 4 i and the three below.
    constexpr int kPer = kBins / kThreads;
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
    int above = incl - sum;
    for (int w = 0; w < tk.warp; ++w) above += red[w];
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
    const int bin = misc[0], members = misc[2];
    r -= misc[1];
    if (members <= kList) {
      get([&](int, int key) {
        if (key >= lo && key <= hi && bin_of(key) == bin) list[atomicAdd(misc + 3, 1)] = key;
      });
      __syncthreads();
      for (int i = tk.tid; i < members; i += kThreads) {
        const int v = list[i];
        int more = 0, same = 0;
        for (int k = 0; k < members; ++k) {
          more += list[k] > v;
          same += list[k] == v;
        }
        if (more < r && r <= more + same) misc[0] = v;
      }
      __syncthreads();
      const int found = misc[0];
      __syncthreads();
      return found;
    }
    int ends[2] = {INT32_MAX, INT32_MIN};
    get([&](int, int key) {
      if (key >= lo && key <= hi && bin_of(key) == bin) {
        ends[0] = min(ends[0], key);
        ends[1] = max(ends[1], key);
      }
    });
    tk.template reduce<2, true>(ends);
    lo = ends[0];
    hi = ends[1];
  }
  return lo;
}

// The token's choice, with more candidates than choices.  kReg: the keys stay in
// registers (up to kThreads kItems candidates), else they are read again by every pass.
template <int D, bool kPaged, bool kReg>
__device__ __forceinline__ void choose(Token<D, kPaged>& tk) {
  using L = SelLayout<D, kPaged>;
  const TopkParams& p = tk.p;
  const int bs = 1 << p.block_shift, nb = (tk.n + bs - 1) >> p.block_shift, want = p.topk >> p.block_shift;
  const int eshift = entry_shift(p.block_shift), per = 1 << (p.block_shift - eshift), entries = (tk.n + (1 << eshift) - 1) >> eshift;
  int32_t* row = p.rows + (tk.t - p.tok0) * p.ld;
  int* misc = reinterpret_cast<int*>(tk.smem + L::kOffMisc);
  int* idx = reinterpret_cast<int*>(tk.smem + L::kOffIdx);
  double* val = reinterpret_cast<double*>(tk.smem + L::kOffVal);
  // A warp has a run of candidates, lane by lane.
  const int run = ((nb + kWarps - 1) / kWarps + 31) & ~31, c0 = tk.warp * run, steps = run / 32;
  auto fetch = [&](int c) {
    if (c >= nb) return kKeyNever;
    if (per == 1) return load(row + c);
    int key = kKeyNever;
    for (int i = 0; i < per; ++i)
      if (c * per + i < entries) key = max(key, load(row + c * per + i));
    return key;
  };
  auto store = [&](int c, int key) {                     // (all of a block in its first entry)
    row[static_cast<int64_t>(c) * per] = key;
    for (int i = 1; i < per; ++i)
      if (c * per + i < entries) row[static_cast<int64_t>(c) * per + i] = kKeyNever;
  };
  int reg[kReg ? kItems : 1];
  auto refresh = [&] {
    if constexpr (kReg) {
#pragma unroll
      for (int i = 0; i < kItems; ++i) reg[i] = i < steps ? fetch(c0 + i * 32 + tk.lane) : kKeyNever;
    }
  };
  auto get = [&](auto f) {
    if constexpr (kReg) {
#pragma unroll
      for (int i = 0; i < kItems; ++i)
        if (i < steps) f(c0 + i * 32 + tk.lane, reg[i]);
    } else {
#pragma unroll 4
      for (int i = 0; i < steps; ++i) f(c0 + i * 32 + tk.lane, fetch(c0 + i * 32 + tk.lane));
    }
  };
  refresh();

  // E and the margin of plain scores: four threads per head.
  float e0 = 0.f, margin = 0.f;
  {
    const int h = tk.tid >> 2, part = tk.tid & 3;
    float len = 0.f, rest = 0.f, wh = 0.f;
    if (h < p.H) {
      const uint4* qr = reinterpret_cast<const uint4*>(tk.smem + L::kOffQ) + h * (D / 8);
      uint4 v[D / 32];
      uint32_t m = 0;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        v[c] = qr[(part * (D / 32) + c) ^ (h & 7)];
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(v[c].x & 0x7fff7fffu, v[c].y & 0x7fff7fffu), __vmaxu2(v[c].z & 0x7fff7fffu, v[c].w & 0x7fff7fffu)));
      }
      m = max(m & 0xffffu, m >> 16);
      m = max(m, __shfl_xor_sync(0xfu << (tk.lane & 28), m, 1));
      m = max(m, __shfl_xor_sync(0xfu << (tk.lane & 28), m, 2));
      const int k = query_exponent(m);
      const float f = pow2f(k), back = pow2f(-k);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const uint32_t w4[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = make_float2(__uint_as_float(w4[i] << 16) * f, __uint_as_float(w4[i] & 0xffff0000u) * f);
          len = fmaf(x.x, x.x, fmaf(x.y, x.y, len));
          if constexpr (kPaged) {
            uint16_t hi, lo;
            split_query(x, hi, lo);
            const float2 a = e4m3x2_value(hi), b = e4m3x2_value(lo);
            const float dx = x.x - a.x - b.x, dy = x.y - a.y - b.y;
            rest = fmaf(dx, dx, fmaf(dy, dy, rest));
          }
        }
      }
      len += __shfl_xor_sync(0xfu << (tk.lane & 28), len, 1);
      rest += __shfl_xor_sync(0xfu << (tk.lane & 28), rest, 1);
      len += __shfl_xor_sync(0xfu << (tk.lane & 28), len, 2);
      rest += __shfl_xor_sync(0xfu << (tk.lane & 28), rest, 2);
      wh = part == 0 ? fabsf(reinterpret_cast<const float*>(tk.smem + L::kOffW)[h]) * back : 0.f;
      len = wh * sqrtf(len);
      rest = wh * sqrtf(rest);
    }
    // The longest row of the tiles that the token sees.
    const int tiles = (tk.n + kTile - 1) / kTile;
    const float* norms = p.norms + (kPaged ? tk.t - p.tok0 : static_cast<int64_t>(tk.req)) * p.norm_ld;
    float top = 0.f;
    for (int i = tk.tid; i < tiles; i += kThreads) top = fmaxf(top, load(norms + i));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      len += __shfl_xor_sync(0xffffffffu, len, off);
      rest += __shfl_xor_sync(0xffffffffu, rest, off);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    }
    float* red = reinterpret_cast<float*>(tk.smem + L::kOffRed);
    if (tk.lane == 0) {
      red[tk.warp] = len;
      red[kWarps + tk.warp] = rest;
      red[2 * kWarps + tk.warp] = top;
    }
    __syncthreads();
    len = rest = top = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      len += red[w];
      rest += red[kWarps + w];
      top = fmaxf(top, red[2 * kWarps + w]);
    }
    __syncthreads();
    // (1.01 for the rounding of these sums, 2^-110 for what underflows: a lone factor of 0
    // leaves scores of exactly 0.)
    const float c = kDotError + (static_cast<float>(p.H) * 0.25f + 4.f) * 0x1p-24f;
    e0 = len * top == 0.f ? 0.f : 1.01f * top * (len * c + rest) + top * 0x1p-110f;
    margin = 1.01f * top * len * 0x1p-17f + top * 0x1p-110f;
    if (!(e0 < INFINITY)) e0 = INFINITY;
  }

  // `level` 0: the score kernel's values.  Where more candidates than the list holds lie
  // in the window, their exact scores less T take the values' place, off by a rounding
  // of what is left (level 1), and so again (level 2: what is still equal ties).
  int klo = 0, khi = 0, r = 0;                           // chosen: above khi, and the first r of [klo, khi]
  double base = 0.;
  for (int level = 0;; ++level) {
    int v[7] = {INT32_MAX, INT32_MIN, 0, 0, 0, 0, 0};    // finite: least, largest, number; >= inf; always; NaN; never
    get([&](int c, int key) {
      if (key > kKeyNegInf && key < kKeyInf) {
        v[0] = min(v[0], key);
        v[1] = max(v[1], key);
        ++v[2];
      }
      v[3] += key >= kKeyInf;
      v[4] += key == kKeyAlways;
      v[5] += key == kKeyNan;
      v[6] += c < nb && key == kKeyNever;
    });
    tk.template reduce<7, true>(v);
    if (nb - v[6] <= want) {                             // all there are
      klo = khi = kKeyNever;
      r = 0;
      break;
    }
    if (want <= v[3]) {
      klo = khi = want <= v[4] ? kKeyAlways : kKeyInf;
      r = want <= v[4] ? want : want - v[4];
      break;
    }
    if (want > v[3] + v[2]) {
      const int neg = nb - v[6] - v[5] - v[3] - v[2];
      r = want - v[3] - v[2];
      klo = khi = r <= neg ? kKeyNegInf : kKeyNan;
      if (r > neg) r -= neg;
      break;
    }
    const int32_t at = find<D, kPaged>(tk, v[0], v[1], want - v[3], get);
    const float mid = value_of(at);
    const float e = level == 0 ? e0 : level == 1 ? fmaxf(fabsf(value_of(v[0])), fabsf(value_of(v[1]))) * 0x1p-23f : 0.f;
    klo = max(key_of(__fadd_rd(mid, -2.f * e)), kKeyNegInf + 1);
    khi = min(key_of(__fadd_ru(mid, 2.f * e)), kKeyInf - 1);
    if (tk.tid == 0) misc[3] = 0;
    __syncthreads();
    int cnt[2] = {0, 0};
    get([&](int c, int key) {
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
    if (m == r || klo == khi) break;
    if (m <= kList) {
      for (int i = tk.warp; i < m; i += kWarps) {
        const double x = tk.exact(idx[i], margin);
        if (tk.lane == 0) val[i] = x;
      }
      __syncthreads();
      for (int i = tk.tid; i < m; i += kThreads) {
        const double x = val[i];
        const int c = idx[i];
        int before = 0;
        for (int k = 0; k < m; ++k) before += val[k] > x || (val[k] == x && idx[k] < c);
        store(c, before < r ? kKeyAlways : kKeyNever);
      }
      __syncthreads();
      r = 0;
      if constexpr (kReg) {
#pragma unroll
        for (int i = 0; i < kItems; ++i)
          if (i < steps && reg[i] >= klo && reg[i] <= khi) reg[i] = fetch(c0 + i * 32 + tk.lane);
      }
      klo = khi;
      break;
    }
    // (base: of the values so far; the new ones' is T.)
    base += static_cast<double>(mid);
    for (int i = 0; i < steps; ++i) {
      const int c = c0 + i * 32 + tk.lane, key = fetch(c);
      const bool in = c < nb && key >= klo && key <= khi;
      for (unsigned todo = __ballot_sync(0xffffffffu, in); todo != 0; todo &= todo - 1) {
        const int cc = c0 + i * 32 + __ffs(todo) - 1;
        const double x = tk.exact(cc, margin);
        if (tk.lane == 0) store(cc, key_of(static_cast<float>(x - base)));
      }
      if (c < nb && !in) store(c, key > khi ? kKeyAlways : kKeyNever);
      __syncwarp();
    }
    __syncthreads();
    refresh();
  }

  // Positions in order: the warps' numbers of ties, then of rows, then the rows.
  int* red = reinterpret_cast<int*>(tk.smem + L::kOffRed);
  auto before_warp = [&](int mine) {                     // sum over the warps before, and over all in red[kWarps]
    if (tk.lane == 0) red[tk.warp] = mine;
    __syncthreads();
    int sum = 0;
    for (int w = 0; w < tk.warp; ++w) sum += red[w];
    return sum;
  };
  int ties = 0;
  if (r > 0) get([&](int, int key) { ties += key >= klo && key <= khi; });
  ties = __reduce_add_sync(0xffffffffu, ties);
  int tie0 = before_warp(ties);
  __syncthreads();
  // Rows of a chosen block: those the token sees, on pages that are there.
  auto rows_of = [&](int c) {
    const int j0 = c << p.block_shift, j1 = min(j0 + bs, tk.n);
    int rows = j1 - j0;
    if constexpr (kPaged)
      if (p.block_shift > p.page_shift)
        for (int j = j0; j < j1; j += 1 << p.page_shift)
          if (tk.page_of(j) < 0) rows -= min(1 << p.page_shift, j1 - j);
    return rows;
  };
  const unsigned below = (1u << tk.lane) - 1;
  auto chosen = [&](int key, int& tie) {                 // (a warp's candidates in order; tie: ties so far)
    const bool is_tie = r > 0 && key >= klo && key <= khi;
    const unsigned m = __ballot_sync(0xffffffffu, is_tie);
    const bool in = (key > khi) || (is_tie && tie + __popc(m & below) < r);
    tie += __popc(m);
    return in;
  };
  int rows = 0, tie = tie0;
  get([&](int c, int key) {
    const bool in = chosen(key, tie);
    if (in) rows += rows_of(c);
  });
  rows = __reduce_add_sync(0xffffffffu, rows);
  int at = before_warp(rows);
  int32_t* out = p.out + tk.t * p.topk;
  tie = tie0;
  get([&](int c, int key) {
    const bool in = chosen(key, tie);
    unsigned m = __ballot_sync(0xffffffffu, in);
    if (p.block_shift == 0) {
      if (in && at + __popc(m & below) < p.topk) out[at + __popc(m & below)] = c;
      at += __popc(m);
    } else {
      for (; m != 0; m &= m - 1) {
        const int cc = __shfl_sync(0xffffffffu, c, __ffs(m) - 1);
        const int j0 = cc << p.block_shift, j1 = min(j0 + bs, tk.n);
        for (int j = j0; j < j1; j += 32) {
          bool there = j + tk.lane < j1;
          if constexpr (kPaged) there = there && tk.page_of(j + tk.lane) >= 0;
          const unsigned rm = __ballot_sync(0xffffffffu, there);
          if (there && at + __popc(rm & below) < p.topk) out[at + __popc(rm & below)] = j + tk.lane;
          at += __popc(rm);
        }
      }
    }
  });
  // Nothing behind the last row.
  int total = 0;
  for (int w = 0; w < kWarps; ++w) total += red[w];
  for (int i = total + tk.tid; i < p.topk; i += kThreads) out[i] = -1;
}

template <int D, bool kPaged>
__global__ void __launch_bounds__(kThreads) smqa_topk_select_kernel(const TopkParams p) {
  using L = SelLayout<D, kPaged>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x;
  const int64_t t = p.tok0 + blockIdx.x;
  grid_dependency_wait();
  grid_dependents_launch();
  if (*reinterpret_cast<volatile int*>(p.status) != 0) return;  // (scores are missing)
  int req;
  const int n = visible<kPaged>(p, t, req);
  int32_t* out = p.out + t * p.topk;
  if (req < 0) {
    if (p.zero_padding)
      for (int i = tid; i < p.topk; i += kThreads) out[i] = -1;
    return;
  }
  Token<D, kPaged> tk{p, smem, t, n, req, tid, tid >> 5, tid & 31};
  if (n <= p.topk) {
    // All that the token sees.
    if constexpr (kPaged) {
      int* red = reinterpret_cast<int*>(smem + L::kOffRed);
      int at = 0;
      for (int j0 = 0; j0 < p.topk; j0 += kThreads) {
        const int j = j0 + tid;
        const bool there = j < n && tk.page_of(j) >= 0;
        const unsigned m = __ballot_sync(0xffffffffu, there);
        if (tk.lane == 0) red[tk.warp] = __popc(m);
        __syncthreads();
        int before = at;
        for (int w = 0; w < kWarps; ++w) {
          before += w < tk.warp ? red[w] : 0;
          at += red[w];
        }
        if (there) out[before + __popc(m & ((1u << tk.lane) - 1))] = j;
        __syncthreads();
      }
      for (int i = at + tid; i < p.topk; i += kThreads) out[i] = -1;
    } else {
      for (int i = tid; i < p.topk; i += kThreads) out[i] = i < n ? i : -1;
    }
    return;
  }
  // Queries and weights.
  const uint32_t q_at = smem_u32(smem) + L::kOffQ;
  const __nv_bfloat16* q = p.q + t * p.H * D;
  for (int i = tid; i < p.H * (D / 8); i += kThreads) {
    const int h = i / (D / 8), c = i % (D / 8);
    cp_async_16(q_at + h * D * 2 + ((c ^ (h & 7)) << 4), q + static_cast<int64_t>(i) * 8);
  }
  if (tid < p.H) reinterpret_cast<float*>(smem + L::kOffW)[tid] = load(p.w + t * p.H + tid);
  cp_async_wait_all();
  __syncthreads();
  const int nb = (n + (1 << p.block_shift) - 1) >> p.block_shift;
  if (nb <= kThreads * kItems)
    choose<D, kPaged, true>(tk);
  else
    choose<D, kPaged, false>(tk);
}

template <int D, bool kPaged>
cudaError_t launch_select(const TopkParams& p, cudaStream_t stream) {
  using L = SelLayout<D, kPaged>;
  const auto kern = smqa_topk_select_kernel<D, kPaged>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), L::kSmem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.toks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
constexpr int64_t kLim = int64_t{1} << 31;
// Bytes of scores that a chunk of tokens may take.
constexpr int64_t kChunkBytes = int64_t{512} << 20;

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
  pl.norm_ld = (rows + kTile - 1) / kTile;
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
  if (bs < 0 || topk % block_size != 0)
    return refuse(SMQA_ERR_UNSUPPORTED, "unsupported topk (need block_size a power of two up to 128, topk a multiple of it)");
  // (The last `recent` positions touch this many blocks at most.)
  if (recent > 0 && (static_cast<int64_t>(recent) - 2 + block_size) / block_size + 1 > topk / block_size)
    return refuse(SMQA_ERR_INVALID_ARG, "recent positions take more blocks than topk has");
  return SMQA_OK;
}
smqa_status check_flat(const smqa_shape& s) {
  if (s.B <= 0 || s.S <= 0 || s.S_kv <= 0 || s.H <= 0 || s.D <= 0)
    return refuse(SMQA_ERR_INVALID_ARG, "non-positive size in shape");
  if (s.H > 128 || (s.D != 64 && s.D != 128) || s.S_kv > kLim - 256 || static_cast<int64_t>(s.B) * s.S_kv >= kLim ||
      static_cast<int64_t>(s.B) * s.S >= kLim)
    return refuse(SMQA_ERR_UNSUPPORTED, "unsupported indexer shape (need 1<=H<=128, D in {64,128}, B*S, B*S_kv < 2^31)");
  return SMQA_OK;
}
smqa_status check_paged_topk(const smqa_paged_shape& s) {
  if (s.T < 0 || s.R <= 0 || s.H <= 0 || s.D <= 0 || s.page_size <= 0 || s.max_pages <= 0 || s.n_pages <= 0)
    return refuse(SMQA_ERR_INVALID_ARG, "non-positive size in paged shape");
  if (s.H > 128 || (s.D != 64 && s.D != 128) || shift_of(s.page_size) < 4 ||
      static_cast<int64_t>(s.n_pages) * s.page_size >= kLim ||
      static_cast<int64_t>(s.max_pages) * s.page_size > kLim - 256)
    return refuse(SMQA_ERR_UNSUPPORTED,
                  "unsupported paged indexer shape (need 1<=H<=128, D in {64,128}, page_size in {16,32,64,128}, "
                  "n_pages * page_size < 2^31, max_pages * page_size <= 2^31 - 256)");
  return SMQA_OK;
}

// Key rows as 8-bit or bf16 boxes of `box_rows` rows, swizzled as the tensor core reads them.
bool encode_keys(CUtensorMap* m, const void* ptr, bool codes, int D, uint64_t rows, uint32_t box_rows) {
  const auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!fn) {
    set_last_error("cuTensorMapEncodeTiled unavailable");
    return false;
  }
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), rows};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * (codes ? 1 : 2)};
  const cuuint32_t box[2] = {codes ? static_cast<cuuint32_t>(D) : 64u, box_rows}, estr[2] = {1, 1};
  const CUresult r = fn(m, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        codes && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) set_last_error("cuTensorMapEncodeTiled failed");
  return r == CUDA_SUCCESS;
}

// The chunks of one call, one after another.
smqa_status run_topk(TopkParams p, const TopkPlan& pl, const CUtensorMap& tm, int D, bool paged, int64_t per_batch_units,
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
    e = launch_topk_score(tm, p, D, paged, stream);
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
  CUtensorMap tm;
  if (!encode_keys(&tm, index_k, false, s.D, static_cast<uint64_t>(s.B) * s.S_kv, kTile)) return SMQA_ERR_CUDA;
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
  return run_topk(p, pl, tm, s.D, false, (s.S + group_tokens(s.H) - 1) / group_tokens(s.H), workspace, stream);
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
  return run_topk(p, pl, tm, s.D, true, pl.units, workspace, stream);
}

}  // extern "C"

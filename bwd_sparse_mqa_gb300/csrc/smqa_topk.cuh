// smqa_topk.cuh -- what the two kernels of the indexer's selection share: their
// parameters, the visible length of a token, the order of scores as integers,
// and the two e4m3 pieces of a query.
#pragma once

#include "smqa_internal.h"
#include "smqa_paged.cuh"

namespace smqa {

// One call, or one chunk of its tokens.  Contiguous: token t = b * S + s, keys
// bf16 [B, S_kv, D].  Paged: token t of request token_req[t], keys e4m3
// [n_pages, page, D] with one scale per page.
struct TopkParams {
  const __nv_bfloat16* q;    // [T, H, D]
  const float* w;            // [T, H]
  const __nv_bfloat16* k;    // contiguous
  const uint8_t* codes;      // paged
  const float* scales;       // [n_pages]
  const int32_t* table;      // [R, max_pages]
  const int32_t* seq_lens;   // [R]
  const int32_t* token_req;  // [T]
  const int32_t* positions;  // [T] (null: a token sees its request's whole length)
  int T, H, S, S_kv, B;
  int R, max_pages, n_pages, page_shift;
  int64_t first;             // position of a batch element's query 0
  int topk, block_shift, recent;
  int64_t unit0, units;      // groups of consecutive tokens (of one batch element): the chunk's first, and their number
  int64_t tok0, toks;        // the chunk's tokens
  int64_t ld;                // entries of a token's row of scores
  int64_t norm_ld;           // bounds of a token's rows (paged), or a batch element's
  int32_t* rows;             // [toks][ld] scores as ordered integers, of entry_rows rows each
  float* norms;              // [toks or B][norm_ld] upper bounds of the key rows' lengths, one per 32 rows
  int32_t* out;              // [T, topk]
  int zero_padding;
  int* status;
  uint64_t limit_ns;
  int stall_cta;
};

constexpr int kTile = 128;               // key rows per tile of the score kernel

// Rows of an entry of the score rows: a block of up to 32 positions has one
// entry, a larger one several (a warp's 32 lanes hold 32 rows).
__host__ __device__ inline int entry_shift(int block_shift) { return block_shift < 5 ? block_shift : 5; }

// Query heads of a token in the score kernel's tile, and tokens of a group.
inline int padded_heads(int H) { return H <= 16 ? 16 : H <= 32 ? 32 : H <= 64 ? 64 : 128; }
inline int group_tokens(int H) { return 256 / padded_heads(H); }

// (tm_q: contiguous keys only.)
cudaError_t launch_topk_score(const CUtensorMap& tm_k, const CUtensorMap& tm_q, const TopkParams& p, int D, bool paged, cudaStream_t stream);
cudaError_t launch_topk_select(const TopkParams& p, int D, bool paged, cudaStream_t stream);

// Scores as integers that order like them, equal ones (0 and -0) alike; a NaN
// ranks below every number, what is not to be chosen below that, and a position
// that is always chosen above every number.
constexpr int32_t kKeyNever = INT32_MIN, kKeyNan = INT32_MIN + 1, kKeyAlways = INT32_MAX;
constexpr int32_t kKeyInf = 0x7f800000;
__device__ __forceinline__ int32_t key_of(float x) {
  const int32_t b = __float_as_int(x + 0.f);
  return x != x ? kKeyNan : b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float value_of(int32_t key) { return __int_as_float(key ^ ((key >> 31) & 0x7fffffff)); }

// Rows token t sees (0: none, or a padding token), and its request or batch element.
template <bool kPaged>
__device__ __forceinline__ int visible(const TopkParams& p, int64_t t, int& req) {
  if constexpr (kPaged) {
    req = load(p.token_req + t);
    if (static_cast<unsigned>(req) >= static_cast<unsigned>(p.R)) {
      req = -1;
      return 0;
    }
    int64_t n = load(p.seq_lens + req);
    if (p.positions) n = min(n, static_cast<int64_t>(load(p.positions + t)) + 1);
    n = min(n, static_cast<int64_t>(p.max_pages) << p.page_shift);
    return static_cast<int>(max(n, static_cast<int64_t>(0)));
  } else {
    req = static_cast<int>(t / p.S);
    const int64_t n = p.first + (t - static_cast<int64_t>(req) * p.S) + 1;
    return static_cast<int>(max(static_cast<int64_t>(0), min(n, static_cast<int64_t>(p.S_kv))));
  }
}

// A query row's largest magnitude m (as bf16 bits) sets a power of two 2^k with
// 2^k m in [128, 256) (k = 126 at most: a normal number).
__device__ __forceinline__ int query_exponent(uint32_t m) { return min(7 - (static_cast<int>(m >> 7) - 127), 126); }
// Two elements x 2^k as two e4m3 pieces: hi the nearest code, lo that of the rest.
// Together they hold bf16's 8 bits down to 2^-9, which is 2^-17 of m.
__device__ __forceinline__ void split_query(float2 x, uint16_t& hi, uint16_t& lo) {
  hi = e4m3x2(x.x, x.y);
  const float2 h = e4m3x2_value(hi);
  lo = e4m3x2(x.x - h.x, x.y - h.y);
}

}  // namespace smqa

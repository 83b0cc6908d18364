// smqa_paged.cuh -- building blocks of the 8-bit paged cache's kernels: e4m3
// conversions, tcgen05 MMAs on e4m3 operands (plain and block-scaled), TMEM
// accesses, and the start-up beside the kernel before.
#pragma once

#include "smqa_ptx.cuh"

namespace smqa {

// Two values -> two e4m3 codes (nearest even, saturating), `lo` in the low byte.
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// The values of two codes (exact).
__device__ __forceinline__ __half2 e4m3x2_half2(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return *reinterpret_cast<__half2*>(&h);
}
__device__ __forceinline__ float2 e4m3x2_value(uint16_t v) { return __half22float2(e4m3x2_half2(v)); }

// Instruction descriptor for kind::f8f6f4 with e4m3 A/B (format 0) and an fp32
// accumulator; the other fields are those of idesc_bf16_f32.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N, bool a_mn_major) {
  return (1u << 4) | (static_cast<uint32_t>(a_mn_major) << 15) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// As mma_ss / mma_ts / mma_commit, on e4m3 operands (32 elements of K per
// instruction; a TMEM A holds four elements per 32-bit column), called by a
// whole converged warp of which one lane issues: descriptors stay in uniform
// registers, where a branch on the lane moves six of them there for every
// instruction.
__device__ __forceinline__ void mma8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void mma8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

// Instruction descriptor for kind::mxf8f6f4: e4m3 A/B, an fp32 accumulator and
// ue8m0 scale factors (a power of two by its exponent's bits), one per row of A
// and of B and 32 elements of K: B's is byte `b_byte` of its row's word in TMEM,
// A's byte 0.  Rows of a factor go by lane (row mod 32, the same in all four
// lane quarters) and column (row / 32).
__host__ __device__ constexpr uint32_t idesc_mx_e4m3_f32(int M, int N, bool a_mn_major, int b_byte) {
  return (static_cast<uint32_t>(b_byte) << 4) | (static_cast<uint32_t>(a_mn_major) << 15) |
         (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 7) << 27);
}
// A kept in the tensor core's collector, and the A that the instruction before
// left there (the same descriptor): its bytes are read from shared memory once
// for both.
__device__ __forceinline__ void mma_mx_ss_keep(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t a_scale, uint32_t b_scale,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X.collector::a::fill "
      "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate));
}
__device__ __forceinline__ void mma_mx_ss_again(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t a_scale, uint32_t b_scale,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X.collector::a::lastuse "
      "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate));
}
__device__ __forceinline__ void mma_commit_elect(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          bar)
      : "memory");
}

// 16 lanes x 64 columns, four times: lanes 0-15 and 16-31 of the warp's quarter
// (a, b), columns from t and from t + 64 (the first and last 32 of a and b), one
// wait.  Thread i of the warp gets, for each group j of eight columns, lane i / 4
// at columns 8j + 2 (i mod 4) and the next (v[4j], v[4j+1]) and lane i / 4 + 8 at
// the same columns (v[4j+2], v[4j+3]).
__device__ __forceinline__ void tmem_ld16x128x2(uint32_t t, float (&a)[64], float (&b)[64]) {
  uint32_t r0[32], r1[32], s0[32], s1[32];
  const uint32_t u = t + (16u << 16);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%128];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%129];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, %80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95}, [%130];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, %112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%131];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r0[0]), "=r"(r0[1]), "=r"(r0[2]), "=r"(r0[3]), "=r"(r0[4]), "=r"(r0[5]), "=r"(r0[6]), "=r"(r0[7]), "=r"(r0[8]), "=r"(r0[9]), "=r"(r0[10]), "=r"(r0[11]), "=r"(r0[12]), "=r"(r0[13]), "=r"(r0[14]), "=r"(r0[15]), "=r"(r0[16]), "=r"(r0[17]), "=r"(r0[18]), "=r"(r0[19]), "=r"(r0[20]), "=r"(r0[21]), "=r"(r0[22]), "=r"(r0[23]), "=r"(r0[24]), "=r"(r0[25]), "=r"(r0[26]), "=r"(r0[27]), "=r"(r0[28]), "=r"(r0[29]), "=r"(r0[30]), "=r"(r0[31]),
        "=r"(s0[0]), "=r"(s0[1]), "=r"(s0[2]), "=r"(s0[3]), "=r"(s0[4]), "=r"(s0[5]), "=r"(s0[6]), "=r"(s0[7]), "=r"(s0[8]), "=r"(s0[9]), "=r"(s0[10]), "=r"(s0[11]), "=r"(s0[12]), "=r"(s0[13]), "=r"(s0[14]), "=r"(s0[15]), "=r"(s0[16]), "=r"(s0[17]), "=r"(s0[18]), "=r"(s0[19]), "=r"(s0[20]), "=r"(s0[21]), "=r"(s0[22]), "=r"(s0[23]), "=r"(s0[24]), "=r"(s0[25]), "=r"(s0[26]), "=r"(s0[27]), "=r"(s0[28]), "=r"(s0[29]), "=r"(s0[30]), "=r"(s0[31]),
        "=r"(r1[0]), "=r"(r1[1]), "=r"(r1[2]), "=r"(r1[3]), "=r"(r1[4]), "=r"(r1[5]), "=r"(r1[6]), "=r"(r1[7]), "=r"(r1[8]), "=r"(r1[9]), "=r"(r1[10]), "=r"(r1[11]), "=r"(r1[12]), "=r"(r1[13]), "=r"(r1[14]), "=r"(r1[15]), "=r"(r1[16]), "=r"(r1[17]), "=r"(r1[18]), "=r"(r1[19]), "=r"(r1[20]), "=r"(r1[21]), "=r"(r1[22]), "=r"(r1[23]), "=r"(r1[24]), "=r"(r1[25]), "=r"(r1[26]), "=r"(r1[27]), "=r"(r1[28]), "=r"(r1[29]), "=r"(r1[30]), "=r"(r1[31]),
        "=r"(s1[0]), "=r"(s1[1]), "=r"(s1[2]), "=r"(s1[3]), "=r"(s1[4]), "=r"(s1[5]), "=r"(s1[6]), "=r"(s1[7]), "=r"(s1[8]), "=r"(s1[9]), "=r"(s1[10]), "=r"(s1[11]), "=r"(s1[12]), "=r"(s1[13]), "=r"(s1[14]), "=r"(s1[15]), "=r"(s1[16]), "=r"(s1[17]), "=r"(s1[18]), "=r"(s1[19]), "=r"(s1[20]), "=r"(s1[21]), "=r"(s1[22]), "=r"(s1[23]), "=r"(s1[24]), "=r"(s1[25]), "=r"(s1[26]), "=r"(s1[27]), "=r"(s1[28]), "=r"(s1[29]), "=r"(s1[30]), "=r"(s1[31])
      : "r"(t), "r"(u), "r"(t + 64), "r"(u + 64)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    a[i] = __uint_as_float(r0[i]);
    a[32 + i] = __uint_as_float(r1[i]);
    b[i] = __uint_as_float(s0[i]);
    b[32 + i] = __uint_as_float(s1[i]);
  }
}
// The same layout, 32 columns of both halves of the quarter.
__device__ __forceinline__ void tmem_ld16x32x2(uint32_t t, float (&a)[16], float (&b)[16]) {
  uint32_t r[16], s[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(s[0]), "=r"(s[1]), "=r"(s[2]), "=r"(s[3]), "=r"(s[4]), "=r"(s[5]), "=r"(s[6]), "=r"(s[7]), "=r"(s[8]), "=r"(s[9]), "=r"(s[10]), "=r"(s[11]), "=r"(s[12]), "=r"(s[13]), "=r"(s[14]), "=r"(s[15])
      : "r"(t), "r"(t + (16u << 16))
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    a[i] = __uint_as_float(r[i]);
    b[i] = __uint_as_float(s[i]);
  }
}
// Four 8 x 8 matrices of 16-bit pairs, transposed: a thread's register holds
// rows 2 (i mod 4), + 1 at column i / 4; `addr` is the address of row i mod 8 of
// matrix i / 8.
__device__ __forceinline__ void stmatrix_trans_x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

// One 32-bit column of the warp's 32 lanes at N places (1 or 4), `step` columns
// apart; one wait.
template <int N, int kStep>
__device__ __forceinline__ void tmem_ld1xn(uint32_t t, float (&v)[N]) {
  static_assert(N == 1 || N == 4, "tmem_ld1xn: one or four columns");
  uint32_t r[4] = {};
  if constexpr (N == 4)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%4];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%1}, [%5];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%2}, [%6];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%3}, [%7];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(t), "r"(t + kStep), "r"(t + 2 * kStep), "r"(t + 3 * kStep)
        : "memory");
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0])
        : "r"(t)
        : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}
// (Stores: tmem_wait_st waits for them.)
__device__ __forceinline__ void tmem_st1(uint32_t t, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(t), "r"(__float_as_uint(v)) : "memory");
}
// Four and eight consecutive columns from this thread's lane.
__device__ __forceinline__ void tmem_st4u(uint32_t t, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(t), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void tmem_st8u(uint32_t t, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Registers per thread of the calling warpgroup from here on (all its warps
// call it).
template <int N>
__device__ __forceinline__ void reg_alloc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dealloc() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Barrier `id` over `threads` threads (whole warps).
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Loads of what the kernel before may have written: through L1, but not by its
// read-only path, which is for data that nothing writes while this kernel lives.
// (As PTX: with the compiler's own plain loads, which it keeps behind every store
// and barrier, the attention of 1024 tokens took 509 us, not 500; with loads past L1
// that of 111 dense ones 26.4, not 23.5.)
__device__ __forceinline__ int load(const int* p) {
  int v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float load(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 load(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// cp.async of 16 bytes, or of 16 zero bytes (nothing is read then).
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool copy) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(copy ? 16u : 0u)
               : "memory");
}

// Programmatic dependent launch: lets the kernel behind start (its blocks take
// what room there is), and, in that one, waits until the kernel before has
// completed and its writes are visible.
__device__ __forceinline__ void grid_dependents_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace smqa

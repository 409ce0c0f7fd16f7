// Building blocks of the tcgen05 attention kernels.
//
// A block holds 128 resident rows and streams tiles of 64 rows of the other
// side.  Warps 0-3 and 4-7 (two groups of 128 threads, one resident row per
// thread) take the stream tiles in turn; warp 8 issues the matrix products;
// warps 9-11 bring in the stream tiles by tiled TMA.  A tile is stored as
// panels of 64 values (128 bytes) per row with the 128-byte swizzle: chunk c of
// 16 bytes of row r sits at r 128 + (c ^ r%8) 16.  That serves both as a
// K-major operand (rows = M or N, the head dimension contracted) and as an
// MN-major one (the head dimension = N, rows contracted), so that keys and
// values are stored once.  Structures begin and end at any row and senders may
// be hidden: the copying warp overwrites such rows of a tile with zeros before
// it hands the tile on (0 x NaN).
//
// Every wait is bounded, as in the ladder's kernels; a wait that gives up sets
// the error word that fc_device_error reads.
#pragma once
#include <cuda.h>

#include "fc_attention.cuh"
#include "fc_device.cuh"

namespace fc {

constexpr int kAtRows = 128, kAtStep = 64, kAtThreads = 384;
constexpr int kAtCopiers = 3;             // copying warps: 9, 10, 11
constexpr uint32_t kAtPanel = kAtStep * 128;   // bytes of a stream tile's panel
constexpr uint64_t kAtDrainNs = 2000000000ull;

// Instruction descriptor: F32 accumulator, A and B of one 16-bit type, A
// K-major, B K-major or MN-major.
template <class T>
__device__ __forceinline__ uint32_t at_idesc(int n, bool b_mn) {
  const uint32_t f = __is_same(T, __half) ? 0u : 1u;
  return (1u << 4) | (f << 7) | (f << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kAtRows >> 4) << 24);
}
// True in one thread of the (whole) warp.  Inside `if (elect_one())` the
// compiler knows that one thread runs and issues each product in some 50
// cycles; under `if (lane == 0)` it took 100 to 150 (64 x 128 x 16 products
// back to back, where the tensor core needs 32 to 64).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(p));
  return p != 0;
}
// D[tmem] (+)= A[smem] B[smem]^T
__device__ __forceinline__ void mma_ss16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
      :
      : "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// D[tmem] (+)= A[tmem] B[smem]: A is 128 rows, two 16-bit values per column
__device__ __forceinline__ void mma_ts16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
      :
      : "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate));
}

// Whole warp: 32 columns of each thread's TMEM lane; the values are there
// after tmem_wait_ld on the same array (which ties them to the wait).
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29])
               :
               : "memory");
  asm volatile("" : "+r"(r[30]), "+r"(r[31]) : : "memory");
}
__device__ __forceinline__ float2 pair_at(const uint32_t (&r)[32], int e) {
  return make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
}
// Four rows of a panel: lane/8 of the rows, 16-byte chunk lane%8; dead rows and
// chunks past the head become zeros.  dst: the panel's address at the first row.
__device__ __forceinline__ void copy_rows4(uint32_t dst, int row, int lane, const void* src, bool live) {
  const int r = row + (lane >> 3);
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               :
               : "r"(dst + r * 128 + (((lane & 7) ^ (r & 7)) << 4)), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
// Zeros one row of a panel (16 bytes per lane of eight).
__device__ __forceinline__ void zero_row(uint32_t panel, int r, int lane) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" : : "r"(panel + r * 128 + (lane & 7) * 16), "r"(0) : "memory");
}
// Tiled TMA copy of one panel: 64 values of the head dimension from x on, head
// h, 64 rows from row on; values and rows past the array are zeros.
__device__ __forceinline__ void load_panel(uint32_t dst, const CUtensorMap* map, int x, int h, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      :
      : "r"(dst), "l"(map), "r"(x), "r"(h), "r"(row), "r"(tc::smem_addr(bar))
      : "memory");
}
// [rows][heads][D] of 16-bit values, row step ld, as {D, heads, rows}; the box
// is one panel: `group` heads of 64 / group rows (rounded down).  False if the
// driver refuses it.
bool at_tensor_map(CUtensorMap* m, bool half, const void* base, int D, int heads, long long ld, int rows, int group = 1);

// Descriptors (128-byte swizzle) of a tile whose panels have R rows, from byte
// address a, and their 16-value or 16-row steps.
constexpr uint64_t kSwizzle128 = 2ull << 61;
template <int R>
__device__ __forceinline__ uint64_t desc_k(uint32_t a) {
  return tc::smem_desc(a, 16, 1024) | kSwizzle128;
}
template <int R>
__device__ __forceinline__ constexpr uint64_t step_k(int k) {
  return (uint64_t)((k >> 2) * R * 128 + (k & 3) * 32) >> 4;
}
template <int R>
__device__ __forceinline__ uint64_t desc_mn(uint32_t a) {
  return tc::smem_desc(a, R * 128, 1024) | kSwizzle128;
}
__device__ __forceinline__ constexpr uint64_t step_mn(int k) { return (uint64_t)(k * 2048) >> 4; }

__device__ __forceinline__ float2 pair(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 lds2(const float* p) { return *reinterpret_cast<const float2*>(p); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// largest of 2 N values, in four chains
template <int N>
__device__ __forceinline__ float max_pairs(const float2 (&x)[N]) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < N; ++i) m[i & 3] = max3(m[i & 3], x[i].x, x[i].y);
  return max3(fmaxf(m[0], m[1]), m[2], m[3]);
}

// f tanh(mul s) / s for |mul s| <= 0.6, as a polynomial in s^2 with the powers of
// mul in its coefficients (degree 4, least largest relative error, fitted to
// tanh(x)/x; 9.1e-8 with FP32 coefficients).  The FP32 pipe is what the score arithmetic fills first, so
// the narrower range of strip_tanh's 0.8 is given for two operations less.
constexpr float kAtTanhMax = 0.6f;
struct TanhPoly {
  float2 c[5];
  float lim;   // of |s|; where a coefficient under- or overflows there is no range
  __device__ __forceinline__ TanhPoly(float f, float mul) {
    const float k[5] = {0.9999999403953552f, -0.33332309126853943f, 0.13310173153877258f, -0.05210148170590401f,
                        0.015475427731871605f};
    const float m2 = mul * mul;
    float p = f * mul;
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      c[i] = pair(p * k[i]);
      p *= m2;
    }
    const float lo = fminf(fabsf(c[0].x), fabsf(c[4].x)), hi = fmaxf(fabsf(c[0].x), fabsf(c[4].x));
    lim = lo > 1e-37f && hi < 1e37f ? kAtTanhMax / fabsf(mul) : -1.0f;
  }
  __device__ __forceinline__ float2 operator()(float2 z) const {
    float2 p = fma2(z, c[4], c[3]);
    p = fma2(z, p, c[2]);
    p = fma2(z, p, c[1]);
    return fma2(z, p, c[0]);
  }
};
}  // namespace fc

// Building blocks of the node attention kernels: tile lookup in a batch of
// structures, asynchronous tile loads, warp-level matrix products on 16-row
// strips, and the score of a pair.
//
// Rows of a tile.  The receivers of a structure and the G heads that share one
// key head form "virtual rows" v = i G + g, so that keys and values are read
// once for the group.  A tile never crosses structures: zero weights times the
// rows of another structure would carry its NaN over.
#pragma once
#include "fc_nodes.cuh"
#include "fc_tc.cuh"

namespace fc {

struct AttnArgs {
  int B, nr, ns, H, KV, G, D;
  float scale, cap;
  long long ldq, ldk, ldv, ldo, ldg;
  const int32_t *recv_ptr, *send_ptr;
  const void *q, *k, *v, *g;
  const float *pos_r, *pos_s, *slope;   // pos_s is never NULL when pos_r is not
  const uint8_t* mask;
  void* out;
  float *lse, *o32;
  int splits;           // parts of the key range
  float* part;          // [splits][nr H][D] partial rows
  float2* part_ml;      // forward: [splits][nr H] maximum and sum
  const float2* stat;   // gradient: [nr H] log-sum (base 2), delta
  float4* rowpart;      // gradient: [splits][nr H] position and slope sums
  float4* rowmean;      // 16-bit gradient: the same sums of the weights alone, and
  float* rowrest;       // the row's sum of dt, which an exact delta makes 0
  float4* colpart;      // gradient: [kv_splits][KV][ns] position sums
  int kv_splits;        // parts of the receivers (key and value gradients)
  float *part_k, *part_v;   // [kv_splits][ns KV][D] partial rows
  void *qb, *kb, *vb;
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rsq(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh of a score over its cap.  FP32 rows take the library function; for
// 16-bit rows 1 - 2 / (1 + e^{2x}) is enough (absolute error about 1e-7).
template <class T>
__device__ __forceinline__ float cap_tanh(float x) {
  if constexpr (sizeof(T) == 4)
    return tanhf(x);
  else
    return 1.0f - 2.0f * rcp(1.0f + ex2(2.0f * kLog2e * x));
}

// Squared distances carry 1e-36 where they are inverted, so that a coincident
// pair has a finite inverse (its distance is then 0, its direction 0).
constexpr float kD2Seed = 1e-36f;

// tanh of scores over the cap for |x| <= 0.8 as x P(x^2): degree 5, least
// largest relative error (fitted to tanh(x)/x); with its FP32 coefficients
// 6.7e-8, about one FP32 rounding.
constexpr float kTanhMax = 0.8f;
__host__ __device__ constexpr float tanh_c(int i) {
  return i == 0   ? 0.9999999403953552f
         : i == 1 ? -0.3333267569541931f
         : i == 2 ? 0.13321048021316528f
         : i == 3 ? -0.05311431363224983f
         : i == 4 ? 0.01909329928457737f
                  : -0.004355299286544323f;
}
__device__ __forceinline__ float tanh_poly(float x) {
  const float z = x * x;
  float p = tanh_c(5);
#pragma unroll
  for (int i = 4; i >= 0; --i) p = fmaf(z, p, tanh_c(i));
  return x * p;
}
// s = tanh(s mul) of a strip.  Scores are a fraction of the cap nearly always:
// the polynomial then spares the special-function unit; a warp that holds a
// larger one takes cap_tanh.
template <class T, int NT>
__device__ __forceinline__ void strip_tanh(float (&s)[NT][4], float mul) {
  float m = 0.0f;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[n][e] *= mul;
      m = fmaxf(m, fabsf(s[n][e]));
    }
  if (__any_sync(0xffffffffu, !(m <= kTanhMax))) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = cap_tanh<T>(s[n][e]);
  } else {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = tanh_poly(s[n][e]);
  }
}

// Tile t of the rows of all structures, `mult` virtual rows per row and `tile`
// virtual rows per tile.  The rows before the first structure and after the
// last count as two more structures (0 and B + 1), which have nothing on the
// other side.  Structure b owns the tile numbers from
// floor(start_b mult / tile) + b on; these ranges are disjoint, so that the
// structure follows from a search in ptr alone.  Every lane of a warp calls.
constexpr int kMaxStruct = INT32_MAX - 64;   // the search looks up to 31 past structure B + 1
struct TileAt {
  int b;               // structure, 0 .. B + 1
  long long v0, v1;    // virtual rows from the tile's first to the structure's end
};
__device__ __forceinline__ int clamp_row(int v, int n) { return v < 0 ? 0 : v > n ? n : v; }
// first row of structure b (0 .. B + 2)
__device__ __forceinline__ int row_bound(const int32_t* __restrict__ ptr, int B, int n, int b) {
  return b == 0 ? 0 : b == B + 2 ? n : clamp_row(ptr[b - 1], n);
}
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ ptr, int B, int n, int mult, int tile, int t,
                                          TileAt& out) {
  const int lane = threadIdx.x & 31;
  auto slot = [&](int b) { return (long long)row_bound(ptr, B, n, b) * mult / tile + b; };
  int lo = 0, hi = B + 2;
  for (;;) {
    const int step = (hi - lo + 31) / 32;
    const int b = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, b < hi && slot(b < hi ? b : lo) <= t);
    const int cnt = le == 0xffffffffu ? 32 : __ffs(~le) - 1;
    if (cnt == 0) return false;
    lo += (cnt - 1) * step;
    hi = lo + step < hi ? lo + step : hi;
    if (step == 1) break;
  }
  out.b = lo;
  out.v0 = (long long)row_bound(ptr, B, n, lo) * mult + (long long)(t - slot(lo)) * tile;
  out.v1 = (long long)row_bound(ptr, B, n, lo + 1) * mult;
  return out.v0 < out.v1;
}
// rows of structure b on the other side
__device__ __forceinline__ void other_side(const int32_t* __restrict__ ptr, int B, int n, int b, int& lo, int& hi) {
  const bool real = b >= 1 && b <= B;
  lo = real ? clamp_row(ptr[b - 1], n) : 0;
  hi = real ? clamp_row(ptr[b], n) : 0;
}
// upper bound of the tile count
inline long long tile_slots(int B, int n, int mult, int tile) { return (long long)n * mult / tile + B + 2; }

// ------------------------------------------------------------------- copies

__device__ __forceinline__ void cp16(void* dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" : : "r"(tc::smem_addr(dst)), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" : : "n"(N) : "memory");
}

__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Row stride of a shared tile in values: 16 bytes more than the row, so that
// eight rows at one column start in eight different 16-byte bank groups.
template <class T, int DP>
constexpr int kStride = DP + 16 / (int)sizeof(T);

// ROWS rows of head_dim values, zeros beyond the head and in rows that `live`
// refuses; row r comes from src(r).
template <class T, int DP, int ROWS, int THREADS, class Src, class Live>
__device__ __forceinline__ void load_rows(T* tile, int D, int tid, Src src, Live live) {
  constexpr int VEC = 16 / sizeof(T), CH = DP / VEC;
#pragma unroll 4
  for (int i = tid; i < ROWS * CH; i += THREADS) {
    const int r = i / CH, c = (i - r * CH) * VEC;
    const bool ok = c < D && live(r);
    const T* p = src(ok ? r : 0);
    cp16(tile + r * kStride<T, DP> + c, p + (ok ? c : 0), ok);
  }
}

// The same for two arrays that share `live` (keys and values): its loads go out
// together, ahead of the copies they decide on.
template <class T, int DP, int ROWS, int THREADS, class Src1, class Src2, class Live>
__device__ __forceinline__ void load_rows2(T* tile1, T* tile2, int D, int tid, Src1 src1, Src2 src2, Live live) {
  constexpr int VEC = 16 / sizeof(T), CH = DP / VEC, U = 8;
#pragma unroll 1
  for (int i0 = tid; i0 < ROWS * CH; i0 += U * THREADS) {
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * THREADS, r = i / CH;
      ok[u] = i < ROWS * CH && (i - r * CH) * VEC < D && live(r);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * THREADS;
      if (i >= ROWS * CH) break;
      const int r = i / CH, c = (i - r * CH) * VEC;
      cp16(tile1 + r * kStride<T, DP> + c, src1(ok[u] ? r : 0) + (ok[u] ? c : 0), ok[u]);
      cp16(tile2 + r * kStride<T, DP> + c, src2(ok[u] ? r : 0) + (ok[u] ? c : 0), ok[u]);
    }
  }
}

// ----------------------------------------------------------------- products

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(tc::smem_addr(p)));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(tc::smem_addr(p)));
}
template <class T>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (sizeof(T) == 2) {
    if constexpr (__is_same(T, __half))
      asm volatile(
          "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
          : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
          : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
      asm volatile(
          "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
          : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
          : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}
__device__ __forceinline__ void mma8(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Accumulator fragment of a 16 x 8 NT strip: element e of tile n is row
// lane/4 + 8 (e/2), column 8 n + 2 (lane%4) + e%2.

// s = A B^T over DP: 16 rows at a, 8 NT rows at b, both in shared tiles; column
// tiles from nl on are not there and stay 0.  FP32 rows as three TF32 products
// (hi lo, lo hi, hi hi), error near 2^-21.  The tensor core truncates every
// step of its sum (measured: steps below one unit in the last place add
// nothing), so the FP32 sums are taken out every 32 values and added in FP32,
// the small products in a sum of their own.
template <class T, int DP, int NT>
__device__ __forceinline__ void strip_nt(float (&s)[NT][4], const T* a, const T* b, int nl) {
  constexpr int S = kStride<T, DP>;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
  if constexpr (sizeof(T) == 2) {
    const T* pa = a + (lane & 15) * S + (lane >> 4) * 8;
    const T* pb = b + ((lane & 7) + ((lane >> 4) << 3)) * S + ((lane >> 3) & 1) * 8;
#pragma unroll
    for (int k = 0; k < DP; k += 16) {
      uint32_t fa[4];
      ldsm4(fa, pa + k);
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        if (n >= nl) break;
        uint32_t fb[4];
        ldsm4(fb, pb + n * 8 * S + k);
        mma16<T>(s[n], fa, fb[0], fb[1]);
        mma16<T>(s[n + 1], fa, fb[2], fb[3]);
      }
    }
  } else {
    const int g = lane >> 2, t = lane & 3;
    const float* pa = a + g * S + t;
    const float* pb = b + g * S + t;
    constexpr int KC = DP < 32 ? DP : 32;
#pragma unroll 1
    for (int k0 = 0; k0 < DP; k0 += KC) {
      uint32_t hi[KC / 8][4], lo[KC / 8][4];
#pragma unroll
      for (int k = 0; k < KC / 8; ++k) {
        const float* p = pa + k0 + 8 * k;
        tc::split_tf32(p[0], hi[k][0], lo[k][0]);
        tc::split_tf32(p[8 * S], hi[k][1], lo[k][1]);
        tc::split_tf32(p[4], hi[k][2], lo[k][2]);
        tc::split_tf32(p[8 * S + 4], hi[k][3], lo[k][3]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n >= nl) break;
        float big[4] = {0.f, 0.f, 0.f, 0.f}, small[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KC / 8; ++k) {
          uint32_t h0, l0, h1, l1;
          tc::split_tf32(pb[n * 8 * S + k0 + 8 * k], h0, l0);
          tc::split_tf32(pb[n * 8 * S + k0 + 8 * k + 4], h1, l1);
          mma8(small, hi[k], l0, l1);
          mma8(big, hi[k], h0, h1);
          mma8(small, lo[k], h0, h1);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] += big[e] + small[e];
      }
    }
  }
}

// acc = alpha acc + P B: P the 16 x 8 NT strip, B 8 NT rows of a shared tile, of
// which the column tiles (rows) from nl on are not there.  Each call sums into
// a fresh fragment that is added to acc in FP32, for the same reason.  Two:
// 16-bit P as two terms (its rounding error and that again), else one rounding
// to 16 bits, half a unit of 2^-8 (BF16) or 2^-11 (FP16) per weight, which
// averages over the row.
template <class T, int DP, int NT, bool Two>
__device__ __forceinline__ void strip_pn(float (&acc)[DP / 8][4], const float (&p)[NT][4], const T* b, float alpha0,
                                         float alpha1, int nl) {
  constexpr int S = kStride<T, DP>;
  const int lane = threadIdx.x & 31;
  if constexpr (sizeof(T) == 2) {
    uint32_t fa[NT / 2][4], fl[Two ? NT / 2 : 1][4];
#pragma unroll
    for (int n = 0; n < NT; n += 2)
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float x = p[n + (h >> 1)][2 * (h & 1)], y = p[n + (h >> 1)][2 * (h & 1) + 1];
        fa[n / 2][h] = pack2<T>(x, y);
        if constexpr (Two)
          fl[n / 2][h] = pack2<T>(x - RowType<T>::to(RowType<T>::from(x)), y - RowType<T>::to(RowType<T>::from(y)));
      }
    const T* pb = b + ((lane & 7) + ((lane >> 3) & 1) * 8) * S + (lane >> 4) * 8;
#pragma unroll
    for (int d = 0; d < DP / 8; d += 2) {
      float f0[4] = {0.f, 0.f, 0.f, 0.f}, f1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        if (n >= nl) break;
        uint32_t fb[4];
        ldsm4t(fb, pb + n * 8 * S + d * 8);
        if constexpr (Two) {
          mma16<T>(f0, fl[n / 2], fb[0], fb[1]);
          mma16<T>(f1, fl[n / 2], fb[2], fb[3]);
        }
        mma16<T>(f0, fa[n / 2], fb[0], fb[1]);
        mma16<T>(f1, fa[n / 2], fb[2], fb[3]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[d][e] = fmaf(acc[d][e], e < 2 ? alpha0 : alpha1, f0[e]);
        acc[d + 1][e] = fmaf(acc[d + 1][e], e < 2 ? alpha0 : alpha1, f1[e]);
      }
    }
  } else {
    // k slot t of the product is row 2t, slot t + 4 row 2t + 1: the layout that P already has
    const int g = lane >> 2, t = lane & 3;
    const float* pb = b + 2 * t * S + g;
    constexpr int DC = DP / 8 < 4 ? DP / 8 : 4;
#pragma unroll
    for (int d = 0; d < DP / 8; d += DC) {
      float f[DC][4], fs[DC][4];
#pragma unroll
      for (int i = 0; i < DC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) f[i][e] = fs[i][e] = 0.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n >= nl) break;
        uint32_t hi[4], lo[4];
        tc::split_tf32(p[n][0], hi[0], lo[0]);
        tc::split_tf32(p[n][2], hi[1], lo[1]);
        tc::split_tf32(p[n][1], hi[2], lo[2]);
        tc::split_tf32(p[n][3], hi[3], lo[3]);
#pragma unroll
        for (int i = 0; i < DC; ++i) {
          uint32_t h0, l0, h1, l1;
          tc::split_tf32(pb[n * 8 * S + (d + i) * 8], h0, l0);
          tc::split_tf32(pb[(n * 8 + 1) * S + (d + i) * 8], h1, l1);
          mma8(fs[i], hi, l0, l1);
          mma8(f[i], hi, h0, h1);
          mma8(fs[i], lo, h0, h1);
        }
      }
#pragma unroll
      for (int i = 0; i < DC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[d + i][e] = fmaf(acc[d + i][e], e < 2 ? alpha0 : alpha1, f[i][e] + fs[i][e]);
    }
  }
}

// Keys (or rows) of one product step: 64, and 32 for wide FP32 heads, whose
// tiles are twice the bytes.
template <class T, int DP>
constexpr int kStep = sizeof(T) == 4 && DP > 64 ? 32 : 64;

// How a call runs (fc_attention.cu): on the tcgen05 kernels or the strip
// kernels, and in how many parts of the senders (forward, query gradient) or
// of the receivers (key and value gradients).
struct AttnPlan {
  bool tc, few, tc_vjp;
  int splits, q_splits, kv_splits;
};
int check_attn(const fc_attn_desc* d, int n_struct, int n_recv, int n_send);
AttnPlan attn_plan(const fc_attn_desc* d, int n_struct, int n_recv, int n_send);
int attn_pad(int head_dim);
// fc_attention_tc.cu: 16-bit types
int launch_attn_fwd_tc(int dtype, const AttnArgs& a, cudaStream_t s);
// fc_attention_tc_vjp.cu: 16-bit types, at most 64 heads to a key head
int launch_attn_vjp_tc(int dtype, bool kv, const AttnArgs& a, cudaStream_t s);
int launch_attn_row_fix(const AttnArgs& a, float2* stat, cudaStream_t s);

}  // namespace fc

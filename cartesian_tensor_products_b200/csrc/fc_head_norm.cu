// RMS norm of query and key heads with the rotation by node positions, and
// its VJP, one pass over the rows each.
//
// Near the rows read and written: neither their bytes nor the instructions fill
// the time (52 and 40 of 78 us in the first case below), a third of the warps
// leave both waiting in turn.  A group of 1 to 32 lanes takes every
// hs-th head of a node, so that a warp reads one stretch of a row and the node's
// angles stay in registers over the group's heads (a block forms them once, in
// shared memory; one group per node instead read 64-byte pieces of eight rows
// at a time: 98 against 75 us at 65,536 nodes of 16 + 4 BF16 heads of 64).  A lane
// holds units of W values f .. f+W-1 together with their rotation partners
// f+R .. f+R+W-1: both loads of a pair are its own and the rotation needs no
// exchange.  W is the widest vector that R is a multiple of (any R is valid:
// odd ones take scalar units).  Angles are formed in FP64 and reduced to half
// turns, since FP32 would lose the phase of positions far from the origin.
// 65,536 nodes of 16 + 4 BF16 heads of 64: 336 MB in 78 us (4.3 TB/s; some 17
// instructions a value, angles included); the VJP at
// 32,769 nodes of 8 + 2 BF16 heads of 128: 252 MB in 100 us (its registers leave
// two blocks per SM, and at 128 a thread the 16-bit rows of whole vectors spill
// some 390 bytes).
#include <math.h>

#include "fc_device.cuh"
#include "fc_nodes.cuh"

namespace fc {

struct HeadArgs {
  int n, hq, hk, d, R, units, lg, hs;   // lg: log2 of the lanes of a group; hs: groups that share a node's heads
  float eps, inv_d;
  long long ldx, ldy, ldg, ldxb;
  const float *gq, *gk, *pos, *freq;
  float *gpart, *pos_bar;
};

// cos and sin of t half turns.  The quarter turns are taken off in FP64 (adding
// and subtracting 1.5 2^52 rounds to a whole number, whose low bits are the
// quadrant), the rest |f| <= 1/4 goes through polynomials in f^2 of least
// largest error, fitted to sin(pi f)/f (relative) and cos(pi f).  With their
// coefficients rounded to FP32 they are 3.4e-8 and 6.7e-9 off.
__device__ __forceinline__ float2 half_turns(double t) {
  constexpr double kRound = 6755399441055744.0;
  const double m = fma(t, 2.0, kRound);
  const int quad = __double2loint(m);
  const float f = (float)fma(m - kRound, -0.5, t), z = f * f;
  float s = fmaf(z, -0.5890122f, 2.549761f);
  s = fmaf(z, s, -5.167708f);
  s = f * fmaf(z, s, 3.1415927f);
  float c = fmaf(z, 0.23132971f, -1.3350446f);
  c = fmaf(z, c, 4.058707f);
  c = fmaf(z, c, -4.934802f);
  c = fmaf(z, c, 1.0f);
  const float x = quad & 1 ? s : c, y = quad & 1 ? c : s;   // quarter turn: cos -> -sin, sin -> cos
  return make_float2((quad + 1) & 2 ? -x : x, quad & 2 ? -y : y);
}

// First value of unit u: rotated pairs first (partner at + R), then the rest.
template <int W>
__device__ __forceinline__ int unit_at(const HeadArgs& a, int u) {
  const int p = a.R / W;
  return u < p ? u * W : 2 * a.R + (u - p) * W;
}

// Arithmetic on the W values of a unit, two per instruction (both kernels are
// bound by instructions before they are by memory at one value each).
template <int W>
__device__ __forceinline__ void vmul(const float (&a)[W], const float (&b)[W], float (&o)[W]) {
  if constexpr (W % 2 == 0) {
#pragma unroll
    for (int i = 0; i < W; i += 2) {
      const float2 v = __fmul2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
      o[i] = v.x;
      o[i + 1] = v.y;
    }
  } else {
    o[0] = a[0] * b[0];
  }
}
template <int W>
__device__ __forceinline__ void vscale(const float (&a)[W], float f, float (&o)[W]) {
  if constexpr (W % 2 == 0) {
#pragma unroll
    for (int i = 0; i < W; i += 2) {
      const float2 v = __fmul2_rn(make_float2(a[i], a[i + 1]), make_float2(f, f));
      o[i] = v.x;
      o[i + 1] = v.y;
    }
  } else {
    o[0] = a[0] * f;
  }
}
// o = a b + c
template <int W>
__device__ __forceinline__ void vfma(const float (&a)[W], const float (&b)[W], const float (&c)[W], float (&o)[W]) {
  if constexpr (W % 2 == 0) {
#pragma unroll
    for (int i = 0; i < W; i += 2) {
      const float2 v = __ffma2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), make_float2(c[i], c[i + 1]));
      o[i] = v.x;
      o[i + 1] = v.y;
    }
  } else {
    o[0] = fmaf(a[0], b[0], c[0]);
  }
}
// o = a f + c
template <int W>
__device__ __forceinline__ void vfmas(const float (&a)[W], float f, const float (&c)[W], float (&o)[W]) {
  if constexpr (W % 2 == 0) {
#pragma unroll
    for (int i = 0; i < W; i += 2) {
      const float2 v = __ffma2_rn(make_float2(a[i], a[i + 1]), make_float2(f, f), make_float2(c[i], c[i + 1]));
      o[i] = v.x;
      o[i + 1] = v.y;
    }
  } else {
    o[0] = fmaf(a[0], f, c[0]);
  }
}
// o = a b - c d
template <int W>
__device__ __forceinline__ void vcross(const float (&a)[W], const float (&b)[W], const float (&c)[W],
                                       const float (&d)[W], float (&o)[W]) {
  float t[W];
  vmul(c, d, t);
#pragma unroll
  for (int i = 0; i < W; ++i) o[i] = fmaf(a[i], b[i], -t[i]);
}
// s += sum of a b, in two chains
template <int W>
__device__ __forceinline__ void vdot(const float (&a)[W], const float (&b)[W], float2& s) {
  if constexpr (W % 2 == 0) {
#pragma unroll
    for (int i = 0; i < W; i += 2) s = __ffma2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), s);
  } else {
    s.x = fmaf(a[0], b[0], s.x);
  }
}

// What a lane keeps of a node: its units' places and angles.
template <int W, int NIT>
struct LaneUnits {
  int at[NIT];          // -1: no unit
  bool pair[NIT];
  float c[NIT][W], s[NIT][W];

  __device__ __forceinline__ LaneUnits(const HeadArgs& a, int lane) {
#pragma unroll
    for (int j = 0; j < NIT; ++j) {
      const int u = lane + (j << a.lg);
      at[j] = u < a.units ? unit_at<W>(a, u) : -1;
      pair[j] = at[j] >= 0 && at[j] < a.R;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        c[j][i] = 1.0f;
        s[j][i] = 0.0f;
      }
    }
  }
  // angles of a node from the block's table
  __device__ __forceinline__ void node(const float2* turn) {
#pragma unroll
    for (int j = 0; j < NIT; ++j)
      if (pair[j])
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float2 t = turn[at[j] + i];
          c[j][i] = t.x;
          s[j][i] = t.y;
        }
  }
  // a head's values as they are stored; what the lane has no unit for stays as
  // it is (clear), a head that is not there is zeros
  template <class T>
  static __device__ __forceinline__ void clear(Pack<T, W> (&p)[NIT], Pack<T, W> (&q)[NIT]) {
#pragma unroll
    for (int j = 0; j < NIT; ++j) {
      p[j].clear();
      q[j].clear();
    }
  }
  template <class T>
  __device__ __forceinline__ void fetch(const T* row, int R, bool live, Pack<T, W> (&p)[NIT], Pack<T, W> (&q)[NIT]) const {
#pragma unroll
    for (int j = 0; j < NIT; ++j) {
      if (live) {
        if (at[j] >= 0) p[j] = *reinterpret_cast<const Pack<T, W>*>(row + at[j]);
        if (pair[j]) q[j] = *reinterpret_cast<const Pack<T, W>*>(row + at[j] + R);
      } else {
        p[j].clear();
        q[j].clear();
      }
    }
  }
  // to FP32; the sum of squares
  template <class T>
  __device__ __forceinline__ float widen(const Pack<T, W> (&a)[NIT], const Pack<T, W> (&b)[NIT], float (&p)[NIT][W],
                                         float (&q)[NIT][W]) const {
    float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < NIT; ++j) {
      a[j].get(p[j]);
      b[j].get(q[j]);
      vdot(p[j], p[j], ss);
      vdot(q[j], q[j], ss);
    }
    return ss.x + ss.y;
  }
};

__device__ __forceinline__ float group_sum(float v, int lg) {
  if (lg > 0) v += __shfl_xor_sync(0xffffffffu, v, 1);
  if (lg > 1) v += __shfl_xor_sync(0xffffffffu, v, 2);
  if (lg > 2) v += __shfl_xor_sync(0xffffffffu, v, 4);
  if (lg > 3) v += __shfl_xor_sync(0xffffffffu, v, 8);
  if (lg > 4) v += __shfl_xor_sync(0xffffffffu, v, 16);
  return v;
}
// One thread's part of the angle table: frequency f of the nodes first, first +
// stride, ..
struct Angles {
  int f, first, stride;
  double w[3];   // frequency in half turns per unit of length
  __device__ __forceinline__ explicit Angles(const HeadArgs& a) {
    f = first = 0;
    stride = 1 << 30;
    if (a.R == 0) {
      first = stride;
      return;
    }
    const int rows = 256 / a.R;   // R <= 64
    first = threadIdx.x / a.R;
    f = threadIdx.x - first * a.R;
    stride = first < rows ? rows : stride;
    if (first >= rows) first = stride;
#pragma unroll
    for (int c = 0; c < 3; ++c) w[c] = (double)a.freq[c * a.R + f] * 0.31830988618379067154;
  }
  // the angles of nodes n0 .. n0 + nodes - 1, [nodes][R]
  __device__ __forceinline__ void table(const HeadArgs& a, long long n0, int nodes, float2* turn) const {
    for (int t = first; t < nodes && n0 + t < a.n; t += stride) {
      const float* p = a.pos + 3 * (n0 + t);
      turn[t * a.R + f] = half_turns(fma((double)p[0], w[0], fma((double)p[1], w[1], (double)p[2] * w[2])));
    }
  }
};
// gamma of both kinds in shared memory, [2][d] (16-byte aligned there, which
// the caller's need not be)
__device__ __forceinline__ void block_weights(const HeadArgs& a, float* gam) {
  for (int i = threadIdx.x; i < 2 * a.d; i += 256) {
    const float* g = i < a.d ? a.gq : a.gk;
    gam[i] = g ? g[i < a.d ? i : i - a.d] : 1.0f;
  }
}
template <class T, int W, int NIT>
__global__ void __launch_bounds__(256, 3) head_norm_kernel(HeadArgs a, const T* __restrict__ x, T* __restrict__ y) {
  extern __shared__ float sm[];
  float* gam = sm;                                          // [2][d]
  float2* turn = reinterpret_cast<float2*>(sm + 2 * a.d);   // [nodes][R]
  const int lane = threadIdx.x & ((1 << a.lg) - 1), group = threadIdx.x >> a.lg, nodes = (256 >> a.lg) / a.hs;
  const long long n0 = (long long)blockIdx.x * nodes;
  const int t = group / a.hs, part = group - t * a.hs;
  const long long node = n0 + t;
  const bool there = node < a.n;
  LaneUnits<W, NIT> u(a, lane);
  // The group's heads: part, part + hs, .. of the queries, then of the keys.  A
  // head's loads run beside the work on the one before (the first's beside the
  // angles).
  const T* xr = x + (there ? node * a.ldx + (long long)part * a.d : 0);
  T* yr = y + (there ? node * a.ldy + (long long)part * a.d : 0);
  Pack<T, W> rp[NIT], rq[NIT];
  u.clear(rp, rq);
  auto fetch = [&](int h, int Hn) { u.fetch(xr, a.R, there && h < Hn, rp, rq); };
  fetch(part, a.hq ? a.hq : a.hk);
  block_weights(a, gam);
  const Angles angles(a);
  angles.table(a, n0, nodes, turn);
  __syncthreads();
  if (there) u.node(turn + t * a.R);
  const int step = a.hs * a.d;
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const int Hn = kind == 0 ? a.hq : a.hk;
    if (Hn == 0) continue;
    const float* gm = gam + kind * a.d;
    for (int hb = 0; hb < Hn; hb += a.hs) {   // the same count in every lane
      const bool live = there && hb + part < Hn, last = hb + a.hs >= Hn;
      float p[NIT][W], q[NIT][W];
      const float ss = group_sum(u.widen(rp, rq, p, q), a.lg);
      const int move = last && kind == 0 ? a.hq * a.d - hb * a.d : step;   // to the group's next head
      xr += move;
      if (!last)
        fetch(hb + a.hs + part, Hn);
      else if (kind == 0)
        fetch(part, a.hk);
      const float r = rsqrtf(ss * a.inv_d + a.eps);
      if (live) {
#pragma unroll
        for (int j = 0; j < NIT; ++j) {
          if (u.at[j] < 0) continue;
          float v[W], w[W], gw[W];
          load_pack<float, W>(gm + u.at[j], gw);
          vscale(p[j], r, p[j]);
          vmul(p[j], gw, v);
          if (u.pair[j]) {
            vscale(q[j], r, q[j]);
            load_pack<float, W>(gm + u.at[j] + a.R, gw);
            vmul(q[j], gw, q[j]);   // v and q: the normed pair
            vmul(v, u.s[j], w);
            vfma(q[j], u.c[j], w, w);
            vcross(v, u.c[j], q[j], u.s[j], v);
            store_pack<T, W>(yr + u.at[j] + a.R, w);
          }
          store_pack<T, W>(yr + u.at[j], v);
        }
      }
      yr += move;
    }
  }
}

// The VJP: x, g read once, x_bar written once.  With u = x r gamma and ub the
// gradient turned back, x_bar = r (gamma ub - xn mean(gamma ub xn)), xn = x r.
// The gamma gradient stays in registers over all the nodes of a block and is
// added over blocks by head_gamma_kernel; the angle gradients of a node stay
// there over the group's heads.
template <class T, int W, int NIT>
__global__ void __launch_bounds__(256, 2) head_norm_vjp_kernel(HeadArgs a, const T* __restrict__ x,
                                                               const T* __restrict__ g, T* __restrict__ xb) {
  extern __shared__ float sm[];
  float* gam = sm;                                                  // [2][d]
  float* red = gam + 2 * a.d;                                       // [8][2][d] gamma sums
  float* psum = red + 16 * a.d;                                     // [groups][3] position sums
  float2* turn = reinterpret_cast<float2*>(psum + 3 * 256);         // [nodes][R]
  const int tid = threadIdx.x, lane = tid & ((1 << a.lg) - 1), group = tid >> a.lg, nodes = (256 >> a.lg) / a.hs;
  const int t = group / a.hs, part = group - t * a.hs;
  LaneUnits<W, NIT> u(a, lane);
  const Angles angles(a);
  const bool want_pos = a.pos_bar && a.R;
  const int step = a.hs * a.d;
  block_weights(a, gam);
  float acc[2][2][NIT][W];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < NIT; ++j)
#pragma unroll
      for (int i = 0; i < W; ++i) acc[k][0][j][i] = acc[k][1][j][i] = 0.0f;
  for (long long n0 = (long long)blockIdx.x * nodes; n0 < a.n; n0 += (long long)gridDim.x * nodes) {
    const long long node = n0 + t;
    const bool there = node < a.n;
    const long long h0 = (long long)part * a.d;
    const T* xr = x + (there ? node * a.ldx + h0 : 0);
    const T* gr = g + (there ? node * a.ldg + h0 : 0);
    T* br = xb + (there ? node * a.ldxb + h0 : 0);
    Pack<T, W> rp[NIT], rq[NIT], sp[NIT], sq[NIT];
    u.clear(rp, rq);
    u.clear(sp, sq);
    auto fetch = [&](int h, int Hn) {
      u.fetch(xr, a.R, there && h < Hn, rp, rq);
      u.fetch(gr, a.R, there && h < Hn, sp, sq);
    };
    fetch(part, a.hq ? a.hq : a.hk);
    __syncthreads();
    angles.table(a, n0, nodes, turn);
    __syncthreads();
    if (there) u.node(turn + t * a.R);
    float th[NIT][W];
#pragma unroll
    for (int j = 0; j < NIT; ++j)
#pragma unroll
      for (int i = 0; i < W; ++i) th[j][i] = 0.0f;
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const int Hn = kind == 0 ? a.hq : a.hk;
      if (Hn == 0) continue;
      const float* gm = gam + kind * a.d;
      for (int hb = 0; hb < Hn; hb += a.hs) {   // the same count in every lane
        const bool live = there && hb + part < Hn;
        float p[NIT][W], q[NIT][W], gp[NIT][W], gq[NIT][W];
        u.widen(sp, sq, gp, gq);
        const float ss = group_sum(u.widen(rp, rq, p, q), a.lg);
        const bool last = hb + a.hs >= Hn;
        const int move = last && kind == 0 ? a.hq * a.d - hb * a.d : step;   // to the group's next head
        xr += move;
        gr += move;
        if (!last)
          fetch(hb + a.hs + part, Hn);
        else if (kind == 0)
          fetch(part, a.hk);
        const float r = live ? rsqrtf(ss * a.inv_d + a.eps) : 0.0f;
        float2 dots = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < NIT; ++j) {
          if (u.at[j] < 0) continue;
          float ga[W];
          load_pack<float, W>(gm + u.at[j], ga);
          vscale(p[j], r, p[j]);
          if (u.pair[j]) {
            float t1[W], t2[W], gb[W];
            vscale(q[j], r, q[j]);
            // turned back: (ua, ub) = (g_a c + g_b s, g_b c - g_a s)
            vmul(gq[j], u.s[j], t1);
            vfma(gp[j], u.c[j], t1, t2);
            vcross(gq[j], u.c[j], gp[j], u.s[j], gq[j]);
#pragma unroll
            for (int i = 0; i < W; ++i) gp[j][i] = t2[i];
            vfma(gq[j], q[j], acc[kind][1][j], acc[kind][1][j]);
            // g_b y_a - g_a y_b with y turned forward is ub va - ua vb with both
            // turned back; va = xa ga, vb = xb gb, and ga, gb go into ub, ua
            load_pack<float, W>(gm + u.at[j] + a.R, gb);
            vmul(gq[j], ga, t1);
            vfma(t1, p[j], th[j], th[j]);
            vmul(gp[j], gb, t1);
#pragma unroll
            for (int i = 0; i < W; ++i) th[j][i] = fmaf(-t1[i], q[j][i], th[j][i]);
            vmul(gq[j], gb, gq[j]);
            vdot(gq[j], q[j], dots);
          }
          vfma(gp[j], p[j], acc[kind][0][j], acc[kind][0][j]);
          vmul(gp[j], ga, gp[j]);
          vdot(gp[j], p[j], dots);
        }
        const float m = group_sum(dots.x + dots.y, a.lg) * a.inv_d;
        if (live && xb) {
#pragma unroll
          for (int j = 0; j < NIT; ++j) {
            if (u.at[j] < 0) continue;
            float v[W];
            vfmas(p[j], -m, gp[j], v);
            vscale(v, r, v);
            store_pack<T, W>(br + u.at[j], v);
            if (u.pair[j]) {
              vfmas(q[j], -m, gq[j], v);
              vscale(v, r, v);
              store_pack<T, W>(br + u.at[j] + a.R, v);
            }
          }
        }
        br += move;
      }
    }
    if (want_pos) {
      float v[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < NIT; ++j)
        if (u.pair[j])
#pragma unroll
          for (int i = 0; i < W; ++i)
#pragma unroll
            for (int c = 0; c < 3; ++c) v[c] += th[j][i] * a.freq[c * a.R + u.at[j] + i];
#pragma unroll
      for (int c = 0; c < 3; ++c) v[c] = group_sum(v[c], a.lg);
      if (lane == 0)
#pragma unroll
        for (int c = 0; c < 3; ++c) psum[3 * group + c] = v[c];
      __syncthreads();
      for (int i = tid; i < 3 * nodes; i += 256) {
        const int n = i / 3, c = i - 3 * n;
        float s = 0.0f;
        for (int k = 0; k < a.hs; ++k) s += psum[3 * (n * a.hs + k) + c];
        if (n0 + n < a.n) a.pos_bar[3 * n0 + i] = s;
      }
    }
  }
  if (!a.gpart) return;
  // groups of a warp, then warps
  for (int i = tid; i < 16 * a.d; i += 256) red[i] = 0.0f;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < NIT; ++j)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        float va = acc[k][0][j][i], vb = acc[k][1][j][i];
        for (int o = 16; o >= 1 << a.lg; o >>= 1) {
          va += __shfl_xor_sync(0xffffffffu, va, o);
          vb += __shfl_xor_sync(0xffffffffu, vb, o);
        }
        if ((tid & 31) < 1 << a.lg && u.at[j] >= 0) {
          float* to = red + ((tid >> 5) * 2 + k) * a.d;
          to[u.at[j] + i] = va;
          if (u.pair[j]) to[u.at[j] + a.R + i] = vb;
        }
      }
  __syncthreads();
  for (int i = tid; i < 2 * a.d; i += 256) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += red[w * 2 * a.d + i];
    a.gpart[(long long)blockIdx.x * 2 * a.d + i] = v;
  }
}

// gamma gradients: 32 columns of [blocks][2 d] per block, in a fixed order
__global__ void __launch_bounds__(1024) head_gamma_kernel(int blocks, int d, const float* __restrict__ part,
                                                          float* __restrict__ gq, float* __restrict__ gk) {
  __shared__ float sum[32][33];
  const int l = threadIdx.x & 31, c = blockIdx.x * 32 + l, w = threadIdx.x >> 5;
  float v = 0.0f;
  if (c < 2 * d)
#pragma unroll 8
    for (int b = w; b < blocks; b += 32) v += part[(long long)b * 2 * d + c];
  sum[w][l] = v;
  __syncthreads();
  v = sum[l][w];   // column w of this block
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int col = blockIdx.x * 32 + w;
  if (l == 0 && col < 2 * d) {
    if (col < d) {
      if (gq) gq[col] = v;
    } else if (gk) {
      gk[col - d] = v;
    }
  }
}

// ----------------------------------------------------------------- launches

static int check_heads(const fc_head_desc* d, int n) {
  if (!d || !row_dtype(d->dtype) || n < 0) return FC_ERR_ARG;
  if (d->heads_q < 0 || d->heads_k < 0 || d->heads_q > 1024 || d->heads_k > 1024) return FC_ERR_ARG;
  const int H = d->heads_q + d->heads_k;
  if (H < 1 || H > 1024 || d->head_dim < 8 || d->head_dim > 128) return FC_ERR_ARG;
  if (d->pairs < 0 || 2 * d->pairs > d->head_dim) return FC_ERR_ARG;
  if (!(d->eps >= 0.0f) || !isfinite(d->eps)) return FC_ERR_ARG;
  if (d->head_dim % 8) return FC_ERR_ALIGN;
  return FC_OK;
}

// Widest unit, up to 16 bytes, that the pairs are a multiple of.
static int unit_width(const fc_head_desc* d) {
  int w = d->dtype == FC_F32 ? 4 : 8;
  while (d->pairs % w) w >>= 1;
  return w;
}

// Groups: the heads of a node are shared by hs of them, a power of two: a
// warp's worth, and more while that leaves SMs idle.
static void head_geom(const fc_head_desc* d, int n, HeadArgs& a) {
  const int W = unit_width(d), H = d->heads_q + d->heads_k;
  a.n = n; a.hq = d->heads_q; a.hk = d->heads_k; a.d = d->head_dim; a.R = d->pairs; a.eps = d->eps;
  a.inv_d = 1.0f / (float)d->head_dim;
  a.units = d->pairs / W + (d->head_dim - 2 * d->pairs) / W;
  a.lg = 0;
  while (a.lg < 5 && (1 << a.lg) < a.units) ++a.lg;
  const int groups = 256 >> a.lg;
  a.hs = 1;
  while (2 * a.hs <= H && 2 * a.hs <= groups &&
         (a.hs < 32 >> a.lg || (long long)n * a.hs / groups < 2 * device_sm_count()))
    a.hs *= 2;
  // not more than an eighth of the groups without a head, while 256 bytes stay together
  const auto rounds = [&](int h) { return (h + a.hs - 1) / a.hs * a.hs; };
  while (a.hs > 1 && rounds(d->heads_q) + rounds(d->heads_k) > H + H / 8 && (a.hs >> 1) << a.lg >= 16) a.hs >>= 1;
}
static long long head_blocks(const HeadArgs& a) {
  const int nodes = (256 >> a.lg) / a.hs;
  return ((long long)a.n + nodes - 1) / nodes;
}
static size_t angle_bytes(const HeadArgs& a) { return sizeof(float2) * (size_t)((256 >> a.lg) / a.hs) * a.R; }
static int vjp_blocks(const HeadArgs& a) {
  const long long all = head_blocks(a), most = 4LL * device_sm_count();
  return (int)(all < most ? all : most);
}

template <class T, int W, int NIT>
static int run_fwd(const HeadArgs& a, const void* x, void* y, cudaStream_t s) {
  const size_t smem = sizeof(float) * 2 * a.d + angle_bytes(a);
  head_norm_kernel<T, W, NIT><<<(unsigned)head_blocks(a), 256, smem, s>>>(a, static_cast<const T*>(x), static_cast<T*>(y));
  return cudaGetLastError() == cudaSuccess ? FC_OK : FC_ERR_CUDA;
}
template <class T, int W, int NIT>
static int run_vjp(const HeadArgs& a, const void* x, const void* g, void* xb, cudaStream_t s) {
  const size_t smem = sizeof(float) * (3 * 256 + 18 * (size_t)a.d) + angle_bytes(a);
  head_norm_vjp_kernel<T, W, NIT><<<vjp_blocks(a), 256, smem, s>>>(a, static_cast<const T*>(x),
                                                                   static_cast<const T*>(g), static_cast<T*>(xb));
  return cudaGetLastError() == cudaSuccess ? FC_OK : FC_ERR_CUDA;
}

// units of a lane: a head has at most 128 / W of them and 32 lanes
template <class T>
static int launch_fwd(const fc_head_desc* desc, const HeadArgs& a, const void* x, void* y, cudaStream_t s) {
  switch (unit_width(desc)) {
    case 8: return run_fwd<T, sizeof(T) == 2 ? 8 : 4, 1>(a, x, y, s);
    case 4: return run_fwd<T, 4, 1>(a, x, y, s);
    case 2: return run_fwd<T, 2, 2>(a, x, y, s);
    default: return run_fwd<T, 1, 4>(a, x, y, s);
  }
}
template <class T>
static int launch_vjp(const fc_head_desc* desc, const HeadArgs& a, const void* x, const void* g, void* xb,
                      cudaStream_t s) {
  switch (unit_width(desc)) {
    case 8: return run_vjp<T, sizeof(T) == 2 ? 8 : 4, 1>(a, x, g, xb, s);
    case 4: return run_vjp<T, 4, 1>(a, x, g, xb, s);
    case 2: return run_vjp<T, 2, 2>(a, x, g, xb, s);
    default: return run_vjp<T, 1, 4>(a, x, g, xb, s);
  }
}

static bool row_step(long long ld, int heads, int d) { return ld >= (long long)heads * d; }

}  // namespace fc

using namespace fc;

extern "C" {

int fc_head_norm_rotate(const fc_head_desc* desc, int n_nodes, const void* x, int64_t ldx, const float* gamma_q,
                        const float* gamma_k, const float* pos, const float* freq, void* y, int64_t ldy,
                        fc_stream_t stream) {
  const int st = check_heads(desc, n_nodes);
  if (st != FC_OK) return st;
  if (n_nodes == 0) return FC_OK;
  const int H = desc->heads_q + desc->heads_k;
  if (!x || !y || (desc->pairs && (!pos || !freq))) return FC_ERR_ARG;
  if (!row_step(ldx, H, desc->head_dim) || !row_step(ldy, H, desc->head_dim)) return FC_ERR_ARG;
  if (!aligned16(x) || !aligned16(y) || ldx % 8 || ldy % 8 || !aligned4(gamma_q) || !aligned4(gamma_k) ||
      !aligned4(pos) || !aligned4(freq))
    return FC_ERR_ALIGN;
  HeadArgs a{};
  head_geom(desc, n_nodes, a);
  a.ldx = ldx; a.ldy = ldy; a.gq = gamma_q; a.gk = gamma_k; a.pos = pos; a.freq = freq;
  cudaStream_t s = (cudaStream_t)stream;
  if (desc->dtype == FC_F32) return launch_fwd<float>(desc, a, x, y, s);
  if (desc->dtype == FC_BF16) return launch_fwd<__nv_bfloat16>(desc, a, x, y, s);
  return launch_fwd<__half>(desc, a, x, y, s);
}

size_t fc_head_norm_rotate_vjp_workspace_size(const fc_head_desc* desc, int n_nodes) {
  if (check_heads(desc, n_nodes) != FC_OK || n_nodes == 0) return 0;
  HeadArgs a{};
  head_geom(desc, n_nodes, a);
  return round16(sizeof(float) * 2 * (size_t)a.d * vjp_blocks(a));
}

int fc_head_norm_rotate_vjp(const fc_head_desc* desc, int n_nodes, const void* x, int64_t ldx, const void* g,
                            int64_t ldg, const float* gamma_q, const float* gamma_k, const float* pos,
                            const float* freq, void* x_bar, int64_t ldxb, float* gamma_q_bar, float* gamma_k_bar,
                            float* pos_bar, void* workspace, size_t ws_bytes, fc_stream_t stream) {
  const int st = check_heads(desc, n_nodes);
  if (st != FC_OK) return st;
  const int H = desc->heads_q + desc->heads_k, D = desc->head_dim;
  cudaStream_t s = (cudaStream_t)stream;
  if (!aligned4(gamma_q_bar) || !aligned4(gamma_k_bar) || !aligned4(pos_bar)) return FC_ERR_ALIGN;
  if (n_nodes > 0) {
    if (!x || !g || (desc->pairs && (!pos || !freq))) return FC_ERR_ARG;
    if (!row_step(ldx, H, D) || !row_step(ldg, H, D) || (x_bar && !row_step(ldxb, H, D))) return FC_ERR_ARG;
    if (!aligned16(x) || !aligned16(g) || (x_bar && (!aligned16(x_bar) || ldxb % 8)) || ldx % 8 || ldg % 8 ||
        !aligned4(gamma_q) || !aligned4(gamma_k) || !aligned4(pos) || !aligned4(freq))
      return FC_ERR_ALIGN;
  }
  const bool gamma = gamma_q_bar || gamma_k_bar;
  if (n_nodes == 0) {
    if ((gamma_q_bar && cudaMemsetAsync(gamma_q_bar, 0, 4 * (size_t)D, s) != cudaSuccess) ||
        (gamma_k_bar && cudaMemsetAsync(gamma_k_bar, 0, 4 * (size_t)D, s) != cudaSuccess))
      return FC_ERR_CUDA;
    return FC_OK;
  }
  HeadArgs a{};
  head_geom(desc, n_nodes, a);
  if (gamma) {
    if (!workspace || ws_bytes < fc_head_norm_rotate_vjp_workspace_size(desc, n_nodes)) return FC_ERR_WORKSPACE;
    if (!aligned16(workspace)) return FC_ERR_ALIGN;
    a.gpart = static_cast<float*>(workspace);
  }
  if (pos_bar && !desc->pairs && cudaMemsetAsync(pos_bar, 0, 12 * (size_t)n_nodes, s) != cudaSuccess)
    return FC_ERR_CUDA;
  if (!x_bar && !gamma && !(pos_bar && desc->pairs)) return FC_OK;
  a.ldx = ldx; a.ldg = ldg; a.ldxb = ldxb; a.gq = gamma_q; a.gk = gamma_k; a.pos = pos; a.freq = freq;
  a.pos_bar = pos_bar;
  const int rc = desc->dtype == FC_F32    ? launch_vjp<float>(desc, a, x, g, x_bar, s)
                 : desc->dtype == FC_BF16 ? launch_vjp<__nv_bfloat16>(desc, a, x, g, x_bar, s)
                                          : launch_vjp<__half>(desc, a, x, g, x_bar, s);
  if (rc != FC_OK || !gamma) return rc;
  head_gamma_kernel<<<(2 * D + 31) / 32, 1024, 0, s>>>(vjp_blocks(a), D, a.gpart, gamma_q_bar, gamma_k_bar);
  return cudaGetLastError() == cudaSuccess ? FC_OK : FC_ERR_CUDA;
}

}  // extern "C"

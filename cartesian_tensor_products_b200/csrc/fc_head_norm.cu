// RMS norm of query and key heads with the rotation by node positions, and
// its VJP, one pass over the rows each.
//
// Bound by the rows read and written.  A group of 1 to 32 lanes takes every
// hs-th head of a node, so that a warp reads one stretch of a row and the node's
// angles stay in registers over the group's heads (a block forms them once, in
// shared memory; one group per node instead read 64-byte pieces of eight rows
// at a time: 98 against 75 us at 65,536 nodes of 16 + 4 BF16 heads of 64).  A lane
// holds units of W values f .. f+W-1 together with their rotation partners
// f+R .. f+R+W-1: both loads of a pair are its own and the rotation needs no
// exchange.  W is the widest vector that R is a multiple of (any R is valid:
// odd ones take scalar units).  Angles are formed in FP64 and reduced to half
// turns, since FP32 would lose the phase of positions far from the origin.
#include <math.h>

#include "fc_nodes.cuh"

namespace fc {

struct HeadArgs {
  int n, hq, hk, d, R, units, lg, hs;   // lg: log2 of the lanes of a group; hs: groups that share a node's heads
  float eps;
  long long ldx, ldy, ldg, ldxb;
  const float *gq, *gk, *pos, *freq;
  float *gpart, *pos_bar;
};

// cos and sin of angle f of a node
__device__ __forceinline__ float2 node_angle(const HeadArgs& a, const double (&p)[3], int f) {
  const double th = p[0] * a.freq[f] + p[1] * a.freq[a.R + f] + p[2] * a.freq[2 * a.R + f];
  const double t = th * 0.31830988618379067154;   // half turns
  float s, c;
  sincospif((float)(t - 2.0 * rint(0.5 * t)), &s, &c);
  return make_float2(c, s);
}

// First value of unit u: rotated pairs first (partner at + R), then the rest.
template <int W>
__device__ __forceinline__ int unit_at(const HeadArgs& a, int u) {
  const int p = a.R / W;
  return u < p ? u * W : 2 * a.R + (u - p) * W;
}

// What a lane keeps of a node: its units' places and angles.
template <int W, int NIT>
struct LaneUnits {
  int at[NIT];          // -1: no unit
  bool pair[NIT];
  float2 cs[NIT][W];

  __device__ __forceinline__ LaneUnits(const HeadArgs& a, int lane) {
#pragma unroll
    for (int j = 0; j < NIT; ++j) {
      const int u = lane + (j << a.lg);
      at[j] = u < a.units ? unit_at<W>(a, u) : -1;
      pair[j] = at[j] >= 0 && at[j] < a.R;
#pragma unroll
      for (int i = 0; i < W; ++i) cs[j][i] = make_float2(1.0f, 0.0f);
    }
  }
  // angles of a node from the block's table
  __device__ __forceinline__ void node(const float2* turn) {
#pragma unroll
    for (int j = 0; j < NIT; ++j)
      if (pair[j])
#pragma unroll
        for (int i = 0; i < W; ++i) cs[j][i] = turn[at[j] + i];
  }
  // a head's values as they are stored, zeros where the lane has none
  template <class T>
  __device__ __forceinline__ void fetch(const T* row, int R, bool live, Pack<T, W> (&p)[NIT], Pack<T, W> (&q)[NIT]) const {
#pragma unroll
    for (int j = 0; j < NIT; ++j) {
      p[j].clear();
      q[j].clear();
      if (live && at[j] >= 0) p[j] = *reinterpret_cast<const Pack<T, W>*>(row + at[j]);
      if (live && pair[j]) q[j] = *reinterpret_cast<const Pack<T, W>*>(row + at[j] + R);
    }
  }
  // to FP32; the sum of squares
  template <class T>
  __device__ __forceinline__ float widen(const Pack<T, W> (&a)[NIT], const Pack<T, W> (&b)[NIT], float (&p)[NIT][W],
                                         float (&q)[NIT][W]) const {
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < NIT; ++j) {
      a[j].get(p[j]);
      b[j].get(q[j]);
#pragma unroll
      for (int i = 0; i < W; ++i) ss += p[j][i] * p[j][i] + q[j][i] * q[j][i];
    }
    return ss;
  }
};

__device__ __forceinline__ float group_sum(float v, int lg) {
  for (int o = (1 << lg) >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// the weights of both kinds, [2][d], and the angles of a block's nodes from n0 on, [nodes][R]
__device__ __forceinline__ void load_weights(const HeadArgs& a, float* gam) {
  for (int i = threadIdx.x; i < 2 * a.d; i += 256) {
    const float* g = i < a.d ? a.gq : a.gk;
    gam[i] = g ? g[i < a.d ? i : i - a.d] : 1.0f;
  }
}
__device__ __forceinline__ void load_angles(const HeadArgs& a, long long n0, int nodes, float2* turn) {
  for (int i = threadIdx.x; i < nodes * a.R; i += 256) {
    const int t = i / a.R;
    const long long n = n0 + t;
    if (n >= a.n) break;
    const double p[3] = {a.pos[3 * n], a.pos[3 * n + 1], a.pos[3 * n + 2]};
    turn[i] = node_angle(a, p, i - t * a.R);
  }
}

template <class T, int W, int NIT>
__global__ void __launch_bounds__(256) head_norm_kernel(HeadArgs a, const T* __restrict__ x, T* __restrict__ y) {
  extern __shared__ float sm[];
  float* gam = sm;
  float2* turn = reinterpret_cast<float2*>(sm + 2 * a.d);
  const int lane = threadIdx.x & ((1 << a.lg) - 1), group = threadIdx.x >> a.lg, nodes = (256 >> a.lg) / a.hs;
  const long long n0 = (long long)blockIdx.x * nodes;
  const int t = group / a.hs, part = group - t * a.hs, H = a.hq + a.hk;
  const long long node = n0 + t;
  const bool there = node < a.n;
  LaneUnits<W, NIT> u(a, lane);
  // a head's loads run beside the work on the one before (the first's beside the angles)
  Pack<T, W> rp[NIT], rq[NIT];
  auto fetch = [&](int h) {
    const bool live = there && h < H;
    u.fetch(x + (live ? node * a.ldx + (long long)h * a.d : 0), a.R, live, rp, rq);
  };
  fetch(part);
  load_weights(a, gam);
  load_angles(a, n0, nodes, turn);
  __syncthreads();
  if (there) u.node(turn + t * a.R);
  for (int hb = 0; hb < H; hb += a.hs) {   // the same count in every lane
    const int h = hb + part;
    const bool live = there && h < H;
    const long long hd = (long long)h * a.d;
    float p[NIT][W], q[NIT][W];
    const float ss = group_sum(u.widen(rp, rq, p, q), a.lg);
    fetch(h + a.hs);
    const float r = rsqrtf(ss / (float)a.d + a.eps);
    if (!live) continue;
    const float* gm = gam + (h < a.hq ? 0 : a.d);
    T* out = y + node * a.ldy + hd;
#pragma unroll
    for (int j = 0; j < NIT; ++j) {
      if (u.at[j] < 0) continue;
      float v[W], w[W], ga[W], gb[W];
      load_pack<float, W>(gm + u.at[j], ga);
      if (u.pair[j]) {
        load_pack<float, W>(gm + u.at[j] + a.R, gb);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float ua = p[j][i] * r * ga[i], ub = q[j][i] * r * gb[i];
          v[i] = ua * u.cs[j][i].x - ub * u.cs[j][i].y;
          w[i] = ua * u.cs[j][i].y + ub * u.cs[j][i].x;
        }
        store_pack<T, W>(out + u.at[j] + a.R, w);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = p[j][i] * r * ga[i];
      }
      store_pack<T, W>(out + u.at[j], v);
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
  float* red = gam + 2 * a.d;                                       // [8][2][d] gamma sums, at the end
  float* psum = red + 16 * a.d;                                     // [groups][3] position sums
  float2* turn = reinterpret_cast<float2*>(psum + 3 * 256);         // [nodes][R]
  const int tid = threadIdx.x, lane = tid & ((1 << a.lg) - 1), group = tid >> a.lg, nodes = (256 >> a.lg) / a.hs;
  const int t = group / a.hs, part = group - t * a.hs, H = a.hq + a.hk;
  LaneUnits<W, NIT> u(a, lane);
  float acc[2][2][NIT][W];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < NIT; ++j)
#pragma unroll
      for (int i = 0; i < W; ++i) acc[k][0][j][i] = acc[k][1][j][i] = 0.0f;
  const bool want_pos = a.pos_bar && a.R;
  load_weights(a, gam);
  for (long long n0 = (long long)blockIdx.x * nodes; n0 < a.n; n0 += (long long)gridDim.x * nodes) {
    const long long node = n0 + t;
    const bool there = node < a.n;
    Pack<T, W> rp[NIT], rq[NIT], sp[NIT], sq[NIT];
    auto fetch = [&](int h) {
      const bool live = there && h < H;
      u.fetch(x + (live ? node * a.ldx + (long long)h * a.d : 0), a.R, live, rp, rq);
      u.fetch(g + (live ? node * a.ldg + (long long)h * a.d : 0), a.R, live, sp, sq);
    };
    fetch(part);
    __syncthreads();
    load_angles(a, n0, nodes, turn);
    __syncthreads();
    if (there) u.node(turn + t * a.R);
    float th[NIT][W];
#pragma unroll
    for (int j = 0; j < NIT; ++j)
#pragma unroll
      for (int i = 0; i < W; ++i) th[j][i] = 0.0f;
    for (int hb = 0; hb < H; hb += a.hs) {
      const int h = hb + part;
      const bool live = there && h < H;
      const float fk = h < a.hq ? 0.0f : 1.0f, fq = 1.0f - fk;
      const float* gm = gam + (h < a.hq ? 0 : a.d);
      const long long hd = (long long)h * a.d;
      float p[NIT][W], q[NIT][W], gp[NIT][W], gq[NIT][W];
      u.widen(sp, sq, gp, gq);
      const float ss = group_sum(u.widen(rp, rq, p, q), a.lg);
      fetch(h + a.hs);
      const float r = live ? rsqrtf(ss / (float)a.d + a.eps) : 0.0f;
      float dot = 0.0f;
#pragma unroll
      for (int j = 0; j < NIT; ++j) {
        if (u.at[j] < 0) continue;
        float ga[W], gb[W];
        load_pack<float, W>(gm + u.at[j], ga);
        if (u.pair[j]) load_pack<float, W>(gm + u.at[j] + a.R, gb);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float xa = p[j][i] * r;
          float ua = gp[j][i];
          p[j][i] = xa;
          if (u.pair[j]) {
            const float2 cs = u.cs[j][i];
            const float xq = q[j][i] * r, ub = gq[j][i] * cs.x - gp[j][i] * cs.y;
            q[j][i] = xq;
            ua = gp[j][i] * cs.x + gq[j][i] * cs.y;
            // g_b y_a - g_a y_b with y turned forward is ub va - ua vb with both turned back
            th[j][i] += ub * (xa * ga[i]) - ua * (xq * gb[i]);
            const float c = ub * xq;
            acc[0][1][j][i] = fmaf(c, fq, acc[0][1][j][i]);
            acc[1][1][j][i] = fmaf(c, fk, acc[1][1][j][i]);
            gq[j][i] = ub * gb[i];
            dot += gq[j][i] * xq;
          }
          const float c = ua * xa;
          acc[0][0][j][i] = fmaf(c, fq, acc[0][0][j][i]);
          acc[1][0][j][i] = fmaf(c, fk, acc[1][0][j][i]);
          gp[j][i] = ua * ga[i];
          dot += gp[j][i] * xa;
        }
      }
      const float m = group_sum(dot, a.lg) / (float)a.d;
      if (!live || !xb) continue;
      T* out = xb + node * a.ldxb + hd;
#pragma unroll
      for (int j = 0; j < NIT; ++j) {
        if (u.at[j] < 0) continue;
        float v[W];
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = r * (gp[j][i] - p[j][i] * m);
        store_pack<T, W>(out + u.at[j], v);
        if (u.pair[j]) {
#pragma unroll
          for (int i = 0; i < W; ++i) v[i] = r * (gq[j][i] - q[j][i] * m);
          store_pack<T, W>(out + u.at[j] + a.R, v);
        }
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
  for (int i = tid; i < 8 * 2 * a.d; i += 256) red[i] = 0.0f;
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
  a.units = d->pairs / W + (d->head_dim - 2 * d->pairs) / W;
  a.lg = 0;
  while (a.lg < 5 && (1 << a.lg) < a.units) ++a.lg;
  const int groups = 256 >> a.lg;
  a.hs = 1;
  while (2 * a.hs <= H && 2 * a.hs <= groups &&
         (a.hs < 32 >> a.lg || (long long)n * a.hs / groups < 2 * device_sm_count()))
    a.hs *= 2;
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
#define FC_HEAD_DISPATCH(RUN, ...)                                                                       \
  do {                                                                                                   \
    const int w = unit_width(desc);                                                                      \
    if (desc->dtype == FC_F32)                                                                           \
      return w == 4   ? RUN<float, 4, 1>(__VA_ARGS__)                                                    \
             : w == 2 ? RUN<float, 2, 2>(__VA_ARGS__)                                                    \
                      : RUN<float, 1, 4>(__VA_ARGS__);                                                   \
    if (desc->dtype == FC_BF16)                                                                          \
      return w == 8   ? RUN<__nv_bfloat16, 8, 1>(__VA_ARGS__)                                            \
             : w == 4 ? RUN<__nv_bfloat16, 4, 1>(__VA_ARGS__)                                            \
             : w == 2 ? RUN<__nv_bfloat16, 2, 2>(__VA_ARGS__)                                            \
                      : RUN<__nv_bfloat16, 1, 4>(__VA_ARGS__);                                           \
    return w == 8   ? RUN<__half, 8, 1>(__VA_ARGS__)                                                     \
           : w == 4 ? RUN<__half, 4, 1>(__VA_ARGS__)                                                     \
           : w == 2 ? RUN<__half, 2, 2>(__VA_ARGS__)                                                     \
                    : RUN<__half, 1, 4>(__VA_ARGS__);                                                    \
  } while (0)

static int launch_fwd(const fc_head_desc* desc, const HeadArgs& a, const void* x, void* y, cudaStream_t s) {
  FC_HEAD_DISPATCH(run_fwd, a, x, y, s);
}
static int launch_vjp(const fc_head_desc* desc, const HeadArgs& a, const void* x, const void* g, void* xb,
                      cudaStream_t s) {
  FC_HEAD_DISPATCH(run_vjp, a, x, g, xb, s);
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
  return launch_fwd(desc, a, x, y, (cudaStream_t)stream);
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
  const int rc = launch_vjp(desc, a, x, g, x_bar, s);
  if (rc != FC_OK || !gamma) return rc;
  head_gamma_kernel<<<(2 * D + 31) / 32, 1024, 0, s>>>(vjp_blocks(a), D, a.gpart, gamma_q_bar, gamma_k_bar);
  return cudaGetLastError() == cudaSuccess ? FC_OK : FC_ERR_CUDA;
}

}  // extern "C"

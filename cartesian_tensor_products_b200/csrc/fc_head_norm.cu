// RMS norm of query and key heads with the rotation by node positions, and
// its VJP, one pass over the rows each.
//
// Bound by the rows read and written.  A head is spread over a group of 1 to
// 32 lanes; a lane holds units of W values f .. f+W-1 together with their
// rotation partners f+R .. f+R+W-1, so that both 16-byte loads of a pair stay
// in one lane and the rotation needs no exchange.  W is the widest vector
// that R is a multiple of (any R is valid: odd ones take scalar units).  The
// angles of a block's nodes are formed once for all heads, in FP64 reduced to
// half turns, since FP32 would lose the phase of positions far from the
// origin.
#include <math.h>

#include "fc_nodes.cuh"

namespace fc {

struct HeadArgs {
  int n, hq, hk, d, R, units, lg, tn;   // lg: log2 of the lanes per head; tn: nodes per block step
  float eps;
  long long ldx, ldy, ldg, ldxb;
  const float *gq, *gk, *pos, *freq;
  float *gpart, *pos_bar;
};

// cos and sin of angle f of a node
__device__ __forceinline__ float2 node_angle(const HeadArgs& a, long long node, int f) {
  const double th = (double)a.pos[3 * node] * a.freq[f] + (double)a.pos[3 * node + 1] * a.freq[a.R + f] +
                    (double)a.pos[3 * node + 2] * a.freq[2 * a.R + f];
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

template <class T, int W, int NIT>
__global__ void __launch_bounds__(256) head_norm_kernel(HeadArgs a, const T* __restrict__ x, T* __restrict__ y) {
  extern __shared__ float sm[];
  float* gam = sm;                                                 // [2][d]
  float2* turn = reinterpret_cast<float2*>(sm + 2 * a.d);          // [tn][R]
  const int tid = threadIdx.x, H = a.hq + a.hk, G = 1 << a.lg;
  const long long n0 = (long long)blockIdx.x * a.tn;
  const int here = (int)(a.n - n0 < a.tn ? a.n - n0 : a.tn);
  for (int i = tid; i < 2 * a.d; i += 256) {
    const float* g = i < a.d ? a.gq : a.gk;
    gam[i] = g ? g[i < a.d ? i : i - a.d] : 1.0f;
  }
  for (int i = tid; i < here * a.R; i += 256) {
    const int t = i / a.R;
    turn[i] = node_angle(a, n0 + t, i - t * a.R);
  }
  __syncthreads();
  const int lane = tid & (G - 1), group = tid >> a.lg, groups = 256 >> a.lg;
  const int items = here * H;
  const int first = (tid & ~31) >> a.lg;   // the warp's first group: loop bounds are per warp
  for (int base = first; base < items; base += groups) {
    const int it = base + (group - first);
    const bool live = it < items;
    const int t = live ? it / H : 0, h = live ? it - t * H : 0;
    const T* row = x + (n0 + t) * a.ldx + (long long)h * a.d;
    float p[NIT][W], q[NIT][W], ss = 0.0f;
#pragma unroll
    for (int j = 0; j < NIT; ++j) {
      const int u = lane + j * G;
#pragma unroll
      for (int i = 0; i < W; ++i) p[j][i] = q[j][i] = 0.0f;
      if (live && u < a.units) {
        const int at = unit_at<W>(a, u);
        load_pack<T, W>(row + at, p[j]);
        if (at < a.R) load_pack<T, W>(row + at + a.R, q[j]);
      }
#pragma unroll
      for (int i = 0; i < W; ++i) ss += p[j][i] * p[j][i] + q[j][i] * q[j][i];
    }
    for (int o = G >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss / (float)a.d + a.eps);
    if (!live) continue;
    const float* gm = gam + (h < a.hq ? 0 : a.d);
    T* out = y + (n0 + t) * a.ldy + (long long)h * a.d;
#pragma unroll
    for (int j = 0; j < NIT; ++j) {
      const int u = lane + j * G;
      if (u >= a.units) continue;
      const int at = unit_at<W>(a, u);
      float v[W], w[W];
      if (at < a.R) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float2 cs = turn[t * a.R + at + i];
          const float ua = p[j][i] * r * gm[at + i], ub = q[j][i] * r * gm[at + a.R + i];
          v[i] = ua * cs.x - ub * cs.y;
          w[i] = ua * cs.y + ub * cs.x;
        }
        store_pack<T, W>(out + at + a.R, w);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = p[j][i] * r * gm[at + i];
      }
      store_pack<T, W>(out + at, v);
    }
  }
}

// The VJP: x, g read once, x_bar written once.  With u = x r gamma and ub the
// gradient turned back, x_bar = r (gamma ub - xn mean(gamma ub xn)), xn = x r.
// The gamma gradient stays in registers over all the nodes of a block and is
// added over blocks by head_gamma_kernel; the position gradient of a node is
// summed over its heads in shared memory.
template <class T, int W, int NIT>
__global__ void __launch_bounds__(256) head_norm_vjp_kernel(HeadArgs a, const T* __restrict__ x,
                                                            const T* __restrict__ g, T* __restrict__ xb) {
  extern __shared__ float sm[];
  const int tid = threadIdx.x, H = a.hq + a.hk, G = 1 << a.lg;
  float* gam = sm;                                                 // [2][d]
  float* fr = gam + 2 * a.d;                                       // [3][R], padded to 4 R
  float2* turn = reinterpret_cast<float2*>(fr + 4 * a.R);          // [tn][R]
  float* pacc = reinterpret_cast<float*>(turn + a.tn * a.R);       // [tn H][3]
  for (int i = tid; i < 2 * a.d; i += 256) {
    const float* gg = i < a.d ? a.gq : a.gk;
    gam[i] = gg ? gg[i < a.d ? i : i - a.d] : 1.0f;
  }
  for (int i = tid; i < 3 * a.R; i += 256) fr[i] = a.freq[i];
  const int lane = tid & (G - 1), group = tid >> a.lg, groups = 256 >> a.lg;
  const int first = (tid & ~31) >> a.lg;
  float acc[2][NIT][2][W];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < NIT; ++j)
#pragma unroll
      for (int i = 0; i < W; ++i) acc[k][j][0][i] = acc[k][j][1][i] = 0.0f;

  for (long long n0 = (long long)blockIdx.x * a.tn; n0 < a.n; n0 += (long long)gridDim.x * a.tn) {
    const int here = (int)(a.n - n0 < a.tn ? a.n - n0 : a.tn);
    __syncthreads();
    for (int i = tid; i < here * a.R; i += 256) {
      const int t = i / a.R;
      turn[i] = node_angle(a, n0 + t, i - t * a.R);
    }
    __syncthreads();
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const int Hn = kind == 0 ? a.hq : a.hk, h0 = kind == 0 ? 0 : a.hq;
      const float* gm = gam + kind * a.d;
      const int items = here * Hn;
      for (int base = first; base < items; base += groups) {
        const int it = base + (group - first);
        const bool live = it < items;
        const int t = live ? it / Hn : 0, h = live ? h0 + it - t * Hn : h0;
        const T* row = x + (n0 + t) * a.ldx + (long long)h * a.d;
        const T* grow = g + (n0 + t) * a.ldg + (long long)h * a.d;
        float p[NIT][W], q[NIT][W], gp[NIT][W], gq[NIT][W], ss = 0.0f;
#pragma unroll
        for (int j = 0; j < NIT; ++j) {
          const int u = lane + j * G;
#pragma unroll
          for (int i = 0; i < W; ++i) p[j][i] = q[j][i] = gp[j][i] = gq[j][i] = 0.0f;
          if (live && u < a.units) {
            const int at = unit_at<W>(a, u);
            load_pack<T, W>(row + at, p[j]);
            load_pack<T, W>(grow + at, gp[j]);
            if (at < a.R) {
              load_pack<T, W>(row + at + a.R, q[j]);
              load_pack<T, W>(grow + at + a.R, gq[j]);
            }
          }
#pragma unroll
          for (int i = 0; i < W; ++i) ss += p[j][i] * p[j][i] + q[j][i] * q[j][i];
        }
        for (int o = G >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss / (float)a.d + a.eps);
        float dot = 0.0f, px = 0.0f, py = 0.0f, pz = 0.0f;
#pragma unroll
        for (int j = 0; j < NIT; ++j) {
          const int u = lane + j * G;
          if (u >= a.units) continue;
          const int at = unit_at<W>(a, u);
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const float xa = p[j][i] * r, ga = gm[at + i];
            p[j][i] = xa;
            float ua = gp[j][i];
            if (at < a.R) {
              const float2 cs = turn[t * a.R + at + i];
              const float xq = q[j][i] * r, gb = gm[at + a.R + i];
              q[j][i] = xq;
              const float va = xa * ga, vb = xq * gb;
              const float ya = va * cs.x - vb * cs.y, yb = va * cs.y + vb * cs.x;
              const float th = gq[j][i] * ya - gp[j][i] * yb;
              px += th * fr[at + i];
              py += th * fr[a.R + at + i];
              pz += th * fr[2 * a.R + at + i];
              ua = gp[j][i] * cs.x + gq[j][i] * cs.y;
              const float ub = gq[j][i] * cs.x - gp[j][i] * cs.y;
              acc[kind][j][1][i] += ub * xq;
              gq[j][i] = ub * gb;
              dot += gq[j][i] * xq;
            }
            acc[kind][j][0][i] += ua * xa;
            gp[j][i] = ua * ga;
            dot += gp[j][i] * xa;
          }
        }
        for (int o = G >> 1; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (a.pos_bar && a.R)
          for (int o = G >> 1; o > 0; o >>= 1) {
            px += __shfl_xor_sync(0xffffffffu, px, o);
            py += __shfl_xor_sync(0xffffffffu, py, o);
            pz += __shfl_xor_sync(0xffffffffu, pz, o);
          }
        if (!live) continue;
        if (a.pos_bar && a.R && lane == 0) {
          float* pa = pacc + 3 * (t * H + h);
          pa[0] = px; pa[1] = py; pa[2] = pz;
        }
        if (!xb) continue;
        const float m = dot / (float)a.d;
        T* out = xb + (n0 + t) * a.ldxb + (long long)h * a.d;
#pragma unroll
        for (int j = 0; j < NIT; ++j) {
          const int u = lane + j * G;
          if (u >= a.units) continue;
          const int at = unit_at<W>(a, u);
          float v[W];
#pragma unroll
          for (int i = 0; i < W; ++i) v[i] = r * (gp[j][i] - p[j][i] * m);
          store_pack<T, W>(out + at, v);
          if (at < a.R) {
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] = r * (gq[j][i] - q[j][i] * m);
            store_pack<T, W>(out + at + a.R, v);
          }
        }
      }
    }
    if (a.pos_bar && a.R) {
      __syncthreads();
      for (int i = tid; i < here * 3; i += 256) {
        const int t = i / 3, c = i - 3 * t;
        float v = 0.0f;
        for (int h = 0; h < H; ++h) v += pacc[3 * (t * H + h) + c];
        a.pos_bar[3 * n0 + i] = v;
      }
    }
  }
  if (!a.gpart) return;
  // groups of a warp, then warps: [8][2][d] in shared memory
  __syncthreads();
  float* red = sm;
  for (int i = tid; i < 8 * 2 * a.d; i += 256) red[i] = 0.0f;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < NIT; ++j) {
      const int u = lane + j * G;
      const int at = unit_at<W>(a, u);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        float va = acc[k][j][0][i], vb = acc[k][j][1][i];
        for (int o = 16; o >= G; o >>= 1) {
          va += __shfl_xor_sync(0xffffffffu, va, o);
          vb += __shfl_xor_sync(0xffffffffu, vb, o);
        }
        if ((tid & 31) < G && u < a.units) {
          float* to = red + ((tid >> 5) * 2 + k) * a.d;
          to[at + i] = va;
          if (at < a.R) to[at + a.R + i] = vb;
        }
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
__global__ void __launch_bounds__(256) head_gamma_kernel(int blocks, int d, const float* __restrict__ part,
                                                         float* __restrict__ gq, float* __restrict__ gk) {
  __shared__ float sum[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  float v = 0.0f;
  if (c < 2 * d)
#pragma unroll 8
    for (int b = w; b < blocks; b += 8) v += part[(long long)b * 2 * d + c];
  sum[w][threadIdx.x & 31] = v;
  __syncthreads();
  if (w == 0 && c < 2 * d) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += sum[k][threadIdx.x];
    if (c < d) {
      if (gq) gq[c] = s;
    } else if (gk) {
      gk[c - d] = s;
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

// Geometry shared by both directions; vjp also keeps one [3] per head and node.
static void head_geom(const fc_head_desc* d, int n, HeadArgs& a) {
  const int W = unit_width(d), H = d->heads_q + d->heads_k;
  a.n = n; a.hq = d->heads_q; a.hk = d->heads_k; a.d = d->head_dim; a.R = d->pairs; a.eps = d->eps;
  a.units = d->pairs / W + (d->head_dim - 2 * d->pairs) / W;
  a.lg = 0;
  while (a.lg < 5 && (1 << a.lg) < a.units) ++a.lg;
  // four heads per lane group and step, fewer while that leaves SMs idle
  int tn = (4 * (256 >> a.lg) + H - 1) / H;
  const int even = n / (2 * device_sm_count());
  if (tn > even) tn = even;
  if (tn > 32) tn = 32;
  a.tn = tn < 1 ? 1 : tn;
}
static int vjp_blocks(const HeadArgs& a) {
  const long long tiles = ((long long)a.n + a.tn - 1) / a.tn;
  const long long most = 4LL * device_sm_count();
  return (int)(tiles < most ? tiles : most);
}

template <class T, int W, int NIT>
static int run_fwd(const HeadArgs& a, const void* x, void* y, cudaStream_t s) {
  const size_t smem = 8 * (size_t)a.d + 8 * (size_t)a.tn * a.R;
  const int grid = (int)(((long long)a.n + a.tn - 1) / a.tn);
  head_norm_kernel<T, W, NIT><<<grid, 256, smem, s>>>(a, static_cast<const T*>(x), static_cast<T*>(y));
  return cudaGetLastError() == cudaSuccess ? FC_OK : FC_ERR_CUDA;
}
template <class T, int W, int NIT>
static int run_vjp(const HeadArgs& a, const void* x, const void* g, void* xb, cudaStream_t s) {
  size_t smem = 8 * (size_t)a.d + 16 * (size_t)a.R + 8 * (size_t)a.tn * a.R +
                12 * (size_t)a.tn * (a.hq + a.hk);
  if (smem < 64 * (size_t)a.d) smem = 64 * (size_t)a.d;
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
  head_gamma_kernel<<<(2 * D + 31) / 32, 256, 0, s>>>(vjp_blocks(a), D, a.gpart, gamma_q_bar, gamma_k_bar);
  return cudaGetLastError() == cudaSuccess ? FC_OK : FC_ERR_CUDA;
}

}  // extern "C"

// Node attention, forward: entry point, plan and the strip kernel.
//
// A block takes 16 WM virtual rows (receivers x heads of a key head) of one
// structure and walks over its senders with a running maximum and sum: scores,
// cap, distance bias and mask stay in registers, keys and values pass through
// a double-buffered shared tile.  A warp holds 16 of the rows and one of WN
// parts of every key tile, with a running state of its own; the parts are
// merged at the end.  WM = 4, WN = 1 or 2 in general; WM = 1, WN = 4 where a
// structure has few rows (three of four warps had none).  With few blocks the
// senders are split over blocks, whose partial rows a second kernel joins.
// Bound by the latency of its few tiles (128 molecules of 9 to 70 atoms, 8 FP32
// heads of 16: 21 us) and, on long FP32 structures, by the three TF32 products of
// mma.sync (2 of 1000 nodes, 8 heads of 128, cap and bias: 335 us, 24 TFLOP/s of
// 4 n^2 H D).
#include <math.h>

#include "fc_attention.cuh"

namespace fc {

template <class T, int DP, int WM, int WN>
struct StripSmem {
  static constexpr int BW = WM == 1 || (sizeof(T) == 4 && DP > 64) ? 16 : 32;   // a warp's part of a key tile
  static constexpr int ROWS = 16 * WM, BN = WN * BW, S = kStride<T, DP>, threads = 32 * WM * WN;
  static constexpr size_t kv = sizeof(T) * BN * S, q = sizeof(T) * ROWS * S;
  static constexpr size_t merge = WN * ROWS * (DP + 2) * sizeof(float);   // over keys and values
  static constexpr size_t bytes = q + 4 * kv + 2 * BN * sizeof(float4);
  static_assert(merge <= 4 * kv && bytes <= 232448, "shared memory");
};

// The two rows of a thread (lane/4 and 8 more of a strip) and their running state.
struct StripRows {
  float px[2], py[2], pz[2], sl[2], mul, cap2;
  __device__ __forceinline__ StripRows(const AttnArgs& a, long long first, long long end, int kvh) {
    const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long r = first + g + 8 * h < end ? first + g + 8 * h : end - 1;
      px[h] = py[h] = pz[h] = sl[h] = 0.0f;
      if (a.pos_r) {
        const float* p = a.pos_r + 3 * (r / a.G);
        px[h] = p[0]; py[h] = p[1]; pz[h] = p[2];
        sl[h] = a.slope[kvh * a.G + r % a.G] * kLog2e;
      }
    }
    mul = a.cap > 0.0f ? a.scale / a.cap : a.scale * kLog2e;
    cap2 = a.cap * kLog2e;
  }
};
template <int DP>
struct StripState {
  float acc[DP / 8][4], m[2], l[2];
  __device__ __forceinline__ StripState() {
#pragma unroll
    for (int d = 0; d < DP / 8; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[d][e] = 0.0f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.0f;
  }
};

// One warp: 16 rows at q against 8 nl keys and values; in: position of each, w = 1 if not there.
template <class T, int DP, int NT, bool Two>
__device__ __forceinline__ void strip_step(const AttnArgs& a, const StripRows& r, StripState<DP>& state, const T* q,
                                           const T* k, const T* v, const float4* in, int nl, bool ragged) {
  const int c2 = 2 * (threadIdx.x & 3);
  float s[NT][4];
  strip_nt<T, DP, NT>(s, q, k, nl);
  if (a.cap > 0.0f) strip_tanh<T, NT>(s, r.mul);
  const float f = a.cap > 0.0f ? r.cap2 : r.mul;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[n][e] *= f;
  if (a.pos_r) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float4 p = in[n * 8 + c2 + c];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float dx = r.px[h] - p.x, dy = r.py[h] - p.y, dz = r.pz[h] - p.z;
          const float d2 = dx * dx + dy * dy + dz * dz;
          s[n][2 * h + c] -= r.sl[h] * (d2 * rsq(d2 + kD2Seed));
        }
      }
  }
  if (ragged) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (in[n * 8 + c2 + c].w != 0.0f) s[n][c] = s[n][2 + c] = -INFINITY;
  }
  float alpha[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float mx = state.m[h];
#pragma unroll
    for (int n = 0; n < NT; ++n) mx = fmaxf(mx, fmaxf(s[n][2 * h], s[n][2 * h + 1]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const float base = mx == -INFINITY ? 0.0f : mx;
    alpha[h] = ex2(state.m[h] - base);
    state.m[h] = mx;
    float sum = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float p = ex2(s[n][2 * h + c] - base);
        s[n][2 * h + c] = p;
        sum += p;
      }
    state.l[h] = state.l[h] * alpha[h] + sum;
  }
  strip_pn<T, DP, NT, Two>(state.acc, s, v, alpha[0], alpha[1], nl);
}

template <class T, int DP, bool Two, int WM, int WN>
__global__ void __launch_bounds__(32 * WM * WN) attn_strip_kernel(AttnArgs a) {
  using L = StripSmem<T, DP, WM, WN>;
  constexpr int BN = L::BN, NT = L::BW / 8, S = kStride<T, DP>, ROWS = L::ROWS, TH = L::threads;
  extern __shared__ __align__(16) unsigned char smem[];
  T* qs = reinterpret_cast<T*>(smem);
  T* ks = qs + ROWS * S;           // two stages
  T* vs = ks + 2 * BN * S;
  float4* info = reinterpret_cast<float4*>(vs + 2 * BN * S);   // [2][BN]: sender position, w = 1 if not there
  TileAt at;
  if (!find_tile(a.recv_ptr, a.B, a.nr, a.G, ROWS, blockIdx.x, at)) return;
  const int kvh = blockIdx.y, tid = threadIdx.x, lane = tid & 31, wm = (tid >> 5) % WM, wn = (tid >> 5) / WM;
  int slo, shi;
  other_side(a.send_ptr, a.B, a.ns, at.b, slo, shi);
  const long long all = shi > slo ? ((long long)shi - slo + BN - 1) / BN : 0;
  const int t0 = (int)(all * blockIdx.z / a.splits), t1 = (int)(all * (blockIdx.z + 1) / a.splits);
  const T* q = static_cast<const T*>(a.q);
  const T* k = static_cast<const T*>(a.k) + (long long)kvh * a.D;
  const T* v = static_cast<const T*>(a.v) + (long long)kvh * a.D;
  auto qrow = [&](int r) {
    const long long vr = at.v0 + r < at.v1 ? at.v0 + r : at.v0;
    return q + vr / a.G * a.ldq + (kvh * a.G + vr % a.G) * (long long)a.D;
  };
  load_rows<T, DP, ROWS, TH>(qs, a.D, tid, qrow, [&](int r) { return at.v0 + r < at.v1; });
  auto load_kv = [&](int t, int st) {
    const long long j0 = slo + (long long)t * BN;
    auto live = [&](int r) { return j0 + r < shi && (!a.mask || a.mask[j0 + r]); };
    load_rows2<T, DP, BN, TH>(
        ks + st * BN * S, vs + st * BN * S, a.D, tid, [&](int r) { return k + (j0 + r) * a.ldk; },
        [&](int r) { return v + (j0 + r) * a.ldv; }, live);
    for (int r = tid; r < BN; r += TH) {
      float4 f = make_float4(0.f, 0.f, 0.f, live(r) ? 0.f : 1.f);
      if (a.pos_r && live(r)) {
        const float* p = a.pos_s + 3 * (j0 + r);
        f.x = p[0]; f.y = p[1]; f.z = p[2];
      }
      info[st * BN + r] = f;
    }
  };
  if (t0 < t1) load_kv(t0, 0);
  cp_commit();

  StripRows rows(a, at.v0 + wm * 16, at.v1, kvh);
  StripState<DP> state;
  const bool idle = at.v0 + wm * 16 >= at.v1;   // none of the warp's rows is there
  for (int t = t0; t < t1; ++t) {
    const int st = (t - t0) & 1;
    if (t + 1 < t1) load_kv(t + 1, st ^ 1);
    cp_commit();
    cp_wait<1>();
    __syncthreads();
    const int b = st * BN + wn * L::BW;
    const long long left = shi - slo - (long long)t * BN - wn * L::BW;
    const int nl = idle || left <= 0 ? 0 : left >= L::BW ? NT : (int)(left + 7) / 8;
    if (nl > 0)
      strip_step<T, DP, NT, Two>(a, rows, state, qs + wm * 16 * S, ks + b * S, vs + b * S, info + b, nl, a.mask || left < L::BW);
    __syncthreads();
  }
  cp_wait<0>();

  // merge: [part][rows] of DP values, maximum and sum
  float* mg = reinterpret_cast<float*>(ks);
  constexpr int MS = DP + 2;
  const int g = lane >> 2, c2 = 2 * (lane & 3);
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float sum = state.l[h];
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    float* to = mg + (wn * ROWS + wm * 16 + g + 8 * h) * MS;
#pragma unroll
    for (int d = 0; d < DP / 8; ++d) {
      to[d * 8 + c2] = state.acc[d][2 * h];
      to[d * 8 + c2 + 1] = state.acc[d][2 * h + 1];
    }
    if ((lane & 3) == 0) {
      to[DP] = state.m[h];
      to[DP + 1] = sum;
    }
  }
  __syncthreads();
  const int quads = a.D / 4;
  for (int i = tid; i < ROWS * quads; i += TH) {
    const int r = i / quads, c = (i - r * quads) * 4;
    const long long vr = at.v0 + r;
    if (vr >= at.v1) break;
    float m = -INFINITY, sum = 0.0f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WN; ++w) m = fmaxf(m, mg[(w * ROWS + r) * MS + DP]);
    const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int w = 0; w < WN; ++w) {
      const float* f = mg + (w * ROWS + r) * MS;
      const float e = ex2(f[DP] - base);
      sum += e * f[DP + 1];
#pragma unroll
      for (int n = 0; n < 4; ++n) x[n] += e * f[c + n];
    }
    const long long node = vr / a.G;
    const int head = kvh * a.G + (int)(vr % a.G);
    const long long row = node * a.H + head;
    if (a.splits > 1) {
      const long long pr = (long long)blockIdx.z * a.nr * a.H + row;
      if (c == 0) a.part_ml[pr] = make_float2(m, sum);
      store_pack<float, 4>(a.part + pr * a.D + c, x);
      continue;
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (a.lse && c == 0) a.lse[row] = (m + log2f(sum)) * kLn2;
#pragma unroll
    for (int n = 0; n < 4; ++n) x[n] *= inv;
    store_pack<T, 4>(static_cast<T*>(a.out) + node * a.ldo + (long long)head * a.D + c, x);
    if (a.o32) store_pack<float, 4>(a.o32 + row * a.D + c, x);
  }
}

// Joins the parts of a row: the largest maximum, the parts rescaled to it.
// One warp per row and head.
template <class T>
__global__ void __launch_bounds__(256) attn_join_kernel(AttnArgs a) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const long long node = row / a.H;
  const int head = (int)(row - node * a.H);
  if (node >= a.nr) return;
  const long long step = (long long)a.nr * a.H;
  float m = -INFINITY;
  for (int s = lane; s < a.splits; s += 32) m = fmaxf(m, a.part_ml[s * step + row].x);
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float base = m == -INFINITY ? 0.0f : m;
  float sum = 0.0f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  const int c = lane * 4;
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    const float2 ml = a.part_ml[s * step + row];
    const float w = ex2(ml.x - base);
    sum += w * ml.y;
    if (c < a.D) {
      const float4 v = *reinterpret_cast<const float4*>(a.part + (s * step + row) * a.D + c);
      acc[0] += w * v.x; acc[1] += w * v.y; acc[2] += w * v.z; acc[3] += w * v.w;
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (a.lse && lane == 0) a.lse[row] = (m + log2f(sum)) * kLn2;
  if (c < a.D) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] *= inv;
    store_pack<T, 4>(static_cast<T*>(a.out) + node * a.ldo + (long long)head * a.D + c, acc);
    if (a.o32) store_pack<float, 4>(a.o32 + row * a.D + c, acc);
  }
}

// ----------------------------------------------------------------- launches

int check_attn(const fc_attn_desc* d, int n_struct, int n_recv, int n_send) {
  if (!d || !row_dtype(d->dtype) || n_struct < 0 || n_recv < 0 || n_send < 0) return FC_ERR_ARG;
  if (n_struct > kMaxStruct) return FC_ERR_ARG;
  if (d->heads < 1 || d->kv_heads < 1 || d->heads > 1024 || d->kv_heads > d->heads || d->heads % d->kv_heads)
    return FC_ERR_ARG;
  if (d->head_dim < 8 || d->head_dim > 128) return FC_ERR_ARG;
  if (!isfinite(d->scale * kLog2e) || !isfinite(d->cap * kLog2e) || d->cap < 0.0f) return FC_ERR_ARG;
  if (d->cap > 0.0f && !isfinite(d->scale / d->cap)) return FC_ERR_ARG;   // 0 times it would be NaN
  if (d->head_dim % 8) return FC_ERR_ALIGN;
  return FC_OK;
}

int attn_pad(int head_dim) { return head_dim <= 16 ? 16 : head_dim <= 32 ? 32 : head_dim <= 64 ? 64 : 128; }

// Parts of the streamed side: enough blocks to fill the card, each part at
// least four product steps of an average structure.
static int parts(long long blocks, long long fill, long long per, int step) {
  const long long want = blocks > 0 ? fill / blocks : 1, most = per / (4 * step);
  long long s = want < most ? want : most;
  if (s > 64) s = 64;
  return s < 1 ? 1 : (int)s;
}

// 16-bit rows go to the tcgen05 kernels from this many rows of an average
// structure on (and 64 senders).  They hold 128 rows and pad the head to 64 or
// 128 values, so wide heads gain first; strips fill the second tile of 130 to 200
// rows better, but only where there are blocks for more than two waves (`many`; 24
// structures of 160 rows of 64: 26/36, 16 of them 25/25).
// B structures, 8 BF16 heads, capped and biased, strips against tcgen05 in us:
//   forward, D 128: B 64: 64 rows 40/40, 72 rows 60/48;  B 16: 72 rows 23/19
//     D 64: B 64: 128 rows 42/46, 160 rows 66/81, 192 rows 76/83, 200 rows 103/91, 300 rows 170/146;
//           B 16: 128 rows 20/19, 192 rows 28/25;  B 4: 128 rows 24/19, 192 rows 21/19
//     D 32: B 64: 256 rows 79/91, 448 rows 202/209, 512 rows 251/226;  B 16: 256 rows 31/27, 448 rows 69/60;
//           B 4: 512 rows 39/22
//     D 16: B 64: 512 rows 210/222, 640 rows 316/316, 768 rows 444/419;  B 16: 256 rows 27/27;  B 4: 512 rows 34/23
//   gradient, D 128: B 64: 64 rows 130/106
//     D 64: B 64: 64 rows 67/92, 72 rows 124/105, 192 rows 275/222
//     D 32: B 64, no bias: 192 rows 137/144, 224 rows 196/157;  biased: 256 rows 279/237
//     D 16: B 64: 256 rows 238/227, 320 rows 344/361, 384 rows 455/397
static int tc_rows(int D, bool vjp, bool many) {
  if (vjp) return D > 64 ? 48 : D > 32 ? 72 : D > 16 ? 224 : 384;
  if (D > 64) return 72;
  if (!many) return D > 32 ? 128 : 256;
  return D > 32 ? 200 : D > 16 ? 448 : 640;
}
AttnPlan attn_plan(const fc_attn_desc* d, int B, int nr, int ns) {
  AttnPlan p;
  const int G = d->heads / d->kv_heads, KV = d->kv_heads, sms = device_sm_count();
  const long long rows = (long long)nr * G, per_r = B > 0 ? rows / B : 0, per_s = B > 0 ? ns / B : 0;
  const int step = d->dtype == FC_F32 && d->head_dim > 64 ? 32 : 64;
  // (rows and the end of a tensor copy's box past the last sender fit 31 bits)
  const bool can = d->dtype != FC_F32 && per_s >= 64 && rows <= INT32_MAX - 64 && ns <= INT32_MAX - 64;
  const auto tiles = [&](long long n, int tile) { return (n + tile - 1) / tile > B ? (n + tile - 1) / tile : B; };
  const bool many = B * ((per_r + 127) / 128) * KV > 2 * sms;   // more than two waves of tiles of 128
  p.tc = can && per_r >= tc_rows(d->head_dim, false, many);
  p.tc_vjp = can && per_r >= tc_rows(d->head_dim, true, many) && G <= 64;
  // few: up to two 16-row tiles a structure
  p.few = !p.tc && per_r <= 32;
  p.splits = p.tc    ? parts(tiles(rows, 128) * KV, sms, per_s, 64)
             : p.few ? parts(tiles(rows, 16) * KV, 4 * sms, per_s, 64)
                     : parts(tiles(rows, 64) * KV, 2 * sms, per_s, step);
  p.q_splits = p.tc_vjp ? parts(tiles(rows, 128) * KV, sms, per_s, 64)
                        : parts(tiles(rows, 64) * KV, 2 * sms, per_s, step);
  p.kv_splits = p.tc_vjp ? parts(tiles(ns, 128) * KV, sms, per_r, 64)
                         : parts(tiles(ns, 64) * KV, 2 * sms, per_r, step);
  return p;
}

template <class T, int DP, bool Two, int WM, int WN>
static int run_strip(const AttnArgs& a, cudaStream_t s) {
  static DeviceFlags ready;
  using L = StripSmem<T, DP, WM, WN>;
  if (set_smem_once(ready, attn_strip_kernel<T, DP, Two, WM, WN>, L::bytes) != FC_OK) return FC_ERR_CUDA;
  attn_strip_kernel<T, DP, Two, WM, WN>
      <<<dim3((unsigned)tile_slots(a.B, a.nr, a.G, L::ROWS), a.KV, a.splits), L::threads, L::bytes, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? FC_OK : FC_ERR_CUDA;
}
template <class T, int DP, bool Two>
static int run_attn(bool few, const AttnArgs& a, cudaStream_t s) {
  if (few) return run_strip<T, DP, Two, 1, 4>(a, s);
  // two halves of a key tile where a tile's bytes leave one block per SM: 128 molecules of 9 to 70
  // atoms take 23 us with one and 30 with two, 2048 nodes of 8 FP32 heads of 128 the other way round
  return run_strip<T, DP, Two, 4, (sizeof(T) == 4 && DP > 64) ? 2 : 1>(a, s);
}

template <class T>
static int run_strips(bool few, const AttnArgs& a, cudaStream_t s) {
  const bool two = sizeof(T) == 2 && a.o32;
  switch (attn_pad(a.D)) {
    case 16: return two ? run_attn<T, 16, sizeof(T) == 2>(few, a, s) : run_attn<T, 16, false>(few, a, s);
    case 32: return two ? run_attn<T, 32, sizeof(T) == 2>(few, a, s) : run_attn<T, 32, false>(few, a, s);
    case 64: return two ? run_attn<T, 64, sizeof(T) == 2>(few, a, s) : run_attn<T, 64, false>(few, a, s);
    default: return two ? run_attn<T, 128, sizeof(T) == 2>(few, a, s) : run_attn<T, 128, false>(few, a, s);
  }
}

template <class T>
static int run_attn_type(int dtype, const AttnPlan& plan, const AttnArgs& a, cudaStream_t s) {
  const int rc = plan.tc && a.ns > 0 ? launch_attn_fwd_tc(dtype, a, s) : run_strips<T>(plan.few, a, s);
  if (rc != FC_OK || a.splits == 1) return rc;
  attn_join_kernel<T><<<(unsigned)(((long long)a.nr * a.H + 7) / 8), 256, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? FC_OK : FC_ERR_CUDA;
}

}  // namespace fc

using namespace fc;

extern "C" {

size_t fc_node_attention_workspace_size(const fc_attn_desc* desc, int n_struct, int n_recv, int n_send) {
  if (check_attn(desc, n_struct, n_recv, n_send) != FC_OK || n_recv == 0) return 0;
  const int sp = attn_plan(desc, n_struct, n_recv, n_send).splits;
  if (sp == 1) return 0;
  const size_t rows = (size_t)sp * n_recv * desc->heads;
  return round16(rows * desc->head_dim * sizeof(float)) + round16(rows * sizeof(float2));
}

int fc_node_attention_on_tcgen05(const fc_attn_desc* desc, int n_struct, int n_recv, int n_send, int vjp) {
  if (check_attn(desc, n_struct, n_recv, n_send) != FC_OK) return -1;
  const AttnPlan plan = attn_plan(desc, n_struct, n_recv, n_send);
  return n_recv > 0 && n_send > 0 && (vjp ? plan.tc_vjp : plan.tc);
}

int fc_node_attention(const fc_attn_desc* desc, int n_struct, int n_recv, int n_send, const int32_t* recv_ptr,
                      const int32_t* send_ptr, const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v,
                      int64_t ldv, const float* pos_recv, const float* pos_send, const float* slope,
                      const uint8_t* send_mask, void* out, int64_t ldo, float* lse, float* out_f32, void* workspace,
                      size_t ws_bytes, fc_stream_t stream) {
  const int st = check_attn(desc, n_struct, n_recv, n_send);
  if (st != FC_OK) return st;
  if (n_recv == 0) return FC_OK;
  const int D = desc->head_dim, H = desc->heads, KV = desc->kv_heads;
  if (!recv_ptr || !send_ptr || !q || !out || (n_send > 0 && (!k || !v))) return FC_ERR_ARG;
  if (!pos_recv != !slope || (pos_send && !pos_recv)) return FC_ERR_ARG;
  if (pos_recv && !pos_send && n_recv != n_send) return FC_ERR_ARG;
  if (ldq < (int64_t)H * D || ldo < (int64_t)H * D || (n_send > 0 && (ldk < (int64_t)KV * D || ldv < (int64_t)KV * D)))
    return FC_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(k) || !aligned16(v) || !aligned16(out_f32) || ldq % 8 || ldk % 8 ||
      ldv % 8 || ldo % 8 || !aligned4(recv_ptr) || !aligned4(send_ptr) || !aligned4(pos_recv) || !aligned4(pos_send) ||
      !aligned4(slope) || !aligned4(lse))
    return FC_ERR_ALIGN;
  AttnArgs a{};
  a.B = n_struct; a.nr = n_recv; a.ns = n_send; a.H = H; a.KV = KV; a.G = H / KV; a.D = D;
  a.scale = desc->scale; a.cap = desc->cap;
  a.ldq = ldq; a.ldk = ldk; a.ldv = ldv; a.ldo = ldo;
  a.recv_ptr = recv_ptr; a.send_ptr = send_ptr; a.q = q; a.k = k; a.v = v;
  a.pos_r = pos_recv; a.pos_s = pos_send ? pos_send : pos_recv; a.slope = slope; a.mask = send_mask;
  a.out = out; a.lse = lse; a.o32 = out_f32;
  const AttnPlan plan = attn_plan(desc, n_struct, n_recv, n_send);
  a.splits = plan.splits;
  if (tile_slots(a.B, a.nr, a.G, 16) > INT32_MAX) return FC_ERR_ARG;
  if (a.splits > 1) {
    const size_t need = fc_node_attention_workspace_size(desc, n_struct, n_recv, n_send);
    if (!workspace || ws_bytes < need) return FC_ERR_WORKSPACE;
    if (!aligned16(workspace)) return FC_ERR_ALIGN;
    a.part = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) +
                                          round16((size_t)a.splits * n_recv * H * D * sizeof(float)));
  }
  cudaStream_t s = (cudaStream_t)stream;
  if (desc->dtype == FC_F32) return run_attn_type<float>(FC_F32, plan, a, s);
  if (desc->dtype == FC_BF16) return run_attn_type<__nv_bfloat16>(FC_BF16, plan, a, s);
  return run_attn_type<__half>(FC_F16, plan, a, s);
}

}  // extern "C"

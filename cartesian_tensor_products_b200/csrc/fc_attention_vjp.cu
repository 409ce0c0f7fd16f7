// Node attention, gradient.
//
// Two passes over the score matrix, both recomputing the weights from the
// saved log-sums, so that every gradient is a sum held by one block and no
// atomics are needed: one block per 64 virtual rows for the query gradient
// (with the receiver and slope sums), one per 64 senders and key head for the
// key and value gradients (with the sender position sums; the heads of the
// group are virtual rows and sum by themselves).  A small kernel first forms
// delta = g . out from the FP32 output, and small ones at the end add the
// position and slope sums over heads and nodes.  Bound as the forward's strips
// are: 128 molecules of 9 to 70 atoms, 8 FP32 heads of 16, 74 us; 2 structures of
// 1000 nodes, 8 FP32 heads of 128, cap and bias, 1078 us.
#include <math.h>

#include "fc_attention.cuh"

namespace fc {

// [nr H]: log-sum in base 2 (+inf for rows without senders, whose weights are
// then 0) and delta.  Eight lanes per row and head.
template <class T>
__global__ void __launch_bounds__(256) attn_stat_kernel(AttnArgs a, const float* __restrict__ o32,
                                                        const float* __restrict__ lse, float2* __restrict__ stat) {
  const long long row = (long long)blockIdx.x * 32 + (threadIdx.x >> 3);
  const int lane = threadIdx.x & 7;
  const bool live = row < (long long)a.nr * a.H;
  const long long node = live ? row / a.H : 0;
  const T* g = static_cast<const T*>(a.g) + node * a.ldg + (live ? row - node * a.H : 0) * a.D;
  float d = 0.0f;
  if (live)
    for (int c = lane * 4; c < a.D; c += 32) {
      float x[4], y[4];
      load_pack<T, 4>(g + c, x);
      load_pack<float, 4>(o32 + row * a.D + c, y);
      d += x[0] * y[0] + x[1] * y[1] + x[2] * y[2] + x[3] * y[3];
    }
  for (int o = 4; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (live && lane == 0) {
    const float l = lse[row];
    stat[row] = make_float2(l == -INFINITY ? INFINITY : l * kLog2e, d);
  }
}

// Eight warps: 16 of the 64 resident rows and one half of every streamed tile
// each; the halves' sums meet at the end.
template <class T, int DP>
struct VjpSmem {
  static constexpr int BN = kStep<T, DP> == 64 && DP > 64 ? 32 : kStep<T, DP>;   // streamed rows
  static constexpr int S = kStride<T, DP>;
  static constexpr size_t tiles = sizeof(T) * 64 * S * 2 + sizeof(T) * BN * S * 4;
  static constexpr size_t bytes = tiles + 4 * BN * sizeof(float4);
  // Blocks per SM that the registers are held to.  A short structure is one tile
  // per block, whose latency a second block hides: 128 molecules of 9 to 70
  // atoms, 8 heads, gradient in us with one / two: FP32 32-wide 156/115, BF16
  // 64-wide 128/106 (spills and all).  FP32 64-wide is the other way round on
  // long structures (4 of 300 to 900 nodes 601/651; the molecules 233/201).
  static constexpr int blocks = sizeof(T) == 2 || DP <= 32 ? 2 : 1;
  static_assert(64 * (DP + 9) * sizeof(float) <= tiles && 64 * (2 * DP + 3) * sizeof(float) <= tiles && bytes <= 232448, "shared memory");
};

// Query gradient, receiver position sums and slope sums.  16-bit rows: delta is
// as exact as a forward with 16-bit weights, dP truncated by the tensor core, and
// what they miss adds up over a row (4e-6 of a BF16 slope gradient at 49 rows of
// some 90 senders).  The weights sum to 1, so that e = sum dt is that rest: the
// sums of P (dP - delta) x are those of dt x less e times those of P x.
template <class T, int DP>
__global__ void __launch_bounds__(256, VjpSmem<T, DP>::blocks) attn_vjp_q_kernel(AttnArgs a) {
  constexpr int BN = VjpSmem<T, DP>::BN, BH = BN / 2, NT = BH / 8, S = kStride<T, DP>;
  constexpr bool Rest = sizeof(T) == 2;
  constexpr int NS = Rest ? 9 : 4;   // sums of a row: position, slope; of the weights: the same; dt
  extern __shared__ __align__(16) unsigned char smem[];
  T* qs = reinterpret_cast<T*>(smem);
  T* gs = qs + 64 * S;
  T* ks = gs + 64 * S;
  T* vs = ks + 2 * BN * S;
  float4* info = reinterpret_cast<float4*>(vs + 2 * BN * S);
  TileAt at;
  if (!find_tile(a.recv_ptr, a.B, a.nr, a.G, 64, blockIdx.x, at)) return;
  const int kvh = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = (tid >> 5) & 3, half = tid >> 7;
  int slo, shi;
  other_side(a.send_ptr, a.B, a.ns, at.b, slo, shi);
  const long long all = shi > slo ? ((long long)shi - slo + BN - 1) / BN : 0;
  const int t0 = (int)(all * blockIdx.z / a.splits), t1 = (int)(all * (blockIdx.z + 1) / a.splits);
  const T* k = static_cast<const T*>(a.k) + (long long)kvh * a.D;
  const T* v = static_cast<const T*>(a.v) + (long long)kvh * a.D;
  auto rowat = [&](const T* base, long long ld, int r) {
    const long long vr = at.v0 + r < at.v1 ? at.v0 + r : at.v0;
    return base + vr / a.G * ld + (kvh * a.G + vr % a.G) * (long long)a.D;
  };
  auto inside = [&](int r) { return at.v0 + r < at.v1; };
  load_rows<T, DP, 64, 256>(qs, a.D, tid, [&](int r) { return rowat(static_cast<const T*>(a.q), a.ldq, r); }, inside);
  load_rows<T, DP, 64, 256>(gs, a.D, tid, [&](int r) { return rowat(static_cast<const T*>(a.g), a.ldg, r); }, inside);
  auto load_kv = [&](int t, int st) {
    const long long j0 = slo + (long long)t * BN;
    auto live = [&](int r) { return j0 + r < shi && (!a.mask || a.mask[j0 + r]); };
    load_rows2<T, DP, BN, 256>(
        ks + st * BN * S, vs + st * BN * S, a.D, tid, [&](int r) { return k + (j0 + r) * a.ldk; },
        [&](int r) { return v + (j0 + r) * a.ldv; }, live);
    if (tid < BN) {
      float4 f = make_float4(0.f, 0.f, 0.f, live(tid) ? 0.f : 1.f);
      if (a.pos_r && live(tid)) {
        const float* p = a.pos_s + 3 * (j0 + tid);
        f.x = p[0]; f.y = p[1]; f.z = p[2];
      }
      info[st * BN + tid] = f;
    }
  };
  if (t0 < t1) load_kv(t0, 0);
  cp_commit();

  const int g = lane >> 2, c2 = 2 * (lane & 3);
  long long vr[2];
  float px[2], py[2], pz[2], sl[2], lse2[2], delta[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    vr[h] = at.v0 + warp * 16 + g + 8 * h;
    const long long r = vr[h] < at.v1 ? vr[h] : at.v0;
    const int head = kvh * a.G + (int)(r % a.G);
    px[h] = py[h] = pz[h] = sl[h] = 0.0f;
    if (a.pos_r) {
      const float* p = a.pos_r + 3 * (r / a.G);
      px[h] = p[0]; py[h] = p[1]; pz[h] = p[2];
      sl[h] = a.slope[head];
    }
    const float2 st = a.stat[r / a.G * a.H + head];
    lse2[h] = vr[h] < at.v1 ? st.x : INFINITY;
    delta[h] = st.y;
  }
  const float mul = a.cap > 0.0f ? a.scale / a.cap : a.scale * kLog2e;
  const float cap2 = a.cap * kLog2e;
  float acc[DP / 8][4], sum[NS][2];
#pragma unroll
  for (int n = 0; n < NS; ++n) sum[n][0] = sum[n][1] = 0.0f;
#pragma unroll
  for (int d = 0; d < DP / 8; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[d][e] = 0.0f;

  const bool idle = at.v0 + warp * 16 >= at.v1;
  for (int t = t0; t < t1; ++t) {
    const int st = (t - t0) & 1;
    if (t + 1 < t1) load_kv(t + 1, st ^ 1);
    cp_commit();
    cp_wait<1>();
    __syncthreads();
    if (idle) {   // none of the warp's rows is there
      __syncthreads();
      continue;
    }
    const T *kt = ks + (st * BN + half * BH) * S, *vt = vs + (st * BN + half * BH) * S;
    const float4* in = info + st * BN + half * BH;
    const long long left = shi - slo - (long long)t * BN - half * BH;
    const int nl = left >= BH ? NT : left <= 0 ? 0 : (int)(left + 7) / 8;   // column tiles that are there
    float s[NT][4], dp[NT][4];
    strip_nt<T, DP, NT>(s, qs + warp * 16 * S, kt, nl);
    strip_nt<T, DP, NT>(dp, gs + warp * 16 * S, vt, nl);
    if (a.cap > 0.0f) strip_tanh<T, NT>(s, mul);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n >= nl) break;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float4 f = in[n * 8 + c2 + c];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float th = s[n][2 * h + c];
          float tt = fmaf(th, a.cap > 0.0f ? cap2 : mul, -lse2[h]);
          const float dc = a.cap > 0.0f ? fmaf(-th, th, 1.0f) : 1.0f;
          float dx = 0.f, dy = 0.f, dz = 0.f, inv = 0.f, dist = 0.f;
          if (a.pos_r) {
            dx = px[h] - f.x; dy = py[h] - f.y; dz = pz[h] - f.z;
            const float d2 = dx * dx + dy * dy + dz * dz;
            inv = rsq(d2 + kD2Seed);
            dist = d2 * inv;
            tt -= sl[h] * kLog2e * dist;
          }
          const float p = ex2(tt);
          const float dt = f.w != 0.0f ? 0.0f : p * (dp[n][2 * h + c] - delta[h]);
          if (a.pos_r) {
            const float w = dt * inv;
            sum[0][h] += w * dx; sum[1][h] += w * dy; sum[2][h] += w * dz;
            sum[3][h] += dt * dist;
            if constexpr (Rest) {
              const float pw = f.w != 0.0f ? 0.0f : p, wp = pw * inv;
              sum[4][h] += wp * dx; sum[5][h] += wp * dy; sum[6][h] += wp * dz;
              sum[7][h] += pw * dist;
              sum[8][h] += dt;
            }
          }
          s[n][2 * h + c] = dt * dc;
        }
      }
    }
    strip_pn<T, DP, NT, false>(acc, s, kt, 1.0f, 1.0f, nl);
    __syncthreads();
  }
  cp_wait<0>();
  __syncthreads();
  float* mg = reinterpret_cast<float*>(smem);   // [64] rows of the second half: DP values, NS sums

#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int o = 1; o < 4; o <<= 1)
#pragma unroll
      for (int n = 0; n < NS; ++n) sum[n][h] += __shfl_xor_sync(0xffffffffu, sum[n][h], o);
    float* m = mg + (warp * 16 + g + 8 * h) * (DP + NS);
    if (half == 1) {
#pragma unroll
      for (int d = 0; d < DP / 8; ++d) {
        m[d * 8 + c2] = acc[d][2 * h];
        m[d * 8 + c2 + 1] = acc[d][2 * h + 1];
      }
      if ((lane & 3) == 0)
#pragma unroll
        for (int n = 0; n < NS; ++n) m[DP + n] = sum[n][h];
    }
  }
  __syncthreads();
  if (half == 1) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (vr[h] >= at.v1) continue;
    const float* m = mg + (warp * 16 + g + 8 * h) * (DP + NS);
#pragma unroll
    for (int n = 0; n < NS; ++n) sum[n][h] += m[DP + n];
    const long long row = vr[h] / a.G * a.H + kvh * a.G + (int)(vr[h] % a.G);
    const long long pr = (long long)blockIdx.z * a.nr * a.H + row;
    if (a.rowpart && (lane & 3) == 0) {
      if constexpr (Rest) {
        if (a.splits > 1) {   // the row's parts meet in attn_row_fix_kernel
          a.rowmean[pr] = make_float4(-sl[h] * sum[4][h], -sl[h] * sum[5][h], -sl[h] * sum[6][h], -sum[7][h]);
          a.rowrest[pr] = sum[8][h];
        } else {
#pragma unroll
          for (int n = 0; n < 4; ++n) sum[n][h] -= sum[8][h] * sum[4 + n][h];
        }
      }
      a.rowpart[pr] = make_float4(-sl[h] * sum[0][h], -sl[h] * sum[1][h], -sl[h] * sum[2][h], -sum[3][h]);
    }
    if (!a.qb) continue;
#pragma unroll
    for (int d = 0; d < DP / 8; ++d) {
      if (d * 8 >= a.D) continue;
      const float v2[2] = {(acc[d][2 * h] + m[d * 8 + c2]) * a.scale, (acc[d][2 * h + 1] + m[d * 8 + c2 + 1]) * a.scale};
      if (a.splits > 1)
        store_pack<float, 2>(a.part + pr * a.D + d * 8 + c2, v2);
      else
        store_pack<T, 2>(static_cast<T*>(a.qb) + row * a.D + d * 8 + c2, v2);
    }
  }
}

// Key and value gradients and sender position sums.
template <class T, int DP>
__global__ void __launch_bounds__(256, VjpSmem<T, DP>::blocks) attn_vjp_kv_kernel(AttnArgs a) {
  constexpr int BN = VjpSmem<T, DP>::BN, BH = BN / 2, NT = BH / 8, S = kStride<T, DP>;
  extern __shared__ __align__(16) unsigned char smem[];
  T* ks = reinterpret_cast<T*>(smem);
  T* vs = ks + 64 * S;
  T* qs = vs + 64 * S;
  T* gs = qs + 2 * BN * S;
  float4* rpos = reinterpret_cast<float4*>(gs + 2 * BN * S);   // [2][BN]: receiver position, slope
  float4* rst = rpos + 2 * BN;                                 // [2][BN]: log-sum, delta
  TileAt at;
  if (!find_tile(a.send_ptr, a.B, a.ns, 1, 64, blockIdx.x, at)) return;
  const int kvh = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = (tid >> 5) & 3, half = tid >> 7;
  int rlo, rhi;
  other_side(a.recv_ptr, a.B, a.nr, at.b, rlo, rhi);
  const long long r0 = (long long)rlo * a.G, r1 = (long long)rhi * a.G;
  const long long all = r1 > r0 ? (r1 - r0 + BN - 1) / BN : 0;
  const long long t0 = all * blockIdx.z / a.kv_splits, steps = all * (blockIdx.z + 1) / a.kv_splits - t0;
  auto shown = [&](long long j) { return j < at.v1 && (!a.mask || a.mask[j]); };
  auto live = [&](int r) { return shown(at.v0 + r); };
  load_rows<T, DP, 64, 256>(
      ks, a.D, tid, [&](int r) { return static_cast<const T*>(a.k) + (at.v0 + r) * a.ldk + (long long)kvh * a.D; }, live);
  load_rows<T, DP, 64, 256>(
      vs, a.D, tid, [&](int r) { return static_cast<const T*>(a.v) + (at.v0 + r) * a.ldv + (long long)kvh * a.D; }, live);
  auto load_q = [&](long long t, int st) {
    const long long b = r0 + (t0 + t) * BN;
    auto at_row = [&](const T* base, long long ld, int r) {
      return base + (b + r) / a.G * ld + (kvh * a.G + (b + r) % a.G) * (long long)a.D;
    };
    auto in = [&](int r) { return b + r < r1; };
    load_rows<T, DP, BN, 256>(qs + st * BN * S, a.D, tid,
                              [&](int r) { return at_row(static_cast<const T*>(a.q), a.ldq, r); }, in);
    load_rows<T, DP, BN, 256>(gs + st * BN * S, a.D, tid,
                              [&](int r) { return at_row(static_cast<const T*>(a.g), a.ldg, r); }, in);
    if (tid < BN) {
      float4 p = make_float4(0.f, 0.f, 0.f, 0.f), s = make_float4(INFINITY, 0.f, 0.f, 0.f);
      if (b + tid < r1) {
        const long long node = (b + tid) / a.G;
        const int head = kvh * a.G + (int)((b + tid) % a.G);
        if (a.pos_r) p = make_float4(a.pos_r[3 * node], a.pos_r[3 * node + 1], a.pos_r[3 * node + 2], a.slope[head]);
        const float2 ld = a.stat[node * a.H + head];
        s.x = ld.x;
        s.y = ld.y;
      }
      rpos[st * BN + tid] = p;
      rst[st * BN + tid] = s;
    }
  };
  if (steps > 0) load_q(0, 0);
  cp_commit();

  const int g = lane >> 2, c2 = 2 * (lane & 3);
  long long vj[2];
  float px[2], py[2], pz[2];
  bool keep[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    vj[h] = at.v0 + warp * 16 + g + 8 * h;
    keep[h] = shown(vj[h]);
    px[h] = py[h] = pz[h] = 0.0f;
    if (a.pos_r && keep[h]) {
      const float* p = a.pos_s + 3 * vj[h];
      px[h] = p[0]; py[h] = p[1]; pz[h] = p[2];
    }
  }
  const float mul = a.cap > 0.0f ? a.scale / a.cap : a.scale * kLog2e;
  const float cap2 = a.cap * kLog2e;
  float dk[DP / 8][4], dv[DP / 8][4], bx[2] = {0.f, 0.f}, by[2] = {0.f, 0.f}, bz[2] = {0.f, 0.f};
#pragma unroll
  for (int d = 0; d < DP / 8; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) dk[d][e] = dv[d][e] = 0.0f;

  const bool idle = at.v0 + warp * 16 >= at.v1;
  for (long long t = 0; t < steps; ++t) {
    const int st = (int)(t & 1);
    if (t + 1 < steps) load_q(t + 1, st ^ 1);
    cp_commit();
    cp_wait<1>();
    __syncthreads();
    if (idle) {   // none of the warp's senders is there
      __syncthreads();
      continue;
    }
    const T *qt = qs + (st * BN + half * BH) * S, *gt = gs + (st * BN + half * BH) * S;
    const float4 *rp = rpos + st * BN + half * BH, *rs = rst + st * BN + half * BH;
    const long long left = r1 - r0 - (t0 + t) * BN - half * BH;
    const int nl = left >= BH ? NT : left <= 0 ? 0 : (int)(left + 7) / 8;   // column tiles that are there
    float s[NT][4], dp[NT][4];
    strip_nt<T, DP, NT>(s, ks + warp * 16 * S, qt, nl);
    strip_nt<T, DP, NT>(dp, vs + warp * 16 * S, gt, nl);
    if (a.cap > 0.0f) strip_tanh<T, NT>(s, mul);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n >= nl) break;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float4 f = rp[n * 8 + c2 + c];
        const float2 ld = *reinterpret_cast<const float2*>(&rs[n * 8 + c2 + c]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float th = s[n][2 * h + c];
          float tt = fmaf(th, a.cap > 0.0f ? cap2 : mul, -ld.x);
          const float dc = a.cap > 0.0f ? fmaf(-th, th, 1.0f) : 1.0f;
          float dx = 0.f, dy = 0.f, dz = 0.f, inv = 0.f;
          if (a.pos_r) {
            dx = f.x - px[h]; dy = f.y - py[h]; dz = f.z - pz[h];
            const float d2 = dx * dx + dy * dy + dz * dz;
            inv = rsq(d2 + kD2Seed);
            tt -= f.w * kLog2e * (d2 * inv);
          }
          const float p = keep[h] ? ex2(tt) : 0.0f;
          const float dt = keep[h] ? p * (dp[n][2 * h + c] - ld.y) : 0.0f;
          if (a.pos_r) {
            const float w = dt * f.w * inv;
            bx[h] += w * dx; by[h] += w * dy; bz[h] += w * dz;
          }
          s[n][2 * h + c] = p;
          dp[n][2 * h + c] = dt * dc;
        }
      }
    }
    strip_pn<T, DP, NT, false>(dv, s, gt, 1.0f, 1.0f, nl);
    strip_pn<T, DP, NT, false>(dk, dp, qt, 1.0f, 1.0f, nl);
    __syncthreads();
  }
  cp_wait<0>();
  __syncthreads();
  float* mg = reinterpret_cast<float*>(smem);   // [64] rows of the second half: DP and DP values, three sums
  constexpr int MS = 2 * DP + 3;

#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      bx[h] += __shfl_xor_sync(0xffffffffu, bx[h], o);
      by[h] += __shfl_xor_sync(0xffffffffu, by[h], o);
      bz[h] += __shfl_xor_sync(0xffffffffu, bz[h], o);
    }
    float* m = mg + (warp * 16 + g + 8 * h) * MS;
    if (half == 1) {
#pragma unroll
      for (int d = 0; d < DP / 8; ++d)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[d * 8 + c2 + e] = dk[d][2 * h + e];
          m[DP + d * 8 + c2 + e] = dv[d][2 * h + e];
        }
      if ((lane & 3) == 0) {
        m[2 * DP] = bx[h]; m[2 * DP + 1] = by[h]; m[2 * DP + 2] = bz[h];
      }
    }
  }
  __syncthreads();
  if (half == 1) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (vj[h] >= at.v1) continue;
    const float* m = mg + (warp * 16 + g + 8 * h) * MS;
    bx[h] += m[2 * DP]; by[h] += m[2 * DP + 1]; bz[h] += m[2 * DP + 2];
    if (a.colpart && (lane & 3) == 0)
      a.colpart[((long long)blockIdx.z * a.KV + kvh) * a.ns + vj[h]] =
          keep[h] ? make_float4(bx[h], by[h], bz[h], 0.f) : make_float4(0.f, 0.f, 0.f, 0.f);
    const long long row = vj[h] * a.KV + kvh;
    // a hidden sender's row is 0 even where the receivers hold NaN
#pragma unroll
    for (int d = 0; d < DP / 8; ++d) {
      if (d * 8 >= a.D) continue;
      float k2[2], v2[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        k2[e] = keep[h] ? (dk[d][2 * h + e] + m[d * 8 + c2 + e]) * a.scale : 0.0f;
        v2[e] = keep[h] ? dv[d][2 * h + e] + m[DP + d * 8 + c2 + e] : 0.0f;
      }
      if (a.kv_splits > 1) {
        const long long pr = ((long long)blockIdx.z * a.ns * a.KV + row) * a.D + d * 8 + c2;
        if (a.kb) store_pack<float, 2>(a.part_k + pr, k2);
        if (a.vb) store_pack<float, 2>(a.part_v + pr, v2);
        continue;
      }
      if (a.kb) store_pack<T, 2>(static_cast<T*>(a.kb) + row * a.D + d * 8 + c2, k2);
      if (a.vb) store_pack<T, 2>(static_cast<T*>(a.vb) + row * a.D + d * 8 + c2, v2);
    }
  }
}

// Adds the parts of gradient rows, one warp per row: to[row] = sum of part[s][row].
template <class T>
__global__ void __launch_bounds__(256) attn_vjp_join_kernel(long long rows, int D, int splits,
                                                            const float* __restrict__ part, T* __restrict__ to) {
  const int c = (threadIdx.x & 31) * 4;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows || c >= D) return;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float4 v = *reinterpret_cast<const float4*>(part + (s * rows + row) * D + c);
    acc[0] += v.x; acc[1] += v.y; acc[2] += v.z; acc[3] += v.w;
  }
  store_pack<T, 4>(to + row * D + c, acc);
}

// The sums over heads and nodes, in one launch (the parts are small: 128
// molecules took 4 us for the positions and 6 for the slopes one after the
// other).  Blocks 0 .. slopes - 1: the slope gradient of one head, summed in
// FP64, as the terms of a row cancel and there is one for every row.  Then the
// position gradients, one warp per node: `recv` blocks for the receivers' parts
// and heads (with the sender's key heads where the senders are the receivers),
// the rest for the senders' key heads.
__global__ void __launch_bounds__(256) attn_sums_kernel(AttnArgs a, int slopes, int recv, bool self,
                                                        float* __restrict__ pos_recv, float* __restrict__ pos_send,
                                                        float* __restrict__ slope) {
  __shared__ double sum[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, block = (int)blockIdx.x - slopes;
  if (block < 0) {
    const int h = blockIdx.x;
    double v = 0.0;
    for (int s = 0; s < a.splits; ++s)
#pragma unroll 8
      for (long long i = threadIdx.x; i < a.nr; i += 256) v += a.rowpart[((long long)s * a.nr + i) * a.H + h].w;
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) sum[warp] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < 8; ++w) v += sum[w];
      slope[h] = (float)v;
    }
    return;
  }
  const bool of_recv = block < recv, of_send = !of_recv || self;
  const long long i = (long long)(of_recv ? block : block - recv) * 8 + warp;
  if (i >= (of_recv ? a.nr : a.ns)) return;
  float x = 0.f, y = 0.f, z = 0.f;
  if (of_recv)
    for (int e = lane; e < a.splits * a.H; e += 32) {
      const int sp = e / a.H;
      const float4 v = a.rowpart[((long long)sp * a.nr + i) * a.H + (e - sp * a.H)];
      x += v.x; y += v.y; z += v.z;
    }
  if (of_send)
    for (int e = lane; e < a.KV * a.kv_splits; e += 32) {
      const float4 v = a.colpart[(long long)e * a.ns + i];
      x += v.x; y += v.y; z += v.z;
    }
  for (int o = 16; o > 0; o >>= 1) {
    x += __shfl_xor_sync(0xffffffffu, x, o);
    y += __shfl_xor_sync(0xffffffffu, y, o);
    z += __shfl_xor_sync(0xffffffffu, z, o);
  }
  if (lane == 0) {
    float* bar = (of_recv ? pos_recv : pos_send) + 3 * i;
    bar[0] = x; bar[1] = y; bar[2] = z;
  }
}

// ----------------------------------------------------------------- launches

struct VjpLayout {
  AttnPlan plan;
  size_t stat, part, rowpart, rowmean, rowrest, colpart, part_k, part_v, bytes;
};
static VjpLayout vjp_layout(const fc_attn_desc* d, int B, int nr, int ns) {
  VjpLayout l;
  l.plan = attn_plan(d, B, nr, ns);
  const size_t rows = (size_t)nr * d->heads, cols = (size_t)ns * d->kv_heads;
  const size_t rp = rows * l.plan.q_splits, cp = cols * l.plan.kv_splits;
  const size_t pq = l.plan.q_splits > 1 ? round16(rp * d->head_dim * sizeof(float)) : 0;
  const size_t pk = l.plan.kv_splits > 1 ? round16(cp * d->head_dim * sizeof(float)) : 0;
  l.stat = 0;
  l.rowpart = round16(rows * sizeof(float2));
  l.rowmean = l.rowpart + rp * sizeof(float4);
  const bool rest = l.plan.tc_vjp || (d->dtype != FC_F32 && l.plan.q_splits > 1);
  l.rowrest = l.rowmean + (rest ? rp * sizeof(float4) : 0);
  l.colpart = l.rowrest + (rest ? round16(rp * sizeof(float)) : 0);
  l.part = l.colpart + cp * sizeof(float4);
  l.part_k = l.part + pq;
  l.part_v = l.part_k + pk;
  l.bytes = l.part_v + pk;
  return l;
}

struct VjpWants {
  bool kv, self;
  float *pos_recv_bar, *pos_send_bar, *slope_bar;
};

template <class T, int DP>
static int run_strips(bool kv, const AttnArgs& a, cudaStream_t s) {
  static DeviceFlags ready_q, ready_kv;
  constexpr size_t bytes = VjpSmem<T, DP>::bytes;
  if (kv) {
    if (set_smem_once(ready_kv, attn_vjp_kv_kernel<T, DP>, bytes) != FC_OK) return FC_ERR_CUDA;
    attn_vjp_kv_kernel<T, DP>
        <<<dim3((unsigned)tile_slots(a.B, a.ns, 1, 64), a.KV, a.kv_splits), 256, bytes, s>>>(a);
  } else {
    if (set_smem_once(ready_q, attn_vjp_q_kernel<T, DP>, bytes) != FC_OK) return FC_ERR_CUDA;
    attn_vjp_q_kernel<T, DP><<<dim3((unsigned)tile_slots(a.B, a.nr, a.G, 64), a.KV, a.splits), 256, bytes, s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? FC_OK : FC_ERR_CUDA;
}

template <class T>
static int run_side(int dtype, bool tc, bool kv, const AttnArgs& a, cudaStream_t s) {
  if (tc) return launch_attn_vjp_tc(dtype, kv, a, s);
  switch (attn_pad(a.D)) {
    case 16: return run_strips<T, 16>(kv, a, s);
    case 32: return run_strips<T, 32>(kv, a, s);
    case 64: return run_strips<T, 64>(kv, a, s);
    default: return run_strips<T, 128>(kv, a, s);
  }
}

template <class T>
static int run_vjp(int dtype, const AttnArgs& a, const VjpWants& w, bool tc, const float* o32, float2* stat,
                   cudaStream_t s) {
  const auto blocks = [](long long rows, int per) { return (unsigned)((rows + per - 1) / per); };
  const long long rows = (long long)a.nr * a.H, cols = (long long)a.ns * a.KV;
  int rc = FC_OK;
  if (a.nr > 0) attn_stat_kernel<T><<<blocks(rows, 32), 256, 0, s>>>(a, o32, a.lse, stat);
  AttnArgs sums = a;   // as the sums over heads and nodes see it
  if (a.nr > 0 && (a.qb || a.rowpart)) {
    rc = run_side<T>(dtype, tc, false, a, s);
    if (rc == FC_OK && a.rowpart && (tc || (sizeof(T) == 2 && a.splits > 1))) {
      // the strips leave delta as it is: it is what they are given for q_bar too
      rc = launch_attn_row_fix(a, tc ? stat : nullptr, s);
      sums.splits = 1;
    }
    if (a.qb && a.splits > 1)
      attn_vjp_join_kernel<T><<<blocks(rows, 8), 256, 0, s>>>(rows, a.D, a.splits, a.part, static_cast<T*>(a.qb));
  }
  if (rc == FC_OK && a.ns > 0 && w.kv) {
    rc = run_side<T>(dtype, tc, true, a, s);
    if (a.kv_splits > 1) {
      if (a.kb)
        attn_vjp_join_kernel<T><<<blocks(cols, 8), 256, 0, s>>>(cols, a.D, a.kv_splits, a.part_k, static_cast<T*>(a.kb));
      if (a.vb)
        attn_vjp_join_kernel<T><<<blocks(cols, 8), 256, 0, s>>>(cols, a.D, a.kv_splits, a.part_v, static_cast<T*>(a.vb));
    }
  }
  if (rc != FC_OK) return rc;
  const int slopes = w.slope_bar ? a.H : 0;
  const unsigned recv = w.pos_recv_bar ? blocks(a.nr, 8) : 0, send = w.pos_send_bar ? blocks(a.ns, 8) : 0;
  if (slopes + recv + send > 0)
    attn_sums_kernel<<<slopes + recv + send, 256, 0, s>>>(sums, slopes, (int)recv, w.self, w.pos_recv_bar, w.pos_send_bar,
                                                          w.slope_bar);
  return cudaGetLastError() == cudaSuccess ? FC_OK : FC_ERR_CUDA;
}

}  // namespace fc

using namespace fc;

extern "C" {

size_t fc_node_attention_vjp_workspace_size(const fc_attn_desc* desc, int n_struct, int n_recv, int n_send) {
  if (check_attn(desc, n_struct, n_recv, n_send) != FC_OK || (n_recv == 0 && n_send == 0)) return 0;
  return vjp_layout(desc, n_struct, n_recv, n_send).bytes;
}

int fc_node_attention_vjp(const fc_attn_desc* desc, int n_struct, int n_recv, int n_send, const int32_t* recv_ptr,
                          const int32_t* send_ptr, const void* q, int64_t ldq, const void* k, int64_t ldk,
                          const void* v, int64_t ldv, const float* pos_recv, const float* pos_send,
                          const float* slope, const uint8_t* send_mask, const float* out_f32, const float* lse,
                          const void* g, int64_t ldg, void* q_bar, void* k_bar, void* v_bar, float* pos_recv_bar,
                          float* pos_send_bar, float* slope_bar, void* workspace, size_t ws_bytes,
                          fc_stream_t stream) {
  const int st = check_attn(desc, n_struct, n_recv, n_send);
  if (st != FC_OK) return st;
  const int D = desc->head_dim, H = desc->heads, KV = desc->kv_heads;
  cudaStream_t s = (cudaStream_t)stream;
  if (!pos_recv != !slope || (pos_send && !pos_recv)) return FC_ERR_ARG;
  if (pos_recv && !pos_send && n_recv != n_send) return FC_ERR_ARG;
  if (!pos_recv && (pos_recv_bar || slope_bar)) return FC_ERR_ARG;
  if (!pos_send && pos_send_bar) return FC_ERR_ARG;
  if (!aligned4(slope_bar)) return FC_ERR_ALIGN;
  if (n_recv == 0 && n_send == 0) {
    if (slope_bar && cudaMemsetAsync(slope_bar, 0, sizeof(float) * H, s) != cudaSuccess) return FC_ERR_CUDA;
    return FC_OK;
  }
  if (!recv_ptr || !send_ptr || (n_recv > 0 && (!q || !g || !out_f32 || !lse)) || (n_send > 0 && (!k || !v)))
    return FC_ERR_ARG;
  if ((n_recv > 0 && (ldq < (int64_t)H * D || ldg < (int64_t)H * D)) ||
      (n_send > 0 && (ldk < (int64_t)KV * D || ldv < (int64_t)KV * D)))
    return FC_ERR_ARG;
  if (!aligned16(q) || !aligned16(g) || !aligned16(k) || !aligned16(v) || !aligned16(out_f32) || !aligned16(q_bar) ||
      !aligned16(k_bar) || !aligned16(v_bar) || ldq % 8 || ldk % 8 || ldv % 8 || ldg % 8 || !aligned4(recv_ptr) ||
      !aligned4(send_ptr) || !aligned4(pos_recv) || !aligned4(pos_send) || !aligned4(slope) || !aligned4(lse) ||
      !aligned4(pos_recv_bar) || !aligned4(pos_send_bar))
    return FC_ERR_ALIGN;
  const VjpLayout l = vjp_layout(desc, n_struct, n_recv, n_send);
  if (!workspace || ws_bytes < l.bytes) return FC_ERR_WORKSPACE;
  if (!aligned16(workspace)) return FC_ERR_ALIGN;
  if (tile_slots(n_struct, n_recv, H / KV, 64) > INT32_MAX || tile_slots(n_struct, n_send, 1, 64) > INT32_MAX)
    return FC_ERR_ARG;
  char* ws = static_cast<char*>(workspace);
  float2* stat = reinterpret_cast<float2*>(ws + l.stat);
  VjpWants w{};
  w.self = pos_recv && !pos_send;
  w.pos_recv_bar = pos_recv_bar;
  w.pos_send_bar = pos_send_bar;
  w.slope_bar = slope_bar;
  w.kv = k_bar || v_bar || pos_send_bar || (w.self && pos_recv_bar);
  AttnArgs a{};
  a.B = n_struct; a.nr = n_recv; a.ns = n_send; a.H = H; a.KV = KV; a.G = H / KV; a.D = D;
  a.scale = desc->scale; a.cap = desc->cap;
  a.ldq = ldq; a.ldk = ldk; a.ldv = ldv; a.ldg = ldg;
  a.recv_ptr = recv_ptr; a.send_ptr = send_ptr; a.q = q; a.k = k; a.v = v; a.g = g;
  a.pos_r = pos_recv; a.pos_s = pos_send ? pos_send : pos_recv; a.slope = slope; a.mask = send_mask;
  a.lse = const_cast<float*>(lse);
  a.splits = l.plan.q_splits;
  a.kv_splits = l.plan.kv_splits;
  a.part_k = reinterpret_cast<float*>(ws + l.part_k);
  a.part_v = reinterpret_cast<float*>(ws + l.part_v);
  a.stat = stat;
  // With a bias the tcgen05 kernels put delta right for the senders' side from the
  // row sums of the query gradient's kernel, which therefore runs for k_bar too:
  // what a gradient holds does not depend on which others are asked for.
  const bool tc = l.plan.tc_vjp && n_recv > 0 && n_send > 0;   // the tensor maps need rows on both sides
  const bool fix = tc && pos_recv && (k_bar || pos_send_bar);
  a.rowpart = pos_recv_bar || slope_bar || fix ? reinterpret_cast<float4*>(ws + l.rowpart) : nullptr;
  a.rowmean = reinterpret_cast<float4*>(ws + l.rowmean);
  a.rowrest = reinterpret_cast<float*>(ws + l.rowrest);
  a.colpart = pos_send_bar || (w.self && pos_recv_bar) ? reinterpret_cast<float4*>(ws + l.colpart) : nullptr;
  a.part = reinterpret_cast<float*>(ws + l.part);
  a.qb = q_bar; a.kb = k_bar; a.vb = v_bar;
  if (desc->dtype == FC_F32) return run_vjp<float>(FC_F32, a, w, false, out_f32, stat, s);
  if (desc->dtype == FC_BF16) return run_vjp<__nv_bfloat16>(FC_BF16, a, w, tc, out_f32, stat, s);
  return run_vjp<__half>(FC_F16, a, w, tc, out_f32, stat, s);
}

}  // extern "C"

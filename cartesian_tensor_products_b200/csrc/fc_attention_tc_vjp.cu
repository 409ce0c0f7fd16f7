// Node attention on the tensor cores (tcgen05), gradient.
//
// Both kernels hold two resident tiles R1, R2 of 128 rows and stream tiles T1,
// T2 of 64 rows.  Per stream tile, S = R1 T1^T and dP = R2 T2^T land in tensor
// memory; a group of 128 threads, one resident row each, turns them into the
// weights P and dS = P (dP - delta) (1 - tanh^2), written back over them in 16
// bits (half a unit of 2^-8 or 2^-11 each, averaged by the products), and the
// accumulating products stay in tensor memory:
//   query gradient         R = q, g; T = k, v:  q_bar += dS k
//   key, value gradients   R = k, v; T = q, g:  k_bar += dS q,  v_bar += P g
// The position and slope sums come from the FP32 values in registers.  Delta as
// it comes in is as exact as the forward's output, whose long sum the tensor
// core truncates (8e-6 of a slope gradient at 2300 senders, 1.6e-5 at 8192); the
// query gradient's kernel therefore sums dt and the weights' own position and
// slope sums too, from which attn_row_fix_kernel takes the rest out.  The two
// groups take the tiles in turn, so that one's arithmetic runs beside the
// other's products.  The heads of a key head are rows of the stream tile
// (64 / G receivers by G heads), so their sum needs no atomics.
//
// Bound like the forward, with the FP32 pipe ahead of the special functions (60 and
// 32 % busy in the query gradient, 50 and 33 % in the other).  Forward and
// gradient of 4096 nodes, 8 BF16 heads of 64, cap and bias: 651 us, the two
// kernels here 246 and 241 us of it.
#include <math.h>

#include "fc_attention_tc.cuh"

namespace fc {

__device__ int g_av_error = 0;
__device__ unsigned long long g_av_wait_ns = 500000000ull;

template <int DP, bool KV>
struct AtVjp {
  static constexpr int panels = DP / 64;
  static constexpr int stages = DP == 128 ? 4 : 6;
  static constexpr int bufs = DP == 128 && KV ? 2 : 3;   // S and dP tiles in tensor memory
  static constexpr uint32_t acc = bufs * 128;            // first accumulator column
  static constexpr int cols = KV ? 6 : 4;                // floats per stream row
  static constexpr size_t tile = (size_t)panels * kAtPanel, res = 2 * tile;
  static constexpr size_t info = cols * kAtStep * sizeof(float);
  static constexpr size_t off_stage = 2 * res, off_info = off_stage + stages * 2 * tile;
  static constexpr size_t off_bar = off_info + stages * info;
  static constexpr size_t bytes = off_bar + 8 * (3 * stages + 3 * bufs + 2) + 16;
  static_assert(bytes <= 232448 && acc + (KV ? 2 : 1) * DP <= 512, "shared or tensor memory");
};

// One resident row: its constants and sums.
template <class T, bool Cap, bool Bias, bool KV>
struct RowGrad {
  float2 mul, cap2, px, py, pz, sl, nl, nd;   // negated: slope (base 2), log-sum, delta
  TanhPoly poly;
  __device__ __forceinline__ explicit RowGrad(float m) : mul(pair(m)), poly(1.0f, m) {}
  // P (KV) and dS of 64 columns as 16-bit pairs; sums: position x, y, z, slope (query gradient)
  // (and, for the query gradient: the weights' sums of the same four, and the sum of dt)
  static constexpr int kSums = KV ? 3 : 9;
  template <bool Easy, bool Flags>
  __device__ __forceinline__ void tile(uint32_t st, const float* in, uint32_t (&w)[KV ? 2 : 1][32],
                                       float2 (&sum)[kSums], float& big) const {
    float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kSums; ++i) sum[i] = pair(0.0f);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t rs[32], rp[32];
      tmem_ld32_async(st + 32 * hf, rs);
      tmem_ld32_async(st + kAtStep + 32 * hf, rp);
      tmem_wait_ld(rs);
      tmem_wait_ld(rp);
      const float* f = in + 32 * hf;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float2 cl = KV ? lds2(f + 3 * kAtStep + 2 * e) : nl;
        float2 t, dc;
        if (Cap) {
          const float2 v = pair_at(rs, e);
          float2 th;
          if (Easy) {
            b[e & 3] = max3_abs(b[e & 3], v.x, v.y);
            th = mul2(v, poly(mul2(v, v)));
          } else {
            const float2 x = mul2(v, mul);
            th = make_float2(cap_tanh<T>(x.x), cap_tanh<T>(x.y));
          }
          t = fma2(th, cap2, cl);
          dc = fma2(make_float2(-th.x, -th.y), th, pair(1.0f));
        } else {
          t = fma2(pair_at(rs, e), mul, cl);
        }
        float2 dx, dy, dz, inv, dist, cs = sl;
        if (Bias) {
          dx = add2(px, lds2(f + 2 * e));
          dy = add2(py, lds2(f + kAtStep + 2 * e));
          dz = add2(pz, lds2(f + 2 * kAtStep + 2 * e));
          if (KV) cs = lds2(f + 5 * kAtStep + 2 * e);
          const float2 d2 = fma2(dx, dx, fma2(dy, dy, fma2(dz, dz, pair(kD2Seed))));
          inv = make_float2(rsq(d2.x), rsq(d2.y));
          dist = mul2(d2, inv);
          t = fma2(dist, cs, t);
        }
        if (Flags && !KV) t = add2(t, lds2(f + 3 * kAtStep + 2 * e));
        const float2 p = make_float2(ex2(t.x), ex2(t.y));
        const float2 dt = mul2(p, add2(pair_at(rp, e), KV ? lds2(f + 4 * kAtStep + 2 * e) : nd));
        if (Bias) {
          float2 wt = mul2(dt, inv);
          if (KV) wt = mul2(wt, cs);
          sum[0] = fma2(wt, dx, sum[0]);
          sum[1] = fma2(wt, dy, sum[1]);
          sum[2] = fma2(wt, dz, sum[2]);
          if constexpr (!KV) {
            const float2 wp = mul2(p, inv);
            sum[3] = fma2(dt, dist, sum[3]);
            sum[4] = fma2(wp, dx, sum[4]);
            sum[5] = fma2(wp, dy, sum[5]);
            sum[6] = fma2(wp, dz, sum[6]);
            sum[7] = fma2(p, dist, sum[7]);
            sum[8] = add2(sum[8], dt);
          }
        }
        const float2 ds = Cap ? mul2(dt, dc) : dt;
        w[0][16 * hf + e] = pack2<T>(ds.x, ds.y);
        if (KV) w[KV ? 1 : 0][16 * hf + e] = pack2<T>(p.x, p.y);
      }
    }
    if (Cap && Easy) big = max3(fmaxf(b[0], b[1]), b[2], b[3]);
  }
};

template <class T, int DP, bool KV, bool Cap, bool Bias>
__global__ void __launch_bounds__(kAtThreads, 1) attn_vjp_tc_kernel(AttnArgs a, const __grid_constant__ CUtensorMap map1,
                                                                const __grid_constant__ CUtensorMap map2) {
  using L = AtVjp<DP, KV>;
  constexpr int NST = L::stages, NB = L::bufs;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = tc::smem_addr(smem);
  auto kst = [&](int s) { return base + (uint32_t)(L::off_stage + s * 2 * L::tile); };   // T1, then T2
  auto info = [&](int s) { return reinterpret_cast<float*>(smem + L::off_info + s * L::info); };
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::off_bar);
  uint64_t *freeb = full + NST, *land = freeb + NST, *s_full = land + NST, *p_full = s_full + NB, *done = p_full + NB,
           *drain = done + NB, *r_full = drain + 1;
  uint32_t* slot = reinterpret_cast<uint32_t*>(r_full + 1);

  // resident rows: virtual receiver rows, or senders
  TileAt at;
  if (KV) {
    if (!find_tile(a.send_ptr, a.B, a.ns, 1, kAtRows, blockIdx.x, at)) return;
  } else {
    if (!find_tile(a.recv_ptr, a.B, a.nr, a.G, kAtRows, blockIdx.x, at)) return;
  }
  const int kvh = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // stream rows: senders, or `npt` receivers by G heads
  int slo, shi;
  if (KV)
    other_side(a.recv_ptr, a.B, a.nr, at.b, slo, shi);
  else
    other_side(a.send_ptr, a.B, a.ns, at.b, slo, shi);
  const int npt = KV ? kAtStep / a.G : kAtStep, group = KV ? a.G : 1;
  const int splits = KV ? a.kv_splits : a.splits;
  const int all = shi > slo ? (int)(((long long)shi - slo + npt - 1) / npt) : 0;
  const int t0 = (int)((long long)all * blockIdx.z / splits);
  const int nt = (int)((long long)all * (blockIdx.z + 1) / splits) - t0;

  if (warp == 8) tc::tmem_alloc(slot, 512);
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      tc::bar_init(&full[s], 1);
      tc::bar_init(&freeb[s], 1);
      tc::bar_init(&land[s], 1);
    }
    for (int b = 0; b < NB; ++b) {
      tc::bar_init(&s_full[b], 1);
      tc::bar_init(&p_full[b], 4);
      tc::bar_init(&done[b], 1);
    }
    tc::bar_init(drain, 1);
    tc::bar_init(r_full, kAtCopiers);
    tc::fence_bar_init();
  }
  // stream rows past npt receivers by G heads are never written: zeros
  if (KV && npt * group < kAtStep)
    for (int i = warp; i < NST * 2 * L::panels; i += 12)
      for (int r = npt * group + (lane >> 3); r < kAtStep; r += 4)
        zero_row(base + (uint32_t)L::off_stage + i * kAtPanel, r, lane);
  tc::fence_proxy_async();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *slot;
  const uint64_t lim = g_av_wait_ns;
  bool fail = false;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 8) {
      // ---------------- matrix products ----------------
      if (elect_one()) {
        const int ks = (a.D + 15) / 16;
        const uint32_t idesc_s = at_idesc<T>(kAtStep, false), idesc_o = at_idesc<T>(ks * 16, true);
        const uint64_t r1 = desc_k<kAtRows>(base), r2 = desc_k<kAtRows>(base + (uint32_t)L::res);
        auto scores = [&](int i) {
          if (!tc::bar_wait(&full[i % NST], (i / NST) & 1, lim)) return false;
          tc::fence_after_sync();
          const uint32_t ta = kst(i % NST), sd = tmem + (i % NB) * 128;
          const uint64_t d1 = desc_k<kAtStep>(ta), d2 = desc_k<kAtStep>(ta + (uint32_t)L::tile);
#pragma unroll
          for (int k = 0; k < DP / 16; ++k)
            if (k < ks) mma_ss16(sd, r1 + step_k<kAtRows>(k), d1 + step_k<kAtStep>(k), idesc_s, k != 0);
#pragma unroll
          for (int k = 0; k < DP / 16; ++k)
            if (k < ks) mma_ss16(sd + kAtStep, r2 + step_k<kAtRows>(k), d2 + step_k<kAtStep>(k), idesc_s, k != 0);
          tc::commit(&s_full[i % NB]);
          return true;
        };
        fail = !tc::bar_wait(r_full, 0, lim);
        for (int i = 0; i < NB && i < nt && !fail; ++i) fail = !scores(i);
        for (int i = 0; i < nt && !fail; ++i) {
          const int b = i % NB;
          if (!tc::bar_wait(&p_full[b], (i / NB) & 1, lim)) {
            fail = true;
            break;
          }
          tc::fence_after_sync();
          const uint32_t ta = kst(i % NST), sd = tmem + b * 128;
          const uint64_t d1 = desc_mn<kAtStep>(ta), d2 = desc_mn<kAtStep>(ta + (uint32_t)L::tile);
#pragma unroll
          for (int k = 0; k < kAtStep / 16; ++k)   // dS over dP
            mma_ts16(tmem + L::acc, sd + kAtStep + 8 * k, d1 + step_mn(k), idesc_o, (i | k) != 0);
          if (KV)
#pragma unroll
            for (int k = 0; k < kAtStep / 16; ++k)   // P over S
              mma_ts16(tmem + L::acc + DP, sd + 8 * k, d2 + step_mn(k), idesc_o, (i | k) != 0);
          tc::commit(&done[b]);
          tc::commit(&freeb[i % NST]);
          // the next scores into these columns once P and dS are read
          if (i + NB < nt) fail = !tc::bar_wait(&done[b], (i / NB) & 1, lim) || !scores(i + NB);
        }
        tc::commit(drain);
        if (!tc::bar_wait(drain, 0, kAtDrainNs)) fail = true;
      }
      __syncwarp();
    } else {
      // ---------------- copies ----------------
      const int cw = warp - 9;
      const T *s1 = static_cast<const T*>(KV ? a.k : a.q), *s2 = static_cast<const T*>(KV ? a.v : a.g);
      const long long ld1 = KV ? a.ldk : a.ldq, ld2 = KV ? a.ldv : a.ldg;
      // (none without a tile to meet: the sums at the end go over their place)
      for (int r0 = cw * 4; r0 < kAtRows && nt > 0; r0 += 12) {
        const long long vr = at.v0 + r0 + (lane >> 3);
        bool ok = vr < at.v1;
        if (KV) ok = ok && (!a.mask || a.mask[vr]);
        const uint32_t u = (uint32_t)(ok ? vr : at.v0), node = KV ? u : u / (uint32_t)a.G;
        const long long head = KV ? kvh : kvh * a.G + (int)(u - node * a.G);
#pragma unroll
        for (int p = 0; p < L::panels; ++p) {
          const int c = p * 64 + (lane & 7) * 8;
          const bool live = ok && c < a.D;
          copy_rows4(base + p * kAtRows * 128, r0, lane, s1 + node * ld1 + head * a.D + (live ? c : 0), live);
          copy_rows4(base + (uint32_t)L::res + p * kAtRows * 128, r0, lane, s2 + node * ld2 + head * a.D + (live ? c : 0), live);
        }
      }
      cp_wait_all();
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(r_full);
      const uint32_t bytes = (uint32_t)(2 * L::panels * npt * group * 128);
      for (int i = cw; i < nt; i += kAtCopiers) {
        const int s = i % NST, round = i / NST;
        if (round > 0 && !tc::warp_wait(&freeb[s], (round - 1) & 1, lim)) {
          fail = true;
          break;
        }
        const long long j0 = slo + (long long)(t0 + i) * npt;   // first sender or receiver
        if (elect_one()) {
          tc::bar_arrive_expect_tx(&land[s], bytes);
#pragma unroll
          for (int p = 0; p < L::panels; ++p) {
            load_panel(kst(s) + p * kAtPanel, &map1, p * 64, kvh * group, (int)j0, &land[s]);
            load_panel(kst(s) + (uint32_t)L::tile + p * kAtPanel, &map2, p * 64, kvh * group, (int)j0, &land[s]);
          }
        }
        __syncwarp();
        unsigned dead[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int r = 32 * n + lane, dn = r / group;
          const long long j = j0 + dn;
          float* f = info(s) + r;
          const bool tail = dn >= npt;   // rows that stay zero
          const bool ok = !tail && j < shi && (KV || !a.mask || a.mask[j]);
          const float* p = KV ? a.pos_r : a.pos_s;
          const bool there = Bias && ok;
          f[0] = there ? -p[3 * j] : 0.0f;
          f[kAtStep] = there ? -p[3 * j + 1] : 0.0f;
          f[2 * kAtStep] = there ? -p[3 * j + 2] : 0.0f;
          if (KV) {   // a row not there has log-sum +infinity: weight 0
            const int head = kvh * group + (r - dn * group);
            const float2 st = ok ? a.stat[j * a.H + head] : make_float2(INFINITY, 0.0f);
            f[3 * kAtStep] = -st.x;
            f[4 * kAtStep] = -st.y;
            f[5 * kAtStep] = there ? -a.slope[head] * kLog2e : 0.0f;
          } else {
            f[3 * kAtStep] = ok ? 0.0f : -INFINITY;
          }
          dead[n] = __ballot_sync(0xffffffffu, !ok && !tail);
        }
        if (!tc::warp_wait(&land[s], round & 1, lim)) {
          tc::warp_wait(&land[s], round & 1, kAtDrainNs);   // let the copy land
          fail = true;
          break;
        }
        if (dead[0] | dead[1]) {
          for (int r = lane >> 3; r < kAtStep; r += 4)
            if ((dead[r >> 5] >> (r & 31)) & 1)
#pragma unroll
              for (int p = 0; p < 2 * L::panels; ++p) zero_row(kst(s) + p * kAtPanel, r, lane);
          tc::fence_proxy_async();
        }
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&full[s]);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---------------- rows ----------------
    const int wg = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const long long vr = at.v0 + row;
    const bool mine = vr < at.v1;
    const bool keep = mine && (!KV || !a.mask || a.mask[vr]);
    const uint32_t u = (uint32_t)(keep ? vr : at.v0);
    const long long node = KV ? u : u / (uint32_t)a.G;
    const int head = KV ? kvh : kvh * a.G + (int)(u - (uint32_t)node * a.G);
    RowGrad<T, Cap, Bias, KV> grad(Cap ? a.scale / a.cap : a.scale * kLog2e);
    grad.cap2 = pair(a.cap * kLog2e);
    grad.px = grad.py = grad.pz = grad.sl = grad.nd = pair(0.0f);
    grad.nl = pair(-INFINITY);
    if (Bias) {
      const float* p = (KV ? a.pos_s : a.pos_r) + 3 * node;
      grad.px = pair(p[0]);
      grad.py = pair(p[1]);
      grad.pz = pair(p[2]);
      if (!KV) grad.sl = pair(-a.slope[head] * kLog2e);
    }
    if (!KV && mine) {
      const float2 st = a.stat[node * a.H + head];
      grad.nl = pair(-st.x);
      grad.nd = pair(-st.y);
    }
    constexpr int NS = RowGrad<T, Cap, Bias, KV>::kSums;
    float2 sum[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) sum[n] = pair(0.0f);
    bool easy = true;   // the last tile's scores were in the polynomial's range
    for (int i = wg; i < nt; i += 2) {
      const int s = i % NST, b = i % NB;
      if (!__all_sync(0xffffffffu, tc::bar_wait(&full[s], (i / NST) & 1, lim) && tc::bar_wait(&s_full[b], (i / NB) & 1, lim))) {
        fail = true;
        break;
      }
      tc::fence_after_sync();
      const uint32_t st = tmem + lanes + b * 128;
      const float* in = info(s);
      const bool flags = !KV && (a.mask || (t0 + i + 1) * (long long)kAtStep > shi - slo);
      uint32_t w[KV ? 2 : 1][32];
      float2 add[NS];
      float big = 0.0f;
      bool ok = false;
      if (!Cap || easy) {
        if (flags)
          grad.template tile<true, true>(st, in, w, add, big);
        else
          grad.template tile<true, false>(st, in, w, add, big);
        ok = !Cap || !__any_sync(0xffffffffu, !(big <= grad.poly.lim));
        easy = ok;
      } else {
        easy = (i & 14) == 0;   // try the polynomial again now and then
      }
      if (!ok) grad.template tile<false, true>(st, in, w, add, big);
#pragma unroll
      for (int n = 0; n < NS; ++n) sum[n] = add2(sum[n], add[n]);
      tc::tmem_st32(st + kAtStep, w[0]);
      if (KV) tc::tmem_st32(st, w[KV ? 1 : 0]);
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&p_full[b]);
    }
    // The accumulators are complete: drain has one phase.  (The last tile's done
    // barrier has one per tile of its buffer: the group that did not hold that
    // tile could pass on the phase before last.)
    if (nt > 0 && !fail && !tc::warp_wait(drain, 0, lim)) fail = true;
    tc::fence_after_sync();
    asm volatile("bar.sync 1, 256;" ::: "memory");
    float* mg = reinterpret_cast<float*>(smem);   // [NS][128]
    if (wg == 1)
#pragma unroll
      for (int n = 0; n < NS; ++n) mg[n * kAtRows + row] = sum[n].x + sum[n].y;
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (wg == 0 && mine && !fail) {
      float t[NS];
#pragma unroll
      for (int n = 0; n < NS; ++n) t[n] = sum[n].x + sum[n].y + mg[n * kAtRows + row];
      if constexpr (KV) {
        if (a.colpart) {   // the slopes went in as -slope log2(e); towards the receiver
          const float f = keep ? kLn2 : 0.0f;
          a.colpart[((long long)blockIdx.z * a.KV + kvh) * a.ns + vr] =
              keep ? make_float4(f * t[0], f * t[1], f * t[2], 0.0f) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      } else if (a.rowpart) {
        const float sl = Bias ? -a.slope[head] : 0.0f;
        const long long pr = (long long)blockIdx.z * a.nr * a.H + node * a.H + head;
        a.rowpart[pr] = make_float4(sl * t[0], sl * t[1], sl * t[2], -t[3]);
        a.rowmean[pr] = make_float4(sl * t[4], sl * t[5], sl * t[6], -t[7]);
        a.rowrest[pr] = t[8];
      }
    }
    // accumulators: KV: one per group; else the groups take the 32-column blocks in turn
    const long long out_row = KV ? vr * a.KV + kvh : node * a.H + head;
    const long long rows = KV ? (long long)a.ns * a.KV : (long long)a.nr * a.H;
    T* to = static_cast<T*>(KV ? (wg == 0 ? a.kb : a.vb) : a.qb);
    float* part = splits > 1 ? (KV ? (wg == 0 ? a.part_k : a.part_v) : a.part) : nullptr;
    if (to) {
      const uint32_t acc = tmem + lanes + L::acc + (KV && wg == 1 ? DP : 0);
      const float f = KV && wg == 1 ? 1.0f : a.scale;
#pragma unroll 1
      for (int c = KV ? 0 : 32 * wg; c < a.D; c += KV ? 32 : 64) {
        uint32_t r[32];
        if (nt > 0 && !fail) {
          tmem_ld32_async(acc + c, r);
          tmem_wait_ld(r);
        }
        const bool have = nt > 0 && keep;   // hidden senders' rows are 0 even where the receivers hold NaN
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          if (!mine || fail || c + e >= a.D) continue;
          float y[8];
#pragma unroll
          for (int n = 0; n < 8; ++n) y[n] = have ? __uint_as_float(r[e + n]) * f : 0.0f;
          if (part) {
            float* pp = part + ((long long)blockIdx.z * rows + out_row) * a.D + c + e;
            *reinterpret_cast<float4*>(pp) = make_float4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<float4*>(pp + 4) = make_float4(y[4], y[5], y[6], y[7]);
          } else {
            store_pack<T, 8>(to + out_row * a.D + c + e, y);
          }
        }
      }
    }
  }
  if (fail) atomicExch(&g_av_error, 1);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 8) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <class T, int DP, bool KV, bool Cap, bool Bias>
static int run(const AttnArgs& a, cudaStream_t s) {
  static DeviceFlags ready;
  using L = AtVjp<DP, KV>;
  if (set_smem_once(ready, attn_vjp_tc_kernel<T, DP, KV, Cap, Bias>, L::bytes) != FC_OK) return FC_ERR_CUDA;
  CUtensorMap m1, m2;
  constexpr bool half = __is_same(T, __half);
  const bool ok = KV ? at_tensor_map(&m1, half, a.q, a.D, a.H, a.ldq, a.nr, a.G) &&
                           at_tensor_map(&m2, half, a.g, a.D, a.H, a.ldg, a.nr, a.G)
                     : at_tensor_map(&m1, half, a.k, a.D, a.KV, a.ldk, a.ns) &&
                           at_tensor_map(&m2, half, a.v, a.D, a.KV, a.ldv, a.ns);
  if (!ok) return FC_ERR_CUDA;
  const long long slots = KV ? tile_slots(a.B, a.ns, 1, kAtRows) : tile_slots(a.B, a.nr, a.G, kAtRows);
  attn_vjp_tc_kernel<T, DP, KV, Cap, Bias>
      <<<dim3((unsigned)slots, a.KV, KV ? a.kv_splits : a.splits), kAtThreads, L::bytes, s>>>(a, m1, m2);
  return cudaGetLastError() == cudaSuccess ? FC_OK : FC_ERR_CUDA;
}
template <class T, int DP, bool KV>
static int run_kind(const AttnArgs& a, cudaStream_t s) {
  if (a.cap > 0.0f) return a.pos_r ? run<T, DP, KV, true, true>(a, s) : run<T, DP, KV, true, false>(a, s);
  return a.pos_r ? run<T, DP, KV, false, true>(a, s) : run<T, DP, KV, false, false>(a, s);
}
template <class T>
static int run_dim(bool kv, const AttnArgs& a, cudaStream_t s) {
  if (a.D <= 64) return kv ? run_kind<T, 64, true>(a, s) : run_kind<T, 64, false>(a, s);
  return kv ? run_kind<T, 128, true>(a, s) : run_kind<T, 128, false>(a, s);
}

// Takes the rest of delta out of a row's sums, parts added: with e = sum dt (the
// error of delta, as the weights sum to 1), the sums of P (dP - delta) x are
// those of dt x less e times those of P x.  They go to the first part; delta
// itself is put right for the sender side if stat is given.
__global__ void __launch_bounds__(256) attn_row_fix_kernel(AttnArgs a, float2* __restrict__ stat) {
  const long long rows = (long long)a.nr * a.H, row = (long long)blockIdx.x * 256 + threadIdx.x;
  if (row >= rows) return;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f), m = s;
  float e = 0.0f;
  for (int p = 0; p < a.splits; ++p) {
    const float4 x = a.rowpart[p * rows + row], y = a.rowmean[p * rows + row];
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    m.x += y.x; m.y += y.y; m.z += y.z; m.w += y.w;
    e += a.rowrest[p * rows + row];
  }
  a.rowpart[row] = make_float4(s.x - e * m.x, s.y - e * m.y, s.z - e * m.z, s.w - e * m.w);
  if (stat) stat[row].y += e;
}
int launch_attn_row_fix(const AttnArgs& a, float2* stat, cudaStream_t s) {
  const long long rows = (long long)a.nr * a.H;
  attn_row_fix_kernel<<<(unsigned)((rows + 255) / 256), 256, 0, s>>>(a, stat);
  return cudaGetLastError() == cudaSuccess ? FC_OK : FC_ERR_CUDA;
}

int launch_attn_vjp_tc(int dtype, bool kv, const AttnArgs& a, cudaStream_t s) {
  return dtype == FC_BF16 ? run_dim<__nv_bfloat16>(kv, a, s) : run_dim<__half>(kv, a, s);
}

int attn_vjp_tc_take_error(int* flag, cudaStream_t s) {
  if (cudaMemcpyFromSymbolAsync(flag, g_av_error, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return FC_ERR_CUDA;
  const int zero = 0;
  if (*flag && (cudaMemcpyToSymbolAsync(g_av_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
                cudaStreamSynchronize(s) != cudaSuccess))
    return FC_ERR_CUDA;
  return FC_OK;
}
int attn_vjp_tc_set_wait(unsigned long long ns) {
  return cudaMemcpyToSymbol(g_av_wait_ns, &ns, sizeof(ns)) == cudaSuccess ? FC_OK : FC_ERR_CUDA;
}

}  // namespace fc

// Node attention on the tensor cores (tcgen05), forward.
//
// Per stream tile of 64 senders: S = Q K^T into tensor memory; a group of 128
// threads, one receiver row each, reads its 64 scores, applies cap, distance
// bias and mask, keeps a running reference and sum, and writes the weights as
// 16-bit terms over the scores; O += P V stays in tensor memory and is rescaled
// only when the reference is raised.  The two groups take the tiles in turn,
// each with its own state and output columns; they are merged at the end.
//
// The score arithmetic takes the time: two special functions (exp, and the root
// of a distance, formed again for every head) and some 20 FP32 operations a pair
// of nodes and head against 4 D tensor operations.  16,384 nodes, 8 BF16 heads of
// 64, cap and bias: 2.04 ms, 1.05e12 pairs/s, 270 TFLOP/s (47 % of the special
// functions' rate, FP32 pipe 41 %, tensor core 15 %; the bytes would take 10 us);
// 4096 such nodes 157 us.  No pipe is full: eight warps of rows are all that
// their registers leave room for, two a scheduler, which cannot hide the latency
// of the tensor-memory reads and of each other's chains.
#include <cudaTypedefs.h>
#include <math.h>

#include "fc_attention_tc.cuh"

namespace fc {

__device__ int g_at_error = 0;
__device__ unsigned long long g_at_wait_ns = 500000000ull;

template <int DP>
struct AtFwd {
  static constexpr int panels = DP / 64;
  static constexpr int stages = DP == 128 ? 5 : 8;
  static constexpr size_t tile = (size_t)panels * kAtPanel, q = 2 * tile;
  static constexpr size_t info = 4 * kAtStep * sizeof(float);
  static constexpr size_t off_stage = q, off_info = off_stage + stages * 2 * tile;
  static constexpr size_t off_bar = off_info + stages * info;
  static constexpr size_t bytes = off_bar + 8 * (3 * stages + 12) + 16;
  static constexpr uint32_t col_o = 4 * kAtStep;   // four score tiles (their weights on top), two outputs
  // the merge of the groups goes over the tiles
  static_assert((DP + 2) * kAtRows * sizeof(float) <= off_info, "merge");
  static_assert(bytes <= 232448 && col_o + 2 * DP <= 512, "shared or tensor memory");
};

// The scores of one row against a tile, in base 2 and relative to a reference.
template <class T, bool Cap, bool Bias>
struct RowScore {
  float2 mul, cap2, px, py, pz, sl;   // slope negated
  TanhPoly poly;
  __device__ __forceinline__ RowScore(const AttnArgs& a, long long node, int head)
      : mul(pair(Cap ? a.scale / a.cap : a.scale * kLog2e)), cap2(pair(a.cap * kLog2e)), poly(a.cap * kLog2e, mul.x) {
    if (!Cap) poly.lim = INFINITY;
    px = py = pz = sl = pair(0.0f);
    if (Bias) {
      px = pair(a.pos_r[3 * node]);
      py = pair(a.pos_r[3 * node + 1]);
      pz = pair(a.pos_r[3 * node + 2]);
      sl = pair(-a.slope[head] * kLog2e);
    }
  }
  // y += slope distance + (0 or -infinity), 32 columns; in: positions and flags of the tile
  template <bool Flags>
  __device__ __forceinline__ void bias(float2* y, const float* in) const {
    if (Bias) {
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float4 fx = *reinterpret_cast<const float4*>(in + 2 * e),
                     fy = *reinterpret_cast<const float4*>(in + kAtStep + 2 * e),
                     fz = *reinterpret_cast<const float4*>(in + 2 * kAtStep + 2 * e);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 dx = add2(px, h ? hi2(fx) : lo2(fx)), dy = add2(py, h ? hi2(fy) : lo2(fy)),
                       dz = add2(pz, h ? hi2(fz) : lo2(fz));
          const float2 d2 = fma2(dx, dx, fma2(dy, dy, fma2(dz, dz, pair(kD2Seed))));
          y[e + h] = fma2(mul2(d2, make_float2(rsq(d2.x), rsq(d2.y))), sl, y[e + h]);
        }
      }
    }
    if (Flags)
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = add2(y[e], lds2(in + 3 * kAtStep + 2 * e));
  }
  // 64 columns with the cap's polynomial; big: the largest product
  template <bool Flags>
  __device__ __forceinline__ void easy(uint32_t st, const float* in, float neg_m, float2 (&x)[32], float& big) const {
    const float2 nm = pair(neg_m);
    uint32_t r[2][32];
    tmem_ld32_async(st, r[0]);
    float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      tmem_wait_ld(r[hf]);
      if (hf == 0) tmem_ld32_async(st + 32, r[1]);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (Cap) {
          const float2 v = pair_at(r[hf], e);
          b[e & 3] = max3_abs(b[e & 3], v.x, v.y);
          x[16 * hf + e] = fma2(v, poly(mul2(v, v)), nm);
        } else {
          x[16 * hf + e] = fma2(pair_at(r[hf], e), mul, nm);
        }
      }
      bias<Flags>(x + 16 * hf, in + 32 * hf);
    }
    if (Cap) big = max3(fmaxf(b[0], b[1]), b[2], b[3]);
  }
  // any scores; whether the polynomial would have served the warp
  __device__ __forceinline__ bool any(uint32_t st, const float* in, float neg_m, bool flags, float2 (&x)[32]) const {
    const float2 nm = pair(neg_m);
    float big = 0.0f;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t r[32];
      tmem_ld32_async(st + 32 * hf, r);
      tmem_wait_ld(r);
      float2 y[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = Cap ? mul2(pair_at(r, e), mul) : fma2(pair_at(r, e), mul, nm);
      if (Cap) {
#pragma unroll
        for (int e = 0; e < 16; ++e) big = max3_abs(big, y[e].x, y[e].y);
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = fma2(make_float2(cap_tanh<T>(y[e].x), cap_tanh<T>(y[e].y)), cap2, nm);
      }
      if (flags)
        bias<true>(y, in + 32 * hf);
      else
        bias<false>(y, in + 32 * hf);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[16 * hf + e] = y[e];
    }
    return !Cap || !__any_sync(0xffffffffu, !(big <= kAtTanhMax && poly.lim > 0.0f));
  }
};

// The weights of 64 scores as PT 16-bit terms, and their sum.
template <class T, int PT>
__device__ __forceinline__ float weigh(float2 (&x)[32], uint32_t (&w)[PT][32]) {
  float2 sum[2] = {pair(0.0f), pair(0.0f)};
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    x[e] = make_float2(ex2(x[e].x), ex2(x[e].y));
    sum[e & 1] = add2(sum[e & 1], x[e]);
    w[0][e] = pack2<T>(x[e].x, x[e].y);
    if (PT == 2) {   // what the rounding left
      const T* h = reinterpret_cast<const T*>(&w[0][e]);
      w[PT - 1][e] = pack2<T>(x[e].x - RowType<T>::to(h[0]), x[e].y - RowType<T>::to(h[1]));
    }
  }
  sum[0] = add2(sum[0], sum[1]);
  return sum[0].x + sum[0].y;
}

template <class T, int DP, int PT, bool Cap, bool Bias>
__global__ void __launch_bounds__(kAtThreads, 1) attn_fwd_tc_kernel(AttnArgs a, const __grid_constant__ CUtensorMap kmap,
                                                                const __grid_constant__ CUtensorMap vmap) {
  using L = AtFwd<DP>;
  constexpr int NST = L::stages;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t qs = tc::smem_addr(smem);
  auto kst = [&](int s) { return qs + (uint32_t)(L::off_stage + s * 2 * L::tile); };   // keys, then values
  auto info = [&](int s) { return reinterpret_cast<float*>(smem + L::off_info + s * L::info); };
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::off_bar);
  uint64_t *freeb = full + NST, *land = freeb + NST, *s_full = land + NST, *p_full = s_full + 4, *o_full = p_full + 4, *drain = o_full + 2, *q_full = drain + 1;
  uint32_t* slot = reinterpret_cast<uint32_t*>(q_full + 1);

  TileAt at;
  if (!find_tile(a.recv_ptr, a.B, a.nr, a.G, kAtRows, blockIdx.x, at)) return;
  const int kvh = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int slo, shi;
  other_side(a.send_ptr, a.B, a.ns, at.b, slo, shi);
  const int all = (shi > slo ? shi - slo + kAtStep - 1 : 0) / kAtStep;
  const int t0 = (int)((long long)all * blockIdx.z / a.splits);
  const int nt = (int)((long long)all * (blockIdx.z + 1) / a.splits) - t0;

  if (warp == 8) tc::tmem_alloc(slot, 512);
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      tc::bar_init(&full[s], 1);
      tc::bar_init(&freeb[s], 1);
      tc::bar_init(&land[s], 1);
    }
    for (int b = 0; b < 4; ++b) {   // one per score tile: a group may be two tiles ahead of the products
      tc::bar_init(&s_full[b], 1);
      tc::bar_init(&p_full[b], 4);
    }
    for (int b = 0; b < 2; ++b) tc::bar_init(&o_full[b], 1);
    tc::bar_init(drain, 1);
    tc::bar_init(q_full, 3);
    tc::fence_bar_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *slot;
  const uint64_t lim = g_at_wait_ns;
  bool fail = false;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 8) {
      // ---------------- matrix products ----------------
      if (elect_one()) {
        const int ks = (a.D + 15) / 16;
        const uint32_t idesc_s = at_idesc<T>(kAtStep, false), idesc_o = at_idesc<T>(ks * 16, true);
        const uint64_t qd = desc_k<kAtRows>(qs);
        auto scores = [&](int i) {
          if (!tc::bar_wait(&full[i % NST], (i / NST) & 1, lim)) return false;
          tc::fence_after_sync();
          const uint64_t kd = desc_k<kAtStep>(kst(i % NST));
          const uint32_t sd = tmem + (i & 3) * kAtStep;
#pragma unroll
          for (int k = 0; k < DP / 16; ++k)
            if (k < ks) mma_ss16(sd, qd + step_k<kAtRows>(k), kd + step_k<kAtStep>(k), idesc_s, k != 0);
          tc::commit(&s_full[i & 3]);
          return true;
        };
        // Scores run three tiles ahead.  Their columns are those of the weights of
        // the tile before last, whose product is awaited first (by then it is done).
        fail = !tc::bar_wait(q_full, 0, lim);
        for (int i = 0; i < 3 && i < nt && !fail; ++i) fail = !scores(i);
        for (int i = 0; i < nt && !fail; ++i) {
          const int b = i & 1;
          if (!tc::bar_wait(&p_full[i & 3], (i >> 2) & 1, lim)) {
            fail = true;
            break;
          }
          tc::fence_after_sync();
          const uint64_t vd = desc_mn<kAtStep>(kst(i % NST) + (uint32_t)L::tile);
          const uint32_t od = tmem + L::col_o + b * DP, pd = tmem + (i & 3) * kAtStep;
#pragma unroll
          for (int p = PT - 1; p >= 0; --p)
#pragma unroll
            for (int k = 0; k < kAtStep / 16; ++k)
              mma_ts16(od, pd + 32 * p + 8 * k, vd + step_mn(k), idesc_o, i > 1 || p != PT - 1 || k != 0);
          tc::commit(&o_full[b]);
          tc::commit(&freeb[i % NST]);
          if (i + 3 < nt)
            fail = (i > 0 && !tc::bar_wait(&o_full[b ^ 1], ((i - 1) >> 1) & 1, lim)) || !scores(i + 3);
        }
        // every product issued above has finished before tensor and shared memory are released
        tc::commit(drain);
        if (!tc::bar_wait(drain, 0, kAtDrainNs)) fail = true;
      }
      __syncwarp();
    } else {
      // ---------------- copies ----------------
      // Warp cw brings in tiles cw, cw + 3, ..; all three copy the receivers' rows first.
      const int cw = warp - 9;
      const T* q = static_cast<const T*>(a.q);
      // (none without a tile to meet: the merge at the end goes over their place)
      for (int r0 = cw * 4; r0 < kAtRows && nt > 0; r0 += 12) {
        const long long vr = at.v0 + r0 + (lane >> 3);
        const bool ok = vr < at.v1;
        const uint32_t u = (uint32_t)(ok ? vr : at.v0), node = u / (uint32_t)a.G;
        const T* src = q + node * a.ldq + (kvh * a.G + (int)(u - node * a.G)) * (long long)a.D;
#pragma unroll
        for (int p = 0; p < L::panels; ++p) {
          const int c = p * 64 + (lane & 7) * 8;
          const bool live = ok && c < a.D;
          copy_rows4(qs + p * kAtRows * 128, r0, lane, src + (live ? c : 0), live);
        }
      }
      cp_wait_all();
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(q_full);
      for (int i = cw; i < nt; i += kAtCopiers) {
        const int s = i % NST, round = i / NST;
        if (round > 0 && !tc::warp_wait(&freeb[s], (round - 1) & 1, lim)) {
          fail = true;
          break;
        }
        const long long j0 = slo + (long long)(t0 + i) * kAtStep;
        if (elect_one()) {
          tc::bar_arrive_expect_tx(&land[s], 2 * (uint32_t)L::tile);
#pragma unroll
          for (int p = 0; p < L::panels; ++p) {
            load_panel(kst(s) + p * kAtPanel, &kmap, p * 64, kvh, (int)j0, &land[s]);
            load_panel(kst(s) + (uint32_t)L::tile + p * kAtPanel, &vmap, p * 64, kvh, (int)j0, &land[s]);
          }
        }
        __syncwarp();
        // negated positions, and what is added to the score: 0, or -infinity for a row not there
        unsigned dead[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const long long j = j0 + 32 * n + lane;
          const bool ok = j < shi && (!a.mask || a.mask[j]), there = Bias && ok;
          float* f = info(s) + 32 * n + lane;
          f[0] = there ? -a.pos_s[3 * j] : 0.0f;
          f[kAtStep] = there ? -a.pos_s[3 * j + 1] : 0.0f;
          f[2 * kAtStep] = there ? -a.pos_s[3 * j + 2] : 0.0f;
          f[3 * kAtStep] = ok ? 0.0f : -INFINITY;
          dead[n] = __ballot_sync(0xffffffffu, !ok);
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
    // ---------------- rows ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int wg = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const long long vr = at.v0 + row;
    const bool mine = vr < at.v1;
    const uint32_t ot = tmem + lanes + L::col_o + wg * DP;
    const uint32_t u = (uint32_t)(mine ? vr : at.v0);
    const int node = (int)(u / (uint32_t)a.G), head = kvh * a.G + (int)(u - (uint32_t)node * a.G);
    RowScore<T, Cap, Bias> score(a, node, head);
    // m: what the scores are taken relative to (base 2).  It is set by the
    // row's first score and raised only when a tile exceeds it by 2^8, so that
    // most tiles fold its subtraction into the score and need no rescaling.
    float m = 0.0f, l = 0.0f;
    bool set = false;
    bool easy = false;   // the last tile's scores were in the polynomial's range
    int j = 0;   // tiles of this group
    for (int i = wg; i < nt; i += 2, ++j) {
      const int s = i % NST;
      if (!__all_sync(0xffffffffu, tc::bar_wait(&full[s], (i / NST) & 1, lim) && tc::bar_wait(&s_full[i & 3], (i >> 2) & 1, lim))) {
        fail = true;
        break;
      }
      tc::fence_after_sync();
      const uint32_t st = tmem + lanes + (i & 3) * kAtStep;
      const float* in = info(s);
      const bool ragged = a.mask || (t0 + i + 1) * (long long)kAtStep > shi - slo;
      float2 x[32];
      bool done = false;
      if (easy) {
        // Straight through on the present reference, without a branch from the
        // scores to the packed weights, so that one column's exp and square
        // root overlap the next one's arithmetic; kept if nothing was out of
        // range, else done again below.
        float big = 0.0f;
        if (ragged)
          score.template easy<true>(st, in, -m, x, big);
        else
          score.template easy<false>(st, in, -m, x, big);
        const float mx = max_pairs(x);
        uint32_t w[PT][32];
        const float sum = weigh<T, PT>(x, w);
        if (!__any_sync(0xffffffffu, !(big <= score.poly.lim) || mx > (set ? 8.0f : -INFINITY))) {
#pragma unroll
          for (int p = 0; p < PT; ++p) tc::tmem_st32(st + 32 * p, w[p]);
          l += sum;
          done = true;
        }
      }
      if (!done) {
        easy = score.any(st, in, -m, ragged, x);
        const float mx = max_pairs(x);
        const bool raise = mx > (set ? 8.0f : -INFINITY);
        if (__any_sync(0xffffffffu, raise)) {
          const float up = raise ? mx : 0.0f;
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = add2(x[e], pair(-up));
          m += up;
          if (j > 0) {   // rescale the sum and the output so far (0 before the row's first score)
            const float al = set ? ex2(-up) : 1.0f;
            l *= al;
            if (!tc::warp_wait(&o_full[wg], (j - 1) & 1, lim)) {
              fail = true;
              break;
            }
            tc::fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < a.D; c += 32) {
              uint32_t o[32];
              tmem_ld32_async(ot + c, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
              tc::tmem_st32(ot + c, o);
            }
          }
          set |= raise;
        }
        uint32_t w[PT][32];
        l += weigh<T, PT>(x, w);
#pragma unroll
        for (int p = 0; p < PT; ++p) tc::tmem_st32(st + 32 * p, w[p]);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&p_full[i & 3]);
    }
    // Every product is complete: drain has one phase.  (o_full[wg] has one per tile,
    // and the product of the tile before last may still be open here, whose
    // predecessor has the parity of the last.)
    if (j > 0 && !fail && !tc::warp_wait(drain, 0, lim)) fail = true;
    tc::fence_after_sync();
    if (!set) m = -INFINITY;
    const bool have = j > 0 && !fail;   // else this group's output columns hold nothing

    // merge the groups: all products and copies are done, shared memory is free
    asm volatile("bar.sync 1, 256;" ::: "memory");
    float* mg = reinterpret_cast<float*>(smem);
    if (wg == 1) {
      mg[row] = m;
      mg[kAtRows + row] = l;
      if (have)
#pragma unroll 1
        for (int c = 0; c < a.D; c += 32) {
          uint32_t o[32];
          tmem_ld32_async(ot + c, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) mg[(2 + c + e) * kAtRows + row] = __uint_as_float(o[e]);
        }
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (wg == 0) {
      const float m1 = mg[row], mx = fmaxf(m, m1), base = mx == -INFINITY ? 0.0f : mx;
      const float w0 = ex2(m - base), w1 = ex2(m1 - base);
      const float sum = l * w0 + mg[kAtRows + row] * w1;
      const bool other = nt > 1, store = mine && !fail, part = a.splits > 1;
      const long long rw = (long long)node * a.H + head;
      const long long pr = (long long)blockIdx.z * a.nr * a.H + rw;
      const float inv = part ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
      if (store) {
        if (part)
          a.part_ml[pr] = make_float2(mx, sum);
        else if (a.lse)
          a.lse[rw] = (mx + log2f(sum)) * kLn2;
      }
      float* pp = part ? a.part + pr * a.D : a.o32 ? a.o32 + rw * a.D : nullptr;
      T* o = part ? nullptr : static_cast<T*>(a.out) + node * a.ldo + (long long)head * a.D;
#pragma unroll 1
      for (int c = 0; c < a.D; c += 32) {
        float v[32];
        {
          uint32_t r[32];
          tmem_ld32_async(ot + c, r);
          tmem_wait_ld(r);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = have ? __uint_as_float(r[e]) * w0 : 0.0f;
        }
        if (other)
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] += mg[(2 + c + e) * kAtRows + row] * w1;
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          if (!store || c + e >= a.D) continue;
          float y[8];
#pragma unroll
          for (int n = 0; n < 8; ++n) y[n] = v[e + n] * inv;
          if (pp) {
            *reinterpret_cast<float4*>(pp + c + e) = make_float4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<float4*>(pp + c + e + 4) = make_float4(y[4], y[5], y[6], y[7]);
          }
          if (o) store_pack<T, 8>(o + c + e, y);
        }
      }
    }
  }
  if (fail) atomicExch(&g_at_error, 1);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 8) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (CUDA 12.0
// ABI), looked up once.
static PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !f)
      return nullptr;
    fn.store(f, std::memory_order_release);
  }
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}
bool at_tensor_map(CUtensorMap* m, bool half, const void* base, int D, int heads, long long ld, int rows, int group) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)(kAtStep / group)}, es[3] = {1, 1, 1};
  return enc(m, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
             dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, int DP, int PT, bool Cap, bool Bias>
static int run_fwd_tc(const AttnArgs& a, cudaStream_t s) {
  static DeviceFlags ready;
  if (set_smem_once(ready, attn_fwd_tc_kernel<T, DP, PT, Cap, Bias>, AtFwd<DP>::bytes) != FC_OK) return FC_ERR_CUDA;
  CUtensorMap km, vm;
  constexpr bool half = __is_same(T, __half);
  if (!at_tensor_map(&km, half, a.k, a.D, a.KV, a.ldk, a.ns) || !at_tensor_map(&vm, half, a.v, a.D, a.KV, a.ldv, a.ns))
    return FC_ERR_CUDA;
  attn_fwd_tc_kernel<T, DP, PT, Cap, Bias>
      <<<dim3((unsigned)tile_slots(a.B, a.nr, a.G, kAtRows), a.KV, a.splits), kAtThreads, AtFwd<DP>::bytes, s>>>(a, km, vm);
  return cudaGetLastError() == cudaSuccess ? FC_OK : FC_ERR_CUDA;
}
template <class T, int DP, int PT>
static int run_fwd_terms(const AttnArgs& a, cudaStream_t s) {
  if (a.cap > 0.0f) return a.pos_r ? run_fwd_tc<T, DP, PT, true, true>(a, s) : run_fwd_tc<T, DP, PT, true, false>(a, s);
  return a.pos_r ? run_fwd_tc<T, DP, PT, false, true>(a, s) : run_fwd_tc<T, DP, PT, false, false>(a, s);
}
template <class T, int PT>
static int run_fwd_dim(const AttnArgs& a, cudaStream_t s) {
  return a.D <= 64 ? run_fwd_terms<T, 64, PT>(a, s) : run_fwd_terms<T, 128, PT>(a, s);
}

int launch_attn_fwd_tc(int dtype, const AttnArgs& a, cudaStream_t s) {
  if (dtype == FC_BF16)
    return a.o32 ? run_fwd_dim<__nv_bfloat16, 2>(a, s) : run_fwd_dim<__nv_bfloat16, 1>(a, s);
  return a.o32 ? run_fwd_dim<__half, 2>(a, s) : run_fwd_dim<__half, 1>(a, s);
}

int attn_vjp_tc_take_error(int* flag, cudaStream_t s);
int attn_vjp_tc_set_wait(unsigned long long ns);

int attn_tc_take_error(int* flag, cudaStream_t s) {
  int vjp = 0;
  if (cudaMemcpyFromSymbolAsync(flag, g_at_error, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess || attn_vjp_tc_take_error(&vjp, s) != FC_OK)
    return FC_ERR_CUDA;
  const int zero = 0;
  if (*flag && (cudaMemcpyToSymbolAsync(g_at_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
                cudaStreamSynchronize(s) != cudaSuccess))
    return FC_ERR_CUDA;
  *flag |= vjp;
  return FC_OK;
}
int attn_tc_set_wait(unsigned long long ns) {
  if (cudaMemcpyToSymbol(g_at_wait_ns, &ns, sizeof(ns)) != cudaSuccess) return FC_ERR_CUDA;
  return attn_vjp_tc_set_wait(ns);
}

}  // namespace fc

// Species embedding and its gradient.
//
// Forward: x[n, rank 0, :] = scale table[species[n]], other ranks zero.  Bound
// by the bytes written ((lmax+1)^2 C values per node); the table stays in L2.
// One thread moves 16-byte vectors, a block a run of whole rows (65,537 nodes of
// rank 2 and 128 FP32 channels: 302 MB in 45 us, 6.7 TB/s).
//
// Gradient: table_bar[s] = scale sum of g over the nodes of species s.  The
// nodes are sorted by species (stable radix sort, one pass of 8 bits for tables
// of up to 255 rows), the sorted list is cut into spans of 32 to 128 nodes, one
// warp sums each span and writes the species that lie inside it; a species that
// crosses spans leaves one partial row per span, which a last kernel adds in
// span order.  That kernel also clears the rows of species without nodes, so
// that every row is written once.  A species with nearly all nodes costs no
// more than an even spread, and no sum depends on the order of atomics.  Bound
// by its launches and the latency of their loads: 100,003 nodes of few species
// (128 FP32 channels, 51 MB) in 38 us, 50,001 nodes of 32,000 species (512 BF16
// channels, two sort passes) in 66 us.
#include <math.h>

#include "fc_nodes.cuh"

namespace fc {

constexpr int kDigits = 256;

// ------------------------------------------------------------------ forward

template <class T>
__global__ void __launch_bounds__(256) species_embed_kernel(int n, int V, int vec0, int rowvec, int rows, float scale,
                                                            const int32_t* __restrict__ species,
                                                            const T* __restrict__ table, T* __restrict__ x) {
  constexpr int W = RowType<T>::kVec;
  const long long r0 = (long long)blockIdx.x * rows;
  const int here = (int)(n - r0 < rows ? n - r0 : rows);
  const int total = here * rowvec;
  T* out = x + r0 * rowvec * W;
  for (int i = threadIdx.x; i < total; i += 256) {
    const int r = i / rowvec, c = i - r * rowvec;
    float v[W];
#pragma unroll
    for (int k = 0; k < W; ++k) v[k] = 0.0f;
    if (c < vec0) {
      const int s = species[r0 + r];
      if (s >= 0 && s < V) {
        load_pack<T, W>(table + ((long long)s * vec0 + c) * W, v);
#pragma unroll
        for (int k = 0; k < W; ++k) v[k] *= scale;
      }
    }
    store_pack<T, W>(out + (long long)i * W, v);
  }
}

// --------------------------------------------------------------------- sort

// Chunks of the sort: `rows` nodes each (a multiple of 256), at most 512.
// Spans of the sums: as long as eight warps per SM allow, since every span of a
// frequent species leaves a partial row (100,003 nodes of few species, 128
// channels: joining them took as long as the sums at 32).
struct SortGeom {
  int n, V, rows, chunks, passes, span;
};
static SortGeom sort_geom(int n, int V, int C) {
  SortGeom g{n, V, 1024, 0, 1, 32};
  while (g.span < 128 && (long long)n / (2 * g.span) * ((C + 127) / 128) >= 8 * device_sm_count()) g.span *= 2;
  const long long per = ((long long)n + 511) / 512;
  if (per > g.rows) g.rows = (int)((per + 255) / 256 * 256);
  g.chunks = (int)(((long long)n + g.rows - 1) / g.rows);
  while (g.passes < 4 && ((long long)V >> (8 * g.passes)) != 0) ++g.passes;   // keys 0 .. V
  return g;
}

// Sort key of node i: its species, or V if it has none.
__device__ __forceinline__ int sort_key(const int32_t* __restrict__ keys, bool raw, long long i, int V) {
  const int k = keys[i];
  return raw && (k < 0 || k >= V) ? V : k;
}

// Digit counts of every chunk.
__global__ void __launch_bounds__(256) sort_count_kernel(SortGeom g, int shift, bool raw,
                                                         const int32_t* __restrict__ keys, int* __restrict__ counts) {
  __shared__ int hist[kDigits];
  hist[threadIdx.x] = 0;
  __syncthreads();
  const long long b = (long long)blockIdx.x * g.rows;
  const long long e = b + g.rows < g.n ? b + g.rows : g.n;
  for (long long i = b + threadIdx.x; i < e; i += 256)
    atomicAdd(&hist[(sort_key(keys, raw, i, g.V) >> shift) & 255], 1);
  __syncthreads();
  counts[blockIdx.x * kDigits + threadIdx.x] = hist[threadIdx.x];
}

// Stable scatter of one 8-bit digit: a warp owns a contiguous eighth of the
// chunk and ranks 32 nodes at a time among equal digits.
__global__ void __launch_bounds__(256) sort_scatter_kernel(SortGeom g, int shift, bool raw,
                                                           const int32_t* __restrict__ keys,
                                                           const int32_t* __restrict__ from,
                                                           const int* __restrict__ counts, int32_t* __restrict__ okeys,
                                                           int32_t* __restrict__ oidx) {
  __shared__ int off[8][kDigits];
  __shared__ int scan[kDigits];
  const int t = threadIdx.x, w = t >> 5, lane = t & 31;
  int total = 0, before = 0;
#pragma unroll 8
  for (int c = 0; c < g.chunks; ++c) {
    const int v = counts[c * kDigits + t];
    total += v;
    if (c < (int)blockIdx.x) before += v;
  }
  scan[t] = total;
#pragma unroll
  for (int k = 0; k < 8; ++k) off[k][t] = 0;
  __syncthreads();
  for (int o = 1; o < kDigits; o <<= 1) {
    const int v = t >= o ? scan[t - o] : 0;
    __syncthreads();
    scan[t] += v;
    __syncthreads();
  }
  const int base = scan[t] - total + before;
  const int sub = g.rows / 8;
  const long long b = (long long)blockIdx.x * g.rows + (long long)w * sub;
  const long long lim = b + sub < g.n ? b + sub : g.n;
  for (long long i = b + lane; i < lim; i += 32) atomicAdd(&off[w][(sort_key(keys, raw, i, g.V) >> shift) & 255], 1);
  __syncthreads();
  int run = base;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int v = off[k][t];
    off[k][t] = run;
    run += v;
  }
  __syncthreads();
  for (long long i0 = b; i0 < lim; i0 += 32) {
    const long long i = i0 + lane;
    const bool live = i < lim;
    const int key = live ? sort_key(keys, raw, i, g.V) : 0;
    const int digit = live ? (key >> shift) & 255 : 256 + lane;
    const unsigned peers = __match_any_sync(0xffffffffu, digit);
    const int rank = __popc(peers & ((1u << lane) - 1u));
    int at = 0;
    if (live) at = off[w][digit] + rank;
    __syncwarp();
    if (live && rank == 0) off[w][digit] += __popc(peers);
    __syncwarp();
    if (live) {
      okeys[at] = key;
      oidx[at] = from ? from[i] : (int32_t)i;
    }
  }
}

// --------------------------------------------------------------------- sums

// One warp: the sums of one span over one tile of 128 columns, four per lane (so
// that the FP32 rows it writes are whole lines for 16-bit gradients too).
// Runs: species of many nodes, whose groups of 16 rows are mostly of one (with
// 32,000 species among 50,001 nodes looking for such groups took 6 of 72 us).
template <class T, bool Runs>
__global__ void __launch_bounds__(256) span_sum_kernel(int n, int V, int C, int span_rows, long long ldg, float scale,
                                                       const int32_t* __restrict__ keys,
                                                       const int32_t* __restrict__ idx, const T* __restrict__ g,
                                                       float* __restrict__ bar, float* __restrict__ part) {
  const int lane = threadIdx.x & 31;
  const long long span = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const long long start = span * span_rows;
  if (start >= n) return;
  const int cnt = (int)(n - start < span_rows ? n - start : span_rows);
  const int col = blockIdx.y * 128 + lane * 4;
  const bool in = col < C;
  const int prev = start > 0 ? keys[start - 1] : -1;
  const int next = start + cnt < n ? keys[start + cnt] : -1;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  int cur = -1;
  bool begins = false;
  auto flush = [&](bool ends) {
    if (cur < 0 || cur >= V || !in) return;
    float* to = begins && ends ? bar + (long long)cur * C : part + (2 * span + (begins ? 1 : 0)) * C;
    const float f = begins && ends ? scale : 1.0f;
    *reinterpret_cast<float4*>(to + col) = make_float4(acc[0] * f, acc[1] * f, acc[2] * f, acc[3] * f);
  };
  auto meet = [&](int k, int row) {   // the span's row of species k
    if (k == cur) return;
    flush(true);
    cur = k;
    begins = row > 0 || prev != k;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = 0.0f;
  };
  // Every load is made (rows past the span repeat its first, lanes past the
  // columns read column 0), so that they go out together.
  constexpr int U = 16;   // rows in flight per lane
  const T* gc = g + (in ? col : 0);
  int key = 0, row = 0;
  auto next_rows = [&](int b0) {
    const long long at = start + (b0 + lane < cnt ? b0 + lane : 0);
    key = keys[at];
    row = idx[at];
  };
  next_rows(0);
  for (int b0 = 0; b0 < cnt; b0 += 32) {
    const int k32 = key, r32 = row;
    next_rows(b0 + 32);
#pragma unroll 1
    for (int r0 = 0; r0 < 32 && b0 + r0 < cnt; r0 += U) {
      float v[U][4];
#pragma unroll
      for (int u = 0; u < U; ++u)
        load_pack<T, 4>(gc + (long long)__shfl_sync(0xffffffffu, r32, r0 + u) * ldg, v[u]);
      if constexpr (Runs) {
        // All of one species: in halves, so that a long sum is rounded in few
        // places (100,003 nodes of few species, added in turn: 1.8e-7 off).
        const int k = __shfl_sync(0xffffffffu, k32, r0);
        const unsigned same = __ballot_sync(0xffffffffu, k32 == k && b0 + lane < cnt);
        if (((same >> r0) & 0xffffu) == 0xffffu) {
          meet(k, b0 + r0);
#pragma unroll
          for (int o = U / 2; o > 0; o >>= 1)
#pragma unroll
            for (int u = 0; u < o; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i) v[u][i] += v[u + o][i];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] += v[0][i];
          continue;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = __shfl_sync(0xffffffffu, k32, r0 + u);
        if (b0 + r0 + u < cnt) {
          meet(k, b0 + r0 + u);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] += v[u][i];
        }
      }
    }
  }
  flush(next != cur);
}

// Joins the species that cross spans.  A warp looks at one span: if a species
// begins in it and runs on, the warp adds its partial rows (at most 64 spans;
// longer ones are added by the whole block).  Blocks from join_blocks on clear
// the species without nodes: a lane searches one species in the sorted list.
__global__ void __launch_bounds__(1024) span_join_kernel(int n, int V, int C, int span_rows, int join_blocks, float scale,
                                                         const int32_t* __restrict__ keys,
                                                         const float* __restrict__ part, float* __restrict__ bar) {
  __shared__ int lng[32];
  __shared__ float sum[32][128];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long spans = ((long long)n + span_rows - 1) / span_rows;
  const long long s = (long long)blockIdx.x * 32 + w;
  const int col = blockIdx.y * 128 + lane * 4;
  const bool in = col < C;
  if ((int)blockIdx.x >= join_blocks) {
    const long long v = ((long long)(blockIdx.x - join_blocks) * 32 + w) * 32 + lane;
    bool none = false;
    if (v < V) {
      int lo = 0, hi = n;   // first node of species >= v
      while (lo < hi) {
        const int mid = (int)(((unsigned)lo + (unsigned)hi) >> 1);
        if (keys[mid] < v)
          lo = mid + 1;
        else
          hi = mid;
      }
      none = lo == n || keys[lo] != v;
    }
    unsigned todo = __ballot_sync(0xffffffffu, none);
    for (; todo; todo &= todo - 1) {
      const long long row = v - lane + (__ffs(todo) - 1);
      if (in) *reinterpret_cast<float4*>(bar + row * C + col) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    return;
  }
  auto head = [&](long long sp) { return keys[sp * span_rows]; };
  auto add = [&](float4& a, long long slot) {
    const float4 v = *reinterpret_cast<const float4*>(part + slot * C + col);
    a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
  };
  if (lane == 0) lng[w] = 0;
  int k = -1;
  if (s + 1 < spans) {
    k = keys[(s + 1) * span_rows - 1];
    const bool runs_on = head(s + 1) == k;
    const bool begins = head(s) != k || s == 0 || keys[s * span_rows - 1] != k;
    if (!runs_on || !begins || k >= V) k = -1;
  }
  if (k >= 0) {
    int m = 0;   // spans after s that start with k
    bool open = true;
    for (int round = 0; round < 2 && open; ++round) {
      const long long sp = s + 1 + m + lane;
      const unsigned same = __ballot_sync(0xffffffffu, sp < spans && head(sp < spans ? sp : 0) == k);
      const int run = same == 0xffffffffu ? 32 : __ffs(~same) - 1;
      m += run;
      open = run == 32;
    }
    if (open) {
      if (lane == 0) lng[w] = 1;
    } else if (in) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b[4] = {a, a, a, a};
      add(a, 2 * s + 1);
      for (int i = 1; i <= m; i += 4)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e <= m) add(b[e], 2 * (s + i + e));
      a.x += (b[0].x + b[1].x) + (b[2].x + b[3].x);
      a.y += (b[0].y + b[1].y) + (b[2].y + b[3].y);
      a.z += (b[0].z + b[1].z) + (b[2].z + b[3].z);
      a.w += (b[0].w + b[1].w) + (b[2].w + b[3].w);
      *reinterpret_cast<float4*>(bar + (long long)k * C + col) =
          make_float4(a.x * scale, a.y * scale, a.z * scale, a.w * scale);
    }
  }
  __syncthreads();
  for (int j = 0; j < 32; ++j) {
    if (!lng[j]) continue;
    const long long sj = (long long)blockIdx.x * 32 + j;
    const int kj = keys[(sj + 1) * span_rows - 1];
    long long m = 0;
    int run = 1024;
    while (run == 1024) {
      const long long sp = sj + 1 + m + threadIdx.x;
      run = __syncthreads_count(sp < spans && head(sp < spans ? sp : 0) == kj);
      m += run;
    }
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
      if (w == 0) add(a, 2 * sj + 1);
#pragma unroll 8
      for (long long i = 1 + w; i <= m; i += 32) add(a, 2 * (sj + i));
    }
    *reinterpret_cast<float4*>(&sum[w][lane * 4]) = a;
    __syncthreads();
    if (threadIdx.x < 128 && blockIdx.y * 128 + threadIdx.x < C) {
      float v[16];
#pragma unroll
      for (int q = 0; q < 16; ++q) v[q] = sum[q][threadIdx.x] + sum[q + 16][threadIdx.x];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
#pragma unroll
        for (int q = 0; q < o; ++q) v[q] += v[q + o];
      bar[(long long)kj * C + blockIdx.y * 128 + threadIdx.x] = v[0] * scale;
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------------- launches

struct EmbedLayout {
  SortGeom g;
  size_t keys[2], idx[2], counts, part, bytes;
};
static EmbedLayout embed_layout(int n, int V, int C) {
  EmbedLayout l;
  l.g = sort_geom(n, V, C);
  size_t at = 0;
  const size_t list = round16(4 * (size_t)n);
  for (int i = 0; i < 2; ++i) {
    l.keys[i] = at;
    at += i == 0 || l.g.passes > 1 ? list : 0;
    l.idx[i] = at;
    at += i == 0 || l.g.passes > 1 ? list : 0;
  }
  l.counts = at;
  at += 4 * (size_t)kDigits * l.g.chunks;
  l.part = at;
  at += 2 * (((size_t)n + l.g.span - 1) / l.g.span) * C * 4;
  l.bytes = at;
  return l;
}

static int check_embed(int dtype, int n, int V, int lmax, int C, float scale) {
  if (!row_dtype(dtype) || n < 0 || V < 1 || V == INT32_MAX || lmax < 0 || lmax > 8 || C <= 0 || !isfinite(scale))
    return FC_ERR_ARG;
  if (C > (1 << 20)) return FC_ERR_ARG;
  if (C % (dtype == FC_F32 ? 4 : 8)) return FC_ERR_ALIGN;
  return FC_OK;
}

template <class T>
static int embed_fwd(int n, int V, int lmax, int C, float scale, const int32_t* species, const void* table, void* x,
                     cudaStream_t s) {
  constexpr int W = RowType<T>::kVec;
  const int vec0 = C / W, rowvec = vec0 * (lmax + 1) * (lmax + 1);
  // about 2048 vectors (32 KB) a block, fewer while that leaves SMs idle
  int rows = 2048 / rowvec;
  const int even = n / (4 * device_sm_count());
  if (rows > even) rows = even;
  if (rows < 1) rows = 1;
  const int blocks = (int)(((long long)n + rows - 1) / rows);
  species_embed_kernel<T><<<blocks, 256, 0, s>>>(n, V, vec0, rowvec, rows, scale, species,
                                                 static_cast<const T*>(table), static_cast<T*>(x));
  return cudaGetLastError() == cudaSuccess ? FC_OK : FC_ERR_CUDA;
}

template <class T>
static void span_sum(const EmbedLayout& l, int C, long long ldg, float scale, const int32_t* keys, const int32_t* idx,
                     const void* g, float* bar, float* part, cudaStream_t s) {
  const long long spans = ((long long)l.g.n + l.g.span - 1) / l.g.span;
  const auto kernel = l.g.n / 16 >= l.g.V ? span_sum_kernel<T, true> : span_sum_kernel<T, false>;
  kernel<<<dim3((unsigned)((spans + 7) / 8), (C + 127) / 128), 256, 0, s>>>(
      l.g.n, l.g.V, C, l.g.span, ldg, scale, keys, idx, static_cast<const T*>(g), bar, part);
}

}  // namespace fc

using namespace fc;

extern "C" {

int fc_species_embed(int dtype, int n_nodes, int n_species, int lmax, int channels, float scale,
                     const int32_t* species, const void* table, void* x, fc_stream_t stream) {
  const int st = check_embed(dtype, n_nodes, n_species, lmax, channels, scale);
  if (st != FC_OK) return st;
  if (n_nodes == 0) return FC_OK;
  if (!species || !table || !x) return FC_ERR_ARG;
  if (!aligned4(species) || !aligned16(table) || !aligned16(x)) return FC_ERR_ALIGN;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == FC_F32) return embed_fwd<float>(n_nodes, n_species, lmax, channels, scale, species, table, x, s);
  if (dtype == FC_BF16)
    return embed_fwd<__nv_bfloat16>(n_nodes, n_species, lmax, channels, scale, species, table, x, s);
  return embed_fwd<__half>(n_nodes, n_species, lmax, channels, scale, species, table, x, s);
}

size_t fc_species_embed_vjp_workspace_size(int n_nodes, int n_species, int channels) {
  if (n_nodes <= 0 || n_species < 1 || n_species == INT32_MAX || channels <= 0 || channels > (1 << 20)) return 0;
  return embed_layout(n_nodes, n_species, channels).bytes;
}

int fc_species_embed_vjp(int dtype, int n_nodes, int n_species, int lmax, int channels, float scale,
                         const int32_t* species, const void* g, float* table_bar, void* workspace, size_t ws_bytes,
                         fc_stream_t stream) {
  const int st = check_embed(dtype, n_nodes, n_species, lmax, channels, scale);
  if (st != FC_OK) return st;
  if (!table_bar || (n_nodes > 0 && (!species || !g))) return FC_ERR_ARG;
  if (!aligned16(table_bar) || (n_nodes > 0 && (!aligned4(species) || !aligned16(g)))) return FC_ERR_ALIGN;
  cudaStream_t s = (cudaStream_t)stream;
  const size_t bar_bytes = sizeof(float) * (size_t)n_species * channels;
  if (n_nodes == 0)
    return cudaMemsetAsync(table_bar, 0, bar_bytes, s) == cudaSuccess ? FC_OK : FC_ERR_CUDA;
  const EmbedLayout l = embed_layout(n_nodes, n_species, channels);
  if (!workspace || ws_bytes < l.bytes) return FC_ERR_WORKSPACE;
  if (!aligned16(workspace)) return FC_ERR_ALIGN;
  char* ws = static_cast<char*>(workspace);
  int* counts = reinterpret_cast<int*>(ws + l.counts);
  float* part = reinterpret_cast<float*>(ws + l.part);
  const int32_t* keys = species;
  const int32_t* idx = nullptr;
  for (int p = 0; p < l.g.passes; ++p) {
    int32_t* okeys = reinterpret_cast<int32_t*>(ws + l.keys[p & 1]);
    int32_t* oidx = reinterpret_cast<int32_t*>(ws + l.idx[p & 1]);
    sort_count_kernel<<<l.g.chunks, 256, 0, s>>>(l.g, 8 * p, p == 0, keys, counts);
    sort_scatter_kernel<<<l.g.chunks, 256, 0, s>>>(l.g, 8 * p, p == 0, keys, idx, counts, okeys, oidx);
    keys = okeys;
    idx = oidx;
  }
  const long long ldg = (long long)(lmax + 1) * (lmax + 1) * channels;
  if (dtype == FC_F32)
    span_sum<float>(l, channels, ldg, scale, keys, idx, g, table_bar, part, s);
  else if (dtype == FC_BF16)
    span_sum<__nv_bfloat16>(l, channels, ldg, scale, keys, idx, g, table_bar, part, s);
  else
    span_sum<__half>(l, channels, ldg, scale, keys, idx, g, table_bar, part, s);
  const long long spans = ((long long)n_nodes + l.g.span - 1) / l.g.span;
  const int join = spans > 1 ? (int)((spans + 31) / 32) : 0, clear = (int)(((long long)n_species + 1023) / 1024);
  span_join_kernel<<<dim3((unsigned)(join + clear), (channels + 127) / 128), 1024, 0, s>>>(
      n_nodes, n_species, channels, l.g.span, join, scale, keys, part, table_bar);
  return cudaGetLastError() == cudaSuccess ? FC_OK : FC_ERR_CUDA;
}

}  // extern "C"

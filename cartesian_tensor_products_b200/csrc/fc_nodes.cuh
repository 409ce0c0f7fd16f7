// Row types and small helpers shared by the node operators (species
// embedding, head norm with rotation, node attention).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fc_common.cuh"
#include "flashcart_nodes.h"

namespace fc {

template <class T>
struct RowType;
template <>
struct RowType<float> {
  static constexpr int kVec = 4;   // values of a 16-byte vector
  static __device__ __forceinline__ float to(float v) { return v; }
  static __device__ __forceinline__ float from(float v) { return v; }
};
template <>
struct RowType<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float to(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct RowType<__half> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float to(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from(float v) { return __float2half_rn(v); }
};

// W consecutive values as one aligned load or store (W sizeof(T) <= 16 bytes).
template <class T, int W>
struct alignas(sizeof(T) * W) Pack {
  T v[W];
};
template <class T, int W>
__device__ __forceinline__ void load_pack(const T* p, float (&out)[W]) {
  const Pack<T, W> a = *reinterpret_cast<const Pack<T, W>*>(p);
#pragma unroll
  for (int i = 0; i < W; ++i) out[i] = RowType<T>::to(a.v[i]);
}
template <class T, int W>
__device__ __forceinline__ void store_pack(T* p, const float (&in)[W]) {
  Pack<T, W> a;
#pragma unroll
  for (int i = 0; i < W; ++i) a.v[i] = RowType<T>::from(in[i]);
  *reinterpret_cast<Pack<T, W>*>(p) = a;
}

inline bool row_dtype(int dtype) { return dtype == FC_F32 || dtype == FC_BF16 || dtype == FC_F16; }
inline size_t row_size(int dtype) { return dtype == FC_F32 ? 4 : 2; }
inline size_t round16(size_t b) { return (b + 15) & ~(size_t)15; }

}  // namespace fc

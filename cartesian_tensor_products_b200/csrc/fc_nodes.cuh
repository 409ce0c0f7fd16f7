// Row types and small helpers shared by the node operators (species
// embedding, head norm with rotation, node attention).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

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

// Two 16-bit values in a word, the first in the low half.
template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// W consecutive values as one aligned load or store (W sizeof(T) <= 16 bytes),
// held as words: 16-bit values are converted two at a time (one at a time, with
// their packing, cost more instructions than a head's norm).
template <class T, int W>
struct alignas(sizeof(T) * W) Pack {
  static constexpr bool kPairs = sizeof(T) == 2 && W >= 2;
  using Word = typename std::conditional<kPairs, uint32_t, T>::type;
  static constexpr int kWords = kPairs ? W / 2 : W;
  Word w[kWords];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (kPairs)
        w[i] = 0u;
      else
        w[i] = RowType<T>::from(0.0f);
    }
  }
  __device__ __forceinline__ void get(float (&v)[W]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (kPairs) {
        const float2 f = unpack2<T>(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      } else {
        v[i] = RowType<T>::to(w[i]);
      }
    }
  }
  __device__ __forceinline__ void set(const float (&v)[W]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (kPairs)
        w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
      else
        w[i] = RowType<T>::from(v[i]);
    }
  }
};
template <class T, int W>
__device__ __forceinline__ void load_pack(const T* p, float (&out)[W]) {
  constexpr int P = sizeof(T) * W > 16 ? 16 / (int)sizeof(T) : W;   // values of one load
#pragma unroll
  for (int i = 0; i < W; i += P) {
    const Pack<T, P> a = *reinterpret_cast<const Pack<T, P>*>(p + i);
    float v[P];
    a.get(v);
#pragma unroll
    for (int k = 0; k < P; ++k) out[i + k] = v[k];
  }
}
template <class T, int W>
__device__ __forceinline__ void store_pack(T* p, const float (&in)[W]) {
  Pack<T, W> a;
  a.set(in);
  *reinterpret_cast<Pack<T, W>*>(p) = a;
}

inline bool row_dtype(int dtype) { return dtype == FC_F32 || dtype == FC_BF16 || dtype == FC_F16; }
inline size_t round16(size_t b) { return (b + 15) & ~(size_t)15; }

}  // namespace fc

// elem.cuh -- element types of the fp32-arithmetic kernels (gated scan, layer norm): packed
// loads of bf16, fp16 or fp32 values as floats, and their stores with one rounding.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace gla {

template <class T>
__device__ __forceinline__ float to_f32(T x) {
  if constexpr (sizeof(T) == 4) return x;
  else if constexpr (sizeof(T) == 2 && __is_same(T, __half)) return __half2float(x);
  else return __bfloat162float(x);
}
template <class T>
__device__ __forceinline__ T from_f32(float x) {
  if constexpr (sizeof(T) == 4) return x;
  else if constexpr (__is_same(T, __half)) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// V consecutive elements of type T as one access of V * sizeof(T) bytes (2, 4, 8, 16; 32 bytes
// as two of 16), which the address must be a multiple of.
template <class T, int V>
struct Pack {
  static constexpr int BYTES = V * (int)sizeof(T);
  static constexpr int WORDS = BYTES < 4 ? 1 : BYTES / 4;
  uint32_t w[WORDS];

  template <bool STREAM = true>
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (BYTES == 2) {
      w[0] = __ldg(reinterpret_cast<const unsigned short*>(p));
    } else if constexpr (BYTES == 4) {
      w[0] = STREAM ? __ldcs(reinterpret_cast<const uint32_t*>(p))
                    : __ldg(reinterpret_cast<const uint32_t*>(p));
    } else if constexpr (BYTES == 8) {
      const uint2 u = STREAM ? __ldcs(reinterpret_cast<const uint2*>(p))
                             : __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = u.x; w[1] = u.y;
    } else {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i) {
        const uint4 u = STREAM ? __ldcs(reinterpret_cast<const uint4*>(p) + i)
                               : __ldg(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (BYTES == 2) {
      *reinterpret_cast<unsigned short*>(p) = (unsigned short)w[0];
    } else if constexpr (BYTES == 4) {
      __stcs(reinterpret_cast<uint32_t*>(p), w[0]);
    } else if constexpr (BYTES == 8) {
      __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
    } else {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i)
        __stcs(reinterpret_cast<uint4*>(p) + i,
               make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
    }
  }
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int i = 0; i < V; ++i) set(i, x);
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[i]);
    } else {
      const uint32_t h = (i & 1) ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu;
      if constexpr (__is_same(T, __half)) return __half2float(__ushort_as_half((unsigned short)h));
      else return __uint_as_float(h << 16);
    }
  }
  __device__ __forceinline__ void set(int i, float x) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(x);
    } else {
      uint32_t h;
      if constexpr (__is_same(T, __half)) h = __half_as_ushort(__float2half_rn(x));
      else h = __bfloat16_as_ushort(__float2bfloat16_rn(x));
      if constexpr (V == 1) w[0] = h;
      else w[i / 2] = (i & 1) ? (w[i / 2] & 0xFFFFu) | (h << 16) : (w[i / 2] & 0xFFFF0000u) | h;
    }
  }
};

}  // namespace gla

// elem.cuh -- element types of the fp32-arithmetic kernels (gated scan, layer norm): packed
// loads of bf16, fp16 or fp32 values as floats, and their stores with one rounding.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace gla {

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
  // elements 2 i and 2 i + 1
  __device__ __forceinline__ float2 get2(int i) const {
    if constexpr (sizeof(T) == 4) return make_float2(get(2 * i), get(2 * i + 1));
    else if constexpr (__is_same(T, __half)) return __half22float2(reinterpret_cast<const __half2&>(w[i]));
    else return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  __device__ __forceinline__ void set2(int i, float2 x) {
    if constexpr (sizeof(T) == 4) {
      set(2 * i, x.x);
      set(2 * i + 1, x.y);
    } else if constexpr (__is_same(T, __half)) {
      reinterpret_cast<__half2&>(w[i]) = __floats2half2_rn(x.x, x.y);
    } else {
      reinterpret_cast<__nv_bfloat162&>(w[i]) = __floats2bfloat162_rn(x.x, x.y);
    }
  }
  // from shared memory
  __device__ __forceinline__ void load_shared(const T* p) {
    static_assert(BYTES >= 16, "whole 16-byte pieces");
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
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

// Two fp32 operations in one instruction: a * b + c, a + b, a * b.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}

}  // namespace gla

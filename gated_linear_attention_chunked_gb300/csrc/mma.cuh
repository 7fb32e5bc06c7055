// mma.cuh -- warp-level 16-bit matrix products (m16n8k16, fp32 accumulation) on swizzled
// shared-memory tiles, and the asynchronous copies that fill them.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "ptx.cuh"

namespace gla {

// A tile of rows of CHUNKS 16-byte chunks.  The chunk index is XORed with row bits so that the
// eight rows of one chunk column that a matrix load touches fall into different banks: three
// bits where the row is a multiple of 128 bytes, two (of row / 2) where it is one of 64.
template <int CHUNKS>
__device__ __forceinline__ uint32_t tile_off(int row, int chunk) {
  static_assert(CHUNKS % 4 == 0, "rows are multiples of 64 bytes");
  const int x = CHUNKS % 8 == 0 ? (row & 7) : ((row >> 1) & 3);
  return (uint32_t)(row * CHUNKS + (chunk ^ x)) * 16u;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// A operand: 16 rows from `row`, channels 8 chunk .. 8 chunk + 15.
template <int CHUNKS>
__device__ __forceinline__ void load_a(uint32_t (&a)[4], uint32_t tile, int row, int chunk) {
  const int l = threadIdx.x & 31;
  ldsm4(a, tile + tile_off<CHUNKS>(row + (l & 15), chunk + (l >> 4)));
}
// B operands of two 8-column blocks whose columns are the tile's rows (row, row + 8), the
// product running along the channels 8 chunk .. 8 chunk + 15: b[0..1] and b[2..3].
template <int CHUNKS>
__device__ __forceinline__ void load_b(uint32_t (&b)[4], uint32_t tile, int row, int chunk) {
  const int l = threadIdx.x & 31;
  ldsm4(b, tile + tile_off<CHUNKS>(row + (l & 7) + ((l >> 4) << 3), chunk + ((l >> 3) & 1)));
}
// B operands of two 8-column blocks whose columns are channels 8 chunk .. 8 chunk + 15, the
// product running along 16 rows from `row`.
template <int CHUNKS>
__device__ __forceinline__ void load_bt(uint32_t (&b)[4], uint32_t tile, int row, int chunk) {
  const int l = threadIdx.x & 31;
  ldsm4t(b, tile + tile_off<CHUNKS>(row + (l & 15), chunk + (l >> 4)));
}

template <class T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (__is_same(T, __half))
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (__is_same(T, __half)) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
// Two adjacent outputs of type TO.
template <class TO>
__device__ __forceinline__ void store2(TO* p, float a, float b) {
  if constexpr (sizeof(TO) == 4) *reinterpret_cast<float2*>(p) = make_float2(a, b);
  else *reinterpret_cast<uint32_t*>(p) = pack2<TO>(a, b);
}

// 16 bytes global -> shared, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// True in one lane of a converged warp.  Inside the branch on it the compiler knows that one lane
// runs and keeps tensor-core descriptors in uniform registers: a 128 x 64 x 16 product from tensor
// memory issues in 29 cycles, in 45 inside a branch on the lane's number.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

}  // namespace gla

// code8.cuh -- rows of a page in 8 bits.  A row x of 96 or 192 values of a 16-bit type is held as whole
// numbers c and one exponent e,
//
//   e = floor(log2(max |x|)) - 6, at least kLowest,   c = x 2^-e rounded to even, within +-127
//
// so a value is off by at most 2^(e-1), less than 1/128 of the row's largest, but for one above
// 127.5 2^e, which an fp16 row can have (off by less than 2^e).  A power of two in place of max / 127 costs
// half a bit on average and makes c 2^e a value of the row's own type, exactly: the products take the same
// operands as with pages of 16 bits, and nothing is rounded a second time.  (Below 2^-24 there are no
// fp16 values, below 2^-126 no normal fp32 scales: kLowest.)
#pragma once
#include "elem.cuh"

namespace gla {

// Infinities are held as the largest code, at most 127 2^kHighest, and NaN as 0.
template <class T>
constexpr int kLowest = __is_same(T, __half) ? -24 : -126;
template <class T>
constexpr int kHighest = __is_same(T, __half) ? 15 - 6 : 127 - 6;

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
// The scale of a stored exponent; below -126 is none that was written.
__device__ __forceinline__ float scale_of(int e) { return pow2(max(e, -126)); }

// Sixteen-bit words of two values as floats.
template <class T>
__device__ __forceinline__ float2 halves(uint32_t w) {
  if constexpr (__is_same(T, __half)) return __half22float2(reinterpret_cast<const __half2&>(w));
  else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// The larger magnitudes of two words' values; NaN counts for nothing beside a number.
template <class T>
__device__ __forceinline__ uint32_t top2(uint32_t a, uint32_t b) {
  a &= 0x7FFF7FFFu;
  b &= 0x7FFF7FFFu;
  if constexpr (__is_same(T, __half)) {
    const __half2 x = __hmax2(reinterpret_cast<__half2&>(a), reinterpret_cast<__half2&>(b));
    return reinterpret_cast<const uint32_t&>(x);
  } else {
    const __nv_bfloat162 x =
        __hmax2(reinterpret_cast<__nv_bfloat162&>(a), reinterpret_cast<__nv_bfloat162&>(b));
    return reinterpret_cast<const uint32_t&>(x);
  }
}
// NaN where one of them is.
template <class T>
__device__ __forceinline__ uint32_t top2_nan(uint32_t a, uint32_t b) {
  if constexpr (__is_same(T, __half)) {
    const __half2 x = __hmax2_nan(reinterpret_cast<__half2&>(a), reinterpret_cast<__half2&>(b));
    return reinterpret_cast<const uint32_t&>(x);
  } else {
    const __nv_bfloat162 x =
        __hmax2_nan(reinterpret_cast<__nv_bfloat162&>(a), reinterpret_cast<__nv_bfloat162&>(b));
    return reinterpret_cast<const uint32_t&>(x);
  }
}
// The exponent of a row whose largest magnitudes these are.
template <class T>
__device__ __forceinline__ int exponent_of(uint32_t top) {
  const float2 f = halves<T>(top & 0x7FFF7FFFu);
  const float x = fmaxf(fmaxf(f.x, f.y), 0.f);
  return min(max((int)(__float_as_uint(x) >> 23) - 127 - 6, kLowest<T>), kHighest<T>);
}
// Codes of eight values; NAN_: NaN among them, as 0.  3 2^22 + x, within fp32's whole numbers, has x rounded to
// even in its last bits (a conversion goes a quarter as fast).
template <class T, bool NAN_>
__device__ __forceinline__ uint2 codes_of(uint4 x, float inv) {
  uint2 c;
  const uint32_t* w = &x.x;
  uint32_t* o = &c.x;
  auto code = [&](float f) {
    constexpr float whole = 12582912.f;
    const float y = fminf(fmaxf(fmaf(f, inv, whole), whole - 127.f), whole + 127.f);
    return __float_as_uint(NAN_ && f != f ? whole : y);
  };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = halves<T>(w[2 * i]), b = halves<T>(w[2 * i + 1]);
    o[i] = __byte_perm(__byte_perm(code(a.x), code(a.y), 0x0040), __byte_perm(code(b.x), code(b.y), 0x0040), 0x5410);
  }
  return c;
}
// A row by L adjacent lanes (of a group aligned to L), each with three 16-byte chunks: chunk
// i L + l of x[i].  Returns the exponent; all of the warp's lanes take part.
template <class T, int L>
__device__ __forceinline__ int code_row(const uint4 (&x)[3], uint2 (&c)[3]) {
  uint32_t top = 0, any = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    top = top2<T>(top, top2<T>(top2<T>(x[i].x, x[i].y), top2<T>(x[i].z, x[i].w)));
    any = top2_nan<T>(any, top2_nan<T>(top2_nan<T>(x[i].x, x[i].y), top2_nan<T>(x[i].z, x[i].w)));
  }
#pragma unroll
  for (int s = 1; s < L; s <<= 1) top = top2<T>(top, __shfl_xor_sync(0xffffffffu, top, s));
  const int e = exponent_of<T>(top);
  const float inv = pow2(-e);
  const float2 f = halves<T>(any);
  if (f.x != f.x || f.y != f.y) {
#pragma unroll
    for (int i = 0; i < 3; ++i) c[i] = codes_of<T, true>(x[i], inv);
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i) c[i] = codes_of<T, false>(x[i], inv);
  }
  return e;
}

// Codes to 16-bit operands: four codes of a word as two words of two values each, whole numbers of
// at most 127 exactly.  even: codes 0, 2 (lo) and 1, 3 (hi); else 0, 1 and 2, 3.
template <class T, bool EVEN>
__device__ __forceinline__ void whole_of(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;  // c + 128
  if constexpr (__is_same(T, __half)) {
    // 0x6400 | u is 1024 + u
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    uint32_t a = __byte_perm(u, 0x64646464u, EVEN ? 0x4240 : 0x4140);
    uint32_t b = __byte_perm(u, 0x64646464u, EVEN ? 0x4341 : 0x4342);
    const __half2 x = __hsub2(reinterpret_cast<__half2&>(a), off);
    const __half2 y = __hsub2(reinterpret_cast<__half2&>(b), off);
    lo = reinterpret_cast<const uint32_t&>(x);
    hi = reinterpret_cast<const uint32_t&>(y);
  } else {
    // 0x4B000000 | u is 2^23 + u as fp32; the upper half of a whole number up to 127 is its bf16
    const float2 off = make_float2(-8388736.f, -8388736.f);
    const uint32_t m = 0x4B000000u;
    const float2 x = add2(make_float2(__uint_as_float(__byte_perm(u, m, 0x7440)),
                                      __uint_as_float(__byte_perm(u, m, EVEN ? 0x7442 : 0x7441))),
                          off);
    const float2 y = add2(make_float2(__uint_as_float(__byte_perm(u, m, EVEN ? 0x7441 : 0x7442)),
                                      __uint_as_float(__byte_perm(u, m, 0x7443))),
                          off);
    lo = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
    hi = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x7632);
  }
}
// Times a power of two (exact while the result is a value of the type).
template <class T>
__device__ __forceinline__ uint32_t scaled(uint32_t w, float s) {
  if constexpr (__is_same(T, __half)) {
    const __half2 x = __hmul2(reinterpret_cast<__half2&>(w), __half2half2(__float2half_rn(s)));
    return reinterpret_cast<const uint32_t&>(x);
  } else {
    const __nv_bfloat162 x =
        __hmul2(reinterpret_cast<__nv_bfloat162&>(w), __bfloat162bfloat162(__float2bfloat16_rn(s)));
    return reinterpret_cast<const uint32_t&>(x);
  }
}

}  // namespace gla

// window_common.cuh -- which keys a query of the windowed attention sees, shared by its kernels.
#pragma once
#include "elem.cuh"
#include "mma.cuh"
#include "window_attn.h"

namespace gla {

constexpr int kCK = kDK / 8, kCV = kDV / 8;  // 16-byte chunks of a key and a value row

// Query t sees key s if s <= t and (t - s < window or s < sink), within the sequence's len tokens.  As
// bits of a 32-bit word, 0 .. n (none for n < 0):
__device__ __forceinline__ uint32_t bits_to(int n) {
  return n < 0 ? 0u : n >= 31 ? ~0u : (2u << n) - 1;
}
// the keys c0 .. c0 + 31 that query t sees,
__device__ __forceinline__ uint32_t keys_seen(int t, int c0, int len, int window, int sink) {
  return bits_to(min(t, len - 1) - c0) & (~bits_to(t - window - c0) | bits_to(sink - 1 - c0));
}
// and the queries c0 .. c0 + 31 that see key s.
__device__ __forceinline__ uint32_t queries_seeing(int s, int c0, int len, int window, int sink) {
  const int end = s < sink ? len - 1 : (int)min((long long)len, (long long)s + window) - 1;
  return bits_to(end - c0) & ~bits_to(s - 1 - c0);
}

// The key tiles (of BN keys) that the queries [q0, q1) see: those of the window, lo .. hi, and
// in front of them the first `far` tiles, which hold the sinks.
struct KeyTiles {
  int lo, far, n;
  __device__ __forceinline__ KeyTiles(int q0, int q1, int BN, int window, int sink) {
    lo = max(0, q0 - window + 1) / BN;
    far = min((min(sink, q1) + BN - 1) / BN, lo);
    n = far + (q1 - 1) / BN - lo + 1;
  }
  __device__ __forceinline__ int tile(int i) const { return i < far ? i : lo + i - far; }
};

}  // namespace gla

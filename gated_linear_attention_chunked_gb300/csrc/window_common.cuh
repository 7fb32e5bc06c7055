// window_common.cuh -- which keys a query of the windowed attention sees, shared by its kernels.
#pragma once
#include "elem.cuh"
#include "mma.cuh"
#include "window_attn.h"

namespace gla {

constexpr int kCK = kDK / 8, kCV = kDV / 8;  // 16-byte chunks of a key and a value row

// Query t sees key s: itself, the window - 1 tokens before it, and the first `sink` tokens.
__device__ __forceinline__ bool window_sees(int t, int s, int window, int sink) {
  return s <= t && (t - s < window || s < sink);
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

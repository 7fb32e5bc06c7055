// window_wait.cuh -- the bounded waits of the windowed attention's forward and gradient.  Some of them
// last a whole item (the output rows' for its sums, the loader's for the roles to take it), and an item
// grows with the sequence: with a window of all of T it streams T / 128 tiles forward and
// (H / KV) T / 64 in the gradient, 0.9 and 0.7 us each.  So the limit counts from the last step that
// the CTA made: a tile whose product with the weights the issuer sent off, or an item that the output
// warps finished.
#pragma once
#include "scan_common.cuh"

namespace gla {

// Behind the CTA's abort flag: steps of the issuer and of the output warps.
constexpr uint32_t kWaitWords = 3;
enum Step : int { STEP_TILE = 1, STEP_ITEM = 2 };
__device__ __forceinline__ void made_step(const scan::Cta& cta, Step which, int n) {
  cta.abort_flag()[which] = n;
}

static __device__ __noinline__ bool wait_moving(volatile int* words, uint32_t bar, uint32_t parity,
                                                int* err, unsigned long long wait_ns) {
  uint64_t t0 = globaltimer();
  int tile = words[STEP_TILE], item = words[STEP_ITEM];
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 31u) == 0) {
      if (words[0]) return false;
      const int tile_now = words[STEP_TILE], item_now = words[STEP_ITEM];
      const uint64_t now = globaltimer();
      if (tile_now != tile || item_now != item) {
        tile = tile_now;
        item = item_now;
        t0 = now;
      } else if (now - t0 > wait_ns) {
        DevCtl c;
        c.err = err;
        c.wait_ns = wait_ns;
        record_error(c, DEV_TIMEOUT);
        words[0] = 1;
        return false;
      }
    }
  }
}
// As scan::wait and scan::wait_warp, with that limit.
__device__ __forceinline__ bool await(const scan::Cta& cta, uint32_t bar, uint32_t parity,
                                     const DevCtl& ctl) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_moving(cta.abort_flag(), bar, parity, ctl.err, ctl.wait_ns);
}
__device__ __forceinline__ bool await_warp(const scan::Cta& cta, uint32_t bar, uint32_t parity,
                                          const DevCtl& ctl) {
  return __all_sync(0xffffffffu, await(cta, bar, parity, ctl));
}

}  // namespace gla

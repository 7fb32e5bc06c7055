// window_chunk8.cu -- chunks of new tokens over pages of 8 bits (window_chunk.cuh).
#include "window_chunk.cuh"

namespace gla {
namespace chunk {

cudaError_t launch8(const ChunkArgs& a, const Plan& plan, DevCtl ctl, cudaStream_t stream) {
  return a.cache.c.type == GLA_BF16 ? run<__nv_bfloat16, true>(a, plan, ctl, stream)
                                    : run<__half, true>(a, plan, ctl, stream);
}

}  // namespace chunk
}  // namespace gla

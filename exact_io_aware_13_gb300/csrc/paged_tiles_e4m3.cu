// The paged tile kernel over an e4m3 cache, in a translation unit of its own so that it
// compiles in parallel.
#include "paged_tiles.cuh"

namespace attn {
cudaError_t launch_paged_tiles_e4m3(const PagedAttention& a, cudaStream_t st) {
  return pt::launch_tiles<true>(a, PagedMaps{}, st);
}
}  // namespace attn

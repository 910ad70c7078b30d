// The paged tile kernel over a bf16 cache.
#include "paged_tiles.cuh"

namespace attn {
cudaError_t launch_paged_tiles_bf16(const PagedAttention& a, const PagedMaps& maps, cudaStream_t st) {
  return pt::launch_tiles<false>(a, maps, st);
}
}  // namespace attn

// Attention of drafted trees over a paged cache: cross attention's kernel
// (cross_kernel.cuh) with the trees' masks, over bf16 and e4m3 caches.
#include "cross_kernel.cuh"

namespace splitkv {

cudaError_t launch_tree(const CrossArgs& a, int64_t row_tiles, const CrossMaps& maps, bool fp8, void* stream) {
  cudaError_t e = fp8 ? launch_cross_kernel<true, true>(a, maps, stream) : launch_cross_kernel<true, false>(a, maps, stream);
  return e == cudaSuccess ? launch_cross_merge(a, row_tiles, stream) : e;
}

}  // namespace splitkv

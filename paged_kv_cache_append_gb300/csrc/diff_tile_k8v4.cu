// diff_tile_k8v4.cu -- differential attention tiles of the K8V4 profile.
#include "diff_tile.cuh"

namespace nk {

cudaError_t diff_tile_k8v4(const nk_pool* p, int layer, const DiffTileArgs& a, bool both, dim3 grid, cudaStream_t s) {
  return diff_tile_dispatch<KIND_FP8, KIND_NVFP4>(p, layer, a, both, grid, s);
}

}  // namespace nk

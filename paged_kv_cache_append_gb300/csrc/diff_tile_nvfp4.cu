// diff_tile_nvfp4.cu -- differential attention tiles of the NVFP4-G16 profile.
#include "diff_tile.cuh"

namespace nk {

cudaError_t diff_tile_nvfp4(const nk_pool* p, int layer, const DiffTileArgs& a, bool both, dim3 grid, cudaStream_t s) {
  return diff_tile_dispatch<KIND_NVFP4, KIND_NVFP4>(p, layer, a, both, grid, s);
}

}  // namespace nk

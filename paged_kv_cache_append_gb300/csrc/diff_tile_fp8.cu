// diff_tile_fp8.cu -- differential attention tiles of the FP8-row profile.
#include "diff_tile.cuh"

namespace nk {

cudaError_t diff_tile_fp8(const nk_pool* p, int layer, const DiffTileArgs& a, bool both, dim3 grid, cudaStream_t s) {
  return diff_tile_dispatch<KIND_FP8, KIND_FP8>(p, layer, a, both, grid, s);
}

}  // namespace nk

// diff_tile_bf16.cu -- differential attention tiles of the BF16 profile.
#include "diff_tile.cuh"

namespace nk {

cudaError_t diff_tile_bf16(const nk_pool* p, int layer, const DiffTileArgs& a, bool both, dim3 grid, cudaStream_t s) {
  return diff_tile_dispatch<KIND_BF16, KIND_BF16>(p, layer, a, both, grid, s);
}

}  // namespace nk

// diff_tile_int8.cu -- differential attention tiles of the INT8-G64 profile.
#include "diff_tile.cuh"

namespace nk {

cudaError_t diff_tile_int8(const nk_pool* p, int layer, const DiffTileArgs& a, bool both, dim3 grid, cudaStream_t s) {
  return diff_tile_dispatch<KIND_INT8, KIND_INT8>(p, layer, a, both, grid, s);
}

}  // namespace nk

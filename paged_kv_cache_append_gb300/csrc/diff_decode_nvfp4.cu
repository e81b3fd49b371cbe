// diff_decode_nvfp4.cu -- differential decode instantiations of the NVFP4-G16 profile.
#include "diff_decode.cuh"

namespace nk {

cudaError_t diff_decode_nvfp4(const nk_pool* p, int layer, const DiffDecodeArgs& a, bool pack, cudaStream_t s) {
  return diff_decode_dispatch<KIND_NVFP4, KIND_NVFP4>(p, layer, a, pack, s);
}

}  // namespace nk

// diff_decode_fp8.cu -- differential decode instantiations of the FP8-row profile.
#include "diff_decode.cuh"

namespace nk {

cudaError_t diff_decode_fp8(const nk_pool* p, int layer, const DiffDecodeArgs& a, bool pack, cudaStream_t s) {
  return diff_decode_dispatch<KIND_FP8, KIND_FP8>(p, layer, a, pack, s);
}

}  // namespace nk

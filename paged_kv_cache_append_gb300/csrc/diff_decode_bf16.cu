// diff_decode_bf16.cu -- differential decode instantiations of the BF16 profile.
#include "diff_decode.cuh"

namespace nk {

cudaError_t diff_decode_bf16(const nk_pool* p, int layer, const DiffDecodeArgs& a, bool pack, cudaStream_t s) {
  return diff_decode_dispatch<KIND_BF16, KIND_BF16>(p, layer, a, pack, s);
}

}  // namespace nk

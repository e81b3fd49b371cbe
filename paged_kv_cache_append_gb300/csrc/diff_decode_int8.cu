// diff_decode_int8.cu -- differential decode instantiations of the INT8-G64 profile.
#include "diff_decode.cuh"

namespace nk {

cudaError_t diff_decode_int8(const nk_pool* p, int layer, const DiffDecodeArgs& a, bool pack, cudaStream_t s) {
  return diff_decode_dispatch<KIND_INT8, KIND_INT8>(p, layer, a, pack, s);
}

}  // namespace nk

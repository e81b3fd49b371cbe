// diff_decode_k8v4.cu -- differential decode instantiations of the K8V4 profile.
#include "diff_decode.cuh"

namespace nk {

cudaError_t diff_decode_k8v4(const nk_pool* p, int layer, const DiffDecodeArgs& a, bool pack, cudaStream_t s) {
  return diff_decode_dispatch<KIND_FP8, KIND_NVFP4>(p, layer, a, pack, s);
}

}  // namespace nk

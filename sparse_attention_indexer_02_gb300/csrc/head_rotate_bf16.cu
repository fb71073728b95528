// The bf16 instantiations of the head rotation (head_rotate.cuh).
#include "head_rotate.cuh"

namespace qsa {

cudaError_t launch_rotate_bf16(const RotateParams& p, cudaStream_t stream) {
  return rot::launch_rotate_t<false>(p, stream);
}

}  // namespace qsa

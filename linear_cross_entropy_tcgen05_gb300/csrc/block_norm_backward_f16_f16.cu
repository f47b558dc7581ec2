// block_norm_backward_f16_f16.cu -- the block norm's backward kernels for f16 activations and a f16 residual stream.
#include "block_norm_kernels.cuh"

namespace flce {

cudaError_t bn_backward_f16_f16(const BlockNormParams& p, const BlockNormShape& s, bool vec, int feat, unsigned blocks,
                                cudaStream_t stream) {
  using TX = __half;
  using TR = __half;
  constexpr bool BACKWARD = true;
#define KERNEL flce_block_norm_backward_kernel
  FLCE_BN_DISPATCH();
}

}  // namespace flce

// block_norm_backward_f32_f32.cu -- the block norm's backward kernels for f32 activations and an f32 residual stream.
#include "block_norm_kernels.cuh"

namespace flce {

cudaError_t bn_backward_f32_f32(const BlockNormParams& p, const BlockNormShape& s, bool vec, int feat, unsigned blocks,
                                cudaStream_t stream) {
  using TX = float;
  using TR = float;
  constexpr bool BACKWARD = true;
#define KERNEL flce_block_norm_backward_kernel
  FLCE_BN_DISPATCH();
}

}  // namespace flce

// block_norm_backward_bf16_bf16.cu -- the block norm's backward kernels for bf16 activations and a bf16 residual stream.
#include "block_norm_kernels.cuh"

namespace flce {

cudaError_t bn_backward_bf16_bf16(const BlockNormParams& p, const BlockNormShape& s, bool vec, int feat, unsigned blocks,
                                  cudaStream_t stream) {
  using TX = __nv_bfloat16;
  using TR = __nv_bfloat16;
  constexpr bool BACKWARD = true;
#define KERNEL flce_block_norm_backward_kernel
  FLCE_BN_DISPATCH();
}

}  // namespace flce

// block_norm_forward_f16_f16.cu -- the block norm's forward kernels for f16 activations and a f16 residual stream.
#include "block_norm_kernels.cuh"

namespace flce {

cudaError_t bn_forward_f16_f16(const BlockNormParams& p, const BlockNormShape& s, bool vec, int feat, unsigned blocks,
                               cudaStream_t stream) {
  using TX = __half;
  using TR = __half;
  constexpr bool BACKWARD = false;
#define KERNEL flce_block_norm_forward_kernel
  FLCE_BN_DISPATCH(FLCE_BN_WIDE_CASES);
}

}  // namespace flce

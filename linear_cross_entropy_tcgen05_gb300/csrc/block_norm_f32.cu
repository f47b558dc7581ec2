// block_norm_f32.cu -- the block norm's kernels for fp32 activations.
#include "block_norm_kernels.cuh"

namespace flce {

cudaError_t bn_forward_f32(const BlockNormParams& p, const BlockNormShape& s, bool, bool vec, int feat, unsigned blocks,
                           cudaStream_t stream) {
  return bn_forward_typed<float, float>(p, s, vec, feat, blocks, stream);
}

cudaError_t bn_backward_f32(const BlockNormParams& p, const BlockNormShape& s, bool, bool vec, int feat,
                            unsigned blocks, cudaStream_t stream) {
  return bn_backward_typed<float, float>(p, s, vec, feat, blocks, stream);
}

}  // namespace flce

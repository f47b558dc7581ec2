// block_norm_bf16.cu -- the block norm's kernels for bf16 activations (bf16 or fp32 residual stream).
#include "block_norm_kernels.cuh"

namespace flce {

cudaError_t bn_forward_bf16(const BlockNormParams& p, const BlockNormShape& s, bool res_f32, bool vec, int feat, unsigned blocks,
                          cudaStream_t stream) {
  return res_f32 ? bn_forward_typed<__nv_bfloat16, float>(p, s, vec, feat, blocks, stream)
                 : bn_forward_typed<__nv_bfloat16, __nv_bfloat16>(p, s, vec, feat, blocks, stream);
}

cudaError_t bn_backward_bf16(const BlockNormParams& p, const BlockNormShape& s, bool res_f32, bool vec, int feat,
                           unsigned blocks, cudaStream_t stream) {
  return res_f32 ? bn_backward_typed<__nv_bfloat16, float>(p, s, vec, feat, blocks, stream)
                 : bn_backward_typed<__nv_bfloat16, __nv_bfloat16>(p, s, vec, feat, blocks, stream);
}

}  // namespace flce

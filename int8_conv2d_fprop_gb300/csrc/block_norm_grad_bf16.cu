// block_norm_grad_bf16.cu -- the block norm's gradient for x of bfloat16.
#include "block_norm_grad.cuh"

namespace i8c {

bool launch_block_norm_grad_bf16(const BlockNormGradArgs &a, const Held &h, bool wide_stream, int64_t grid, size_t smem, cudaStream_t s) {
    return wide_stream ? launch_backward<__nv_bfloat16, float>(a, h, grid, smem, s) : launch_backward<__nv_bfloat16, __nv_bfloat16>(a, h, grid, smem, s);
}

}  // namespace i8c

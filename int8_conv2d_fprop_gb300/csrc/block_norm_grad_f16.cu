// block_norm_grad_f16.cu -- the block norm's gradient for x of float16.
#include "block_norm_grad.cuh"

namespace i8c {

bool launch_block_norm_grad_f16(const BlockNormGradArgs &a, const Held &h, bool wide_stream, int64_t grid, size_t smem, cudaStream_t s) {
    return wide_stream ? launch_backward<__half, float>(a, h, grid, smem, s) : launch_backward<__half, __half>(a, h, grid, smem, s);
}

}  // namespace i8c

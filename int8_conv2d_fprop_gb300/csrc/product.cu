// product.cu -- D[a,b] = epilogue(sum_k A[a,k] * B[b,k]) for 16-bit float
// operands with any strides.
#include <cuda_runtime.h>

#include "channel.h"
#include "channel_math.cuh"

namespace i8c {

bool product_in_place(const void *p, int64_t rows, int64_t rs, int64_t cols, int64_t cs) {
    if (rows <= 1) rs = 0;
    if (cols <= 1) cs = 0;
    if ((uintptr_t)p % 16) return false;
    return (cs <= 1 && rs % 8 == 0) || (rs <= 1 && cs % 8 == 0);
}

namespace {

constexpr int T = 64, KT = 16;

// 64 x 64 outputs per block, 4 x 4 per thread, both operands staged as
// floats in shared memory.
template <int kAct>
__global__ void __launch_bounds__(256) product_simple_kernel(Product pr) {
    __shared__ float sa[KT][T + 1], sb[KT][T + 1];
    const int64_t a0 = (int64_t)blockIdx.x * T, b0 = (int64_t)blockIdx.y * T;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < pr.k; k0 += KT) {
        for (int i = threadIdx.x; i < T * KT; i += 256) {
            const int kk = i % KT, r = i / KT;
            const bool kin = k0 + kk < pr.k;
            sa[kk][r] = (kin && a0 + r < pr.ma)
                            ? load_as_float(pr.a.p, (a0 + r) * pr.a.s_mn + (k0 + kk) * pr.a.s_k, pr.in_dtype) : 0.0f;
            sb[kk][r] = (kin && b0 + r < pr.nb)
                            ? load_as_float(pr.b.p, (b0 + r) * pr.b.s_mn + (k0 + kk) * pr.b.s_k, pr.in_dtype) : 0.0f;
        }
        __syncthreads();
        for (int kk = 0; kk < KT; ++kk)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] += sa[kk][ty + 16 * i] * sb[kk][tx + 16 * j];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t a = a0 + ty + 16 * i, b = b0 + tx + 16 * j;
            if (a >= pr.ma || b >= pr.nb) continue;
            float z = acc[i][j];
            if (pr.bias) z += load_as_float(pr.bias, pr.bias_along_a ? a : b, pr.bias_dtype);
            if (pr.pre) store_from_float(pr.pre, a * pr.pre_sa + b * pr.pre_sb, pr.in_dtype, z);
            float v = activate<kAct>(z);
            if (pr.res) v += load_as_float(pr.res, a * pr.res_sa + b * pr.res_sb, pr.d_dtype);
            store_from_float(pr.d, a * pr.d_sa + b * pr.d_sb, pr.d_dtype, v);
        }
}

template <int kAct>
conv_status launch(const Product &pr, cudaStream_t s) {
    const dim3 grid((unsigned)((pr.ma + T - 1) / T), (unsigned)((pr.nb + T - 1) / T));
    if (grid.y > 65535) return CONV_ERR_TOO_LARGE;
    product_simple_kernel<kAct><<<grid, 256, 0, s>>>(pr);
    return cudaGetLastError() == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

}  // namespace

conv_status product_launch(const Product &pr, void *stream) {
    if (pr.ma == 0 || pr.nb == 0) return CONV_OK;
    const cudaStream_t s = (cudaStream_t)stream;
    switch (pr.act) {
        case CONV_ACT_RELU: return launch<CONV_ACT_RELU>(pr, s);
        case CONV_ACT_GELU: return launch<CONV_ACT_GELU>(pr, s);
        case CONV_ACT_GELU_TANH: return launch<CONV_ACT_GELU_TANH>(pr, s);
        case CONV_ACT_SILU: return launch<CONV_ACT_SILU>(pr, s);
        default: return launch<CONV_ACT_NONE>(pr, s);
    }
}

}  // namespace i8c

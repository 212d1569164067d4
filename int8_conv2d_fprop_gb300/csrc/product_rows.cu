// product_rows.cu -- the product for up to four rows of activations: a call's
// latency and the stream of weights are all there is, and the tensor-core
// kernel's set-up (tensor memory, barriers, a cluster's partial sums) takes
// longer than the work.
//
// y[m,n] = epilogue(sum_k x[m,k] w[n,k]): a block takes four rows of w, its
// eight warps a stretch of k each; a lane reads 16 bytes of every row at a
// time and multiplies on the CUDA cores in 32 bits (at 6.8 TB/s an SM gets 12
// weights per clock, which leaves room for one row and not for many more).
// The warps' sums meet in shared memory in a fixed order.  (Whole rows to a
// warp, without the meeting, measured 33 us against 28 on 4096 x 16384.)
#include <cuda_runtime.h>

#include "channel.h"
#include "channel_launch.cuh"
#include "channel_math.cuh"
#include "tc_ptx.cuh"

namespace i8c {
namespace {

constexpr int kRowsW = 4;  // rows of w per block
constexpr int kWarps = 8;

template <int kAct>
__device__ __forceinline__ float activate_one(float z) {
    float other = 0.0f;
    activate<kAct>(z, other);
    return z;
}

template <int kM>
__global__ void __launch_bounds__(32 * kWarps) product_rows_kernel(const Product pr) {
    __shared__ float part[kWarps][kM][kRowsW];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t n0 = (int64_t)blockIdx.x * kRowsW;
    const int64_t groups = pr.k / 8, per = (groups + kWarps * 32 - 1) / (kWarps * 32) * 32;
    const int64_t g1 = min(groups, (warp + 1) * per);
    const uint16_t *w = (const uint16_t *)pr.b.p, *x = (const uint16_t *)pr.a.p;
    const bool half = pr.in_dtype == CONV_FLOAT16;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    float sum[kM][kRowsW] = {};
    auto rows = [&](auto f) {
#pragma unroll 2
        for (int64_t g = warp * per + lane; g < g1; g += 32) {
            uint4 q[kRowsW], u[kM];
#pragma unroll
            for (int r = 0; r < kRowsW; ++r)
                q[r] = n0 + r < pr.nb ? *reinterpret_cast<const uint4 *>(w + (n0 + r) * pr.b.s_mn + g * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int m = 0; m < kM; ++m) u[m] = *reinterpret_cast<const uint4 *>(x + m * pr.a.s_mn + g * 8);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 a[kM];
#pragma unroll
                for (int m = 0; m < kM; ++m) a[m] = f((&u[m].x)[i]);
#pragma unroll
                for (int r = 0; r < kRowsW; ++r) {
                    const float2 b = f((&q[r].x)[i]);
#pragma unroll
                    for (int m = 0; m < kM; ++m) sum[m][r] = fmaf(a[m].y, b.y, fmaf(a[m].x, b.x, sum[m][r]));
                }
            }
        }
    };
    if (half) rows([](uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); });
    else rows([](uint32_t v) { return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)); });
    // the last k mod 8, a lane each
    const int64_t tail = groups * 8 + lane;
    if (warp == 0 && tail < pr.k) {
#pragma unroll
        for (int r = 0; r < kRowsW; ++r) {
            if (n0 + r >= pr.nb) break;
            const float b = load_as_float(pr.b.p, (n0 + r) * pr.b.s_mn + tail, pr.in_dtype);
#pragma unroll
            for (int m = 0; m < kM; ++m) sum[m][r] = fmaf(load_as_float(pr.a.p, m * pr.a.s_mn + tail, pr.in_dtype), b, sum[m][r]);
        }
    }
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int r = 0; r < kRowsW; ++r) {
            float s = sum[m][r];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) part[warp][m][r] = s;
        }
    __syncthreads();
    if (threadIdx.x >= kM * kRowsW) return;
    const int m = threadIdx.x / kRowsW, r = threadIdx.x % kRowsW;
    const int64_t n = n0 + r;
    if (n >= pr.nb) return;
    float z = 0.0f;
    for (int i = 0; i < kWarps; ++i) z += part[i][m][r];
    if (pr.bias) z += load_as_float(pr.bias, n, pr.bias_dtype);
    if (pr.pre) store_from_float(pr.pre, m * pr.pre_sa + n * pr.pre_sb, pr.in_dtype, z);
    switch (pr.act) {
        case CONV_ACT_RELU: z = activate_one<CONV_ACT_RELU>(z); break;
        case CONV_ACT_GELU: z = activate_one<CONV_ACT_GELU>(z); break;
        case CONV_ACT_GELU_TANH: z = activate_one<CONV_ACT_GELU_TANH>(z); break;
        case CONV_ACT_SILU: z = activate_one<CONV_ACT_SILU>(z); break;
        default: break;
    }
    if (pr.res) z += load_as_float(pr.res, m * pr.res_sa + n * pr.res_sb, pr.d_dtype);
    store_from_float(pr.d, m * pr.d_sa + n * pr.d_sb, pr.d_dtype, z);
}

}  // namespace

bool product_rows_applies(const Product &pr) {
    // w and x with k contiguous (and so, being readable in place, aligned rows)
    // (one row: 3.4 us against 7.6 at 1024 x 1024, as fast at 4096 x 16384;
    // four: 3.2 against 6.7, but 44 against 27, where the multiplications
    // outlast the stream)
    return pr.ma <= 4 && !pr.bias_along_a && pr.nb >= 64 && pr.k >= 64 && pr.a.s_k == 1 && pr.b.s_k == 1 &&
           (pr.ma == 1 || pr.ma * pr.nb * pr.k <= 48 << 20);
}

conv_status product_rows_launch(const Product &pr, void *stream) {
    const dim3 grid((unsigned)((pr.nb + kRowsW - 1) / kRowsW));
    const cudaStream_t s = (cudaStream_t)stream;
    bool ok;
    switch (pr.ma) {
        case 1: ok = launch_behind(product_rows_kernel<1>, grid, 32 * kWarps, 0, s, pr); break;
        case 2: ok = launch_behind(product_rows_kernel<2>, grid, 32 * kWarps, 0, s, pr); break;
        case 3: ok = launch_behind(product_rows_kernel<3>, grid, 32 * kWarps, 0, s, pr); break;
        default: ok = launch_behind(product_rows_kernel<4>, grid, 32 * kWarps, 0, s, pr); break;
    }
    return ok ? CONV_OK : CONV_ERR_CUDA;
}

}  // namespace i8c

// scaled_rows.cu -- the product of 8-bit operands for a few rows of
// activations: the stream of weights is all there is.
//
// A block takes 16 rows of w, its eight warps the blocks of 128 k in turn; a
// lane reads 32 bytes of two rows of w and of a row of x in each.  The
// multiplications run on the tensor cores' warp-level form (16 rows of w by 8
// of x, f16 operands, which hold the 8-bit values exactly, 32-bit sums): a
// lane's bytes go to the instruction in the order in which they lie in
// memory, for both operands alike, so that nothing is rearranged.  Each block's
// sums are scaled and added in 32 bits; the warps' sums meet in shared memory
// in a fixed order.
#include <cuda_runtime.h>

#include <algorithm>

#include "channel.h"
#include "channel_launch.cuh"
#include "channel_math.cuh"
#include "eight_bit.cuh"
#include "tc_ptx.cuh"

namespace i8c {
namespace {

constexpr int kRowsW = 16;  // rows of w per block
constexpr int kWarps = 8;

// Bytes k0 .. k0 + 31 of a row, zeros from k on.
__device__ __forceinline__ void load32(const uint8_t *row, int64_t k0, int64_t k, bool valid, uint32_t (&v)[8]) {
    if (valid && k0 + 32 <= k) {
        const uint4 a = reinterpret_cast<const uint4 *>(row + k0)[0], b = reinterpret_cast<const uint4 *>(row + k0)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = 0;
        if (valid && k0 + 4 * i < k) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k0 + 4 * i + j < k) v[i] |= (uint32_t)row[k0 + 4 * i + j] << (8 * j);
        }
    }
}

// c += A (16 x 16) B (16 x 8), f16 operands.
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float activate_value(float z, int32_t act) {
    float other = 0.0f;
    switch (act) {
        case CONV_ACT_RELU: activate<CONV_ACT_RELU>(z, other); break;
        case CONV_ACT_GELU: activate<CONV_ACT_GELU>(z, other); break;
        case CONV_ACT_GELU_TANH: activate<CONV_ACT_GELU_TANH>(z, other); break;
        case CONV_ACT_SILU: activate<CONV_ACT_SILU>(z, other); break;
        default: break;
    }
    return z;
}

// kG: groups of 8 rows of x.
template <int kG, bool kXE5m2, bool kWE5m2>
__global__ void __launch_bounds__(32 * kWarps) scaled_rows_kernel(const ScaledProduct pr) {
    __shared__ float part[kWarps][8 * kG][kRowsW + 1];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, t = lane & 3;
    const int64_t n0 = (int64_t)blockIdx.x * kRowsW;
    const int blocks = (int)((pr.k + kScaleBlock - 1) / kScaleBlock);
    const bool w_in[2] = {n0 + g < pr.nb, n0 + g + 8 < pr.nb};
    const uint8_t *w = pr.b.p + (n0 + g) * pr.b.rs;
    const float *ws[2] = {pr.b.scale + ((n0 + g) >> pr.b.shift) * pr.b.s_rs, pr.b.scale + ((n0 + g + 8) >> pr.b.shift) * pr.b.s_rs};
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    for (int64_t m0 = (int64_t)blockIdx.y * 8 * kG; m0 < pr.ma; m0 += (int64_t)gridDim.y * 8 * kG) {
        float acc[kG][4] = {};
#pragma unroll 2
        for (int kb = warp; kb < blocks; kb += kWarps) {
            const int64_t k0 = (int64_t)kb * kScaleBlock + t * 32;
            uint32_t wq[2][8], xq[kG][8];
#pragma unroll
            for (int h = 0; h < 2; ++h) load32(w + 8 * h * pr.b.rs, k0, pr.k, w_in[h], wq[h]);
            float sw[2], sx[kG][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) sw[h] = w_in[h] ? ws[h][kb * pr.b.s_cs] : 0.0f;
#pragma unroll
            for (int j = 0; j < kG; ++j) {
                load32(pr.a.p + (m0 + 8 * j + g) * pr.a.rs, k0, pr.k, m0 + 8 * j + g < pr.ma, xq[j]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t m = m0 + 8 * j + 2 * t + h;
                    sx[j][h] = m < pr.ma ? pr.a.scale[(m >> pr.a.shift) * pr.a.s_rs + kb * pr.a.s_cs] : 0.0f;
                }
            }
            float c[kG][4] = {};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t a[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    a[h] = unpack_eight_bit<kWE5m2>((uint16_t)wq[h][i]);
                    a[2 + h] = unpack_eight_bit<kWE5m2>((uint16_t)(wq[h][i] >> 16));
                }
#pragma unroll
                for (int j = 0; j < kG; ++j)
                    mma_16816(c[j], a[0], a[1], a[2], a[3], unpack_eight_bit<kXE5m2>((uint16_t)xq[j][i]),
                              unpack_eight_bit<kXE5m2>((uint16_t)(xq[j][i] >> 16)));
            }
#pragma unroll
            for (int j = 0; j < kG; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(sw[e >> 1] * sx[j][e & 1], c[j][e], acc[j][e]);
        }
        __syncthreads();  // (the previous rows' sums have been read)
#pragma unroll
        for (int j = 0; j < kG; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[warp][8 * j + 2 * t + (e & 1)][g + 8 * (e >> 1)] = acc[j][e];
        __syncthreads();
        for (int i = threadIdx.x; i < 8 * kG * kRowsW; i += 32 * kWarps) {
            const int64_t m = m0 + i / kRowsW, n = n0 + i % kRowsW;
            if (m >= pr.ma || n >= pr.nb) continue;
            float z = 0.0f;
#pragma unroll
            for (int v = 0; v < kWarps; ++v) z += part[v][i / kRowsW][i % kRowsW];
            if (pr.bias) z += load_as_float(pr.bias, n, pr.bias_dtype);
            if (pr.pre) store_from_float(pr.pre, m * pr.pre_sa + n * pr.pre_sb, pr.pre_dtype, z);
            z = activate_value(z, pr.act);
            if (pr.res) z += load_as_float(pr.res, m * pr.res_sa + n * pr.res_sb, pr.d_dtype);
            store_from_float(pr.d, m * pr.d_sa + n * pr.d_sb, pr.d_dtype, z);
        }
    }
}

template <int kG>
bool launch(const ScaledProduct &pr, dim3 grid, cudaStream_t s) {
    if (pr.a.e5m2)
        return pr.b.e5m2 ? launch_behind(scaled_rows_kernel<kG, true, true>, grid, 32 * kWarps, 0, s, pr)
                         : launch_behind(scaled_rows_kernel<kG, true, false>, grid, 32 * kWarps, 0, s, pr);
    return pr.b.e5m2 ? launch_behind(scaled_rows_kernel<kG, false, true>, grid, 32 * kWarps, 0, s, pr)
                     : launch_behind(scaled_rows_kernel<kG, false, false>, grid, 32 * kWarps, 0, s, pr);
}

}  // namespace

bool scaled_rows_applies(int64_t ma, int64_t nb, int64_t k) { return ma <= 32 || k == 0; }

conv_status scaled_rows_launch(const ScaledProduct &pr, void *stream) {
    const int64_t groups = std::min<int64_t>((pr.ma + 7) / 8, 4);
    const int64_t tiles = (pr.ma + 8 * groups - 1) / (8 * groups);
    const dim3 grid((unsigned)((pr.nb + kRowsW - 1) / kRowsW), (unsigned)std::min<int64_t>(tiles, 65535));
    const cudaStream_t s = (cudaStream_t)stream;
    bool ok;
    switch (groups) {
        case 1: ok = launch<1>(pr, grid, s); break;
        case 2: ok = launch<2>(pr, grid, s); break;
        case 3: ok = launch<3>(pr, grid, s); break;
        default: ok = launch<4>(pr, grid, s); break;
    }
    return ok ? CONV_OK : CONV_ERR_CUDA;
}

}  // namespace i8c

// scaled_rows.cu -- the product of 8-bit operands for a few rows of
// activations: the stream of weights is all there is.
//
// A warp takes 16 rows of w and every split-th block of 128 k, as many warps to
// the same rows as fill the GPU (16 per SM, which all run at once); a lane
// reads 32 bytes of two rows of w and of a row of x, a block ahead of the one
// it multiplies.  The multiplications run on the tensor cores' warp-level form
// (16 rows of w by 8 of x, f16 operands, which hold the 8-bit values exactly,
// 32-bit sums): a lane's bytes go to the instruction in the order in which
// they lie in memory, for both operands alike, so that nothing is rearranged.
// Each block's sums are scaled and added in 32 bits; the warps' sums meet in
// shared memory in a fixed order.  One row through 4096 x 4096 takes 4.8 us, 8
// rows through 4096 x 16384 15.9 us (4.2 TB/s), 16 rows 18.4; 33 rows through
// 4096 x 4096 take the tensor-core tiles 10.6 us, 16 rows here 5.7.
#include <cuda_runtime.h>

#include <algorithm>

#include "channel.h"
#include "channel_launch.cuh"
#include "channel_math.cuh"
#include "eight_bit.cuh"
#include "tc_ptx.cuh"

namespace i8c {
namespace {

constexpr int kRowsW = 16;  // rows of w per warp
constexpr int kWarps = 8;

// Bytes k0 .. k0 + 31 of a row, zeros from k on.
__device__ __forceinline__ void load32(const uint8_t *row, int64_t k0, int64_t k, uint32_t (&v)[8]) {
    if (k0 + 32 <= k) {
        const uint4 a = reinterpret_cast<const uint4 *>(row + k0)[0], b = reinterpret_cast<const uint4 *>(row + k0)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (k0 + 4 * i + j < k) v[i] |= (uint32_t)row[k0 + 4 * i + j] << (8 * j);
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

// What a lane has of one block of k.
template <int kG>
struct Loaded {
    uint32_t w[2][8], x[kG][8];
    float sw[2], sx[kG][2];
};

// kG: groups of 8 rows of x.  split: warps to the same rows of w.
template <int kG, bool kXE5m2, bool kWE5m2>
__global__ void __launch_bounds__(32 * kWarps, 2) scaled_rows_kernel(const ScaledProduct pr, int split) {
    __shared__ float part[kWarps][8 * kG][kRowsW + 1];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, t = lane & 3;
    const int tiles = kWarps / split;  // of 16 rows of w, in this block
    const int64_t n0 = ((int64_t)blockIdx.x * tiles + warp / split) * kRowsW;
    const int blocks = (int)((pr.k + kScaleBlock - 1) / kScaleBlock);
    // (rows past the last are read as the first: nothing of theirs is stored, and rows do not meet)
    const uint8_t *w[2], *x[kG];
    const float *ws[2], *xs[kG][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t n = n0 + g + 8 * h < pr.nb ? n0 + g + 8 * h : 0;
        w[h] = pr.b.p + n * pr.b.rs;
        ws[h] = pr.b.scale + (n >> pr.b.shift) * pr.b.s_rs;
    }
#pragma unroll
    for (int j = 0; j < kG; ++j) {
        x[j] = pr.a.p + (8 * j + g < pr.ma ? 8 * j + g : 0) * pr.a.rs;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t m = 8 * j + 2 * t + h < pr.ma ? 8 * j + 2 * t + h : 0;
            xs[j][h] = pr.a.scale + (m >> pr.a.shift) * pr.a.s_rs;
        }
    }
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    auto load = [&](Loaded<kG> &f, int kb) {
        const int64_t k0 = (int64_t)kb * kScaleBlock + t * 32;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            load32(w[h], k0, pr.k, f.w[h]);
            f.sw[h] = ws[h][kb * pr.b.s_cs];
        }
#pragma unroll
        for (int j = 0; j < kG; ++j) {
            load32(x[j], k0, pr.k, f.x[j]);
#pragma unroll
            for (int h = 0; h < 2; ++h) f.sx[j][h] = xs[j][h][kb * pr.a.s_cs];
        }
    };
    float acc[kG][4] = {};
    auto multiply = [&](const Loaded<kG> &f) {
        float c[kG][4] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t a[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                a[h] = unpack_eight_bit<kWE5m2>((uint16_t)f.w[h][i]);
                a[2 + h] = unpack_eight_bit<kWE5m2>((uint16_t)(f.w[h][i] >> 16));
            }
#pragma unroll
            for (int j = 0; j < kG; ++j)
                mma_16816(c[j], a[0], a[1], a[2], a[3], unpack_eight_bit<kXE5m2>((uint16_t)f.x[j][i]),
                          unpack_eight_bit<kXE5m2>((uint16_t)(f.x[j][i] >> 16)));
        }
#pragma unroll
        for (int j = 0; j < kG; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(f.sw[e >> 1] * f.sx[j][e & 1], c[j][e], acc[j][e]);
    };
    Loaded<kG> f0, f1;
    int kb = warp % split;
    if (kb < blocks) load(f0, kb);
#pragma unroll 1
    for (; kb < blocks; kb += 2 * split) {
        if (kb + split < blocks) load(f1, kb + split);
        multiply(f0);
        if (kb + 2 * split < blocks) load(f0, kb + 2 * split);
        if (kb + split < blocks) multiply(f1);
    }
#pragma unroll
    for (int j = 0; j < kG; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[warp][8 * j + 2 * t + (e & 1)][g + 8 * (e >> 1)] = acc[j][e];
    __syncthreads();
    for (int i = threadIdx.x; i < tiles * 8 * kG * kRowsW; i += 32 * kWarps) {
        const int tile = i / (8 * kG * kRowsW), m = i / kRowsW % (8 * kG);
        const int64_t n = ((int64_t)blockIdx.x * tiles + tile) * kRowsW + i % kRowsW;
        if (m >= pr.ma || n >= pr.nb) continue;
        float z = 0.0f;
        for (int v = 0; v < split; ++v) z += part[tile * split + v][m][i % kRowsW];
        if (pr.bias) z += load_as_float(pr.bias, n, pr.bias_dtype);
        if (pr.pre) store_from_float(pr.pre, m * pr.pre_sa + n * pr.pre_sb, pr.pre_dtype, z);
        z = activate_value(z, pr.act);
        if (pr.res) z += load_as_float(pr.res, m * pr.res_sa + n * pr.res_sb, pr.d_dtype);
        store_from_float(pr.d, m * pr.d_sa + n * pr.d_sb, pr.d_dtype, z);
    }
}

template <int kG>
bool launch(const ScaledProduct &pr, cudaStream_t s) {
    // warps to the same 16 rows of w: as many as 16 per SM allow
    const int64_t rows = (pr.nb + kRowsW - 1) / kRowsW;
    int split = kWarps;
    while (split > 1 && rows * split > 16 * 152) split /= 2;
    const int64_t tiles = kWarps / split;
    const dim3 grid((unsigned)((rows + tiles - 1) / tiles));
    const int threads = 32 * kWarps;
    if (pr.a.e5m2)
        return pr.b.e5m2 ? launch_behind(scaled_rows_kernel<kG, true, true>, grid, threads, 0, s, pr, split)
                         : launch_behind(scaled_rows_kernel<kG, true, false>, grid, threads, 0, s, pr, split);
    return pr.b.e5m2 ? launch_behind(scaled_rows_kernel<kG, false, true>, grid, threads, 0, s, pr, split)
                     : launch_behind(scaled_rows_kernel<kG, false, false>, grid, threads, 0, s, pr, split);
}

}  // namespace

// (More rows than two groups of 8 do not fit the registers with a block ahead.)
bool scaled_rows_applies(int64_t ma, int64_t nb, int64_t k) { return ma <= 16; }

conv_status scaled_rows_launch(const ScaledProduct &pr, void *stream) {
    const cudaStream_t s = (cudaStream_t)stream;
    return (pr.ma <= 8 ? launch<1>(pr, s) : launch<2>(pr, s)) ? CONV_OK : CONV_ERR_CUDA;
}

}  // namespace i8c

// quantize.cu -- conv_quantize: 8-bit floats with a scale for each block of
// 128, by rows, by columns (transposed), or both.
//
// A block of 256 threads holds a tile of 128 x 128 in registers, thread t the
// rows 8 (t / 16) .. + 7 of columns 8 (t % 16) .. + 7: it is read once, in
// 16-byte vectors, and every scale of either form is the maximum over threads
// that meet in a half warp (a row) or in shared memory (a column, the tile).
// The row form is written from the registers, 128 bytes of a row by 16
// threads; the column form is turned through 16 KB of shared memory in pieces
// of 8 bytes, so that it too leaves in runs of 128.  A stream: what bounds it
// is memory.
#include <cuda_runtime.h>

#include "channel.h"
#include "channel_launch.cuh"
#include "channel_math.cuh"
#include "channel_rows.cuh"
#include "eight_bit.cuh"
#include "tc_ptx.cuh"

namespace i8c {
namespace {

constexpr int kTile = 128;

struct QuantizeArgs {
    MatRef x, pre, q, scale, qt, scale_t;
    int64_t rows, cols;
    int32_t tiles_c;
    int32_t act, whole;       // whole: one scale for the tile
    int32_t pre_vec;          // preact in aligned vectors
    int32_t q_vec, qt_vec;    // outputs in aligned pieces of 8 bytes
};

// 8 elements of a row from column c on, zeros from `cols` on.
template <typename X, bool kVec>
__device__ __forceinline__ void load8(const MatRef &m, int64_t r, int64_t c, int64_t cols, float (&v)[8]) {
    const X *p = (const X *)m.p + r * m.rs + c * (kVec ? 1 : m.cs);
    if (kVec && c + 8 <= cols) {
        if constexpr (kIs16<X>) {
            unpack8(*reinterpret_cast<const uint4 *>(p), std::is_same_v<X, __half> ? CONV_FLOAT16 : CONV_BFLOAT16, v);
        } else {
            const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int32_t type = std::is_same_v<X, float> ? CONV_FLOAT32 : std::is_same_v<X, __half> ? CONV_FLOAT16 : CONV_BFLOAT16;
        v[j] = c + j < cols ? load_as_float(p, kVec ? j : j * m.cs, type) : 0.0f;
    }
}

// v * act'(z) for 8 elements of preact, whose type is its own.
__device__ __noinline__ void slopes8(const MatRef &pre, int64_t r, int64_t c, int64_t cols, bool vec, int32_t act,
                                     float *v) {
    float z[8];
    const int64_t at = r * pre.rs + c * pre.cs;
    if (vec && c + 8 <= cols) {
        unpack8(*reinterpret_cast<const uint4 *>((const uint16_t *)pre.p + at), pre.dtype, z);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = c + j < cols ? load_as_float(pre.p, at + j * pre.cs, pre.dtype) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        switch (act) {
            case CONV_ACT_RELU: activation_slope<CONV_ACT_RELU>(z[j], z[j + 1]); break;
            case CONV_ACT_GELU: activation_slope<CONV_ACT_GELU>(z[j], z[j + 1]); break;
            case CONV_ACT_GELU_TANH: activation_slope<CONV_ACT_GELU_TANH>(z[j], z[j + 1]); break;
            default: activation_slope<CONV_ACT_SILU>(z[j], z[j + 1]); break;
        }
        v[j] *= z[j];
        v[j + 1] *= z[j + 1];
    }
}

// 8 bytes of a line from element c on.
__device__ __forceinline__ void store8(const MatRef &m, int64_t r, int64_t c, int64_t cols, bool vec, uint32_t lo,
                                       uint32_t hi) {
    uint8_t *p = (uint8_t *)const_cast<void *>(m.p) + r * m.rs + c * m.cs;
    if (vec && c + 8 <= cols) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (c + j < cols) p[j * m.cs] = (uint8_t)((j < 4 ? lo : hi) >> (j % 4 * 8));
}

template <typename X, bool kVec, bool kSlope, bool kE5m2>
__global__ void __launch_bounds__(256, 2) quantize_kernel(const QuantizeArgs a) {
    __shared__ __align__(16) uint32_t most[8][kTile];
    __shared__ __align__(16) uint2 turned[kTile][kTile / 8];
    const int cg = threadIdx.x % 16, rg = threadIdx.x / 16, warp = threadIdx.x / 32;
    const int64_t tr = blockIdx.x / a.tiles_c, tc = blockIdx.x - tr * a.tiles_c;
    const int64_t r0 = tr * kTile + rg * 8, c0 = tc * kTile + cg * 8;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (r0 + i < a.rows) {
            load8<X, kVec>(a.x, r0 + i, c0, a.cols, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
        }
    }
    if constexpr (kSlope) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (r0 + i < a.rows) slopes8(a.pre, r0 + i, c0, a.cols, a.pre_vec, a.act, v[i]);
    }

    // a magnitude for the tile, or for every row and every column of it
    BlockScale tile_scale{};
    if (a.whole) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, magnitude(v[i][j]));
        m = __reduce_max_sync(0xffffffffu, m);
        if (threadIdx.x % 32 == 0) most[0][warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w) m = max(m, most[0][w]);
        tile_scale = block_scale<kE5m2>(m);
        if (threadIdx.x == 0) {
            if (a.q.p) ((float *)const_cast<void *>(a.scale.p))[tr * a.scale.rs + tc * a.scale.cs] = tile_scale.scale;
            if (a.qt.p) ((float *)const_cast<void *>(a.scale_t.p))[tc * a.scale_t.rs + tr * a.scale_t.cs] = tile_scale.scale;
        }
    }
    if (a.q.p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            BlockScale s = tile_scale;
            if (!a.whole) {
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = max(m, magnitude(v[i][j]));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                s = block_scale<kE5m2>(m);
                if (cg == i && r0 + i < a.rows)
                    ((float *)const_cast<void *>(a.scale.p))[(r0 + i) * a.scale.rs + tc * a.scale.cs] = s.scale;
            }
            const float f = s.factor;
            if (r0 + i < a.rows)
                store8(a.q, r0 + i, c0, a.cols, a.q_vec,
                       pack_eight_bit<kE5m2>(v[i][0] * f, v[i][1] * f, v[i][2] * f, v[i][3] * f),
                       pack_eight_bit<kE5m2>(v[i][4] * f, v[i][5] * f, v[i][6] * f, v[i][7] * f));
        }
    }
    if (!a.qt.p) return;
    float f[8];
    if (a.whole) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = tile_scale.factor;
    } else {
        uint32_t m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m[j] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m[j] = max(m[j], magnitude(v[i][j]));
            m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
        }
        if (threadIdx.x % 32 < 16) {
            *reinterpret_cast<uint4 *>(&most[warp][cg * 8]) = make_uint4(m[0], m[1], m[2], m[3]);
            *reinterpret_cast<uint4 *>(&most[warp][cg * 8 + 4]) = make_uint4(m[4], m[5], m[6], m[7]);
        }
        __syncthreads();
        // a column's scale by one thread, its factor to the others
        if (threadIdx.x < kTile) {
            uint32_t c = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) c = max(c, most[w][threadIdx.x]);
            const BlockScale s = block_scale<kE5m2>(c);
            const int64_t col = tc * kTile + threadIdx.x;
            if (col < a.cols) ((float *)const_cast<void *>(a.scale_t.p))[col * a.scale_t.rs + tr * a.scale_t.cs] = s.scale;
            most[0][threadIdx.x] = __float_as_uint(s.factor);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(most[0][cg * 8 + j]);
    }
    // (pieces exchanged so that 16 threads' meet all banks)
#pragma unroll
    for (int j = 0; j < 8; ++j)
        turned[cg * 8 + j][rg ^ cg] =
            make_uint2(pack_eight_bit<kE5m2>(v[0][j] * f[j], v[1][j] * f[j], v[2][j] * f[j], v[3][j] * f[j]),
                       pack_eight_bit<kE5m2>(v[4][j] * f[j], v[5][j] * f[j], v[6][j] * f[j], v[7][j] * f[j]));
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int col = i * 16 + rg;
        const uint2 b = turned[col][cg ^ (col >> 3)];
        if (tc * kTile + col < a.cols)
            store8(a.qt, tc * kTile + col, tr * kTile + cg * 8, a.rows, a.qt_vec, b.x, b.y);
    }
}

template <typename X, bool kVec, bool kSlope>
bool launch(const QuantizeArgs &a, int64_t grid, bool e5m2, cudaStream_t s) {
    return e5m2 ? launch_behind(quantize_kernel<X, kVec, kSlope, true>, dim3((unsigned)grid), 256, 0, s, a)
                : launch_behind(quantize_kernel<X, kVec, kSlope, false>, dim3((unsigned)grid), 256, 0, s, a);
}

template <typename X>
bool launch_for(const QuantizeArgs &a, int64_t grid, bool e5m2, cudaStream_t s) {
    const bool vec = vector_rows(a.x);
    if (a.pre.p) return vec ? launch<X, true, true>(a, grid, e5m2, s) : launch<X, false, true>(a, grid, e5m2, s);
    return vec ? launch<X, true, false>(a, grid, e5m2, s) : launch<X, false, false>(a, grid, e5m2, s);
}

int64_t blocks_of(int64_t n) { return (n + kScaleBlock - 1) / kScaleBlock; }

// One form's output and its scales: of the right types and extents.
conv_status check_pair(const conv_matrix_desc *q, const void *q_dev, const conv_matrix_desc *scale, const void *scale_dev,
                       int64_t rows, int64_t cols, int32_t tile) {
    if (!scale) return CONV_ERR_NULL_PTR;
    conv_status st;
    if ((st = check_matrix(q)) || (st = check_matrix(scale))) return st;
    if (!is_eight_bit_type(q->dtype) || scale->dtype != CONV_FLOAT32) return CONV_ERR_DTYPE;
    if (q->rows != rows || q->cols != cols || scale->rows != (rows + tile - 1) / tile || scale->cols != blocks_of(cols))
        return CONV_ERR_SHAPE_MISMATCH;
    if ((st = check_address(q, q_dev)) || (st = check_address(scale, scale_dev))) return st;
    return CONV_OK;
}

}  // namespace
}  // namespace i8c

using namespace i8c;

extern "C" conv_status conv_quantize(const conv_matrix_desc *x, const void *x_dev, const conv_matrix_desc *preact,
                                     const void *preact_dev, const conv_matrix_desc *q, void *q_dev,
                                     const conv_matrix_desc *scale, void *scale_dev, const conv_matrix_desc *qt,
                                     void *qt_dev, const conv_matrix_desc *scale_t, void *scale_t_dev,
                                     const conv_quantize_params *p, void *stream) {
    if (!x || !p || (!q && !qt) || (!q && scale) || (!qt && scale_t)) return CONV_ERR_NULL_PTR;
    conv_status st;
    if ((st = check_matrix(x))) return st;
    if (!is_float_type(x->dtype)) return CONV_ERR_DTYPE;
    if ((p->tile != 1 && p->tile != kTile) || p->activation < CONV_ACT_NONE || p->activation > CONV_ACT_SILU ||
        p->reserved[0] != 0 || p->reserved[1] != 0)
        return CONV_ERR_BAD_PARAM;
    if ((st = check_address(x, x_dev))) return st;
    const int64_t m = x->rows, c = x->cols;
    if (p->activation == CONV_ACT_NONE) preact = nullptr;
    else if (!preact) return CONV_ERR_NULL_PTR;
    if (preact) {
        if ((st = check_matrix(preact))) return st;
        if (!is_half_type(preact->dtype) && preact->dtype != x->dtype) return CONV_ERR_DTYPE;
        if (preact->rows != m || preact->cols != c) return CONV_ERR_SHAPE_MISMATCH;
        if ((st = check_address(preact, preact_dev))) return st;
    }
    if (q && (st = check_pair(q, q_dev, scale, scale_dev, m, c, p->tile))) return st;
    if (qt && (st = check_pair(qt, qt_dev, scale_t, scale_t_dev, c, m, p->tile))) return st;
    if (q && qt && q->dtype != qt->dtype) return CONV_ERR_DTYPE;
    if (m == 0 || c == 0) return CONV_OK;
    const conv_matrix_desc *d[] = {x, preact, q, scale, qt, scale_t};
    const void *at[] = {x_dev, preact_dev, q_dev, scale_dev, qt_dev, scale_t_dev};
    for (int i = 2; i < 6; ++i)
        for (int j = 0; j < i; ++j)
            if (d[i] && d[j] && matrices_overlap(d[i], at[i], d[j], at[j])) return CONV_ERR_OVERLAP;
    const int64_t tiles_c = blocks_of(c), grid = blocks_of(m) * tiles_c;
    if (grid > INT32_MAX) return CONV_ERR_TOO_LARGE;
    if ((st = check_device())) return st;
    QuantizeArgs a;
    a.x = mat_ref(x, x_dev), a.pre = mat_ref(preact, preact_dev);
    a.q = mat_ref(q, q_dev), a.scale = mat_ref(scale, scale_dev);
    a.qt = mat_ref(qt, qt_dev), a.scale_t = mat_ref(scale_t, scale_t_dev);
    a.rows = m, a.cols = c, a.tiles_c = (int32_t)tiles_c;
    a.act = p->activation, a.whole = p->tile == kTile;
    auto pieces = [](const MatRef &r, int64_t cols) {
        return (r.cs == 1 || cols == 1) && r.rs % 8 == 0 && (uintptr_t)r.p % 8 == 0;
    };
    a.pre_vec = preact && is_half_type(preact->dtype) && vector_rows(a.pre);
    a.q_vec = q && pieces(a.q, c), a.qt_vec = qt && pieces(a.qt, m);
    const bool e5m2 = (q ? q : qt)->dtype == CONV_FLOAT8_E5M2;
    const cudaStream_t s = (cudaStream_t)stream;
    bool ok;
    switch (x->dtype) {
        case CONV_FLOAT32: ok = launch_for<float>(a, grid, e5m2, s); break;
        case CONV_FLOAT16: ok = launch_for<__half>(a, grid, e5m2, s); break;
        default: ok = launch_for<__nv_bfloat16>(a, grid, e5m2, s); break;
    }
    return ok ? CONV_OK : CONV_ERR_CUDA;
}

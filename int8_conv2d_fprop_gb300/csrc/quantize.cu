// quantize.cu -- conv_quantize: 8-bit floats with a scale for each block of
// 128, by rows, by columns (transposed), or both.
//
// A block of 512 threads holds a tile of 128 x 128 in registers, thread t the
// rows 4 (t / 16) .. + 3 of columns 8 (t % 16) .. + 7: it is read once, in
// 16-byte vectors (of rows that begin anywhere: aligned ones joined by
// shifts), and every scale of either form is the maximum over threads that
// meet in a half warp (a row) or in shared memory (a column, the tile).  The
// row form is written from the registers, 128 bytes of a row by 16 threads;
// the column form is turned through 16 KB of shared memory in pieces of 4
// bytes, so that it too leaves in runs of 128.  A stream: 16384 x 4096 bf16 to
// rows takes 36.6 us (5.6 TB/s).  With slopes and both forms the instructions
// bound it (59 per element; 35.3 us for 2047 x 5001 f16 with odd strides).
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
constexpr int kThreads = 512;
constexpr int kRows = 4;  // of a thread

// How a matrix's rows are read.
enum Reads : int32_t {
    kReadVectors,  // 16-byte aligned
    kReadShifted,  // 16-bit elements, adjacent, from any address
    kReadAny,      // an element at a time
};

struct QuantizeArgs {
    MatRef x, pre, q, scale, qt, scale_t;
    const uint16_t *x_end, *pre_end;  // of the matrices, for reads that are shifted
    int64_t rows, cols;
    int32_t tiles_c;
    int32_t act, whole;       // whole: one scale for the tile
    int32_t pre_reads;
    int32_t q_vec, qt_vec;    // outputs in aligned pieces of 8 bytes
};

// 16 bytes from element c of a row that begins anywhere, c = 8 (lane % 16) + a
// multiple of 128: the aligned vector and the next lane's, moved together by
// the row's offset.  Vectors reach into the row's neighbours but not past the
// matrix, [lo, hi); where they would, the elements are read one by one.  What
// lies from `cols` on is not of the row.  (The whole warp takes part; without
// a row p is NULL.)
__device__ __forceinline__ uint4 load16_shifted(const uint16_t *row, int64_t c, int64_t cols, const uint16_t *lo,
                                                const uint16_t *hi) {
    const int lead = (int)((uintptr_t)row / 2 & 7);
    const uint16_t *v = row - lead + c;
    const bool mine = row && v >= lo && v + 8 <= hi, whole = mine && (lead == 0 || v + 16 <= hi);
    const uint4 q = mine ? *reinterpret_cast<const uint4 *>(v) : make_uint4(0, 0, 0, 0);
    uint32_t w[8] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[4 + i] = __shfl_down_sync(0xffffffffu, w[i], 1, 16);
    if (threadIdx.x % 16 == 15 && whole && lead) {
        const uint4 n = *reinterpret_cast<const uint4 *>(v + 8);
        w[4] = n.x, w[5] = n.y, w[6] = n.z, w[7] = n.w;
    }
    if (lead & 4) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (lead & 2) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (lead & 1) * 16);
    if (row && !whole) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t u = c + e < cols ? row[c + e] : 0u;
            w[e / 2] = e % 2 ? w[e / 2] | u << 16 : u;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 elements of row r from column c on, as stored; what lies from `cols` on is
// not to be used.
template <typename X, int kReads>
__device__ __forceinline__ void load8(const MatRef &m, const uint16_t *end, int64_t r, int64_t rows, int64_t c, int64_t cols,
                                      Group<X> &g) {
    if constexpr (kReads == kReadShifted) {
        const uint4 q = load16_shifted(r < rows && c < cols + 8 ? (const uint16_t *)m.p + r * m.rs : nullptr, c, cols,
                                       (const uint16_t *)m.p, end);
        g.w[0] = q.x, g.w[1] = q.y, g.w[2] = q.z, g.w[3] = q.w;
        return;
    }
    if (r >= rows) {
#pragma unroll
        for (int j = 0; j < (int)(sizeof(g.w) / 4); ++j) g.w[j] = 0;
        return;
    }
    const X *p = (const X *)m.p + r * m.rs + c * (kReads == kReadVectors ? 1 : m.cs);
    if (kReads == kReadVectors && c + 8 <= cols) {
        const uint4 a = reinterpret_cast<const uint4 *>(p)[0];
        g.w[0] = a.x, g.w[1] = a.y, g.w[2] = a.z, g.w[3] = a.w;
        if constexpr (!kIs16<X>) {
            const uint4 b = reinterpret_cast<const uint4 *>(p)[1];
            g.w[4] = b.x, g.w[5] = b.y, g.w[6] = b.z, g.w[7] = b.w;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t at = kReads == kReadVectors ? j : j * m.cs;
        if constexpr (kIs16<X>) {
            const uint32_t v = c + j < cols ? reinterpret_cast<const uint16_t *>(p)[at] : 0u;
            g.w[j / 2] = j % 2 ? g.w[j / 2] | v << 16 : v;
        } else {
            g.w[j] = c + j < cols ? reinterpret_cast<const uint32_t *>(p)[at] : 0u;
        }
    }
}

// 8 values of preact as stored, where it is read in vectors (and has 16 bits):
// like x's, none of them from past the matrix.
__device__ __forceinline__ uint4 load_preact(const QuantizeArgs &a, int64_t r, int64_t c) {
    const MatRef &m = a.pre;
    if (a.pre_reads == kReadShifted)
        return load16_shifted(r < a.rows && c < a.cols + 8 ? (const uint16_t *)m.p + r * m.rs : nullptr, c, a.cols,
                              (const uint16_t *)m.p, a.pre_end);
    Group<__half> g;  // (either type, as stored)
    load8<__half, kReadVectors>(m, nullptr, r, a.rows, c, a.cols, g);
    return make_uint4(g.w[0], g.w[1], g.w[2], g.w[3]);
}

template <int kAct>
__device__ __forceinline__ void times_slope(const QuantizeArgs &a, int64_t r, int64_t c, const uint4 &zq, float (&v)[8]) {
    float z[8];
    if (a.pre_reads != kReadAny) {
        unpack8(zq, a.pre.dtype, z);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            z[j] = r < a.rows && c + j < a.cols ? load_as_float(a.pre.p, r * a.pre.rs + (c + j) * a.pre.cs, a.pre.dtype) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        activation_slope<kAct>(z[j], z[j + 1]);
        v[j] *= z[j];
        v[j + 1] *= z[j + 1];
    }
}

// Larger of each half's 16 bits.
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// The 32-bit float's bits of a magnitude in the 16 bits of type X.
template <typename X>
__device__ __forceinline__ uint32_t widened(uint32_t m) {
    if constexpr (std::is_same_v<X, __half>) return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
    else return m << 16;
}

// A thread's values: as they were read (16 bits), or as 32-bit floats.
template <typename X, bool kRaw>
struct Values {
    Group<X> g[kRows];
    __device__ __forceinline__ Pair at(int i, int j) const { return element2(g[i], j); }  // of row i, elements 2j and 2j + 1
    __device__ __forceinline__ uint32_t row_most(int i) const {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max16x2(m, g[i].w[j] & 0x7fff7fffu);
        return widened<X>(max(m & 0xffffu, m >> 16));
    }
    __device__ __forceinline__ void column_most(uint32_t (&m)[8]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w = 0;
#pragma unroll
            for (int i = 0; i < kRows; ++i) w = max16x2(w, g[i].w[j] & 0x7fff7fffu);
            w = max16x2(w, __shfl_xor_sync(0xffffffffu, w, 16));
            m[2 * j] = widened<X>(w & 0xffffu), m[2 * j + 1] = widened<X>(w >> 16);
        }
    }
};
template <typename X>
struct Values<X, false> {
    float v[kRows][8];
    __device__ __forceinline__ Pair at(int i, int j) const { return pair(v[i][2 * j], v[i][2 * j + 1]); }
    __device__ __forceinline__ uint32_t row_most(int i) const {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, magnitude(v[i][j]));
        return m;
    }
    __device__ __forceinline__ void column_most(uint32_t (&m)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m[j] = 0;
#pragma unroll
            for (int i = 0; i < kRows; ++i) m[j] = max(m[j], magnitude(v[i][j]));
            m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
        }
    }
};

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

// kColumns: also (or only) the column form.
template <typename X, int kReads, bool kSlope, bool kE5m2, bool kColumns>
__global__ void __launch_bounds__(kThreads, kIs16<X> && !kSlope ? 3 : 2) quantize_kernel(const QuantizeArgs a) {
    __shared__ __align__(16) uint32_t most[kThreads / 32][kColumns ? kTile : 1];
    __shared__ __align__(16) uint32_t turned[kColumns ? kTile : 1][kTile / 4];
    const int cg = threadIdx.x % 16, rg = threadIdx.x / 16, warp = threadIdx.x / 32;
    const int64_t tr = blockIdx.x / a.tiles_c, tc = blockIdx.x - tr * a.tiles_c;
    const int64_t r0 = tr * kTile + rg * kRows, c0 = tc * kTile + cg * 8;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    constexpr bool kRaw = kIs16<X> && !kSlope;
    Values<X, kRaw> v;
    {
        Group<X> g[kRows];
        uint4 z[kSlope ? kRows : 1];
#pragma unroll
        for (int i = 0; i < kRows; ++i) load8<X, kReads>(a.x, a.x_end, r0 + i, a.rows, c0, a.cols, g[i]);
        if constexpr (kSlope) {
            if (a.pre_reads != kReadAny) {
#pragma unroll
                for (int i = 0; i < kRows; ++i) z[i] = load_preact(a, r0 + i, c0);
            }
        }
        if constexpr (kRaw) {
#pragma unroll
            for (int i = 0; i < kRows; ++i) v.g[i] = g[i];
        } else {
#pragma unroll
            for (int i = 0; i < kRows; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) v.v[i][j] = element(g[i], j);
        }
        if constexpr (kSlope) {
            auto all = [&](auto act) {
#pragma unroll
                for (int i = 0; i < kRows; ++i) times_slope<decltype(act)::value>(a, r0 + i, c0, z[i], v.v[i]);
            };
            switch (a.act) {
                case CONV_ACT_RELU: all(std::integral_constant<int, CONV_ACT_RELU>()); break;
                case CONV_ACT_GELU: all(std::integral_constant<int, CONV_ACT_GELU>()); break;
                case CONV_ACT_GELU_TANH: all(std::integral_constant<int, CONV_ACT_GELU_TANH>()); break;
                default: all(std::integral_constant<int, CONV_ACT_SILU>()); break;
            }
        }
    }
    if (c0 + 8 > a.cols) {  // (what is not of the row may be anything)
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + j >= a.cols) {
                    if constexpr (kRaw) v.g[i].w[j / 2] &= j % 2 ? 0x0000ffffu : 0xffff0000u;
                    else v.v[i][j] = 0.0f;
                }
    }

    // a magnitude for the tile, or for every row and every column of it
    BlockScale tile_scale{};
    if (a.whole) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kRows; ++i) m = max(m, v.row_most(i));
        m = __reduce_max_sync(0xffffffffu, m);
        if (threadIdx.x % 32 == 0) most[warp][0] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = max(m, most[w][0]);
        tile_scale = block_scale<kE5m2>(m);
        if (threadIdx.x == 0) {
            if (a.q.p) ((float *)const_cast<void *>(a.scale.p))[tr * a.scale.rs + tc * a.scale.cs] = tile_scale.scale;
            if (a.qt.p) ((float *)const_cast<void *>(a.scale_t.p))[tc * a.scale_t.rs + tr * a.scale_t.cs] = tile_scale.scale;
        }
    }
    if (!kColumns || a.q.p) {
        // (thread i of a half warp writes row i's scale: neighbouring rows' in one access)
        BlockScale s = tile_scale;
        if (!a.whole) {
            uint32_t mine = 0;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                uint32_t m = v.row_most(i);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                if (cg == i) mine = m;
            }
            s = block_scale<kE5m2>(mine);  // (the divisions once for a row, by its thread)
            if (cg < kRows && r0 + cg < a.rows)
                ((float *)const_cast<void *>(a.scale.p))[(r0 + cg) * a.scale.rs + tc * a.scale.cs] = s.scale;
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const Pair f = pair(__shfl_sync(0xffffffffu, s.factor, i, 16)), rest = pair(__shfl_sync(0xffffffffu, s.rest, i, 16));
            float q[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) split(quotient(v.at(i, j), f, rest), &q[2 * j], &q[2 * j + 1]);
            if (r0 + i < a.rows)
                store8(a.q, r0 + i, c0, a.cols, a.q_vec, pack_eight_bit<kE5m2>(q[0], q[1], q[2], q[3]),
                       pack_eight_bit<kE5m2>(q[4], q[5], q[6], q[7]));
        }
    }
    if constexpr (kColumns) {
        if (!a.whole) {
            uint32_t m[8];
            v.column_most(m);
            if (threadIdx.x % 32 < 16) {
                *reinterpret_cast<uint4 *>(&most[warp][cg * 8]) = make_uint4(m[0], m[1], m[2], m[3]);
                *reinterpret_cast<uint4 *>(&most[warp][cg * 8 + 4]) = make_uint4(m[4], m[5], m[6], m[7]);
            }
            __syncthreads();
            // a column's scale by one thread, its factors to the others
            if (threadIdx.x < kTile) {
                uint32_t c = 0;
#pragma unroll
                for (int w = 0; w < kThreads / 32; ++w) c = max(c, most[w][threadIdx.x]);
                const BlockScale s = block_scale<kE5m2>(c);
                const int64_t col = tc * kTile + threadIdx.x;
                if (col < a.cols) ((float *)const_cast<void *>(a.scale_t.p))[col * a.scale_t.rs + tr * a.scale_t.cs] = s.scale;
                most[0][threadIdx.x] = __float_as_uint(s.factor);
                most[1][threadIdx.x] = __float_as_uint(s.rest);
            }
            __syncthreads();
        }
        // (pieces exchanged in pairs so that a warp's meet all banks)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float4 f = make_float4(tile_scale.factor, tile_scale.factor, tile_scale.factor, tile_scale.factor);
            float4 rest = make_float4(tile_scale.rest, tile_scale.rest, tile_scale.rest, tile_scale.rest);
            if (!a.whole) {
                f = *reinterpret_cast<const float4 *>(&most[0][cg * 8 + h * 4]);
                rest = *reinterpret_cast<const float4 *>(&most[1][cg * 8 + h * 4]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float q[2][kRows];
#pragma unroll
                for (int i = 0; i < kRows; ++i)
                    split(quotient(v.at(i, h * 2 + j), j ? pair(f.z, f.w) : pair(f.x, f.y), j ? pair(rest.z, rest.w) : pair(rest.x, rest.y)),
                          &q[0][i], &q[1][i]);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    turned[cg * 8 + h * 4 + j * 2 + k][rg ^ (cg * 2)] = pack_eight_bit<kE5m2>(q[k][0], q[k][1], q[k][2], q[k][3]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTile * 16 / kThreads; ++i) {
            const int col = i * (kThreads / 16) + rg;
            const uint2 b = *reinterpret_cast<const uint2 *>(&turned[col][(cg ^ (col >> 3)) * 2]);
            if (tc * kTile + col < a.cols)
                store8(a.qt, tc * kTile + col, tr * kTile + cg * 8, a.rows, a.qt_vec, b.x, b.y);
        }
    }
}

template <typename X, int kReads, bool kSlope>
bool launch(const QuantizeArgs &a, int64_t grid, bool e5m2, cudaStream_t s) {
    const dim3 g((unsigned)grid);
    if (a.qt.p)
        return e5m2 ? launch_behind(quantize_kernel<X, kReads, kSlope, true, true>, g, kThreads, 0, s, a)
                    : launch_behind(quantize_kernel<X, kReads, kSlope, false, true>, g, kThreads, 0, s, a);
    return e5m2 ? launch_behind(quantize_kernel<X, kReads, kSlope, true, false>, g, kThreads, 0, s, a)
                : launch_behind(quantize_kernel<X, kReads, kSlope, false, false>, g, kThreads, 0, s, a);
}

int reads_of(const MatRef &m) {
    if (vector_rows(m)) return kReadVectors;
    return m.cs == 1 && is_half_type(m.dtype) ? kReadShifted : kReadAny;
}

template <typename X>
bool launch_for(const QuantizeArgs &a, int64_t grid, bool e5m2, cudaStream_t s) {
    const int reads = reads_of(a.x);
    if constexpr (kIs16<X>) {
        if (reads == kReadShifted)
            return a.pre.p ? launch<X, kReadShifted, true>(a, grid, e5m2, s) : launch<X, kReadShifted, false>(a, grid, e5m2, s);
    }
    if (reads == kReadVectors)
        return a.pre.p ? launch<X, kReadVectors, true>(a, grid, e5m2, s) : launch<X, kReadVectors, false>(a, grid, e5m2, s);
    return a.pre.p ? launch<X, kReadAny, true>(a, grid, e5m2, s) : launch<X, kReadAny, false>(a, grid, e5m2, s);
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
    a.pre_reads = !preact ? kReadAny : is_half_type(preact->dtype) ? reads_of(a.pre) : kReadAny;
    auto end = [](const conv_matrix_desc *e, const void *p) {
        return e ? (const uint16_t *)((const char *)p + matrix_extent_bytes(e)) : nullptr;
    };
    a.x_end = end(x, x_dev), a.pre_end = end(preact, preact_dev);
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

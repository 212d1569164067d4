// linear.cu -- conv_linear and conv_linear_grad: argument checks, workspace
// layout, the packed copies of operands the product cannot read in place,
// and dz with the bias gradient.
#include <cuda_runtime.h>

#include <algorithm>

#include "channel.h"
#include "channel_launch.cuh"
#include "channel_math.cuh"
#include "tc_ptx.cuh"

namespace i8c {
namespace {

// ---------------------------------------------------------------- packing
// Copies of up to two matrices of 16-bit elements as lines of `len` elements
// `ld` apart (a multiple of 8, so that every line is 16-byte aligned; the
// padding is never read), in one launch.  A line is a row, or a column where
// columns have the smaller stride: the product takes either order, so nothing
// is transposed.  Lines whose elements are adjacent are read in aligned
// 16-byte vectors, a neighbour's half joined on by shifts; vectors that reach
// past the matrix are read by elements.
struct PackJob {
    const uint16_t *src;
    uint16_t *dst;
    int64_t line_stride, elem_stride, lines, len, ld;
    const uint16_t *end;  // of the matrix's elements
    int32_t pieces;       // pieces of 1024 elements per line
    int32_t blocks;       // eight pieces each
};
struct PackJobs {
    PackJob job[2];
    int count = 0;
};

template <int kWord>
__device__ __forceinline__ uint4 shifted(const uint4 &a, const uint4 &b, bool odd) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = odd ? __funnelshift_r(w[kWord + i], w[kWord + i + 1], 16) : w[kWord + i];
    return make_uint4(o[0], o[1], o[2], o[3]);
}

__global__ void __launch_bounds__(256) pack_matrix_kernel(const PackJobs jobs) {
    const bool second = (int)blockIdx.x >= jobs.job[0].blocks;
    const PackJob &j = jobs.job[second];
    const int64_t p = (int64_t)((int)blockIdx.x - (second ? jobs.job[0].blocks : 0)) * 8 + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    const int64_t line = p / j.pieces, c0 = (p - line * j.pieces) * 1024;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (line >= j.lines) return;
    const uint16_t *src = j.src + line * j.line_stride;
    uint16_t *dst = j.dst + line * j.ld;
    if (j.elem_stride > 1) {
#pragma unroll 8
        for (int i = 0; i < 32; ++i) {
            const int64_t c = c0 + i * 32 + lane;
            if (c < j.len) dst[c] = src[c * j.elem_stride];
        }
        return;
    }
    const int lead = (int)((uintptr_t)src / 2 & 7);  // elements past a 16-byte boundary, on the whole line
    const uint16_t *base = src - lead;
    uint4 q[4], last[4];
    bool whole[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t c = c0 + i * 256 + lane * 8;
        // (the vector at c, and beyond it the one at c + 8 unless lead is 0)
        const uint16_t *v = base + c;
        const bool mine = v >= j.src && v + 8 <= j.end, next = lead == 0 || v + 16 <= j.end;
        whole[i] = c < j.len && mine && next;
        q[i] = mine ? *reinterpret_cast<const uint4 *>(v) : make_uint4(0, 0, 0, 0);
        last[i] = lane == 31 && whole[i] && lead ? *reinterpret_cast<const uint4 *>(v + 8) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t c = c0 + i * 256 + lane * 8;
        uint4 n;
        n.x = __shfl_down_sync(0xffffffffu, q[i].x, 1);
        n.y = __shfl_down_sync(0xffffffffu, q[i].y, 1);
        n.z = __shfl_down_sync(0xffffffffu, q[i].z, 1);
        n.w = __shfl_down_sync(0xffffffffu, q[i].w, 1);
        if (lane == 31) n = last[i];
        if (whole[i]) {
            const bool odd = lead & 1;
            uint4 o;
            switch (lead >> 1) {  // the same for the whole warp
                case 0: o = shifted<0>(q[i], n, odd); break;
                case 1: o = shifted<1>(q[i], n, odd); break;
                case 2: o = shifted<2>(q[i], n, odd); break;
                default: o = shifted<3>(q[i], n, odd); break;
            }
            *reinterpret_cast<uint4 *>(dst + c) = o;
        } else {
            for (int e = 0; e < 8 && c + e < j.len; ++e) dst[c + e] = src[c + e];
        }
    }
}

conv_status run_packs(PackJobs &jobs, cudaStream_t s) {
    if (jobs.count == 0) return CONV_OK;
    const int64_t blocks = (int64_t)jobs.job[0].blocks + (jobs.count > 1 ? jobs.job[1].blocks : 0);
    if (blocks > INT32_MAX) return CONV_ERR_TOO_LARGE;
    return launch_behind(pack_matrix_kernel, dim3((unsigned)blocks), 256, 0, s, jobs) ? CONV_OK : CONV_ERR_CUDA;
}

struct Packed {  // a packed copy in the workspace, or none
    size_t off = 0, bytes = 0;
    int64_t ld = 0;
    bool by_rows = false;  // lines are rows, else columns
};

void plan_pack(const conv_matrix_desc *d, const void *p, size_t *total, Packed *k) {
    *k = Packed();
    if (d->rows == 0 || d->cols == 0 || product_in_place(p, d->rows, d->row_stride, d->cols, d->col_stride)) return;
    // along the smaller stride (a dim of extent 1 has none)
    k->by_rows = d->rows == 1 || (d->cols > 1 && d->col_stride <= d->row_stride);
    k->ld = round_up(k->by_rows ? d->cols : d->rows, 8);
    k->off = *total;
    k->bytes = (size_t)round_up((k->by_rows ? d->rows : d->cols) * k->ld * 2, 256);
    *total += k->bytes;
}

// Operand as the product reads it: in place, or its packed copy, which the
// jobs then have to make.
conv_status operand(const conv_matrix_desc *d, const void *p, const Packed &k, void *workspace, PackJobs *jobs,
                    MatRef *m) {
    *m = mat_ref(d, p);
    if (!k.bytes) return CONV_OK;
    PackJob &j = jobs->job[jobs->count++];
    j.src = (const uint16_t *)p;
    j.dst = (uint16_t *)((char *)workspace + k.off);
    j.lines = k.by_rows ? d->rows : d->cols;
    j.len = k.by_rows ? d->cols : d->rows;
    j.line_stride = k.by_rows ? m->rs : m->cs;
    j.elem_stride = k.by_rows ? m->cs : m->rs;
    j.ld = k.ld;
    j.end = j.src + matrix_extent_bytes(d) / 2;
    j.pieces = (int32_t)((j.len + 1023) / 1024);
    const int64_t blocks = (j.lines * j.pieces + 7) / 8;
    if (blocks > INT32_MAX / 2) return CONV_ERR_TOO_LARGE;
    j.blocks = (int32_t)blocks;
    m->p = j.dst;
    m->rs = d->rows > 1 ? (k.by_rows ? k.ld : 1) : 0;
    m->cs = d->cols > 1 ? (k.by_rows ? 1 : k.ld) : 0;
    return CONV_OK;
}

conv_status check_linear_params(const conv_linear_params *p, const conv_matrix_desc *x, bool has_bias) {
    if (!p) return CONV_ERR_NULL_PTR;
    if (p->activation < CONV_ACT_NONE || p->activation > CONV_ACT_SILU) return CONV_ERR_BAD_PARAM;
    if (p->reserved[0] != 0 || p->reserved[1] != 0) return CONV_ERR_BAD_PARAM;
    if (has_bias && p->bias_dtype != CONV_FLOAT32 && p->bias_dtype != x->dtype) return CONV_ERR_DTYPE;
    return CONV_OK;
}

conv_status check_operands(const conv_matrix_desc *x, const conv_matrix_desc *w) {
    conv_status st;
    if ((st = check_matrix(x)) || (st = check_matrix(w))) return st;
    if (!is_half_type(x->dtype) || w->dtype != x->dtype) return CONV_ERR_DTYPE;
    if (x->cols != w->cols) return CONV_ERR_SHAPE_MISMATCH;
    return CONV_OK;
}

conv_status check_like(const conv_matrix_desc *d, const void *p, int64_t rows, int64_t cols) {
    conv_status st = check_matrix(d);
    if (st) return st;
    if (d->rows != rows || d->cols != cols) return CONV_ERR_SHAPE_MISMATCH;
    return check_address(d, p);
}

conv_status check_vector(const void *p, int64_t n, int32_t dtype, const conv_matrix_desc *out, const void *out_dev) {
    if (!p || n == 0) return CONV_OK;
    if ((uintptr_t)p % (uintptr_t)channel_elem_size(dtype)) return CONV_ERR_ALIGNMENT;
    if (out && overlaps(p, (uint64_t)(n * channel_elem_size(dtype)), out_dev, matrix_extent_bytes(out)))
        return CONV_ERR_OVERLAP;
    return CONV_OK;
}

conv_status check_workspace(const void *workspace, size_t have, size_t need) {
    if (need == 0) return CONV_OK;
    if (!workspace || have < need || (uintptr_t)workspace % 256) return CONV_ERR_WORKSPACE;
    return CONV_OK;
}

struct LinearPlan {
    Packed x, w;
    size_t part_off = 0;  // partial sums of the product
    size_t bytes = 0;
};

LinearPlan plan_linear(const conv_matrix_desc *x, const void *x_dev, const conv_matrix_desc *w, const void *w_dev) {
    LinearPlan pl;
    plan_pack(x, x_dev, &pl.bytes, &pl.x);
    plan_pack(w, w_dev, &pl.bytes, &pl.w);
    pl.part_off = pl.bytes;
    if (x->rows > 0 && w->rows > 0) pl.bytes += product_plan(x->rows, w->rows, x->cols).part_bytes;
    return pl;
}

// ---------------------------------------------------------------- dz
// dz = dy * act'(preact) in 16 bits, and the column sums of the unrounded dz
// over this block's rows: 32 columns, a row per warp at a time.  One block to
// the column's rows writes dbias itself.
template <int kAct>
__global__ void __launch_bounds__(1024) linear_dz_kernel(MatRef dy, MatRef pre, int64_t rows, int64_t cols,
                                                        int64_t rows_per_block, void *dz, int64_t dz_ld,
                                                        float *part, void *dbias, int32_t bias_dtype) {
    __shared__ float red[32][32];
    const int x = threadIdx.x % 32, y = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + x;
    const int64_t r0 = (int64_t)blockIdx.y * rows_per_block;
    const int64_t r1 = r0 + rows_per_block < rows ? r0 + rows_per_block : rows;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    float sum = 0.0f;
    const int warps = blockDim.x / 32;
    if (c < cols) {
#pragma unroll 4
        for (int64_t r = r0 + y; r < r1; r += warps) {
            float v = load_as_float(dy.p, r * dy.rs + c * dy.cs, dy.dtype);
            if constexpr (kAct != CONV_ACT_NONE) {
                float slope = load_as_float(pre.p, r * pre.rs + c * pre.cs, pre.dtype), unused = 0.0f;
                activation_slope<kAct>(slope, unused);
                v *= slope;
            }
            if (dz) store_from_float(dz, r * dz_ld + c, dy.dtype, v);
            sum += v;
        }
    }
    if (!part && !dbias) return;
    red[y][x] = sum;
    __syncthreads();
    if (y == 0 && c < cols) {
        for (int i = 1; i < warps; ++i) sum += red[i][x];
        if (part) part[(int64_t)blockIdx.y * cols + c] = sum;
        else store_from_float(dbias, c, bias_dtype, sum);
    }
}

// Elements c .. c + 7 of a row, c = 8 lane + a multiple of 256, for a warp that
// is on one row: the aligned vector and the next lane's, joined by shifts.
// Vectors reach into the row's neighbours but not past the matrix, [lo, hi);
// where they would, the elements are read one by one (0 past cols).
__device__ __forceinline__ uint4 load8_shifted(const uint16_t *row, int64_t c, int64_t cols, const uint16_t *lo,
                                               const uint16_t *hi) {
    const int lane = threadIdx.x % 32, lead = (int)((uintptr_t)row / 2 & 7);
    const uint16_t *v = row - lead + c;
    const bool mine = v >= lo && v + 8 <= hi, whole = mine && (lead == 0 || v + 16 <= hi);
    const uint4 q = mine ? *reinterpret_cast<const uint4 *>(v) : make_uint4(0, 0, 0, 0);
    uint4 n;
    n.x = __shfl_down_sync(0xffffffffu, q.x, 1);
    n.y = __shfl_down_sync(0xffffffffu, q.y, 1);
    n.z = __shfl_down_sync(0xffffffffu, q.z, 1);
    n.w = __shfl_down_sync(0xffffffffu, q.w, 1);
    if (lane == 31 && whole && lead) n = *reinterpret_cast<const uint4 *>(v + 8);
    const bool odd = lead & 1;
    uint4 o;
    switch (lead >> 1) {  // the same for the whole warp
        case 0: o = shifted<0>(q, n, odd); break;
        case 1: o = shifted<1>(q, n, odd); break;
        case 2: o = shifted<2>(q, n, odd); break;
        default: o = shifted<3>(q, n, odd); break;
    }
    if (!whole) {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < cols) w[e / 2] |= (uint32_t)row[c + e] << (e % 2 * 16);
        o = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return o;
}

// The same for rows of adjacent elements: 32 x 8 threads of 8 columns each, a
// row per warp, several rows in flight.  kShift: rows of any alignment and
// length, else 16-byte aligned ones of a multiple of 8.  A stream (50176 x
// 1024 GELU: 55-58 us, 5.3-5.6 TB/s of dy, preact and dz); the slope's arithmetic
// takes about half the issue slots.
template <int kAct, bool kShift>
__global__ void __launch_bounds__(256, 3) linear_dz_rows_kernel(MatRef dy, MatRef pre, const uint16_t *dy_end,
                                                             const uint16_t *pre_end, int64_t rows, int64_t cols,
                                                             int64_t rows_per_block, void *dz, int64_t dz_ld,
                                                             float *part) {
    __shared__ float red[8][256];
    const int x = threadIdx.x % 32, y = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 256 + x * 8;
    const int64_t r0 = (int64_t)blockIdx.y * rows_per_block;
    const int64_t r1 = r0 + rows_per_block < rows ? r0 + rows_per_block : rows;
    const uint16_t *const g0 = (const uint16_t *)dy.p, *const z0 = (const uint16_t *)pre.p;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    float sum[8] = {};
    if (kShift || c < cols) {
        constexpr int kRows = kShift ? 2 : 4;
        for (int64_t r = r0 + y; r < r1; r += 8 * kRows) {
            uint4 g[kRows], z[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                if (r + 8 * i >= r1) break;  // (the whole warp)
                const uint16_t *gr = g0 + (r + 8 * i) * dy.rs, *zr = z0 + (r + 8 * i) * pre.rs;
                if constexpr (kShift) {
                    g[i] = load8_shifted(gr, c, cols, g0, dy_end);
                    if constexpr (kAct != CONV_ACT_NONE) z[i] = load8_shifted(zr, c, cols, z0, pre_end);
                } else {
                    g[i] = *reinterpret_cast<const uint4 *>(gr + c);
                    if constexpr (kAct != CONV_ACT_NONE) z[i] = *reinterpret_cast<const uint4 *>(zr + c);
                }
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                if (r + 8 * i >= r1) break;
                float v[8];
                unpack8(g[i], dy.dtype, v);
                if constexpr (kAct != CONV_ACT_NONE) {
                    float p[8];
                    unpack8(z[i], dy.dtype, p);
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        activation_slope<kAct>(p[j], p[j + 1]);
                        v[j] *= p[j];
                        v[j + 1] *= p[j + 1];
                    }
                }
                // (past the last column stand a neighbour's elements: their
                // sums are not written, their dz lies in the padding)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += v[j];
                if (dz && (!kShift || c < cols))
                    *reinterpret_cast<uint4 *>((uint16_t *)dz + (r + 8 * i) * dz_ld + c) = pack8(v, dy.dtype);
            }
        }
    }
    if (!part) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) red[y][x * 8 + j] = sum[j];
    __syncthreads();
    const int64_t mine = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (mine < cols) {
        float s = red[0][threadIdx.x];
        for (int i = 1; i < 8; ++i) s += red[i][threadIdx.x];
        part[(int64_t)blockIdx.y * cols + mine] = s;
    }
}

// Adds the blocks' partial sums: 32 columns per block, 32 threads per column.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *part, int64_t parts, int64_t cols, void *out,
                                                         int32_t dtype) {
    __shared__ float red[32][32];
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int64_t i = ty; i < parts; i += 32) s += part[i * cols + c];
    }
    red[ty][tx] = s;
    __syncthreads();
    if (ty || c >= cols) return;
    for (int i = 1; i < 32; ++i) s += red[i][tx];
    store_from_float(out, c, dtype, s);
}

struct GradPlan {
    bool dz = false;  // dz is made in the workspace
    size_t dz_off = 0, part_off = 0;  // part: column sums of dz
    size_t sums_off = 0;              // partial sums of the products, one after the other
    int64_t dz_ld = 0, parts = 0, rows_per_part = 0;
    Packed x, w;
    size_t bytes = 0;
};

GradPlan plan_grad(const conv_matrix_desc *dy, const void *dy_dev, const conv_matrix_desc *x, const void *x_dev,
                   const conv_matrix_desc *w, const void *w_dev, const conv_linear_params *p) {
    GradPlan pl;
    const int64_t m = dy->rows, n = dy->cols;
    if (m > 0 && n > 0) {
        pl.dz = p->activation != CONV_ACT_NONE ||
                !product_in_place(dy_dev, m, dy->row_stride, n, dy->col_stride);
        if (pl.dz) {
            pl.dz_ld = round_up(n, 8);
            pl.dz_off = pl.bytes;
            pl.bytes += (size_t)round_up(m * pl.dz_ld * 2, 256);
        }
        // two rounds of three blocks per SM, whichever kernel runs
        // (few rows: one block to a column, without a second kernel)
        const int64_t wanted = m <= 512 ? 1 : std::min<int64_t>(512, std::max<int64_t>(1, 912 / ((n + 255) / 256)));
        pl.rows_per_part = round_up((m + wanted - 1) / wanted, 8);
        pl.parts = (m + pl.rows_per_part - 1) / pl.rows_per_part;
        pl.part_off = pl.bytes;
        pl.bytes += (size_t)round_up(pl.parts * n * 4, 256);
    }
    plan_pack(x, x_dev, &pl.bytes, &pl.x);
    plan_pack(w, w_dev, &pl.bytes, &pl.w);
    pl.sums_off = pl.bytes;
    if (x->cols > 0) {
        size_t dx = 0, dw = 0;
        if (m > 0) dx = product_plan(m, x->cols, n).part_bytes;
        if (n > 0) dw = product_plan(n, x->cols, m).part_bytes;
        pl.bytes += std::max(dx, dw);
    }
    return pl;
}

template <int kAct>
bool launch_dz(const GradPlan &pl, const MatRef &dy, const MatRef &pre, int64_t m, int64_t n, void *ws, void *dbias,
               int32_t bias_dtype, cudaStream_t s) {
    void *dz = pl.dz ? (char *)ws + pl.dz_off : nullptr;
    float *part = dbias && pl.parts > 1 ? (float *)((char *)ws + pl.part_off) : nullptr;
    const dim3 wide((unsigned)((n + 255) / 256), (unsigned)pl.parts);
    auto end = [&](const MatRef &a) { return a.p ? (const uint16_t *)a.p + (m - 1) * a.rs + n : nullptr; };
    if (pl.parts > 1 && n % 8 == 0 && vector_rows(dy) && vector_rows(pre))
        return launch_behind(linear_dz_rows_kernel<kAct, false>, wide, 256, 0, s, dy, pre, end(dy), end(pre), m, n,
                             pl.rows_per_part, dz, pl.dz_ld, part);
    if (pl.parts > 1 && dy.cs == 1 && (!pre.p || pre.cs == 1))
        return launch_behind(linear_dz_rows_kernel<kAct, true>, wide, 256, 0, s, dy, pre, end(dy), end(pre), m, n,
                             pl.rows_per_part, dz, pl.dz_ld, part);
    return launch_behind(linear_dz_kernel<kAct>, dim3((unsigned)((n + 31) / 32), (unsigned)pl.parts),
                         pl.parts > 1 ? 256 : 1024, 0, s, dy, pre, m, n, pl.rows_per_part, dz, pl.dz_ld, part,
                         part ? nullptr : dbias, bias_dtype);
}

conv_status make_dz(const GradPlan &pl, int32_t act, const MatRef &dy, const MatRef &pre, int64_t m, int64_t n,
                    void *ws, void *dbias, int32_t bias_dtype, cudaStream_t s) {
    bool ok;
    switch (act) {
        case CONV_ACT_RELU: ok = launch_dz<CONV_ACT_RELU>(pl, dy, pre, m, n, ws, dbias, bias_dtype, s); break;
        case CONV_ACT_GELU: ok = launch_dz<CONV_ACT_GELU>(pl, dy, pre, m, n, ws, dbias, bias_dtype, s); break;
        case CONV_ACT_GELU_TANH: ok = launch_dz<CONV_ACT_GELU_TANH>(pl, dy, pre, m, n, ws, dbias, bias_dtype, s); break;
        case CONV_ACT_SILU: ok = launch_dz<CONV_ACT_SILU>(pl, dy, pre, m, n, ws, dbias, bias_dtype, s); break;
        default: ok = launch_dz<CONV_ACT_NONE>(pl, dy, pre, m, n, ws, dbias, bias_dtype, s); break;
    }
    if (ok && dbias && pl.parts > 1)
        ok = launch_behind(column_sum_kernel, dim3((unsigned)((n + 31) / 32)), 1024, 0, s,
                           (const float *)((char *)ws + pl.part_off), pl.parts, n, dbias, bias_dtype);
    return ok ? CONV_OK : CONV_ERR_CUDA;
}

}  // namespace
}  // namespace i8c

using namespace i8c;

extern "C" {

conv_status conv_linear_workspace_size(const conv_matrix_desc *x, const void *x_dev, const conv_matrix_desc *w,
                                       const void *w_dev, size_t *bytes) {
    if (!x || !w || !bytes) return CONV_ERR_NULL_PTR;
    conv_status st = check_operands(x, w);
    if (st) return st;
    *bytes = plan_linear(x, x_dev, w, w_dev).bytes;
    return CONV_OK;
}

conv_status conv_linear(const conv_matrix_desc *x, const void *x_dev, const conv_matrix_desc *w, const void *w_dev,
                        const void *bias_dev, const conv_matrix_desc *residual, const void *residual_dev,
                        const conv_matrix_desc *preact, void *preact_dev, const conv_matrix_desc *y, void *y_dev,
                        const conv_linear_params *p, void *workspace, size_t workspace_bytes, void *stream) {
    if (!x || !w || !y || !p) return CONV_ERR_NULL_PTR;
    conv_status st;
    if ((st = check_operands(x, w)) || (st = check_linear_params(p, x, bias_dev != nullptr))) return st;
    const int64_t m = x->rows, n = w->rows, k = x->cols;
    if ((st = check_like(y, y_dev, m, n))) return st;
    if (y->dtype != x->dtype && y->dtype != CONV_FLOAT32) return CONV_ERR_DTYPE;
    if ((st = check_address(x, x_dev)) || (st = check_address(w, w_dev))) return st;
    if (residual) {
        if ((st = check_like(residual, residual_dev, m, n))) return st;
        if (residual->dtype != y->dtype) return CONV_ERR_DTYPE;
    }
    if (preact) {
        if ((st = check_like(preact, preact_dev, m, n))) return st;
        if (preact->dtype != x->dtype) return CONV_ERR_DTYPE;
    }
    if ((st = check_vector(bias_dev, n, p->bias_dtype, y, y_dev))) return st;
    if (preact && (st = check_vector(bias_dev, n, p->bias_dtype, preact, preact_dev))) return st;
    if (m == 0 || n == 0) return CONV_OK;
    if (matrices_overlap(y, y_dev, x, x_dev) || matrices_overlap(y, y_dev, w, w_dev) ||
        (residual && !same_matrix(y, y_dev, residual, residual_dev) &&
         matrices_overlap(y, y_dev, residual, residual_dev)) ||
        (preact && (matrices_overlap(preact, preact_dev, x, x_dev) || matrices_overlap(preact, preact_dev, w, w_dev) ||
                    matrices_overlap(preact, preact_dev, y, y_dev) ||
                    (residual && matrices_overlap(preact, preact_dev, residual, residual_dev)))))
        return CONV_ERR_OVERLAP;
    const LinearPlan pl = plan_linear(x, x_dev, w, w_dev);
    if ((st = check_workspace(workspace, workspace_bytes, pl.bytes))) return st;
    if (pl.bytes) {
        const conv_matrix_desc *d[] = {x, w, y, residual, preact};
        const void *a[] = {x_dev, w_dev, y_dev, residual_dev, preact_dev};
        for (int i = 0; i < 5; ++i)
            if (d[i] && overlaps(workspace, pl.bytes, a[i], matrix_extent_bytes(d[i]))) return CONV_ERR_OVERLAP;
        if (bias_dev && overlaps(workspace, pl.bytes, bias_dev, (uint64_t)(n * channel_elem_size(p->bias_dtype))))
            return CONV_ERR_OVERLAP;
    }
    if ((st = check_device())) return st;
    MatRef xr, wr;
    PackJobs jobs;
    if ((st = operand(x, x_dev, pl.x, workspace, &jobs, &xr)) || (st = operand(w, w_dev, pl.w, workspace, &jobs, &wr)) ||
        (st = run_packs(jobs, (cudaStream_t)stream)))
        return st;
    Product pr;
    pr.ma = m, pr.nb = n, pr.k = k;
    pr.a = {xr.p, xr.rs, xr.cs};
    pr.b = {wr.p, wr.rs, wr.cs};
    pr.in_dtype = x->dtype;
    const MatRef yr = mat_ref(y, y_dev), rr = mat_ref(residual, residual_dev), zr = mat_ref(preact, preact_dev);
    pr.d = y_dev, pr.d_sa = yr.rs, pr.d_sb = yr.cs, pr.d_dtype = y->dtype;
    pr.res = residual ? residual_dev : nullptr, pr.res_sa = rr.rs, pr.res_sb = rr.cs;
    pr.pre = preact ? preact_dev : nullptr, pr.pre_sa = zr.rs, pr.pre_sb = zr.cs;
    pr.bias = bias_dev, pr.bias_dtype = p->bias_dtype;
    pr.act = p->activation;
    return product_launch(pr, (char *)workspace + pl.part_off, stream);
}

conv_status conv_linear_grad_workspace_size(const conv_matrix_desc *dy, const void *dy_dev,
                                            const conv_matrix_desc *x, const void *x_dev, const conv_matrix_desc *w,
                                            const void *w_dev, const conv_linear_params *p, size_t *bytes) {
    if (!dy || !x || !w || !p || !bytes) return CONV_ERR_NULL_PTR;
    conv_status st;
    if ((st = check_operands(x, w)) || (st = check_linear_params(p, x, false)) || (st = check_matrix(dy))) return st;
    if (dy->dtype != x->dtype) return CONV_ERR_DTYPE;
    if (dy->rows != x->rows || dy->cols != w->rows) return CONV_ERR_SHAPE_MISMATCH;
    *bytes = plan_grad(dy, dy_dev, x, x_dev, w, w_dev, p).bytes;
    return CONV_OK;
}

conv_status conv_linear_grad(const conv_matrix_desc *dy, const void *dy_dev, const conv_matrix_desc *x,
                             const void *x_dev, const conv_matrix_desc *w, const void *w_dev,
                             const conv_matrix_desc *preact, const void *preact_dev, const conv_matrix_desc *dx,
                             void *dx_dev, const conv_matrix_desc *dw, void *dw_dev, void *dbias_dev,
                             const conv_linear_params *p, void *workspace, size_t workspace_bytes, void *stream) {
    if (!dy || !x || !w || !p || (!dx && !dw && !dbias_dev)) return CONV_ERR_NULL_PTR;
    conv_status st;
    if ((st = check_operands(x, w)) || (st = check_linear_params(p, x, dbias_dev != nullptr))) return st;
    const int64_t m = x->rows, n = w->rows, k = x->cols;
    if ((st = check_like(dy, dy_dev, m, n))) return st;
    if (dy->dtype != x->dtype) return CONV_ERR_DTYPE;
    if ((st = check_address(x, x_dev)) || (st = check_address(w, w_dev))) return st;
    if (p->activation == CONV_ACT_NONE) preact = nullptr;
    else if (!preact) return CONV_ERR_NULL_PTR;
    if (preact) {
        if ((st = check_like(preact, preact_dev, m, n))) return st;
        if (preact->dtype != x->dtype) return CONV_ERR_DTYPE;
    }
    if (dx) {
        if ((st = check_like(dx, dx_dev, m, k))) return st;
        if (dx->dtype != x->dtype && dx->dtype != CONV_FLOAT32) return CONV_ERR_DTYPE;
    }
    if (dw) {
        if ((st = check_like(dw, dw_dev, n, k))) return st;
        if (dw->dtype != x->dtype && dw->dtype != CONV_FLOAT32) return CONV_ERR_DTYPE;
    }
    const conv_matrix_desc *in[] = {dy, x, w, preact};
    const void *in_dev[] = {dy_dev, x_dev, w_dev, preact_dev};
    for (int i = 0; i < 4; ++i) {
        if (!in[i]) continue;
        if (dx && matrices_overlap(dx, dx_dev, in[i], in_dev[i])) return CONV_ERR_OVERLAP;
        if (dw && matrices_overlap(dw, dw_dev, in[i], in_dev[i])) return CONV_ERR_OVERLAP;
        if ((st = check_vector(dbias_dev, n, p->bias_dtype, in[i], in_dev[i]))) return st;
    }
    if (dx && dw && matrices_overlap(dx, dx_dev, dw, dw_dev)) return CONV_ERR_OVERLAP;
    if (dx && (st = check_vector(dbias_dev, n, p->bias_dtype, dx, dx_dev))) return st;
    if (dw && (st = check_vector(dbias_dev, n, p->bias_dtype, dw, dw_dev))) return st;
    const GradPlan pl = plan_grad(dy, dy_dev, x, x_dev, w, w_dev, p);
    if ((st = check_workspace(workspace, workspace_bytes, pl.bytes))) return st;
    if (pl.bytes) {
        const conv_matrix_desc *d[] = {dy, x, w, preact, dx, dw};
        const void *a[] = {dy_dev, x_dev, w_dev, preact_dev, dx_dev, dw_dev};
        for (int i = 0; i < 6; ++i)
            if (d[i] && overlaps(workspace, pl.bytes, a[i], matrix_extent_bytes(d[i]))) return CONV_ERR_OVERLAP;
        if (dbias_dev && overlaps(workspace, pl.bytes, dbias_dev, (uint64_t)(n * channel_elem_size(p->bias_dtype))))
            return CONV_ERR_OVERLAP;
    }
    if ((st = check_device())) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    MatRef dz = mat_ref(dy, dy_dev);
    if (m > 0 && n > 0 && (pl.dz || dbias_dev)) {
        if ((st = make_dz(pl, p->activation, dz, mat_ref(preact, preact_dev), m, n, workspace, dbias_dev,
                          p->bias_dtype, s)))
            return st;
        if (pl.dz) {
            dz.p = (char *)workspace + pl.dz_off;
            dz.rs = m > 1 ? pl.dz_ld : 0;
            dz.cs = n > 1 ? 1 : 0;
        }
    } else if (m == 0 && n > 0 && dbias_dev) {
        if (cudaMemsetAsync(dbias_dev, 0, (size_t)(n * channel_elem_size(p->bias_dtype)), s) != cudaSuccess)
            return CONV_ERR_CUDA;
    }
    MatRef xr, wr;
    PackJobs jobs;
    const bool want_dx = dx && m > 0 && k > 0, want_dw = dw && n > 0 && k > 0;
    if ((want_dx && (st = operand(w, w_dev, pl.w, workspace, &jobs, &wr))) ||
        (want_dw && (st = operand(x, x_dev, pl.x, workspace, &jobs, &xr))) || (st = run_packs(jobs, s)))
        return st;
    if (want_dx) {
        Product pr;
        pr.ma = m, pr.nb = k, pr.k = n;
        pr.a = {dz.p, dz.rs, dz.cs};
        pr.b = {wr.p, wr.cs, wr.rs};
        // dx waits for dz, not for the sum of its columns
        pr.beside_previous = m > 0 && n > 0 && dbias_dev && pl.parts > 1 && jobs.count == 0;
        pr.in_dtype = x->dtype;
        const MatRef o = mat_ref(dx, dx_dev);
        pr.d = dx_dev, pr.d_sa = o.rs, pr.d_sb = o.cs, pr.d_dtype = dx->dtype;
        if ((st = product_launch(pr, (char *)workspace + pl.sums_off, stream))) return st;
    }
    if (want_dw) {
        Product pr;
        pr.ma = n, pr.nb = k, pr.k = m;
        pr.a = {dz.p, dz.cs, dz.rs};
        pr.b = {xr.p, xr.cs, xr.rs};
        // dw does not wait for dx (unless dx's joining kernel still reads the
        // partial sums' workspace)
        pr.beside_previous = want_dx && product_plan(m, k, n).parts == 1;
        pr.in_dtype = x->dtype;
        const MatRef o = mat_ref(dw, dw_dev);
        pr.d = dw_dev, pr.d_sa = o.rs, pr.d_sb = o.cs, pr.d_dtype = dw->dtype;
        if ((st = product_launch(pr, (char *)workspace + pl.sums_off, stream))) return st;
    }
    return CONV_OK;
}

}  // extern "C"

// linear_fp8.cu -- conv_linear_fp8: argument checks, the packed copies of
// operands whose rows are not aligned, and which product takes the call.
#include <cuda_runtime.h>

#include <algorithm>

#include "channel.h"
#include "channel_launch.cuh"
#include "tc_ptx.cuh"

namespace i8c {
namespace {

// Rows of `len` bytes, `rs` apart, to rows of `ld` bytes (a multiple of 16;
// what lies behind a row's end is not read): 16 bytes per thread, from aligned
// words joined by shifts where those lie inside the matrix.
struct PackRows {
    const uint8_t *src, *end;
    uint8_t *dst;
    int64_t rows, len, rs, ld;
};
__global__ void __launch_bounds__(256) pack_rows_kernel(const PackRows a, const PackRows b) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const PackRows &j = blockIdx.y ? b : a;
    const int64_t pieces = j.ld / 16;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < j.rows * pieces; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / pieces, c = (i - r * pieces) * 16;
        const uint8_t *p = j.src + r * j.rs + c;
        const int off = (int)((uintptr_t)p & 3);
        const uint8_t *q = p - off;
        uint32_t w[5] = {};
        if (q >= j.src && q + 20 <= j.end) {
#pragma unroll
            for (int k = 0; k < 5; ++k) w[k] = reinterpret_cast<const uint32_t *>(q)[k];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 8 * off);
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (c + k < j.len) w[k / 4] |= (uint32_t)p[k] << (k % 4 * 8);
        }
        *reinterpret_cast<uint4 *>(j.dst + r * j.ld + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

bool in_place(const conv_matrix_desc *d, const void *p) {
    return (uintptr_t)p % 16 == 0 && (d->rows <= 1 || d->row_stride % 16 == 0);
}

struct Plan {
    size_t x_off = 0, w_off = 0, part_off = 0, bytes = 0;
    bool pack_x = false, pack_w = false;
};
Plan plan_of(const conv_matrix_desc *x, const void *x_dev, const conv_matrix_desc *w, const void *w_dev) {
    Plan pl;
    if (x->rows == 0 || w->rows == 0 || x->cols == 0) return pl;
    pl.pack_x = !in_place(x, x_dev), pl.pack_w = !in_place(w, w_dev);
    if (pl.pack_x) pl.x_off = pl.bytes, pl.bytes += (size_t)round_up(x->rows * round_up(x->cols, 16), 256);
    if (pl.pack_w) pl.w_off = pl.bytes, pl.bytes += (size_t)round_up(w->rows * round_up(w->cols, 16), 256);
    pl.part_off = pl.bytes;
    if (!scaled_rows_applies(x->rows, w->rows, x->cols)) pl.bytes += scaled_plan(x->rows, w->rows, x->cols).part_bytes;
    return pl;
}

conv_status check_operand(const conv_matrix_desc *d) {
    conv_status st = check_matrix(d);
    if (st) return st;
    if (!is_eight_bit_type(d->dtype)) return CONV_ERR_DTYPE;
    if (d->rows > 0 && d->cols > 1 && d->col_stride != 1) return CONV_ERR_BAD_STRIDES;
    return CONV_OK;
}

conv_status check_scale(const conv_matrix_desc *s, const void *p, const conv_matrix_desc *of, int32_t *shift) {
    conv_status st = check_matrix(s);
    if (st) return st;
    if (s->dtype != CONV_FLOAT32) return CONV_ERR_DTYPE;
    const int64_t squares = (of->rows + kScaleBlock - 1) / kScaleBlock;
    if (s->cols != (of->cols + kScaleBlock - 1) / kScaleBlock || (s->rows != of->rows && s->rows != squares))
        return CONV_ERR_SHAPE_MISMATCH;
    *shift = s->rows == of->rows ? 0 : 7;
    return check_address(s, p);
}

conv_status check_result(const conv_matrix_desc *d, const void *p, int64_t rows, int64_t cols) {
    conv_status st = check_matrix(d);
    if (st) return st;
    if (d->rows != rows || d->cols != cols) return CONV_ERR_SHAPE_MISMATCH;
    return check_address(d, p);
}

}  // namespace
}  // namespace i8c

using namespace i8c;

extern "C" {

conv_status conv_linear_fp8_workspace_size(const conv_matrix_desc *x, const void *x_dev, const conv_matrix_desc *w,
                                           const void *w_dev, size_t *bytes) {
    if (!x || !w || !bytes) return CONV_ERR_NULL_PTR;
    conv_status st;
    if ((st = check_operand(x)) || (st = check_operand(w))) return st;
    if (x->cols != w->cols) return CONV_ERR_SHAPE_MISMATCH;
    *bytes = plan_of(x, x_dev, w, w_dev).bytes;
    return CONV_OK;
}

conv_status conv_linear_fp8(const conv_matrix_desc *x, const void *x_dev, const conv_matrix_desc *x_scale,
                            const void *x_scale_dev, const conv_matrix_desc *w, const void *w_dev,
                            const conv_matrix_desc *w_scale, const void *w_scale_dev, const void *bias_dev,
                            const conv_matrix_desc *residual, const void *residual_dev,
                            const conv_matrix_desc *preact, void *preact_dev, const conv_matrix_desc *y, void *y_dev,
                            const conv_linear_params *p, void *workspace, size_t workspace_bytes, void *stream) {
    if (!x || !x_scale || !w || !w_scale || !y || !p) return CONV_ERR_NULL_PTR;
    conv_status st;
    ScaledProduct pr;
    if ((st = check_operand(x)) || (st = check_operand(w))) return st;
    if (x->cols != w->cols) return CONV_ERR_SHAPE_MISMATCH;
    if ((st = check_scale(x_scale, x_scale_dev, x, &pr.a.shift)) || (st = check_scale(w_scale, w_scale_dev, w, &pr.b.shift)) ||
        (st = check_address(x, x_dev)) || (st = check_address(w, w_dev)))
        return st;
    const int64_t m = x->rows, n = w->rows;
    if (p->activation < CONV_ACT_NONE || p->activation > CONV_ACT_SILU || p->reserved[0] != 0 || p->reserved[1] != 0)
        return CONV_ERR_BAD_PARAM;
    if ((st = check_result(y, y_dev, m, n))) return st;
    if (!is_float_type(y->dtype)) return CONV_ERR_DTYPE;
    if (residual) {
        if ((st = check_result(residual, residual_dev, m, n))) return st;
        if (residual->dtype != y->dtype) return CONV_ERR_DTYPE;
    }
    if (preact) {
        if ((st = check_result(preact, preact_dev, m, n))) return st;
        if (!is_half_type(preact->dtype)) return CONV_ERR_DTYPE;
    }
    uint64_t bias_bytes = 0;
    if (bias_dev) {
        if (p->bias_dtype != CONV_FLOAT32 && p->bias_dtype != y->dtype) return CONV_ERR_DTYPE;
        if ((uintptr_t)bias_dev % (uintptr_t)channel_elem_size(p->bias_dtype)) return CONV_ERR_ALIGNMENT;
        bias_bytes = (uint64_t)(n * channel_elem_size(p->bias_dtype));
    }
    if (m == 0 || n == 0) return CONV_OK;
    const Plan pl = plan_of(x, x_dev, w, w_dev);
    const conv_matrix_desc *d[] = {x, x_scale, w, w_scale, residual, preact, y};
    const void *at[] = {x_dev, x_scale_dev, w_dev, w_scale_dev, residual_dev, preact_dev, y_dev};
    for (int i = 5; i < 7; ++i) {
        if (!d[i]) continue;
        for (int j = 0; j < i; ++j)
            if (d[j] && !(i == 6 && j == 4 && same_matrix(y, y_dev, residual, residual_dev)) &&
                matrices_overlap(d[i], at[i], d[j], at[j]))
                return CONV_ERR_OVERLAP;
        if (overlaps(bias_dev, bias_bytes, at[i], matrix_extent_bytes(d[i]))) return CONV_ERR_OVERLAP;
    }
    if (pl.bytes) {
        if (!workspace || workspace_bytes < pl.bytes || (uintptr_t)workspace % 256) return CONV_ERR_WORKSPACE;
        for (int i = 0; i < 7; ++i)
            if (d[i] && overlaps(workspace, pl.bytes, at[i], matrix_extent_bytes(d[i]))) return CONV_ERR_OVERLAP;
        if (overlaps(workspace, pl.bytes, bias_dev, bias_bytes)) return CONV_ERR_OVERLAP;
    }
    if ((st = check_device())) return st;
    auto operand = [&](const conv_matrix_desc *e, const void *e_dev, const conv_matrix_desc *s, const void *s_dev, bool packed,
                       size_t off, ScaledOperand *o) {
        const MatRef r = mat_ref(e, e_dev), sr = mat_ref(s, s_dev);
        o->p = packed ? (const uint8_t *)workspace + off : (const uint8_t *)r.p;
        o->rs = e->rows <= 1 ? 0 : packed ? round_up(e->cols, 16) : r.rs;
        o->scale = (const float *)sr.p, o->s_rs = sr.rs, o->s_cs = sr.cs;
        o->e5m2 = e->dtype == CONV_FLOAT8_E5M2;
        return PackRows{(const uint8_t *)r.p, (const uint8_t *)r.p + matrix_extent_bytes(e), (uint8_t *)workspace + off,
                        packed ? e->rows : 0, e->cols, r.rs, round_up(e->cols, 16)};
    };
    const PackRows px = operand(x, x_dev, x_scale, x_scale_dev, pl.pack_x, pl.x_off, &pr.a);
    const PackRows pw = operand(w, w_dev, w_scale, w_scale_dev, pl.pack_w, pl.w_off, &pr.b);
    if (pl.pack_x || pl.pack_w) {
        const int64_t pieces = std::max(px.rows, pw.rows) * (px.ld / 16);
        const dim3 grid((unsigned)std::min<int64_t>((pieces + 255) / 256, 4096), 2);
        if (!launch_behind(pack_rows_kernel, grid, 256, 0, (cudaStream_t)stream, px, pw)) return CONV_ERR_CUDA;
    }
    pr.ma = m, pr.nb = n, pr.k = x->cols;
    const MatRef yr = mat_ref(y, y_dev), rr = mat_ref(residual, residual_dev), zr = mat_ref(preact, preact_dev);
    pr.d = y_dev, pr.d_sa = yr.rs, pr.d_sb = yr.cs, pr.d_dtype = y->dtype;
    pr.res = residual ? residual_dev : nullptr, pr.res_sa = rr.rs, pr.res_sb = rr.cs;
    pr.pre = preact ? preact_dev : nullptr, pr.pre_sa = zr.rs, pr.pre_sb = zr.cs, pr.pre_dtype = zr.dtype;
    pr.bias = bias_dev, pr.bias_dtype = p->bias_dtype;
    pr.act = p->activation;
    if (scaled_rows_applies(m, n, pr.k)) return scaled_rows_launch(pr, stream);
    return scaled_launch(pr, (char *)workspace + pl.part_off, stream);
}

}  // extern "C"

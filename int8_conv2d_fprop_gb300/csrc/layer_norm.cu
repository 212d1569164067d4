// layer_norm.cu -- conv_layer_norm and conv_layer_norm_grad.
#include <cuda_runtime.h>

#include <cmath>

#include "channel.h"
#include "channel_math.cuh"

namespace i8c {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the block, the same value in every thread.
__device__ __forceinline__ float block_sum(float v, float *red) {
    v = warp_sum(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    float t = red[0];
    for (int i = 1; i < kThreads / 32; ++i) t += red[i];
    return t;
}

__global__ void __launch_bounds__(kThreads) layer_norm_kernel(MatRef x, const void *gain, const void *shift,
                                                              MatRef y, float *mean_out, float *rstd_out, int64_t cols,
                                                              float eps, float scale, int32_t param_dtype) {
    __shared__ float red[kThreads / 32];
    const int64_t r = blockIdx.x;
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += kThreads) s += scale * load_as_float(x.p, r * x.rs + c * x.cs, x.dtype);
    const float mean = block_sum(s, red) / (float)cols;
    s = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
        const float d = scale * load_as_float(x.p, r * x.rs + c * x.cs, x.dtype) - mean;
        s += d * d;
    }
    const float rstd = rsqrtf(block_sum(s, red) / (float)cols + eps);
    for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
        const float d = scale * load_as_float(x.p, r * x.rs + c * x.cs, x.dtype) - mean;
        const float g = gain ? load_as_float(gain, c, param_dtype) : 1.0f;
        const float b = shift ? load_as_float(shift, c, param_dtype) : 0.0f;
        store_from_float((void *)y.p, r * y.rs + c * y.cs, y.dtype, d * rstd * g + b);
    }
    if (threadIdx.x == 0) {
        if (mean_out) mean_out[r] = mean;
        if (rstd_out) rstd_out[r] = rstd;
    }
}

__global__ void __launch_bounds__(kThreads) layer_norm_dx_kernel(MatRef dy, MatRef x, const void *gain,
                                                                 const float *mean, const float *rstd, MatRef res,
                                                                 MatRef dx, int64_t cols, int32_t param_dtype) {
    __shared__ float red[kThreads / 32];
    const int64_t r = blockIdx.x;
    const float mu = mean[r], rs = rstd[r];
    float st = 0.0f, stn = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
        const float n = (load_as_float(x.p, r * x.rs + c * x.cs, x.dtype) - mu) * rs;
        const float t = load_as_float(dy.p, r * dy.rs + c * dy.cs, dy.dtype) *
                        (gain ? load_as_float(gain, c, param_dtype) : 1.0f);
        st += t;
        stn += t * n;
    }
    st = block_sum(st, red) / (float)cols;
    stn = block_sum(stn, red) / (float)cols;
    for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
        const float n = (load_as_float(x.p, r * x.rs + c * x.cs, x.dtype) - mu) * rs;
        const float t = load_as_float(dy.p, r * dy.rs + c * dy.cs, dy.dtype) *
                        (gain ? load_as_float(gain, c, param_dtype) : 1.0f);
        float d = rs * (t - st - n * stn);
        if (res.p) d += load_as_float(res.p, r * res.rs + c * res.cs, res.dtype);
        store_from_float((void *)dx.p, r * dx.rs + c * dx.cs, dx.dtype, d);
    }
}

// Column sums of dy * n and dy over this block's rows: 32 columns, 8 rows at
// a time.
__global__ void __launch_bounds__(kThreads) layer_norm_params_kernel(MatRef dy, MatRef x, const float *mean,
                                                                     const float *rstd, int64_t rows, int64_t cols,
                                                                     int64_t rows_per_block, float *part) {
    __shared__ float red[2][8][32];
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;
    const int64_t r0 = (int64_t)blockIdx.y * rows_per_block;
    const int64_t r1 = r0 + rows_per_block < rows ? r0 + rows_per_block : rows;
    float sg = 0.0f, sb = 0.0f;
    if (c < cols)
        for (int64_t r = r0 + ty; r < r1; r += 8) {
            const float d = load_as_float(dy.p, r * dy.rs + c * dy.cs, dy.dtype);
            sg += d * ((load_as_float(x.p, r * x.rs + c * x.cs, x.dtype) - mean[r]) * rstd[r]);
            sb += d;
        }
    red[0][ty][tx] = sg;
    red[1][ty][tx] = sb;
    __syncthreads();
    if (ty == 0 && c < cols) {
        for (int i = 1; i < 8; ++i) {
            sg += red[0][i][tx];
            sb += red[1][i][tx];
        }
        float *p = part + (int64_t)blockIdx.y * 2 * cols;
        p[c] = sg;
        p[cols + c] = sb;
    }
}

__global__ void __launch_bounds__(kThreads) layer_norm_params_sum_kernel(const float *part, int64_t parts,
                                                                         int64_t cols, void *dgain, void *dshift,
                                                                         int32_t dtype) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= 2 * cols) return;
    void *out = c < cols ? dgain : dshift;
    if (!out) return;
    float s = 0.0f;
    for (int64_t i = 0; i < parts; ++i) s += part[i * 2 * cols + c];
    store_from_float(out, c < cols ? c : c - cols, dtype, s);
}

bool is_float_type(int32_t t) { return t == CONV_FLOAT32 || is_half_type(t); }

conv_status check_norm_params(const conv_layer_norm_params *p, int32_t out_dtype) {
    if (p->reserved != 0 || !(p->eps > 0.0f) || !std::isfinite(p->eps) || !std::isfinite(p->scale) || p->scale == 0.0f)
        return CONV_ERR_BAD_PARAM;
    if (p->param_dtype != CONV_FLOAT32 && p->param_dtype != out_dtype) return CONV_ERR_DTYPE;
    return CONV_OK;
}

// A vector the call reads or writes: aligned to its element, and apart from
// the matrix `m`.
conv_status check_vector(const void *p, int64_t n, int64_t size, const conv_matrix_desc *m, const void *m_dev) {
    if (!p || n == 0) return CONV_OK;
    if ((uintptr_t)p % (uintptr_t)size) return CONV_ERR_ALIGNMENT;
    if (m && overlaps(p, (uint64_t)(n * size), m_dev, matrix_extent_bytes(m))) return CONV_ERR_OVERLAP;
    return CONV_OK;
}

struct NormGradPlan {
    int64_t parts = 0, rows_per_part = 0;
    size_t bytes = 0;
};

NormGradPlan plan_norm_grad(int64_t rows, int64_t cols) {
    NormGradPlan pl;
    if (rows == 0 || cols == 0) return pl;
    pl.rows_per_part = round_up((rows + 255) / 256, 8);
    pl.parts = (rows + pl.rows_per_part - 1) / pl.rows_per_part;
    pl.bytes = (size_t)round_up(pl.parts * 2 * cols * 4, 256);
    return pl;
}

}  // namespace
}  // namespace i8c

using namespace i8c;

extern "C" {

conv_status conv_layer_norm(const conv_matrix_desc *x, const void *x_dev, const void *gain_dev,
                            const void *shift_dev, const conv_matrix_desc *y, void *y_dev, float *mean_dev,
                            float *rstd_dev, const conv_layer_norm_params *p, void *stream) {
    if (!x || !y || !p) return CONV_ERR_NULL_PTR;
    conv_status st;
    if ((st = check_matrix(x)) || (st = check_matrix(y))) return st;
    if ((x->dtype != CONV_INT32 && !is_float_type(x->dtype)) || !is_float_type(y->dtype)) return CONV_ERR_DTYPE;
    if ((st = check_norm_params(p, y->dtype))) return st;
    if (x->rows != y->rows || x->cols != y->cols) return CONV_ERR_SHAPE_MISMATCH;
    if (x->cols < 1) return CONV_ERR_BAD_PARAM;
    if ((st = check_address(x, x_dev)) || (st = check_address(y, y_dev))) return st;
    const int64_t rows = x->rows, cols = x->cols, psize = channel_elem_size(p->param_dtype);
    if ((st = check_vector(gain_dev, cols, psize, y, y_dev)) || (st = check_vector(shift_dev, cols, psize, y, y_dev)))
        return st;
    float *stats[] = {mean_dev, rstd_dev};
    for (float *v : stats) {
        if ((st = check_vector(v, rows, 4, x, x_dev)) || (st = check_vector(v, rows, 4, y, y_dev))) return st;
        if (v && (overlaps(v, rows * 4, gain_dev, cols * psize) || overlaps(v, rows * 4, shift_dev, cols * psize)))
            return CONV_ERR_OVERLAP;
    }
    if (overlaps(mean_dev, rows * 4, rstd_dev, rows * 4)) return CONV_ERR_OVERLAP;
    if (matrices_overlap(x, x_dev, y, y_dev) &&
        !(same_matrix(x, x_dev, y, y_dev) && channel_elem_size(x->dtype) == channel_elem_size(y->dtype)))
        return CONV_ERR_OVERLAP;
    if (rows == 0) return CONV_OK;
    if ((st = check_device())) return st;
    layer_norm_kernel<<<(unsigned)rows, kThreads, 0, (cudaStream_t)stream>>>(
        mat_ref(x, x_dev), gain_dev, shift_dev, mat_ref(y, y_dev), mean_dev, rstd_dev, cols, p->eps, p->scale,
        p->param_dtype);
    return cudaGetLastError() == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

conv_status conv_layer_norm_grad_workspace_size(const conv_matrix_desc *x, size_t *bytes) {
    if (!x || !bytes) return CONV_ERR_NULL_PTR;
    conv_status st = check_matrix(x);
    if (st) return st;
    if (!is_float_type(x->dtype)) return CONV_ERR_DTYPE;
    if (x->cols < 1) return CONV_ERR_BAD_PARAM;
    *bytes = plan_norm_grad(x->rows, x->cols).bytes;
    return CONV_OK;
}

conv_status conv_layer_norm_grad(const conv_matrix_desc *dy, const void *dy_dev, const conv_matrix_desc *x,
                                 const void *x_dev, const void *gain_dev, const float *mean_dev,
                                 const float *rstd_dev, const conv_matrix_desc *residual_grad,
                                 const void *residual_grad_dev, const conv_matrix_desc *dx, void *dx_dev,
                                 void *dgain_dev, void *dshift_dev, const conv_layer_norm_params *p, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    if (!dy || !x || !p || (!dx && !dgain_dev && !dshift_dev)) return CONV_ERR_NULL_PTR;
    conv_status st;
    const conv_matrix_desc *all[] = {dy, x, residual_grad, dx};
    const void *all_dev[] = {dy_dev, x_dev, residual_grad_dev, dx_dev};
    for (int i = 0; i < 4; ++i) {
        if (!all[i]) continue;
        if ((st = check_matrix(all[i]))) return st;
        if (!is_float_type(all[i]->dtype) || all[i]->dtype != x->dtype) return CONV_ERR_DTYPE;
        if (all[i]->rows != x->rows || all[i]->cols != x->cols) return CONV_ERR_SHAPE_MISMATCH;
    }
    if ((st = check_norm_params(p, x->dtype))) return st;
    if (p->scale != 1.0f || x->cols < 1) return CONV_ERR_BAD_PARAM;
    for (int i = 0; i < 4; ++i)
        if (all[i] && (st = check_address(all[i], all_dev[i]))) return st;
    const int64_t rows = x->rows, cols = x->cols, psize = channel_elem_size(p->param_dtype);
    if (rows > 0 && (!mean_dev || !rstd_dev)) return CONV_ERR_NULL_PTR;
    if ((st = check_vector(mean_dev, rows, 4, dx, dx_dev)) || (st = check_vector(rstd_dev, rows, 4, dx, dx_dev)) ||
        (st = check_vector(gain_dev, cols, psize, dx, dx_dev)))
        return st;
    void *grads[] = {dgain_dev, dshift_dev};
    for (void *g : grads) {
        for (int i = 0; i < 4; ++i)
            if (all[i] && (st = check_vector(g, cols, psize, all[i], all_dev[i]))) return st;
        if (g && (overlaps(g, cols * psize, mean_dev, rows * 4) || overlaps(g, cols * psize, rstd_dev, rows * 4) ||
                  overlaps(g, cols * psize, gain_dev, cols * psize)))
            return CONV_ERR_OVERLAP;
    }
    if (overlaps(dgain_dev, cols * psize, dshift_dev, cols * psize)) return CONV_ERR_OVERLAP;
    if (dx && (matrices_overlap(dx, dx_dev, x, x_dev) || matrices_overlap(dx, dx_dev, dy, dy_dev) ||
               (residual_grad && matrices_overlap(dx, dx_dev, residual_grad, residual_grad_dev) &&
                !same_matrix(dx, dx_dev, residual_grad, residual_grad_dev))))
        return CONV_ERR_OVERLAP;
    const NormGradPlan pl = plan_norm_grad(rows, cols);
    if (pl.bytes) {
        if (!workspace || workspace_bytes < pl.bytes || (uintptr_t)workspace % 256) return CONV_ERR_WORKSPACE;
        for (int i = 0; i < 4; ++i)
            if (all[i] && overlaps(workspace, pl.bytes, all_dev[i], matrix_extent_bytes(all[i])))
                return CONV_ERR_OVERLAP;
        const void *vec[] = {gain_dev, dgain_dev, dshift_dev, mean_dev, rstd_dev};
        for (int i = 0; i < 5; ++i)
            if (overlaps(workspace, pl.bytes, vec[i], i < 3 ? cols * psize : rows * 4)) return CONV_ERR_OVERLAP;
    }
    if ((st = check_device())) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    if (rows == 0) {
        for (void *g : grads)
            if (g && cudaMemsetAsync(g, 0, (size_t)(cols * psize), s) != cudaSuccess) return CONV_ERR_CUDA;
        return CONV_OK;
    }
    const MatRef dyr = mat_ref(dy, dy_dev), xr = mat_ref(x, x_dev);
    if (dx)
        layer_norm_dx_kernel<<<(unsigned)rows, kThreads, 0, s>>>(
            dyr, xr, gain_dev, mean_dev, rstd_dev, mat_ref(residual_grad, residual_grad_dev), mat_ref(dx, dx_dev),
            cols, p->param_dtype);
    if (dgain_dev || dshift_dev) {
        const dim3 grid((unsigned)((cols + 31) / 32), (unsigned)pl.parts);
        layer_norm_params_kernel<<<grid, kThreads, 0, s>>>(dyr, xr, mean_dev, rstd_dev, rows, cols, pl.rows_per_part,
                                                           (float *)workspace);
        layer_norm_params_sum_kernel<<<(unsigned)((2 * cols + kThreads - 1) / kThreads), kThreads, 0, s>>>(
            (const float *)workspace, pl.parts, cols, dgain_dev, dshift_dev, p->param_dtype);
    }
    return cudaGetLastError() == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

}  // extern "C"

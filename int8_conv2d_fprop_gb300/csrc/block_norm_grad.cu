// block_norm_grad.cu -- conv_block_norm_grad: the kernel for any strides, the
// joining of the workers' shares, argument checks and launches.
#include <cuda_runtime.h>

#include <algorithm>

#include "block_norm_grad.cuh"

namespace i8c {

bool launch_block_norm_grad_f32(const BlockNormGradArgs &a, const Held &h, int64_t grid, size_t smem, cudaStream_t s) {
    return launch_backward<float, float>(a, h, grid, smem, s);
}

namespace {

// Any strides, types and widths: a block per row, held in shared memory; every
// thread adds to its own columns of the block's shares.
__global__ void __launch_bounds__(kAnyThreads) block_norm_grad_any_kernel(const BlockNormGradArgs a) {
    __shared__ __align__(16) BlockSums sums;
    Summer block_sum{&sums};
    extern __shared__ __align__(16) float shared[];
    float *const dhs = shared, *const vs = shared + a.cols;
    const float per = 1.0f / (float)a.cols;
    const int64_t worker = blockIdx.x, first = worker * a.per_worker, end = min(a.rows, first + a.per_worker);
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (first >= end) return;
    float *const dg = a.part_gain ? a.part_gain + worker * a.part_cols : nullptr;
    float *const dp = a.part_post ? a.part_post + worker * a.part_cols : nullptr;
    float *const sv = a.part_post || a.dgate.p ? a.scratch + worker * a.part_cols : nullptr;  // S of the gate
    for (int c = threadIdx.x; c < a.cols; c += kAnyThreads) {
        if (dg) dg[c] = 0.0f;
        if (dp) dp[c] = 0.0f;
        if (sv) sv[c] = 0.0f;
    }
    for (int64_t r = first; r < end; ++r) {
        const int64_t which = r / a.rows_per_gate, gate = which * a.gate.rs;
        const float rs = a.dy.p ? a.rstd[r] : 0.0f, rx = a.post ? a.post_rstd[r] : 1.0f;
        float s = 0.0f;
        if (a.dy.p) {
            for (int c = threadIdx.x; c < a.cols; c += kAnyThreads) {
                const float d = load_as_float(a.dy.p, r * a.dy.rs + c * a.dy.cs, a.dy.dtype);
                const float w = load_as_float(a.h.p, r * a.h.rs + c * a.h.cs, a.h.dtype) * rs;
                const float t = d * (a.gain ? load_as_float(a.gain, c, a.param_dtype) : 1.0f);
                dhs[c] = t;
                vs[c] = w;
                s = fmaf(t, w, s);
                if (dg) dg[c] += d * w;
            }
            s = block_sum(s) * per;
        }
        float s2 = 0.0f;
        for (int c = threadIdx.x; c < a.cols; c += kAnyThreads) {
            float dh = a.dy.p ? rs * (dhs[c] - vs[c] * s) : 0.0f;
            if (a.dsum.p) dh += load_as_float(a.dsum.p, r * a.dsum.rs + c * a.dsum.cs, a.dsum.dtype);
            if (a.dskip.p)
                store_from_float(const_cast<void *>(a.dskip.p), r * a.dskip.rs + c * a.dskip.cs, a.dskip.dtype, a.skip_scale * dh);
            float dn = dh * a.branch_scale;
            if (a.gate.p) dn *= load_as_float(a.gate.p, gate + c * a.gate.cs, a.gate.dtype);
            if (a.post && a.post_gain) dn *= load_as_float(a.post_gain, c, a.param_dtype);
            if (a.x.p) {
                const float v = load_as_float(a.x.p, r * a.x.rs + c * a.x.cs, a.x.dtype) * rx;
                vs[c] = v;
                s2 = fmaf(dn, v, s2);
                if (sv) sv[c] += dh * v;
            }
            dhs[c] = dn;
        }
        if (a.dx.p) {
            s2 = a.post ? block_sum(s2) * per : 0.0f;
            for (int c = threadIdx.x; c < a.cols; c += kAnyThreads)
                store_from_float(const_cast<void *>(a.dx.p), r * a.dx.rs + c * a.dx.cs, a.dx.dtype,
                                 a.post ? rx * (dhs[c] - vs[c] * s2) : dhs[c]);
        }
        if (!sv || (r + 1 < end && r + 1 < (which + 1) * a.rows_per_gate)) continue;
        for (int c = threadIdx.x; c < a.cols; c += kAnyThreads) {
            const float t = sv[c];
            sv[c] = 0.0f;
            const float b = a.branch_scale * t;
            if (dp) dp[c] += b * (a.gate.p ? load_as_float(a.gate.p, gate + c * a.gate.cs, a.gate.dtype) : 1.0f);
            if (a.part_gate) a.part_gate[(worker + which) * a.part_cols + c] = t;
            else if (a.dgate.p)
                store_from_float(const_cast<void *>(a.dgate.p), which * a.dgate.rs + c * a.dgate.cs, a.dgate.dtype,
                                 b * (a.post && a.post_gain ? load_as_float(a.post_gain, c, a.param_dtype) : 1.0f));
        }
    }
}

// Adds the shares.  blockIdx.y 0: dgain, 1: dpost_gain, of the blocks (8
// columns and 64 lines at a time, 20 loads of a thread in flight: one round
// covers them), 2 + i: dgate of gates 16 i to 16 i + 15 of the workers, a warp
// each on 32 columns.  The shares of worker w (of a block, where it is one)
// start at (lead + w lead_step) mod 8.
struct BlockNormJoin {
    const float *part_gain, *part_post, *part_gate;
    MatRef dgate;
    const void *post_gain;
    void *dgain, *dpost_gain;
    int64_t gates, rows_per_gate, per_worker;
    int32_t blocks, warps, workers, cols, part_cols, lead, lead_step, param_dtype, post;
    float branch_scale;
};
__global__ void __launch_bounds__(512) block_norm_join_kernel(const BlockNormJoin a) {
    __shared__ float red[16][8];
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (blockIdx.y >= 2) {
        const int64_t g = ((int64_t)blockIdx.y - 2) * 16 + threadIdx.x / 32;
        const int c = blockIdx.x * 32 + threadIdx.x % 32;
        if (g >= a.gates || c >= a.cols) return;
        // the workers whose stretches meet the gate's rows
        const int lo = a.per_worker ? (int)(g * a.rows_per_gate / a.per_worker) : 0;
        const int hi = a.per_worker ? (int)(((g + 1) * a.rows_per_gate - 1) / a.per_worker) : a.workers - 1;
        const float *p = a.part_gate + g * a.part_cols + c;
        float s = 0.0f;
#pragma unroll 1
        for (int w0 = lo; w0 <= hi; w0 += 20) {
            float v[20];
#pragma unroll
            for (int u = 0; u < 20; ++u)
                v[u] = w0 + u <= hi ? p[(int64_t)(w0 + u) * a.part_cols + ((a.lead + (w0 + u) * a.lead_step) & 7)] : 0.0f;
#pragma unroll
            for (int u = 0; u < 20; ++u) s += v[u];
        }
        s *= a.branch_scale;
        if (a.post && a.post_gain) s *= load_as_float(a.post_gain, c, a.param_dtype);
        store_from_float(const_cast<void *>(a.dgate.p), g * a.dgate.rs + c * a.dgate.cs, a.dgate.dtype, s);
        return;
    }
    void *out = blockIdx.y ? a.dpost_gain : a.dgain;
    if (!out) return;
    const int tx = threadIdx.x % 8, ty = threadIdx.x / 8;
    const int c = blockIdx.x * 8 + tx;
    const float *p = (blockIdx.y ? a.part_post : a.part_gain) + c;
    const int lead = a.warps ? 0 : a.lead, lead_step = a.warps ? 0 : a.lead_step;
    float s = 0.0f;
    if (c < a.cols) {
#pragma unroll 1
        for (int w0 = ty; w0 < a.blocks; w0 += 64 * 20) {
            float v[20];
#pragma unroll
            for (int u = 0; u < 20; ++u) {
                const int w = w0 + 64 * u;
                v[u] = w < a.blocks ? p[(int64_t)w * a.part_cols + ((lead + w * lead_step) & 7)] : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < 20; ++u) s += v[u];
        }
    }
    s += __shfl_xor_sync(0xffffffffu, s, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    if (threadIdx.x % 32 < 8) red[threadIdx.x / 32][tx] = s;
    __syncthreads();
    if (ty || c >= a.cols) return;
    s = red[0][tx];
#pragma unroll
    for (int i = 1; i < 16; ++i) s += red[i][tx];
    store_from_float(out, c, a.param_dtype, s);
}

__global__ void __launch_bounds__(256) zero_matrix_kernel(MatRef m, int64_t rows, int64_t cols) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int64_t c = threadIdx.x; c < cols; c += 256) store_from_float(const_cast<void *>(m.p), r * m.rs + c * m.cs, m.dtype, 0.0f);
}

// Rows on their way, and the shared memory with them (two blocks to an SM where
// a warp holds a row).
size_t grad_smem(const BlockNormGradArgs &a, const Held &h, bool aligned, int64_t ts, int64_t ss, int *stages) {
    const uint32_t t_slot = row_slot_bytes(a.cols, (uint32_t)ts), s_slot = row_slot_bytes(a.cols, (uint32_t)ss);
    const uint32_t stage = (a.dy.p ? t_slot + s_slot : 0) + (a.dsum.p ? s_slot : 0) + (a.x.p ? t_slot : 0);
    const int workers = h.warp ? 8 : 1;
    auto space = [&](int n) {
        return row_space(workers, n, stage, kept_sets(aligned, h.warp, 2), h.warp ? 32 : h.threads, h.nv).total;
    };
    *stages = stages_for(space(0), workers * stage, std::min(16, 512 / h.threads));
    // (at the end the warps' shares lie over all of it)
    return std::max<size_t>(space(*stages), h.warp ? (size_t)a.cols * 64 : 0);
}

// (room for a lead and for whole groups)
int64_t part_columns(int64_t cols) { return round_up(cols, 8) + 8; }

// Workers there are at most, whatever the device: 8 warps of two blocks on each
// SM of the part this library is for, or eight blocks of 64 threads, or four.
int64_t most_workers(int64_t rows, int64_t cols) {
    return std::min<int64_t>(rows, cols <= 512 ? 16 * 152 : 4 * 152);
}

// Lines of shares: each worker's of dgain and of dpost_gain, S's slots (the
// gates of stretches are at most as many as the workers), and a scratch line
// for each block.
size_t block_norm_grad_bytes(int64_t rows, int64_t cols) {
    if (rows == 0) return 0;
    return (size_t)round_up(5 * most_workers(rows, cols) * part_columns(cols) * 4, 256);
}

}  // namespace
}  // namespace i8c

using namespace i8c;

extern "C" {

conv_status conv_block_norm_grad_workspace_size(const conv_matrix_desc *x, int64_t groups, size_t *bytes) {
    if (!x || !bytes) return CONV_ERR_NULL_PTR;
    conv_status st = check_matrix(x);
    if (st) return st;
    if (!is_float_type(x->dtype)) return CONV_ERR_DTYPE;
    if (x->cols < 1 || groups < 0) return CONV_ERR_BAD_PARAM;
    if (groups == 0 ? x->rows != 0 : x->rows % groups != 0) return CONV_ERR_SHAPE_MISMATCH;
    if (x->cols > kMostGradColumns) return CONV_ERR_TOO_LARGE;
    *bytes = block_norm_grad_bytes(x->rows, x->cols);
    return CONV_OK;
}

conv_status conv_block_norm_grad(const conv_matrix_desc *dy, const void *dy_dev, const conv_matrix_desc *dsum,
                                 const void *dsum_dev, const conv_matrix_desc *x, const void *x_dev,
                                 const conv_matrix_desc *sum, const void *sum_dev, const conv_matrix_desc *gate,
                                 const void *gate_dev, const void *post_gain_dev, const void *gain_dev,
                                 const float *post_rstd_dev, const float *rstd_dev, const conv_matrix_desc *dx,
                                 void *dx_dev, const conv_matrix_desc *dskip, void *dskip_dev,
                                 const conv_matrix_desc *dgate, void *dgate_dev, void *dpost_gain_dev,
                                 void *dgain_dev, const conv_block_norm_params *p, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    if (!p || (!dy && !dsum) || (!dx && !dskip && !dgate && !dpost_gain_dev && !dgain_dev)) return CONV_ERR_NULL_PTR;
    if (p->post_norm != 1) post_gain_dev = nullptr, post_rstd_dev = nullptr;
    // what the wanted gradients need
    const bool need_x = p->post_norm == 1 ? dx || dgate || dpost_gain_dev : dgate != nullptr;
    if ((dpost_gain_dev && p->post_norm != 1) || (dgain_dev && !dy)) return CONV_ERR_BAD_PARAM;
    if ((need_x && !x) || (dy && !sum)) return CONV_ERR_NULL_PTR;
    const conv_matrix_desc *like = dy ? dy : dsum;
    const int64_t rows = like->rows, cols = like->cols, psize = channel_elem_size(p->param_dtype);
    const conv_matrix_desc *all[] = {dy, dsum, x, sum, dx, dskip};
    const void *all_dev[] = {dy_dev, dsum_dev, x_dev, sum_dev, dx_dev, dskip_dev};
    conv_status st;
    int32_t x_type = 0, s_type = 0;
    for (int i = 0; i < 6; ++i) {
        if (!all[i]) continue;
        if ((st = check_matrix(all[i]))) return st;
        if (!is_float_type(all[i]->dtype)) return CONV_ERR_DTYPE;
        int32_t &type = i == 0 || i == 2 || i == 4 ? x_type : s_type;
        if (type && type != all[i]->dtype) return CONV_ERR_DTYPE;
        type = all[i]->dtype;
        if (all[i]->rows != rows || all[i]->cols != cols) return CONV_ERR_SHAPE_MISMATCH;
    }
    if (!x_type) x_type = s_type;
    if (!s_type) s_type = x_type;
    if (!stream_type(s_type, x_type)) return CONV_ERR_DTYPE;
    if ((st = check_block_params(p, x_type))) return st;
    if (cols < 1) return CONV_ERR_BAD_PARAM;
    if (cols > kMostGradColumns) return CONV_ERR_TOO_LARGE;
    for (int i = 0; i < 6; ++i)
        if (all[i] && (st = check_address(all[i], all_dev[i]))) return st;
    if ((st = check_gate(gate, gate_dev, rows, cols, x_type)) || (st = check_gate(dgate, dgate_dev, rows, cols, x_type))) return st;
    if (gate && dgate && gate->rows != dgate->rows) return CONV_ERR_SHAPE_MISMATCH;
    if (!dy) gain_dev = nullptr, rstd_dev = nullptr, sum = nullptr;
    if (!need_x) x = nullptr;
    if (rows > 0 && ((dy && !rstd_dev) || (need_x && p->post_norm && !post_rstd_dev))) return CONV_ERR_NULL_PTR;
    if (!need_x) post_rstd_dev = nullptr;
    const void *vectors[] = {post_gain_dev, gain_dev, dpost_gain_dev, dgain_dev};
    for (const void *v : vectors)
        if ((uintptr_t)v % psize) return CONV_ERR_ALIGNMENT;
    if ((uintptr_t)post_rstd_dev % 4 || (uintptr_t)rstd_dev % 4) return CONV_ERR_ALIGNMENT;
    const Buffer in[] = {matrix_of(dy, dy_dev), matrix_of(dsum, dsum_dev), matrix_of(x, x_dev), matrix_of(sum, sum_dev),
                         matrix_of(gate, gate_dev), vector_of(post_gain_dev, cols * psize), vector_of(gain_dev, cols * psize),
                         vector_of(post_rstd_dev, rows * 4), vector_of(rstd_dev, rows * 4)};
    const size_t need = block_norm_grad_bytes(rows, cols);
    const Buffer out[] = {matrix_of(dx, dx_dev), matrix_of(dskip, dskip_dev), matrix_of(dgate, dgate_dev),
                          vector_of(dpost_gain_dev, cols * psize), vector_of(dgain_dev, cols * psize),
                          vector_of(workspace, (int64_t)need)};
    if (need && (!workspace || workspace_bytes < need || (uintptr_t)workspace % 256)) return CONV_ERR_WORKSPACE;
    for (int i = 0; i < 6; ++i) {
        for (int j = 0; j < 9; ++j) {
            const bool same = (i == 0 && j == 0 && dx && dy && same_matrix(dx, dx_dev, dy, dy_dev)) ||
                              (i == 1 && j == 1 && dskip && dsum && same_matrix(dskip, dskip_dev, dsum, dsum_dev));
            if (!same && share(out[i], in[j])) return CONV_ERR_OVERLAP;
        }
        for (int j = 0; j < i; ++j)
            if (share(out[i], out[j])) return CONV_ERR_OVERLAP;
    }
    if ((st = check_device())) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    if (rows == 0) {
        for (void *g : {dpost_gain_dev, dgain_dev})
            if (g && cudaMemsetAsync(g, 0, (size_t)(cols * psize), s) != cudaSuccess) return CONV_ERR_CUDA;
        if (dgate && dgate->rows > 0 &&
            !launch_behind(zero_matrix_kernel, dim3((unsigned)std::min<int64_t>(dgate->rows, 65536)), 256, 0, s,
                           mat_ref(dgate, dgate_dev), dgate->rows, cols))
            return CONV_ERR_CUDA;
        return CONV_OK;
    }
    BlockNormGradArgs a;
    a.dy = mat_ref(dy, dy_dev), a.dsum = mat_ref(dsum, dsum_dev), a.x = mat_ref(x, x_dev), a.h = mat_ref(sum, sum_dev);
    a.gate = mat_ref(gate, gate_dev), a.dx = mat_ref(dx, dx_dev), a.dskip = mat_ref(dskip, dskip_dev);
    a.dgate = mat_ref(dgate, dgate_dev);
    a.post_gain = post_gain_dev, a.gain = gain_dev, a.post_rstd = post_rstd_dev, a.rstd = rstd_dev;
    a.rows = rows, a.cols = (int32_t)cols, a.part_cols = (int32_t)part_columns(cols);
    a.gates = gate ? gate->rows : dgate ? dgate->rows : 1;
    a.rows_per_gate = rows / a.gates;
    a.skip_scale = p->skip_scale, a.branch_scale = p->branch_scale;
    a.param_dtype = p->param_dtype, a.post = p->post_norm && x;
    const MatRef &ref = dy ? a.dy : a.dsum;
    const bool one = one_lead({&ref, &a.dsum, &a.x, &a.h});
    a.shift_dx = dx && !one_lead({&ref, &a.dx});
    a.shift_dskip = dskip && !one_lead({&ref, &a.dskip});
    const bool unit = unit_columns(a.dy) && unit_columns(a.dsum) && unit_columns(a.x) && unit_columns(a.h) &&
                      unit_columns(a.dx) && unit_columns(a.dskip) && unit_columns(a.gate) && unit_columns(a.dgate);
    const bool aligned = aligned_rows(ref);
    a.wait_limit_ns = wait_limit_ns(), a.status = device_status_word();
    if (!a.status) return CONV_ERR_CUDA;
    // (gates' gradients leave in aligned groups, whole gates' in even rows)
    Held h = unit && one && ((aligned && aligned_rows(a.dgate)) || a.gates == 1)
                 ? held(cols, aligned, cols % 8 == 0 && aligned && aligned_rows(a.dx) && aligned_rows(a.dskip) && aligned_rows(a.dgate))
                 : Held();
    const int64_t ts = channel_elem_size(x_type), ss = channel_elem_size(s_type);
    size_t smem = 0;
    int64_t most = 0;
    if (h.nv) {
        smem = grad_smem(a, h, aligned, ts, ss, &a.stages);
        most = std::min(workers_at_once(h, 512, smem), most_workers(rows, cols));
        if (smem > 216 << 10 || (!h.even && a.gates > most)) h = Held();
    }
    if (!h.nv) {
        smem = (size_t)cols * 8;
        most = device_sm_count() * std::max<int64_t>(1, std::min<int64_t>(4, (int64_t)((224 << 10) / (smem + 2048))));
        most = std::min(most, most_workers(rows, cols));
    }
    const int64_t per_block = h.warp ? 8 : 1;
    int64_t workers;
    a.whole = a.gates > most;
    if (h.nv && !aligned) {
        // (one gate: steps of a multiple of 8, so that a worker's rows share their lead, or a row each)
        workers = rows <= most ? rows : std::max<int64_t>(8, most / per_block / 8 * 8 * per_block);
        if (h.warp && rows > most) workers = std::max<int64_t>(8, most / 64 * 64);
        a.per_worker = 0;
    } else {
        a.per_worker = a.whole ? stretch_of(a.gates, most) * a.rows_per_gate : stretch_of(rows, most);
        workers = (rows + a.per_worker - 1) / a.per_worker;
    }
    const int64_t grid = (workers + per_block - 1) / per_block;
    const int64_t lines = most_workers(rows, cols);
    a.part_gain = dgain_dev ? (float *)workspace : nullptr;
    a.part_post = dpost_gain_dev ? (float *)workspace + lines * a.part_cols : nullptr;
    a.part_gate = dgate && !a.whole ? (float *)workspace + 2 * lines * a.part_cols : nullptr;
    a.scratch = (float *)workspace + 4 * lines * a.part_cols;
    bool ok;
    if (h.nv)
        ok = x_type == CONV_FLOAT32   ? launch_block_norm_grad_f32(a, h, grid, smem, s)
             : x_type == CONV_FLOAT16 ? launch_block_norm_grad_f16(a, h, s_type == CONV_FLOAT32, grid, smem, s)
                                      : launch_block_norm_grad_bf16(a, h, s_type == CONV_FLOAT32, grid, smem, s);
    else
        ok = launch_large<block_norm_grad_any_kernel>(dim3((unsigned)grid), kAnyThreads, smem, s, a);
    const bool gates_left = dgate && !a.whole;
    if (ok && (dgain_dev || dpost_gain_dev || gates_left)) {
        BlockNormJoin j;
        j.part_gain = a.part_gain, j.part_post = a.part_post, j.part_gate = a.part_gate;
        j.dgate = a.dgate, j.post_gain = post_gain_dev;
        j.dgain = dgain_dev, j.dpost_gain = dpost_gain_dev;
        j.gates = a.gates, j.rows_per_gate = a.rows_per_gate, j.per_worker = a.per_worker;
        j.blocks = (int32_t)grid, j.warps = h.warp, j.workers = (int32_t)workers, j.cols = a.cols, j.part_cols = a.part_cols;
        const Lead lead = h.nv && !aligned ? lead_of_rows(ref) : Lead{0, 0};
        j.lead = (int32_t)lead.base, j.lead_step = (int32_t)lead.step;
        j.param_dtype = p->param_dtype, j.post = a.post, j.branch_scale = p->branch_scale;
        ok = launch_behind(block_norm_join_kernel, dim3((unsigned)((cols + 7) / 8), (unsigned)(2 + (gates_left ? (a.gates + 15) / 16 : 0))),
                           512, 0, s, j);
    }
    return ok ? CONV_OK : CONV_ERR_CUDA;
}

}  // extern "C"

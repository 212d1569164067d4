// block_norm.cu -- conv_block_norm: the norm behind a residual block, its gate,
// the residual sum and the norm before the next block, as one pass over the
// rows.
//
// A stream.  A row is held in the registers of a worker: a warp (up to 512
// columns where all rows are of whole aligned groups of 8, else up to 256 of
// aligned rows and 249 of others) or a block (up to 8192, of unaligned rows
// 8185).  Its matrices come in by bulk copies, one for each row and matrix, one
// to three rows ahead as shared memory allows: that takes an instruction of a
// lane where asynchronous copies took two of every thread.  Wider rows, and some
// widths below whose rows and parameters do not fit shared memory beside each
// other, go an element at a time.  The sums of squares run over registers, and every output is
// written once.  A worker takes a stretch of rows, so that it reads its gates
// once each.  50176 x 512 bf16 with 64 gates: 40.6 us (5.1 TB/s).
#include <cuda_runtime.h>

#include <algorithm>

#include "block_norm.cuh"

namespace i8c {
namespace {

struct BlockNormArgs {
    MatRef x, skip, gate, sum, y, y_scale;
    const void *post_gain, *gain;
    float *post_rstd, *rstd;
    int64_t rows, rows_per_gate;
    int32_t cols;
    float eps, skip_scale, branch_scale;
    int32_t param_dtype;
    int32_t post;
    int32_t shift_sum, shift_y;  // rows of another lead than x's
    int64_t per_worker;        // rows of a worker's stretch; 0: rows that begin anywhere, in steps
    int32_t stages;
    uint64_t wait_limit_ns;
    int *status;
};

// ---------------------------------------------------------------- forward
// kEven: all matrices in aligned rows of whole groups.
template <typename T, typename S, int kNv, bool kWarp, bool kEven>
__global__ void __launch_bounds__(kWarp ? 256 : 512, kWarp ? 3 : kNv == 1 ? 2 : 1)
    block_norm_rows_kernel(const BlockNormArgs a) {
    __shared__ __align__(16) float sums[2][32];
    RowSummer block_sum{sums};
    extern __shared__ __align__(128) uint8_t smem[];
    const int local = kWarp ? threadIdx.x / 32 : 0, workers = kWarp ? 8 : 1;
    const int64_t worker = (int64_t)blockIdx.x * workers + local;
    const bool skip = a.skip.p;
    Stretch rows;
    rows.first = a.per_worker ? worker * a.per_worker : worker;
    rows.end = a.per_worker ? min(a.rows, rows.first + a.per_worker) : a.rows;
    rows.step = a.per_worker ? 1 : (int64_t)gridDim.x * workers;
    S *sum = (S *)const_cast<void *>(a.sum.p) + (a.sum.p ? rows.first * a.sum.rs : 0);
    T *y = (T *)const_cast<void *>(a.y.p) + (a.y.p && !a.y_scale.p ? rows.first * a.y.rs : 0);
    Place<true> at;
    at.t = kWarp ? threadIdx.x % 32 : threadIdx.x;
    at.threads = kWarp ? 32 : blockDim.x;
    at.cols = a.cols;
    at.lead = kEven ? 0 : lead_of((const T *)a.x.p + rows.first * a.x.rs);
    const float per = 1.0f / (float)a.cols;
    const uint32_t x_slot = row_slot_bytes(a.cols, sizeof(T)), stage_bytes = x_slot + (skip ? row_slot_bytes(a.cols, sizeof(S)) : 0);
    // (the gains are every worker's own where rows begin anywhere, the gate always)
    const int own = a.per_worker ? 0 : local, first_gate = a.per_worker ? 2 : 2 * workers;
    const RowSpace space = row_space(workers, a.stages, stage_bytes, first_gate + workers, at.threads, kNv);
    const uint32_t base = ptx::smem_addr(smem), bars = base + local * 8 * kMostStages, ring = base + space.rows + local * a.stages * stage_bytes;
    const uint32_t set = kNv * 32 * at.threads, stride = at.threads * 16, kept = base + space.kept + at.t * 16;
    const Kept post_gain{kept + 2 * own * set, stride}, gain{kept + (2 * own + 1) * set, stride}, gate{kept + (first_gate + local) * set, stride};
    RowFeed feed;
    feed.on = false;
    if (at.t == 0) feed.set(a.x, a.rows, a.cols, sizeof(T), 0, rows.first, rows.step);
    if (at.t == 1 && skip) feed.set(a.skip, a.rows, a.cols, sizeof(S), x_slot, rows.first, rows.step);
    if (at.t == 0) {
        for (int i = 0; i < a.stages; ++i) ptx::mbar_init(bars + 8 * i, skip ? 2 : 1);
        ptx::fence_mbar_init();
    }
    row_sync<kWarp>();
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    RowWait wait{a.wait_limit_ns, a.status};
    int64_t to_fill = rows.first;  // the row that is fetched next
    auto fill = [&](int stage) {
        if (feed.on && to_fill < rows.end) feed.fill<kEven>(ring + stage * stage_bytes, bars + 8 * stage);
        to_fill += rows.step;
    };
    for (int d = 0; d < a.stages; ++d) fill(d);
    if (!a.per_worker || local == 0) {
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            float g[8];
            load_params(a.post_gain, a.param_dtype, 1.0f, at, i, g);
            post_gain.keep(i, g);
            load_params(a.gain, a.param_dtype, 1.0f, at, i, g);
            gain.keep(i, g);
        }
    }
    __syncthreads();
    const Pair skip_scale = pair(a.skip_scale);
    int64_t gate_end = rows.first;  // the row from which on another gate is wanted
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t r = rows.first; r < rows.end; r += rows.step) {
        if (r >= gate_end) {
            const int64_t which = r / a.rows_per_gate;
            gate_end = (which + 1) * a.rows_per_gate;
#pragma unroll
            for (int i = 0; i < kNv; ++i) keep_gate(gate, a.gate, which, post_gain, a.post, a.branch_scale, at, i);
        }
        const uint32_t slot = ring + stage * stage_bytes;
        wait(bars + 8 * stage, phase);
        Pair v[kNv][4];
        Pair s2 = pair(0.0f);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            Group<T> gx;
            slot_group<kEven>(slot, at, i, gx);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i][j] = element2(gx, j);
                s2 = fma2(v[i][j], v[i][j], s2);
            }
        }
        float rx = 1.0f;
        if (a.post) {
            const float s = sum_of(s2);
            rx = inverse_root(kWarp ? warp_sum(s) : block_sum(s), per, a.eps);
            if (at.t == 0 && a.post_rstd) a.post_rstd[r] = rx;
        }
        s2 = pair(0.0f);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            Pair g[4];
            gate.get(i, g);
            Group<S> gs;
            slot_group<kEven>(slot + x_slot, at, i, gs, skip);
            // (without a post norm rx is 1, without a skip its values 0: no branch costs less)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i][j] = fma2(skip_scale, element2(gs, j), mul2(mul2(v[i][j], pair(rx)), g[j]));
                s2 = fma2(v[i][j], v[i][j], s2);
            }
        }
        if (a.sum.p) {
#pragma unroll
            for (int i = 0; i < kNv; ++i) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) split(v[i][j], &o[2 * j], &o[2 * j + 1]);
                if (!kEven && a.shift_sum) store_shifted(sum, at, i, o);
                else store_group<true, S, kEven>(sum, at, i, o);
            }
        }
        float rs = 1.0f;
        if (a.y.p) {
            const float s = sum_of(s2);
            rs = inverse_root(kWarp ? warp_sum(s) : block_sum(s), per, a.eps);
            if (at.t == 0 && a.rstd) a.rstd[r] = rs;
        }
        // everything of the slots has been read: they take the row `stages` steps on
        if (kWarp || !a.y.p) row_sync<kWarp>();
        fill(stage);
        if (++stage == a.stages) stage = 0, phase ^= 1;
        if (a.y.p) {
#pragma unroll
            for (int i = 0; i < kNv; ++i) {
                Pair g[4];
                gain.get(i, g);
                float o[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) split(mul2(mul2(v[i][j], pair(rs)), g[j]), &o[2 * j], &o[2 * j + 1]);
                if (a.y_scale.p) {
                    // (lead 0: sixteen threads hold a block of 128)
                    uint32_t m = 0;
                    const int c = at.column(i, 0);
#pragma unroll
                    for (int j = 0; j < 8; ++j) m = max(m, c + j < a.cols ? magnitude(o[j]) : 0u);
#pragma unroll
                    for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
                    const BlockScale b = block_scale<false>(m);
                    if (c >= a.cols) continue;
                    if (at.t % 16 == 0)
                        ((float *)const_cast<void *>(a.y_scale.p))[r * a.y_scale.rs + c / 128 * a.y_scale.cs] = b.scale;
#pragma unroll
                    for (int j = 0; j < 8; j += 2)
                        split(quotient(pair(o[j], o[j + 1]), pair(b.factor), pair(b.rest)), &o[j], &o[j + 1]);
                    const uint2 q = make_uint2(pack_eight_bit<false>(o[0], o[1], o[2], o[3]), pack_eight_bit<false>(o[4], o[5], o[6], o[7]));
                    uint8_t *p = (uint8_t *)const_cast<void *>(a.y.p) + r * a.y.rs + c;
                    if (c + 8 <= a.cols) {
                        *reinterpret_cast<uint2 *>(p) = q;
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (c + j < a.cols) p[j] = (uint8_t)((j < 4 ? q.x : q.y) >> (j % 4 * 8));
                    }
                } else if (!kEven && a.shift_y) {
                    store_shifted(y, at, i, o);
                } else {
                    store_group<true, T, kEven>(y, at, i, o);
                }
            }
        }
        if (a.sum.p) sum += rows.step * a.sum.rs;
        if (a.y.p && !a.y_scale.p) y += rows.step * a.y.rs;
    }
    wait.settle(feed.on);
}

// Any strides, types and widths: a block per row, held in shared memory.
__global__ void __launch_bounds__(kAnyThreads) block_norm_any_kernel(const BlockNormArgs a) {
    __shared__ __align__(16) BlockSums sums;
    Summer block_sum{&sums};
    extern __shared__ __align__(16) float row[];
    const float per = 1.0f / (float)a.cols;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        float s = 0.0f;
        for (int c = threadIdx.x; c < a.cols; c += kAnyThreads) {
            const float v = load_as_float(a.x.p, r * a.x.rs + c * a.x.cs, a.x.dtype);
            row[c] = v;
            s = fmaf(v, v, s);
        }
        float rx = 1.0f;
        if (a.post) {
            rx = inverse_root(block_sum(s), per, a.eps);
            if (threadIdx.x == 0 && a.post_rstd) a.post_rstd[r] = rx;
        }
        const int64_t gate = a.gate.p ? r / a.rows_per_gate * a.gate.rs : 0;
        s = 0.0f;
        for (int c = threadIdx.x; c < a.cols; c += kAnyThreads) {
            float v = row[c];
            if (a.post) v = v * rx * (a.post_gain ? load_as_float(a.post_gain, c, a.param_dtype) : 1.0f);
            float h = a.branch_scale * v;
            if (a.gate.p) h *= load_as_float(a.gate.p, gate + c * a.gate.cs, a.gate.dtype);
            if (a.skip.p) h = fmaf(a.skip_scale, load_as_float(a.skip.p, r * a.skip.rs + c * a.skip.cs, a.skip.dtype), h);
            row[c] = h;
            s = fmaf(h, h, s);
            if (a.sum.p) store_from_float(const_cast<void *>(a.sum.p), r * a.sum.rs + c * a.sum.cs, a.sum.dtype, h);
        }
        if (!a.y.p) continue;
        const float rs = inverse_root(block_sum(s), per, a.eps);
        if (threadIdx.x == 0 && a.rstd) a.rstd[r] = rs;
        if (!a.y_scale.p) {
            for (int c = threadIdx.x; c < a.cols; c += kAnyThreads)
                store_from_float(const_cast<void *>(a.y.p), r * a.y.rs + c * a.y.cs, a.y.dtype,
                                 row[c] * rs * (a.gain ? load_as_float(a.gain, c, a.param_dtype) : 1.0f));
            continue;
        }
        // (the other threads' elements: behind the sum's barrier)
        const int lane = threadIdx.x % 32;
        for (int b = threadIdx.x / 32; b * 128 < a.cols; b += kAnyThreads / 32) {
            float o[4];
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = b * 128 + j * 32 + lane;
                o[j] = c < a.cols ? row[c] * rs * (a.gain ? load_as_float(a.gain, c, a.param_dtype) : 1.0f) : 0.0f;
                m = max(m, magnitude(o[j]));
            }
            const BlockScale q = block_scale<false>(__reduce_max_sync(0xffffffffu, m));
            if (lane == 0) ((float *)const_cast<void *>(a.y_scale.p))[r * a.y_scale.rs + b * a.y_scale.cs] = q.scale;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = b * 128 + j * 32 + lane;
                if (c < a.cols)
                    ((uint8_t *)const_cast<void *>(a.y.p))[r * a.y.rs + c * a.y.cs] =
                        (uint8_t)pack_eight_bit<false>(quotient(o[j], q), 0.0f, 0.0f, 0.0f);
            }
        }
        __syncthreads();  // (before the next row is written over this one)
    }
}

// Threads of an SM that the kernel's launch bounds leave registers for.
int forward_threads(const Held &h) { return h.warp ? 768 : h.nv == 1 ? 1024 : 512; }

// Rows on their way, and the shared memory with them.
size_t forward_smem(const BlockNormArgs &a, const Held &h, bool aligned, int64_t ts, int64_t ss, int *stages) {
    const uint32_t stage = row_slot_bytes(a.cols, (uint32_t)ts) + (a.skip.p ? row_slot_bytes(a.cols, (uint32_t)ss) : 0);
    const int workers = h.warp ? 8 : 1;
    auto space = [&](int n) {
        return row_space(workers, n, stage, kept_sets(aligned, h.warp, 1), h.warp ? 32 : h.threads, h.nv).total;
    };
    *stages = stages_for(space(0), workers * stage, std::min(16, forward_threads(h) / h.threads));
    return space(*stages);
}

template <typename T, typename S, int kNv, bool kWarp, bool kEven>
bool launch_rows(BlockNormArgs a, const Held &h, bool aligned, cudaStream_t s) {
    const int workers = kWarp ? 8 : 1;
    const size_t smem = forward_smem(a, h, aligned, sizeof(T), sizeof(S), &a.stages);
    const int64_t most = workers_at_once(h, forward_threads(h), smem);
    int64_t grid;
    if (aligned) {
        a.per_worker = stretch_of(a.rows, most);
        grid = ((a.rows + a.per_worker - 1) / a.per_worker + workers - 1) / workers;
    } else {
        // (steps of a multiple of 8, so that a worker's rows share their lead)
        a.per_worker = 0;
        grid = std::min<int64_t>((a.rows + workers - 1) / workers, std::max<int64_t>(8, most / workers / 8 * 8));
    }
    return launch_large<block_norm_rows_kernel<T, S, kNv, kWarp, kEven>>(dim3((unsigned)grid), h.threads, smem, s, a);
}

template <typename T, typename S>
bool launch_forward(const BlockNormArgs &a, const Held &h, bool aligned, cudaStream_t s) {
    if (h.even) {
        if (h.warp) return h.nv == 1 ? launch_rows<T, S, 1, true, true>(a, h, true, s) : launch_rows<T, S, 2, true, true>(a, h, true, s);
        return h.nv == 1 ? launch_rows<T, S, 1, false, true>(a, h, true, s) : launch_rows<T, S, 2, false, true>(a, h, true, s);
    }
    if (h.warp) return launch_rows<T, S, 1, true, false>(a, h, aligned, s);
    return h.nv == 1 ? launch_rows<T, S, 1, false, false>(a, h, aligned, s) : launch_rows<T, S, 2, false, false>(a, h, aligned, s);
}

}  // namespace
}  // namespace i8c

using namespace i8c;

extern "C" {

conv_status conv_block_norm(const conv_matrix_desc *x, const void *x_dev, const conv_matrix_desc *skip,
                            const void *skip_dev, const conv_matrix_desc *gate, const void *gate_dev,
                            const void *post_gain_dev, const void *gain_dev, const conv_matrix_desc *sum,
                            void *sum_dev, const conv_matrix_desc *y, void *y_dev, const conv_matrix_desc *y_scale,
                            void *y_scale_dev, float *post_rstd_dev, float *rstd_dev,
                            const conv_block_norm_params *p, void *stream) {
    if (!x || !p || (!sum && !y)) return CONV_ERR_NULL_PTR;
    conv_status st;
    if ((st = check_matrix(x))) return st;
    if (!is_float_type(x->dtype)) return CONV_ERR_DTYPE;
    if ((st = check_block_params(p, x->dtype))) return st;
    const int64_t rows = x->rows, cols = x->cols, psize = channel_elem_size(p->param_dtype);
    if (cols < 1) return CONV_ERR_BAD_PARAM;
    if (cols > kMostColumns) return CONV_ERR_TOO_LARGE;
    if ((st = check_address(x, x_dev)) || (st = check_operand(skip, skip_dev, rows, cols)) ||
        (st = check_operand(sum, sum_dev, rows, cols)) || (st = check_operand(y, y_dev, rows, cols)) ||
        (st = check_gate(gate, gate_dev, rows, cols, x->dtype)))
        return st;
    if ((skip && !stream_type(skip->dtype, x->dtype)) || (sum && !stream_type(sum->dtype, x->dtype)) ||
        (skip && sum && skip->dtype != sum->dtype))
        return CONV_ERR_DTYPE;
    if (y) {
        if (y->dtype != x->dtype && y->dtype != CONV_FLOAT8_E4M3) return CONV_ERR_DTYPE;
        if (y->dtype == CONV_FLOAT8_E4M3) {
            if (!y_scale) return CONV_ERR_NULL_PTR;
            if ((st = check_operand(y_scale, y_scale_dev, rows, (cols + kScaleBlock - 1) / kScaleBlock))) return st;
            if (y_scale->dtype != CONV_FLOAT32) return CONV_ERR_DTYPE;
        }
    }
    if (!y || y->dtype != CONV_FLOAT8_E4M3) y_scale = nullptr;
    if (!p->post_norm) post_gain_dev = nullptr, post_rstd_dev = nullptr;
    if (!y) gain_dev = nullptr, rstd_dev = nullptr;
    if ((uintptr_t)post_gain_dev % psize || (uintptr_t)gain_dev % psize || (uintptr_t)post_rstd_dev % 4 || (uintptr_t)rstd_dev % 4)
        return CONV_ERR_ALIGNMENT;
    if (rows == 0) return CONV_OK;
    const Buffer in[] = {matrix_of(x, x_dev), matrix_of(skip, skip_dev), matrix_of(gate, gate_dev),
                         vector_of(post_gain_dev, cols * psize), vector_of(gain_dev, cols * psize)};
    const Buffer out[] = {matrix_of(sum, sum_dev), matrix_of(y, y_dev), matrix_of(y_scale, y_scale_dev),
                          vector_of(post_rstd_dev, rows * 4), vector_of(rstd_dev, rows * 4)};
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < 5; ++j) {
            // in place: sum on skip or x, y on x
            const bool same = (i == 0 && (j == 1 || j == 0) && in[j].d && sum && sum->dtype == in[j].d->dtype &&
                               same_matrix(sum, sum_dev, in[j].d, in[j].p)) ||
                              (i == 1 && j == 0 && y && y->dtype == x->dtype && same_matrix(y, y_dev, x, x_dev));
            if (!same && share(out[i], in[j])) return CONV_ERR_OVERLAP;
        }
        for (int j = 0; j < i; ++j)
            if (share(out[i], out[j])) return CONV_ERR_OVERLAP;
    }
    if ((st = check_device())) return st;
    BlockNormArgs a;
    a.x = mat_ref(x, x_dev), a.skip = mat_ref(skip, skip_dev), a.gate = mat_ref(gate, gate_dev);
    a.sum = mat_ref(sum, sum_dev), a.y = mat_ref(y, y_dev), a.y_scale = mat_ref(y_scale, y_scale_dev);
    a.post_gain = post_gain_dev, a.gain = gain_dev, a.post_rstd = post_rstd_dev, a.rstd = rstd_dev;
    a.rows = rows, a.rows_per_gate = gate ? rows / gate->rows : rows;
    a.cols = (int32_t)cols;
    a.eps = p->eps, a.skip_scale = p->skip_scale, a.branch_scale = p->branch_scale;
    a.param_dtype = p->param_dtype, a.post = p->post_norm;
    a.per_worker = 0, a.wait_limit_ns = wait_limit_ns(), a.status = device_status_word();
    if (!a.status) return CONV_ERR_CUDA;
    const bool eight = y_scale != nullptr;
    // (8-bit rows are written in pieces of 8 bytes, their blocks counted from an aligned row's start)
    a.shift_sum = sum && !one_lead({&a.x, &a.sum});
    a.shift_y = y && !eight && !one_lead({&a.x, &a.y});
    const bool unit = unit_columns(a.x) && unit_columns(a.skip) && unit_columns(a.sum) && unit_columns(a.y) && unit_columns(a.gate);
    Held h = unit && one_lead({&a.x, &a.skip}) && (!eight || (aligned_rows(a.x) && aligned_rows(a.y)))
                       ? held(cols, aligned_rows(a.x),
                              cols % 8 == 0 && aligned_rows(a.x) && aligned_rows(a.sum) && (eight || aligned_rows(a.y)))
                       : Held();
    const int32_t s_type = skip ? skip->dtype : sum ? sum->dtype : x->dtype;
    int stages;
    if (h.nv && forward_smem(a, h, aligned_rows(a.x), channel_elem_size(x->dtype), channel_elem_size(s_type), &stages) > 216 << 10) h = Held();
    const cudaStream_t s = (cudaStream_t)stream;
    bool ok;
    if (h.nv == 0) {
        const size_t smem = (size_t)cols * 4;
        const int64_t per_sm = std::max<int64_t>(1, std::min<int64_t>(4, (int64_t)((224 << 10) / (smem + 2048))));
        ok = launch_large<block_norm_any_kernel>(dim3((unsigned)std::min<int64_t>(rows, device_sm_count() * per_sm)), kAnyThreads,
                                                 smem, s, a);
    } else {
        ok = by_types(x->dtype, s_type,
                      [&](auto t, auto u) { return launch_forward<decltype(t), decltype(u)>(a, h, aligned_rows(a.x), s); });
    }
    return ok ? CONV_OK : CONV_ERR_CUDA;
}

}  // extern "C"

// block_norm.cuh -- what the block norm and its gradient share: how a worker's
// rows, parameters and shared memory are laid out, how many workers there are,
// and the checks of their arguments.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "channel.h"
#include "channel_launch.cuh"
#include "channel_math.cuh"
#include "channel_rows.cuh"
#include "eight_bit.cuh"
#include "tc_ptx.cuh"

namespace i8c {

constexpr int kAnyThreads = 512;                 // of the kernels for any strides
constexpr int64_t kMostColumns = 49152;          // a row in 192 KB of shared memory
constexpr int64_t kMostGradColumns = kMostColumns / 2;

// 1 / sqrt(mean + eps).  A sum that has overflowed (of an infinity, or of
// finite squares) would give 0: NaN says so instead.
__device__ __forceinline__ float inverse_root(float sum, float per, float eps) {
    return sum <= 3.402823466e38f ? rsqrtf(sum * per + eps) : __uint_as_float(0x7fffffffu);
}

// A worker's parameters in shared memory: 8 of them for group i of thread t,
// two pieces of 16 bytes a worker's width apart.
struct Kept {
    uint32_t base, stride;  // this thread's first piece
    __device__ __forceinline__ uint32_t at(int i) const { return base + i * 2 * stride; }
    __device__ __forceinline__ void keep(int i, const float (&v)[8]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            ptx::st_shared_v4(at(i) + h * stride, make_uint4(__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                                                             __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])));
    }
    __device__ __forceinline__ void get(int i, Pair (&g)[4]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 w = ptx::ld_shared_v4(at(i) + h * stride);
            g[2 * h] = pair(__uint_as_float(w.x), __uint_as_float(w.y));
            g[2 * h + 1] = pair(__uint_as_float(w.z), __uint_as_float(w.w));
        }
    }
};

__device__ __forceinline__ float sum_of(Pair p) {
    float a, b;
    split(p, &a, &b);
    return a + b;
}

__device__ __forceinline__ const void *gate_row(const MatRef &gate, int64_t row) {
    return gate.p ? (const char *)gate.p + row * gate.rs * (gate.dtype == CONV_FLOAT32 ? 4 : 2) : nullptr;
}

// The gate (with the branch's scale) and the post gain, in one: what a row of
// gate `which` is multiplied by.
__device__ __forceinline__ void keep_gate(const Kept &kept, const MatRef &gate, int64_t which, const Kept &post_gain, bool post,
                                          float branch_scale, const Place<true> &at, int i) {
    float g[8];
    load_params(gate_row(gate, which), gate.dtype, 1.0f, at, i, g);
    Pair p[4];
    if (post) post_gain.get(i, p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        Pair w = mul2(pair(g[2 * j], g[2 * j + 1]), pair(branch_scale));
        if (post) w = mul2(w, p[j]);
        split(w, &g[2 * j], &g[2 * j + 1]);
    }
    kept.keep(i, g);
}

// The rows of a worker: a stretch, or (rows that begin anywhere) every
// step-th, the steps being a multiple of 8 so that all begin alike.
struct Stretch {
    int64_t first, end, step;
};

// Shared memory of the row kernels: barriers, rows, kept parameters (offsets;
// the same on both sides of a launch).
struct RowSpace {
    uint32_t rows, kept, total;
};
constexpr int kMostStages = 4;  // rows on their way, the one being read among them
__host__ __device__ inline RowSpace row_space(int workers, int stages, uint32_t stage_bytes, int kept_sets, int worker_threads,
                                              int nv) {
    RowSpace s;
    s.rows = 8 * 8 * kMostStages;  // (behind the barriers of 8 workers)
    s.kept = s.rows + workers * stages * stage_bytes;
    s.total = s.kept + kept_sets * nv * 32 * worker_threads;
    return s;
}

// ---------------------------------------------------------------- launches
// How rows are held: by a warp of one group of 8 per lane (of even rows, two),
// else by a block of one group per thread up to 512 of them, two up to 1024.
// (The code for the ends of rows would not fit the registers beside two
// groups of a warp.)
struct Held {
    int nv = 0, threads = 0;  // nv == 0: in shared memory
    bool warp = false, even = false;
};
inline Held held(int64_t cols, bool aligned, bool even) {
    Held h;
    h.even = even;
    const int64_t groups = aligned ? (cols + 7) / 8 : (cols + 14) / 8;
    if (groups <= (even ? 64 : 32)) {
        h.warp = true, h.threads = 256;
        h.nv = groups <= 32 ? 1 : 2;
    } else if (groups <= 1024) {
        h.nv = groups <= 512 ? 1 : 2;
        h.threads = (int)round_up((groups + h.nv - 1) / h.nv, 32);
    }
    return h;
}

// Whether every row of a matrix begins on a boundary of 8 elements.
inline bool aligned_rows(const MatRef &m) {
    if (!m.p) return true;
    const Lead l = lead_of_rows(m);
    return l.base == 0 && l.step == 0;
}

// A matrix of the call: given (with its address) or not, of one of two types.
inline conv_status check_operand(const conv_matrix_desc *d, const void *p, int64_t rows, int64_t cols) {
    if (!d) return CONV_OK;
    conv_status st = check_matrix(d);
    if (st) return st;
    if (d->rows != rows || d->cols != cols) return CONV_ERR_SHAPE_MISMATCH;
    return check_address(d, p);
}

inline conv_status check_block_params(const conv_block_norm_params *p, int32_t x_type) {
    if (!(p->eps > 0.0f) || !std::isfinite(p->eps) || !std::isfinite(p->skip_scale) || !std::isfinite(p->branch_scale) ||
        (p->post_norm != 0 && p->post_norm != 1) || p->reserved[0] != 0 || p->reserved[1] != 0 || p->reserved[2] != 0)
        return CONV_ERR_BAD_PARAM;
    if (p->param_dtype != CONV_FLOAT32 && p->param_dtype != x_type) return CONV_ERR_DTYPE;
    return CONV_OK;
}

inline bool stream_type(int32_t t, int32_t x_type) { return t == CONV_FLOAT32 || t == x_type; }

// A gate (or its gradient) for `rows` rows.
inline conv_status check_gate(const conv_matrix_desc *g, const void *p, int64_t rows, int64_t cols, int32_t x_type) {
    if (!g) return CONV_OK;
    conv_status st = check_matrix(g);
    if (st) return st;
    if (!stream_type(g->dtype, x_type)) return CONV_ERR_DTYPE;
    if (g->cols != cols || (g->rows == 0 ? rows != 0 : rows % g->rows != 0)) return CONV_ERR_SHAPE_MISMATCH;
    return check_address(g, p);
}

// One buffer of a call, for the overlap checks: a matrix, or a vector of n elements of `size` bytes.
struct Buffer {
    const conv_matrix_desc *d;
    const void *p;
    int64_t bytes;
};
inline bool share(const Buffer &a, const Buffer &b) {
    if (a.d && b.d) return matrices_overlap(a.d, a.p, b.d, b.p);
    return overlaps(a.p, (uint64_t)a.bytes, b.p, (uint64_t)b.bytes);
}
inline Buffer matrix_of(const conv_matrix_desc *d, const void *p) { return {d, d ? p : nullptr, d ? (int64_t)matrix_extent_bytes(d) : 0}; }
inline Buffer vector_of(const void *p, int64_t bytes) { return {nullptr, p, bytes}; }

// Workers that run at once: blocks of an SM by threads (the launch bounds) and
// shared memory, times their warps.
inline int64_t workers_at_once(const Held &h, int threads_bound, size_t smem) {
    const int64_t per_sm = std::max<int64_t>(1, std::min<int64_t>({threads_bound / h.threads, (int64_t)((224 << 10) / (smem + 2048)), 16}));
    return device_sm_count() * per_sm * (h.warp ? 8 : 1);
}

// Rows of each of `most` workers: all stretches alike but the last one.
inline int64_t stretch_of(int64_t rows, int64_t most) { return (rows + most - 1) / most; }

// Sets of kept parameters: two gains for all workers, or (rows that begin
// anywhere) for each, and `more` for each.
inline int kept_sets(bool stretches, bool warp, int more) { return (stretches ? 2 : warp ? 16 : 2) + more * (warp ? 8 : 1); }

// As many rows on their way as leave room for `blocks` blocks on an SM, two at least.
inline int stages_for(uint32_t fixed, uint32_t per_stage, int blocks) {
    const int64_t room = ((224 << 10) / blocks - 2048 - (int64_t)fixed) / (int64_t)per_stage;
    return (int)std::max<int64_t>(2, std::min<int64_t>(kMostStages, room));
}

// The types of x and of the stream, as a call of f.
template <typename F>
inline bool by_types(int32_t x, int32_t stream, F f) {
    if (x == CONV_FLOAT32) return f(0.0f, 0.0f);
    if (x == CONV_FLOAT16) return stream == CONV_FLOAT32 ? f(__half(), 0.0f) : f(__half(), __half());
    return stream == CONV_FLOAT32 ? f(__nv_bfloat16(), 0.0f) : f(__nv_bfloat16(), __nv_bfloat16());
}

}  // namespace i8c

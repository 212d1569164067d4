// block_norm.cu -- conv_block_norm and conv_block_norm_grad: the norm behind a
// residual block, its gate, the residual sum and the norm before the next
// block, as one pass over the rows.
//
// Both are streams.  A row is held by a warp (up to 512 columns) or a block;
// its matrices come in by asynchronous copies two or three rows ahead, into
// slots that only the reading thread uses, the sums of squares run over
// registers, and every output is written once.  In the gradient the two sums
// over rows that the parameters want are S = sum dh * v and sum dy * u: from S
// follow both dgate (times the post gain) and dpost_gain (times the gate), so
// a thread carries two vectors and not three.  Blocks are dealt to gates
// ("units": a gate's rows, or every splits-th of them), keep their shares in
// registers over their rows, and a second kernel adds the shares in order.
// Where there are more gates than blocks, a unit is a gate and its dgate
// leaves with its last row.
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
namespace {

constexpr int kAnyThreads = 512;                 // of the kernels for any strides
constexpr int64_t kMostColumns = 49152;          // a row in 192 KB of shared memory
constexpr int64_t kMostGradColumns = kMostColumns / 2;
constexpr int64_t kMaxParts = 608;               // shares of the sums over rows: four blocks per SM

struct BlockNormArgs {
    MatRef x, skip, gate, sum, y, y_scale;
    const void *post_gain, *gain;
    float *post_rstd, *rstd;
    int64_t rows, rows_per_gate;
    int32_t cols;
    float eps, skip_scale, branch_scale;
    int32_t param_dtype;
    int32_t post;
    int32_t turn_sum, turn_y;  // rows of another lead than x's
};

// 1 / sqrt(mean + eps).  A sum that has overflowed (of an infinity, or of
// finite squares) would give 0: NaN says so instead.
__device__ __forceinline__ float inverse_root(float sum, float per, float eps) {
    return sum <= 3.402823466e38f ? rsqrtf(sum * per + eps) : __uint_as_float(0x7fffffffu);
}

// Pieces of 16 bytes in a group of 8.
template <typename X>
__device__ __forceinline__ uint32_t pieces() { return kIs16<X> ? 1u : 2u; }

// A thread's 8 parameters in shared memory (two pieces of 16 bytes).
__device__ __forceinline__ void keep_params(uint32_t slot, uint32_t stride, const float (&v)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        ptx::st_shared_v4(slot + h * stride, make_uint4(__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                                                        __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])));
}
__device__ __forceinline__ void kept_params(uint32_t slot, uint32_t stride, Pair (&g)[4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint4 w = ptx::ld_shared_v4(slot + h * stride);
        g[2 * h] = pair(__uint_as_float(w.x), __uint_as_float(w.y));
        g[2 * h + 1] = pair(__uint_as_float(w.z), __uint_as_float(w.w));
    }
}

__device__ __forceinline__ float sum_of(Pair p) {
    float a, b;
    split(p, &a, &b);
    return a + b;
}

template <typename T, typename S>
constexpr int stages_of() { return kIs16<T> && kIs16<S> ? 3 : 2; }

// ---------------------------------------------------------------- forward
template <typename T, typename S, int kNv, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 256 : 512, kWarp ? 3 : kNv == 1 ? 2 : 1)
    block_norm_rows_kernel(const BlockNormArgs a) {
    __shared__ __align__(16) BlockSums sums;
    Summer block_sum{&sums};
    // gains [group][post, pre][half][thread] of 16 bytes; the rows on their
    // way; rows being turned
    extern __shared__ __align__(16) float shared[];
    constexpr int kStages = stages_of<T, S>();
    const int64_t first = kWarp ? (int64_t)blockIdx.x * 8 + threadIdx.x / 32 : blockIdx.x;
    const int64_t step = kWarp ? (int64_t)gridDim.x * 8 : gridDim.x;
    const T *x = (const T *)a.x.p;
    const S *skip = (const S *)a.skip.p;
    S *sum = (S *)const_cast<void *>(a.sum.p);
    Place<true> at;
    at.t = kWarp ? threadIdx.x % 32 : threadIdx.x;
    at.threads = kWarp ? 32 : blockDim.x;
    at.cols = a.cols;
    at.lead = lead_of(x + first * a.x.rs);
    const float per = 1.0f / (float)a.cols;
    const uint32_t stride = blockDim.x * 16;
    const uint32_t gains = ptx::smem_addr(shared) + threadIdx.x * 16;
    const uint32_t ring = gains + kNv * 4 * stride;
    const uint32_t stage_bytes = (pieces<T>() + (skip ? pieces<S>() : 0u)) * kNv * stride;
    char *turned = (char *)shared + kNv * 4 * stride + kStages * stage_bytes;
    const int turn_at = kWarp ? threadIdx.x / 32 * turn_elems(a.cols) : 0;
    const Turn<S> turn_sum{(S *)turned + turn_at, lead_of(sum + first * a.sum.rs)};
    if (a.turn_sum) turned += (int64_t)turn_elems(a.cols) * sizeof(S) * (kWarp ? 8 : 1);
    const Turn<T> turn_y{(T *)turned + turn_at, lead_of((const T *)a.y.p + first * a.y.rs)};
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    auto fetch = [&](int64_t r, int stage) {
        if (r < a.rows) {
#pragma unroll
            for (int i = 0; i < kNv; ++i) {
                const uint32_t to = ring + stage * stage_bytes + i * pieces<T>() * stride;
                fetch_group(x + r * a.x.rs, at, i, to, stride);
                if (skip) fetch_group(skip + r * a.skip.rs, at, i, ring + stage * stage_bytes + (kNv * pieces<T>() + i * pieces<S>()) * stride, stride);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int d = 0; d < kStages; ++d) fetch(first + d * step, d);
#pragma unroll
    for (int i = 0; i < kNv; ++i) {
        float g[8];
        load_params(a.post_gain, a.param_dtype, 1.0f, at, i, g);
        keep_params(gains + i * 4 * stride, stride, g);
        load_params(a.gain, a.param_dtype, 1.0f, at, i, g);
        keep_params(gains + (i * 4 + 2) * stride, stride, g);
    }
    const Pair skip_scale = pair(a.skip_scale), branch_scale = pair(a.branch_scale);
    int stage = 0;
    for (int64_t r = first; r < a.rows; r += step) {
        Group<T> gx[kNv];
        Group<S> gs[kNv];
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            read_group(ring + stage * stage_bytes + i * pieces<T>() * stride, stride, gx[i]);
            if (skip) read_group(ring + stage * stage_bytes + (kNv * pieces<T>() + i * pieces<S>()) * stride, stride, gs[i]);
        }
        Pair v[kNv][4];
        Pair s2 = pair(0.0f);
#pragma unroll
        for (int i = 0; i < kNv; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i][j] = element2(gx[i], j);
                s2 = fma2(v[i][j], v[i][j], s2);
            }
        // the slots just read take the row kStages steps on
        fetch(r + kStages * step, stage);
        if (++stage == kStages) stage = 0;
        if (a.post) {
            const float s = sum_of(s2), rx = inverse_root(kWarp ? warp_sum(s) : block_sum(s), per, a.eps);
            if (at.t == 0 && a.post_rstd) a.post_rstd[r] = rx;
#pragma unroll
            for (int i = 0; i < kNv; ++i) {
                Pair g[4];
                kept_params(gains + i * 4 * stride, stride, g);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = mul2(mul2(v[i][j], pair(rx)), g[j]);
            }
        }
        const int64_t gate_row = a.gate.p ? r / a.rows_per_gate * a.gate.rs : 0;
        s2 = pair(0.0f);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            float g[8];
            if (a.gate.p)
                load_params((const char *)a.gate.p + gate_row * (a.gate.dtype == CONV_FLOAT32 ? 4 : 2), a.gate.dtype, 0.0f, at, i, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                Pair h = mul2(branch_scale, v[i][j]);
                if (a.gate.p) h = mul2(h, pair(g[2 * j], g[2 * j + 1]));
                if (skip) h = fma2(skip_scale, element2(gs[i], j), h);
                v[i][j] = h;
                s2 = fma2(h, h, s2);
            }
        }
        if (sum) {
#pragma unroll
            for (int i = 0; i < kNv; ++i) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) split(v[i][j], &o[2 * j], &o[2 * j + 1]);
                if (a.turn_sum) turn_group(turn_sum, at, i, o);
                else store_group(sum + r * a.sum.rs, at, i, o);
            }
        }
        if (a.y.p) {
            const float s = sum_of(s2), rs = inverse_root(kWarp ? warp_sum(s) : block_sum(s), per, a.eps);
            if (at.t == 0 && a.rstd) a.rstd[r] = rs;
#pragma unroll
            for (int i = 0; i < kNv; ++i) {
                Pair g[4];
                kept_params(gains + (i * 4 + 2) * stride, stride, g);
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
                    const uint2 q = make_uint2(
                        pack_eight_bit<false>(o[0] * b.factor, o[1] * b.factor, o[2] * b.factor, o[3] * b.factor),
                        pack_eight_bit<false>(o[4] * b.factor, o[5] * b.factor, o[6] * b.factor, o[7] * b.factor));
                    uint8_t *p = (uint8_t *)const_cast<void *>(a.y.p) + r * a.y.rs + c;
                    if (c + 8 <= a.cols) {
                        *reinterpret_cast<uint2 *>(p) = q;
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (c + j < a.cols) p[j] = (uint8_t)((j < 4 ? q.x : q.y) >> (j % 4 * 8));
                    }
                } else if (a.turn_y) {
                    turn_group(turn_y, at, i, o);
                } else {
                    store_group((T *)const_cast<void *>(a.y.p) + r * a.y.rs, at, i, o);
                }
            }
        }
        if (a.turn_sum || a.turn_y) {
            row_sync<kWarp>();
            if (a.turn_sum) store_turned(sum + r * a.sum.rs, turn_sum, at);
            if (a.turn_y) store_turned((T *)const_cast<void *>(a.y.p) + r * a.y.rs, turn_y, at);
            row_sync<kWarp>();
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
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
                        (uint8_t)pack_eight_bit<false>(o[j] * q.factor, 0.0f, 0.0f, 0.0f);
            }
        }
        __syncthreads();  // (before the next row is written over this one)
    }
}

// ---------------------------------------------------------------- gradient
struct BlockNormGradArgs {
    MatRef dy, dsum, x, h, gate, dx, dskip, dgate;
    const void *post_gain, *gain;
    const float *post_rstd, *rstd;
    float *part;               // [blocks][3][part_cols], or NULL: shares of sum dy u, then of S, or of sum db v where units are whole
    int64_t rows, rows_per_gate, gates;
    int32_t cols, part_cols;
    float skip_scale, branch_scale;
    int32_t param_dtype;
    int32_t post;
    int32_t splits;            // units of a gate's rows; 0: units are whole gates, several to a block
    int32_t turn_dx, turn_dskip;
};

// The rows of unit u: first, first + step, ... below end.
struct Unit {
    int64_t gate, first, end, step;
};
__device__ __forceinline__ Unit unit_at(const BlockNormGradArgs &a, int64_t u) {
    Unit n;
    const int64_t parts = a.splits ? a.splits : 1;
    n.gate = u / parts;
    n.first = n.gate * a.rows_per_gate + (u - n.gate * parts);
    n.end = (n.gate + 1) * a.rows_per_gate;
    n.step = parts;
    return n;
}

// (one stage where two do not fit: a row's slots are filled again as soon as they have been read)
__host__ __device__ constexpr int grad_stages(int nv, bool warp) { return nv == 2 && !warp ? 1 : 2; }

// kWhole: a worker (warp or block) takes whole gates.
template <typename T, typename S, int kNv, bool kWarp, bool kWhole>
__global__ void __launch_bounds__(kWarp ? 256 : 512, kWarp ? 2 : 1) block_norm_grad_rows_kernel(const BlockNormGradArgs a) {
    __shared__ __align__(16) BlockSums sums;
    Summer block_sum{&sums};
    // [group][gain, post gain, gate][half][thread] of 16 bytes; the rows on
    // their way; rows being turned; kWarp: at the end [8 warps][2][cols] sums
    // over all of it
    extern __shared__ __align__(16) float shared[];
    constexpr int kStages = grad_stages(kNv, kWarp);
    const T *dy = (const T *)a.dy.p, *x = (const T *)a.x.p;
    const S *ds = (const S *)a.dsum.p, *hs = (const S *)a.h.p;
    T *dx = (T *)const_cast<void *>(a.dx.p);
    S *dskip = (S *)const_cast<void *>(a.dskip.p);
    const int worker = kWarp && kWhole ? blockIdx.x * 8 + threadIdx.x / 32 : blockIdx.x;
    const int64_t workers = kWarp && kWhole ? (int64_t)gridDim.x * 8 : gridDim.x;
    const int64_t units = a.splits ? a.gates * a.splits : a.gates;
    // rows of a unit are dealt to the block's warps, unless a warp has a unit of its own
    const int deal = kWarp && !kWhole ? 8 : 1, mine = kWarp && !kWhole ? threadIdx.x / 32 : 0;
    Place<true> at;
    at.t = kWarp ? threadIdx.x % 32 : threadIdx.x;
    at.threads = kWarp ? 32 : blockDim.x;
    at.cols = a.cols;
    {
        // (one lead for all matrices and, where there are several units, for all rows)
        const Unit n = unit_at(a, worker);
        const int64_t r = n.first + mine * n.step;
        at.lead = dy ? lead_of(dy + r * a.dy.rs) : lead_of(ds + r * a.dsum.rs);
    }
    const float per = 1.0f / (float)a.cols;
    const uint32_t stride = blockDim.x * 16;
    const uint32_t params = ptx::smem_addr(shared) + threadIdx.x * 16;
    const uint32_t ring = params + kNv * 6 * stride;
    // offsets of the matrices in a stage
    const uint32_t of_ds = dy ? (pieces<T>() + pieces<S>()) * kNv * stride : 0u;
    const uint32_t of_x = of_ds + (ds ? pieces<S>() * kNv * stride : 0u);
    const uint32_t of_h = pieces<T>() * kNv * stride;  // behind dy, with which it comes
    const uint32_t stage_bytes = of_x + (x ? pieces<T>() * kNv * stride : 0u);
    char *turned = (char *)shared + kNv * 6 * stride + kStages * stage_bytes;
    const int turn_at = kWarp ? threadIdx.x / 32 * turn_elems(a.cols) : 0;
    Turn<S> turn_dskip{(S *)turned + turn_at, 0};
    if (a.turn_dskip) turned += (int64_t)turn_elems(a.cols) * sizeof(S) * (kWarp ? 8 : 1);
    Turn<T> turn_dx{(T *)turned + turn_at, 0};
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    auto fetch = [&](int64_t r, const Unit &n, int stage) {
        if (r < n.end) {
            const uint32_t to = ring + stage * stage_bytes;
#pragma unroll
            for (int i = 0; i < kNv; ++i) {
                if (dy) {
                    fetch_group(dy + r * a.dy.rs, at, i, to + i * pieces<T>() * stride, stride);
                    fetch_group(hs + r * a.h.rs, at, i, to + of_h + i * pieces<S>() * stride, stride);
                }
                if (ds) fetch_group(ds + r * a.dsum.rs, at, i, to + of_ds + i * pieces<S>() * stride, stride);
                if (x) fetch_group(x + r * a.x.rs, at, i, to + of_x + i * pieces<T>() * stride, stride);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // (parameters of units: the gains once, the gate with each)
#pragma unroll
    for (int i = 0; i < kNv; ++i) {
        float g[8];
        load_params(a.gain, a.param_dtype, 1.0f, at, i, g);
        keep_params(params + i * 6 * stride, stride, g);
        load_params(a.post_gain, a.param_dtype, 1.0f, at, i, g);
        keep_params(params + (i * 6 + 2) * stride, stride, g);
    }
    Pair dg[kNv][4], sv[kNv][4], dp[kWhole ? kNv : 1][4];
#pragma unroll
    for (int i = 0; i < kNv; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            dg[i][j] = sv[i][j] = pair(0.0f);
            if constexpr (kWhole) dp[i][j] = pair(0.0f);
        }
    const Pair skip_scale = pair(a.skip_scale), branch_scale = pair(a.branch_scale);
    for (int64_t u = worker; u < units; u += workers) {
        const Unit n = unit_at(a, u);
        const int64_t first = n.first + mine * n.step, step = n.step * deal;
#pragma unroll
        for (int d = 0; d < kStages; ++d) fetch(first + d * step, n, d);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            float g[8];
            load_params(a.gate.p ? (const char *)a.gate.p + n.gate * a.gate.rs * (a.gate.dtype == CONV_FLOAT32 ? 4 : 2) : nullptr,
                        a.gate.dtype, 1.0f, at, i, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] *= a.branch_scale;
            keep_params(params + (i * 6 + 4) * stride, stride, g);  // (with the branch's scale)
        }
        int stage = 0;
        for (int64_t r = first; r < n.end; r += step) {
            const float rs = dy ? a.rstd[r] : 0.0f, rx = a.post ? a.post_rstd[r] : 1.0f;
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            const uint32_t from = ring + stage * stage_bytes;
            Pair dh[kNv][4];
            Group<T> gx[kNv];
            if (dy) {
                Group<T> gy[kNv];
                Group<S> gh[kNv];
                Pair s2 = pair(0.0f);
#pragma unroll
                for (int i = 0; i < kNv; ++i) {
                    read_group(from + i * pieces<T>() * stride, stride, gy[i]);
                    read_group(from + of_h + i * pieces<S>() * stride, stride, gh[i]);
                    Pair g[4];
                    kept_params(params + i * 6 * stride, stride, g);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const Pair d = element2(gy[i], j), w = mul2(element2(gh[i], j), pair(rs));
                        dh[i][j] = mul2(d, g[j]);
                        s2 = fma2(dh[i][j], w, s2);
                        dg[i][j] = fma2(d, w, dg[i][j]);
                    }
                }
                const float s = sum_of(s2), minus = -(kWarp ? warp_sum(s) : block_sum(s)) * per * rs * rs;
#pragma unroll
                for (int i = 0; i < kNv; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        dh[i][j] = fma2(element2(gh[i], j), pair(minus), mul2(dh[i][j], pair(rs)));
            } else {
#pragma unroll
                for (int i = 0; i < kNv; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) dh[i][j] = pair(0.0f);
            }
            if (ds) {
#pragma unroll
                for (int i = 0; i < kNv; ++i) {
                    Group<S> g;
                    read_group(from + of_ds + i * pieces<S>() * stride, stride, g);
#pragma unroll
                    for (int j = 0; j < 4; ++j) dh[i][j] = add2(dh[i][j], element2(g, j));
                }
            }
            if (x) {
#pragma unroll
                for (int i = 0; i < kNv; ++i) read_group(from + of_x + i * pieces<T>() * stride, stride, gx[i]);
            }
            fetch(r + kStages * step, n, stage);
            if (++stage == kStages) stage = 0;
            if (dskip) {
                if (a.turn_dskip) turn_dskip.lead = lead_of(dskip + r * a.dskip.rs);
#pragma unroll
                for (int i = 0; i < kNv; ++i) {
                    float o[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) split(mul2(skip_scale, dh[i][j]), &o[2 * j], &o[2 * j + 1]);
                    if (a.turn_dskip) turn_group(turn_dskip, at, i, o);
                    else store_group(dskip + r * a.dskip.rs, at, i, o);
                }
            }
            // S, and dn (in dh's place) with its sum
            Pair s2 = pair(0.0f);
#pragma unroll
            for (int i = 0; i < kNv; ++i) {
                Pair g[4], p[4];
                kept_params(params + (i * 6 + 4) * stride, stride, g);
                if (a.post) kept_params(params + (i * 6 + 2) * stride, stride, p);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (x) {
                        const Pair v = mul2(element2(gx[i], j), pair(rx));
                        sv[i][j] = fma2(dh[i][j], v, sv[i][j]);
                        dh[i][j] = mul2(dh[i][j], g[j]);
                        if (a.post) {
                            dh[i][j] = mul2(dh[i][j], p[j]);
                            s2 = fma2(dh[i][j], v, s2);
                        }
                    } else {
                        dh[i][j] = mul2(dh[i][j], g[j]);
                    }
                }
            }
            if (dx) {
                float minus = 0.0f;
                if (a.post) {
                    const float s = sum_of(s2);
                    minus = -(kWarp ? warp_sum(s) : block_sum(s)) * per * rx * rx;
                }
                if (a.turn_dx) turn_dx.lead = lead_of(dx + r * a.dx.rs);
#pragma unroll
                for (int i = 0; i < kNv; ++i) {
                    float o[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        Pair w = dh[i][j];
                        if (a.post) w = fma2(element2(gx[i], j), pair(minus), mul2(w, pair(rx)));
                        split(w, &o[2 * j], &o[2 * j + 1]);
                    }
                    if (a.turn_dx) turn_group(turn_dx, at, i, o);
                    else store_group(dx + r * a.dx.rs, at, i, o);
                }
            }
            if (a.turn_dskip || a.turn_dx) {
                row_sync<kWarp>();
                if (a.turn_dskip) store_turned(dskip + r * a.dskip.rs, turn_dskip, at);
                if (a.turn_dx) store_turned(dx + r * a.dx.rs, turn_dx, at);
                row_sync<kWarp>();
            }
        }
        if constexpr (kWhole) {
            // the gate's sum is complete: its gradient, and its share of the post gain's
#pragma unroll
            for (int i = 0; i < kNv; ++i) {
                Pair g[4], p[4];
                kept_params(params + (i * 6 + 4) * stride, stride, g);
                kept_params(params + (i * 6 + 2) * stride, stride, p);
                float o[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    dp[i][j] = fma2(g[j], sv[i][j], dp[i][j]);
                    split(mul2(mul2(sv[i][j], p[j]), branch_scale), &o[2 * j], &o[2 * j + 1]);
                    sv[i][j] = pair(0.0f);
                }
                if (a.dgate.p) {
                    if (a.dgate.dtype == CONV_FLOAT32) store_group((float *)const_cast<void *>(a.dgate.p) + n.gate * a.dgate.rs, at, i, o);
                    else store_group((T *)const_cast<void *>(a.dgate.p) + n.gate * a.dgate.rs, at, i, o);
                }
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!a.part) return;
    float *part = a.part + (int64_t)blockIdx.x * 3 * a.part_cols;
    auto second = [&](int i, int j) -> Pair & {
        if constexpr (kWhole) return dp[i][j];
        else return sv[i][j];
    };
    if constexpr (!kWarp) {
        // (a block's shares start at its lead: whole groups are aligned)
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            const int c = at.column(i, 0) + at.lead;
            if (c >= a.cols + at.lead) continue;
            float g[8], b[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) split(dg[i][j], &g[2 * j], &g[2 * j + 1]), split(second(i, j), &b[2 * j], &b[2 * j + 1]);
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                *reinterpret_cast<float4 *>(part + c + j) = make_float4(g[j], g[j + 1], g[j + 2], g[j + 3]);
                *reinterpret_cast<float4 *>(part + a.part_cols + c + j) = make_float4(b[j], b[j + 1], b[j + 2], b[j + 3]);
            }
        }
        return;
    }
    __syncthreads();  // nothing in shared memory is read any more
    float *warp_part = shared + threadIdx.x / 32 * 2 * a.cols;
#pragma unroll
    for (int i = 0; i < kNv; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = at.column(i, j);
            float lo, hi;
            if (at.inside(c)) {
                split(dg[i][j / 2], &lo, &hi);
                warp_part[c] = j % 2 ? hi : lo;
                split(second(i, j / 2), &lo, &hi);
                warp_part[a.cols + c] = j % 2 ? hi : lo;
            }
        }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.cols; c += 256) {
        float s = shared[c];
#pragma unroll
        for (int w = 1; w < 8; ++w) s += shared[w * 2 * a.cols + c];
        part[c < a.cols ? c : a.part_cols + c - a.cols] = s;
    }
}

// Any strides, types and widths: a block per unit's row, held in shared
// memory; every thread adds to its own columns of the block's shares.
__global__ void __launch_bounds__(kAnyThreads) block_norm_grad_any_kernel(const BlockNormGradArgs a) {
    __shared__ __align__(16) BlockSums sums;
    Summer block_sum{&sums};
    extern __shared__ __align__(16) float shared[];
    float *const dhs = shared, *const vs = shared + a.cols;
    const float per = 1.0f / (float)a.cols;
    const int64_t units = a.splits ? a.gates * a.splits : a.gates;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    float *const dg = a.part ? a.part + (int64_t)blockIdx.x * 3 * a.part_cols : nullptr;
    float *const second = dg + a.part_cols, *const whole = dg + 2 * a.part_cols;
    float *const sv = a.splits ? second : whole;  // S of the unit
    if (dg)
        for (int c = threadIdx.x; c < a.cols; c += kAnyThreads) dg[c] = second[c] = whole[c] = 0.0f;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const Unit n = unit_at(a, u);
        const int64_t gate = n.gate * a.gate.rs;
        for (int64_t r = n.first; r < n.end; r += n.step) {
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
                    if (dg) sv[c] += dh * v;
                }
                dhs[c] = dn;
            }
            if (!a.dx.p) continue;
            s2 = a.post ? block_sum(s2) * per : 0.0f;
            for (int c = threadIdx.x; c < a.cols; c += kAnyThreads)
                store_from_float(const_cast<void *>(a.dx.p), r * a.dx.rs + c * a.dx.cs, a.dx.dtype,
                                 a.post ? rx * (dhs[c] - vs[c] * s2) : dhs[c]);
        }
        if (a.splits || !dg) continue;
        for (int c = threadIdx.x; c < a.cols; c += kAnyThreads) {
            const float t = a.branch_scale * whole[c];
            second[c] += t * (a.gate.p ? load_as_float(a.gate.p, gate + c * a.gate.cs, a.gate.dtype) : 1.0f);
            if (a.dgate.p)
                store_from_float(const_cast<void *>(a.dgate.p), n.gate * a.dgate.rs + c * a.dgate.cs, a.dgate.dtype,
                                 t * (a.post && a.post_gain ? load_as_float(a.post_gain, c, a.param_dtype) : 1.0f));
            whole[c] = 0.0f;
        }
    }
}

// Adds the blocks' shares: 32 columns per block, 16 threads per column.
// blockIdx.y 0: dgain, 1: dpost_gain, 2 + g: dgate of gate g.  Block i's
// shares start at (lead + i lead_step) mod 8.
struct BlockNormJoin {
    const float *part;
    MatRef gate, dgate;
    const void *post_gain;
    void *dgain, *dpost_gain;
    int64_t gates;
    int32_t parts, cols, part_cols, splits, lead, lead_step, param_dtype, post;
    float branch_scale;
};
__global__ void __launch_bounds__(512) block_norm_join_kernel(const BlockNormJoin a) {
    __shared__ float red[16][32];
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const int c = blockIdx.x * 32 + tx;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    for (int64_t what = blockIdx.y; what < 2 + (a.splits && a.dgate.p ? a.gates : 0); what += gridDim.y) {
        if (what == 0 ? !a.dgain : what == 1 && !a.dpost_gain) continue;
        const int lo = what >= 2 ? (int)(what - 2) * a.splits : 0, hi = what >= 2 ? lo + a.splits : a.parts;
        const bool weigh = what == 1 && a.splits && a.gate.p;
        float s = 0.0f;
        if (c < a.cols) {
#pragma unroll 1
            for (int i0 = lo + ty; i0 < hi; i0 += 16 * 8) {
                float v[8], g[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int i = i0 + 16 * u;
                    v[u] = i < hi ? a.part[((int64_t)3 * i + (what > 0)) * a.part_cols + c + ((a.lead + i * a.lead_step) & 7)] : 0.0f;
                    g[u] = weigh && i < hi ? load_as_float(a.gate.p, i / a.splits * a.gate.rs + c * a.gate.cs, a.gate.dtype) : 1.0f;
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) s += i0 + 16 * u < hi ? v[u] * g[u] : 0.0f;
            }
        }
        __syncthreads();
        red[ty][tx] = s;
        __syncthreads();
        if (ty || c >= a.cols) continue;
        for (int i = 1; i < 16; ++i) s += red[i][tx];
        if (what == 0) {
            store_from_float(a.dgain, c, a.param_dtype, s);
        } else if (what == 1) {
            store_from_float(a.dpost_gain, c, a.param_dtype, a.splits ? s * a.branch_scale : s);
        } else {
            s *= a.branch_scale;
            if (a.post && a.post_gain) s *= load_as_float(a.post_gain, c, a.param_dtype);
            store_from_float(const_cast<void *>(a.dgate.p), (what - 2) * a.dgate.rs + c * a.dgate.cs, a.dgate.dtype, s);
        }
    }
}

__global__ void __launch_bounds__(256) zero_matrix_kernel(MatRef m, int64_t rows, int64_t cols) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int64_t c = threadIdx.x; c < cols; c += 256) store_from_float(const_cast<void *>(m.p), r * m.rs + c * m.cs, m.dtype, 0.0f);
}

// ---------------------------------------------------------------- launches
// How rows are held: by a warp up to 64 groups of 8, else by a block of one
// group per thread up to 512 of them, two up to 1024.
struct Held {
    int nv = 0, threads = 0;  // nv == 0: in shared memory
    bool warp = false;
};
Held held(int64_t cols, bool aligned) {
    Held h;
    const int64_t groups = aligned ? (cols + 7) / 8 : (cols + 14) / 8;
    if (groups <= 64) {
        h.warp = true, h.threads = 256;
        h.nv = groups <= 32 ? 1 : 2;
    } else if (groups <= 1024) {
        h.nv = groups <= 512 ? 1 : 2;
        h.threads = (int)round_up((groups + h.nv - 1) / h.nv, 32);
    }
    return h;
}

// Whether every row of a matrix begins on a boundary of 8 elements.
bool aligned_rows(const MatRef &m) {
    if (!m.p) return true;
    const Lead l = lead_of_rows(m);
    return l.base == 0 && l.step == 0;
}

// A matrix of the call: given (with its address) or not, of one of two types.
conv_status check_operand(const conv_matrix_desc *d, const void *p, int64_t rows, int64_t cols) {
    if (!d) return CONV_OK;
    conv_status st = check_matrix(d);
    if (st) return st;
    if (d->rows != rows || d->cols != cols) return CONV_ERR_SHAPE_MISMATCH;
    return check_address(d, p);
}

conv_status check_block_params(const conv_block_norm_params *p, int32_t x_type) {
    if (!(p->eps > 0.0f) || !std::isfinite(p->eps) || !std::isfinite(p->skip_scale) || !std::isfinite(p->branch_scale) ||
        (p->post_norm != 0 && p->post_norm != 1) || p->reserved[0] != 0 || p->reserved[1] != 0 || p->reserved[2] != 0)
        return CONV_ERR_BAD_PARAM;
    if (p->param_dtype != CONV_FLOAT32 && p->param_dtype != x_type) return CONV_ERR_DTYPE;
    return CONV_OK;
}

bool stream_type(int32_t t, int32_t x_type) { return t == CONV_FLOAT32 || t == x_type; }

// A gate (or its gradient) for `rows` rows.
conv_status check_gate(const conv_matrix_desc *g, const void *p, int64_t rows, int64_t cols, int32_t x_type) {
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
bool share(const Buffer &a, const Buffer &b) {
    if (a.d && b.d) return matrices_overlap(a.d, a.p, b.d, b.p);
    return overlaps(a.p, (uint64_t)a.bytes, b.p, (uint64_t)b.bytes);
}
Buffer matrix_of(const conv_matrix_desc *d, const void *p) { return {d, d ? p : nullptr, d ? (int64_t)matrix_extent_bytes(d) : 0}; }
Buffer vector_of(const void *p, int64_t bytes) { return {nullptr, p, bytes}; }

template <typename T, typename S, int kNv, bool kWarp>
bool launch_rows(const BlockNormArgs &a, const Held &h, cudaStream_t s) {
    const size_t stage = (sizeof(T) + (a.skip.p ? sizeof(S) : 0)) * 8 * kNv * h.threads;
    const size_t turn = (size_t)turn_elems(a.cols) * (kWarp ? 8 : 1);
    const size_t smem = (size_t)kNv * 64 * h.threads + stages_of<T, S>() * stage + (a.turn_sum ? turn * sizeof(S) : 0) +
                        (a.turn_y ? turn * sizeof(T) : 0);
    // blocks that run at once, by threads (the launch bounds) and shared memory; a multiple of 8, so that a block's
    // rows share their lead
    const int64_t by_threads = kWarp ? 3 : (kNv == 1 ? 1024 : 512) / h.threads;
    const int64_t per_sm = std::max<int64_t>(1, std::min<int64_t>({by_threads, (int64_t)((224 << 10) / (smem + 2048)), 16}));
    const int64_t wanted = kWarp ? (a.rows + 7) / 8 : a.rows, most = device_sm_count() * per_sm / 8 * 8;
    return launch_large<block_norm_rows_kernel<T, S, kNv, kWarp>>(dim3((unsigned)std::min(wanted, most)), h.threads, smem, s, a);
}

template <typename T, typename S>
bool launch_forward(const BlockNormArgs &a, const Held &h, cudaStream_t s) {
    if (h.warp) return h.nv == 1 ? launch_rows<T, S, 1, true>(a, h, s) : launch_rows<T, S, 2, true>(a, h, s);
    return h.nv == 1 ? launch_rows<T, S, 1, false>(a, h, s) : launch_rows<T, S, 2, false>(a, h, s);
}

size_t grad_smem(const BlockNormGradArgs &a, const Held &h, int64_t ts, int64_t ss) {
    const size_t stage = (size_t)((a.dy.p ? ts + ss : 0) + (a.dsum.p ? ss : 0) + (a.x.p ? ts : 0)) * 8 * h.nv * h.threads;
    const size_t turn = (size_t)turn_elems(a.cols) * (h.warp ? 8 : 1);
    const size_t rows = (size_t)h.nv * 96 * h.threads + grad_stages(h.nv, h.warp) * stage + (a.turn_dskip ? turn * ss : 0) + (a.turn_dx ? turn * ts : 0);
    return std::max(rows, h.warp && a.part ? (size_t)a.cols * 64 : 0);
}
int64_t grad_blocks_per_sm(const Held &h, size_t smem) {
    const int64_t by_threads = h.warp ? 2 : 512 / h.threads;
    return std::max<int64_t>(1, std::min<int64_t>({by_threads, (int64_t)((224 << 10) / (smem + 2048)), 4}));
}

template <typename T, typename S, int kNv, bool kWarp>
bool launch_grad_rows(const BlockNormGradArgs &a, const Held &h, int64_t grid, size_t smem, cudaStream_t s) {
    return a.splits ? launch_large<block_norm_grad_rows_kernel<T, S, kNv, kWarp, false>>(dim3((unsigned)grid), h.threads, smem, s, a)
                    : launch_large<block_norm_grad_rows_kernel<T, S, kNv, kWarp, true>>(dim3((unsigned)grid), h.threads, smem, s, a);
}
template <typename T, typename S>
bool launch_backward(const BlockNormGradArgs &a, const Held &h, int64_t grid, size_t smem, cudaStream_t s) {
    if (h.warp)
        return h.nv == 1 ? launch_grad_rows<T, S, 1, true>(a, h, grid, smem, s) : launch_grad_rows<T, S, 2, true>(a, h, grid, smem, s);
    return h.nv == 1 ? launch_grad_rows<T, S, 1, false>(a, h, grid, smem, s) : launch_grad_rows<T, S, 2, false>(a, h, grid, smem, s);
}

// (room for a lead and for whole groups)
int64_t part_columns(int64_t cols) { return round_up(cols, 8) + 8; }

size_t block_norm_grad_bytes(int64_t rows, int64_t cols) {
    if (rows == 0) return 0;
    return (size_t)round_up(std::min(kMaxParts, rows) * 3 * part_columns(cols) * 4, 256);
}

// The types of x and of the stream, as a call of f.
template <typename F>
bool by_types(int32_t x, int32_t stream, F f) {
    if (x == CONV_FLOAT32) return f(0.0f, 0.0f);
    if (x == CONV_FLOAT16) return stream == CONV_FLOAT32 ? f(__half(), 0.0f) : f(__half(), __half());
    return stream == CONV_FLOAT32 ? f(__nv_bfloat16(), 0.0f) : f(__nv_bfloat16(), __nv_bfloat16());
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
    const bool eight = y_scale != nullptr;
    // (8-bit rows are written in pieces of 8 bytes, their blocks counted from an aligned row's start)
    a.turn_sum = sum && !one_lead({&a.x, &a.sum});
    a.turn_y = y && !eight && !one_lead({&a.x, &a.y});
    const bool unit = unit_columns(a.x) && unit_columns(a.skip) && unit_columns(a.sum) && unit_columns(a.y) && unit_columns(a.gate);
    const bool fits = (!a.turn_sum && !a.turn_y) || cols <= 4096;
    const Held h = unit && fits && one_lead({&a.x, &a.skip}) && (!eight || (aligned_rows(a.x) && aligned_rows(a.y)))
                       ? held(cols, aligned_rows(a.x))
                       : Held();
    const cudaStream_t s = (cudaStream_t)stream;
    bool ok;
    if (h.nv == 0) {
        const size_t smem = (size_t)cols * 4;
        const int64_t per_sm = std::max<int64_t>(1, std::min<int64_t>(4, (int64_t)((224 << 10) / (smem + 2048))));
        ok = launch_large<block_norm_any_kernel>(dim3((unsigned)std::min<int64_t>(rows, device_sm_count() * per_sm)), kAnyThreads,
                                                 smem, s, a);
    } else {
        ok = by_types(x->dtype, skip ? skip->dtype : sum ? sum->dtype : x->dtype,
                      [&](auto t, auto u) { return launch_forward<decltype(t), decltype(u)>(a, h, s); });
    }
    return ok ? CONV_OK : CONV_ERR_CUDA;
}

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
    a.part = dgate || dpost_gain_dev || dgain_dev ? (float *)workspace : nullptr;
    a.rows = rows, a.cols = (int32_t)cols, a.part_cols = (int32_t)part_columns(cols);
    a.gates = gate ? gate->rows : dgate ? dgate->rows : 1;
    a.rows_per_gate = rows / a.gates;
    a.skip_scale = p->skip_scale, a.branch_scale = p->branch_scale;
    a.param_dtype = p->param_dtype, a.post = p->post_norm && x;
    const MatRef &ref = dy ? a.dy : a.dsum;
    const bool one = one_lead({&ref, &a.dsum, &a.x, &a.h});
    a.turn_dx = dx && !one_lead({&ref, &a.dx});
    a.turn_dskip = dskip && !one_lead({&ref, &a.dskip});
    const bool unit = unit_columns(a.dy) && unit_columns(a.dsum) && unit_columns(a.x) && unit_columns(a.h) &&
                      unit_columns(a.dx) && unit_columns(a.dskip) && unit_columns(a.gate) && unit_columns(a.dgate);
    const bool aligned = aligned_rows(ref);
    Held h = unit && one && (aligned || a.gates == 1) ? held(cols, aligned) : Held();
    // (with more gates than blocks dgate leaves in aligned groups)
    if (a.gates > kMaxParts && !(aligned_rows(a.dgate) && aligned)) h = Held();
    const int64_t ts = channel_elem_size(x_type), ss = channel_elem_size(s_type);
    size_t smem = 0;
    int64_t per_sm = 1;
    if (h.nv) {
        smem = grad_smem(a, h, ts, ss);
        if (smem > 216 << 10) h = Held();
        else per_sm = grad_blocks_per_sm(h, smem);
    }
    if (!h.nv) {
        smem = (size_t)cols * 8;
        per_sm = std::max<int64_t>(1, std::min<int64_t>(4, (int64_t)((224 << 10) / (smem + 2048))));
    }
    // units: gates in `splits` parts, to fill the GPU, or whole gates where there are more of them than blocks
    const int64_t most = std::min<int64_t>(kMaxParts, device_sm_count() * per_sm);
    const int64_t per_unit = h.warp ? 8 : 1;  // rows of a unit at a time
    int64_t grid;
    if (a.gates > most) {
        a.splits = 0;
        grid = h.warp ? std::min(most, (a.gates + 7) / 8) : std::min(most, a.gates);
    } else {
        int64_t splits = std::min(most / a.gates, (a.rows_per_gate + per_unit - 1) / per_unit);
        // (rows that begin anywhere: a block's rows are a multiple of 8 apart, or one)
        if (h.nv && !h.warp && !aligned && splits < a.rows_per_gate) splits = std::max<int64_t>(8, splits / 8 * 8);
        splits = std::max<int64_t>(1, std::min(splits, a.rows_per_gate));
        a.splits = (int32_t)splits;
        grid = a.gates * splits;
    }
    bool ok;
    if (h.nv)
        ok = by_types(x_type, s_type, [&](auto t, auto u) { return launch_backward<decltype(t), decltype(u)>(a, h, grid, smem, s); });
    else
        ok = launch_large<block_norm_grad_any_kernel>(dim3((unsigned)grid), kAnyThreads, smem, s, a);
    if (ok && a.part) {
        BlockNormJoin j;
        j.part = a.part, j.gate = a.gate, j.dgate = a.dgate, j.post_gain = post_gain_dev;
        j.dgain = dgain_dev, j.dpost_gain = dpost_gain_dev;
        j.gates = a.gates, j.parts = (int32_t)grid, j.cols = a.cols, j.part_cols = a.part_cols, j.splits = a.splits;
        const Lead lead = h.nv && !h.warp ? lead_of_rows(ref) : Lead{0, 0};
        j.lead = (int32_t)lead.base, j.lead_step = (int32_t)lead.step;
        j.param_dtype = p->param_dtype, j.post = a.post, j.branch_scale = p->branch_scale;
        const int64_t what = 2 + (a.splits && dgate ? a.gates : 0);
        if (dgain_dev || dpost_gain_dev || what > 2)
            ok = launch_behind(block_norm_join_kernel, dim3((unsigned)((cols + 31) / 32), (unsigned)std::min<int64_t>(what, 32768)),
                               512, 0, s, j);
    }
    return ok ? CONV_OK : CONV_ERR_CUDA;
}

}  // extern "C"

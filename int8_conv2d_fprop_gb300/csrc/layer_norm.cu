// layer_norm.cu -- conv_layer_norm and conv_layer_norm_grad.
//
// Both are streams: every row is read once into registers, its sums are taken
// there (the variance from the differences to the mean, as the definition
// has it), and the result is written.  The gradient also sums two vectors
// over the rows; each block keeps its share in registers over its rows and a
// second kernel adds the blocks' shares in order, so that no atomics are
// needed.  Measured (bytes of the operands and results over time): 100352 x
// 256 int32 -> bf16 27 us, 5.8 TB/s; 16384 x 4096 bf16 forward 51 us,
// 5.3 TB/s; gradient of 50176 x 512 bf16 with a residual 40 us, 5.2 TB/s, of
// 16384 x 4096 100 us, 4.0 TB/s (one barrier per row); of 2047 x 5001 f16 with
// odd strides 36 us, where seven rows per block leave their start and end
// bare.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <initializer_list>
#include <type_traits>

#include "channel.h"
#include "channel_launch.cuh"
#include "channel_math.cuh"
#include "tc_ptx.cuh"

namespace i8c {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums of two values over the block (at most 32 warps), the same in every
// thread and in the same order in all of them, with one barrier: consecutive
// sums use the two buffers in turn, and no warp can be two sums ahead.
struct BlockSums {
    float2 part[2][32];
};

struct Summer {
    BlockSums *s;
    int turn = 0;
    __device__ __forceinline__ float2 operator()(float u, float v) {
        u = warp_sum(u);
        v = warp_sum(v);
        float2 *p = s->part[turn];
        turn ^= 1;
        if (threadIdx.x % 32 == 0) p[threadIdx.x / 32] = make_float2(u, v);
        __syncthreads();
        const int warps = blockDim.x / 32;
        float2 t = make_float2(0.0f, 0.0f);
        const float4 *q = reinterpret_cast<const float4 *>(p);
#pragma unroll 4
        for (int i = 0; i < warps / 2; ++i) {
            const float4 w = q[i];
            t.x += w.x + w.z;
            t.y += w.y + w.w;
        }
        if (warps & 1) t.x += p[warps - 1].x, t.y += p[warps - 1].y;
        return t;
    }
    __device__ __forceinline__ float operator()(float u) { return (*this)(u, 0.0f).x; }
};

// ---------------------------------------------------------------- rows in registers
// A row is held by a warp (kWarp: eight rows per block) or by the block, 8 kNv
// elements per thread, so that it is read once and every sum runs over
// registers.
//
// kVec: thread t holds the aligned groups of 8 elements t, t + T, ...: one
// 16-byte vector of a 16-bit type, two of a 32-bit one.  A row that starts
// `lead` elements past such a boundary starts with a partial group and ends
// with one.  Blocks step over the rows in multiples of 8, so a block (or
// warp) meets the same lead on all its rows whatever the row stride, and its
// columns stay in the same registers: odd widths cost two partial groups per
// row.  This wants one lead for all the matrices a call reads; an output with
// another one is turned through shared memory, a row at a time.  The gradient of
// matrices with several leads has thread t hold elements t, t + T, ..., one per
// access.
template <typename T>
constexpr bool kIs16 = sizeof(T) == 2;

template <typename T>
struct Group {  // 8 elements as stored
    uint32_t w[kIs16<T> ? 4 : 8];
};

template <typename T>
__device__ __forceinline__ float element(const Group<T> &g, int j) {
    if constexpr (std::is_same_v<T, float>) return __uint_as_float(g.w[j]);
    else if constexpr (std::is_same_v<T, int32_t>) return (float)(int32_t)g.w[j];
    else if constexpr (std::is_same_v<T, __half>)
        return __half2float(__ushort_as_half((unsigned short)(g.w[j / 2] >> (j % 2 * 16))));
    else return __uint_as_float(j % 2 ? g.w[j / 2] & 0xffff0000u : g.w[j / 2] << 16);
}

// Elements 2j and 2j + 1 as a pair of floats.
template <typename T>
__device__ __forceinline__ Pair element2(const Group<T> &g, int j) {
    if constexpr (std::is_same_v<T, __half>) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&g.w[j]));
        return pair(f.x, f.y);
    } else {
        return pair(element(g, 2 * j), element(g, 2 * j + 1));
    }
}

__device__ __forceinline__ uint32_t bits16(float v, const __half *) { return __half_as_ushort(__float2half_rn(v)); }
__device__ __forceinline__ uint32_t bits16(float v, const __nv_bfloat16 *) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Where a thread's elements lie in its rows.
template <bool kVec>
struct Place {
    int t, threads, cols, lead;
    // column of element j of the thread's group i; outside the row if not below cols
    __device__ __forceinline__ int column(int i, int j) const {
        return kVec ? (i * threads + t) * 8 - lead + j : (i * 8 + j) * threads + t;
    }
    __device__ __forceinline__ bool inside(int c) const { return (uint32_t)c < (uint32_t)cols; }
    __device__ __forceinline__ bool whole(int i) const {
        return kVec ? inside(column(i, 0)) && inside(column(i, 7)) : inside(column(i, 7));
    }
};

// Elements past the boundary of 8 at which p lies.
template <typename T>
__device__ __forceinline__ int lead_of(const T *p) {
    return (int)((uintptr_t)p / sizeof(T)) & 7;
}

// Group i of the row that starts at p; zeros outside the row.
template <bool kVec, typename T>
__device__ __forceinline__ void load_group(const T *p, const Place<kVec> &at, int i, Group<T> &g) {
    if (kVec && at.whole(i)) {
        const uint4 *q = reinterpret_cast<const uint4 *>(p + at.column(i, 0));
        const uint4 a = q[0];
        g.w[0] = a.x, g.w[1] = a.y, g.w[2] = a.z, g.w[3] = a.w;
        if constexpr (!kIs16<T>) {
            const uint4 b = q[1];
            g.w[4] = b.x, g.w[5] = b.y, g.w[6] = b.z, g.w[7] = b.w;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = at.column(i, j);
        if constexpr (kIs16<T>) {
            const uint32_t v = at.inside(c) ? reinterpret_cast<const uint16_t *>(p)[c] : 0u;
            if (j % 2) g.w[j / 2] |= v << 16;
            else g.w[j / 2] = v;
        } else {
            g.w[j] = at.inside(c) ? reinterpret_cast<const uint32_t *>(p)[c] : 0u;
        }
    }
}

template <bool kVec, typename T>
__device__ __forceinline__ void store_group(T *p, const Place<kVec> &at, int i, const float (&v)[8]) {
    if (kVec && at.whole(i)) {
        const int c = at.column(i, 0);
        if constexpr (kIs16<T>) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = pack2(v[2 * j], v[2 * j + 1], std::is_same_v<T, __half> ? CONV_FLOAT16 : CONV_BFLOAT16);
            *reinterpret_cast<uint4 *>(p + c) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            *reinterpret_cast<float4 *>(p + c) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(p + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = at.column(i, j);
        if (!at.inside(c)) continue;
        if constexpr (kIs16<T>) reinterpret_cast<uint16_t *>(p)[c] = (uint16_t)bits16(v[j], p);
        else p[c] = v[j];
    }
}

// The same for an output whose lead differs from the rows read: its groups
// are put together in shared memory, element c of the row at c + lead.
template <typename T>
struct Turn {
    T *buf;     // shared memory of the row's warp or block: cols + 16 elements
    int lead;   // of the output's rows
};

template <bool kVec, typename T>
__device__ __forceinline__ void turn_group(const Turn<T> &u, const Place<kVec> &at, int i, const float (&v)[8]) {
    if (at.whole(i)) {
        T *to = u.buf + at.column(i, 0) + u.lead;
        if constexpr (kIs16<T>) {
            if (((u.lead ^ at.lead) & 1) == 0) {
#pragma unroll
                for (int j = 0; j < 8; j += 2)
                    reinterpret_cast<uint32_t *>(to)[j / 2] =
                        pack2(v[j], v[j + 1], std::is_same_v<T, __half> ? CONV_FLOAT16 : CONV_BFLOAT16);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) reinterpret_cast<uint16_t *>(to)[j] = (uint16_t)bits16(v[j], u.buf);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) to[j] = v[j];
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = at.column(i, j);
        if (!at.inside(c)) continue;
        if constexpr (kIs16<T>) reinterpret_cast<uint16_t *>(u.buf)[c + u.lead] = (uint16_t)bits16(v[j], u.buf);
        else u.buf[c + u.lead] = v[j];
    }
}

template <bool kVec, typename T>
__device__ __forceinline__ void store_turned(T *p, const Turn<T> &u, const Place<kVec> &at) {
    for (int g = at.t; g * 8 < at.cols + u.lead; g += at.threads) {
        const int c = g * 8 - u.lead;
        if (c >= 0 && c + 8 <= at.cols) {
            const uint4 *q = reinterpret_cast<const uint4 *>(u.buf + g * 8);
            uint4 *o = reinterpret_cast<uint4 *>(p + c);
            o[0] = q[0];
            if constexpr (!kIs16<T>) o[1] = q[1];
        } else {
            for (int j = max(0, -c); j < 8 && c + j < at.cols; ++j) p[c + j] = u.buf[g * 8 + j];
        }
    }
}

template <bool kWarp>
__device__ __forceinline__ void row_sync() {
    if constexpr (kWarp) __syncwarp();
    else __syncthreads();
}

// 8 values of a parameter vector (any alignment; absent or outside: `fill`).
template <bool kVec>
__device__ __forceinline__ void load_params(const void *p, int32_t dtype, float fill, const Place<kVec> &at, int i,
                                            float (&v)[8]) {
    if (kVec && p && at.whole(i)) {
        const int c = at.column(i, 0);
        const char *q = (const char *)p + (int64_t)c * (dtype == CONV_FLOAT32 ? 4 : 2);
        if ((uintptr_t)q % 16 == 0) {
            if (dtype == CONV_FLOAT32) {
                const float4 a = reinterpret_cast<const float4 *>(q)[0], b = reinterpret_cast<const float4 *>(q)[1];
                v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
            } else {
                unpack8(*reinterpret_cast<const uint4 *>(q), dtype, v);
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = at.column(i, j);
        v[j] = p && at.inside(c) ? load_as_float(p, c, dtype) : fill;
    }
}

// Elements of a row being turned, a multiple of 16.
__host__ __device__ constexpr int turn_elems(int cols) { return (cols + 31) / 16 * 16; }

// Threads of a block that holds a row in kNv groups per thread, and the
// blocks of that size that registers are kept for.  (More elements per thread
// share one sum's shuffles and barrier; the gradient's sums take twice the
// registers.)
constexpr int norm_threads(int nv) { return nv == 2 ? 256 : 512; }
constexpr int norm_blocks(int nv) { return nv == 2 ? 3 : 1; }
constexpr int grad_threads(int nv) { return nv == 1 ? 128 : nv == 2 ? 320 : 512; }
constexpr int grad_blocks(int nv) { return nv == 1 ? 6 : nv == 2 ? 2 : 1; }

struct NormArgs {
    MatRef x, y;
    const void *gain, *shift;
    float *mean, *rstd;
    int64_t rows;
    int32_t cols;
    float eps, scale;
    int32_t param_dtype;
    int32_t turn;  // y's rows have another lead than x's
};

template <typename X, typename Y, int kNv, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 256 : norm_threads(kNv), kWarp ? (kNv == 4 ? 2 : 1) : norm_blocks(kNv))
    layer_norm_rows_kernel(const NormArgs a) {
    __shared__ __align__(16) BlockSums sums;
    Summer block_sum{&sums};
    // every thread's own gains and shifts unless kKeep ([group][gain, shift]
    // [half][thread] of 16 bytes), then rows being turned
    extern __shared__ __align__(16) float shared[];
    const int64_t first = kWarp ? (int64_t)blockIdx.x * 8 + threadIdx.x / 32 : blockIdx.x;
    const int64_t step = kWarp ? (int64_t)gridDim.x * 8 : gridDim.x;
    const X *x = (const X *)a.x.p;
    Y *y = (Y *)const_cast<void *>(a.y.p);
    Place<true> at;
    at.t = kWarp ? threadIdx.x % 32 : threadIdx.x;
    at.threads = kWarp ? 32 : blockDim.x;
    at.cols = a.cols;
    at.lead = lead_of(x + first * a.x.rs);
    const float per = 1.0f / (float)a.cols;
    constexpr bool kKeep = kNv <= 2;  // parameters in registers over the rows
    const Turn<Y> turn{(Y *)(shared + (kKeep ? 0 : kNv * 16 * blockDim.x)) +
                           (kWarp ? threadIdx.x / 32 * turn_elems(a.cols) : 0),
                       lead_of(y + first * a.y.rs)};
    float gain[kKeep ? kNv : 1][8], shift[kKeep ? kNv : 1][8];
    const uint32_t slot = ptx::smem_addr(shared) + threadIdx.x * 16, stride = blockDim.x * 16;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if constexpr (kKeep) {
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            load_params(a.gain, a.param_dtype, 1.0f, at, i, gain[i]);
            load_params(a.shift, a.param_dtype, 0.0f, at, i, shift[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            load_params(a.gain, a.param_dtype, 1.0f, at, i, gain[0]);
            load_params(a.shift, a.param_dtype, 0.0f, at, i, shift[0]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float *g = gain[0] + 4 * h, *b = shift[0] + 4 * h;
                ptx::st_shared_v4(slot + (4 * i + h) * stride, make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]),
                                                                          __float_as_uint(g[2]), __float_as_uint(g[3])));
                ptx::st_shared_v4(slot + (4 * i + 2 + h) * stride,
                                  make_uint4(__float_as_uint(b[0]), __float_as_uint(b[1]), __float_as_uint(b[2]),
                                             __float_as_uint(b[3])));
            }
        }
    }
    Group<X> next[kNv];
    if (first < a.rows) {
#pragma unroll
        for (int i = 0; i < kNv; ++i) load_group(x + first * a.x.rs, at, i, next[i]);
    }
    for (int64_t r = first; r < a.rows; r += step) {
        float v[kNv][8];
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kNv; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = a.scale * element(next[i], j);
                s += v[i][j];
            }
        if (r + step < a.rows) {
#pragma unroll
            for (int i = 0; i < kNv; ++i) load_group(x + (r + step) * a.x.rs, at, i, next[i]);
        }
        const float mean = (kWarp ? warp_sum(s) : block_sum(s)) * per;
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] -= mean;
            if (!at.whole(i)) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (!at.inside(at.column(i, j))) v[i][j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[i][j] * v[i][j];
        }
        const float rstd = rsqrtf((kWarp ? warp_sum(s) : block_sum(s)) * per + a.eps);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            if constexpr (kKeep) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * gain[i][j] + shift[i][j];
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 g = ptx::ld_shared_v4(slot + (4 * i + h) * stride);
                    const uint4 b = ptx::ld_shared_v4(slot + (4 * i + 2 + h) * stride);
                    float *w = v[i] + 4 * h;
                    w[0] = w[0] * rstd * __uint_as_float(g.x) + __uint_as_float(b.x);
                    w[1] = w[1] * rstd * __uint_as_float(g.y) + __uint_as_float(b.y);
                    w[2] = w[2] * rstd * __uint_as_float(g.z) + __uint_as_float(b.z);
                    w[3] = w[3] * rstd * __uint_as_float(g.w) + __uint_as_float(b.w);
                }
            }
            if (a.turn) turn_group(turn, at, i, v[i]);
            else store_group(y + r * a.y.rs, at, i, v[i]);
        }
        if (a.turn) {
            row_sync<kWarp>();
            store_turned(y + r * a.y.rs, turn, at);
            if (kWarp) __syncwarp();  // (a block's next row has barriers before it writes again)
        }
        if (at.t == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

struct NormGradArgs {
    MatRef dy, x, res, dx;
    const void *gain;
    const float *mean, *rstd;
    float *part;  // [blocks][2][part_cols], or NULL
    int64_t rows;
    int32_t cols;
    int32_t param_dtype;
    int32_t part_cols;
    int32_t turn;  // dx's rows have another lead than the matrices read
};

// Rows on their way: a thread's groups of the next kDepth rows come in by
// asynchronous copies into slots that only this thread reads, so that the
// loads in flight cost no registers and no barriers.
template <typename X>
constexpr int kDepth = kIs16<X> ? 3 : 2;

__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <typename X>
struct Slots {
    uint32_t base;    // this thread's first 16 bytes
    uint32_t stride;  // 16 bytes of every thread of the block
    __device__ __forceinline__ uint32_t at(int stage, int matrix, int matrices, int i, int nv) const {
        return base + ((stage * matrices + matrix) * nv + i) * (kIs16<X> ? 1 : 2) * stride;
    }
};

template <typename X>
__device__ __forceinline__ void fetch_group(const X *p, const Place<true> &at, int i, uint32_t slot, uint32_t stride) {
    if (at.whole(i)) {
        copy_async16(slot, p + at.column(i, 0));
        if constexpr (!kIs16<X>) copy_async16(slot + stride, p + at.column(i, 4));
        return;
    }
    Group<X> g;
    load_group(p, at, i, g);
    ptx::st_shared_v4(slot, make_uint4(g.w[0], g.w[1], g.w[2], g.w[3]));
    if constexpr (!kIs16<X>) ptx::st_shared_v4(slot + stride, make_uint4(g.w[4], g.w[5], g.w[6], g.w[7]));
}

template <typename X>
__device__ __forceinline__ void read_group(uint32_t slot, uint32_t stride, Group<X> &g) {
    const uint4 a = ptx::ld_shared_v4(slot);
    g.w[0] = a.x, g.w[1] = a.y, g.w[2] = a.z, g.w[3] = a.w;
    if constexpr (!kIs16<X>) {
        const uint4 b = ptx::ld_shared_v4(slot + stride);
        g.w[4] = b.x, g.w[5] = b.y, g.w[6] = b.z, g.w[7] = b.w;
    }
}

// dx of every row and this block's partial sums of dy * n and dy, in
// registers over its rows.
template <typename X, int kNv, bool kVec, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 256 : grad_threads(kNv), kWarp ? (kNv == 1 ? 3 : 2) : grad_blocks(kNv))
    layer_norm_grad_rows_kernel(const NormGradArgs a) {
    __shared__ __align__(16) BlockSums sums;
    Summer block_sum{&sums};
    // every thread's own gains if kKeep ([group][half][thread] of 16 bytes);
    // the rows on their way (kAhead); rows being turned; kWarp: at the end
    // [8 warps][2][cols] sums over all of it
    extern __shared__ __align__(16) float shared[];
    const int64_t first = kWarp ? (int64_t)blockIdx.x * 8 + threadIdx.x / 32 : blockIdx.x;
    const int64_t step = kWarp ? (int64_t)gridDim.x * 8 : gridDim.x;
    const X *x = (const X *)a.x.p, *dy = (const X *)a.dy.p, *res = (const X *)a.res.p;
    X *dx = (X *)const_cast<void *>(a.dx.p);
    Place<kVec> at;
    at.t = kWarp ? threadIdx.x % 32 : threadIdx.x;
    at.threads = kWarp ? 32 : blockDim.x;
    at.cols = a.cols;
    at.lead = kVec ? lead_of(x + first * a.x.rs) : 0;
    const float per = 1.0f / (float)a.cols;
    constexpr bool kKeep = kNv <= 2;
    constexpr bool kAhead = kVec && kNv <= 2;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int gain_elems = kKeep ? kNv * 8 * blockDim.x : 0;
    const int matrices = res ? 3 : 2;
    Slots<X> slots;
    slots.stride = blockDim.x * 16;
    slots.base = ptx::smem_addr(shared + gain_elems) + threadIdx.x * 16;
    const uint32_t ring_bytes = kAhead ? kDepth<X> * matrices * kNv * (kIs16<X> ? 1 : 2) * slots.stride : 0;
    const Turn<X> turn{(X *)((char *)(shared + gain_elems) + ring_bytes) + (kWarp ? threadIdx.x / 32 * turn_elems(a.cols) : 0),
                       lead_of(dx + first * a.dx.rs)};
    auto fetch = [&](int64_t r, int stage) {
        if constexpr (kAhead) {
            if (r < a.rows) {
#pragma unroll
                for (int i = 0; i < kNv; ++i) {
                    fetch_group(x + r * a.x.rs, at, i, slots.at(stage, 0, matrices, i, kNv), slots.stride);
                    fetch_group(dy + r * a.dy.rs, at, i, slots.at(stage, 1, matrices, i, kNv), slots.stride);
                    if (res) fetch_group(res + r * a.res.rs, at, i, slots.at(stage, 2, matrices, i, kNv), slots.stride);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
#pragma unroll
    for (int d = 0; d < kDepth<X>; ++d) fetch(first + d * step, d);
    const uint32_t my_gain = ptx::smem_addr(shared) + threadIdx.x * 16;
    if constexpr (kKeep) {
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            float g[8];
            load_params(a.gain, a.param_dtype, 1.0f, at, i, g);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                ptx::st_shared_v4(my_gain + (2 * i + h) * slots.stride,
                                  make_uint4(__float_as_uint(g[4 * h]), __float_as_uint(g[4 * h + 1]),
                                             __float_as_uint(g[4 * h + 2]), __float_as_uint(g[4 * h + 3])));
        }
    }
    // gains 4h .. 4h + 3 of group i
    auto load_gain = [&](int i, Pair (&g)[4]) {
        if constexpr (kKeep) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 w = ptx::ld_shared_v4(my_gain + (2 * i + h) * slots.stride);
                g[2 * h] = pair(__uint_as_float(w.x), __uint_as_float(w.y));
                g[2 * h + 1] = pair(__uint_as_float(w.z), __uint_as_float(w.w));
            }
        } else {
            float f[8];
            load_params(a.gain, a.param_dtype, 1.0f, at, i, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = pair(f[2 * j], f[2 * j + 1]);
        }
    };
    Pair dg[kNv][4], db[kNv][4];
#pragma unroll
    for (int i = 0; i < kNv; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) dg[i][j] = db[i][j] = pair(0.0f);
    float mu = 0.0f, rs = 0.0f;
    if (first < a.rows) mu = a.mean[first], rs = a.rstd[first];
    int stage = 0;
    for (int64_t r = first; r < a.rows; r += step) {
        Group<X> gx[kNv], gy[kNv], gr[kNv];
        if constexpr (kAhead) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kDepth<X> - 1) : "memory");
#pragma unroll
            for (int i = 0; i < kNv; ++i) {
                read_group(slots.at(stage, 0, matrices, i, kNv), slots.stride, gx[i]);
                read_group(slots.at(stage, 1, matrices, i, kNv), slots.stride, gy[i]);
                if (res) read_group(slots.at(stage, 2, matrices, i, kNv), slots.stride, gr[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kNv; ++i) {
                load_group(x + r * a.x.rs, at, i, gx[i]);
                load_group(dy + r * a.dy.rs, at, i, gy[i]);
                if (res) load_group(res + r * a.res.rs, at, i, gr[i]);
            }
        }
        const float m = mu, rr = rs;
        if (r + step < a.rows) mu = a.mean[r + step], rs = a.rstd[r + step];
        // n = (x - mean) rstd: the difference first, whose rounding is its own
        // (x rstd - mean rstd in one instruction is off by the rounding of
        // mean rstd: dgain by 2e-5 where the mean is 1000 deviations)
        const Pair scale = pair(rr), minus_mean = pair(-m);
        Pair st2 = pair(0.0f), stn2 = pair(0.0f);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            Pair gain[4];
            load_gain(i, gain);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // (outside the row dy is 0, and so is every term)
                const Pair d = element2(gy[i], j), n = mul2(add2(element2(gx[i], j), minus_mean), scale);
                const Pair u = mul2(d, gain[j]);
                st2 = add2(st2, u);
                stn2 = fma2(u, n, stn2);
                dg[i][j] = fma2(d, n, dg[i][j]);
                db[i][j] = add2(db[i][j], d);
            }
        }
        // the slots just read take the row kDepth steps on
        fetch(r + kDepth<X> * step, stage);
        if (++stage == kDepth<X>) stage = 0;
        if (!dx) continue;
        float st, stn, other;
        split(st2, &st, &other);
        st += other;
        split(stn2, &stn, &other);
        stn += other;
        if constexpr (kWarp) {
            st = warp_sum(st);
            stn = warp_sum(stn);
        } else {
            const float2 s = block_sum(st, stn);
            st = s.x, stn = s.y;
        }
        const Pair minus_st = pair(-st * per * rr), minus_stn = pair(-stn * per * rr);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            float v[8];
            Pair gain[4];
            load_gain(i, gain);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const Pair n = mul2(add2(element2(gx[i], j), minus_mean), scale);
                Pair w = fma2(mul2(element2(gy[i], j), gain[j]), scale, minus_st);
                w = fma2(n, minus_stn, w);
                if (res) w = add2(w, element2(gr[i], j));
                split(w, &v[2 * j], &v[2 * j + 1]);
            }
            if (kVec && a.turn) turn_group(turn, at, i, v);
            else store_group(dx + r * a.dx.rs, at, i, v);
        }
        if (kVec && a.turn) {
            row_sync<kWarp>();
            store_turned(dx + r * a.dx.rs, turn, at);
            if (kWarp) __syncwarp();  // (a block's next row has barriers before it writes again)
        }
    }
    if constexpr (kAhead) asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!a.part) return;
    float *part = a.part + (int64_t)blockIdx.x * 2 * a.part_cols;
    if constexpr (kVec && !kWarp) {
        // (a block's sums start at its lead: whole groups are aligned)
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            const int c = at.column(i, 0) + at.lead;
            if (c >= a.cols + at.lead) continue;
            float g[8], b[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) split(dg[i][j], &g[2 * j], &g[2 * j + 1]), split(db[i][j], &b[2 * j], &b[2 * j + 1]);
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                *reinterpret_cast<float4 *>(part + c + j) = make_float4(g[j], g[j + 1], g[j + 2], g[j + 3]);
                *reinterpret_cast<float4 *>(part + a.part_cols + c + j) = make_float4(b[j], b[j + 1], b[j + 2], b[j + 3]);
            }
        }
        return;
    }
    if constexpr (kWarp) __syncthreads();  // nothing in shared memory is read any more
    float *mine = kWarp ? shared + threadIdx.x / 32 * 2 * a.cols : part;
    const int second = kWarp ? a.cols : a.part_cols;
#pragma unroll
    for (int i = 0; i < kNv; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = at.column(i, j);
            float lo, hi;
            if (at.inside(c)) {
                split(dg[i][j / 2], &lo, &hi);
                mine[c] = j % 2 ? hi : lo;
                split(db[i][j / 2], &lo, &hi);
                mine[second + c] = j % 2 ? hi : lo;
            }
        }
    if constexpr (kWarp) {
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * a.cols; c += 256) {
            float s = shared[c];
#pragma unroll
            for (int w = 1; w < 8; ++w) s += shared[w * 2 * a.cols + c];
            part[c < a.cols ? c : a.part_cols + c - a.cols] = s;
        }
    }
}

// Adds the blocks' partial sums: 32 columns per block, 16 threads per column;
// blockIdx.y 0: dgain, 1: dshift.  Block i's sums start at (lead + i lead_step)
// mod 8.
__global__ void __launch_bounds__(512) layer_norm_params_sum_kernel(const float *part, int parts, int cols, int part_cols,
                                                                    int lead, int lead_step, void *dgain, void *dshift,
                                                                    int32_t dtype) {
    __shared__ float red[16][32];
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const int c = blockIdx.x * 32 + tx;
    void *out = blockIdx.y ? dshift : dgain;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (!out) return;
    float s = 0.0f;
    if (c < cols) {
        // All of a thread's loads in flight at once (two blocks per SM leave 304
        // parts, 19 for each thread): 4.2 us for 1024 sums, 6.7 us in batches of 8.
#pragma unroll 1
        for (int i0 = ty; i0 < parts; i0 += 16 * 20) {
            float v[20];
#pragma unroll
            for (int u = 0; u < 20; ++u) {
                const int i = i0 + 16 * u;
                v[u] = i < parts ? part[((int64_t)2 * i + blockIdx.y) * part_cols + c + ((lead + i * lead_step) & 7)] : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < 20; ++u) s += v[u];
        }
    }
    red[ty][tx] = s;
    __syncthreads();
    if (ty || c >= cols) return;
    for (int i = 1; i < 16; ++i) s += red[i][tx];
    store_from_float(out, c, dtype, s);
}

// ---------------------------------------------------------------- any width, any strides
// Rows too wide for registers and matrices whose columns are not contiguous:
// a block per row, the row read again for each pass (from L2 mostly).
__global__ void __launch_bounds__(1024) layer_norm_any_kernel(const NormArgs a) {
    __shared__ __align__(16) BlockSums sums;
    Summer block_sum{&sums};
    const MatRef &x = a.x, &y = a.y;
    const int64_t r = blockIdx.x, cols = a.cols;
    ptx::grid_dependency_wait();
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += (int)blockDim.x) s += a.scale * load_as_float(x.p, r * x.rs + c * x.cs, x.dtype);
    const float mean = block_sum(s) / (float)cols;
    s = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += (int)blockDim.x) {
        const float d = a.scale * load_as_float(x.p, r * x.rs + c * x.cs, x.dtype) - mean;
        s += d * d;
    }
    const float rstd = rsqrtf(block_sum(s) / (float)cols + a.eps);
    for (int64_t c = threadIdx.x; c < cols; c += (int)blockDim.x) {
        const float d = a.scale * load_as_float(x.p, r * x.rs + c * x.cs, x.dtype) - mean;
        const float g = a.gain ? load_as_float(a.gain, c, a.param_dtype) : 1.0f;
        const float b = a.shift ? load_as_float(a.shift, c, a.param_dtype) : 0.0f;
        store_from_float((void *)y.p, r * y.rs + c * y.cs, y.dtype, d * rstd * g + b);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
    }
}

__global__ void __launch_bounds__(1024) layer_norm_dx_any_kernel(const NormGradArgs a) {
    __shared__ __align__(16) BlockSums sums;
    Summer block_sum{&sums};
    const MatRef &x = a.x, &dy = a.dy, &res = a.res, &dx = a.dx;
    const int64_t r = blockIdx.x, cols = a.cols;
    ptx::grid_dependency_wait();
    const float mu = a.mean[r], rs = a.rstd[r];
    float st = 0.0f, stn = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += (int)blockDim.x) {
        const float n = (load_as_float(x.p, r * x.rs + c * x.cs, x.dtype) - mu) * rs;
        const float t = load_as_float(dy.p, r * dy.rs + c * dy.cs, dy.dtype) *
                        (a.gain ? load_as_float(a.gain, c, a.param_dtype) : 1.0f);
        st += t;
        stn += t * n;
    }
    const float2 s = block_sum(st, stn);
    st = s.x / (float)cols;
    stn = s.y / (float)cols;
    for (int64_t c = threadIdx.x; c < cols; c += (int)blockDim.x) {
        const float n = (load_as_float(x.p, r * x.rs + c * x.cs, x.dtype) - mu) * rs;
        const float t = load_as_float(dy.p, r * dy.rs + c * dy.cs, dy.dtype) *
                        (a.gain ? load_as_float(a.gain, c, a.param_dtype) : 1.0f);
        float d = rs * (t - st - n * stn);
        if (res.p) d += load_as_float(res.p, r * res.rs + c * res.cs, res.dtype);
        store_from_float((void *)dx.p, r * dx.rs + c * dx.cs, dx.dtype, d);
    }
}

// Column sums of dy * n and dy over this block's rows: 32 columns, 8 rows at
// a time.
__global__ void __launch_bounds__(kThreads) layer_norm_params_any_kernel(const NormGradArgs a, int64_t rows_per_block) {
    __shared__ float sg_red[8][32], sb_red[8][32];
    const MatRef &x = a.x, &dy = a.dy;
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;
    const int64_t r0 = (int64_t)blockIdx.y * rows_per_block;
    const int64_t r1 = r0 + rows_per_block < a.rows ? r0 + rows_per_block : a.rows;
    ptx::grid_dependency_wait();
    float sg = 0.0f, sb = 0.0f;
    if (c < a.cols)
        for (int64_t r = r0 + ty; r < r1; r += 8) {
            const float d = load_as_float(dy.p, r * dy.rs + c * dy.cs, dy.dtype);
            sg += d * ((load_as_float(x.p, r * x.rs + c * x.cs, x.dtype) - a.mean[r]) * a.rstd[r]);
            sb += d;
        }
    sg_red[ty][tx] = sg;
    sb_red[ty][tx] = sb;
    __syncthreads();
    if (ty == 0 && c < a.cols) {
        for (int i = 1; i < 8; ++i) {
            sg += sg_red[i][tx];
            sb += sb_red[i][tx];
        }
        float *p = a.part + (int64_t)blockIdx.y * 2 * a.part_cols;
        p[c] = sg;
        p[a.part_cols + c] = sb;
    }
}

// ---------------------------------------------------------------- launches
bool unit_columns(const MatRef &m) { return !m.p || m.cs <= 1; }

// Lead of a matrix's rows: 8 values for the rows modulo 8, as base and step.
struct Lead {
    int64_t base, step;
};
Lead lead_of_rows(const MatRef &m) {
    const int64_t size = channel_elem_size(m.dtype);
    return {(int64_t)((uintptr_t)m.p / (uintptr_t)size & 7), m.rs & 7};
}

// Whether the rows of all matrices (those given) have one lead.
bool one_lead(std::initializer_list<const MatRef *> all) {
    const Lead l = lead_of_rows(**all.begin());
    for (const MatRef *m : all) {
        if (!m->p) continue;
        const Lead k = lead_of_rows(*m);
        if (k.base != l.base || k.step != l.step) return false;
    }
    return true;
}

// Whether an output row can be turned in shared memory.
bool turnable(int64_t cols, int32_t out_dtype) {
    const int64_t rows = cols <= 1024 ? 8 : 1;
    return rows * turn_elems((int)std::min<int64_t>(cols, 1 << 20)) * channel_elem_size(out_dtype) <= 40 << 10;
}

// How rows are held: by a warp up to 64 groups of 8 (128 in the forward
// pass), else by a block of `threads`, nv groups each.
struct RowShape {
    int nv = 0, threads = 0;  // nv == 0: not in registers
    bool warp = false, vec = false;
};

RowShape row_shape(int64_t cols, const MatRef &x, bool vec, bool grad) {
    RowShape s;
    s.vec = vec;
    const Lead l = lead_of_rows(x);
    const bool aligned = l.base == 0 && l.step == 0;
    const int64_t groups = vec && !aligned ? (cols + 14) / 8 : (cols + 7) / 8;
    if (groups <= (grad ? 64 : 128)) {
        s.warp = true;
        s.threads = 256;
        s.nv = groups <= 32 ? 1 : groups <= 64 ? 2 : 4;
        return s;
    }
    for (int nv = grad ? 1 : 2; nv <= (vec ? 4 : 2); nv *= 2) {
        const int64_t threads = round_up((groups + nv - 1) / nv, 32);
        if (threads <= (grad ? grad_threads(nv) : norm_threads(nv))) {
            s.nv = nv;
            s.threads = (int)threads;
            return s;
        }
    }
    return s;
}

// Blocks for `rows` rows: all at once, or a multiple of 8 that fills the GPU
// (so that a block's rows share their lead).
int64_t row_blocks(int64_t rows, const RowShape &sh, int per_sm, int64_t limit) {
    const int64_t blocks = sh.warp ? (rows + 7) / 8 : rows;
    const int64_t most = std::min<int64_t>((int64_t)device_sm_count() * per_sm, limit) / 8 * 8;
    return std::min(blocks, std::max<int64_t>(most, 8));
}

// A launch with more than 48 KB of shared memory.
template <auto kKernel, typename Args>
bool launch_large(dim3 grid, int threads, size_t smem, cudaStream_t s, const Args &a) {
    static std::atomic<bool> ready[64];  // (check_device admits 64 devices)
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (!ready[dev].load()) {
        if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 << 10) != cudaSuccess) return false;
        ready[dev].store(true);
    }
    return launch_behind(kKernel, grid, threads, smem, s, a);
}

template <typename X, typename Y>
bool launch_norm(const NormArgs &a, const RowShape &sh, unsigned grid, cudaStream_t s) {
    const size_t smem = (sh.nv == 4 ? (size_t)sh.threads * 256 : 0) +
                        (a.turn ? (size_t)turn_elems(a.cols) * sizeof(Y) * (sh.warp ? 8 : 1) : 0);
    if (sh.nv == 4)
        return sh.warp ? launch_large<layer_norm_rows_kernel<X, Y, 4, true>>(dim3(grid), sh.threads, smem, s, a)
                       : launch_large<layer_norm_rows_kernel<X, Y, 4, false>>(dim3(grid), sh.threads, smem, s, a);
    if (!sh.warp) return launch_behind(layer_norm_rows_kernel<X, Y, 2, false>, dim3(grid), sh.threads, smem, s, a);
    return sh.nv == 1 ? launch_behind(layer_norm_rows_kernel<X, Y, 1, true>, dim3(grid), sh.threads, smem, s, a)
                      : launch_behind(layer_norm_rows_kernel<X, Y, 2, true>, dim3(grid), sh.threads, smem, s, a);
}

template <typename X>
bool launch_norm_to(const NormArgs &a, const RowShape &sh, unsigned grid, cudaStream_t s) {
    switch (a.y.dtype) {
        case CONV_FLOAT32: return launch_norm<X, float>(a, sh, grid, s);
        case CONV_FLOAT16: return launch_norm<X, __half>(a, sh, grid, s);
        default: return launch_norm<X, __nv_bfloat16>(a, sh, grid, s);
    }
}

template <typename X>
bool launch_norm_grad(const NormGradArgs &a, const RowShape &sh, unsigned grid, cudaStream_t s) {
    const size_t gain = sh.nv <= 2 ? (size_t)sh.nv * sh.threads * 32 : 0;
    const size_t ring = sh.vec && sh.nv <= 2 ? (size_t)kDepth<X> * (a.res.p ? 3 : 2) * sh.nv * 8 * sizeof(X) * sh.threads : 0;
    const size_t turn = a.turn ? (size_t)turn_elems(a.cols) * sizeof(X) * (sh.warp ? 8 : 1) : 0;
    const size_t smem = std::max(gain + ring + turn, sh.warp && a.part ? (size_t)a.cols * 64 : 0);
#define I8C_NORM(NV, W)                                                                                        \
    (sh.vec ? launch_large<layer_norm_grad_rows_kernel<X, NV, true, W>>(dim3(grid), sh.threads, smem, s, a)    \
            : launch_behind(layer_norm_grad_rows_kernel<X, NV, false, W>, dim3(grid), sh.threads, smem, s, a))
    if (sh.warp) return sh.nv == 1 ? I8C_NORM(1, true) : I8C_NORM(2, true);
    if (sh.nv <= 2) return sh.nv == 1 ? I8C_NORM(1, false) : I8C_NORM(2, false);
    return launch_behind(layer_norm_grad_rows_kernel<X, 4, true, false>, dim3(grid), sh.threads, smem, s, a);
#undef I8C_NORM
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

// Partial sums of dgain and dshift: one set per block of the row kernels, at
// most kMaxParts of them whatever the device.
constexpr int64_t kMaxParts = 608;  // four blocks on each of 152 SMs

// (room for a lead and for whole groups)
int64_t part_columns(int64_t cols) { return round_up(cols, 8) + 8; }

size_t norm_grad_bytes(int64_t rows, int64_t cols) {
    if (rows == 0) return 0;
    return (size_t)round_up(std::min(kMaxParts, rows) * 2 * part_columns(cols) * 4, 256);
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
    NormArgs a;
    a.x = mat_ref(x, x_dev), a.y = mat_ref(y, y_dev);
    a.gain = gain_dev, a.shift = shift_dev;
    a.mean = mean_dev, a.rstd = rstd_dev;
    a.rows = rows, a.cols = (int32_t)cols;
    a.eps = p->eps, a.scale = p->scale, a.param_dtype = p->param_dtype;
    const cudaStream_t s = (cudaStream_t)stream;
    a.turn = !one_lead({&a.x, &a.y});
    // (rows too wide to be turned are too wide for an element per access too)
    const RowShape sh = a.turn && !turnable(cols, y->dtype) ? RowShape() : row_shape(cols, a.x, true, false);
    bool ok;
    if (sh.nv == 0 || !unit_columns(a.x) || !unit_columns(a.y)) {
        ok = launch_behind(layer_norm_any_kernel, dim3((unsigned)rows), cols > 4096 ? 1024 : 256, 0, s, a);
    } else {
        const unsigned grid = (unsigned)row_blocks(rows, sh, (sh.nv == 4 ? 512 : sh.warp ? 1024 : 768) / sh.threads, INT32_MAX);
        switch (x->dtype) {
            case CONV_FLOAT32: ok = launch_norm_to<float>(a, sh, grid, s); break;
            case CONV_FLOAT16: ok = launch_norm_to<__half>(a, sh, grid, s); break;
            case CONV_BFLOAT16: ok = launch_norm_to<__nv_bfloat16>(a, sh, grid, s); break;
            default: ok = launch_norm_to<int32_t>(a, sh, grid, s); break;
        }
    }
    return ok ? CONV_OK : CONV_ERR_CUDA;
}

conv_status conv_layer_norm_grad_workspace_size(const conv_matrix_desc *x, size_t *bytes) {
    if (!x || !bytes) return CONV_ERR_NULL_PTR;
    conv_status st = check_matrix(x);
    if (st) return st;
    if (!is_float_type(x->dtype)) return CONV_ERR_DTYPE;
    if (x->cols < 1) return CONV_ERR_BAD_PARAM;
    *bytes = norm_grad_bytes(x->rows, x->cols);
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
    const size_t need = norm_grad_bytes(rows, cols);
    if (need) {
        if (!workspace || workspace_bytes < need || (uintptr_t)workspace % 256) return CONV_ERR_WORKSPACE;
        for (int i = 0; i < 4; ++i)
            if (all[i] && overlaps(workspace, need, all_dev[i], matrix_extent_bytes(all[i])))
                return CONV_ERR_OVERLAP;
        const void *vec[] = {gain_dev, dgain_dev, dshift_dev, mean_dev, rstd_dev};
        for (int i = 0; i < 5; ++i)
            if (overlaps(workspace, need, vec[i], i < 3 ? cols * psize : rows * 4)) return CONV_ERR_OVERLAP;
    }
    if ((st = check_device())) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    if (rows == 0) {
        for (void *g : grads)
            if (g && cudaMemsetAsync(g, 0, (size_t)(cols * psize), s) != cudaSuccess) return CONV_ERR_CUDA;
        return CONV_OK;
    }
    NormGradArgs a;
    a.dy = mat_ref(dy, dy_dev), a.x = mat_ref(x, x_dev);
    a.res = mat_ref(residual_grad, residual_grad_dev), a.dx = mat_ref(dx, dx_dev);
    a.gain = gain_dev, a.mean = mean_dev, a.rstd = rstd_dev;
    a.part = dgain_dev || dshift_dev ? (float *)workspace : nullptr;
    a.rows = rows, a.cols = (int32_t)cols, a.param_dtype = p->param_dtype;
    a.part_cols = (int32_t)part_columns(cols);
    Lead lead{0, 0};  // of the blocks' sums
    const RowShape sh = row_shape(cols, a.x, one_lead({&a.x, &a.dy, &a.res}) &&
                                                 (one_lead({&a.x, &a.dx}) || turnable(cols, x->dtype)), true);
    a.turn = !one_lead({&a.x, &a.dx});
    int64_t parts;
    bool ok = true;
    if (sh.nv == 0 || !unit_columns(a.dy) || !unit_columns(a.x) || !unit_columns(a.res) || !unit_columns(a.dx)) {
        if (dx) ok = launch_behind(layer_norm_dx_any_kernel, dim3((unsigned)rows), cols > 4096 ? 1024 : 256, 0, s, a);
        const int64_t per = round_up((rows + 255) / 256, 8);
        parts = (rows + per - 1) / per;
        if (a.part)
            ok = ok && launch_behind(layer_norm_params_any_kernel, dim3((unsigned)((cols + 31) / 32), (unsigned)parts),
                                     kThreads, 0, s, a, per);
    } else {
        const int per_sm = sh.warp ? (sh.nv == 1 ? 3 : 2) : grad_threads(sh.nv) * grad_blocks(sh.nv) / sh.threads;
        parts = row_blocks(rows, sh, per_sm, kMaxParts);
        if (sh.vec && !sh.warp) lead = lead_of_rows(a.x);
        switch (x->dtype) {
            case CONV_FLOAT32: ok = launch_norm_grad<float>(a, sh, (unsigned)parts, s); break;
            case CONV_FLOAT16: ok = launch_norm_grad<__half>(a, sh, (unsigned)parts, s); break;
            default: ok = launch_norm_grad<__nv_bfloat16>(a, sh, (unsigned)parts, s); break;
        }
    }
    if (ok && a.part)
        ok = launch_behind(layer_norm_params_sum_kernel, dim3((unsigned)((cols + 31) / 32), 2), 512, 0, s,
                           (const float *)workspace, (int)parts, (int)cols, (int)a.part_cols, (int)lead.base,
                           (int)lead.step, dgain_dev, dshift_dev, p->param_dtype);
    return ok ? CONV_OK : CONV_ERR_CUDA;
}

}  // extern "C"

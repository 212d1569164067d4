// layer_norm.cu -- conv_layer_norm and conv_layer_norm_grad.
#include <cuda_runtime.h>

#include <algorithm>
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

// Sums of two values over the block, the same in every thread.
__device__ __forceinline__ float2 block_sum2(float u, float v, float2 *red) {
    const int warps = blockDim.x / 32;
    u = warp_sum(u);
    v = warp_sum(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = make_float2(u, v);
    __syncthreads();
    const float2 mine = threadIdx.x % 32 < warps ? red[threadIdx.x % 32] : make_float2(0.0f, 0.0f);
    return make_float2(warp_sum(mine.x), warp_sum(mine.y));
}

__device__ __forceinline__ float block_sum(float v, float2 *red) { return block_sum2(v, 0.0f, red).x; }

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
// row.  This wants one lead for all matrices of a call.  Otherwise thread t
// holds elements t, t + T, ..., one per access.
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
            for (int j = 0; j < 4; ++j) w[j] = bits16(v[2 * j], p) | bits16(v[2 * j + 1], p) << 16;
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

// 8 values of a parameter vector (any alignment; absent or outside: `fill`).
template <bool kVec>
__device__ __forceinline__ void load_params(const void *p, int32_t dtype, float fill, const Place<kVec> &at, int i,
                                            float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = at.column(i, j);
        v[j] = p && at.inside(c) ? load_as_float(p, c, dtype) : fill;
    }
}

template <bool kWarp>
__device__ __forceinline__ float row_sum(float v, float2 *red) {
    if constexpr (kWarp) return warp_sum(v);
    else return block_sum(v, red);
}

// Threads of a block that holds a row in kNv groups per thread, as registers
// allow; an SM takes as many blocks as fit that many threads.
constexpr int max_threads(int nv) { return nv == 1 ? 640 : 512; }

struct NormArgs {
    MatRef x, y;
    const void *gain, *shift;
    float *mean, *rstd;
    int64_t rows;
    int32_t cols;
    float eps, scale;
    int32_t param_dtype;
};

template <typename X, typename Y, int kNv, bool kVec, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 256 : max_threads(kNv)) layer_norm_rows_kernel(const NormArgs a) {
    __shared__ float2 red[32];
    const int64_t first = kWarp ? (int64_t)blockIdx.x * 8 + threadIdx.x / 32 : blockIdx.x;
    const int64_t step = kWarp ? (int64_t)gridDim.x * 8 : gridDim.x;
    const X *x = (const X *)a.x.p;
    Y *y = (Y *)const_cast<void *>(a.y.p);
    Place<kVec> at;
    at.t = kWarp ? threadIdx.x % 32 : threadIdx.x;
    at.threads = kWarp ? 32 : blockDim.x;
    at.cols = a.cols;
    at.lead = kVec ? lead_of(x + first * a.x.rs) : 0;
    const float per = 1.0f / (float)a.cols;
    constexpr bool kKeep = kNv <= 2;  // parameters in registers over the rows
    float gain[kKeep ? kNv : 1][8], shift[kKeep ? kNv : 1][8];
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if constexpr (kKeep) {
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            load_params(a.gain, a.param_dtype, 1.0f, at, i, gain[i]);
            load_params(a.shift, a.param_dtype, 0.0f, at, i, shift[i]);
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
        const float mean = row_sum<kWarp>(s, red) * per;
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
        const float rstd = rsqrtf(row_sum<kWarp>(s, red) * per + a.eps);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            if constexpr (kKeep) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * gain[i][j] + shift[i][j];
            } else {
                load_params(a.gain, a.param_dtype, 1.0f, at, i, gain[0]);
                load_params(a.shift, a.param_dtype, 0.0f, at, i, shift[0]);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * gain[0][j] + shift[0][j];
            }
            store_group(y + r * a.y.rs, at, i, v[i]);
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
    float *part;  // [blocks][2][cols], or NULL
    int64_t rows;
    int32_t cols;
    int32_t param_dtype;
};

// dx of every row and this block's partial sums of dy * n and dy, in
// registers over its rows.
template <typename X, int kNv, bool kVec, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 256 : max_threads(kNv), kWarp ? 2 : 1)
    layer_norm_grad_rows_kernel(const NormGradArgs a) {
    __shared__ float2 red[32];
    // the gain, placed so that a thread's group is 32 aligned bytes (kWarp:
    // as it is, since the warps' rows have different leads), if kKeep;
    // kWarp: [8 warps][2][cols] sums, after the rows
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
    constexpr bool kAhead = kNv * (kIs16<X> ? 1 : 2) <= 2;  // next row's loads in flight during this one
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int shift = kWarp ? 0 : at.lead;
    if constexpr (kKeep) {
        for (int c = threadIdx.x; c < (kWarp ? a.cols : kNv * at.threads * 8); c += blockDim.x) {
            const int col = c - shift;
            shared[c] = a.gain && at.inside(col) ? load_as_float(a.gain, col, a.param_dtype) : 1.0f;
        }
        __syncthreads();
    }
    auto load_gain = [&](int i, float (&g)[8]) {
        if constexpr (kKeep && kVec) {
            const int c = at.column(i, 0) + shift;
            if (!kWarp || ((at.lead & 3) == 0 && at.whole(i))) {
                const float4 u = *reinterpret_cast<const float4 *>(shared + c), v = *reinterpret_cast<const float4 *>(shared + c + 4);
                g[0] = u.x, g[1] = u.y, g[2] = u.z, g[3] = u.w, g[4] = v.x, g[5] = v.y, g[6] = v.z, g[7] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = at.inside(c + j) ? shared[c + j] : 1.0f;
            }
        } else if constexpr (kKeep) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = at.column(i, j);
                g[j] = at.inside(c) ? shared[c] : 1.0f;
            }
        } else {
            load_params(a.gain, a.param_dtype, 1.0f, at, i, g);
        }
    };
    float dg[kNv][8] = {}, db[kNv][8] = {};
    Group<X> nx[kNv], ny[kNv], nr[kNv];
    float mu = 0.0f, rs = 0.0f;
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            load_group(x + r * a.x.rs, at, i, nx[i]);
            load_group(dy + r * a.dy.rs, at, i, ny[i]);
            if (res) load_group(res + r * a.res.rs, at, i, nr[i]);
        }
        mu = a.mean[r];
        rs = a.rstd[r];
    };
    if (kAhead && first < a.rows) fetch(first);
    for (int64_t r = first; r < a.rows; r += step) {
        if (!kAhead) fetch(r);
        Group<X> gx[kNv], gy[kNv], gr[kNv];
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            gx[i] = nx[i];
            gy[i] = ny[i];
            gr[i] = nr[i];
        }
        const float m = mu, rr = rs;
        if (kAhead && r + step < a.rows) fetch(r + step);
        float st = 0.0f, stn = 0.0f;
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            float gain[8];
            load_gain(i, gain);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // (outside the row dy is 0, and so is every term)
                const float d = element(gy[i], j), n = (element(gx[i], j) - m) * rr;
                const float u = d * gain[j];
                st += u;
                stn += u * n;
                dg[i][j] += d * n;
                db[i][j] += d;
            }
        }
        if (!dx) continue;
        if constexpr (kWarp) {
            st = warp_sum(st);
            stn = warp_sum(stn);
        } else {
            const float2 s = block_sum2(st, stn, red);
            st = s.x, stn = s.y;
        }
        st *= per;
        stn *= per;
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            float v[8], gain[8];
            load_gain(i, gain);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = (element(gx[i], j) - m) * rr;
                v[j] = rr * (element(gy[i], j) * gain[j] - st - n * stn);
                if (res) v[j] += element(gr[i], j);
            }
            store_group(dx + r * a.dx.rs, at, i, v);
        }
    }
    if (!a.part) return;
    float *part = a.part + (int64_t)blockIdx.x * 2 * a.cols;
    if constexpr (kWarp) __syncthreads();  // the gain is no longer read
    float *mine = kWarp ? shared + threadIdx.x / 32 * 2 * a.cols : part;
#pragma unroll
    for (int i = 0; i < kNv; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = at.column(i, j);
            if (at.inside(c)) {
                mine[c] = dg[i][j];
                mine[a.cols + c] = db[i][j];
            }
        }
    if constexpr (kWarp) {
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * a.cols; c += 256) {
            float s = shared[c];
#pragma unroll
            for (int w = 1; w < 8; ++w) s += shared[w * 2 * a.cols + c];
            part[c] = s;
        }
    }
}

// Adds the blocks' partial sums: 32 columns per block, 32 threads per column.
__global__ void __launch_bounds__(1024) layer_norm_params_sum_kernel(const float *part, int64_t parts, int64_t cols,
                                                                     void *dgain, void *dshift, int32_t dtype) {
    __shared__ float red[32][33];
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;
    ptx::grid_dependency_wait();
    float s = 0.0f;
    if (c < 2 * cols)
        for (int64_t i = ty; i < parts; i += 32) s += part[i * 2 * cols + c];
    red[ty][tx] = s;
    __syncthreads();
    const int64_t cc = (int64_t)blockIdx.x * 32 + ty;
    s = warp_sum(red[tx][ty]);
    if (tx == 0 && cc < 2 * cols) {
        void *out = cc < cols ? dgain : dshift;
        if (out) store_from_float(out, cc < cols ? cc : cc - cols, dtype, s);
    }
}

// ---------------------------------------------------------------- any width, any strides
// Rows too wide for registers and matrices whose columns are not contiguous:
// a block per row, the row read again for each pass (from L2 mostly).
__global__ void __launch_bounds__(1024) layer_norm_any_kernel(const NormArgs a) {
    __shared__ float2 red[32];
    const MatRef &x = a.x, &y = a.y;
    const int64_t r = blockIdx.x, cols = a.cols;
    ptx::grid_dependency_wait();
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += (int)blockDim.x) s += a.scale * load_as_float(x.p, r * x.rs + c * x.cs, x.dtype);
    const float mean = block_sum(s, red) / (float)cols;
    s = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += (int)blockDim.x) {
        const float d = a.scale * load_as_float(x.p, r * x.rs + c * x.cs, x.dtype) - mean;
        s += d * d;
    }
    const float rstd = rsqrtf(block_sum(s, red) / (float)cols + a.eps);
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
    __shared__ float2 red[32];
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
    const float2 s = block_sum2(st, stn, red);
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
        float *p = a.part + (int64_t)blockIdx.y * 2 * a.cols;
        p[c] = sg;
        p[a.cols + c] = sb;
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

// How rows are held: by a warp up to 64 groups of 8, else by a block of
// `threads`, nv groups each.
struct RowShape {
    int nv = 0, threads = 0;  // nv == 0: not in registers
    bool warp = false, vec = false;
};

RowShape row_shape(int64_t cols, const MatRef &x, bool vec) {
    RowShape s;
    s.vec = vec;
    const Lead l = lead_of_rows(x);
    const bool aligned = l.base == 0 && l.step == 0;
    const int64_t groups = vec && !aligned ? (cols + 14) / 8 : (cols + 7) / 8;
    if (groups <= 64) {
        s.warp = true;
        s.threads = 256;
        s.nv = groups <= 32 ? 1 : 2;
        return s;
    }
    for (int nv = 1; nv <= (vec ? 4 : 2); nv *= 2) {
        const int64_t threads = round_up((groups + nv - 1) / nv, 32);
        if (threads <= max_threads(nv)) {
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

template <typename X, typename Y>
bool launch_norm(const NormArgs &a, const RowShape &sh, unsigned grid, cudaStream_t s) {
#define I8C_NORM(NV, W)                                                                                       \
    (sh.vec ? launch_behind(layer_norm_rows_kernel<X, Y, NV, true, W>, dim3(grid), sh.threads, 0, s, a)          \
         : launch_behind(layer_norm_rows_kernel<X, Y, NV, false, W>, dim3(grid), sh.threads, 0, s, a))
    if (sh.warp) return sh.nv == 1 ? I8C_NORM(1, true) : I8C_NORM(2, true);
    if (sh.nv <= 2) return sh.nv == 1 ? I8C_NORM(1, false) : I8C_NORM(2, false);
    return launch_behind(layer_norm_rows_kernel<X, Y, 4, true, false>, dim3(grid), sh.threads, 0, s, a);
#undef I8C_NORM
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
    const size_t smem = sh.warp ? (size_t)a.cols * (a.part ? 64 : 4) : sh.nv <= 2 ? (size_t)sh.nv * sh.threads * 32 : 0;
#define I8C_NORM(NV, W)                                                                                        \
    (sh.vec ? launch_behind(layer_norm_grad_rows_kernel<X, NV, true, W>, dim3(grid), sh.threads, smem, s, a)      \
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

size_t norm_grad_bytes(int64_t rows, int64_t cols) {
    if (rows == 0) return 0;
    return (size_t)round_up(std::min(kMaxParts, rows) * 2 * cols * 4, 256);
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
    const RowShape sh = row_shape(cols, a.x, one_lead({&a.x, &a.y}));
    bool ok;
    if (sh.nv == 0 || !unit_columns(a.x) || !unit_columns(a.y)) {
        ok = launch_behind(layer_norm_any_kernel, dim3((unsigned)rows), cols > 4096 ? 1024 : 256, 0, s, a);
    } else {
        const unsigned grid = (unsigned)row_blocks(rows, sh, std::max(1, 1024 / sh.threads), INT32_MAX);
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
    const RowShape sh = row_shape(cols, a.x, one_lead({&a.x, &a.dy, &a.res, &a.dx}));
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
        parts = row_blocks(rows, sh, sh.warp ? 2 : std::max(1, max_threads(sh.nv) / sh.threads), kMaxParts);
        switch (x->dtype) {
            case CONV_FLOAT32: ok = launch_norm_grad<float>(a, sh, (unsigned)parts, s); break;
            case CONV_FLOAT16: ok = launch_norm_grad<__half>(a, sh, (unsigned)parts, s); break;
            default: ok = launch_norm_grad<__nv_bfloat16>(a, sh, (unsigned)parts, s); break;
        }
    }
    if (ok && a.part)
        ok = launch_behind(layer_norm_params_sum_kernel, dim3((unsigned)((2 * cols + 31) / 32)), 1024, 0, s,
                           (const float *)workspace, parts, cols, dgain_dev, dshift_dev, p->param_dtype);
    return ok ? CONV_OK : CONV_ERR_CUDA;
}

}  // extern "C"

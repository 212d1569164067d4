// layer_norm.cu -- conv_layer_norm and conv_layer_norm_grad.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
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
// registers.  kVec: aligned rows of a multiple of 8 elements, in groups of 8
// (one 16-byte vector of a 16-bit type, two of a 32-bit one); otherwise
// thread t holds elements t, t + T, ... and every access is one element wide,
// which still makes whole runs per warp.
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

// Group i of the row that starts at p (element stride 1): T threads to the row.
template <bool kVec, typename T>
__device__ __forceinline__ void load_group(const T *p, int i, int t, int threads, int cols, Group<T> &g) {
    if constexpr (kVec) {
        const int c = (i * threads + t) * 8;
        if (c < cols) {
            const uint4 a = *reinterpret_cast<const uint4 *>(p + c);
            g.w[0] = a.x, g.w[1] = a.y, g.w[2] = a.z, g.w[3] = a.w;
            if constexpr (!kIs16<T>) {
                const uint4 b = *reinterpret_cast<const uint4 *>(p + c + 4);
                g.w[4] = b.x, g.w[5] = b.y, g.w[6] = b.z, g.w[7] = b.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < (kIs16<T> ? 4 : 8); ++j) g.w[j] = 0;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = (i * 8 + j) * threads + t;
            if constexpr (kIs16<T>) {
                const uint32_t v = c < cols ? reinterpret_cast<const uint16_t *>(p)[c] : 0u;
                if (j % 2) g.w[j / 2] |= v << 16;
                else g.w[j / 2] = v;
            } else {
                g.w[j] = c < cols ? reinterpret_cast<const uint32_t *>(p)[c] : 0u;
            }
        }
    }
}

template <bool kVec>
__device__ __forceinline__ int column(int i, int j, int t, int threads) {
    return kVec ? (i * threads + t) * 8 + j : (i * 8 + j) * threads + t;
}

template <bool kVec, typename T>
__device__ __forceinline__ void store_group(T *p, int i, int t, int threads, int cols, const float (&v)[8]) {
    if constexpr (kVec) {
        const int c = (i * threads + t) * 8;
        if (c >= cols) return;
        if constexpr (kIs16<T>) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = bits16(v[2 * j], p) | bits16(v[2 * j + 1], p) << 16;
            *reinterpret_cast<uint4 *>(p + c) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            *reinterpret_cast<float4 *>(p + c) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(p + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = column<false>(i, j, t, threads);
            if (c >= cols) continue;
            if constexpr (kIs16<T>) reinterpret_cast<uint16_t *>(p)[c] = (uint16_t)bits16(v[j], p);
            else p[c] = v[j];
        }
    }
}

// 8 values of a parameter vector (any alignment; absent: `fill`).
template <bool kVec>
__device__ __forceinline__ void load_params(const void *p, int32_t dtype, float fill, int i, int t, int threads, int cols,
                                            float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = column<kVec>(i, j, t, threads);
        v[j] = p && c < cols ? load_as_float(p, c, dtype) : fill;
    }
}

template <bool kWarp>
__device__ __forceinline__ float row_sum(float v, float2 *red) {
    if constexpr (kWarp) return warp_sum(v);
    else return block_sum(v, red);
}

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
__global__ void __launch_bounds__(kWarp ? 256 : 512) layer_norm_rows_kernel(const NormArgs a) {
    __shared__ float2 red[32];
    const int threads = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x % 32 : threadIdx.x;
    const int64_t first = kWarp ? (int64_t)blockIdx.x * 8 + threadIdx.x / 32 : blockIdx.x;
    const int64_t step = kWarp ? (int64_t)gridDim.x * 8 : gridDim.x;
    const float per = 1.0f / (float)a.cols;
    constexpr bool kKeep = kNv <= 2;  // parameters in registers over the rows
    float gain[kKeep ? kNv : 1][8], shift[kKeep ? kNv : 1][8];
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if constexpr (kKeep) {
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            load_params<kVec>(a.gain, a.param_dtype, 1.0f, i, t, threads, a.cols, gain[i]);
            load_params<kVec>(a.shift, a.param_dtype, 0.0f, i, t, threads, a.cols, shift[i]);
        }
    }
    const X *x = (const X *)a.x.p;
    Y *y = (Y *)const_cast<void *>(a.y.p);
    Group<X> next[kNv];
    if (first < a.rows) {
#pragma unroll
        for (int i = 0; i < kNv; ++i) load_group<kVec>(x + first * a.x.rs, i, t, threads, a.cols, next[i]);
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
            for (int i = 0; i < kNv; ++i) load_group<kVec>(x + (r + step) * a.x.rs, i, t, threads, a.cols, next[i]);
        }
        const float mean = row_sum<kWarp>(s, red) * per;
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < kNv; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] -= mean;
                if (column<kVec>(i, j, t, threads) < a.cols) s += v[i][j] * v[i][j];
            }
        const float rstd = rsqrtf(row_sum<kWarp>(s, red) * per + a.eps);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            if constexpr (kKeep) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * gain[i][j] + shift[i][j];
            } else {
                load_params<kVec>(a.gain, a.param_dtype, 1.0f, i, t, threads, a.cols, gain[0]);
                load_params<kVec>(a.shift, a.param_dtype, 0.0f, i, t, threads, a.cols, shift[0]);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * gain[0][j] + shift[0][j];
            }
            store_group<kVec>(y + r * a.y.rs, i, t, threads, a.cols, v[i]);
        }
        if (t == 0) {
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
__global__ void __launch_bounds__(kWarp ? 256 : 512) layer_norm_grad_rows_kernel(const NormGradArgs a) {
    __shared__ float2 red[32];
    extern __shared__ float sums[];  // kWarp: [2][cols]
    const int threads = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x % 32 : threadIdx.x;
    const int64_t first = kWarp ? (int64_t)blockIdx.x * 8 + threadIdx.x / 32 : blockIdx.x;
    const int64_t step = kWarp ? (int64_t)gridDim.x * 8 : gridDim.x;
    const float per = 1.0f / (float)a.cols;
    constexpr bool kKeep = kNv <= 2;
    constexpr bool kAhead = kNv * (kIs16<X> ? 1 : 2) <= 2;  // next row's loads in flight during this one
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    float gain[kKeep ? kNv : 1][8];
    if constexpr (kKeep) {
#pragma unroll
        for (int i = 0; i < kNv; ++i) load_params<kVec>(a.gain, a.param_dtype, 1.0f, i, t, threads, a.cols, gain[i]);
    }
    float dg[kNv][8] = {}, db[kNv][8] = {};
    const X *x = (const X *)a.x.p, *dy = (const X *)a.dy.p, *res = (const X *)a.res.p;
    X *dx = (X *)const_cast<void *>(a.dx.p);
    Group<X> nx[kNv], ny[kNv], nr[kNv];
    float mu = 0.0f, rs = 0.0f;
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            load_group<kVec>(x + r * a.x.rs, i, t, threads, a.cols, nx[i]);
            load_group<kVec>(dy + r * a.dy.rs, i, t, threads, a.cols, ny[i]);
            if (res) load_group<kVec>(res + r * a.res.rs, i, t, threads, a.cols, nr[i]);
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
            if constexpr (!kKeep) load_params<kVec>(a.gain, a.param_dtype, 1.0f, i, t, threads, a.cols, gain[0]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // (outside the row dy is 0, and so is every term)
                const float d = element(gy[i], j), n = (element(gx[i], j) - m) * rr;
                const float u = d * gain[kKeep ? i : 0][j];
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
            float v[8];
            if constexpr (!kKeep) load_params<kVec>(a.gain, a.param_dtype, 1.0f, i, t, threads, a.cols, gain[0]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = (element(gx[i], j) - m) * rr;
                v[j] = rr * (element(gy[i], j) * gain[kKeep ? i : 0][j] - st - n * stn);
                if (res) v[j] += element(gr[i], j);
            }
            store_group<kVec>(dx + r * a.dx.rs, i, t, threads, a.cols, v);
        }
    }
    if (!a.part) return;
    float *part = a.part + (int64_t)blockIdx.x * 2 * a.cols;
    if constexpr (kWarp) {
        // the eight warps add their sums in order
        for (int w = 0; w < 8; ++w) {
            if ((int)threadIdx.x / 32 == w)
#pragma unroll
                for (int i = 0; i < kNv; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int c = column<kVec>(i, j, t, threads);
                        if (c < a.cols) {
                            sums[c] = (w ? sums[c] : 0.0f) + dg[i][j];
                            sums[a.cols + c] = (w ? sums[a.cols + c] : 0.0f) + db[i][j];
                        }
                    }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * a.cols; c += 256) part[c] = sums[c];
    } else {
#pragma unroll
        for (int i = 0; i < kNv; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = column<kVec>(i, j, t, threads);
                if (c < a.cols) {
                    part[c] = dg[i][j];
                    part[a.cols + c] = db[i][j];
                }
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

// How rows of `cols` elements are held: by a warp up to 8 * 32 * nv elements,
// else by a block of `threads`.
struct RowShape {
    int nv = 0, threads = 0;  // nv == 0: not in registers
    bool warp = false;
};

RowShape row_shape(int64_t cols) {
    RowShape s;
    if (cols <= 512) {
        s.warp = true;
        s.threads = 256;
        s.nv = cols <= 256 ? 1 : 2;
        return s;
    }
    for (int nv = 1; nv <= 4; nv *= 2) {
        const int64_t threads = round_up((cols + 8 * nv - 1) / (8 * nv), 32);
        if (threads <= (nv == 1 ? 256 : 512)) {
            s.nv = nv;
            s.threads = (int)threads;
            return s;
        }
    }
    return s;
}

template <typename X, typename Y>
bool launch_norm(const NormArgs &a, const RowShape &sh, bool vec, unsigned grid, cudaStream_t s) {
#define I8C_NORM(NV, W)                                                                                       \
    (vec ? launch_behind(layer_norm_rows_kernel<X, Y, NV, true, W>, dim3(grid), sh.threads, 0, s, a)          \
         : launch_behind(layer_norm_rows_kernel<X, Y, NV, false, W>, dim3(grid), sh.threads, 0, s, a))
    if (sh.warp) return sh.nv == 1 ? I8C_NORM(1, true) : I8C_NORM(2, true);
    return sh.nv == 1 ? I8C_NORM(1, false) : sh.nv == 2 ? I8C_NORM(2, false) : I8C_NORM(4, false);
#undef I8C_NORM
}

template <typename X>
bool launch_norm_to(const NormArgs &a, const RowShape &sh, bool vec, unsigned grid, cudaStream_t s) {
    switch (a.y.dtype) {
        case CONV_FLOAT32: return launch_norm<X, float>(a, sh, vec, grid, s);
        case CONV_FLOAT16: return launch_norm<X, __half>(a, sh, vec, grid, s);
        default: return launch_norm<X, __nv_bfloat16>(a, sh, vec, grid, s);
    }
}

template <typename X>
bool launch_norm_grad(const NormGradArgs &a, const RowShape &sh, bool vec, unsigned grid, cudaStream_t s) {
    const size_t smem = sh.warp ? (size_t)a.cols * 8 : 0;
#define I8C_NORM(NV, W)                                                                                        \
    (vec ? launch_behind(layer_norm_grad_rows_kernel<X, NV, true, W>, dim3(grid), sh.threads, smem, s, a)      \
         : launch_behind(layer_norm_grad_rows_kernel<X, NV, false, W>, dim3(grid), sh.threads, smem, s, a))
    if (sh.warp) return sh.nv == 1 ? I8C_NORM(1, true) : I8C_NORM(2, true);
    return sh.nv == 1 ? I8C_NORM(1, false) : sh.nv == 2 ? I8C_NORM(2, false) : I8C_NORM(4, false);
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
    const RowShape sh = row_shape(cols);
    bool ok;
    if (sh.nv == 0 || !unit_columns(a.x) || !unit_columns(a.y)) {
        ok = launch_behind(layer_norm_any_kernel, dim3((unsigned)rows), cols > 4096 ? 1024 : 256, 0, s, a);
    } else {
        const bool vec = cols % 8 == 0 && vector_rows(a.x) && vector_rows(a.y);
        const int64_t blocks = sh.warp ? (rows + 7) / 8 : rows;
        const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)device_sm_count() * (1024 / sh.threads));
        switch (x->dtype) {
            case CONV_FLOAT32: ok = launch_norm_to<float>(a, sh, vec, grid, s); break;
            case CONV_FLOAT16: ok = launch_norm_to<__half>(a, sh, vec, grid, s); break;
            case CONV_BFLOAT16: ok = launch_norm_to<__nv_bfloat16>(a, sh, vec, grid, s); break;
            default: ok = launch_norm_to<int32_t>(a, sh, vec, grid, s); break;
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
    const RowShape sh = row_shape(cols);
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
        const bool vec = cols % 8 == 0 && vector_rows(a.dy) && vector_rows(a.x) && vector_rows(a.res) &&
                         vector_rows(a.dx);
        const int64_t blocks = sh.warp ? (rows + 7) / 8 : rows;
        parts = std::min<int64_t>({blocks, (int64_t)device_sm_count() * std::max(1, 512 / sh.threads), kMaxParts});
        switch (x->dtype) {
            case CONV_FLOAT32: ok = launch_norm_grad<float>(a, sh, vec, (unsigned)parts, s); break;
            case CONV_FLOAT16: ok = launch_norm_grad<__half>(a, sh, vec, (unsigned)parts, s); break;
            default: ok = launch_norm_grad<__nv_bfloat16>(a, sh, vec, (unsigned)parts, s); break;
        }
    }
    if (ok && a.part)
        ok = launch_behind(layer_norm_params_sum_kernel, dim3((unsigned)((2 * cols + 31) / 32)), 1024, 0, s,
                           (const float *)workspace, parts, cols, dgain_dev, dshift_dev, p->param_dtype);
    return ok ? CONV_OK : CONV_ERR_CUDA;
}

}  // extern "C"

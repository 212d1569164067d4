// clip_grads.cu -- conv_clip_grads: the global norm of many tensors, and the
// tensors scaled by it.
//
// Two kernels over chunks of 16384 elements, dealt to at most four blocks per
// SM: the first leaves each block's sum of squares in the workspace, the
// second adds those sums (every block for itself, in one order: that costs a
// few loads from L2 and saves a counter that would have to be cleared) and
// scales.  It walks the chunks backwards, so that what the first kernel read
// last is still in L2.  The table of tensors travels in the launch's
// parameters, up to 64 of them in a small launch and 960 in a large one; more
// take several launches, whose sums meet in the workspace.  A stream: 268
// million values in 48 tensors take 265 us (read twice and written once, 6.0
// TB/s), six small tensors 9.3 us of launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "channel.h"
#include "channel_launch.cuh"
#include "channel_math.cuh"
#include "channel_rows.cuh"
#include "tc_ptx.cuh"

namespace i8c {
namespace {

constexpr int kClipThreads = 256;
constexpr int64_t kChunk = 16384;                 // elements
constexpr int kGroups = (int)(kChunk / (kClipThreads * 8));  // of 8 elements, per thread and chunk
constexpr int kClipBlocks = 608;                  // four per SM of the part this library is for: fixes the workspace

struct ClipEntry {
    const void *grad;
    void *out;
    int64_t count;
    int32_t first;  // chunk
    int32_t dtype;
};
template <int kMax>
struct ClipTable {
    ClipEntry entry[kMax];
    int32_t n, chunks;
    double *part;      // of this launch's blocks (first kernel), or of all (second)
    int32_t parts;
    float max_norm, eps;
    float *norm;       // written by the first block, or NULL
};

// The entry that chunk c belongs to (empty tensors have no chunk).
template <int kMax>
__device__ __forceinline__ const ClipEntry &entry_of(const ClipTable<kMax> &t, int c) {
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.entry[mid].first <= c) lo = mid;
        else hi = mid - 1;
    }
    return t.entry[lo];
}

// Group i of this thread in a chunk that starts at p and has `left` elements; zeros past the end.
template <typename T>
__device__ __forceinline__ void load_group_of(const T *p, int64_t left, int i, bool vec, Group<T> &g) {
    const int64_t e = ((int64_t)i * kClipThreads + threadIdx.x) * 8;
    if (vec && e + 8 <= left) {
        const uint4 *q = reinterpret_cast<const uint4 *>(p + e);
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
        if constexpr (kIs16<T>) {
            const uint32_t v = e + j < left ? reinterpret_cast<const uint16_t *>(p)[e + j] : 0u;
            if (j % 2) g.w[j / 2] |= v << 16;
            else g.w[j / 2] = v;
        } else {
            g.w[j] = e + j < left ? reinterpret_cast<const uint32_t *>(p)[e + j] : 0u;
        }
    }
}

// Sum of the squares of 32 elements.  In 32 bits where that keeps them (f16
// always; else unless the sum nears either end of the range, or is 0 with
// something there), else in 64.
template <typename T>
__device__ __forceinline__ double squares(const Group<T> (&g)[4]) {
    Pair s = pair(0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const Pair v = element2(g[i], j);
            s = fma2(v, v, s);
        }
    float a, b;
    split(s, &a, &b);
    a += b;
    if (!std::is_same_v<T, __half> && !(a > 0x1p-90f && a < 0x1p120f)) {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < (kIs16<T> ? 4 : 8); ++j) any |= g[i].w[j] & (kIs16<T> ? 0x7fff7fffu : 0x7fffffffu);
        double d = 0.0;
        if (any) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const double v = (double)element(g[i], j);
                    d += v * v;
                }
        }
        return d;
    }
    return (double)a;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const ClipEntry &e, int c) {
    const int64_t at = (int64_t)(c - e.first) * kChunk, left = e.count - at;
    const T *p = (const T *)e.grad + at;
    const bool vec = (uintptr_t)p % 16 == 0;
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kGroups; i += 4) {
        Group<T> g[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) load_group_of(p, left, i + k, vec, g[k]);
        sum += squares(g);
    }
    return sum;
}

// Sum over the block, in every thread.
__device__ __forceinline__ double block_total(double v) {
    __shared__ double part[kClipThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kClipThreads / 32; ++i) s += part[i];
    return s;
}

template <int kMax>
__global__ void __launch_bounds__(kClipThreads, 4) clip_squares_kernel(const __grid_constant__ ClipTable<kMax> t) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    double sum = 0.0;
    for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const ClipEntry &e = entry_of(t, c);
        if (e.dtype == CONV_FLOAT32) sum += chunk_squares<float>(e, c);
        else if (e.dtype == CONV_FLOAT16) sum += chunk_squares<__half>(e, c);
        else sum += chunk_squares<__nv_bfloat16>(e, c);
    }
    sum = block_total(sum);
    if (threadIdx.x == 0) t.part[blockIdx.x] = sum;
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const ClipEntry &e, int c, float factor) {
    const int64_t at = (int64_t)(c - e.first) * kChunk, left = e.count - at;
    const T *p = (const T *)e.grad + at;
    T *o = (T *)e.out + at;
    const bool vec = (uintptr_t)p % 16 == 0, out_vec = (uintptr_t)o % 16 == 0;
#pragma unroll
    for (int i = 0; i < kGroups; i += 4) {
        Group<T> g[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) load_group_of(p, left, i + k, vec, g[k]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t at8 = ((int64_t)(i + k) * kClipThreads + threadIdx.x) * 8;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = element(g[k], j) * factor;
            if (out_vec && at8 + 8 <= left) {
                if constexpr (kIs16<T>) {
                    *reinterpret_cast<uint4 *>(o + at8) = pack8<std::is_same_v<T, __half>>(v);
                } else {
                    *reinterpret_cast<float4 *>(o + at8) = make_float4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<float4 *>(o + at8 + 4) = make_float4(v[4], v[5], v[6], v[7]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (at8 + j < left) {
                        if constexpr (kIs16<T>) reinterpret_cast<uint16_t *>(o)[at8 + j] = (uint16_t)bits16(v[j], o);
                        else o[at8 + j] = v[j];
                    }
            }
        }
    }
}

template <int kMax>
__global__ void __launch_bounds__(kClipThreads, 4) clip_scale_kernel(const __grid_constant__ ClipTable<kMax> t) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    double sum = 0.0;
    for (int i = threadIdx.x; i < t.parts; i += kClipThreads) sum += t.part[i];
    const double norm = sqrt(block_total(sum));
    if (blockIdx.x == 0 && threadIdx.x == 0 && t.norm) *t.norm = (float)norm;
    const double ratio = (double)t.max_norm / (norm + (double)t.eps);
    const float factor = ratio >= 1.0 ? 1.0f : (float)ratio;  // (NaN stays)
    for (int b = blockIdx.x; b < t.chunks; b += gridDim.x) {
        const int c = t.chunks - 1 - b;
        const ClipEntry &e = entry_of(t, c);
        if (e.out == e.grad && factor == 1.0f) continue;
        if (e.dtype == CONV_FLOAT32) scale_chunk<float>(e, c, factor);
        else if (e.dtype == CONV_FLOAT16) scale_chunk<__half>(e, c, factor);
        else scale_chunk<__nv_bfloat16>(e, c, factor);
    }
}

constexpr int kSmallTable = 64, kLargeTable = 960;  // (parameters hold 32764 bytes)
static_assert(sizeof(ClipTable<kLargeTable>) <= 32764);

int64_t launches_of(int64_t n) { return std::max<int64_t>(1, (n + kLargeTable - 1) / kLargeTable); }
size_t clip_bytes(int64_t n) { return (size_t)round_up(launches_of(n) * kClipBlocks * 8, 256); }

// Fills the table with tensors [lo, hi); false where they have too many chunks.
template <int kMax>
bool fill(ClipTable<kMax> &t, const conv_grad_tensor *g, int64_t lo, int64_t hi) {
    int64_t chunks = 0;
    t.n = 0;
    for (int64_t i = lo; i < hi; ++i) {
        if (g[i].count == 0) continue;
        t.entry[t.n++] = {g[i].grad, g[i].out ? g[i].out : const_cast<void *>(g[i].grad), g[i].count, (int32_t)chunks, g[i].dtype};
        chunks += (g[i].count + kChunk - 1) / kChunk;
        if (chunks > INT32_MAX - kClipBlocks) return false;
    }
    t.chunks = (int32_t)chunks;
    return true;
}

template <int kMax>
conv_status run(const conv_grad_tensor *g, int64_t n, float max_norm, float eps, float *norm, double *part, cudaStream_t s) {
    ClipTable<kMax> t;
    int64_t parts = 0;
    const int64_t launches = std::max<int64_t>(1, (n + kMax - 1) / kMax);
    for (int64_t l = 0; l < launches; ++l)  // (all of them before the first launch: a refused call launches nothing)
        if (!fill(t, g, l * kMax, std::min(n, (l + 1) * kMax))) return CONV_ERR_TOO_LARGE;
    for (int64_t l = 0; l < launches; ++l) {
        if (launches > 1) fill(t, g, l * kMax, std::min(n, (l + 1) * kMax));
        if (t.chunks == 0) continue;
        const int grid = std::min(t.chunks, kClipBlocks);
        t.part = part + parts;
        parts += grid;
        if (!launch_behind(clip_squares_kernel<kMax>, dim3((unsigned)grid), kClipThreads, 0, s, t)) return CONV_ERR_CUDA;
    }
    t.part = part, t.parts = (int32_t)parts;
    t.max_norm = max_norm, t.eps = eps;
    // backwards, like the chunks; the norm with the first launch
    for (int64_t l = launches; l-- > 0;) {
        if (launches > 1) fill(t, g, l * kMax, std::min(n, (l + 1) * kMax));
        t.norm = l == launches - 1 ? norm : nullptr;
        if (std::isinf(max_norm)) t.chunks = 0;
        if (t.chunks == 0 && !t.norm) continue;
        if (!launch_behind(clip_scale_kernel<kMax>, dim3((unsigned)std::clamp(t.chunks, 1, kClipBlocks)), kClipThreads, 0, s, t))
            return CONV_ERR_CUDA;
    }
    return CONV_OK;
}

struct Range {
    uintptr_t lo, hi;
    bool operator<(const Range &o) const { return lo < o.lo; }
};

conv_status check_tensors(const conv_grad_tensor *g, int64_t n) {
    if (n < 0) return CONV_ERR_BAD_PARAM;
    if (n > 0 && !g) return CONV_ERR_NULL_PTR;
    if (n > 1 << 24) return CONV_ERR_TOO_LARGE;
    for (int64_t i = 0; i < n; ++i) {
        if (!is_float_type(g[i].dtype)) return CONV_ERR_DTYPE;
        if (g[i].reserved != 0 || g[i].count < 0) return CONV_ERR_BAD_PARAM;
        if (g[i].count >= (int64_t)1 << 45) return CONV_ERR_TOO_LARGE;
    }
    return CONV_OK;
}

}  // namespace
}  // namespace i8c

using namespace i8c;

extern "C" {

conv_status conv_clip_grads_workspace_size(const conv_grad_tensor *tensors, int64_t n, size_t *bytes) {
    if (!bytes) return CONV_ERR_NULL_PTR;
    const conv_status st = check_tensors(tensors, n);
    if (st) return st;
    *bytes = clip_bytes(n);
    return CONV_OK;
}

conv_status conv_clip_grads(const conv_grad_tensor *tensors, int64_t n, float max_norm, float eps, float *norm_dev,
                            void *workspace, size_t workspace_bytes, void *stream) {
    conv_status st = check_tensors(tensors, n);
    if (st) return st;
    if (!norm_dev) return CONV_ERR_NULL_PTR;
    if (!(max_norm >= 0.0f) || !(eps >= 0.0f) || std::isinf(eps)) return CONV_ERR_BAD_PARAM;
    if ((uintptr_t)norm_dev % 4) return CONV_ERR_ALIGNMENT;
    const size_t need = clip_bytes(n);
    if (!workspace || workspace_bytes < need || (uintptr_t)workspace % 256) return CONV_ERR_WORKSPACE;
    // every buffer of the call apart from every other
    Range few[2 * kSmallTable + 2];
    std::unique_ptr<Range[]> many;
    Range *r = few;
    if (n > kSmallTable) {
        many.reset(new (std::nothrow) Range[2 * n + 2]);
        if (!many) return CONV_ERR_TOO_LARGE;
        r = many.get();
    }
    int64_t k = 0;
    r[k++] = {(uintptr_t)norm_dev, (uintptr_t)norm_dev + 4};
    r[k++] = {(uintptr_t)workspace, (uintptr_t)workspace + need};
    const bool scaling = !std::isinf(max_norm);
    for (int64_t i = 0; i < n; ++i) {
        const conv_grad_tensor &g = tensors[i];
        if (g.count == 0) continue;
        if (!g.grad) return CONV_ERR_NULL_PTR;
        const uintptr_t size = (uintptr_t)channel_elem_size(g.dtype), bytes = size * (uintptr_t)g.count;
        if ((uintptr_t)g.grad % size || (uintptr_t)g.out % size) return CONV_ERR_ALIGNMENT;
        r[k++] = {(uintptr_t)g.grad, (uintptr_t)g.grad + bytes};
        if (scaling && g.out && g.out != g.grad) r[k++] = {(uintptr_t)g.out, (uintptr_t)g.out + bytes};
    }
    std::sort(r, r + k);
    for (int64_t i = 1; i < k; ++i)
        if (r[i].lo < r[i - 1].hi) return CONV_ERR_OVERLAP;
    if ((st = check_device())) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    // (the small table's launch copies 2 KB of parameters, the large one's 30 KB)
    return n <= kSmallTable ? run<kSmallTable>(tensors, n, max_norm, eps, norm_dev, (double *)workspace, s)
                            : run<kLargeTable>(tensors, n, max_norm, eps, norm_dev, (double *)workspace, s);
}

}  // extern "C"

// channel_rows.cuh -- rows of channels in registers: how a warp or a block
// holds, loads, sums and stores them; shared by the norms.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <initializer_list>
#include <type_traits>

#include "channel.h"
#include "channel_launch.cuh"
#include "channel_math.cuh"
#include "tc_ptx.cuh"

namespace i8c {

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

// kEven: rows of whole groups.
template <bool kVec, typename T, bool kEven = false>
__device__ __forceinline__ void store_group(T *p, const Place<kVec> &at, int i, const float (&v)[8]) {
    if (kEven ? at.inside(at.column(i, 0)) : kVec && at.whole(i)) {
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
    if constexpr (!kEven) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = at.column(i, j);
            if (!at.inside(c)) continue;
            if constexpr (kIs16<T>) reinterpret_cast<uint16_t *>(p)[c] = (uint16_t)bits16(v[j], p);
            else p[c] = v[j];
        }
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

// Stores group i of a row whose groups begin elsewhere than the thread's
// (another lead): the thread's last elements and the next one's first make up
// an aligned group, except at a warp's ends and the row's, whose elements go
// one by one.  The whole warp takes part.
template <typename T>
__device__ __forceinline__ void store_shifted(T *p, const Place<true> &at, int i, const float (&v)[8]) {
    const int b = (at.lead - lead_of(p)) & 7;  // the thread's first element on the output's boundary
    constexpr int kWords = kIs16<T> ? 4 : 8;
    uint32_t w[2 * kWords];
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
        if constexpr (kIs16<T>) w[j] = pack2(v[2 * j], v[2 * j + 1], std::is_same_v<T, __half> ? CONV_FLOAT16 : CONV_BFLOAT16);
        else w[j] = __float_as_uint(v[j]);
    }
#pragma unroll
    for (int j = 0; j < kWords; ++j) w[kWords + j] = __shfl_down_sync(0xffffffffu, w[j], 1);
    const int c = at.column(i, 0), lane = threadIdx.x % 32;
    const bool whole = (lane < 31 || b == 0) && c + b >= 0 && c + b + 8 <= at.cols;
    // elements that no aligned group has: before the boundary where the previous lane cannot take them, behind it
    // where this one cannot
    const bool first = lane == 0 || c + b - 8 < 0 || c + b > at.cols;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (at.inside(c + j) && (j < b ? first : !whole)) {
            if constexpr (kIs16<T>) reinterpret_cast<uint16_t *>(p)[c + j] = (uint16_t)(w[j / 2] >> (j % 2 * 16));
            else p[c + j] = __uint_as_float(w[j]);
        }
    if constexpr (kIs16<T>) {
        if (b & 4) {
#pragma unroll
            for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
        }
        if (b & 2) {
#pragma unroll
            for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], (b & 1) * 16);
    } else {
#pragma unroll
        for (int s = 4; s > 0; s >>= 1)
            if (b & s) {
#pragma unroll
                for (int j = 0; j < 7 + s; ++j)
                    if (j + s < 16) w[j] = w[j + s];
            }
    }
    if (whole) {
        uint4 *o = reinterpret_cast<uint4 *>(p + c + b);
        o[0] = make_uint4(w[0], w[1], w[2], w[3]);
        if constexpr (!kIs16<T>) o[1] = make_uint4(w[4], w[5], w[6], w[7]);
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

// ---------------------------------------------------------------- rows by bulk copies
// Rows of several matrices on their way to shared memory, one bulk copy per
// row and matrix: lane m of a worker's first warp feeds matrix m.  A copy
// takes whole 16-byte pieces, so a row that begins or ends inside one brings
// bytes of its neighbours along, which the readers mask; where that would
// reach past the matrix (its first or last row) the ends are copied by
// elements.  A row lies in its slot as it does past a boundary of 8 elements.
struct RowFeed {
    const char *p, *end;   // the matrix's memory
    const char *next;      // the row to come
    int64_t step;          // bytes from it to the one after
    uint32_t bytes;        // of a row
    uint32_t off;          // of the matrix's slot in a stage
    uint32_t half;         // 16 where a boundary of 16 bytes may not be one of 8 elements
    bool on;

    __device__ __forceinline__ void set(const MatRef &m, int64_t rows, int32_t cols, uint32_t size, uint32_t at, int64_t first, int64_t row_step) {
        p = (const char *)m.p;
        bytes = (uint32_t)cols * size;
        end = p + (rows - 1) * m.rs * size + bytes;
        next = p + first * m.rs * size;
        step = row_step * m.rs * size;
        off = at;
        half = size == 4 ? 16 : 0;
        on = true;
    }
    // One arrival on `bar` and the next row's bytes.  kEven: rows of whole, aligned groups.
    template <bool kEven>
    __device__ __forceinline__ void fill(uint32_t stage, uint32_t bar) {
        const char *s = next, *e = s + bytes;
        next += step;
        if constexpr (kEven) {
            ptx::mbar_arrive_expect_tx(bar, bytes);
            ptx::bulk_copy_g2s(stage + off, s, bytes, bar);
        } else {
            fill_any(s, e, stage + ((uint32_t)(uintptr_t)s & half), bar);
        }
    }
    __device__ __forceinline__ void fill_any(const char *s, const char *e, uint32_t stage, uint32_t bar) const {
        const char *s0 = s - ((uintptr_t)s & 15), *e0 = e + (-(uintptr_t)e & 15);
        if (s0 >= p && e0 <= end) {
            ptx::mbar_arrive_expect_tx(bar, (uint32_t)(e0 - s0));
            ptx::bulk_copy_g2s(stage + off, s0, (uint32_t)(e0 - s0), bar);
            return;
        }
        const char *s1 = s + (-(uintptr_t)s & 15), *e1 = e - ((uintptr_t)e & 15);
        const char *const lead_end = s1 < e ? s1 : e;
        auto copy = [&](const char *from, const char *to) {
            for (; from < to; from += 2)
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(stage + off + (uint32_t)(from - s0)), "h"(*(const uint16_t *)from) : "memory");
        };
        copy(s, lead_end);
        if (e1 >= s1) copy(e1, e);
        if (e1 > s1) {
            ptx::mbar_arrive_expect_tx(bar, (uint32_t)(e1 - s1));
            ptx::bulk_copy_g2s(stage + off + (uint32_t)(s1 - s0), s1, (uint32_t)(e1 - s1), bar);
        } else {
            ptx::mbar_arrive(bar);
        }
    }
};

// Bytes of a row's slot: the row, and the groups of 8 that its ends lie in.
__host__ __device__ constexpr uint32_t row_slot_bytes(int32_t cols, uint32_t size) {
    return ((uint32_t)cols + 7) / 8 * 8 * size + 8 * size;
}

// Summer for one value.
struct RowSummer {
    float (*part)[32];
    int turn = 0;
    __device__ __forceinline__ float operator()(float u) {
        u = warp_sum(u);
        float *p = part[turn];
        turn ^= 1;
        if (threadIdx.x % 32 == 0) p[threadIdx.x / 32] = u;
        __syncthreads();
        const int warps = blockDim.x / 32;
        float t = 0.0f;
#pragma unroll 4
        for (int i = 0; i < warps; ++i) t += p[i];
        return t;
    }
};

// Waits for a row, not for ever: a thread that has given up once (the status
// word then says so) does not wait again until the end.
struct RowWait {
    uint64_t limit_ns;
    int *status;
    bool gave_up = false;
    __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity) {
        if (gave_up || ptx::mbar_try_wait(bar, parity)) return;
        const uint64_t t0 = ptx::global_timer_ns();
        while (!ptx::mbar_try_wait(bar, parity)) {
            if (ptx::global_timer_ns() - t0 > limit_ns) {
                gave_up = true;
                atomicExch(status, (int)CONV_ERR_DEVICE_TIMEOUT);
                return;
            }
        }
    }

    // Behind the rows: after a wait that ran out copies may still be under way to
    // the block's shared memory.  The lanes that started them stay until they
    // have landed: 10 ms, where a copy takes microseconds (rows were fed on
    // without waiting, so that no phase says which of them is in).
    __device__ __forceinline__ void settle(bool feeds) const {
        if (!gave_up || !feeds) return;
        const uint64_t t0 = ptx::global_timer_ns();
        while (ptx::global_timer_ns() - t0 < 10000000) {
        }
    }
};

// Group i of a row in its slot; zeros outside the row, and where there is no matrix.  kEven: rows of whole
// groups.
template <bool kEven, typename X>
__device__ __forceinline__ void slot_group(uint32_t slot, const Place<true> &at, int i, Group<X> &g, bool there = true) {
    const uint32_t from = slot + (uint32_t)(i * at.threads + at.t) * (uint32_t)(8 * sizeof(X));
    if (there && (kEven ? at.inside(at.column(i, 0)) : at.whole(i))) {
        const uint4 a = ptx::ld_shared_v4(from);
        g.w[0] = a.x, g.w[1] = a.y, g.w[2] = a.z, g.w[3] = a.w;
        if constexpr (!kIs16<X>) {
            const uint4 b = ptx::ld_shared_v4(from + 16);
            g.w[4] = b.x, g.w[5] = b.y, g.w[6] = b.z, g.w[7] = b.w;
        }
        return;
    }
    if constexpr (kEven) {
#pragma unroll
        for (int j = 0; j < (int)(sizeof(g.w) / 4); ++j) g.w[j] = 0;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool in = there && at.inside(at.column(i, j));
            if constexpr (kIs16<X>) {
                uint16_t v = 0;
                if (in) asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(from + j * 2));
                if (j % 2) g.w[j / 2] |= (uint32_t)v << 16;
                else g.w[j / 2] = v;
            } else {
                g.w[j] = in ? ptx::ld_shared_b32(from + j * 4) : 0u;
            }
        }
    }
}

// ---------------------------------------------------------------- host
inline bool unit_columns(const MatRef &m) { return !m.p || m.cs <= 1; }

// Lead of a matrix's rows: 8 values for the rows modulo 8, as base and step.
struct Lead {
    int64_t base, step;
};
inline Lead lead_of_rows(const MatRef &m) {
    const int64_t size = channel_elem_size(m.dtype);
    return {(int64_t)((uintptr_t)m.p / (uintptr_t)size & 7), m.rs & 7};
}

// Whether the rows of all matrices (those given) have one lead.
inline bool one_lead(std::initializer_list<const MatRef *> all) {
    const Lead l = lead_of_rows(**all.begin());
    for (const MatRef *m : all) {
        if (!m->p) continue;
        const Lead k = lead_of_rows(*m);
        if (k.base != l.base || k.step != l.step) return false;
    }
    return true;
}

// A launch with more than 48 KB of shared memory.
template <auto kKernel, typename Args>
inline bool launch_large(dim3 grid, int threads, size_t smem, cudaStream_t s, const Args &a) {
    static std::atomic<bool> ready[64];  // (check_device admits 64 devices)
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (!ready[dev].load()) {
        if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 << 10) != cudaSuccess) return false;
        ready[dev].store(true);
    }
    return launch_behind(kKernel, grid, threads, smem, s, a);
}

// A vector the call reads or writes: aligned to its element, and apart from
// the matrix `m`.
inline conv_status check_vector(const void *p, int64_t n, int64_t size, const conv_matrix_desc *m, const void *m_dev) {
    if (!p || n == 0) return CONV_OK;
    if ((uintptr_t)p % (uintptr_t)size) return CONV_ERR_ALIGNMENT;
    if (m && overlaps(p, (uint64_t)(n * size), m_dev, matrix_extent_bytes(m))) return CONV_ERR_OVERLAP;
    return CONV_OK;
}

}  // namespace i8c

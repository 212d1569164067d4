// product_tiles.cuh -- what the tensor-core products share: waits, tile walks,
// the epilogue from 32-bit sums to stored results, the joining of cut sums,
// and tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "channel.h"
#include "channel_launch.cuh"
#include "channel_math.cuh"
#include "tc_ptx.cuh"

namespace i8c {

constexpr int kTileA = 128;        // accumulator lanes of one CTA
constexpr int kSlotBytes = 2048;   // staging of one epilogue warp
constexpr int64_t kSms = 152;      // of the part this library is for, whatever the device: plans fix workspace sizes

// How an output, residual or pre-activation matrix is walked.
enum Walk : int32_t {
    kWalkNone = 0,
    kWalkRows,    // b contiguous, 16-byte aligned rows: vectors
    kWalkAlongB,  // lanes along b
    kWalkAlongA,  // lanes along a
};

struct Side {
    void *p;
    int64_t sa, sb;
    int32_t dtype;
    int32_t walk;
};

// An output, its residual and pre-activation, and the bias.
struct EpilogueArgs {
    CUtensorMap map_d, map_pre;
    Side d, res, pre;
    const void *bias;
    int32_t bias_dtype, bias_along_a;
    int32_t ma, nb;
    int32_t slots;               // staging slots of an epilogue warp: 2 where a residual is loaded ahead
    int32_t act;                 // read by kernels that take the activation at run time
};

// ... in tiles, some of which may be summed in runs of k.
struct TileArgs : EpilogueArgs {
    int32_t tile_b;              // a multiple of 32
    int32_t tiles_a, tiles_b;
    int32_t parts;               // runs of k, each summed to `part` (1: none),
    int32_t full;                // of the tiles from this one on
    float *part;                 // [run][tile][128-row half][column][row of 128]
};

// Activation code for functions that take the activation at run time.
constexpr int kAnyAct = -1;

// ---------------------------------------------------------------- PTX
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// The address of this CTA's shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Arrival that orders nothing but itself (and, behind tcgen05.fence, the
// tensor-memory reads): a releasing one would first wait for every global
// store of the epilogue to be acknowledged.
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// 2-D load whose completion is counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void *tmap, int32_t x, int32_t y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, int32_t x, int32_t y, int32_t z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void *tmap, int32_t x, int32_t y, int32_t z,
                                                 uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

template <bool kPair>
__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                    uint32_t accumulate) {
    if constexpr (kPair) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    } else {
        ptx::mma_f16_ss(d_tmem, a_desc, b_desc, idesc, accumulate);
    }
}

// Arrives on `bar` (in both CTAs of a pair) when the MMAs issued so far are done.
template <bool kPair>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    if constexpr (kPair) {
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                bar),
            "h"((uint16_t)3)
            : "memory");
    } else {
        ptx::mma_commit(bar);
    }
}

template <bool kPair>
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
    if constexpr (kPair) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
                     "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::"r"(dst), "r"(cols) : "memory");
    } else {
        ptx::tmem_alloc(dst, cols);
        ptx::tmem_relinquish();
    }
}

template <bool kPair>
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
    if constexpr (kPair)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
    else
        ptx::tmem_dealloc(addr, cols);
}

// Shared-memory matrix descriptor, 128-byte swizzle.  k contiguous: rows of
// 64 k elements, 8-row atoms 1024 bytes apart (the leading offset is unused).
// Own dim contiguous: rows of 64 own elements, one per k; 8-k atoms 1024
// bytes apart, the next 64 own elements one box (64 rows) further.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool mn) {
    uint64_t d = 0;
    d |= (uint64_t)((addr & 0x3FFFF) >> 4);
    d |= (uint64_t)(mn ? (64 * 128) >> 4 : 1) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Bounded wait; false when the CTA is giving up (the status word then holds
// the timeout).
static __device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int32_t *abort_flag, uint64_t limit_ns,
                                       int *status, bool spin) {
    const uint64_t t0 = ptx::global_timer_ns();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (spin ? ptx::mbar_test_wait(bar, parity) : ptx::mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (ptx::global_timer_ns() - t0 > limit_ns) {
            *abort_flag = 1;
            atomicExch(status, (int)CONV_ERR_DEVICE_TIMEOUT);
            return false;
        }
    }
}

// spin: poll without suspending (a suspended wait resumes some time after the
// phase completes).
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int32_t *abort_flag,
                                           uint64_t limit_ns, int *status, bool spin = false) {
    if (spin ? ptx::mbar_test_wait(bar, parity) : ptx::mbar_try_wait(bar, parity)) return true;
    return wait_slow(bar, parity, abort_flag, limit_ns, status, spin);
}

struct Ring {
    uint32_t idx = 0, phase = 0;
    __device__ __forceinline__ void next(uint32_t depth) {
        if (++idx == depth) {
            idx = 0;
            phase ^= 1u;
        }
    }
};

// Tile t of the walk over the output: bands of 8 tiles along a, so that the
// tiles in flight share operand rows in L2.
__device__ __forceinline__ void tile_at(const TileArgs &a, int t, int *ia, int *ib) {
    constexpr int kBand = 8;
    const int per_band = kBand * a.tiles_b;
    const int band = t / per_band, in = t - band * per_band;
    const int rows = min(kBand, a.tiles_a - band * kBand);
    *ib = in / rows;
    *ia = band * kBand + (in - *ib * rows);
}

// ---------------------------------------------------------------- epilogue
template <int kAct, int W>
__device__ __forceinline__ void activate_all(const EpilogueArgs &a, float (&v)[W]) {
    if constexpr (kAct == kAnyAct) {
        switch (a.act) {
            case CONV_ACT_RELU: activate_all<CONV_ACT_RELU>(a, v); break;
            case CONV_ACT_GELU: activate_all<CONV_ACT_GELU>(a, v); break;
            case CONV_ACT_GELU_TANH: activate_all<CONV_ACT_GELU_TANH>(a, v); break;
            case CONV_ACT_SILU: activate_all<CONV_ACT_SILU>(a, v); break;
            default: break;
        }
    } else {
#pragma unroll
        for (int j = 0; j < W; j += 2) activate<kAct>(v[j], v[j + 1]);
    }
}

// One warp's 32 rows x up to 32 columns at (row0, b0), lane = row.  The warp
// owns 2 KB of shared memory, the slot, through which every output, residual
// and pre-activation is turned: rows of 64 bytes (32 columns of a 16-bit
// matrix, 16 of a 32-bit one), each lane writing or reading its own row, and
// runs of a row going to or from global memory.
//
// kSlots slots in turn: as many stores may be under way.
struct WarpTile {
    int32_t row0, b0, rows, cols;  // rows, cols: how many are inside the matrix and the tile
    mutable int32_t turn = 0;      // of the slots
    uint32_t slot, bias;           // bias: 128 bytes of shared memory
    int lane;
};

// 16-byte piece i of a slot row, the pieces exchanged so that neither walk
// meets a bank twice; element c of a slot row.
__device__ __forceinline__ uint32_t piece(uint32_t slot, uint32_t row, uint32_t i) {
    return slot + row * 64 + ((i ^ ((row >> 1) & 3)) << 4);
}
__device__ __forceinline__ uint32_t at16(uint32_t slot, uint32_t row, uint32_t c) { return piece(slot, row, c >> 3) + (c & 7) * 2; }
__device__ __forceinline__ uint32_t at32(uint32_t slot, uint32_t row, uint32_t c) { return piece(slot, row, c >> 2) + (c & 3) * 4; }

__device__ __forceinline__ uint16_t ld_shared_b16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ void st_shared_b16(uint32_t addr, uint16_t v) {
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}

// Rows of a side matrix with aligned rows to the slot: 64-byte runs, eight
// rows per access.  p: the first row's 64 bytes.
__device__ __forceinline__ void rows_to_slot(const WarpTile &t, const char *p, int64_t row_bytes) {
    p += (int64_t)(t.lane / 4) * row_bytes + (t.lane & 3) * 16;
    uint4 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[i] = t.lane / 4 + 8 * i < t.rows ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
        p += 8 * row_bytes;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) ptx::st_shared_v4(piece(t.slot, t.lane / 4 + 8 * i, t.lane & 3), q[i]);
}

// 16-bit rows, two at a time, from and to the slot in 32-bit words where a row's alignment has
// them: lane w of a row takes columns 2w - odd and the next, and the last lane
// the column that is left.  p: the first row's first element.
static __device__ __noinline__ void slot_to_words(uint16_t *p, int64_t row, int rows, int cols, uint32_t slot) {
    const int lane = threadIdx.x % 32, w = lane & 15;
#pragma unroll 2
    for (int r = lane >> 4; r < rows; r += 2) {
        uint16_t *q = p + r * row;
        const int e = 2 * w - (int)((uintptr_t)q >> 1 & 1);
        const uint32_t lo = e >= 0 ? ld_shared_b16(at16(slot, r, e)) : 0u, hi = ld_shared_b16(at16(slot, r, e + 1));
        if (e >= 0 && e + 1 < cols) *reinterpret_cast<uint32_t *>(q + e) = lo | hi << 16;
        else if (e >= 0 && e < cols) q[e] = (uint16_t)lo;
        else if (e < 0) q[0] = (uint16_t)hi;
        if (e == 29 && cols == 32) q[31] = ld_shared_b16(at16(slot, r, 31));
    }
}
static __device__ __noinline__ void words_to_slot(const uint16_t *p, int64_t row, int rows, int cols, uint32_t slot) {
    const int lane = threadIdx.x % 32, w = lane & 15;
#pragma unroll 1
    for (int r0 = lane >> 4; r0 < rows; r0 += 16) {
        uint32_t v[8];  // loads in flight
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t *q = p + (r0 + 2 * i) * row;
            const int e = 2 * w - (int)((uintptr_t)q >> 1 & 1);
            v[i] = 0;
            if (r0 + 2 * i >= rows) continue;
            if (e >= 0 && e + 1 < cols) v[i] = *reinterpret_cast<const uint32_t *>(q + e);
            else if (e >= 0 && e < cols) v[i] = q[e];
            else if (e < 0) v[i] = (uint32_t)q[0] << 16;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + 2 * i;
            const uint16_t *q = p + r * row;
            const int e = 2 * w - (int)((uintptr_t)q >> 1 & 1);
            if (r >= rows) continue;
            if (e >= 0) st_shared_b16(at16(slot, r, e), (uint16_t)v[i]);
            st_shared_b16(at16(slot, r, e + 1), (uint16_t)(v[i] >> 16));
            if (e == 29 && cols == 32) st_shared_b16(at16(slot, r, 31), q[31]);
        }
    }
}

// The same for any strides, an element at a time, `cols` columns from column
// b0 + c on: lanes along the rows, or along the columns (32 of 16 bits, or 16
// of 32 bits and two rows).
static __device__ __noinline__ void slot_to_any(Side s, WarpTile t, int c, int cols) {
    const bool wide = s.dtype == CONV_FLOAT32;
    if (s.walk == kWalkAlongA) {
        const int64_t at = (int64_t)(t.row0 + t.lane) * s.sa + (int64_t)(t.b0 + c) * s.sb;
        if (t.lane < t.rows)
#pragma unroll 8
            for (int j = 0; j < cols; ++j) {
                if (wide) ((uint32_t *)s.p)[at + j * s.sb] = ptx::ld_shared_b32(at32(t.slot, t.lane, j));
                else ((uint16_t *)s.p)[at + j * s.sb] = ld_shared_b16(at16(t.slot, t.lane, j));
            }
        return;
    }
    const int col = wide ? t.lane & 15 : t.lane, first = wide ? t.lane >> 4 : 0, step = wide ? 2 : 1;
    const int64_t at = (int64_t)t.row0 * s.sa + (int64_t)(t.b0 + c + col) * s.sb;
    if (col < cols) {
#pragma unroll 4
        for (int r = first; r < t.rows; r += step) {
            if (wide) ((uint32_t *)s.p)[at + r * s.sa] = ptx::ld_shared_b32(at32(t.slot, r, col));
            else ((uint16_t *)s.p)[at + r * s.sa] = ld_shared_b16(at16(t.slot, r, col));
        }
    }
}
static __device__ __noinline__ void any_to_slot(Side s, WarpTile t, int c, int cols) {
    const bool wide = s.dtype == CONV_FLOAT32;
    if (s.walk == kWalkAlongA) {
        const int64_t at = (int64_t)(t.row0 + t.lane) * s.sa + (int64_t)(t.b0 + c) * s.sb;
        if (t.lane < t.rows) {
#pragma unroll 8
            for (int j = 0; j < cols; ++j) {
                if (wide) ptx::st_shared_b32(at32(t.slot, t.lane, j), ((const uint32_t *)s.p)[at + j * s.sb]);
                else st_shared_b16(at16(t.slot, t.lane, j), ((const uint16_t *)s.p)[at + j * s.sb]);
            }
        }
        return;
    }
    const int col = wide ? t.lane & 15 : t.lane, first = wide ? t.lane >> 4 : 0, step = wide ? 2 : 1;
    const int64_t at = (int64_t)t.row0 * s.sa + (int64_t)(t.b0 + c + col) * s.sb;
    if (col < cols) {
#pragma unroll 1
        for (int r = first; r < t.rows; r += 16 * step) {
            // (sixteen loads in flight)
            uint32_t q[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (r + i * step < t.rows)
                    q[i] = wide ? ((const uint32_t *)s.p)[at + (r + i * step) * s.sa]
                                : ((const uint16_t *)s.p)[at + (r + i * step) * s.sa];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (r + i * step < t.rows) {
                    if (wide) ptx::st_shared_b32(at32(t.slot, r + i * step, col), q[i]);
                    else st_shared_b16(at16(t.slot, r + i * step, col), (uint16_t)q[i]);
                }
        }
    }
}

// The slot to `map`'s matrix by TMA, and the wait before the slot is used again.
__device__ __forceinline__ void send_slot(const CUtensorMap *map, const WarpTile &t, int c) {
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (t.lane == 0) {
        ptx::tma_store_2d(map, t.b0 + c, t.row0, t.slot);
        ptx::bulk_commit_group();
    }
}
__device__ __forceinline__ void free_slot(const WarpTile &t) {
    if (t.lane == 0) ptx::bulk_wait_group_read<0>();
    __syncwarp();
}
// ... of the next slot in turn, which t then has: every turn commits a group, so
// that with all but the last kSlots - 1 read this slot's is.
template <int kSlots>
__device__ __forceinline__ void next_slot(WarpTile &t, const WarpTile &given) {
    if (t.lane == 0) ptx::bulk_wait_group_read<kSlots - 1>();
    __syncwarp();
    if constexpr (kSlots > 1) {
        t.slot = given.slot + given.turn * kSlotBytes;
        given.turn = given.turn + 1 == kSlots ? 0 : given.turn + 1;
    }
}

// The slot has been written out without TMA (or not at all): an empty group in
// its place, for next_slot counts one for every turn.
template <int kSlots>
__device__ __forceinline__ void skip_slot(const WarpTile &t) {
    if (kSlots > 1 && t.lane == 0) ptx::bulk_commit_group();
}

template <int kSlots = 1>
__device__ __forceinline__ void store_chunk(const Side &s, const CUtensorMap *map, const WarpTile &given, const float (&v)[32]) {
    WarpTile t = given;
    const bool rows = s.walk == kWalkRows && t.cols == 32;
    if (s.dtype != CONV_FLOAT32) {
        next_slot<kSlots>(t, given);
        if (s.dtype == CONV_FLOAT16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) ptx::st_shared_v4(piece(t.slot, t.lane, i), pack8<true>(v + 8 * i));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) ptx::st_shared_v4(piece(t.slot, t.lane, i), pack8<false>(v + 8 * i));
        }
        if (rows) {
            send_slot(map, t, 0);
        } else {
            __syncwarp();
            if (s.walk != kWalkAlongA && s.sb == 1)
                slot_to_words((uint16_t *)s.p + (int64_t)t.row0 * s.sa + t.b0, s.sa, t.rows, t.cols, t.slot);
            else
                slot_to_any(s, t, 0, t.cols);
            skip_slot<kSlots>(t);
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < 32; c += 16) {
        next_slot<kSlots>(t, given);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            ptx::st_shared_v4(piece(t.slot, t.lane, i),
                              make_uint4(__float_as_uint(v[c + 4 * i]), __float_as_uint(v[c + 4 * i + 1]),
                                         __float_as_uint(v[c + 4 * i + 2]), __float_as_uint(v[c + 4 * i + 3])));
        if (rows) {
            send_slot(map, t, c);
            continue;
        }
        __syncwarp();
        if (c < t.cols) slot_to_any(s, t, c, min(16, t.cols - c));
        skip_slot<kSlots>(t);
    }
}

// (Slot elements outside the matrix are whatever they were: they are added
// to sums that are not stored.)
__device__ __forceinline__ void add_chunk(const Side &s, const WarpTile &t, float (&v)[32]) {
    const bool rows = s.walk == kWalkRows && t.cols == 32;
    if (s.dtype != CONV_FLOAT32) {
        free_slot(t);
        if (rows) rows_to_slot(t, (const char *)s.p + ((int64_t)t.row0 * s.sa + t.b0) * 2, s.sa * 2);
        else if (s.walk != kWalkAlongA && s.sb == 1)
            words_to_slot((const uint16_t *)s.p + (int64_t)t.row0 * s.sa + t.b0, s.sa, t.rows, t.cols, t.slot);
        else any_to_slot(s, t, 0, t.cols);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float r[8];
            unpack8(ptx::ld_shared_v4(piece(t.slot, t.lane, i)), s.dtype, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[8 * i + j] += r[j];
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < 32; c += 16) {
        free_slot(t);
        if (rows) rows_to_slot(t, (const char *)s.p + ((int64_t)t.row0 * s.sa + t.b0 + c) * 4, s.sa * 4);
        else if (c < t.cols) any_to_slot(s, t, c, min(16, t.cols - c));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 q = ptx::ld_shared_v4(piece(t.slot, t.lane, i));
            v[c + 4 * i] += __uint_as_float(q.x), v[c + 4 * i + 1] += __uint_as_float(q.y);
            v[c + 4 * i + 2] += __uint_as_float(q.z), v[c + 4 * i + 3] += __uint_as_float(q.w);
        }
    }
}

// The lane's bias: of its row, or of column b0 + lane for the others to share.
__device__ __forceinline__ float lane_bias(const EpilogueArgs &a, int row0, int b0, int lane) {
    if (!a.bias) return 0.0f;
    const int at = (a.bias_along_a ? row0 : b0) + lane;
    return at < (a.bias_along_a ? a.ma : a.nb) ? load_as_float(a.bias, at, a.bias_dtype) : 0.0f;
}

template <int W>
__device__ __forceinline__ void add_bias(const EpilogueArgs &a, const WarpTile &t, float bias, float (&v)[W]) {
    if (!a.bias) return;
    if (a.bias_along_a) {
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] += bias;
        return;
    }
    // lane j's bias to every row, through 128 bytes of shared memory
    __syncwarp();
    ptx::st_shared_b32(t.bias + t.lane * 4, __float_as_uint(bias));
    __syncwarp();
#pragma unroll
    for (int j = 0; j < W; j += 4) {
        const uint4 b = ptx::ld_shared_v4(t.bias + j * 4);
        split(add2(pair(v[j], v[j + 1]), pair(__uint_as_float(b.x), __uint_as_float(b.y))), &v[j], &v[j + 1]);
        split(add2(pair(v[j + 2], v[j + 3]), pair(__uint_as_float(b.z), __uint_as_float(b.w))), &v[j + 2], &v[j + 3]);
    }
}

__device__ __forceinline__ void load_sums(uint32_t acc, float (&v)[32]) {
    uint32_t u[32];
    ptx::tmem_ld_32x32b_x32(acc, u);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(u[j]);
}

// A 16-bit residual with aligned rows, where the sums are short: the warp's
// second slot takes it by asynchronous copies, a chunk ahead of its use.
__device__ __forceinline__ void fetch_residual(const EpilogueArgs &a, const WarpTile &t, int row0, int rows, int b0) {
    if (a.slots == 2 && b0 + 32 <= a.nb) {
        const char *p = (const char *)a.res.p + ((int64_t)(row0 + t.lane / 4) * a.res.sa + b0) * 2 + (t.lane & 3) * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (t.lane / 4 + 8 * i < rows)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 piece(t.slot + kSlotBytes, t.lane / 4 + 8 * i, t.lane & 3)),
                             "l"(p + (int64_t)(8 * i) * a.res.sa * 2)
                             : "memory");
    }
}

// 32 rows x 32 columns of sums; next: the columns from this chunk to the warp's
// next one in the tile, 0 at the last.
template <int kAct, int kSlots = 1>
__device__ __forceinline__ void finish_values(const EpilogueArgs &a, const WarpTile &t, float (&v)[32], float bias, int next) {
    add_bias(a, t, bias, v);
    if (a.pre.walk) store_chunk<kSlots>(a.pre, &a.map_pre, t, v);
    activate_all<kAct>(a, v);
    if (a.slots == 2 && t.cols == 32) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float r[8];
            unpack8(ptx::ld_shared_v4(piece(t.slot + kSlotBytes, t.lane, i)), a.res.dtype, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[8 * i + j] += r[j];
        }
        __syncwarp();
        if (next) fetch_residual(a, t, t.row0, t.rows, t.b0 + next);
    } else if (a.res.walk) {
        add_chunk(a.res, t, v);
    }
    store_chunk<kSlots>(a.d, &a.map_d, t, v);
}

// ... of those at `acc` in tensor memory.
template <int kAct>
__device__ __forceinline__ void finish_chunk(const EpilogueArgs &a, const WarpTile &t, uint32_t acc, float bias, int next) {
    float v[32];
    load_sums(acc, v);
    finish_values<kAct>(a, t, v, bias, next);
}

// 8 columns of a split tile: every lane on its own row.
__device__ __forceinline__ void store8(const Side &s, const WarpTile &t, const float (&v)[8]) {
    if (t.lane >= t.rows) return;
    const int64_t at = (int64_t)(t.row0 + t.lane) * s.sa + (int64_t)t.b0 * s.sb;
    if (s.walk == kWalkRows && t.cols == 8) {
        if (s.dtype == CONV_FLOAT32) {
            float4 *p = reinterpret_cast<float4 *>((float *)s.p + at);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4 *>((uint16_t *)s.p + at) = pack8(v, s.dtype);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < t.cols) store_from_float(s.p, at + j * s.sb, s.dtype, v[j]);
}

template <int kAct>
__device__ __forceinline__ void finish8(const EpilogueArgs &a, const WarpTile &t, float (&v)[8]) {
    float r[8];
    if (a.res.walk) {
        const int64_t at = (int64_t)(t.row0 + t.lane) * a.res.sa + (int64_t)t.b0 * a.res.sb;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            r[j] = t.lane < t.rows && j < t.cols ? load_as_float(a.res.p, at + j * a.res.sb, a.res.dtype) : 0.0f;
    }
    add_bias(a, t, lane_bias(a, t.row0, t.b0, t.lane), v);
    if (a.pre.walk) store8(a.pre, t, v);
    activate_all<kAct>(a, v);
    if (a.res.walk) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += r[j];
    }
    store8(a.d, t, v);
}

// Adds the runs' partial sums and finishes the product: 32 rows x 8 columns
// per block, lane = row; warp w adds runs w, w + 8, ... and the first warp the
// warps' sums, in order.
template <int kAct>
__device__ __forceinline__ void join_runs(const TileArgs &a, int rows_per_tile) {
    __shared__ __align__(16) float bias[32];
    __shared__ float sums[8][8][32];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    const int tiles = a.tiles_a * a.tiles_b - a.full;  // those cut
    // block: 8 columns of 32 rows, columns fastest
    const int per_half = a.tile_b / 8 * 4, halves = rows_per_tile / kTileA;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int th = blockIdx.x / per_half, in = blockIdx.x - th * per_half;
    const int quad = in / (a.tile_b / 8), c = (in - quad * (a.tile_b / 8)) * 8;
    const int t = th / halves, half = th - t * halves;
    int ia, ib;
    tile_at(a, a.full + t, &ia, &ib);
    WarpTile wt;
    wt.lane = lane;
    wt.slot = 0;  // (unused by 8-column tiles)
    wt.bias = ptx::smem_addr(bias);
    wt.row0 = ia * rows_per_tile + half * kTileA + quad * 32;
    wt.rows = min(32, a.ma - wt.row0);
    wt.b0 = ib * a.tile_b + c;
    wt.cols = min(8, a.nb - wt.b0);
    if (wt.rows <= 0 || wt.cols <= 0) return;
    const float *p = a.part + ((int64_t)th * a.tile_b + c) * kTileA + quad * 32 + lane;
    const int64_t run = (int64_t)tiles * halves * a.tile_b * kTileA;
    float v[8] = {};
#pragma unroll 4
    for (int r = warp; r < a.parts; r += 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += p[r * run + j * kTileA];
    }
    if (warp > 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[warp][j][lane] = v[j];
    }
    __syncthreads();
    if (warp > 0) return;
    for (int w = 1; w < warps; ++w) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += sums[w][j][lane];
    }
    finish8<kAct>(a, wt, v);
}

// ---------------------------------------------------------------- host
inline PFN_cuTensorMapEncodeTiled_v12000 tiled_encoder() {
    static std::atomic<void *> fn{nullptr};
    if (!fn.load()) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(p);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn.load());
}

// Map of a [outer, inner] matrix with `inner` contiguous.
inline bool encode(CUtensorMap *m, int32_t dtype, const void *p, int64_t inner, int64_t outer, int64_t stride, int box_inner,
            int box_outer, CUtensorMapSwizzle swizzle) {
    auto enc = tiled_encoder();
    if (!enc) return false;
    const CUtensorMapDataType t = dtype == CONV_FLOAT32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                  : dtype == CONV_FLOAT16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                  : dtype == CONV_BFLOAT16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                           : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const int64_t size = channel_elem_size(dtype);
    // (one row: any legal stride will do)
    if (outer == 1) stride = round_up(inner * size, 16) / size;
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
    const cuuint64_t strides[1] = {(cuuint64_t)(stride * size)};
    const cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_outer}, ones[2] = {1, 1};
    return enc(m, t, 2, const_cast<void *>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline Side make_side(const void *p, int64_t sa, int64_t sb, int32_t dtype, int64_t ma, int64_t nb) {
    Side s{const_cast<void *>(p), sa, sb, dtype, kWalkNone};
    if (!p) return s;
    const int64_t size = channel_elem_size(dtype);
    // (TMA stores clip to the matrix in units of 16 bytes: rows of other
    // lengths would be written past their end)
    if ((sb == 1 || nb == 1) && (nb * size) % 16 == 0 && (sa * size) % 16 == 0 && (uintptr_t)p % 16 == 0)
        s.walk = kWalkRows;
    else if (nb > 1 && (ma == 1 || sb <= sa))
        s.walk = kWalkAlongB;
    else
        s.walk = kWalkAlongA;
    return s;
}

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace i8c

// product.cu -- D[a,b] = epilogue(sum_k A[a,k] * B[b,k]) for 16-bit float
// operands, on the 5th-generation tensor cores.
//
// Two threads load 64-element k-steps of the operands with TMA (128-byte
// swizzle) into a ring, one thread issues tcgen05.mma into one of two
// accumulators in tensor memory, and twelve warps take the other accumulator
// through bias, pre-activation, activation and residual to the output.
// Either operand may have k or its own dim contiguous: only the tensor map,
// the descriptor strides and the instruction's transpose bits differ, so the
// forward product and both gradients are one kernel.
//
// What bounds it: with long sums the loads' latency over the ring (32 KB per
// k-step and SM; 4 / 5 / 6 stages took 695 / 621 / 582 us on 8192 x 4096 ->
// 16384, as replayed when they were compared) and the power cap (577-626 us
// replayed, 675-680 us among calls on other data: 1.62 PFLOP/s); with short ones what
// an SM moves in and out (50176 x 512 -> 2048: 3.5 us for each round of 76
// tiles, 95 GB/s per SM; 4.9 with GELU and a second output); a single small
// tile takes 3.5 us: 0.6 of set-up, 1.0 for its first loads, 0.3 for the
// sums, 1.5 to finish and leave.
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

bool product_in_place(const void *p, int64_t rows, int64_t rs, int64_t cols, int64_t cs) {
    if (rows <= 1) rs = 0;
    if (cols <= 1) cs = 0;
    if ((uintptr_t)p % 16) return false;
    return (cs <= 1 && rs % 8 == 0) || (rs <= 1 && cs % 8 == 0);
}

namespace {

constexpr int kTileA = 128;        // accumulator lanes of one CTA
constexpr int kStepK = 64;         // k elements per ring stage: one 128-byte row
constexpr int kMaxTileB = 256;     // columns of one accumulator
constexpr int kMaxStages = 12;
constexpr int kThreads = 512;      // 4 control warps, 12 epilogue warps
constexpr int kEpilogueWarps = 12; // (16 would leave 96 registers per thread, and spill)
constexpr int kParts = kEpilogueWarps / 4;                             // epilogue warps on a quarter of the lanes
constexpr int kChunks = (kMaxTileB / 32 + kParts - 1) / kParts;        // 32-column chunks of one of them
constexpr int kSlotBytes = 2048;   // staging of one epilogue warp
constexpr int kBiasBytes = kEpilogueWarps * 128;
constexpr int kRingBytes = 196608;
constexpr int kMaxSplit = 8;       // portable cluster size
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

struct ProductArgs {
    CUtensorMap map_a, map_b, map_d, map_pre;
    Side d, res, pre;
    const void *bias;
    int32_t bias_dtype, bias_along_a;
    int32_t ma, nb;
    int32_t k_steps;
    int32_t tile_b;              // a multiple of 32
    int32_t tiles_a, tiles_b;
    int32_t rows_a;              // rows of a from one tile to the next (and in it)
    int32_t a_mn, b_mn;          // operand's own dim (not k) contiguous
    int32_t a_blocks, b_blocks;  // own dim contiguous and whole blocks of 64: all of a k-step's boxes in one load
    int32_t b_rows, b_boxes;     // rows of B per CTA; TMA boxes per k-step
    int32_t slots;               // staging slots of an epilogue warp: 2 where a residual is loaded ahead
    int32_t stages, stage_bytes; // A is the first 16 KB of a stage
    int32_t split;               // CTAs of a cluster sharing one tile along k (1: none)
    int32_t late_wait;           // waits for the stream's previous kernel at its end, not its start
    int32_t spin;                // short sums: waits poll (latency counts, and nothing else wants the issue slots)
    int32_t parts;               // runs of k, each summed to `part` (1: none),
    int32_t full;                // of the tiles from this one on
    float *part;                 // [run][tile][128-row half][column][row of 128]
    uint32_t idesc;
    uint64_t wait_limit_ns;
    int *status;
};

struct SharedCtl {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2];
    uint32_t tmem_base;
    int32_t abort_flag;
};

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
    d |= (uint64_t)(mn ? (kStepK * 128) >> 4 : 1) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Bounded wait; false when the CTA is giving up (the status word then holds
// the timeout).
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int32_t *abort_flag, uint64_t limit_ns,
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
__device__ __forceinline__ void tile_at(const ProductArgs &a, int t, int *ia, int *ib) {
    constexpr int kBand = 8;
    const int per_band = kBand * a.tiles_b;
    const int band = t / per_band, in = t - band * per_band;
    const int rows = min(kBand, a.tiles_a - band * kBand);
    *ib = in / rows;
    *ia = band * kBand + (in - *ib * rows);
}

// ---------------------------------------------------------------- epilogue
template <int kAct, int W>
__device__ __forceinline__ void activate_all(float (&v)[W]) {
#pragma unroll
    for (int j = 0; j < W; j += 2) activate<kAct>(v[j], v[j + 1]);
}

// One warp's 32 rows x up to 32 columns at (row0, b0), lane = row.  The warp
// owns 2 KB of shared memory, the slot, through which every output, residual
// and pre-activation is turned: rows of 64 bytes (32 columns of a 16-bit
// matrix, 16 of a 32-bit one), each lane writing or reading its own row, and
// runs of a row going to or from global memory.
struct WarpTile {
    int32_t row0, b0, rows, cols;  // rows, cols: how many are inside the matrix and the tile
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
__device__ __noinline__ void slot_to_words(uint16_t *p, int64_t row, int rows, int cols, uint32_t slot) {
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
__device__ __noinline__ void words_to_slot(const uint16_t *p, int64_t row, int rows, int cols, uint32_t slot) {
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
__device__ __noinline__ void slot_to_any(Side s, WarpTile t, int c, int cols) {
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
__device__ __noinline__ void any_to_slot(Side s, WarpTile t, int c, int cols) {
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

__device__ __forceinline__ void store_chunk(const Side &s, const CUtensorMap *map, const WarpTile &t, const float (&v)[32]) {
    const bool rows = s.walk == kWalkRows && t.cols == 32;
    if (s.dtype != CONV_FLOAT32) {
        free_slot(t);
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
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < 32; c += 16) {
        free_slot(t);
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
__device__ __forceinline__ float lane_bias(const ProductArgs &a, int row0, int b0, int lane) {
    if (!a.bias) return 0.0f;
    const int at = (a.bias_along_a ? row0 : b0) + lane;
    return at < (a.bias_along_a ? a.ma : a.nb) ? load_as_float(a.bias, at, a.bias_dtype) : 0.0f;
}

template <int W>
__device__ __forceinline__ void add_bias(const ProductArgs &a, const WarpTile &t, float bias, float (&v)[W]) {
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
__device__ __forceinline__ void fetch_residual(const ProductArgs &a, const WarpTile &t, int row0, int rows, int b0) {
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

// 32 rows x 32 columns of sums at `acc` in tensor memory; next: the columns
// from this chunk to the warp's next one in the tile, 0 at the last.
template <int kAct>
__device__ __forceinline__ void finish_chunk(const ProductArgs &a, const WarpTile &t, uint32_t acc, float bias, int next) {
    float v[32];
    load_sums(acc, v);
    add_bias(a, t, bias, v);
    if (a.pre.walk) store_chunk(a.pre, &a.map_pre, t, v);
    activate_all<kAct>(v);
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
    store_chunk(a.d, &a.map_d, t, v);
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
__device__ __forceinline__ void finish8(const ProductArgs &a, const WarpTile &t, float (&v)[8]) {
    float r[8];
    if (a.res.walk) {
        const int64_t at = (int64_t)(t.row0 + t.lane) * a.res.sa + (int64_t)t.b0 * a.res.sb;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            r[j] = t.lane < t.rows && j < t.cols ? load_as_float(a.res.p, at + j * a.res.sb, a.res.dtype) : 0.0f;
    }
    add_bias(a, t, lane_bias(a, t.row0, t.b0, t.lane), v);
    if (a.pre.walk) store8(a.pre, t, v);
    activate_all<kAct>(v);
    if (a.res.walk) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += r[j];
    }
    store8(a.d, t, v);
}

// ---------------------------------------------------------------- kernel
// kPair: two CTAs of a cluster work on one tile of 256 x tile_b
// (cta_group::2: each holds its 128 rows of A and half the rows of B, the
// first one issues the MMAs for both).  Otherwise one CTA per tile of
// 128 x tile_b, or `split` CTAs of a cluster that each sum part of k and
// then add their partial tiles through distributed shared memory, in order
// of rank.
template <bool kPair, int kAct>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ ProductArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t ring = ptx::smem_addr(smem);
    const uint32_t staging = ring + a.stages * a.stage_bytes;
    const uint32_t bias_smem = staging + kEpilogueWarps * kSlotBytes * a.slots;
    SharedCtl *ctl = reinterpret_cast<SharedCtl *>(smem + (bias_smem - ring) + kBiasBytes);
    if (ring & 1023) {  // the swizzles count on it (true of every launch without static shared memory)
        if (threadIdx.x == 0) atomicExch(a.status, (int)CONV_ERR_ALIGNMENT);
        return;
    }
    volatile int32_t *abort_flag = &ctl->abort_flag;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = (kPair || a.split > 1) ? cluster_rank() : 0;
    const int cluster_size = kPair ? 2 : a.split;
    const int first = blockIdx.x / cluster_size, step = gridDim.x / cluster_size;
    const int tiles = a.tiles_a * a.tiles_b, units = a.full + (tiles - a.full) * a.parts;
    int k_lo = 0, k_hi = a.k_steps;
    if (!kPair && a.split > 1) {
        k_lo = (int)((int64_t)a.k_steps * rank / a.split);
        k_hi = (int)((int64_t)a.k_steps * (rank + 1) / a.split);
    }

    // unit u: a whole tile, then the runs of the cut tiles (the runs of one
    // stretch of k side by side, on the same rows of the operands); sets the
    // k-steps, returns the tile
    auto run_of = [&](int u) {
        if (a.parts > 1) {
            k_lo = 0, k_hi = a.k_steps;
            if (u >= a.full) {
                const int cut = tiles - a.full, p = (u - a.full) / cut;
                k_lo = (int)((int64_t)a.k_steps * p / a.parts);
                k_hi = (int)((int64_t)a.k_steps * (p + 1) / a.parts);
                u -= p * cut;
            }
        }
        return u;
    };

    if (threadIdx.x == 0) {
        ptx::prefetch_tensormap(&a.map_a);
        for (int i = 0; i < a.stages; ++i) {
            ptx::mbar_init(ptx::smem_addr(&ctl->full[i]), 2);  // the two loading threads
            ptx::mbar_init(ptx::smem_addr(&ctl->empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_addr(&ctl->acc_full[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&ctl->acc_empty[i]), kPair ? 2 * kEpilogueWarps : kEpilogueWarps);
        }
        ctl->abort_flag = 0;
        ptx::fence_mbar_init();
    } else if (threadIdx.x == 96) {
        ptx::prefetch_tensormap(&a.map_b);
    }
    __syncthreads();
    // Tensor memory is allocated while the first loads are on their way: the
    // loading warps of a single CTA do not wait for it.  (Those of a pair
    // signal each other's barriers, which have to be there first.)
    uint32_t tmem = 0;
    if (kPair || !(warp == 0 || warp == 3)) {
        if (warp == 2) tmem_alloc<kPair>(ptx::smem_addr(&ctl->tmem_base), 512);
        ptx::tc_fence_before();
        if (kPair) cluster_sync();
        else asm volatile("bar.sync 1, %0;" ::"n"(kThreads - 64) : "memory");
        ptx::tc_fence_after();
        tmem = *(volatile uint32_t *)&ctl->tmem_base;
    }
    // Nothing above reads or writes global memory.  A product beside an
    // independent kernel (the stream's previous one) begins at once: that one
    // let it start only after its own wait (or began the same way behind
    // another such one), so all the kernels before them have ended; it waits
    // before it ends, so that whoever waits for it finds them done.
    if (!a.late_wait) ptx::grid_dependency_wait();
    ptx::launch_dependents();

    if ((warp == 0 || warp == 3) && lane == 0) {
        // ------------------------------------------------ loads: operand A by
        // warp 0, operand B by warp 3 (one thread issuing for both fell behind
        // the MMAs where an operand takes two boxes per k-step)
        const bool is_b = warp == 3;
        const bool mn = is_b ? a.b_mn : a.a_mn;
        const CUtensorMap *map = is_b ? &a.map_b : &a.map_a;
        const int boxes = is_b ? a.b_boxes : 2;
        const bool blocks = is_b ? a.b_blocks : a.a_blocks;
        const uint32_t bytes = (kPair ? 2u : 1u) * (mn ? boxes * 8192u : (is_b ? a.b_rows : kPair ? kTileA : a.rows_a) * 128u);
        Ring rg;
        int64_t issued = 0;
        bool ok = true;
        for (int t = first; t < units && ok; t += step) {
            int ia, ib;
            tile_at(a, run_of(t), &ia, &ib);
            const int own = is_b ? ib * a.tile_b + (kPair ? rank * a.b_rows : 0)
                                 : ia * a.rows_a + (kPair ? rank * kTileA : 0);
            for (int ks = k_lo; ks < k_hi; ++ks) {
                if (!wait_phase(ptx::smem_addr(&ctl->empty[rg.idx]), rg.phase ^ 1u, abort_flag, a.wait_limit_ns, a.status)) {
                    ok = false;
                    break;
                }
                uint32_t bar = ptx::smem_addr(&ctl->full[rg.idx]);
                if (!kPair || rank == 0) ptx::mbar_arrive_expect_tx(bar, bytes);
                if (kPair) bar = map_to_rank(bar, 0);
                const uint32_t dst = ring + rg.idx * a.stage_bytes + (is_b ? 16384 : 0);
                const int k0 = ks * kStepK;
                auto load = [&](uint32_t to, int x, int y) {
                    if constexpr (kPair) tma_load_2d_pair(to, map, x, y, bar);
                    else ptx::tma_load_2d(to, map, x, y, bar);
                };
                if (mn && blocks) {
                    if constexpr (kPair) tma_load_3d_pair(dst, map, 0, k0, own / 64, bar);
                    else tma_load_3d(dst, map, 0, k0, own / 64, bar);
                } else if (mn) {
                    for (int i = 0; i < boxes; ++i) load(dst + i * 8192, own + 64 * i, k0);
                } else {
                    load(dst, k0, own);
                }
                ++issued;
                rg.next(a.stages);
            }
        }
        // Every stage is released by the MMAs that read it; the releases
        // reach both CTAs of a pair, so they have to be in before either
        // leaves.  (A single CTA's are in before its last accumulator is.)
        // After a time-out the copies have to land first (in a pair on the
        // leader's barriers; the cluster barrier below keeps both CTAs), and
        // no release may come.
        const bool drain_copies = *abort_flag && (!kPair || rank == 0);
        for (int s = 0; s < a.stages && (kPair || drain_copies); ++s) {
            const int64_t n = issued / a.stages + (s < issued % a.stages ? 1 : 0);
            if (n == 0) continue;
            const uint32_t bar = ptx::smem_addr(drain_copies ? &ctl->full[s] : &ctl->empty[s]);
            const uint64_t t0 = ptx::global_timer_ns();
            while (!ptx::mbar_try_wait(bar, (uint32_t)((n - 1) & 1)))
                if (ptx::global_timer_ns() - t0 > 10000000) break;
        }
    } else if (warp == 1 && lane == 0 && (!kPair || rank == 0)) {
        // ------------------------------------------------ MMA
        Ring rg;
        int n = 0;
        bool ok = true;
        const uint32_t adv_a = a.a_mn ? 2048 >> 4 : 32 >> 4, adv_b = a.b_mn ? 2048 >> 4 : 32 >> 4;
        for (int t = first; t < units && ok; t += step, ++n) {
            const int slot = n & 1;
            run_of(t);
            if (!wait_phase(ptx::smem_addr(&ctl->acc_empty[slot]), ((n >> 1) & 1) ^ 1u, abort_flag, a.wait_limit_ns, a.status)) break;
            ptx::tc_fence_after();
            const uint32_t d = tmem + slot * kMaxTileB;
            for (int ks = k_lo; ks < k_hi; ++ks) {
                if (!wait_phase(ptx::smem_addr(&ctl->full[rg.idx]), rg.phase, abort_flag, a.wait_limit_ns, a.status, a.spin)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t sa = ring + rg.idx * a.stage_bytes;
                const uint64_t da = operand_desc(sa, a.a_mn), db = operand_desc(sa + 16384, a.b_mn);
#pragma unroll
                for (int i = 0; i < kStepK / 16; ++i)
                    mma<kPair>(d, da + i * adv_a, db + i * adv_b, a.idesc, (ks > k_lo || i > 0) ? 1u : 0u);
                mma_commit<kPair>(ptx::smem_addr(&ctl->empty[rg.idx]));
                rg.next(a.stages);
            }
            if (ok) mma_commit<kPair>(ptx::smem_addr(&ctl->acc_full[slot]));
        }
    } else if (warp >= 4) {
        // ------------------------------------------------ epilogue
        const int e = warp - 4, quad = warp & 3, part = e >> 2;
        WarpTile wt;
        wt.lane = lane;
        wt.slot = staging + e * kSlotBytes * a.slots;
        wt.bias = bias_smem + e * 128;
        int n = 0;
        for (int t = first; t < units; t += step, ++n) {
            int ia, ib;
            tile_at(a, run_of(t), &ia, &ib);
            const int slot = n & 1;
            const int row0 = ia * a.rows_a + (kPair ? rank * kTileA : 0) + quad * 32;
            // this warp's biases, loaded while the tile is being summed
            float bias[kChunks];
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const int c = (part + kParts * i) * 32;
                bias[i] = c < a.tile_b ? lane_bias(a, row0, ib * a.tile_b + c, lane) : 0.0f;
            }
            const int rows = min(32, min(a.ma, (ia + 1) * a.rows_a) - row0);
            if (part * 32 < a.tile_b) fetch_residual(a, wt, row0, rows, ib * a.tile_b + part * 32);
            if (!wait_phase(ptx::smem_addr(&ctl->acc_full[slot]), (n >> 1) & 1, abort_flag, a.wait_limit_ns, a.status, a.spin)) break;
            ptx::tc_fence_after();
            const uint32_t acc = tmem + slot * kMaxTileB + ((uint32_t)(quad * 32) << 16);
            if (k_lo == k_hi) {  // no products: the accumulator was never written
                const uint32_t zero[32] = {};
                for (int c = part * 32; c < a.tile_b; c += 32 * kParts) ptx::tmem_st_32x32b_x32(acc + c, zero);
                ptx::tmem_st_wait();
            }
            wt.row0 = row0;
            wt.rows = rows;
            if (!kPair && a.split > 1) {
                // partial sums to shared memory [column][row], over the
                // ring: its loads and MMAs are done
                for (int c = part * 32; c < a.tile_b; c += 32 * kParts) {
                    uint32_t v[32];
                    ptx::tmem_ld_32x32b_x32(acc + c, v);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        ptx::st_shared_b32(ring + ((c + j) * kTileA + quad * 32 + lane) * 4, v[j]);
                }
                break;  // one tile per cluster; the rest follows the cluster barrier
            }
#pragma unroll 1
            for (int i = 0, c = part * 32; c < a.tile_b; ++i, c += 32 * kParts) {
                wt.b0 = ib * a.tile_b + c;
                wt.cols = min(32, a.nb - wt.b0);
                if (wt.rows <= 0 || wt.cols <= 0) continue;
                if (t >= a.full) {
                    float v[32];
                    load_sums(acc + c, v);
                    float *p = a.part + (((int64_t)(t - a.full) * (kPair ? 2 : 1) + (kPair ? rank : 0)) * a.tile_b + c) * kTileA + quad * 32 + lane;
#pragma unroll
                    for (int j = 0; j < 32; ++j) p[j * kTileA] = v[j];
                    continue;
                }
                finish_chunk<kAct>(a, wt, acc + c, i == 0 ? bias[0] : i == 1 ? bias[1] : bias[kChunks - 1],
                                   c + 32 * kParts < a.tile_b ? 32 * kParts : 0);
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                const uint32_t bar = ptx::smem_addr(&ctl->acc_empty[slot]);
                mbar_arrive_relaxed(kPair ? map_to_rank(bar, 0) : bar);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (lane == 0) ptx::bulk_wait_group_read<0>();
    }

    __syncwarp();
    if (!kPair && a.split > 1) {
        cluster_sync();
        if (warp >= 4 && !*abort_flag) {
            // units of 32 rows x 8 columns, dealt to the cluster's warps
            int ia, ib;
            tile_at(a, first, &ia, &ib);
            const int e = warp - 4;
            WarpTile wt;
            wt.lane = lane;
            wt.slot = 0;  // (unused by 8-column tiles)
            wt.bias = bias_smem + e * 128;
            const int units = a.tile_b / 8 * 4;
            for (int u = e * a.split + (int)rank; u < units; u += kEpilogueWarps * a.split) {
                const int quad = u & 3, c = (u >> 2) * 8;
                wt.row0 = ia * a.rows_a + quad * 32;
                wt.rows = min(32, min(a.ma, (ia + 1) * a.rows_a) - wt.row0);
                wt.b0 = ib * a.tile_b + c;
                wt.cols = min(8, a.nb - wt.b0);
                if (wt.rows <= 0 || wt.cols <= 0) continue;
                float v[8] = {};
#pragma unroll 1
                for (int r0 = 0; r0 < a.split; r0 += 4) {
                    float q[4][8];  // 32 loads in flight
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        // (splits are powers of two: of 2 CTAs, the first is read twice and not added)
                        const uint32_t src = map_to_rank(ring + (c * kTileA + quad * 32 + lane) * 4, r0 + r < a.split ? r0 + r : 0);
#pragma unroll
                        for (int j = 0; j < 8; ++j) q[r][j] = ld_cluster_f32(src + j * kTileA * 4);
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (r0 + r < a.split) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[j] += q[r][j];
                        }
                }
                finish8<kAct>(a, wt, v);
            }
        }
        cluster_sync();  // peers read this CTA's shared memory until here
    } else if (kPair) {
        cluster_sync();
    } else {
        __syncthreads();
    }
    ptx::tc_fence_after();
    if (warp == 2) tmem_dealloc<kPair>(tmem, 512);
    if (a.late_wait) ptx::grid_dependency_wait();
}

// Adds the runs' partial sums and finishes the product: 32 rows x 8 columns
// per block, lane = row; warp w adds runs w, w + 8, ... and the first warp the
// warps' sums, in order.
template <int kAct>
__global__ void __launch_bounds__(256) product_join_kernel(const __grid_constant__ ProductArgs a, int rows_per_tile) {
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
PFN_cuTensorMapEncodeTiled_v12000 tiled_encoder() {
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
bool encode(CUtensorMap *m, int32_t dtype, const void *p, int64_t inner, int64_t outer, int64_t stride, int box_inner,
            int box_outer, CUtensorMapSwizzle swizzle) {
    auto enc = tiled_encoder();
    if (!enc) return false;
    const CUtensorMapDataType t = dtype == CONV_FLOAT32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                  : dtype == CONV_FLOAT16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int64_t size = channel_elem_size(dtype);
    // (one row: any legal stride will do)
    if (outer == 1) stride = round_up(inner * size, 16) / size;
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
    const cuuint64_t strides[1] = {(cuuint64_t)(stride * size)};
    const cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_outer}, ones[2] = {1, 1};
    return enc(m, t, 2, const_cast<void *>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map of an operand whose own dim is contiguous and made of whole blocks of
// 64: [block][k][64], `boxes` blocks of 64 k per load.
bool encode_blocks(CUtensorMap *m, int32_t dtype, const void *p, int64_t own, int64_t k, int64_t stride, int boxes) {
    auto enc = tiled_encoder();
    if (!enc) return false;
    if (k == 1) stride = round_up(own, 8);
    const cuuint64_t dims[3] = {64, (cuuint64_t)k, (cuuint64_t)(own / 64)};
    const cuuint64_t strides[2] = {(cuuint64_t)(stride * 2), 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)kStepK, (cuuint32_t)boxes}, ones[3] = {1, 1, 1};
    return enc(m, dtype == CONV_FLOAT16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
               const_cast<void *>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

Side make_side(const void *p, int64_t sa, int64_t sb, int32_t dtype, int64_t ma, int64_t nb) {
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

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// Clusters of one-CTA-per-SM blocks that run at once (as
// cudaOccupancyMaxActiveClusters counts them on the 152 SMs: processor
// clusters are not all of one size).
int64_t active_clusters(int size) { return size == 1 ? kSms : size == 2 ? kSms / 2 : size == 4 ? 36 : 15; }

ProductPlan product_plan(int64_t ma, int64_t nb, int64_t k) {
    ProductPlan pl;
    // Few rows: the long dim becomes the tile's 128 lanes and the few rows its
    // columns, so that no lanes idle and every CTA streams its own weights.
    if (ma < nb && ma <= 128) {
        pl.swap = true;
        std::swap(ma, nb);
    }
    const int64_t k_steps = cdiv(k, kStepK);
    // Pairs where there are enough tiles to fill the GPU, or enough k-steps in
    // all of them to fill it with runs of at least 16 k-steps: a pair tile
    // loads half the operand bytes per product of a 128 x 128 tile.  (The
    // weight gradient of 50176 rows, 256 -> 1024: 72 us as 128 x 128 tiles in
    // clusters of 8.)
    const int64_t wide = nb > 128 ? 256 : 128;
    const int64_t pair_tiles = cdiv(ma, 256) * cdiv(nb, wide);
    if (nb > 64 && ma > 128 && (pair_tiles * 2 >= kSms || pair_tiles * k_steps >= kSms / 2 * 16)) {
        pl.pair = true;
        pl.tile_b = (int32_t)wide;
        // (a k-step takes 0.34 us at 256 columns and still 0.31 at 192 and 0.30
        // at 128: narrower tiles for a fuller last round do not pay)
        pl.tiles_a = cdiv(ma, 256);
        pl.tiles_b = cdiv(nb, pl.tile_b);
        const int64_t tiles = pl.tiles_a * pl.tiles_b;
        // Fewer tiles than pairs: all of them in runs.  A last round that
        // leaves half the pairs idle or more: its tiles in runs, where that
        // saves 40 k-steps or more (14 us; the joining kernel takes about 8).
        const int64_t last = tiles % (kSms / 2);
        int64_t parts = 1;
        if (tiles * 2 < kSms) parts = std::min(kSms / 2 / tiles, k_steps / 8);
        else if (last > 0) parts = std::min<int64_t>(kSms / 2 / last, 8);
        if (parts > 1 && tiles * 2 >= kSms && k_steps - k_steps / parts < 40) parts = 1;
        pl.full = tiles;
        if (parts > 1) {
            pl.parts = (int32_t)parts;
            pl.full = tiles * 2 < kSms ? 0 : tiles - last;
            pl.part_bytes = (size_t)(parts * (tiles - pl.full) * 256 * pl.tile_b * 4);
        }
        return pl;
    }
    // Single CTAs with narrower tiles, split along k in clusters while that
    // brings more SMs in.
    pl.tile_b = (int32_t)std::min<int64_t>(round_up(nb, 32), 256);
    while (pl.tile_b > 64 && cdiv(ma, kTileA) * cdiv(nb, pl.tile_b) * 2 <= kSms)
        pl.tile_b = (int32_t)round_up(pl.tile_b / 2, 32);
    pl.tiles_a = cdiv(ma, kTileA);
    pl.tiles_b = cdiv(nb, pl.tile_b);
    const int64_t tiles = pl.tiles_a * pl.tiles_b;
    while (pl.split < kMaxSplit && tiles <= active_clusters(pl.split * 2) && k_steps >= pl.split * 4) pl.split *= 2;
    return pl;
}

conv_status product_launch(const Product &given, void *workspace, void *stream) {
    if (given.ma == 0 || given.nb == 0) return CONV_OK;
    if (product_rows_applies(given)) return product_rows_launch(given, stream);
    Product pr = given;
    const ProductPlan pl = product_plan(pr.ma, pr.nb, pr.k);
    if (pl.tiles_a * pl.tiles_b > INT32_MAX / kMaxSplit) return CONV_ERR_TOO_LARGE;
    if (pl.swap) {
        std::swap(pr.ma, pr.nb);
        std::swap(pr.a, pr.b);
        std::swap(pr.d_sa, pr.d_sb);
        std::swap(pr.res_sa, pr.res_sb);
        std::swap(pr.pre_sa, pr.pre_sb);
        pr.bias_along_a = !pr.bias_along_a;
    }
    ProductArgs a;
    a.ma = (int32_t)pr.ma, a.nb = (int32_t)pr.nb;
    a.k_steps = (int32_t)cdiv(pr.k, kStepK);
    a.d = make_side(pr.d, pr.d_sa, pr.d_sb, pr.d_dtype, pr.ma, pr.nb);
    a.res = make_side(pr.res, pr.res_sa, pr.res_sb, pr.d_dtype, pr.ma, pr.nb);
    a.pre = make_side(pr.pre, pr.pre_sa, pr.pre_sb, pr.in_dtype, pr.ma, pr.nb);
    a.bias = pr.bias, a.bias_dtype = pr.bias_dtype, a.bias_along_a = pr.bias_along_a;
    a.wait_limit_ns = wait_limit_ns();
    a.status = device_status_word();
    if (!a.status) return CONV_ERR_CUDA;

    // k contiguous, or else the operand's own dim
    a.a_mn = !(pr.a.s_k == 1 || pr.k <= 1) || (pr.a.s_mn == 1 && pr.k <= 1);
    a.b_mn = !(pr.b.s_k == 1 || pr.k <= 1) || (pr.b.s_mn == 1 && pr.k <= 1);

    const bool pair = pl.pair;
    a.tile_b = pl.tile_b;
    a.tiles_a = (int32_t)pl.tiles_a;
    a.tiles_b = (int32_t)pl.tiles_b;
    a.rows_a = pair ? 256 : kTileA;
    a.split = pl.split;
    a.parts = pl.parts;
    a.part = (float *)workspace;
    if (!pair && !a.a_mn && pl.parts == 1) {
        // Fewer tiles than SMs, each a stream of operand A: shorter tiles for
        // more SMs (at least 64 rows, which keeps the loads of B the smaller
        // part; whole 32-row stores where TMA makes them, since it would not
        // stop at a tile's end).
        const int64_t most = active_clusters(pl.split) / pl.tiles_b;
        const bool sent = a.d.walk == kWalkRows || a.pre.walk == kWalkRows;
        const int64_t rows = round_up(std::max<int64_t>(cdiv(pr.ma, most), 64), sent ? 32 : 4);
        if (rows < kTileA && pl.tiles_a < most) {
            a.rows_a = (int32_t)rows;
            a.tiles_a = (int32_t)cdiv(pr.ma, rows);
        }
    }
    a.b_rows = pair ? a.tile_b / 2 : a.tile_b;
    a.late_wait = pr.beside_previous;
    a.spin = !pair && a.k_steps <= 32 * a.split;
    const int64_t tiles = (int64_t)a.tiles_a * a.tiles_b;
    a.full = (int32_t)(pl.parts > 1 ? pl.full : tiles);
    const int64_t units = a.full + (tiles - a.full) * pl.parts;
    const int sms = device_sm_count(), cluster = pair ? 2 : a.split;
    const int grid = a.split > 1 ? (int)units * a.split : (int)std::min<int64_t>(units, sms / cluster) * cluster;
    a.b_boxes = (int32_t)cdiv(a.b_rows, 64);
    a.stage_bytes = 16384 + (int32_t)round_up(a.b_mn ? a.b_boxes * 8192 : a.b_rows * 128, 1024);
    // (long sums hide the epilogue and want the slots' stage of the ring, see
    // the stages' times at the head of this file)
    a.slots = a.res.walk == kWalkRows && a.res.dtype != CONV_FLOAT32 && a.split == 1 && pl.parts == 1 && a.k_steps <= 24 ? 2 : 1;
    a.stages = std::min(kMaxStages, (kRingBytes - (a.slots - 1) * kEpilogueWarps * kSlotBytes) / a.stage_bytes);
    const int tile_a = pair ? 256 : 128;
    a.idesc = (1u << 4) | ((pr.in_dtype == CONV_BFLOAT16 ? 1u : 0u) << 7) | ((pr.in_dtype == CONV_BFLOAT16 ? 1u : 0u) << 10) |
              ((a.a_mn ? 1u : 0u) << 15) | ((a.b_mn ? 1u : 0u) << 16) | ((uint32_t)(a.tile_b >> 3) << 17) |
              ((uint32_t)(tile_a >> 4) << 24);

    if (a.k_steps > 0) {
        const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
        // (blocks as the outermost dim step by 128 bytes; a tile starts on one)
        a.a_blocks = a.a_mn && pr.ma % 64 == 0;
        a.b_blocks = a.b_mn && pr.nb % 64 == 0 && a.tile_b % 64 == 0 && a.b_rows % 64 == 0;
        const bool ok_a = a.a_blocks ? encode_blocks(&a.map_a, pr.in_dtype, pr.a.p, pr.ma, pr.k, pr.a.s_k, 2)
                          : a.a_mn ? encode(&a.map_a, pr.in_dtype, pr.a.p, pr.ma, pr.k, pr.a.s_k, 64, kStepK, sw)
                                 : encode(&a.map_a, pr.in_dtype, pr.a.p, pr.k, pr.ma, pr.a.s_mn, kStepK, pair ? kTileA : a.rows_a, sw);
        const bool ok_b = a.b_blocks ? encode_blocks(&a.map_b, pr.in_dtype, pr.b.p, pr.nb, pr.k, pr.b.s_k, a.b_boxes)
                          : a.b_mn ? encode(&a.map_b, pr.in_dtype, pr.b.p, pr.nb, pr.k, pr.b.s_k, 64, kStepK, sw)
                                 : encode(&a.map_b, pr.in_dtype, pr.b.p, pr.k, pr.nb, pr.b.s_mn, kStepK, a.b_rows, sw);
        if (!ok_a || !ok_b) return CONV_ERR_CUDA;
    }
    for (auto [s, m] : {std::pair<Side *, CUtensorMap *>{&a.d, &a.map_d}, {&a.pre, &a.map_pre}})
        if (s->walk == kWalkRows &&
            !encode(m, s->dtype, s->p, pr.nb, pr.ma, s->sa, s->dtype == CONV_FLOAT32 ? 16 : 32, 32,
                    CU_TENSOR_MAP_SWIZZLE_64B))
            return CONV_ERR_CUDA;

    const size_t smem = (size_t)a.stages * a.stage_bytes + kEpilogueWarps * kSlotBytes * a.slots + kBiasBytes + sizeof(SharedCtl);
    // the kernel with the call's activation, for CTA pairs or single CTAs
    typedef void (*Kernel)(ProductArgs);
    static const Kernel kernels[2][5] = {
        {product_kernel<false, CONV_ACT_NONE>, product_kernel<false, CONV_ACT_RELU>, product_kernel<false, CONV_ACT_GELU>,
         product_kernel<false, CONV_ACT_GELU_TANH>, product_kernel<false, CONV_ACT_SILU>},
        {product_kernel<true, CONV_ACT_NONE>, product_kernel<true, CONV_ACT_RELU>, product_kernel<true, CONV_ACT_GELU>,
         product_kernel<true, CONV_ACT_GELU_TANH>, product_kernel<true, CONV_ACT_SILU>}};
    const Kernel kernel = kernels[pair][pr.act];
    static std::atomic<bool> ready[64][2][5];  // (check_device admits 64 devices)
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CONV_ERR_CUDA;
    if (!ready[dev][pair][pr.act].load()) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448) != cudaSuccess)
            return CONV_ERR_CUDA;
        ready[dev][pair][pr.act].store(true);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cluster, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return CONV_ERR_CUDA;
    if (a.parts > 1) {
        typedef void (*Join)(ProductArgs, int);
        static const Join joins[5] = {product_join_kernel<CONV_ACT_NONE>, product_join_kernel<CONV_ACT_RELU>,
                                      product_join_kernel<CONV_ACT_GELU>, product_join_kernel<CONV_ACT_GELU_TANH>,
                                      product_join_kernel<CONV_ACT_SILU>};
        const int64_t blocks = (tiles - a.full) * (tile_a / 32) * (a.tile_b / 8);
        if (!launch_behind(joins[pr.act], dim3((unsigned)blocks), 32 * std::min(8, a.parts), 0, (cudaStream_t)stream, a, tile_a))
            return CONV_ERR_CUDA;
    }
    return CONV_OK;
}

}  // namespace i8c

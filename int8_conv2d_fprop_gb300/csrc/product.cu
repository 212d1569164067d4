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
#include "product_tiles.cuh"
#include "tc_ptx.cuh"

namespace i8c {

bool product_in_place(const void *p, int64_t rows, int64_t rs, int64_t cols, int64_t cs) {
    if (rows <= 1) rs = 0;
    if (cols <= 1) cs = 0;
    if ((uintptr_t)p % 16) return false;
    return (cs <= 1 && rs % 8 == 0) || (rs <= 1 && cs % 8 == 0);
}

namespace {

constexpr int kStepK = 64;         // k elements per ring stage: one 128-byte row
constexpr int kMaxTileB = 256;     // columns of one accumulator
constexpr int kMaxStages = 12;
constexpr int kThreads = 512;      // 4 control warps, 12 epilogue warps
constexpr int kEpilogueWarps = 12; // (16 would leave 96 registers per thread, and spill)
constexpr int kParts = kEpilogueWarps / 4;                             // epilogue warps on a quarter of the lanes
constexpr int kChunks = (kMaxTileB / 32 + kParts - 1) / kParts;        // 32-column chunks of one of them
constexpr int kBiasBytes = kEpilogueWarps * 128;
constexpr int kRingBytes = 196608;
constexpr int kMaxSplit = 8;       // portable cluster size

struct ProductArgs : TileArgs {
    CUtensorMap map_a, map_b;
    int32_t k_steps;
    int32_t rows_a;              // rows of a from one tile to the next (and in it)
    int32_t a_mn, b_mn;          // operand's own dim (not k) contiguous
    int32_t a_blocks, b_blocks;  // own dim contiguous and whole blocks of 64: all of a k-step's boxes in one load
    int32_t b_rows, b_boxes;     // rows of B per CTA; TMA boxes per k-step
    int32_t stages, stage_bytes; // A is the first 16 KB of a stage
    int32_t split;               // CTAs of a cluster sharing one tile along k (1: none)
    int32_t late_wait;           // waits for the stream's previous kernel at its end, not its start
    int32_t spin;                // short sums: waits poll (latency counts, and nothing else wants the issue slots)
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
            // (a warp stops as a whole: its tensor-memory loads take all lanes)
            if (!__all_sync(0xffffffffu, wait_phase(ptx::smem_addr(&ctl->acc_full[slot]), (n >> 1) & 1, abort_flag, a.wait_limit_ns, a.status, a.spin)))
                break;
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

template <int kAct>
__global__ void __launch_bounds__(256) product_join_kernel(const __grid_constant__ ProductArgs a, int rows_per_tile) {
    join_runs<kAct>(a, rows_per_tile);
}

// ---------------------------------------------------------------- host
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

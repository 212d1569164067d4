// scaled_product.cu -- D[a,b] = epilogue(sum over blocks of 128 k of
// scale_a * scale_b * sum_k A[a,k] * B[b,k]) for 8-bit float operands, on the
// 5th-generation tensor cores.
//
// The tensor cores sum one block of 128 k at a time (four MMAs of 32 k) into
// one of two accumulators in tensor memory; eight warps take the other one,
// multiply it by the block's scales and add it to 32-bit sums that they keep
// in registers over all of k.  So every block costs a pass over the
// accumulator: 128 x 256 values per CTA and block, read from tensor memory and
// multiplied in packed pairs, against the 512 cycles that the MMAs take.  Two
// accumulators let the MMAs run a block ahead, and through the epilogue, two.
// What bounds it is that pass: 900 cycles per block with its waits and loads
// (8192 x 4096 -> 16384 540-556 us, 2.0 PFLOP/s; 8192 x 16384 -> 4096 2.2).
// Warps: 0 and 3 load the operands by TMA (128 bytes of k are one swizzled
// row), 1 issues the MMAs, 2 copies the scales, 4 to 11 sum and finish.  The
// control warps give registers to the summing ones, whose 128 columns of sums
// do not fit otherwise.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "channel.h"
#include "channel_launch.cuh"
#include "channel_math.cuh"
#include "product_tiles.cuh"
#include "tc_ptx.cuh"

namespace i8c {
namespace {

constexpr int kBlockK = 128;       // k elements of a block, bytes of a swizzled row
constexpr int kMaxTileB = 256;
constexpr int kMaxStages = 8;
constexpr int kSumWarps = 8;       // two to a quarter of the lanes, each half the columns
constexpr int kThreads = 128 + 32 * kSumWarps;
constexpr int kBatch = 4;          // blocks whose scales come together
constexpr int kScaleSlots = 2;     // batches on their way
constexpr int kScaleBytes = (kTileA + kMaxTileB) * 4;  // of a block
constexpr int kBiasBytes = kSumWarps * 128;
// staging slots of a summing warp: four chunks of 32 columns of 16 bits, a tile's
// all on their way at once (twice as many turns for 32 bits, and a
// pre-activation takes its own)
constexpr int kSlots = 4;
constexpr int kRingBytes = 147456;
// registers: 384 threads start with 168 each; the summing warps' 128 sums, 32
// values on their way and the rest of their state take up to 224
constexpr int kControlRegs = 48, kSumRegs = 224, kLaunchRegs = 168;
static_assert(128 * kControlRegs + 32 * kSumWarps * kSumRegs <= kThreads * kLaunchRegs);

struct ScaleArgs {
    const float *p;
    int64_t rs, cs;
    int32_t shift;               // rows that share a scale: 1 << shift
    int32_t rows;                // of the operand
};

struct ScaledArgs : TileArgs {
    CUtensorMap map_a, map_b;
    ScaleArgs sa, sb;
    int32_t blocks;              // of k
    int32_t stages, stage_bytes; // A is the first 16 KB of a stage
    uint32_t idesc;
    uint64_t wait_limit_ns;
    int *status;
};

struct SharedCtl {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t scale_full[kScaleSlots], scale_empty[kScaleSlots];
    uint32_t tmem_base;
    int32_t abort_flag;
};

// True in one thread of the warp, whose threads are all here.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

__device__ __forceinline__ void mma8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Four bytes to shared memory, zeros where there is nothing to read.
__device__ __forceinline__ void copy_async4(uint32_t dst, const float *src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
// Arrives (once, of the expected count) when this thread's copies so far have landed.
__device__ __forceinline__ void arrive_behind_copies(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// A bounded wait without a call (the summing warps have no registers to put
// away) that polls: a suspended thread resumes some time after its phase is
// complete, and here every block of k waits for the one before.
__device__ __forceinline__ bool wait_polling(uint32_t bar, uint32_t parity, volatile int32_t *abort_flag, uint64_t limit_ns,
                                             int *status) {
    if (ptx::mbar_test_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::global_timer_ns();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (ptx::mbar_test_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (ptx::global_timer_ns() - t0 > limit_ns) {
            *abort_flag = 1;
            atomicExch(status, (int)CONV_ERR_DEVICE_TIMEOUT);
            return false;
        }
    }
}

// Whether all lanes have got what they waited for.  A warp gives up as a whole:
// the tensor-memory loads and the barriers of a warp take all its lanes.
__device__ __forceinline__ bool all_lanes(bool got) { return __all_sync(0xffffffffu, got); }

// sum += {lo, hi} * s
__device__ __forceinline__ void add_scaled(Pair &sum, uint32_t lo, uint32_t hi, Pair s) {
    asm("{\n\t.reg .b64 p;\n\tmov.b64 p, {%1, %2};\n\tfma.rn.f32x2 %0, p, %3, %0;\n\t}" : "+l"(sum.v) : "r"(lo), "r"(hi), "l"(s.v));
}

// One CTA works on a tile of 128 x 2 kCols.
// kPerColumn: B has a scale for each row, else one for the 128 that a summing
// warp's columns lie in.
template <int kCols, bool kPerColumn>
__global__ void __launch_bounds__(kThreads, 1) scaled_product_kernel(const __grid_constant__ ScaledArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int kTileB = 2 * kCols;
    const uint32_t ring = ptx::smem_addr(smem);
    const uint32_t staging = ring + a.stages * a.stage_bytes;
    const uint32_t scales = staging + kSumWarps * kSlots * kSlotBytes;
    const uint32_t bias_smem = scales + kScaleSlots * kBatch * kScaleBytes;
    SharedCtl *ctl = reinterpret_cast<SharedCtl *>(smem + (bias_smem - ring) + kBiasBytes);
    if (ring & 1023) {  // the swizzles count on it (true of every launch without static shared memory)
        if (threadIdx.x == 0) atomicExch(a.status, (int)CONV_ERR_ALIGNMENT);
        return;
    }
    volatile int32_t *abort_flag = &ctl->abort_flag;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int first = blockIdx.x, step = gridDim.x;
    const int tiles = a.tiles_a * a.tiles_b, units = a.full + (tiles - a.full) * a.parts;

    // unit u: a whole tile, then the runs of the cut tiles; sets the blocks of k, returns the tile
    int k_lo = 0, k_hi = a.blocks;
    auto run_of = [&](int u) {
        if (a.parts > 1) {
            k_lo = 0, k_hi = a.blocks;
            if (u >= a.full) {
                const int cut = tiles - a.full, p = (u - a.full) / cut;
                k_lo = (int)((int64_t)a.blocks * p / a.parts);
                k_hi = (int)((int64_t)a.blocks * (p + 1) / a.parts);
                u -= p * cut;
            }
        }
        return u;
    };

    if (threadIdx.x == 0) {
        if (a.blocks > 0) ptx::prefetch_tensormap(&a.map_a);
        for (int i = 0; i < a.stages; ++i) {
            ptx::mbar_init(ptx::smem_addr(&ctl->full[i]), 2);  // the two loading threads
            ptx::mbar_init(ptx::smem_addr(&ctl->empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_addr(&ctl->acc_full[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&ctl->acc_empty[i]), kSumWarps);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            ptx::mbar_init(ptx::smem_addr(&ctl->scale_full[i]), 32);
            ptx::mbar_init(ptx::smem_addr(&ctl->scale_empty[i]), kSumWarps);
        }
        ctl->abort_flag = 0;
        ptx::fence_mbar_init();
    } else if (threadIdx.x == 96 && a.blocks > 0) {
        ptx::prefetch_tensormap(&a.map_b);
    }
    __syncthreads();
    if (warp == 2) tmem_alloc<false>(ptx::smem_addr(&ctl->tmem_base), 512);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *(volatile uint32_t *)&ctl->tmem_base;
    // Nothing above reads or writes global memory.
    ptx::grid_dependency_wait();
    ptx::launch_dependents();

    if (warp < 4) {
        ptx::setmaxnreg_dec<kControlRegs>();
        if ((warp == 0 || warp == 3) && lane == 0) {
            // ------------------------------------------------ loads: operand A by warp 0, operand B by warp 3
            const bool is_b = warp == 3;
            const CUtensorMap *map = is_b ? &a.map_b : &a.map_a;
            const uint32_t bytes = (is_b ? kTileB : kTileA) * kBlockK;
            Ring rg;
            int64_t issued = 0;
            bool ok = true;
            for (int t = first; t < units && ok; t += step) {
                int ia, ib;
                tile_at(a, run_of(t), &ia, &ib);
                const int own = is_b ? ib * kTileB : ia * kTileA;
                for (int kb = k_lo; kb < k_hi; ++kb) {
                    if (!wait_phase(ptx::smem_addr(&ctl->empty[rg.idx]), rg.phase ^ 1u, abort_flag, a.wait_limit_ns, a.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = ptx::smem_addr(&ctl->full[rg.idx]), dst = ring + rg.idx * a.stage_bytes;
                    ptx::mbar_arrive_expect_tx(bar, bytes);
                    ptx::tma_load_2d(dst + (is_b ? 16384 : 0), map, kb * kBlockK, own, bar);
                    ++issued;
                    rg.next(a.stages);
                }
            }
            // (every stage's release is in before the last accumulator is)
            // After a time-out the copies have to land first.
            for (int s = 0; s < a.stages && *abort_flag; ++s) {
                const int64_t n = issued / a.stages + (s < issued % a.stages ? 1 : 0);
                if (n == 0) continue;
                const uint32_t bar = ptx::smem_addr(&ctl->full[s]);
                const uint64_t t0 = ptx::global_timer_ns();
                while (!ptx::mbar_try_wait(bar, (uint32_t)((n - 1) & 1)))
                    if (ptx::global_timer_ns() - t0 > 10000000) break;
            }
        } else if (warp == 1) {
            // ------------------------------------------------ MMA: a block of k to an accumulator
            // (The whole warp walks, one thread issues: descriptors that are
            // uniform over a warp stay in uniform registers.  In a branch of one
            // thread, four MMAs with their commit took 770 cycles to issue
            // instead of the 513 that the tensor cores need for them.)
            const bool issues = elect_one();
            Ring rg;
            uint32_t n = 0, issued = 0;
            bool ok = true;
            for (int t = first; t < units && ok; t += step) {
                run_of(t);
                for (int kb = k_lo; kb < k_hi && ok; ++kb, ++n) {
                    const uint32_t slot = n & 1;
                    ok = wait_polling(ptx::smem_addr(&ctl->acc_empty[slot]), ((n >> 1) & 1) ^ 1u, abort_flag, a.wait_limit_ns, a.status) &&
                         wait_polling(ptx::smem_addr(&ctl->full[rg.idx]), rg.phase, abort_flag, a.wait_limit_ns, a.status);
                    ptx::tc_fence_after();
                    const uint32_t at = ring + rg.idx * a.stage_bytes, d = tmem + slot * kMaxTileB;
                    const uint64_t da = ptx::smem_desc_sw128(at), db = ptx::smem_desc_sw128(at + 16384);
                    if (issues && ok) {
                        issued = n + 1;
#pragma unroll
                        for (int i = 0; i < kBlockK / 32; ++i) mma8(d, da + i * 2, db + i * 2, a.idesc, i > 0 ? 1u : 0u);
                        ptx::mma_commit(ptx::smem_addr(&ctl->acc_full[slot]));
                        ptx::mma_commit(ptx::smem_addr(&ctl->empty[rg.idx]));
                    }
                    ok = all_lanes(ok);  // (behind the MMAs: a vote before them took 2 % of the time)
                    rg.next(a.stages);
                }
            }
            // After a time-out the MMAs under way have to end before their
            // shared and tensor memory goes: the last one's commit covers all.
            // (Else the summing warps have waited for every accumulator.)
            if (*abort_flag && issued > 0) {
                const uint64_t t0 = ptx::global_timer_ns();
                while (!ptx::mbar_test_wait(ptx::smem_addr(&ctl->acc_full[(issued - 1) & 1]), ((issued - 1) >> 1) & 1))
                    if (ptx::global_timer_ns() - t0 > 10000000) break;
            }
        } else if (warp == 2) {
            // ------------------------------------------------ scales: of this CTA's rows, and of the tile's columns
            Ring rg;
            bool ok = true;
            for (int t = first; t < units && ok; t += step) {
                int ia, ib;
                tile_at(a, run_of(t), &ia, &ib);
                const int row0 = ia * kTileA, col0 = ib * kTileB;
                const float *pa[kTileA / 32], *pb[kPerColumn ? kTileB / 32 : 1];
                bool in_a[kTileA / 32], in_b[kPerColumn ? kTileB / 32 : 1];
#pragma unroll
                for (int i = 0; i < kTileA / 32; ++i) {
                    const int r = row0 + i * 32 + lane;
                    in_a[i] = r < a.sa.rows;
                    pa[i] = a.sa.p + (in_a[i] ? (int64_t)(r >> a.sa.shift) * a.sa.rs : 0);
                }
#pragma unroll
                for (int i = 0; i < (kPerColumn ? kTileB / 32 : 1); ++i) {
                    const int r = kPerColumn ? col0 + i * 32 + lane : col0 + (lane & 1) * kCols;
                    in_b[i] = r < a.sb.rows && (kPerColumn || lane < 2);
                    pb[i] = a.sb.p + (in_b[i] ? (int64_t)(r >> a.sb.shift) * a.sb.rs : 0);
                }
                for (int kb = k_lo; kb < k_hi; kb += kBatch) {
                    if (!wait_phase(ptx::smem_addr(&ctl->scale_empty[rg.idx]), rg.phase ^ 1u, abort_flag, a.wait_limit_ns, a.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t to = scales + rg.idx * kBatch * kScaleBytes + lane * 4;
#pragma unroll
                    for (int q = 0; q < kBatch; ++q) {
                        if (kb + q >= k_hi) break;
#pragma unroll
                        for (int i = 0; i < kTileA / 32; ++i) copy_async4(to + q * kScaleBytes + i * 128, pa[i] + (kb + q) * a.sa.cs, in_a[i]);
#pragma unroll
                        for (int i = 0; i < (kPerColumn ? kTileB / 32 : 1); ++i)
                            if (kPerColumn || lane < 2)
                                copy_async4(to + q * kScaleBytes + kTileA * 4 + i * 128, pb[i] + (kb + q) * a.sb.cs, in_b[i]);
                    }
                    arrive_behind_copies(ptx::smem_addr(&ctl->scale_full[rg.idx]));
                    rg.next(kScaleSlots);
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else {
        // ------------------------------------------------ sums
        ptx::setmaxnreg_inc<kSumRegs>();
        const int e = warp - 4, quad = warp & 3, part = e >> 2;
        WarpTile wt;
        wt.lane = lane;
        wt.slot = staging + e * kSlots * kSlotBytes;
        wt.bias = bias_smem + e * 128;
        Ring sr;
        uint32_t n = 0;
        bool ok = true;
        for (int t = first; t < units && ok; t += step) {
            int ia, ib;
            tile_at(a, run_of(t), &ia, &ib);
            Pair sum[kCols / 2];
#pragma unroll
            for (int j = 0; j < kCols / 2; ++j) sum[j] = pair(0.0f);
            for (int k0 = k_lo; k0 < k_hi && ok; k0 += kBatch) {
                // a batch's scales: of the row, and with it the columns' where they have one
                const uint32_t at = scales + sr.idx * kBatch * kScaleBytes;
                // (a lane that has given up goes through the batch with the others,
                // without waiting)
                ok = wait_polling(ptx::smem_addr(&ctl->scale_full[sr.idx]), sr.phase, abort_flag, a.wait_limit_ns, a.status);
                const int k1 = min(k_hi, k0 + kBatch);
#pragma unroll 1
                for (int kb = k0; kb < k1; ++kb, ++n) {
                    const uint32_t slot = n & 1, mine = at + (kb - k0) * kScaleBytes;
                    float s = __uint_as_float(ptx::ld_shared_b32(mine + (quad * 32 + lane) * 4));
                    if constexpr (!kPerColumn) s *= __uint_as_float(ptx::ld_shared_b32(mine + (kTileA + part) * 4));
                    ok = ok && wait_polling(ptx::smem_addr(&ctl->acc_full[slot]), (n >> 1) & 1, abort_flag, a.wait_limit_ns, a.status);
                    ptx::tc_fence_after();
                    const uint32_t acc = tmem + slot * kMaxTileB + part * kCols + ((uint32_t)(quad * 32) << 16);
                    const Pair s2 = pair(s);
                    uint32_t u[2][16];
                    ptx::tmem_ld_32x32b_x16(acc, u[0]);
#pragma unroll
                    for (int c = 0; c < kCols / 16; ++c) {
                        ptx::tmem_ld_wait();
                        if (c + 1 < kCols / 16) {
                            ptx::tmem_ld_32x32b_x16(acc + (c + 1) * 16, u[(c + 1) & 1]);
                        } else {
                            // everything of this accumulator is in registers
                            // (of all lanes: the wait is the warp's)
                            ptx::tc_fence_before();
                            if (lane == 0) mbar_arrive_relaxed(ptx::smem_addr(&ctl->acc_empty[slot]));
                        }
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            Pair &lo = sum[(c * 16 + j) / 2], &hi = sum[(c * 16 + j) / 2 + 1];
                            const uint32_t *const from = u[c & 1] + j;
                            if constexpr (kPerColumn) {
                                // (the row's scale times the column's first, as with one scale for the columns)
                                const uint4 b = ptx::ld_shared_v4(mine + (kTileA + part * kCols + c * 16 + j) * 4);
                                add_scaled(lo, from[0], from[1], mul2(s2, pair(__uint_as_float(b.x), __uint_as_float(b.y))));
                                add_scaled(hi, from[2], from[3], mul2(s2, pair(__uint_as_float(b.z), __uint_as_float(b.w))));
                            } else {
                                add_scaled(lo, from[0], from[1], s2);
                                add_scaled(hi, from[2], from[3], s2);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive_relaxed(ptx::smem_addr(&ctl->scale_empty[sr.idx]));  // (read, and nothing written)
                sr.next(kScaleSlots);
                ok = all_lanes(ok);
            }
            if (!ok) break;
            wt.row0 = ia * kTileA + quad * 32;
            wt.rows = min(32, a.ma - wt.row0);
            // (the sums move down 32 columns at a time, so that the finishing code is there once)
#pragma unroll 1
            for (int c = part * kCols; c < (part + 1) * kCols; c += 32) {
                float v[32];
#pragma unroll
                for (int j = 0; j < 16; ++j) split(sum[j], &v[2 * j], &v[2 * j + 1]);
                if constexpr (kCols > 32) {
#pragma unroll
                    for (int j = 0; j + 16 < kCols / 2; ++j) sum[j] = sum[j + 16];
                }
                wt.b0 = ib * kTileB + c;
                wt.cols = min(32, a.nb - wt.b0);
                if (wt.rows <= 0 || wt.cols <= 0) continue;
                if (t >= a.full) {
                    float *p = a.part + ((int64_t)(t - a.full) * kTileB + c) * kTileA + quad * 32 + lane;
#pragma unroll
                    for (int j = 0; j < 32; ++j) p[j * kTileA] = v[j];
                    continue;
                }
                finish_values<kAnyAct, kSlots>(a, wt, v, lane_bias(a, wt.row0, wt.b0, lane), 0);
            }
        }
        if (lane == 0) ptx::bulk_wait_group_read<0>();
    }

    __syncwarp();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 2) tmem_dealloc<false>(tmem, 512);
}

__global__ void __launch_bounds__(256) scaled_join_kernel(const __grid_constant__ ScaledArgs a, int rows_per_tile) {
    join_runs<kAnyAct>(a, rows_per_tile);
}

}  // namespace

ScaledPlan scaled_plan(int64_t ma, int64_t nb, int64_t k) {
    ScaledPlan pl;
    // Few rows: the long dim becomes the tile's 128 lanes, so that no lanes
    // idle and every CTA streams its own weights.
    if (ma < nb && ma <= 128) {
        pl.swap = true;
        std::swap(ma, nb);
    }
    const int64_t blocks = cdiv(k, kBlockK);
    pl.tile_b = nb <= 64 ? 64 : nb <= 128 ? 128 : 256;
    while (pl.tile_b > 64 && cdiv(ma, kTileA) * cdiv(nb, pl.tile_b) * 2 <= kSms) pl.tile_b /= 2;
    pl.tiles_a = cdiv(ma, kTileA), pl.tiles_b = cdiv(nb, pl.tile_b);
    // Fewer tiles than run at once: all of them in runs.  A last round that
    // leaves half the GPU idle or more: its tiles in runs.
    const int64_t tiles = pl.tiles_a * pl.tiles_b, at_once = kSms, last = tiles % at_once;
    int64_t parts = 1;
    if (tiles * 2 <= at_once) parts = std::min(at_once / tiles, blocks / 4);
    else if (tiles > at_once && last > 0) parts = std::min<int64_t>(at_once / last, 8);
    if (parts > 1 && tiles > at_once && blocks - blocks / parts < 20) parts = 1;
    pl.full = tiles;
    if (parts > 1) {
        pl.parts = (int32_t)parts;
        pl.full = tiles <= at_once ? 0 : tiles - last;
        pl.part_bytes = (size_t)(parts * (tiles - pl.full) * kTileA * pl.tile_b * 4);
    }
    return pl;
}

conv_status scaled_launch(const ScaledProduct &given, void *workspace, void *stream) {
    ScaledProduct pr = given;
    const ScaledPlan pl = scaled_plan(pr.ma, pr.nb, pr.k);
    if (pl.tiles_a * pl.tiles_b > INT32_MAX / 16) return CONV_ERR_TOO_LARGE;
    ScaledArgs a;
    a.bias_along_a = pl.swap;
    if (pl.swap) {
        std::swap(pr.ma, pr.nb);
        std::swap(pr.a, pr.b);
        std::swap(pr.d_sa, pr.d_sb);
        std::swap(pr.res_sa, pr.res_sb);
        std::swap(pr.pre_sa, pr.pre_sb);
    }
    a.ma = (int32_t)pr.ma, a.nb = (int32_t)pr.nb;
    a.blocks = (int32_t)cdiv(pr.k, kBlockK);
    a.d = make_side(pr.d, pr.d_sa, pr.d_sb, pr.d_dtype, pr.ma, pr.nb);
    a.res = make_side(pr.res, pr.res_sa, pr.res_sb, pr.d_dtype, pr.ma, pr.nb);
    a.pre = make_side(pr.pre, pr.pre_sa, pr.pre_sb, pr.pre_dtype, pr.ma, pr.nb);
    a.bias = pr.bias, a.bias_dtype = pr.bias_dtype, a.act = pr.act, a.slots = 1;
    a.sa = {pr.a.scale, pr.a.s_rs, pr.a.s_cs, pr.a.shift, (int32_t)pr.ma};
    a.sb = {pr.b.scale, pr.b.s_rs, pr.b.s_cs, pr.b.shift, (int32_t)pr.nb};
    a.wait_limit_ns = wait_limit_ns();
    a.status = device_status_word();
    if (!a.status) return CONV_ERR_CUDA;
    a.tile_b = pl.tile_b, a.tiles_a = (int32_t)pl.tiles_a, a.tiles_b = (int32_t)pl.tiles_b;
    a.parts = pl.parts, a.full = (int32_t)pl.full, a.part = (float *)workspace;
    a.stage_bytes = 16384 + a.tile_b * kBlockK;
    a.stages = std::min(kMaxStages, kRingBytes / a.stage_bytes);
    a.idesc = (1u << 4) | ((pr.a.e5m2 ? 1u : 0u) << 7) | ((pr.b.e5m2 ? 1u : 0u) << 10) | ((uint32_t)(a.tile_b >> 3) << 17) |
              ((uint32_t)(kTileA >> 4) << 24);
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    // (without products nothing is loaded: there are no maps)
    if (a.blocks > 0 && (!encode(&a.map_a, CONV_FLOAT8_E4M3, pr.a.p, pr.k, pr.ma, pr.a.rs, kBlockK, kTileA, sw) ||
        !encode(&a.map_b, CONV_FLOAT8_E4M3, pr.b.p, pr.k, pr.nb, pr.b.rs, kBlockK, a.tile_b, sw)))
        return CONV_ERR_CUDA;
    for (auto [s, m] : {std::pair<Side *, CUtensorMap *>{&a.d, &a.map_d}, {&a.pre, &a.map_pre}})
        if (s->walk == kWalkRows &&
            !encode(m, s->dtype, s->p, pr.nb, pr.ma, s->sa, s->dtype == CONV_FLOAT32 ? 16 : 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
            return CONV_ERR_CUDA;
    typedef void (*Kernel)(ScaledArgs);
    // [tiles of 64, 128, 256 columns][a scale per row of B]
    static const Kernel kernels[3][2] = {{scaled_product_kernel<32, false>, scaled_product_kernel<32, true>},
                                         {scaled_product_kernel<64, false>, scaled_product_kernel<64, true>},
                                         {scaled_product_kernel<128, false>, scaled_product_kernel<128, true>}};
    const int which = a.tile_b == 64 ? 0 : a.tile_b == 128 ? 1 : 2, per = pr.b.shift == 0;
    const Kernel kernel = kernels[which][per];
    static std::atomic<bool> ready[64][3][2];  // (check_device admits 64 devices)
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CONV_ERR_CUDA;
    if (!ready[dev][which][per].load()) {
        // (the summing warps wait for registers that the block has to have been launched with)
        cudaFuncAttributes attr;
        if (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess ||
            attr.numRegs * kThreads < 128 * kControlRegs + 32 * kSumWarps * kSumRegs ||
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448) != cudaSuccess)
            return CONV_ERR_CUDA;
        ready[dev][which][per].store(true);
    }
    const int64_t tiles = (int64_t)a.tiles_a * a.tiles_b, units = a.full + (tiles - a.full) * a.parts;
    const size_t smem = (size_t)a.stages * a.stage_bytes + kSumWarps * kSlots * kSlotBytes + kScaleSlots * kBatch * kScaleBytes + kBiasBytes + sizeof(SharedCtl);
    if (!launch_behind(kernel, dim3((unsigned)std::min<int64_t>(units, device_sm_count())), kThreads, smem, (cudaStream_t)stream, a))
        return CONV_ERR_CUDA;
    if (a.parts > 1) {
        const int64_t blocks = (tiles - a.full) * (kTileA / 32) * (a.tile_b / 8);
        if (blocks > INT32_MAX) return CONV_ERR_TOO_LARGE;
        if (!launch_behind(scaled_join_kernel, dim3((unsigned)blocks), 32 * std::min(8, a.parts), 0, (cudaStream_t)stream, a, kTileA))
            return CONV_ERR_CUDA;
    }
    return CONV_OK;
}

}  // namespace i8c

// block_norm_grad.cuh -- the gradient of the block norm for rows in registers.
//
// Rows and parameters as in block_norm.cu.  The two sums over rows that the
// parameters want are S = sum dh * v and sum dy * u: from S follow both dgate
// (times the post gain) and dpost_gain (times the gate), so a thread carries
// two vectors and not three; the third, the gates' sum of gate * S, lies in
// shared memory and is added to where a gate ends.  A worker takes a stretch of rows and leaves S
// whenever a gate ends; stretch w leaves gate g's in slot w + g, which no other
// stretch and gate have.  A second kernel adds the slots in order.  Where there
// are more gates than workers, a worker takes whole gates and writes their
// dgate itself.  50176 x 512 bf16 with 64 gates: 70 us (4.4 TB/s; 39
// instructions per element, in half of the issue slots); 2047 x 5001 f16 with odd strides 82 us, a block of 320 threads per SM.
#pragma once

#include "block_norm.cuh"

namespace i8c {

struct BlockNormGradArgs {
    MatRef dy, dsum, x, h, gate, dx, dskip, dgate;
    const void *post_gain, *gain;
    const float *post_rstd, *rstd;
    float *part_gain;          // [blocks][part_cols]: shares of sum dy u, or NULL
    float *part_post;          // [blocks][part_cols]: of sum db v, or NULL
    float *part_gate;          // [workers + gates][part_cols]: of S, or NULL (nobody wants it, or gates are whole)
    float *scratch;            // [blocks][part_cols]: S of a gate, of the kernel for any strides
    int64_t rows, rows_per_gate, gates;
    int64_t per_worker;        // rows of a worker's stretch; 0: rows that begin anywhere, in steps
    int32_t cols, part_cols;
    float skip_scale, branch_scale;
    int32_t param_dtype;
    int32_t post;
    int32_t whole;             // workers take whole gates
    int32_t stages;
    int32_t shift_dx, shift_dskip;  // rows of another lead than those read
    uint64_t wait_limit_ns;
    int *status;
};

// Stores a thread's 8 shares of group i; a worker's shares start at its
// lead, so that whole groups are aligned.
__device__ __forceinline__ void store_share(float *part, const Place<true> &at, int i, const Pair (&v)[4]) {
    const int c = at.column(i, 0) + at.lead;
    if (c >= at.cols + at.lead) return;
    float o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) split(v[j], &o[2 * j], &o[2 * j + 1]);
    *reinterpret_cast<float4 *>(part + c) = make_float4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<float4 *>(part + c + 4) = make_float4(o[4], o[5], o[6], o[7]);
}

// Launches the kernel for x's and the stream's type (T of the one, S of the
// other), in a translation unit for each T.
bool launch_block_norm_grad_bf16(const BlockNormGradArgs &a, const Held &h, bool wide_stream, int64_t grid, size_t smem, cudaStream_t s);
bool launch_block_norm_grad_f16(const BlockNormGradArgs &a, const Held &h, bool wide_stream, int64_t grid, size_t smem, cudaStream_t s);
bool launch_block_norm_grad_f32(const BlockNormGradArgs &a, const Held &h, int64_t grid, size_t smem, cudaStream_t s);

// kWhole: a worker takes whole gates.
template <typename T, typename S, int kNv, bool kWarp, bool kWhole, bool kEven>
__global__ void __launch_bounds__(kWarp ? 256 : 512, kWarp ? 2 : 1) block_norm_grad_rows_kernel(const BlockNormGradArgs a) {
    __shared__ __align__(16) float sums[2][32];
    RowSummer block_sum{sums};
    extern __shared__ __align__(128) uint8_t smem[];
    const bool dy = a.dy.p, ds = a.dsum.p, x = a.x.p;
    const int local = kWarp ? threadIdx.x / 32 : 0, workers = kWarp ? 8 : 1;
    const int64_t worker = (int64_t)blockIdx.x * workers + local;
    Stretch rows;
    rows.first = a.per_worker ? worker * a.per_worker : worker;
    rows.end = a.per_worker ? min(a.rows, rows.first + a.per_worker) : a.rows;
    rows.step = a.per_worker ? 1 : (int64_t)gridDim.x * workers;
    T *dx = (T *)const_cast<void *>(a.dx.p) + (a.dx.p ? rows.first * a.dx.rs : 0);
    S *dskip = (S *)const_cast<void *>(a.dskip.p) + (a.dskip.p ? rows.first * a.dskip.rs : 0);
    Place<true> at;
    at.t = kWarp ? threadIdx.x % 32 : threadIdx.x;
    at.threads = kWarp ? 32 : blockDim.x;
    at.cols = a.cols;
    at.lead = kEven ? 0 : dy ? lead_of((const T *)a.dy.p + rows.first * a.dy.rs) : lead_of((const S *)a.dsum.p + rows.first * a.dsum.rs);
    const float per = 1.0f / (float)a.cols;
    // a stage: dy and h, dsum, x
    const uint32_t t_slot = row_slot_bytes(a.cols, sizeof(T)), s_slot = row_slot_bytes(a.cols, sizeof(S));
    const uint32_t of_ds = dy ? t_slot + s_slot : 0, of_x = of_ds + (ds ? s_slot : 0), stage_bytes = of_x + (x ? t_slot : 0);
    // (the gains are every worker's own where rows begin anywhere; the gate, and the sum of db v, always)
    const int own = a.per_worker ? 0 : local, first_gate = a.per_worker ? 2 : 2 * workers;
    const RowSpace space = row_space(workers, a.stages, stage_bytes, first_gate + 2 * workers, at.threads, kNv);
    const uint32_t base = ptx::smem_addr(smem), bars = base + local * 8 * kMostStages, ring = base + space.rows + local * a.stages * stage_bytes;
    const uint32_t set = kNv * 32 * at.threads, stride = at.threads * 16, kept = base + space.kept + at.t * 16;
    const Kept post_gain{kept + 2 * own * set, stride}, gain{kept + (2 * own + 1) * set, stride};
    const Kept gate{kept + (first_gate + 2 * local) * set, stride}, post_sum{kept + (first_gate + 2 * local + 1) * set, stride};
    RowFeed feed;
    feed.on = false;
    if (at.t == 0 && dy) feed.set(a.dy, a.rows, a.cols, sizeof(T), 0, rows.first, rows.step);
    if (at.t == 1 && dy) feed.set(a.h, a.rows, a.cols, sizeof(S), t_slot, rows.first, rows.step);
    if (at.t == 2 && ds) feed.set(a.dsum, a.rows, a.cols, sizeof(S), of_ds, rows.first, rows.step);
    if (at.t == 3 && x) feed.set(a.x, a.rows, a.cols, sizeof(T), of_x, rows.first, rows.step);
    if (at.t == 0) {
        for (int i = 0; i < a.stages; ++i) ptx::mbar_init(bars + 8 * i, (dy ? 2 : 0) + (ds ? 1 : 0) + (x ? 1 : 0));
        ptx::fence_mbar_init();
    }
    row_sync<kWarp>();
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    RowWait wait{a.wait_limit_ns, a.status};
    int64_t to_fill = rows.first;  // the row that is fetched next
    auto fill = [&](int stage) {
        if (feed.on && to_fill < rows.end) feed.fill<kEven>(ring + stage * stage_bytes, bars + 8 * stage);
        to_fill += rows.step;
    };
    for (int d = 0; d < a.stages; ++d) fill(d);
    if (!a.per_worker || local == 0) {
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            float g[8];
            load_params(a.post_gain, a.param_dtype, 1.0f, at, i, g);
            post_gain.keep(i, g);
            load_params(a.gain, a.param_dtype, 1.0f, at, i, g);
            gain.keep(i, g);
        }
    }
    __syncthreads();
    Pair dg[kNv][4], sv[kNv][4];
#pragma unroll
    for (int i = 0; i < kNv; ++i) {
        const float zero[8] = {};
        post_sum.keep(i, zero);
#pragma unroll
        for (int j = 0; j < 4; ++j) dg[i][j] = sv[i][j] = pair(0.0f);
    }
    int64_t which = 0, gate_end = rows.first;
    // S of gate `which` is complete as far as this worker goes: its shares of the post gain's gradient and of the gate's
    auto leave_gate = [&]() {
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            float g[8], o[8];
            load_params(gate_row(a.gate, which), a.gate.dtype, 1.0f, at, i, g);
            Pair p[4];
            post_sum.get(i, p);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                split(fma2(mul2(pair(g[2 * j], g[2 * j + 1]), pair(a.branch_scale)), sv[i][j], p[j]), &o[2 * j], &o[2 * j + 1]);
            }
            post_sum.keep(i, o);
            if constexpr (kWhole) {
                if (a.dgate.p) {
                    post_gain.get(i, p);
#pragma unroll
                    for (int j = 0; j < 4; ++j) split(mul2(mul2(sv[i][j], p[j]), pair(a.branch_scale)), &o[2 * j], &o[2 * j + 1]);
                    if (a.dgate.dtype == CONV_FLOAT32) store_group<true, float, kEven>((float *)const_cast<void *>(a.dgate.p) + which * a.dgate.rs, at, i, o);
                    else store_group<true, T, kEven>((T *)const_cast<void *>(a.dgate.p) + which * a.dgate.rs, at, i, o);
                }
            } else if (a.part_gate) {
                store_share(a.part_gate + (worker + which) * a.part_cols, at, i, sv[i]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) sv[i][j] = pair(0.0f);
        }
    };
    int stage = 0;
    uint32_t phase = 0;
    float next_rs = dy && rows.first < rows.end ? a.rstd[rows.first] : 0.0f;
    float next_rx = a.post && rows.first < rows.end ? a.post_rstd[rows.first] : 1.0f;
    for (int64_t r = rows.first; r < rows.end; r += rows.step) {
        if (r >= gate_end) {
            if (r > rows.first) leave_gate();
            which = r / a.rows_per_gate;
            gate_end = (which + 1) * a.rows_per_gate;
#pragma unroll
            for (int i = 0; i < kNv; ++i) keep_gate(gate, a.gate, which, post_gain, a.post, a.branch_scale, at, i);
        }
        const float rs = next_rs, rx = next_rx;
        if (r + rows.step < rows.end) {
            if (dy) next_rs = a.rstd[r + rows.step];
            if (a.post) next_rx = a.post_rstd[r + rows.step];
        }
        const uint32_t slot = ring + stage * stage_bytes;
        wait(bars + 8 * stage, phase);
        Pair dh[kNv][4];
        Pair s2 = pair(0.0f);
        float minus = 0.0f;
        // (a matrix that is not there reads as 0, a norm that is not as 1: no branch costs less)
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            Group<T> gy;
            Group<S> gh;
            slot_group<kEven>(slot, at, i, gy, dy);
            slot_group<kEven>(slot + t_slot, at, i, gh, dy);
            Pair g[4];
            gain.get(i, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const Pair d = element2(gy, j), w = mul2(element2(gh, j), pair(rs));
                dh[i][j] = mul2(d, g[j]);
                s2 = fma2(dh[i][j], w, s2);
                dg[i][j] = fma2(d, w, dg[i][j]);
            }
        }
        if (dy) {
            const float s = sum_of(s2);
            minus = -(kWarp ? warp_sum(s) : block_sum(s)) * per * rs * rs;
        }
        // (what was read before the sum is read again, not kept: registers are short)
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            Group<S> gh, gs;
            slot_group<kEven>(slot + t_slot, at, i, gh, dy);
            slot_group<kEven>(slot + of_ds, at, i, gs, ds);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                dh[i][j] = fma2(element2(gh, j), pair(minus), fma2(dh[i][j], pair(rs), element2(gs, j)));
        }
        if (a.dskip.p) {
            const Pair skip_scale = pair(a.skip_scale);
#pragma unroll
            for (int i = 0; i < kNv; ++i) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) split(mul2(skip_scale, dh[i][j]), &o[2 * j], &o[2 * j + 1]);
                if (!kEven && a.shift_dskip) store_shifted(dskip, at, i, o);
                else store_group<true, S, kEven>(dskip, at, i, o);
            }
        }
        // S, and dn (in dh's place) with its sum
        s2 = pair(0.0f);
        Group<T> gx[kNv];
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            slot_group<kEven>(slot + of_x, at, i, gx[i], x);
            Pair g[4];
            gate.get(i, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const Pair v = mul2(element2(gx[i], j), pair(rx));
                sv[i][j] = fma2(dh[i][j], v, sv[i][j]);
                dh[i][j] = mul2(dh[i][j], g[j]);
                s2 = fma2(dh[i][j], v, s2);
            }
        }
        const bool second = a.dx.p && a.post;
        if (second) {
            const float s = sum_of(s2);
            minus = -(kWarp ? warp_sum(s) : block_sum(s)) * per * rx * rx;
        }
        // everything of the slots has been read: they take the row `stages` steps on
        if (kWarp || !second) row_sync<kWarp>();
        fill(stage);
        if (++stage == a.stages) stage = 0, phase ^= 1;
        if (a.dx.p) {
            // (two loops: without a post norm dx is db whatever x is, an infinity among it too)
            auto put = [&](int i, const float (&o)[8]) {
                if (!kEven && a.shift_dx) store_shifted(dx, at, i, o);
                else store_group<true, T, kEven>(dx, at, i, o);
            };
            float o[8];
            if (second) {
#pragma unroll
                for (int i = 0; i < kNv; ++i) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        split(fma2(element2(gx[i], j), pair(minus), mul2(dh[i][j], pair(rx))), &o[2 * j], &o[2 * j + 1]);
                    put(i, o);
                }
            } else {
#pragma unroll
                for (int i = 0; i < kNv; ++i) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) split(dh[i][j], &o[2 * j], &o[2 * j + 1]);
                    put(i, o);
                }
            }
        }
        if (a.dskip.p) dskip += rows.step * a.dskip.rs;
        if (a.dx.p) dx += rows.step * a.dx.rs;
    }
    wait.settle(feed.on);
    // (workers beyond the rows leave no gate, and nothing of theirs is added)
    if (rows.first < rows.end) leave_gate();
    if constexpr (!kWarp) {
        if (rows.first >= rows.end) return;
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            if (a.part_gain) store_share(a.part_gain + worker * a.part_cols, at, i, dg[i]);
            if (a.part_post) {
                Pair p[4];
                post_sum.get(i, p);
                store_share(a.part_post + worker * a.part_cols, at, i, p);
            }
        }
    } else {
        // the warps' shares added in the block: [warp][dgain, dpost_gain][column] over all of shared memory
        Pair ps[kNv][4];
#pragma unroll
        for (int i = 0; i < kNv; ++i) post_sum.get(i, ps[i]);
        __syncthreads();
        float *const shares = reinterpret_cast<float *>(smem);
        float *const mine = shares + local * 2 * a.cols;
#pragma unroll
        for (int i = 0; i < kNv; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = at.column(i, j);
                float lo, hi;
                if (at.inside(c)) {
                    split(dg[i][j / 2], &lo, &hi);
                    mine[c] = j % 2 ? hi : lo;
                    split(ps[i][j / 2], &lo, &hi);
                    mine[a.cols + c] = j % 2 ? hi : lo;
                }
            }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * a.cols; c += 256) {
            float s = shares[c];
#pragma unroll
            for (int w = 1; w < 8; ++w) s += shares[w * 2 * a.cols + c];
            float *const to = c < a.cols ? a.part_gain : a.part_post;
            if (to) to[(int64_t)blockIdx.x * a.part_cols + (c < a.cols ? c : c - a.cols)] = s;
        }
    }
}

template <typename T, typename S, int kNv, bool kWarp>
bool launch_grad_rows(const BlockNormGradArgs &a, const Held &h, int64_t grid, size_t smem, cudaStream_t s) {
    const dim3 g((unsigned)grid);
    if (!h.even) return launch_large<block_norm_grad_rows_kernel<T, S, kNv, kWarp, false, false>>(g, h.threads, smem, s, a);
    return a.whole ? launch_large<block_norm_grad_rows_kernel<T, S, kNv, kWarp, true, true>>(g, h.threads, smem, s, a)
                   : launch_large<block_norm_grad_rows_kernel<T, S, kNv, kWarp, false, true>>(g, h.threads, smem, s, a);
}
template <typename T, typename S>
bool launch_backward(const BlockNormGradArgs &a, const Held &h, int64_t grid, size_t smem, cudaStream_t s) {
    if (h.warp) {
        if (h.nv == 1) return launch_grad_rows<T, S, 1, true>(a, h, grid, smem, s);
        const dim3 g((unsigned)grid);  // (even rows)
        return a.whole ? launch_large<block_norm_grad_rows_kernel<T, S, 2, true, true, true>>(g, h.threads, smem, s, a)
                       : launch_large<block_norm_grad_rows_kernel<T, S, 2, true, false, true>>(g, h.threads, smem, s, a);
    }
    return h.nv == 1 ? launch_grad_rows<T, S, 1, false>(a, h, grid, smem, s) : launch_grad_rows<T, S, 2, false>(a, h, grid, smem, s);
}

}  // namespace i8c

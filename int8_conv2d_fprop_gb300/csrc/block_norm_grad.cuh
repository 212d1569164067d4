// block_norm_grad.cuh -- the gradient of the block norm for rows in registers.
//
// Rows and parameters as in block_norm.cu.  The two sums over rows that the
// parameters want are S = sum dh * v and sum dy * u: from S follow both dgate
// (times the post gain) and dpost_gain (times the gate), so a thread carries
// two vectors and not three.  A worker takes a stretch of rows and leaves S
// whenever a gate ends; stretch w leaves gate g's in slot w + g, which no other
// stretch and gate have.  A second kernel adds the slots in order.  Where there
// are more gates than workers, a worker takes whole gates and writes their
// dgate itself.
#pragma once

#include "block_norm.cuh"

namespace i8c {

struct BlockNormGradArgs {
    MatRef dy, dsum, x, h, gate, dx, dskip, dgate;
    const void *post_gain, *gain;
    const float *post_rstd, *rstd;
    float *part_gain;          // [workers][part_cols]: shares of sum dy u, or NULL
    float *part_gate;          // [workers + gates][part_cols]: of S; whole gates: [workers], of sum db v; or NULL
    float *scratch;            // [blocks][part_cols]: S of a gate, of the kernel for any strides
    int64_t rows, rows_per_gate, gates;
    int64_t per_worker;        // rows of a worker's stretch; 0: rows that begin anywhere, in steps
    int32_t cols, part_cols;
    float skip_scale, branch_scale;
    int32_t param_dtype;
    int32_t post;
    int32_t whole;             // workers take whole gates
    int32_t turn_dx, turn_dskip;
    uint64_t wait_limit_ns;
    int *status;
};

// Adds or stores a thread's 8 shares of group i; a worker's shares start at
// its lead, so that whole groups are aligned.
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
    __shared__ __align__(16) BlockSums sums;
    Summer block_sum{&sums};
    extern __shared__ __align__(128) uint8_t smem[];
    const T *dy = (const T *)a.dy.p, *x = (const T *)a.x.p;
    const S *ds = (const S *)a.dsum.p;
    T *dx = (T *)const_cast<void *>(a.dx.p);
    S *dskip = (S *)const_cast<void *>(a.dskip.p);
    const int local = kWarp ? threadIdx.x / 32 : 0, workers = kWarp ? 8 : 1;
    const int64_t worker = (int64_t)blockIdx.x * workers + local;
    Stretch rows;
    rows.first = a.per_worker ? worker * a.per_worker : worker;
    rows.end = a.per_worker ? min(a.rows, rows.first + a.per_worker) : a.rows;
    rows.step = a.per_worker ? 1 : (int64_t)gridDim.x * workers;
    Place<true> at;
    at.t = kWarp ? threadIdx.x % 32 : threadIdx.x;
    at.threads = kWarp ? 32 : blockDim.x;
    at.cols = a.cols;
    at.lead = kEven ? 0 : dy ? lead_of(dy + rows.first * a.dy.rs) : lead_of(ds + rows.first * a.dsum.rs);
    const float per = 1.0f / (float)a.cols;
    // a stage: dy and h, dsum, x
    const uint32_t t_slot = row_slot_bytes(a.cols, sizeof(T)), s_slot = row_slot_bytes(a.cols, sizeof(S));
    const uint32_t of_ds = dy ? t_slot + s_slot : 0, of_x = of_ds + (ds ? s_slot : 0), stage_bytes = of_x + (x ? t_slot : 0);
    const int own = a.per_worker ? 0 : local;
    const RowSpace space = row_space(workers, stage_bytes, (a.per_worker ? 2 : 2 * workers) + workers, at.threads, kNv,
                                     (a.turn_dskip ? turn_elems(a.cols) * sizeof(S) : 0) + (a.turn_dx ? turn_elems(a.cols) * sizeof(T) : 0));
    const uint32_t base = ptx::smem_addr(smem), bars = base + local * 8 * kStages, ring = base + space.rows + local * kStages * stage_bytes;
    const uint32_t set = kNv * 32 * at.threads, stride = at.threads * 16;
    const Kept post_gain{base + space.kept + (2 * own) * set + at.t * 16, stride}, gain{post_gain.base + set, stride};
    const Kept gate{base + space.kept + ((a.per_worker ? 2 : 2 * workers) + local) * set + at.t * 16, stride};
    uint8_t *turned = smem + space.turned + local * (space.total - space.turned) / workers;
    Turn<S> turn_dskip{(S *)turned, 0};  // (the lead a row at a time: the output's may change where the rows read have one)
    if (a.turn_dskip) turned += turn_elems(a.cols) * sizeof(S);
    Turn<T> turn_dx{(T *)turned, 0};

    RowFeed feed;
    feed.on = false;
    if (at.t == 0 && dy) feed.set(a.dy, a.rows, a.cols, sizeof(T), 0);
    if (at.t == 1 && dy) feed.set(a.h, a.rows, a.cols, sizeof(S), t_slot);
    if (at.t == 2 && ds) feed.set(a.dsum, a.rows, a.cols, sizeof(S), of_ds);
    if (at.t == 3 && x) feed.set(a.x, a.rows, a.cols, sizeof(T), of_x);
    if (at.t == 0) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) ptx::mbar_init(bars + 8 * i, (dy ? 2 : 0) + (ds ? 1 : 0) + (x ? 1 : 0));
        ptx::fence_mbar_init();
    }
    row_sync<kWarp>();
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    RowWait wait{a.wait_limit_ns, a.status};
    auto fill = [&](int64_t r, int stage) {
        if (at.t < 4 && r < rows.end) feed.fill(r, ring + stage * stage_bytes, bars + 8 * stage);
    };
#pragma unroll
    for (int d = 0; d < kStages; ++d) fill(rows.first + d * rows.step, d);
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
    Pair dg[kNv][4], sv[kNv][4], dp[kWhole ? kNv : 1][4];
#pragma unroll
    for (int i = 0; i < kNv; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            dg[i][j] = sv[i][j] = pair(0.0f);
            if constexpr (kWhole) dp[i][j] = pair(0.0f);
        }
    const Pair skip_scale = pair(a.skip_scale), branch_scale = pair(a.branch_scale);
    int64_t which = 0, gate_end = rows.first;
    // S of gate `which` is complete as far as this worker goes
    auto leave_gate = [&]() {
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            if constexpr (kWhole) {
                // its gradient, and its share of the post gain's
                Pair g[4], p[4];
                gate.get(i, g);
                post_gain.get(i, p);
                float o[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    dp[i][j] = fma2(g[j], sv[i][j], dp[i][j]);
                    split(mul2(mul2(sv[i][j], p[j]), branch_scale), &o[2 * j], &o[2 * j + 1]);
                }
                if (a.dgate.p) {
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
            for (int i = 0; i < kNv; ++i) {
                float g[8];
                load_params(gate_row(a.gate, which), a.gate.dtype, 1.0f, at, i, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] *= a.branch_scale;
                gate.keep(i, g);
            }
        }
        const float rs = next_rs, rx = next_rx;
        if (r + rows.step < rows.end) {
            if (dy) next_rs = a.rstd[r + rows.step];
            if (a.post) next_rx = a.post_rstd[r + rows.step];
        }
        if (!kEven && a.turn_dskip) turn_dskip.lead = lead_of(dskip + r * a.dskip.rs);
        if (!kEven && a.turn_dx) turn_dx.lead = lead_of(dx + r * a.dx.rs);
        const uint32_t slot = ring + stage * stage_bytes;
        wait(bars + 8 * stage, phase);
        Pair dh[kNv][4];
        Group<T> gx[kNv];
        Group<S> gs[kNv], gh[kNv];
        Pair s2 = pair(0.0f);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            if (ds) slot_group<kEven>(slot + of_ds, at, i, gs[i]);
            if (x) slot_group<kEven>(slot + of_x, at, i, gx[i]);
            if (dy) {
                Group<T> gy;
                slot_group<kEven>(slot, at, i, gy);
                slot_group<kEven>(slot + t_slot, at, i, gh[i]);
                Pair g[4];
                gain.get(i, g);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Pair d = element2(gy, j), w = mul2(element2(gh[i], j), pair(rs));
                    dh[i][j] = mul2(d, g[j]);
                    s2 = fma2(dh[i][j], w, s2);
                    dg[i][j] = fma2(d, w, dg[i][j]);
                }
            }
        }
        float minus = 0.0f;
        if (dy) {
            const float s = sum_of(s2);
            minus = -(kWarp ? warp_sum(s) : block_sum(s)) * per * rs * rs;
        }
        // the slots just read take the row kStages steps on
        if (kWarp || !dy) row_sync<kWarp>();
        fill(r + kStages * rows.step, stage);
        if (++stage == kStages) stage = 0, phase ^= 1;
#pragma unroll
        for (int i = 0; i < kNv; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (dy) {
                    dh[i][j] = fma2(element2(gh[i], j), pair(minus), mul2(dh[i][j], pair(rs)));
                    if (ds) dh[i][j] = add2(dh[i][j], element2(gs[i], j));
                } else {
                    dh[i][j] = element2(gs[i], j);
                }
            }
        if (dskip) {
#pragma unroll
            for (int i = 0; i < kNv; ++i) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) split(mul2(skip_scale, dh[i][j]), &o[2 * j], &o[2 * j + 1]);
                if (!kEven && a.turn_dskip) turn_group(turn_dskip, at, i, o);
                else store_group<true, S, kEven>(dskip + r * a.dskip.rs, at, i, o);
            }
        }
        // S, and dn (in dh's place) with its sum
        s2 = pair(0.0f);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            Pair g[4], p[4];
            gate.get(i, g);
            if (a.post) post_gain.get(i, p);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (x) {
                    const Pair v = a.post ? mul2(element2(gx[i], j), pair(rx)) : element2(gx[i], j);
                    sv[i][j] = fma2(dh[i][j], v, sv[i][j]);
                    dh[i][j] = mul2(dh[i][j], g[j]);
                    if (a.post) {
                        dh[i][j] = mul2(dh[i][j], p[j]);
                        s2 = fma2(dh[i][j], v, s2);
                    }
                } else {
                    dh[i][j] = mul2(dh[i][j], g[j]);
                }
            }
        }
        if (dx) {
            if (a.post) {
                const float s = sum_of(s2);
                minus = -(kWarp ? warp_sum(s) : block_sum(s)) * per * rx * rx;
            }
#pragma unroll
            for (int i = 0; i < kNv; ++i) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    Pair w = dh[i][j];
                    if (a.post) w = fma2(element2(gx[i], j), pair(minus), mul2(w, pair(rx)));
                    split(w, &o[2 * j], &o[2 * j + 1]);
                }
                if (!kEven && a.turn_dx) turn_group(turn_dx, at, i, o);
                else store_group<true, T, kEven>(dx + r * a.dx.rs, at, i, o);
            }
        }
        if (!kEven && (a.turn_dskip || a.turn_dx)) {
            row_sync<kWarp>();
            if (a.turn_dskip) store_turned(dskip + r * a.dskip.rs, turn_dskip, at);
            if (a.turn_dx) store_turned(dx + r * a.dx.rs, turn_dx, at);
            row_sync<kWarp>();
        }
    }
    // (workers beyond the rows leave nothing, and nothing of theirs is added)
    if (rows.first >= rows.end) return;
    leave_gate();
#pragma unroll
    for (int i = 0; i < kNv; ++i) {
        if (a.part_gain) store_share(a.part_gain + worker * a.part_cols, at, i, dg[i]);
        if constexpr (kWhole) {
            if (a.part_gate) store_share(a.part_gate + worker * a.part_cols, at, i, dp[i]);
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
    if (h.warp) return launch_grad_rows<T, S, 1, true>(a, h, grid, smem, s);
    return h.nv == 1 ? launch_grad_rows<T, S, 1, false>(a, h, grid, smem, s) : launch_grad_rows<T, S, 2, false>(a, h, grid, smem, s);
}

}  // namespace i8c

// rmsnorm.cu -- RMS norm over the channels of each row (pixel or token), with
// the residual's addition before it, and its backward pass.
//
//   t = x + r;  rho = 1 / sqrt(mean_c t^2 + eps);  y = gamma * t * rho
//   E4M3 y: s = max_c |y| / 448, stored value rn(y / s)
//
//   d = dy * gamma;  dx = rho * d - t * rho^3 * mean_c(d t) + dt
//   dgamma = sum_rows dy * t * rho
//
// A row is read once into registers (16-byte loads of each operand), its sums
// run in FP32 over a group of threads, and the outputs are written from the
// registers: the traffic is each input once and each output once, which is
// what bounds these kernels.  max |y| = rho * max |gamma t|, so the 8-bit
// scale comes from the same reduction as the sum of squares.  Measured back to
// back, BF16: forward with both outputs 100352 x 512 67.9 us (6.05 TB/s), backward
// 25088 x 1024 35.6 us (5.8 TB/s); one row 3 us, the cost of a launch.  Slower: FP32
// rows (100352 x 512 248 us, 3.3 TB/s), an FP32 stream beside BF16 branches (a row ahead in registers: 124 us, 5.0 TB/s; backward 209
// us, 3.5 TB/s), channels apart (two passes: 368 us, 1.1 TB/s; backward 610 us, 0.7 TB/s).
#include "norm_rows.cuh"

namespace {

using namespace dlc;

// Blocks of 256 threads an SM is to hold (what the registers are limited for).
constexpr int RMS_FWD_BLOCKS = 4, RMS_BWD_BLOCKS = 2;

// Rows in registers: `tpr` threads a row (8 to 1024: short rows take few, so that a
// block's loads cover several rows), V vectors of W channels a thread.
// The next row's loads are issued before this row's reduction waits.
template <int W, int V, int KIND, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > NORM_THREADS ? 1 : RMS_FWD_BLOCKS)
    rms_rows_kernel(const __grid_constant__ RmsProblem p, int tpr, int gamma_vec) {
    griddep_launch_dependents();
    __shared__ float2 buf[2][NORM_MAX_WARPS];
    const int rpb = (int)blockDim.x / tpr, slot = (int)threadIdx.x / tpr, t = (int)threadIdx.x % tpr;
    const long long step = (long long)gridDim.x * rpb;
    extern __shared__ uint4 ring_s[];
    constexpr int E = V * W;
    const Cols<W, V> cols(t, tpr, p.C);
    const float inv_c = 1.f / (float)p.C;
    const bool e4m3 = p.y.dt == DLC_DATA_FLOAT8_E4M3;
    griddep_wait();
    float g[E];
#pragma unroll
    for (int j = 0; j < V; ++j) load_gamma<W>(p.gamma, (t + j * tpr) * W, p.C, gamma_vec != 0, g + j * W);
    Rows<W, V, KIND, 2, ring_rows<KIND, MAXT>()> rows;
    rows.start(smem_u32(ring_s), t, tpr, slot, p.C);
    long long row = (long long)blockIdx.x * rpb + slot, ahead = row;
    const int c = cols.c[0];
    RowWalk wx(p.x, row, step, c), wr(p.r, row, step, c), wt(p.t, row, step, c), wy(p.y, row, step, c);
    auto fetch = [&]() {
        if (ahead < p.rows) {
            rows.fetch(p.x, 0, wx.at(p.x, ahead, c), cols);
            if (p.r.p) rows.fetch(p.r, 1, wr.at(p.r, ahead, c), cols);
        }
        rows.commit();
        ahead += step;
        wx.next();
        wr.next();
    };
    for (int i = 0; i < rows.AHEAD; ++i) fetch();
    // every thread of the block makes the same number of rounds
    for (int parity = 0; row - slot < p.rows; row += step, parity ^= 1, wt.next(), wy.next()) {
        const bool on = row < p.rows;
        float f[2][E];
        const uint32_t starts[2] = {(uint32_t)(row * p.x.m.ld * 2), (uint32_t)(row * p.r.m.ld * 2)};
        rows.take(f, cols, starts);
        float *v = f[0];
        if (p.r.p) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) set2(v, i, add2(get2(v, i), get2(f[1], i)));
        }
        if (p.t.p && on) store_row<W, V>(p.t.dt, wt.at(p.t, row, c), cols, f[0]);
        fetch();
        float2 sq = make_float2(0.f, 0.f);
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            sq = fma2(get2(v, i), get2(v, i), sq);
            set2(v, i, mul2(get2(v, i), get2(g, i)));
        }
        if (e4m3) {
#pragma unroll
            for (int i = 0; i < E; ++i) mx = fmaxf(mx, fabsf(v[i]));
        }
        const float2 red = row_reduce<true>(sq.x + sq.y, mx, tpr, slot, buf, parity);
        if (!on) continue;
        float rho = rsqrtf(red.x * inv_c + p.eps);
        if (e4m3) {
            const E4m3Row q(red.x, red.y, rho);
            if (t == 0) p.scale[row] = q.scale;
            if (q.first != 1.f) {
#pragma unroll
                for (int i = 0; i < E / 2; ++i) set2(v, i, mul2(get2(v, i), make_float2(q.first, q.first)));
            }
            rho = q.then;
        }
#pragma unroll
        for (int i = 0; i < E / 2; ++i) set2(v, i, mul2(get2(v, i), make_float2(rho, rho)));
        store_row<W, V>(p.y.dt, wy.at(p.y, row, c), cols, f[0]);
    }
}

// The remaining layouts, two passes over a row (see AnyMap).
template <bool LANES>
__global__ void __launch_bounds__(NORM_THREADS) rms_any_kernel(const __grid_constant__ RmsProblem p) {
    using M = AnyMap<LANES>;
    griddep_launch_dependents();
    __shared__ float2 part[NORM_THREADS / 32][32];
    griddep_wait();
    for (long long row0 = (long long)blockIdx.x * M::ROWS; row0 < p.rows; row0 += (long long)gridDim.x * M::ROWS) {
        const long long row = row0 + M::row();
        const bool on = row < p.rows;
        const long long xo = on ? row_off(p.x.m, row) : 0, ro = on && p.r.p ? row_off(p.r.m, row) : 0;
        float sq = 0.f, mx = 0.f;
        float v[AHEAD], r[AHEAD];
        for (int c = M::first(); on && c < p.C; c += AHEAD * M::STEP) {
            const auto in = [&](int i) { return c + i * M::STEP < p.C; };
            load_elems<AHEAD>(p.x.p, p.x.dt, xo + c * p.x.m.cs, M::STEP * p.x.m.cs, in, v);
            if (p.r.p) {
                load_elems<AHEAD>(p.r.p, p.r.dt, ro + c * p.r.m.cs, M::STEP * p.r.m.cs, in, r);
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) v[i] += r[i];
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                sq = fmaf(v[i], v[i], sq);
                mx = fmaxf(mx, fabsf(v[i] * (in(i) ? p.gamma[c + i * M::STEP] : 0.f)));
            }
        }
        const float2 red = M::template join<true>(sq, mx, part);
        if (!on) continue;
        float f = rsqrtf(red.x / (float)p.C + p.eps), first = 1.f;
        if (p.y.dt == DLC_DATA_FLOAT8_E4M3) {
            const E4m3Row q(red.x, red.y, f);
            if (M::first() == 0) p.scale[row] = q.scale;
            first = q.first, f = q.then;
        }
        const long long to = p.t.p ? row_off(p.t.m, row) : 0, yo = row_off(p.y.m, row);
        for (int c = M::first(); c < p.C; c += AHEAD * M::STEP) {
            const auto in = [&](int i) { return c + i * M::STEP < p.C; };
            load_elems<AHEAD>(p.x.p, p.x.dt, xo + c * p.x.m.cs, M::STEP * p.x.m.cs, in, v);
            if (p.r.p) {
                load_elems<AHEAD>(p.r.p, p.r.dt, ro + c * p.r.m.cs, M::STEP * p.r.m.cs, in, r);
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) v[i] += r[i];
            }
            float g[AHEAD];
            load_elems<AHEAD>(p.gamma, DLC_DATA_FLOAT, c, M::STEP, in, g);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int ci = c + i * M::STEP;
                if (ci >= p.C) break;
                if (p.t.p) store_elem(p.t.p, p.t.dt, to + ci * p.t.m.cs, v[i]);
                store_elem(p.y.p, p.y.dt, yo + ci * p.y.m.cs, v[i] * g[i] * first * f);
            }
        }
    }
}

// Backward, rows in registers.  Each thread adds up dgamma of its own channels
// over the rows it visits; a block writes one partial row of sums.
template <int W, int V, int KIND, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > NORM_THREADS ? 1 : RMS_BWD_BLOCKS)
    rms_bwd_rows_kernel(const __grid_constant__ RmsBwdProblem p, int tpr, int gamma_vec) {
    griddep_launch_dependents();
    __shared__ float2 buf[2][NORM_MAX_WARPS];
    extern __shared__ uint4 ring_s[];
    constexpr int E = V * W;
    const int rpb = (int)blockDim.x / tpr, slot = (int)threadIdx.x / tpr, t = (int)threadIdx.x % tpr;
    const long long step = (long long)gridDim.x * rpb;
    const Cols<W, V> cols(t, tpr, p.C);
    const float inv_c = 1.f / (float)p.C;
    griddep_wait();
    float g[E], acc[E];
#pragma unroll
    for (int j = 0; j < V; ++j) load_gamma<W>(p.gamma, (t + j * tpr) * W, p.C, gamma_vec != 0, g + j * W);
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.f;
    Rows<W, V, KIND, 3, ring_rows<KIND, MAXT>()> rows;
    rows.start(smem_u32(ring_s), t, tpr, slot, p.C);
    long long row = (long long)blockIdx.x * rpb + slot, ahead = row;
    const int c = cols.c[0];
    RowWalk wy(p.dy, row, step, c), wt(p.t, row, step, c), ws(p.dt, row, step, c), wx(p.dx, row, step, c);
    auto fetch = [&]() {
        if (ahead < p.rows) {
            rows.fetch(p.dy, 0, wy.at(p.dy, ahead, c), cols);
            rows.fetch(p.t, 1, wt.at(p.t, ahead, c), cols);
            if (p.dt.p) rows.fetch(p.dt, 2, ws.at(p.dt, ahead, c), cols);
        }
        rows.commit();
        ahead += step;
        wy.next();
        wt.next();
        ws.next();
    };
    for (int i = 0; i < rows.AHEAD; ++i) fetch();
    for (int parity = 0; row - slot < p.rows; row += step, parity ^= 1, wx.next()) {
        const bool on = row < p.rows;
        float f[3][E];
        const uint32_t starts[3] = {(uint32_t)(row * p.dy.m.ld * 2), (uint32_t)(row * p.t.m.ld * 2), (uint32_t)(row * p.dt.m.ld * 2)};
        rows.take(f, cols, starts);
        float2 sq = make_float2(0.f, 0.f), dot = sq;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const float2 v = get2(f[1], i);
            sq = fma2(v, v, sq);
            dot = fma2(mul2(get2(f[0], i), get2(g, i)), v, dot);
        }
        fetch();
        const float2 red = row_reduce<false>(sq.x + sq.y, dot.x + dot.y, tpr, slot, buf, parity);
        if (!on) continue;
        const float rho = rsqrtf(red.x * inv_c + p.eps);
        const float k = -row_slope(rho, red.y * inv_c);
        const float2 rho2 = make_float2(rho, rho), k2 = make_float2(k, k);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const float2 d = mul2(get2(f[0], i), rho2), v = get2(f[1], i);
            set2(acc, i, fma2(d, v, get2(acc, i)));
            const float2 s = p.dt.p ? get2(f[2], i) : make_float2(0.f, 0.f);
            set2(f[2], i, fma2(d, get2(g, i), fma2(v, k2, s)));
        }
        store_row<W, V>(p.dx.dt, wx.at(p.dx, row, c), cols, f[2]);
    }
    if (!p.dgamma) return;
    if (rpb > 1) {  // join the block's row slots, in the ring's place: [slot][C]
        float *acc_s = reinterpret_cast<float *>(ring_s);
        cp_async_wait<0>();
        __syncthreads();
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i % W < cols.n[i / W]) acc_s[(long long)slot * p.C + cols.c[i / W] + i % W] = acc[i];
        __syncthreads();
        for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
            float s = 0.f;
            for (int i = 0; i < rpb; ++i) s += acc_s[(long long)i * p.C + c];
            p.ws[(long long)blockIdx.x * p.C + c] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i % W < cols.n[i / W]) p.ws[(long long)blockIdx.x * p.C + cols.c[i / W] + i % W] = acc[i];
    }
}

// Backward for the remaining layouts.  A block's dgamma collects in its row of
// partial sums, a channel always through the same thread (LANES: its warp's
// rows joined by shuffles).
template <bool LANES>
__global__ void __launch_bounds__(NORM_THREADS) rms_bwd_any_kernel(const __grid_constant__ RmsBwdProblem p) {
    using M = AnyMap<LANES>;
    griddep_launch_dependents();
    __shared__ float2 part[NORM_THREADS / 32][32];
    griddep_wait();
    bool first = true;
    for (long long row0 = (long long)blockIdx.x * M::ROWS; row0 < p.rows; row0 += (long long)gridDim.x * M::ROWS) {
        const long long row = row0 + M::row();
        const bool on = row < p.rows;
        const long long yo = on ? row_off(p.dy.m, row) : 0, to = on ? row_off(p.t.m, row) : 0;
        float sq = 0.f, dot = 0.f;
        float v[AHEAD], d[AHEAD], a[AHEAD];
        for (int c = M::first(); on && c < p.C; c += AHEAD * M::STEP) {
            const auto in = [&](int i) { return c + i * M::STEP < p.C; };
            load_elems<AHEAD>(p.t.p, p.t.dt, to + c * p.t.m.cs, M::STEP * p.t.m.cs, in, v);
            load_elems<AHEAD>(p.dy.p, p.dy.dt, yo + c * p.dy.m.cs, M::STEP * p.dy.m.cs, in, d);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                sq = fmaf(v[i], v[i], sq);
                dot = fmaf(d[i] * (in(i) ? p.gamma[c + i * M::STEP] : 0.f), v[i], dot);
            }
        }
        const float2 red = M::template join<false>(sq, dot, part);
        const float rho = on ? rsqrtf(red.x / (float)p.C + p.eps) : 0.f;
        const float k = row_slope(rho, red.y / (float)p.C);
        const long long xo = on ? row_off(p.dx.m, row) : 0, so = on && p.dt.p ? row_off(p.dt.m, row) : 0;
        for (int c = M::first(); c < p.C; c += AHEAD * M::STEP) {
            const auto in = [&](int i) { return on && c + i * M::STEP < p.C; };
            load_elems<AHEAD>(p.t.p, p.t.dt, to + c * p.t.m.cs, M::STEP * p.t.m.cs, in, v);
            load_elems<AHEAD>(p.dy.p, p.dy.dt, yo + c * p.dy.m.cs, M::STEP * p.dy.m.cs, in, d);
            float gain[AHEAD];
            load_elems<AHEAD>(p.gamma, DLC_DATA_FLOAT, c, M::STEP, in, gain);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) a[i] = 0.f;
            if (p.dt.p) load_elems<AHEAD>(p.dt.p, p.dt.dt, so + c * p.dt.m.cs, M::STEP * p.dt.m.cs, in, a);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int ci = c + i * M::STEP;
                if (ci >= p.C) break;
                if (on) store_elem(p.dx.p, p.dx.dt, xo + ci * p.dx.m.cs, a[i] + rho * d[i] * gain[i] - v[i] * k);
                if (!p.dgamma) continue;
                float g = d[i] * rho * v[i];
                if (LANES)
                    for (int o = 16; o > 0; o /= 2) g += __shfl_xor_sync(0xffffffffu, g, o);
                if (!LANES || M::row() == 0) {
                    float *w = p.ws + (long long)blockIdx.x * p.C + ci;
                    *w = first ? g : *w + g;
                }
            }
        }
        first = false;
    }
}

// out[c] = the sum of the blocks' partial rows, in a fixed order: 32 columns a
// block, the partial rows dealt to its 32 warps.  At most a few hundred rows from the
// L2: latency, and the launch, which starts while the grid before it ends (304
// partial rows of 1024 columns add 2.7 us to a backward call).
// Columns from `half` on are those of out2 (either output may be absent).
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *ws, float *out, float *out2, long long half, long long C, int blocks) {
    griddep_launch_dependents();
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + lane;
    griddep_wait();
    float s = 0.f;
    if (c < C) {
#pragma unroll 8
        for (int b = warp; b < blocks; b += 32) s += ws[b * C + c];
    }
    part[warp][lane] = s;
    __syncthreads();
    s = part[lane][warp];  // column `warp`
    for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    const long long k = (long long)blockIdx.x * 32 + warp;
    if (lane == 0 && k < C) {
        if (k < half) {
            if (out) out[k] = s;
        } else if (out2) {
            out2[k - half] = s;
        }
    }
}

// ---- host side ---------------------------------------------------------------

RowPlan plan_fwd(const dlcContext *ctx, const RmsProblem &p) {
    return plan_rows(p.rows, p.C, contiguous(p.x) && contiguous(p.r) && contiguous(p.t) && contiguous(p.y),
                     vec_ok(p.x) && vec_ok(p.r) && vec_ok(p.t) && vec_ok(p.y), ring({p.x, p.r}), RMS_FWD_BLOCKS, ctx->sm_count);
}

RowPlan plan_bwd(const dlcContext *ctx, const RmsBwdProblem &p) {
    return plan_rows(p.rows, p.C, contiguous(p.dy) && contiguous(p.t) && contiguous(p.dt) && contiguous(p.dx),
                     vec_ok(p.dy) && vec_ok(p.t) && vec_ok(p.dt) && vec_ok(p.dx),
                     ring({p.dy, p.t, p.dt}), RMS_BWD_BLOCKS, ctx->sm_count);
}

template <int W, int V, int KIND, int MAXT>
RowKernel fwd_entry(const RowPlan &r, int C) {
    using Ring = Rows<W, V, KIND, 2, ring_rows<KIND, MAXT>()>;
    if constexpr (W == 8 && Ring::smem(MAXT, 0, 0) > NORM_MAX_RING)
        return fwd_entry<W, V, ROWS_REGS, MAXT>(r, C);
    else
        return {(const void *)rms_rows_kernel<W, V, KIND, MAXT>, Ring::smem(r.threads, r.tpr, C)};
}

template <int W, int KIND>
RowKernel fwd_kernel(const RowPlan &r, int C) {
    constexpr int V = W == 8 ? 2 : 8;  // vectors a thread of a long row
    if constexpr (W == 8 && KIND == ROWS_REGS) {
        if (r.v == 1 && r.threads > 512) return fwd_entry<8, 1, KIND, 1024>(r, C);
        if (r.v == 1 && r.threads > NORM_THREADS) return fwd_entry<8, 1, KIND, 512>(r, C);
    }
    if (r.threads > 512) return fwd_entry<W, V, KIND, 1024>(r, C);
    if (r.threads > NORM_THREADS) return fwd_entry<W, V, KIND, 512>(r, C);
    if (r.v == V) return fwd_entry<W, V, KIND, NORM_THREADS>(r, C);
    if (W == 1 && r.v == 4) return fwd_entry<W, W == 1 ? 4 : V, KIND, NORM_THREADS>(r, C);
    return fwd_entry<W, W == 8 ? 1 : 2, KIND, NORM_THREADS>(r, C);
}

template <int W, int V, int KIND, int MAXT>
RowKernel bwd_entry(const RowPlan &r, int C) {
    using Ring = Rows<W, V, KIND, 3, ring_rows<KIND, MAXT>()>;
    if constexpr (W == 8 && Ring::smem(MAXT, 0, 0) > NORM_MAX_RING)
        return {nullptr, 0};  // (two passes)
    else
        return {(const void *)rms_bwd_rows_kernel<W, V, KIND, MAXT>, Ring::smem(r.threads, r.tpr, C)};
}

template <int W, int KIND>
RowKernel bwd_kernel(const RowPlan &r, int C) {
    constexpr int V = W == 8 ? 2 : 8;  // vectors a thread of a long row
    if constexpr (W == 8 && KIND == ROWS_REGS) {
        if (r.v == 1 && r.threads > 512) return bwd_entry<8, 1, KIND, 1024>(r, C);
        if (r.v == 1 && r.threads > NORM_THREADS) return bwd_entry<8, 1, KIND, 512>(r, C);
    }
    if (r.threads > 512) return bwd_entry<W, V, KIND, 1024>(r, C);
    if (r.threads > NORM_THREADS) return bwd_entry<W, V, KIND, 512>(r, C);
    if (r.v == V) return bwd_entry<W, V, KIND, NORM_THREADS>(r, C);
    if (W == 1 && r.v == 4) return bwd_entry<W, W == 1 ? 4 : V, KIND, NORM_THREADS>(r, C);
    return bwd_entry<W, W == 8 ? 1 : 2, KIND, NORM_THREADS>(r, C);
}

}  // namespace

dlcStatus_t dlc_launch_rms(dlcContext *ctx, const RmsProblem &pb) {
    const RowPlan r = plan_fwd(ctx, pb);
    RmsProblem p = pb;
    int tpr = r.tpr, gamma_vec = (uintptr_t)p.gamma % 16 == 0;
    void *args[] = {&p, &tpr, &gamma_vec};
    const RowKernel k =
        r.w == 0 ? RowKernel{r.lanes ? (const void *)rms_any_kernel<true> : (const void *)rms_any_kernel<false>, 0}
        : r.w == 1 ? (pieces_ok(p.x) && pieces_ok(p.r) ? fwd_kernel<1, ROWS_BF16>(r, p.C) : fwd_kernel<1, ROWS_REGS>(r, p.C))
        : all_of(DLC_DATA_BFLOAT16, {p.x, p.r}) ? fwd_kernel<8, ROWS_BF16>(r, p.C)
        : all_of(DLC_DATA_FLOAT, {p.x, p.r}) ? fwd_kernel<8, ROWS_F32>(r, p.C) : fwd_kernel<8, ROWS_REGS>(r, p.C);
    if (!dlc_allow_smem(ctx, k.fn, k.smem)) return DLC_STATUS_EXECUTION_FAILED;
    return dlc_launch(ctx, k.fn, dim3((unsigned)r.blocks), dim3((unsigned)r.threads), k.smem, args);
}

size_t dlc_rms_bwd_workspace(const dlcContext *ctx, const RmsBwdProblem &p) {
    // the most blocks of any layout's plan, so that the pointers' alignment does not matter
    const long long most = (long long)ctx->sm_count * 4;
    const long long blocks = p.rows < most ? p.rows : most;
    return (size_t)blocks * p.C * sizeof(float);
}

dlcStatus_t dlc_launch_rms_bwd(dlcContext *ctx, const RmsBwdProblem &pb) {
    RowPlan r = plan_bwd(ctx, pb);
    RmsBwdProblem p = pb;
    int tpr = r.tpr, gamma_vec = (uintptr_t)p.gamma % 16 == 0;
    void *args[] = {&p, &tpr, &gamma_vec};
    RowKernel k =
        r.w == 0 ? RowKernel{r.lanes ? (const void *)rms_bwd_any_kernel<true> : (const void *)rms_bwd_any_kernel<false>, 0}
        : r.w == 1 ? (pieces_ok(p.dy) && pieces_ok(p.t) && pieces_ok(p.dt) ? bwd_kernel<1, ROWS_BF16>(r, p.C) : bwd_kernel<1, ROWS_REGS>(r, p.C))
        : all_of(DLC_DATA_BFLOAT16, {p.dy, p.t, p.dt}) ? bwd_kernel<8, ROWS_BF16>(r, p.C)
        : all_of(DLC_DATA_FLOAT, {p.dy, p.t, p.dt}) ? bwd_kernel<8, ROWS_F32>(r, p.C) : bwd_kernel<8, ROWS_REGS>(r, p.C);
    if (!k.fn) {
        r = two_pass_rows(p.rows, ctx->sm_count);
        k = RowKernel{(const void *)rms_bwd_any_kernel<false>, 0};
    }
    const int rpb = r.w ? r.threads / r.tpr : 1;
    const size_t smem = std::max(k.smem, rpb > 1 && p.dgamma ? (size_t)rpb * p.C * sizeof(float) : 0);
    if (!dlc_allow_smem(ctx, k.fn, smem)) return DLC_STATUS_EXECUTION_FAILED;
    dlcStatus_t st = dlc_launch(ctx, k.fn, dim3((unsigned)r.blocks), dim3((unsigned)r.threads), smem, args);
    if (st != DLC_STATUS_SUCCESS || !p.dgamma) return st;
    return dlc_launch_column_sum(ctx, p.ws, p.dgamma, p.C, (int)r.blocks);
}

dlcStatus_t dlc_launch_column_sum(dlcContext *ctx, const float *ws, float *out, int C, int blocks) {
    float *out2 = nullptr;
    long long all = C;
    void *args[] = {&ws, &out, &out2, &all, &all, &blocks};
    return dlc_launch(ctx, (const void *)column_sum_kernel, dim3((unsigned)((all + 31) / 32)), dim3(1024), 0, args);
}

dlcStatus_t dlc_launch_column_sums(dlcContext *ctx, const float *ws, float *out, float *out2, int C, int blocks) {
    long long half = C, all = 2 * half;  // (from 2^30 channels on more than an int holds)
    void *args[] = {&ws, &out, &out2, &half, &all, &blocks};
    return dlc_launch(ctx, (const void *)column_sum_kernel, dim3((unsigned)((all + 31) / 32)), dim3(1024), 0, args);
}

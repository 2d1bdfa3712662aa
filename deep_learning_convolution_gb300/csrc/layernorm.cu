// layernorm.cu -- layer norm over the channels of each row (pixel or token), with
// the residual's addition before it, and its backward pass.
//
//   t = x + r;  mu = mean_c t;  rho = 1 / sqrt(mean_c (t - mu)^2 + eps)
//   n = (t - mu) rho;  y = gamma n + beta;  E4M3 y: s = max_c |y| / 448, stored rn(y / s)
//
//   d = dy * gamma;  dx = rho (d - mean_c d - n mean_c(d n)) + dt
//   dgamma = sum_rows dy * n;  dbeta = sum_rows dy
//
// The squares are summed about the row's own mean, in a second reduction over registers: the
// difference of the mean square and the squared mean would lose what a large mean (or
// one large channel) leaves of the small ones.  Rows far from zero are centred twice (far_row).  Rows in the usual layouts are
// layernorm_vec.cu's and layernorm_shift.cu's; here are the others: mixed types, and unaligned rows where that is
// faster, with the rows' way through registers that the RMS norm has (rmsnorm.cu), channels apart and long rows
// read again for each step.  Instructions and latency bound them, measured back to back: 16384 x 1001 FP32
// unaligned with residual and sum 46 us (5.7 TB/s), backward 58 us; an FP32 stream beside BF16
// branches, 100352 x 512, 140 us, backward 228 us; channels apart, 128 images of 512 x 28 x 28 BF16, 262
// us, backward 641 us; 2730 x 12288 FP32 238 us, backward 392 us.
#include "norm_rows.cuh"

namespace {

using namespace dlc;

// Blocks of 256 threads an SM is to hold (what the registers are limited for).
constexpr int LN_FWD_BLOCKS = 3, LN_BWD_BLOCKS = 2;

// v - mean for the channels that exist, 0 for the others.
template <int W, int V>
__device__ __forceinline__ void centre(float (&v)[V * W], const Cols<W, V> &k, float mean) {
    constexpr int E = V * W;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) set2(v, i, add2(get2(v, i), pair_of(-mean)));
    if (k.count < V || k.n[V - 1] < W) {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i % W >= k.n[i / W]) v[i] = 0.f;
    }
}

// A sum of many terms and what its additions round off (Knuth's two-sum): the long rows' means.
struct LongSum {
    float s = 0.f, lost = 0.f;
    __device__ __forceinline__ void add(float v) {
        const float t = s + v, b = t - s;
        lost += (s - (t - b)) + (v - b);
        s = t;
    }
    __device__ __forceinline__ float value() const { return s + lost; }
};

// Centres a thread's part of a row again (far_row), or leaves it where `far` is false.
template <int W, int V>
__device__ __forceinline__ void recentre(float (&v)[V * W], const Cols<W, V> &k, bool far, int C, int tpr, int slot,
                                         float2 (*buf)[NORM_MAX_WARPS], int parity) {
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < V * W / 2; ++i) sum = add2(get2(v, i), sum);
    const float off = row_reduce<false>(sum.x + sum.y, 0.f, tpr, slot, buf, parity).x;
    centre<W, V>(v, k, far ? off / (float)C : 0.f);
}

// Rows in registers, as rms_rows_kernel has them.
template <int W, int V, int KIND, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > NORM_THREADS ? 1 : LN_FWD_BLOCKS)
    layer_rows_kernel(const __grid_constant__ LayerProblem p, int tpr, int gamma_vec) {
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
    float g[E], b[E];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int at = (t + j * tpr) * W;
        load_gamma<W>(p.gamma, at, p.C, gamma_vec != 0, g + j * W);
        if (p.beta) {
            load_gamma<W>(p.beta, at, p.C, gamma_vec != 0, b + j * W);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) b[j * W + i] = 0.f;
        }
    }
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
    for (int parity = 0; row - slot < p.rows; row += step, wt.next(), wy.next()) {
        const bool on = row < p.rows;
        float f[2][E];
        const uint32_t starts[2] = {(uint32_t)(row * p.x.m.ld * 2), (uint32_t)(row * p.r.m.ld * 2)};
        rows.take(f, cols, starts);
        auto &v = f[0];
        if (p.r.p) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) set2(v, i, add2(get2(v, i), get2(f[1], i)));
        }
        if (p.t.p && on) store_row<W, V>(p.t.dt, wt.at(p.t, row, c), cols, v);
        fetch();
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) sum = add2(get2(v, i), sum);
        const float mean = row_reduce<false>(sum.x + sum.y, 0.f, tpr, slot, buf, parity).x * inv_c;
        parity ^= 1;
        centre<W, V>(v, cols, mean);
        auto squares = [&]() {
            float2 sq = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) sq = fma2(get2(v, i), get2(v, i), sq);
            const float ss = row_reduce<false>(sq.x + sq.y, 0.f, tpr, slot, buf, parity).x;
            parity ^= 1;
            return ss;
        };
        float ss = squares();
        const bool far = far_row(mean, ss * inv_c);
        if (__builtin_expect(__any_sync(0xffffffffu, far), 0)) {
            recentre<W, V>(v, cols, far, p.C, tpr, slot, buf, parity);
            parity ^= 1;
            ss = squares();
        }
        const float2 rho = pair_of(rsqrtf(ss * inv_c + p.eps));
#pragma unroll
        for (int i = 0; i < E / 2; ++i) set2(v, i, fma2(mul2(get2(v, i), rho), get2(g, i), get2(b, i)));
        if (e4m3) {
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) mx = fmaxf(mx, fabsf(v[i]));
            mx = row_reduce<true>(0.f, mx, tpr, slot, buf, parity).y;
            parity ^= 1;
            const float scale = fmaxf(mx, SCALE_FLOOR) / E4M3_MAX, inv = 1.f / scale;
            if (t == 0 && on) p.scale[row] = scale;
#pragma unroll
            for (int i = 0; i < E / 2; ++i) set2(v, i, mul2(get2(v, i), pair_of(inv)));
        }
        if (on) store_row<W, V>(p.y.dt, wy.at(p.y, row, c), cols, v);
    }
}

// The remaining layouts (see AnyMap): the row is read again for every step, mostly from
// the L1 or L2, and t is worked out anew each time, so that it may overwrite x or r
// in the last one.
template <bool LANES>
__global__ void __launch_bounds__(NORM_THREADS) layer_any_kernel(const __grid_constant__ LayerProblem p) {
    using M = AnyMap<LANES>;
    griddep_launch_dependents();
    __shared__ float2 part[NORM_THREADS / 32][32];
    griddep_wait();
    const float inv_c = 1.f / (float)p.C;
    for (long long row0 = (long long)blockIdx.x * M::ROWS; row0 < p.rows; row0 += (long long)gridDim.x * M::ROWS) {
        const long long row = row0 + M::row();
        const bool on = row < p.rows;
        const long long xo = on ? row_off(p.x.m, row) : 0, ro = on && p.r.p ? row_off(p.r.m, row) : 0;
        float v[AHEAD], r[AHEAD];
        // fn(channel, t) for this thread's channels of the row
        auto each = [&](auto fn) {
            for (int c = M::first(); on && c < p.C; c += AHEAD * M::STEP) {
                const auto in = [&](int i) { return c + i * M::STEP < p.C; };
                load_elems<AHEAD>(p.x.p, p.x.dt, xo + c * p.x.m.cs, M::STEP * p.x.m.cs, in, v);
                if (p.r.p) {
                    load_elems<AHEAD>(p.r.p, p.r.dt, ro + c * p.r.m.cs, M::STEP * p.r.m.cs, in, r);
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i) v[i] += r[i];
                }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    if (in(i)) fn(c + i * M::STEP, v[i]);
            }
        };
        LongSum sum;
        float mx = 0.f, rest = 0.f;
        each([&](int, float t) { sum.add(t); });
        const float mean = M::template join<false>(sum.value(), 0.f, part).x * inv_c;
        auto squares = [&]() {
            float sq = 0.f;
            each([&](int, float t) {
                const float d = t - mean - rest;
                sq = fmaf(d, d, sq);
            });
            return M::template join<false>(sq, 0.f, part).x;
        };
        float sq = squares();
        const bool far = on && far_row(mean, sq * inv_c);
        if (__syncthreads_or(far)) {
            float off = 0.f;
            each([&](int, float t) { off += t - mean; });
            off = M::template join<false>(off, 0.f, part).x;
            if (far) rest = off / (float)p.C;
            sq = squares();
        }
        const float rho = rsqrtf(sq * inv_c + p.eps);
        auto y_of = [&](int c, float t) { return fmaf((t - mean - rest) * rho, p.gamma[c], p.beta ? p.beta[c] : 0.f); };
        float inv = 1.f;
        if (p.y.dt == DLC_DATA_FLOAT8_E4M3) {
            each([&](int c, float t) { mx = fmaxf(mx, fabsf(y_of(c, t))); });
            const float scale = fmaxf(M::template join<true>(0.f, mx, part).y, SCALE_FLOOR) / E4M3_MAX;
            if (on && M::first() == 0) p.scale[row] = scale;
            inv = 1.f / scale;
        }
        const long long to = on && p.t.p ? row_off(p.t.m, row) : 0, yo = on ? row_off(p.y.m, row) : 0;
        each([&](int c, float t) {
            if (p.t.p) store_elem(p.t.p, p.t.dt, to + c * p.t.m.cs, t);
            store_elem(p.y.p, p.y.dt, yo + c * p.y.m.cs, y_of(c, t) * inv);
        });
    }
}

// Backward, rows in registers.  Each thread adds up dgamma and dbeta of its own
// channels over the rows it visits; a block writes one partial row of each.
template <int W, int V, int KIND, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > NORM_THREADS ? 1 : LN_BWD_BLOCKS)
    layer_bwd_rows_kernel(const __grid_constant__ LayerBwdProblem p, int tpr, int gamma_vec) {
    griddep_launch_dependents();
    __shared__ float2 buf[2][NORM_MAX_WARPS];
    extern __shared__ uint4 ring_s[];
    constexpr int E = V * W;
    const int rpb = (int)blockDim.x / tpr, slot = (int)threadIdx.x / tpr, t = (int)threadIdx.x % tpr;
    const long long step = (long long)gridDim.x * rpb;
    const Cols<W, V> cols(t, tpr, p.C);
    const float inv_c = 1.f / (float)p.C;
    griddep_wait();
    float g[E], dg[E], db[E];
#pragma unroll
    for (int j = 0; j < V; ++j) load_gamma<W>(p.gamma, (t + j * tpr) * W, p.C, gamma_vec != 0, g + j * W);
#pragma unroll
    for (int i = 0; i < E; ++i) dg[i] = db[i] = 0.f;
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
    for (; row - slot < p.rows; row += step, wx.next()) {
        const bool on = row < p.rows;
        float f[3][E];
        const uint32_t starts[3] = {(uint32_t)(row * p.dy.m.ld * 2), (uint32_t)(row * p.t.m.ld * 2), (uint32_t)(row * p.dt.m.ld * 2)};
        rows.take(f, cols, starts);
        fetch();
        float2 sum = make_float2(0.f, 0.f), sd = sum;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            sum = add2(get2(f[1], i), sum);
            sd = fma2(get2(f[0], i), get2(g, i), sd);
        }
        const float2 means = row_reduce<false>(sum.x + sum.y, sd.x + sd.y, tpr, slot, buf, 0);
        centre<W, V>(f[1], cols, means.x * inv_c);
        auto squares = [&]() {
            float2 sq = make_float2(0.f, 0.f), dot = sq;
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const float2 v = get2(f[1], i);
                sq = fma2(v, v, sq);
                dot = fma2(mul2(get2(f[0], i), get2(g, i)), v, dot);
            }
            return row_reduce<false>(sq.x + sq.y, dot.x + dot.y, tpr, slot, buf, 1);
        };
        float2 red = squares();
        const bool far = far_row(means.x * inv_c, red.x * inv_c);
        if (__builtin_expect(__any_sync(0xffffffffu, far), 0)) {
            recentre<W, V>(f[1], cols, far, p.C, tpr, slot, buf, 0);
            red = squares();
        }
        if (!on) continue;
        const float rho = rsqrtf(red.x * inv_c + p.eps);
        // dx = rho d - rho mean(d) - (t - mu) rho^3 mean(d (t - mu))
        const float2 rho2 = pair_of(rho), k2 = pair_of(-row_slope(rho, red.y * inv_c)), m2 = pair_of(-rho * (means.y * inv_c));
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const float2 dy = get2(f[0], i), d = mul2(dy, rho2), v = get2(f[1], i);
            set2(dg, i, fma2(d, v, get2(dg, i)));
            set2(db, i, add2(dy, get2(db, i)));
            const float2 s = p.dt.p ? add2(get2(f[2], i), m2) : m2;
            set2(f[2], i, fma2(d, get2(g, i), fma2(v, k2, s)));
        }
        store_row<W, V>(p.dx.dt, wx.at(p.dx, row, c), cols, f[2]);
    }
    if (!p.dgamma && !p.dbeta) return;
    float *ws0 = p.ws + 2ll * blockIdx.x * p.C;  // [dgamma, dbeta][C] of this block
    if (rpb > 1) {  // join the block's row slots, in the ring's place: [slot][C], one sum after the other
        float *acc_s = reinterpret_cast<float *>(ring_s);
        cp_async_wait<0>();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (i % W < cols.n[i / W]) acc_s[(long long)slot * p.C + cols.c[i / W] + i % W] = h ? db[i] : dg[i];
            __syncthreads();
            for (int k = threadIdx.x; k < p.C; k += blockDim.x) {
                float s = 0.f;
                for (int i = 0; i < rpb; ++i) s += acc_s[(long long)i * p.C + k];
                ws0[(long long)h * p.C + k] = s;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i % W < cols.n[i / W]) {
                const int k = cols.c[i / W] + i % W;
                ws0[k] = dg[i];
                ws0[(long long)p.C + k] = db[i];
            }
    }
}

// Backward for the remaining layouts.  A block's sums collect in its rows of
// partial sums, a channel always through the same thread (LANES: its warp's
// rows joined by shuffles).
template <bool LANES>
__global__ void __launch_bounds__(NORM_THREADS) layer_bwd_any_kernel(const __grid_constant__ LayerBwdProblem p) {
    using M = AnyMap<LANES>;
    griddep_launch_dependents();
    __shared__ float2 part[NORM_THREADS / 32][32];
    griddep_wait();
    const float inv_c = 1.f / (float)p.C;
    float *ws0 = p.ws + 2ll * blockIdx.x * p.C;
    bool first = true;
    for (long long row0 = (long long)blockIdx.x * M::ROWS; row0 < p.rows; row0 += (long long)gridDim.x * M::ROWS) {
        const long long row = row0 + M::row();
        const bool on = row < p.rows;
        const long long yo = on ? row_off(p.dy.m, row) : 0, to = on ? row_off(p.t.m, row) : 0;
        float v[AHEAD], d[AHEAD], g[AHEAD], a[AHEAD];
        auto load = [&](int c, auto in) {
            load_elems<AHEAD>(p.t.p, p.t.dt, to + c * p.t.m.cs, M::STEP * p.t.m.cs, in, v);
            load_elems<AHEAD>(p.dy.p, p.dy.dt, yo + c * p.dy.m.cs, M::STEP * p.dy.m.cs, in, d);
            load_elems<AHEAD>(p.gamma, DLC_DATA_FLOAT, c, M::STEP, in, g);
        };
        LongSum sum;
        float sd = 0.f, rest = 0.f;
        // fn(t - mean - rest, dy, gamma) for this thread's channels of the row
        auto each = [&](float mean, auto fn) {
            for (int c = M::first(); on && c < p.C; c += AHEAD * M::STEP) {
                const auto in = [&](int i) { return c + i * M::STEP < p.C; };
                load(c, in);
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    if (in(i)) fn(v[i] - mean - rest, d[i], g[i]);
            }
        };
        each(0.f, [&](float t, float dy, float gamma) {
            sum.add(t);
            sd = fmaf(dy, gamma, sd);
        });
        const float2 means = M::template join<false>(sum.value(), sd, part);
        const float mean = means.x * inv_c;
        auto squares = [&]() {
            float sq = 0.f, dot = 0.f;
            each(mean, [&](float t, float dy, float gamma) {
                sq = fmaf(t, t, sq);
                dot = fmaf(dy * gamma, t, dot);
            });
            return M::template join<false>(sq, dot, part);
        };
        float2 red = squares();
        const bool far = on && far_row(mean, red.x * inv_c);
        if (__syncthreads_or(far)) {
            float off = 0.f;
            each(mean, [&](float t, float, float) { off += t; });
            off = M::template join<false>(off, 0.f, part).x;
            if (far) rest = off / (float)p.C;
            red = squares();
        }
        const float rho = on ? rsqrtf(red.x * inv_c + p.eps) : 0.f;
        const float k = row_slope(rho, red.y * inv_c), m = rho * (means.y * inv_c);
        const long long xo = on ? row_off(p.dx.m, row) : 0, so = on && p.dt.p ? row_off(p.dt.m, row) : 0;
        for (int c = M::first(); c < p.C; c += AHEAD * M::STEP) {
            const auto in = [&](int i) { return on && c + i * M::STEP < p.C; };
            load(c, in);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) a[i] = 0.f;
            if (p.dt.p) load_elems<AHEAD>(p.dt.p, p.dt.dt, so + c * p.dt.m.cs, M::STEP * p.dt.m.cs, in, a);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int ci = c + i * M::STEP;
                if (ci >= p.C) break;
                const float t = v[i] - mean - rest;
                if (on) store_elem(p.dx.p, p.dx.dt, xo + ci * p.dx.m.cs, a[i] - m + rho * d[i] * g[i] - t * k);
                if (!p.dgamma && !p.dbeta) continue;
                float dg = on ? d[i] * rho * t : 0.f, db = d[i];
                if (LANES)
                    for (int o = 16; o > 0; o /= 2) {
                        dg += __shfl_xor_sync(0xffffffffu, dg, o);
                        db += __shfl_xor_sync(0xffffffffu, db, o);
                    }
                if (!LANES || M::row() == 0) {
                    float *w = ws0 + ci;
                    w[0] = first ? dg : w[0] + dg;
                    w[p.C] = first ? db : w[p.C] + db;
                }
            }
        }
        first = false;
    }
}

// ---- host side ---------------------------------------------------------------

template <int W, int V, int KIND, int MAXT>
RowKernel fwd_entry(const RowPlan &r, int C) {
    using Ring = Rows<W, V, KIND, 2, ring_rows<KIND, MAXT>()>;
    if constexpr (W == 8 && Ring::smem(MAXT, 0, 0) > NORM_MAX_RING)
        return {nullptr, 0};  // (the row read again for each step)
    else
        return {(const void *)layer_rows_kernel<W, V, KIND, MAXT>, Ring::smem(r.threads, r.tpr, C)};
}

template <int W, int V, int KIND, int MAXT>
RowKernel bwd_entry(const RowPlan &r, int C) {
    using Ring = Rows<W, V, KIND, 3, ring_rows<KIND, MAXT>()>;
    if constexpr (W == 8 && Ring::smem(MAXT, 0, 0) > NORM_MAX_RING)
        return {nullptr, 0};
    else
        return {(const void *)layer_bwd_rows_kernel<W, V, KIND, MAXT>, Ring::smem(r.threads, r.tpr, C)};
}

template <int W, int KIND, bool BWD, int V, int MAXT>
RowKernel entry(const RowPlan &r, int C) {
    if constexpr (BWD)
        return bwd_entry<W, V, KIND, MAXT>(r, C);
    else
        return fwd_entry<W, V, KIND, MAXT>(r, C);
}

template <int W, int KIND, bool BWD>
RowKernel kernel_of(const RowPlan &r, int C) {
    constexpr int V = W == 8 ? 2 : 8;  // vectors a thread of a long row
    if constexpr (W == 8 && KIND == ROWS_REGS) {  // a row ahead in registers: one vector a thread
        if (r.v == V) return {nullptr, 0};
        if (r.threads > 512) return entry<8, KIND, BWD, 1, 1024>(r, C);
        if (r.threads > NORM_THREADS) return entry<8, KIND, BWD, 1, 512>(r, C);
        return entry<8, KIND, BWD, 1, NORM_THREADS>(r, C);
    } else {
        if (r.threads > 512) return entry<W, KIND, BWD, V, 1024>(r, C);
        if (r.threads > NORM_THREADS) return entry<W, KIND, BWD, V, 512>(r, C);
        if (r.v == V) return entry<W, KIND, BWD, V, NORM_THREADS>(r, C);
        if (W == 1 && r.v == 4) return entry<W, KIND, BWD, W == 1 ? 4 : V, NORM_THREADS>(r, C);
        return entry<W, KIND, BWD, W == 8 ? 1 : 2, NORM_THREADS>(r, C);
    }
}

// The kernel that reads `ts` by the plan; none where the row does not fit registers.
template <bool BWD>
RowKernel row_kernel(const RowPlan &r, int C, std::initializer_list<RowTensor> ts) {
    if (r.w == 0) return {nullptr, 0};
    if (r.w == 1) {
        bool pieces = true;
        for (const RowTensor &t : ts) pieces = pieces && pieces_ok(t);
        return pieces ? kernel_of<1, ROWS_BF16, BWD>(r, C) : kernel_of<1, ROWS_REGS, BWD>(r, C);
    }
    return all_of(DLC_DATA_BFLOAT16, ts) ? kernel_of<8, ROWS_BF16, BWD>(r, C)
           : all_of(DLC_DATA_FLOAT, ts)  ? kernel_of<8, ROWS_F32, BWD>(r, C)
                                         : kernel_of<8, ROWS_REGS, BWD>(r, C);
}

}  // namespace

dlcStatus_t dlc_launch_layer(dlcContext *ctx, const LayerProblem &pb) {
    LayerProblem p = pb;
    dlcStatus_t done;
    if (dlc_layer_vec(ctx, p, done) || dlc_layer_shift(ctx, p, done)) return done;
    RowPlan r = plan_rows(p.rows, p.C, contiguous(p.x) && contiguous(p.r) && contiguous(p.t) && contiguous(p.y),
                          vec_ok(p.x) && vec_ok(p.r) && vec_ok(p.t) && vec_ok(p.y), ring({p.x, p.r}), LN_FWD_BLOCKS, ctx->sm_count);
    RowKernel k = row_kernel<false>(r, p.C, {p.x, p.r});
    if (!k.fn) {
        if (r.w) r = two_pass_rows(p.rows, ctx->sm_count);
        k.fn = r.lanes ? (const void *)layer_any_kernel<true> : (const void *)layer_any_kernel<false>;
    }
    int tpr = r.tpr, gamma_vec = (uintptr_t)p.gamma % 16 == 0 && (uintptr_t)p.beta % 16 == 0;
    void *args[] = {&p, &tpr, &gamma_vec};
    if (!dlc_allow_smem(ctx, k.fn, k.smem)) return DLC_STATUS_EXECUTION_FAILED;
    return dlc_launch(ctx, k.fn, dim3((unsigned)r.blocks), dim3((unsigned)r.threads), k.smem, args);
}

size_t dlc_layer_bwd_workspace(const dlcContext *ctx, long long rows, int C) {
    // the most blocks of any layout's plan, so that the pointers' alignment does not matter
    return (size_t)std::min((rows + 7) / 8 * 8, (long long)ctx->sm_count * 4) * 2 * C * sizeof(float);
}

dlcStatus_t dlc_launch_layer_bwd(dlcContext *ctx, const LayerBwdProblem &pb) {
    LayerBwdProblem p = pb;
    dlcStatus_t done;
    if (dlc_layer_bwd_vec(ctx, p, done) || dlc_layer_bwd_shift(ctx, p, done)) return done;
    RowPlan r = plan_rows(p.rows, p.C, contiguous(p.dy) && contiguous(p.t) && contiguous(p.dt) && contiguous(p.dx),
                          vec_ok(p.dy) && vec_ok(p.t) && vec_ok(p.dt) && vec_ok(p.dx), ring({p.dy, p.t, p.dt}), LN_BWD_BLOCKS,
                          ctx->sm_count);
    RowKernel k = row_kernel<true>(r, p.C, {p.dy, p.t, p.dt});
    if (!k.fn) {
        if (r.w) r = two_pass_rows(p.rows, ctx->sm_count);
        k.fn = r.lanes ? (const void *)layer_bwd_any_kernel<true> : (const void *)layer_bwd_any_kernel<false>;
    }
    const int rpb = r.w ? r.threads / r.tpr : 1;
    const bool sums = p.dgamma || p.dbeta;
    const size_t smem = std::max(k.smem, rpb > 1 && sums ? (size_t)rpb * p.C * sizeof(float) : 0);
    int tpr = r.tpr, gamma_vec = (uintptr_t)p.gamma % 16 == 0;
    void *args[] = {&p, &tpr, &gamma_vec};
    if (!dlc_allow_smem(ctx, k.fn, smem)) return DLC_STATUS_EXECUTION_FAILED;
    const dlcStatus_t st = dlc_launch(ctx, k.fn, dim3((unsigned)r.blocks), dim3((unsigned)r.threads), smem, args);
    if (st != DLC_STATUS_SUCCESS || !sums) return st;
    return dlc_launch_column_sums(ctx, p.ws, p.dgamma, p.dbeta, p.C, (int)r.blocks);
}

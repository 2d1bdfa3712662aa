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
#include <initializer_list>

#include "channel.cuh"
#include "ptx.cuh"
#include "row_ring.cuh"

namespace {

using namespace dlc;

constexpr float E4M3_MAX = 448.f;
constexpr float SCALE_FLOOR = 1e-30f;  // max |y| of an all-zero row counts as this
constexpr int RMS_THREADS = 256;
constexpr int RMS_MAX_WARPS = 32;
// Blocks of 256 threads an SM is to hold (what the registers are limited for).
constexpr int RMS_FWD_BLOCKS = 4, RMS_BWD_BLOCKS = 2;

// A ring that a block's shared memory cannot hold (FP32 rows of 8193 to 16384 channels:
// 256 KiB forward, 384 backward) gives way to one row ahead in registers forward, and to the
// two-pass kernel backward, where the registers spill.  2730 x 12288: forward 171 us;
// backward 261 us, 433 through registers.
constexpr size_t RMS_MAX_RING = 226 * 1024;

// Rows of the ring.  Measured when chosen, 100352 x 512 forward / 25088 x 1024 backward, BF16:
// 3 rows at 4 / 2 blocks an SM 74.5 / 40.0 us; 4 rows 77.6 / 41.1; one row ahead
// in registers 109 us forward.
// FP32 rows, twice the bytes, and blocks of 1024 threads: 2.
template <int KIND, int MAXT>
constexpr int ring_rows() { return MAXT > 512 || KIND == ROWS_F32 ? 2 : 3; }

// A thread's part of a row: its vectors (W = 8), or single elements (W = 1).
template <int W, int V>
__device__ __forceinline__ void store_row(int dt, char *at, const Cols<W, V> &k, const float (&f)[V * W]) {
    if constexpr (W == 1) {
        if (dt == DLC_DATA_BFLOAT16) {
            unsigned short *p = reinterpret_cast<unsigned short *>(at);
#pragma unroll
            for (int j = 0; j < V; ++j, p += k.step)
                if (j < k.count) *p = (unsigned short)pack_bf16(f[j], 0.f);
        } else if (dt == DLC_DATA_FLOAT) {
            float *p = reinterpret_cast<float *>(at);
#pragma unroll
            for (int j = 0; j < V; ++j, p += k.step)
                if (j < k.count) *p = f[j];
        } else {
            unsigned char *p = reinterpret_cast<unsigned char *>(at);
#pragma unroll
            for (int j = 0; j < V; j += 2, p += 2 * k.step) {
                const uint32_t q = pack_e4m3(f[j], f[j + 1]);
                if (j < k.count) p[0] = (unsigned char)q;
                if (j + 1 < k.count) p[k.step] = (unsigned char)(q >> 8);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float *v = f + j * W;
            const int d = j * k.step;
            if (k.n[j] == W) {
                if (dt == DLC_DATA_BFLOAT16) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < W / 2; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
                    *reinterpret_cast<uint4 *>(at + 2 * d) = make_uint4(w[0], w[1], w[2], w[3]);
                } else if (dt == DLC_DATA_FLOAT) {
                    float4 *p = reinterpret_cast<float4 *>(at + 4 * d);
#pragma unroll
                    for (int i = 0; i < W / 4; ++i) p[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                } else {
                    uint32_t w[2];
#pragma unroll
                    for (int i = 0; i < W / 4; ++i)
                        w[i] = pack_e4m3(v[4 * i], v[4 * i + 1]) | (pack_e4m3(v[4 * i + 2], v[4 * i + 3]) << 16);
                    *reinterpret_cast<uint2 *>(at + d) = make_uint2(w[0], w[1]);
                }
            } else if (k.n[j] > 0) {
#pragma unroll
                for (int i = 0; i < W - 1; ++i)
                    if (i < k.n[j]) store_elem(at, dt, d + i, v[i]);
            }
        }
    }
}

template <int W>
__device__ __forceinline__ void load_gamma(const float *gamma, int c, int C, bool vec, float *v) {
    if (W == 8 && vec && c + W <= C) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const float4 a = reinterpret_cast<const float4 *>(gamma + c)[i];
            v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = a.z, v[4 * i + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = c + i < C ? gamma[c + i] : 0.f;
    }
}

// (sum of a, sum or maximum of b) over the `tpr` threads of a row: a power of
// two, within a warp or whole warps.  The row's threads meet at a named
// barrier of their own; the buffer alternates between calls, so one barrier a
// call is enough.
template <bool MAX_B>
__device__ __forceinline__ float2 row_reduce(float a, float b, int tpr, int slot, float2 (*buf)[RMS_MAX_WARPS], int parity) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        if (o < 8 || o < tpr) {  // (a row has eight threads at least)
            a += __shfl_xor_sync(0xffffffffu, a, o);
            const float ob = __shfl_xor_sync(0xffffffffu, b, o);
            b = MAX_B ? fmaxf(b, ob) : b + ob;
        }
    }
    if (tpr > 32) {
        const int warps = tpr >> 5;
        const float2 *row = buf[parity] + slot * warps;
        if ((threadIdx.x & 31) == 0) buf[parity][threadIdx.x >> 5] = make_float2(a, b);
        asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(tpr) : "memory");
        const float2 v0 = row[0], v1 = row[1];
        a = v0.x + v1.x;
        b = MAX_B ? fmaxf(v0.y, v1.y) : v0.y + v1.y;
        for (int i = 2; i < warps; ++i) {
            const float2 v = row[i];
            a += v.x;
            b = MAX_B ? fmaxf(b, v.y) : b + v.y;
        }
    }
    return make_float2(a, b);
}

// An E4M3 row's scale, and the two factors that take gamma * t to the stored values
// y / scale, one after the other.  Their product rho / scale leaves FP32's range where
// |y| is near the scale's floor and rho large (a zero row under an epsilon of 1e-12):
// infinity times zero would be NaN, so rho then comes first.  A row of zeros is zeros
// without an epsilon too.  NaN stays NaN.
struct E4m3Row {
    float scale, first, then;
    __device__ __forceinline__ E4m3Row(float squares, float amax, float rho) {
        if (squares == 0.f && amax == 0.f) rho = 0.f;
        const float top = amax * rho;
        scale = (top < SCALE_FLOOR ? SCALE_FLOOR : top) / E4M3_MAX;
        first = 1.f;
        then = rho / scale;
        if (isinf(then)) first = rho, then = 1.f / scale;
    }
};

// Rows in registers: `tpr` threads a row (8 to 1024: short rows take few, so that a
// block's loads cover several rows), V vectors of W channels a thread.
// The next row's loads are issued before this row's reduction waits.
template <int W, int V, int KIND, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > RMS_THREADS ? 1 : RMS_FWD_BLOCKS)
    rms_rows_kernel(const __grid_constant__ RmsProblem p, int tpr, int gamma_vec) {
    griddep_launch_dependents();
    __shared__ float2 buf[2][RMS_MAX_WARPS];
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

// The remaining layouts, two passes over a row.  LANES (channels apart): 32
// rows a block, one per lane, the channels dealt to eight warps, so neighbouring
// rows share the loads.  Otherwise (a row too long for registers): one row a
// block, its channels dealt to the threads.  The second pass recomputes t (so t
// may overwrite x or r in place); it finds most of a row in the L1 or L2, and the
// loads' latency bounds these layouts, four a thread in flight.
constexpr int AHEAD = 4;  // channels a thread loads at once

template <bool LANES>
struct AnyMap {
    static constexpr int ROWS = LANES ? 32 : 1, STEP = LANES ? 8 : RMS_THREADS;
    static __device__ __forceinline__ int row() { return LANES ? (int)(threadIdx.x & 31) : 0; }
    static __device__ __forceinline__ int first() { return LANES ? (int)(threadIdx.x >> 5) : (int)threadIdx.x; }
    // sums a (and sums or maximises b) over the threads of this thread's row
    template <bool MAX_B>
    static __device__ float2 join(float a, float b, float2 (*part)[32]) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (!LANES) {
            for (int o = 16; o > 0; o /= 2) {
                a += __shfl_xor_sync(0xffffffffu, a, o);
                const float ob = __shfl_xor_sync(0xffffffffu, b, o);
                b = MAX_B ? fmaxf(b, ob) : b + ob;
            }
        }
        __syncthreads();
        part[warp][lane] = make_float2(a, b);
        __syncthreads();
        a = 0.f, b = 0.f;
        for (int i = 0; i < RMS_THREADS / 32; ++i) {
            const float2 v = part[i][lane];
            a += v.x;
            b = MAX_B ? fmaxf(b, v.y) : b + v.y;
        }
        return make_float2(a, b);
    }
};

template <bool LANES>
__global__ void __launch_bounds__(RMS_THREADS) rms_any_kernel(const __grid_constant__ RmsProblem p) {
    using M = AnyMap<LANES>;
    griddep_launch_dependents();
    __shared__ float2 part[RMS_THREADS / 32][32];
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

// rho^3 * mean(d t): about rho^2 for rows of any size, where rho^3 alone is out of
// FP32's range for rows of 1e-13 or 1e13.
__device__ __forceinline__ float row_slope(float rho, float mean) { return rho * (rho * (rho * mean)); }

// Backward, rows in registers.  Each thread adds up dgamma of its own channels
// over the rows it visits; a block writes one partial row of sums.
template <int W, int V, int KIND, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > RMS_THREADS ? 1 : RMS_BWD_BLOCKS)
    rms_bwd_rows_kernel(const __grid_constant__ RmsBwdProblem p, int tpr, int gamma_vec) {
    griddep_launch_dependents();
    __shared__ float2 buf[2][RMS_MAX_WARPS];
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
__global__ void __launch_bounds__(RMS_THREADS) rms_bwd_any_kernel(const __grid_constant__ RmsBwdProblem p) {
    using M = AnyMap<LANES>;
    griddep_launch_dependents();
    __shared__ float2 part[RMS_THREADS / 32][32];
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
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *ws, float *out, int C, int blocks) {
    griddep_launch_dependents();
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (int)blockIdx.x * 32 + lane;
    griddep_wait();
    float s = 0.f;
    if (c < C) {
#pragma unroll 8
        for (int b = warp; b < blocks; b += 32) s += ws[(long long)b * C + c];
    }
    part[warp][lane] = s;
    __syncthreads();
    s = part[lane][warp];  // column `warp`
    for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0 && (int)blockIdx.x * 32 + warp < C) out[(int)blockIdx.x * 32 + warp] = s;
}

// ---- host side ---------------------------------------------------------------

struct RowPlan {
    int w = 0, v = 0;  // channels per vector (0: the two-pass kernels), vectors per thread
    bool lanes = false;
    int tpr = 0, threads = 0;
    long long blocks = 0;
};

// Whether every row of t can be read in 16-byte vectors of eight channels.
bool vec_ok(const RowTensor &t) {
    if (!t.p) return true;
    const int e = dlc_dtype_bytes((dlcDataType_t)t.dt);
    const long long b = e == 1 ? 8 : 16;
    auto mult = [&](long long s) { return (s * e) % b == 0; };
    return (uintptr_t)t.p % b == 0 &&
           (t.m.uniform ? mult(t.m.ld) : (mult(t.m.s0) && mult(t.m.s2) && mult(t.m.s3)));
}

bool contiguous(const RowTensor &t) { return !t.p || t.m.cs == 1; }

bool all_of(int dt, std::initializer_list<RowTensor> ts) {
    for (const RowTensor &t : ts)
        if (t.p && t.dt != dt) return false;
    return true;
}

bool ring(std::initializer_list<RowTensor> ts) { return all_of(DLC_DATA_BFLOAT16, ts) || all_of(DLC_DATA_FLOAT, ts); }

RowPlan plan_rows(long long rows, int C, bool cs1, bool vec, bool ring, int per_sm, int sm_count) {
    RowPlan r;
    r.threads = RMS_THREADS;
    r.lanes = !cs1;
    if (cs1) {
        r.w = vec ? 8 : 1;
        // vectors a thread: few for short rows (more threads a row); rows held in
        // registers a row ahead take one, or two of a very long row
        const int v_max = vec ? (ring ? 2 : 1) : 8;
        const long long nv = (C + r.w - 1) / r.w;
        int v = vec ? 1 : 2, tpr = 8;
        while (tpr < 32 && tpr * v < nv) tpr *= 2;
        while (v < v_max && tpr * v < nv && tpr == 32) v *= 2;
        while (tpr < 1024 && (long long)tpr * v < nv) tpr *= 2;
        if (vec && (long long)tpr * v < nv) v = 2;
        if ((long long)tpr * v < nv) r.w = 0;  // longer than a block's registers
        r.v = v;
        r.tpr = tpr;
        if (r.w && tpr > RMS_THREADS) r.threads = tpr;
    }
    const int rpb = r.w ? r.threads / r.tpr : (r.lanes ? 32 : 1);
    const long long need = (rows + rpb - 1) / rpb;
    const long long most = (long long)sm_count * (r.w ? (r.threads > RMS_THREADS ? 1 : per_sm) : 4);
    r.blocks = need < most ? need : most;
    return r;
}

// One row a block at a time, twice over it.
RowPlan two_pass_rows(long long rows, int sm_count) {
    RowPlan r;
    r.threads = RMS_THREADS;
    r.blocks = std::min(rows, (long long)sm_count * 4);
    return r;
}

RowPlan plan_fwd(const dlcContext *ctx, const RmsProblem &p) {
    return plan_rows(p.rows, p.C, contiguous(p.x) && contiguous(p.r) && contiguous(p.t) && contiguous(p.y),
                     vec_ok(p.x) && vec_ok(p.r) && vec_ok(p.t) && vec_ok(p.y), ring({p.x, p.r}), RMS_FWD_BLOCKS, ctx->sm_count);
}

RowPlan plan_bwd(const dlcContext *ctx, const RmsBwdProblem &p) {
    return plan_rows(p.rows, p.C, contiguous(p.dy) && contiguous(p.t) && contiguous(p.dt) && contiguous(p.dx),
                     vec_ok(p.dy) && vec_ok(p.t) && vec_ok(p.dt) && vec_ok(p.dx),
                     ring({p.dy, p.t, p.dt}), RMS_BWD_BLOCKS, ctx->sm_count);
}

// Rows that may be copied in the 16-byte pieces they touch: the first row
// starts one, so no piece starts before the tensor.
bool pieces_ok(const RowTensor &t) {
    return !t.p || (t.dt == DLC_DATA_BFLOAT16 && t.m.uniform && (uintptr_t)t.p % 16 == 0);
}

struct RowKernel {
    const void *fn;
    size_t smem;
};

template <int W, int V, int KIND, int MAXT>
RowKernel fwd_entry(const RowPlan &r, int C) {
    using Ring = Rows<W, V, KIND, 2, ring_rows<KIND, MAXT>()>;
    if constexpr (W == 8 && Ring::smem(MAXT, 0, 0) > RMS_MAX_RING)
        return fwd_entry<W, V, ROWS_REGS, MAXT>(r, C);
    else
        return {(const void *)rms_rows_kernel<W, V, KIND, MAXT>, Ring::smem(r.threads, r.tpr, C)};
}

template <int W, int KIND>
RowKernel fwd_kernel(const RowPlan &r, int C) {
    constexpr int V = W == 8 ? 2 : 8;  // vectors a thread of a long row
    if constexpr (W == 8 && KIND == ROWS_REGS) {
        if (r.v == 1 && r.threads > 512) return fwd_entry<8, 1, KIND, 1024>(r, C);
        if (r.v == 1 && r.threads > RMS_THREADS) return fwd_entry<8, 1, KIND, 512>(r, C);
    }
    if (r.threads > 512) return fwd_entry<W, V, KIND, 1024>(r, C);
    if (r.threads > RMS_THREADS) return fwd_entry<W, V, KIND, 512>(r, C);
    if (r.v == V) return fwd_entry<W, V, KIND, RMS_THREADS>(r, C);
    if (W == 1 && r.v == 4) return fwd_entry<W, W == 1 ? 4 : V, KIND, RMS_THREADS>(r, C);
    return fwd_entry<W, W == 8 ? 1 : 2, KIND, RMS_THREADS>(r, C);
}

template <int W, int V, int KIND, int MAXT>
RowKernel bwd_entry(const RowPlan &r, int C) {
    using Ring = Rows<W, V, KIND, 3, ring_rows<KIND, MAXT>()>;
    if constexpr (W == 8 && Ring::smem(MAXT, 0, 0) > RMS_MAX_RING)
        return {nullptr, 0};  // (two passes)
    else
        return {(const void *)rms_bwd_rows_kernel<W, V, KIND, MAXT>, Ring::smem(r.threads, r.tpr, C)};
}

template <int W, int KIND>
RowKernel bwd_kernel(const RowPlan &r, int C) {
    constexpr int V = W == 8 ? 2 : 8;  // vectors a thread of a long row
    if constexpr (W == 8 && KIND == ROWS_REGS) {
        if (r.v == 1 && r.threads > 512) return bwd_entry<8, 1, KIND, 1024>(r, C);
        if (r.v == 1 && r.threads > RMS_THREADS) return bwd_entry<8, 1, KIND, 512>(r, C);
    }
    if (r.threads > 512) return bwd_entry<W, V, KIND, 1024>(r, C);
    if (r.threads > RMS_THREADS) return bwd_entry<W, V, KIND, 512>(r, C);
    if (r.v == V) return bwd_entry<W, V, KIND, RMS_THREADS>(r, C);
    if (W == 1 && r.v == 4) return bwd_entry<W, W == 1 ? 4 : V, KIND, RMS_THREADS>(r, C);
    return bwd_entry<W, W == 8 ? 1 : 2, KIND, RMS_THREADS>(r, C);
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
    void *args[] = {&ws, &out, &C, &blocks};
    return dlc_launch(ctx, (const void *)column_sum_kernel, dim3((unsigned)((C + 31) / 32)), dim3(1024), 0, args);
}

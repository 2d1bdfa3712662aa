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
// scale comes from the same reduction as the sum of squares.
#include "channel.cuh"
#include "ptx.cuh"

namespace {

using namespace dlc;

constexpr float E4M3_MAX = 448.f;
constexpr float SCALE_FLOOR = 1e-30f;  // max |y| of an all-zero row counts as this
constexpr int RMS_THREADS = 256;
constexpr int RMS_MAX_WARPS = 32;

// W consecutive elements (n <= W of them inside the row) as FP32.  W = 8: the
// address is 16-byte aligned; a partial vector is read element by element, so
// nothing past the row is touched.
template <int W>
__device__ __forceinline__ void load_vec(const RowTensor &t, long long off, int n, float *v) {
    if constexpr (W == 1) {
        v[0] = n > 0 ? load_elem(t.p, t.dt, off) : 0.f;
    } else {
        if (n >= W) {
            if (t.dt == DLC_DATA_BFLOAT16) {
                const uint4 q = *reinterpret_cast<const uint4 *>(static_cast<const unsigned short *>(t.p) + off);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[2 * i] = __uint_as_float(w[i] << 16);
                    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                }
            } else {
                const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(t.p) + off);
                const float4 a = f[0], b = f[1];
                v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
                v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] = i < n ? load_elem(t.p, t.dt, off + i) : 0.f;
        }
    }
}

template <int W>
__device__ __forceinline__ void store_vec(const RowTensor &t, long long off, int n, const float *v) {
    if constexpr (W == 1) {
        if (n > 0) store_elem(t.p, t.dt, off, v[0]);
    } else {
        if (n >= W) {
            if (t.dt == DLC_DATA_BFLOAT16) {
                *reinterpret_cast<uint4 *>(static_cast<unsigned short *>(t.p) + off) =
                    make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
            } else if (t.dt == DLC_DATA_FLOAT) {
                float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(t.p) + off);
                f[0] = make_float4(v[0], v[1], v[2], v[3]);
                f[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                *reinterpret_cast<uint2 *>(static_cast<unsigned char *>(t.p) + off) =
                    make_uint2(pack_e4m3(v[0], v[1]) | (pack_e4m3(v[2], v[3]) << 16),
                               pack_e4m3(v[4], v[5]) | (pack_e4m3(v[6], v[7]) << 16));
            }
        } else {
            for (int i = 0; i < W; ++i)
                if (i < n) store_elem(t.p, t.dt, off + i, v[i]);
        }
    }
}

template <int W>
__device__ __forceinline__ void load_gamma(const float *gamma, int c, int C, float *v) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = c + i < C ? __ldg(gamma + c + i) : 0.f;
}

// (sum of a, sum or maximum of b) over the `tpr` threads of a row: a power of
// two, within a warp or whole warps.  All of the block's threads call it; the
// buffer alternates between calls, so one barrier per call is enough.
template <bool MAX_B>
__device__ __forceinline__ float2 row_reduce(float a, float b, int tpr, float2 (*buf)[RMS_MAX_WARPS], int parity) {
    for (int o = (tpr < 32 ? tpr : 32) / 2; o > 0; o /= 2) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        const float ob = __shfl_xor_sync(0xffffffffu, b, o);
        b = MAX_B ? fmaxf(b, ob) : b + ob;
    }
    if (tpr > 32) {
        const int warp = threadIdx.x >> 5, first = (threadIdx.x / tpr) * (tpr >> 5);
        if ((threadIdx.x & 31) == 0) buf[parity][warp] = make_float2(a, b);
        __syncthreads();
        a = 0.f, b = 0.f;
        for (int i = 0; i < (tpr >> 5); ++i) {
            const float2 v = buf[parity][first + i];
            a += v.x;
            b = MAX_B ? fmaxf(b, v.y) : b + v.y;
        }
    }
    return make_float2(a, b);
}

// 1 / scale and scale of an E4M3 row whose largest |y| is `amax` (NaN stays NaN).
__device__ __forceinline__ float e4m3_scale(float amax) {
    return (amax < SCALE_FLOOR ? SCALE_FLOOR : amax) / E4M3_MAX;
}

// Rows in registers: `tpr` threads a row, V vectors of W channels a thread.
template <int W, int V>
__global__ void __launch_bounds__(1024) rms_rows_kernel(const __grid_constant__ RmsProblem p, int tpr) {
    griddep_launch_dependents();
    __shared__ float2 buf[2][RMS_MAX_WARPS];
    const int rpb = (int)blockDim.x / tpr, slot = (int)threadIdx.x / tpr, t = (int)threadIdx.x % tpr;
    griddep_wait();
    int parity = 0;
    for (long long row0 = (long long)blockIdx.x * rpb; row0 < p.rows; row0 += (long long)gridDim.x * rpb, parity ^= 1) {
        const long long row = row0 + slot;
        const bool on = row < p.rows;
        const long long xo = on ? row_off(p.x.m, row) : 0;
        const long long ro = on && p.r.p ? row_off(p.r.m, row) : 0;
        float v[V][W];
        float sq = 0.f, mx = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (t + j * tpr) * W, n = on ? p.C - c : 0;
            load_vec<W>(p.x, xo + c, n, v[j]);
            if (p.r.p) {
                float r[W];
                load_vec<W>(p.r, ro + c, n, r);
#pragma unroll
                for (int i = 0; i < W; ++i) v[j][i] += r[i];
            }
        }
        if (p.t.p && on) {
            const long long to = row_off(p.t.m, row);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (t + j * tpr) * W;
                store_vec<W>(p.t, to + c, p.C - c, v[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float g[W];
            load_gamma<W>(p.gamma, (t + j * tpr) * W, p.C, g);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                sq = fmaf(v[j][i], v[j][i], sq);
                v[j][i] *= g[i];
                mx = fmaxf(mx, fabsf(v[j][i]));
            }
        }
        const float2 red = row_reduce<true>(sq, mx, tpr, buf, parity);
        if (!on) continue;
        float f = rsqrtf(red.x / (float)p.C + p.eps);
        if (p.y.dt == DLC_DATA_FLOAT8_E4M3) {
            const float s = e4m3_scale(red.y * f);
            if (t == 0) p.scale[row] = s;
            f = f / s;
        }
        const long long yo = row_off(p.y.m, row);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (t + j * tpr) * W;
#pragma unroll
            for (int i = 0; i < W; ++i) v[j][i] *= f;
            store_vec<W>(p.y, yo + c, p.C - c, v[j]);
        }
    }
}

// The remaining layouts (channels not contiguous, or too many for registers):
// 32 rows a block, one per lane, the channels dealt to eight warps; the row is
// read twice, the sum t recomputed (so t may overwrite x or r in place).
__global__ void __launch_bounds__(RMS_THREADS) rms_any_kernel(const __grid_constant__ RmsProblem p) {
    griddep_launch_dependents();
    __shared__ float2 part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_wait();
    for (long long row0 = (long long)blockIdx.x * 32; row0 < p.rows; row0 += (long long)gridDim.x * 32) {
        const long long row = row0 + lane;
        const bool on = row < p.rows;
        const long long xo = on ? row_off(p.x.m, row) : 0, ro = on && p.r.p ? row_off(p.r.m, row) : 0;
        float sq = 0.f, mx = 0.f;
        for (int c = warp; on && c < p.C; c += 8) {
            float v = load_elem(p.x.p, p.x.dt, xo + c * p.x.m.cs);
            if (p.r.p) v += load_elem(p.r.p, p.r.dt, ro + c * p.r.m.cs);
            sq = fmaf(v, v, sq);
            mx = fmaxf(mx, fabsf(v * __ldg(p.gamma + c)));
        }
        part[warp][lane] = make_float2(sq, mx);
        __syncthreads();
        sq = 0.f, mx = 0.f;
        for (int i = 0; i < 8; ++i) {
            sq += part[i][lane].x;
            mx = fmaxf(mx, part[i][lane].y);
        }
        __syncthreads();
        if (!on) continue;
        float f = rsqrtf(sq / (float)p.C + p.eps);
        if (p.y.dt == DLC_DATA_FLOAT8_E4M3) {
            const float s = e4m3_scale(mx * f);
            if (warp == 0) p.scale[row] = s;
            f = f / s;
        }
        const long long to = p.t.p ? row_off(p.t.m, row) : 0, yo = row_off(p.y.m, row);
        for (int c = warp; c < p.C; c += 8) {
            float v = load_elem(p.x.p, p.x.dt, xo + c * p.x.m.cs);
            if (p.r.p) v += load_elem(p.r.p, p.r.dt, ro + c * p.r.m.cs);
            if (p.t.p) store_elem(p.t.p, p.t.dt, to + c * p.t.m.cs, v);
            store_elem(p.y.p, p.y.dt, yo + c * p.y.m.cs, v * __ldg(p.gamma + c) * f);
        }
    }
}

// Backward, rows in registers.  Each thread adds up dgamma of its own channels
// over the rows it visits; a block writes one partial row of sums.
template <int W, int V>
__global__ void __launch_bounds__(1024) rms_bwd_rows_kernel(const __grid_constant__ RmsBwdProblem p, int tpr) {
    griddep_launch_dependents();
    __shared__ float2 buf[2][RMS_MAX_WARPS];
    extern __shared__ float acc_s[];  // [rows per block][C], to join the block's row slots
    const int rpb = (int)blockDim.x / tpr, slot = (int)threadIdx.x / tpr, t = (int)threadIdx.x % tpr;
    griddep_wait();
    float acc[V][W];
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < W; ++i) acc[j][i] = 0.f;
    int parity = 0;
    for (long long row0 = (long long)blockIdx.x * rpb; row0 < p.rows; row0 += (long long)gridDim.x * rpb, parity ^= 1) {
        const long long row = row0 + slot;
        const bool on = row < p.rows;
        const long long yo = on ? row_off(p.dy.m, row) : 0, to = on ? row_off(p.t.m, row) : 0;
        float d[V][W], v[V][W];
        float sq = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (t + j * tpr) * W, n = on ? p.C - c : 0;
            load_vec<W>(p.dy, yo + c, n, d[j]);
            load_vec<W>(p.t, to + c, n, v[j]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float g[W];
            load_gamma<W>(p.gamma, (t + j * tpr) * W, p.C, g);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                sq = fmaf(v[j][i], v[j][i], sq);
                dot = fmaf(d[j][i] * g[i], v[j][i], dot);
            }
        }
        const float2 red = row_reduce<false>(sq, dot, tpr, buf, parity);
        if (!on) continue;
        const float rho = rsqrtf(red.x / (float)p.C + p.eps);
        const float k = rho * rho * rho * (red.y / (float)p.C);
        const long long xo = row_off(p.dx.m, row), so = p.dt.p ? row_off(p.dt.m, row) : 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (t + j * tpr) * W, n = p.C - c;
            float g[W], s[W];
            load_gamma<W>(p.gamma, c, p.C, g);
#pragma unroll
            for (int i = 0; i < W; ++i) s[i] = 0.f;
            if (p.dt.p) load_vec<W>(p.dt, so + c, n, s);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                acc[j][i] = fmaf(d[j][i] * rho, v[j][i], acc[j][i]);
                s[i] += rho * d[j][i] * g[i] - v[j][i] * k;
            }
            store_vec<W>(p.dx, xo + c, n, s);
        }
    }
    if (!p.dgamma) return;
    if (rpb > 1) {
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const int c = (t + j * tpr) * W + i;
                if (c < p.C) acc_s[(long long)slot * p.C + c] = acc[j][i];
            }
        __syncthreads();
        for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
            float s = 0.f;
            for (int i = 0; i < rpb; ++i) s += acc_s[(long long)i * p.C + c];
            p.ws[(long long)blockIdx.x * p.C + c] = s;
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const int c = (t + j * tpr) * W + i;
                if (c < p.C) p.ws[(long long)blockIdx.x * p.C + c] = acc[j][i];
            }
    }
}

// Backward for the remaining layouts: one row a lane as above.  A block's
// dgamma is summed over its rows by warp shuffles, one channel at a time, into
// its row of partial sums (only its own warp touches a channel).
__global__ void __launch_bounds__(RMS_THREADS) rms_bwd_any_kernel(const __grid_constant__ RmsBwdProblem p) {
    griddep_launch_dependents();
    __shared__ float2 part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_wait();
    bool first = true;
    for (long long row0 = (long long)blockIdx.x * 32; row0 < p.rows; row0 += (long long)gridDim.x * 32) {
        const long long row = row0 + lane;
        const bool on = row < p.rows;
        const long long yo = on ? row_off(p.dy.m, row) : 0, to = on ? row_off(p.t.m, row) : 0;
        float sq = 0.f, dot = 0.f;
        for (int c = warp; on && c < p.C; c += 8) {
            const float v = load_elem(p.t.p, p.t.dt, to + c * p.t.m.cs);
            const float d = load_elem(p.dy.p, p.dy.dt, yo + c * p.dy.m.cs) * __ldg(p.gamma + c);
            sq = fmaf(v, v, sq);
            dot = fmaf(d, v, dot);
        }
        part[warp][lane] = make_float2(sq, dot);
        __syncthreads();
        sq = 0.f, dot = 0.f;
        for (int i = 0; i < 8; ++i) {
            sq += part[i][lane].x;
            dot += part[i][lane].y;
        }
        __syncthreads();
        const float rho = on ? rsqrtf(sq / (float)p.C + p.eps) : 0.f;
        const float k = rho * rho * rho * (dot / (float)p.C);
        const long long xo = on ? row_off(p.dx.m, row) : 0, so = on && p.dt.p ? row_off(p.dt.m, row) : 0;
        for (int c = warp; c < p.C; c += 8) {
            float a = 0.f;
            if (on) {
                const float v = load_elem(p.t.p, p.t.dt, to + c * p.t.m.cs);
                const float d = load_elem(p.dy.p, p.dy.dt, yo + c * p.dy.m.cs);
                a = d * rho * v;
                float s = p.dt.p ? load_elem(p.dt.p, p.dt.dt, so + c * p.dt.m.cs) : 0.f;
                s += rho * d * __ldg(p.gamma + c) - v * k;
                store_elem(p.dx.p, p.dx.dt, xo + c * p.dx.m.cs, s);
            }
            if (p.dgamma) {
                for (int o = 16; o > 0; o /= 2) a += __shfl_xor_sync(0xffffffffu, a, o);
                if (lane == 0) {
                    float *w = p.ws + (long long)blockIdx.x * p.C + c;
                    *w = first ? a : *w + a;
                }
            }
        }
        first = false;
    }
}

// out[c] = the sum of the blocks' partial rows, in a fixed order.
__global__ void __launch_bounds__(256) column_sum_kernel(const float *ws, float *out, int C, int blocks) {
    griddep_launch_dependents();
    __shared__ float part[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (int)blockIdx.x * 32 + lane;
    griddep_wait();
    float s = 0.f;
    if (c < C)
        for (int b = warp; b < blocks; b += 8) s += ws[(long long)b * C + c];
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < C) {
        for (int i = 1; i < 8; ++i) s += part[i][lane];
        out[c] = s;
    }
}

// ---- host side ---------------------------------------------------------------

struct RowPlan {
    int w = 0, v = 0;  // channels per vector (0: the any-layout kernel), vectors per thread
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

RowPlan plan_rows(long long rows, int C, bool cs1, bool vec, int v_max, int sm_count) {
    RowPlan r;
    r.threads = RMS_THREADS;
    if (cs1) {
        r.w = vec ? 8 : 1;
        const long long nv = (C + r.w - 1) / r.w;
        // vectors a thread: few for short rows (more threads a row), v_max at most
        int v = 1, tpr = 8;
        while (tpr < 32 && tpr * v < nv) tpr *= 2;
        while (v < v_max && tpr * v < nv && tpr == 32) v *= 2;
        while (tpr < 1024 && (long long)tpr * v < nv) tpr *= 2;
        if ((long long)tpr * v < nv) r.w = 0;
        r.v = v;
        r.tpr = tpr;
        if (r.w && tpr > RMS_THREADS) r.threads = tpr;
    }
    const int rpb = r.w ? r.threads / r.tpr : 32;
    const long long need = (rows + rpb - 1) / rpb;
    const long long most = (long long)sm_count * (2048 / r.threads);
    r.blocks = need < most ? need : most;
    return r;
}

RowPlan plan_fwd(const dlcContext *ctx, const RmsProblem &p) {
    return plan_rows(p.rows, p.C, contiguous(p.x) && contiguous(p.r) && contiguous(p.t) && contiguous(p.y),
                     vec_ok(p.x) && vec_ok(p.r) && vec_ok(p.t) && vec_ok(p.y), 4, ctx->sm_count);
}

RowPlan plan_bwd(const dlcContext *ctx, const RmsBwdProblem &p) {
    return plan_rows(p.rows, p.C, contiguous(p.dy) && contiguous(p.t) && contiguous(p.dt) && contiguous(p.dx),
                     vec_ok(p.dy) && vec_ok(p.t) && vec_ok(p.dt) && vec_ok(p.dx), 2, ctx->sm_count);
}

const void *fwd_kernel(const RowPlan &r) {
    if (!r.w) return (const void *)rms_any_kernel;
    if (r.w == 8)
        return r.v == 1 ? (const void *)rms_rows_kernel<8, 1>
                        : r.v == 2 ? (const void *)rms_rows_kernel<8, 2> : (const void *)rms_rows_kernel<8, 4>;
    return r.v == 1 ? (const void *)rms_rows_kernel<1, 1>
                    : r.v == 2 ? (const void *)rms_rows_kernel<1, 2> : (const void *)rms_rows_kernel<1, 4>;
}

const void *bwd_kernel(const RowPlan &r) {
    if (!r.w) return (const void *)rms_bwd_any_kernel;
    if (r.w == 8) return r.v == 1 ? (const void *)rms_bwd_rows_kernel<8, 1> : (const void *)rms_bwd_rows_kernel<8, 2>;
    return r.v == 1 ? (const void *)rms_bwd_rows_kernel<1, 1> : (const void *)rms_bwd_rows_kernel<1, 2>;
}

}  // namespace

dlcStatus_t dlc_launch_rms(dlcContext *ctx, const RmsProblem &pb) {
    const RowPlan r = plan_fwd(ctx, pb);
    RmsProblem p = pb;
    int tpr = r.tpr;
    void *args[] = {&p, &tpr};
    return dlc_launch(ctx, fwd_kernel(r), dim3((unsigned)r.blocks), dim3((unsigned)r.threads), 0, args);
}

size_t dlc_rms_bwd_workspace(const dlcContext *ctx, const RmsBwdProblem &p) {
    // the most blocks of any layout's plan, so that the pointers' alignment does not matter
    const long long most = (long long)ctx->sm_count * (2048 / RMS_THREADS);
    const long long blocks = p.rows < most ? p.rows : most;
    return (size_t)blocks * p.C * sizeof(float);
}

dlcStatus_t dlc_launch_rms_bwd(dlcContext *ctx, const RmsBwdProblem &pb) {
    const RowPlan r = plan_bwd(ctx, pb);
    RmsBwdProblem p = pb;
    int tpr = r.tpr;
    void *args[] = {&p, &tpr};
    const int rpb = r.w ? r.threads / r.tpr : 1;
    const size_t smem = rpb > 1 && p.dgamma ? (size_t)rpb * p.C * sizeof(float) : 0;
    dlcStatus_t st = dlc_launch(ctx, bwd_kernel(r), dim3((unsigned)r.blocks), dim3((unsigned)r.threads), smem, args);
    if (st != DLC_STATUS_SUCCESS || !p.dgamma) return st;
    return dlc_launch_column_sum(ctx, p.ws, p.dgamma, p.C, (int)r.blocks);
}

dlcStatus_t dlc_launch_column_sum(dlcContext *ctx, const float *ws, float *out, int C, int blocks) {
    void *args[] = {&ws, &out, &C, &blocks};
    return dlc_launch(ctx, (const void *)column_sum_kernel, dim3((unsigned)((C + 31) / 32)), dim3(256), 0, args);
}

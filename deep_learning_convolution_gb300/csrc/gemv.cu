// gemv.cu -- the products of the linear and gated layers for one to four rows
// (a decoding step of a few sequences), on the CUDA cores.
//
// Every filter element is used once per row, so the filters' bytes are the
// time, and a launch of this size is worth as little set-up as possible: a warp
// takes four or eight filters (of a gated layer: half as many outputs' gate and up
// filters) along the reduction, each lane 16-byte vectors of filters and rows
// straight from memory, products and sums in FP32.  With few filters the
// warps of a block share them, each a range of the reduction; the partial sums
// meet in shared memory in a fixed order.  Filters or rows that are not on
// 16-byte boundaries are read element by element, in place.
//
// Measured back to back, BF16: 1 x 2048 -> 2 x 8192 gated 12.6 us (67 MB of
// filters, 5.3 TB/s), 4096 -> 1000 3.0 us for one row and 4.1 for four.
#include "channel.cuh"
#include "gemm.h"
#include "ptx.cuh"

namespace {

using namespace dlc;

constexpr int GV_WARPS = 8;

// Filters of a warp.  E4M3 rows are half as long: twice the filters, so that the
// end of a group (joining the lanes, the epilogue) comes as rarely per byte.
template <bool E4M3, int M>
constexpr int gv_filters() { return E4M3 && M == 1 ? 8 : 4; }
// Blocks an SM holds and steps of the ring (16 KiB of filters a step and block).
// E4M3 takes more instructions a byte, so more warps.
template <bool E4M3>
constexpr int gv_blocks() { return 2; }
template <bool E4M3>
constexpr int gv_ring() { return E4M3 ? 3 : 6; }

struct GvParams {
    int N, act;
    long long K;
    RowTensor x, z, r, y;
    const void *w;
    const float *sa, *sb, *bias;
    int ranges;        // warps of a block that share filters
    int groups;        // of gv_filters() filters
};

// One 16-byte vector as pairs of 16-bit values: 8 BF16 as they are, 16 E4M3 as
// FP16 (which holds every E4M3 value exactly).
template <bool E4M3>
struct GvVector {
    uint32_t h[E4M3 ? 8 : 4];
    __device__ __forceinline__ void set(const uint4 &q) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (E4M3) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i] >> (16 * j)), __NV_E4M3);
                    h[2 * i + j] = (uint32_t)r.x | ((uint32_t)r.y << 16);
                }
            } else {
                h[i] = w[i];
            }
        }
    }
};

// c + a . b over a pair, the products and sums in FP32 (operands read as the
// 16-bit values they are: no unpacking).
template <bool E4M3>
__device__ __forceinline__ float gv_fma(uint32_t a, uint32_t b, float c) {
    if constexpr (E4M3)
        asm("{\n\t.reg .b16 a0, a1, b0, b1;\n\tmov.b32 {a0, a1}, %1;\n\tmov.b32 {b0, b1}, %2;\n\t"
            "fma.rn.f32.f16 %0, a0, b0, %0;\n\tfma.rn.f32.f16 %0, a1, b1, %0;\n\t}\n"
            : "+f"(c)
            : "r"(a), "r"(b));
    else
        asm("{\n\t.reg .b16 a0, a1, b0, b1;\n\tmov.b32 {a0, a1}, %1;\n\tmov.b32 {b0, b1}, %2;\n\t"
            "fma.rn.f32.bf16 %0, a0, b0, %0;\n\tfma.rn.f32.bf16 %0, a1, b1, %0;\n\t}\n"
            : "+f"(c)
            : "r"(a), "r"(b));
    return c;
}

// Where a warp's filters start: row f of group `group` (the last filter again past the end).
template <bool GATED, int F>
__device__ __forceinline__ long long gv_row(const GvParams &p, int group, int f) {
    constexpr int OUT = GATED ? F / 2 : F;
    const int n = min(group * OUT + (GATED ? f % OUT : f), p.N - 1);
    return ((GATED && f >= OUT ? (long long)p.N : 0) + n) * p.K;
}

// Sums each of V values (a power of two, at most 32) over the warp: while more
// than one is left, a lane hands half of them to its partner and keeps the
// other half.  Returns the sum of value lane / (32 / V).
template <int V>
__device__ __forceinline__ float gv_reduce(float (&v)[V]) {
    const int lane = threadIdx.x & 31;
    int o = 16;
#pragma unroll
    for (int n = V / 2; n > 0; n /= 2, o /= 2) {
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    float s = v[0];
#pragma unroll
    for (; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// Joins a group's sums over the lanes and the ranges, and applies the epilogue.
template <bool GATED, int F, int M>
__device__ __forceinline__ void gv_finish(const GvParams &p, int group, int range, const float (&acc)[F][M],
                                          float (*part)[32]) {
    constexpr int OUT = GATED ? F / 2 : F;  // outputs of a warp
    constexpr int V = F * M <= 4 ? 4 : F * M <= 8 ? 8 : 16;
    static_assert(F * M <= 16, "a warp reduces sixteen sums at most");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = i < F * M ? acc[i / M][i % M] : 0.f;
    __syncwarp();
    const float s = gv_reduce<V>(v);
    if (lane % (32 / V) == 0) part[warp][lane / (32 / V)] = s;
    if (p.ranges > 1)
        __syncthreads();
    else
        __syncwarp();
    const int o = lane / M, m = lane - o * M, n = group * OUT + o;
    if (range != 0 || group >= p.groups || lane >= OUT * M || n >= p.N) return;
    const float sa = p.sa ? p.sa[m] : 1.f;
    float z[GATED ? 2 : 1];
#pragma unroll
    for (int h = 0; h < (GATED ? 2 : 1); ++h) {
        float t = 0.f;
        for (int i = 0; i < p.ranges; ++i) t += part[warp + i][(h * OUT + o) * M + m];
        const long long k = (long long)h * p.N + n;
        if (p.sb) t *= sa * p.sb[k];
        if (p.bias) t += p.bias[k];
        z[h] = t;
        if (p.z.p) store_elem(p.z.p, p.z.dt, row_off(p.z.m, m) + k * p.z.m.cs, t);
    }
    float y = z[0];
    act_dispatch(p.act, [&](auto act) { y = act_f<decltype(act)::value>(y); });
    if (GATED) y *= z[GATED];
    if (p.r.p) y += load_elem(p.r.p, p.r.dt, row_off(p.r.m, m) + n * p.r.m.cs);
    store_elem(p.y.p, p.y.dt, row_off(p.y.m, m) + n * p.y.m.cs, y);
}

// Vectors.  A lane's next vectors of its filters come asynchronously into a ring
// of its own in shared memory, across the end of one group into the next.
template <bool E4M3, bool GATED, int M>
__global__ void __launch_bounds__(GV_WARPS * 32, gv_blocks<E4M3>()) gemv_kernel(const __grid_constant__ GvParams p) {
    constexpr int F = gv_filters<E4M3, M>(), E = E4M3 ? 16 : 8, P = E / 2;  // elements and pairs of a vector
    constexpr int GV_RING = gv_ring<E4M3>();
    griddep_launch_dependents();
    extern __shared__ uint4 ring_s[];
    __shared__ float part[GV_WARPS][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_block = GV_WARPS / p.ranges, range = warp % p.ranges;
    const int stride = (int)gridDim.x * per_block;  // with several ranges the grid covers all groups at once
    const int vecs = (int)(p.K / E), step = p.ranges * 32, first = range * 32 + lane;
    const uint4 *w = static_cast<const uint4 *>(p.w), *x = static_cast<const uint4 *>(p.x.p);
    const uint32_t slot = smem_u32(ring_s) + threadIdx.x * 16u, vec = 16u * blockDim.x;
    int group = (int)blockIdx.x * per_block + warp / p.ranges;
    griddep_wait();
    long long xo[M];
#pragma unroll
    for (int m = 0; m < M; ++m) xo[m] = row_off(p.x.m, m) / E;
    // every lane of a warp takes the same number of steps (the last may be idle)
    const int steps = (vecs + step - 1) / step;
    int next_group = group, next_step = 0;
    uint32_t put = 0, get = 0;
    const uint4 *from[F];
    auto aim = [&]() {
#pragma unroll
        for (int f = 0; f < F; ++f) from[f] = w + gv_row<GATED, F>(p, next_group, f) / E;
    };
    auto fetch = [&]() {
        if (next_group < p.groups) {
            const int k = first + next_step * step;
            if (k < vecs) {
#pragma unroll
                for (int f = 0; f < F; ++f) cp_async_16(slot + (put * F + (uint32_t)f) * vec, from[f] + k, 16u);
            }
            if (++next_step == steps) {
                next_step = 0;
                next_group += stride;
                if (next_group < p.groups) aim();
            }
        }
        cp_async_commit();
        put = put == GV_RING - 1 ? 0 : put + 1;
    };
    if (group < p.groups) aim();
#pragma unroll
    for (int i = 0; i < GV_RING - 1; ++i) fetch();
    do {
        float acc[F][M];
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
            for (int m = 0; m < M; ++m) acc[f][m] = 0.f;
        if (group < p.groups) {
            uint4 qx[M];
#pragma unroll
            for (int m = 0; m < M; ++m)
                if (first < vecs) qx[m] = x[xo[m] + first];
            for (int k = first; k - first < steps * step; k += step) {
                const bool in = k < vecs;
                GvVector<E4M3> xv[M];
#pragma unroll
                for (int m = 0; m < M; ++m) xv[m].set(qx[m]);
#pragma unroll
                for (int m = 0; m < M; ++m)  // one step ahead
                    if (k + step < vecs) qx[m] = x[xo[m] + k + step];
                cp_async_wait<GV_RING - 2>();
                uint4 qw[F];
#pragma unroll
                for (int f = 0; f < F; ++f)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(qw[f].x), "=r"(qw[f].y), "=r"(qw[f].z), "=r"(qw[f].w)
                                 : "r"(slot + (get * F + (uint32_t)f) * vec)
                                 : "memory");
                get = get == GV_RING - 1 ? 0 : get + 1;
                fetch();
                if (!in) continue;
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    GvVector<E4M3> wv;
                    wv.set(qw[f]);
#pragma unroll
                    for (int i = 0; i < P; ++i)
#pragma unroll
                        for (int m = 0; m < M; ++m) acc[f][m] = gv_fma<E4M3>(wv.h[i], xv[m].h[i], acc[f][m]);
                }
            }
        }
        gv_finish<GATED, F, M>(p, group, range, acc, part);
        group += stride;
    } while (group < p.groups);
    cp_async_wait<0>();
}

// Elements, at any stride and alignment.
template <bool E4M3, bool GATED, int M>
__global__ void __launch_bounds__(GV_WARPS * 32) gemv_elements_kernel(const __grid_constant__ GvParams p) {
    // elements of a filter in flight (one row of 4003 -> 4004: with 12 24.9 us in BF16
    // and 15.0 in E4M3, with 8 27.6 and 24.9)
    constexpr int F = 4, B = M == 1 ? 12 : 8;
    using T = typename std::conditional<E4M3, unsigned char, unsigned short>::type;
    griddep_launch_dependents();
    __shared__ float part[GV_WARPS][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_block = GV_WARPS / p.ranges, range = warp % p.ranges;
    const int group = (int)blockIdx.x * per_block + warp / p.ranges;
    griddep_wait();
    float acc[F][M];
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int m = 0; m < M; ++m) acc[f][m] = 0.f;
    if (group < p.groups) {
        long long row[F], xo[M];
#pragma unroll
        for (int f = 0; f < F; ++f) row[f] = gv_row<GATED, F>(p, group, f);
#pragma unroll
        for (int m = 0; m < M; ++m) xo[m] = row_off(p.x.m, m);
        const T *w = static_cast<const T *>(p.w), *x = static_cast<const T *>(p.x.p);
        auto value = [](T b) {
            if constexpr (E4M3) {
                __nv_fp8_e4m3 v;
                v.__x = b;
                return float(v);
            } else {
                return bf16_bits_f32(b);
            }
        };
        for (long long k = range * 32 + lane; k < p.K; k += (long long)B * p.ranges * 32) {
            T ew[F][B], ex[M][B];
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const long long at = k + (long long)i * p.ranges * 32;
                const bool in = at < p.K;
#pragma unroll
                for (int f = 0; f < F; ++f) ew[f][i] = in ? w[row[f] + at] : (T)0;
#pragma unroll
                for (int m = 0; m < M; ++m) ex[m][i] = in ? x[xo[m] + at * p.x.m.cs] : (T)0;
            }
#pragma unroll
            for (int i = 0; i < B; ++i)
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const float xv = value(ex[m][i]);
#pragma unroll
                    for (int f = 0; f < F; ++f) acc[f][m] = fmaf(value(ew[f][i]), xv, acc[f][m]);
                }
        }
    }
    gv_finish<GATED, F, M>(p, group, range, acc, part);
}

template <bool E4M3, bool GATED>
const void *gv_kernel(long long M, bool vec) {
    if (!vec) return M == 1 ? (const void *)gemv_elements_kernel<E4M3, GATED, 1> : (const void *)gemv_elements_kernel<E4M3, GATED, 2>;
    if (M == 1) return (const void *)gemv_kernel<E4M3, GATED, 1>;
    if (E4M3 || M == 2) return (const void *)gemv_kernel<E4M3, GATED, 2>;
    return M == 3 ? (const void *)gemv_kernel<false, GATED, 3> : (const void *)gemv_kernel<false, GATED, 4>;
}

bool gv_vec(const GemmProblem &g) {
    const long long e = dlc_dtype_bytes((dlcDataType_t)g.a.t.dt);
    auto mult = [&](long long s) { return (s * e) % 16 == 0; };
    const RowMap &x = g.a.t.m;
    return mult(g.K) && (uintptr_t)g.b.t.p % 16 == 0 && (uintptr_t)g.a.t.p % 16 == 0 && x.cs == 1 &&
           (g.M == 1 || (x.uniform ? mult(x.ld) : (mult(x.s0) && mult(x.s2) && mult(x.s3))));
}

}  // namespace

// Whether this is the faster way.  Measured back to back: the few-row kernel
// takes 4.8 us and the filters' bytes at 6.9 (E4M3: 7.6) MB/us whatever the rows;
// this one 2.4 us and, in BF16, 6.5, 5.7, 5.2 and 4.7 MB/us for one to four rows
// (2048 -> 2 x 8192), in E4M3 4.3 and 3.1 MB/us for one and two.  Filters that it
// has to read element by element run at 1.2 MB/us: faster than packing them
// first for one or two rows (4003 -> 4004, two rows: 21.9 us against 35).
bool dlc_gemv_ok(const GemmProblem &g) {
    if (g.a.trans || g.b.trans || (g.N > 1 && g.b.t.m.ld != g.K)) return false;  // (padded rows: copies)
    if (!gv_vec(g)) return g.M <= 2;
    const bool e4m3 = g.a.t.dt == DLC_DATA_FLOAT8_E4M3;
    if (g.M > (e4m3 ? 2 : 4)) return false;
    const double bytes = (double)(g.gated ? 2 : 1) * g.N * g.K * (e4m3 ? 1 : 2), m = (double)g.M;
    return e4m3 ? 2.4 + bytes * (1.0 + 0.5 * m) / 6.4e6 < 4.8 + bytes / 7.6e6
                : 2.4 + bytes * (1.0 + 0.14 * m) / 7.45e6 < 4.8 + bytes / 6.9e6;
}

dlcStatus_t dlc_launch_gemv(dlcContext *ctx, const GemmProblem &g) {
    const bool e4m3 = g.a.t.dt == DLC_DATA_FLOAT8_E4M3;
    GvParams p;
    p.N = g.N;
    p.act = g.act;
    p.K = g.K;
    p.x = g.a.t;
    p.z = g.z;
    p.r = g.r;
    p.y = g.y;
    p.w = g.b.t.p;
    p.sa = g.sa;
    p.sb = g.sb;
    p.bias = g.bias;
    const bool vec = gv_vec(g);
    const int filters = vec && e4m3 && g.M == 1 ? gv_filters<true, 1>() : 4, out = g.gated ? filters / 2 : filters;
    p.groups = (g.N + out - 1) / out;
    // more warps a group while half the resident ones have none and each range
    // keeps two vectors a lane
    const int e = e4m3 ? 1 : 2, blocks_sm = e4m3 ? gv_blocks<true>() : gv_blocks<false>();
    p.ranges = 1;
    while (p.ranges < GV_WARPS && 2LL * p.groups * p.ranges <= (long long)ctx->sm_count * blocks_sm * GV_WARPS &&
           g.K * e >= (long long)p.ranges * 2 * 2 * 32 * 16)
        p.ranges *= 2;
    const int per_block = GV_WARPS / p.ranges;
    void *args[] = {&p};
    const void *kern = e4m3 ? (g.gated ? gv_kernel<true, true>(g.M, vec) : gv_kernel<true, false>(g.M, vec))
                            : (g.gated ? gv_kernel<false, true>(g.M, vec) : gv_kernel<false, false>(g.M, vec));
    const size_t smem = vec ? (size_t)(e4m3 ? gv_ring<true>() : gv_ring<false>()) * filters * 16 * GV_WARPS * 32 : 0;
    if (!dlc_allow_smem(ctx, kern, smem)) return DLC_STATUS_EXECUTION_FAILED;
    int blocks = (p.groups + per_block - 1) / per_block;
    if (vec && p.ranges == 1) blocks = std::min(blocks, blocks_sm * ctx->sm_count);
    return dlc_launch(ctx, kern, dim3((unsigned)blocks), dim3(GV_WARPS * 32), smem, args);
}

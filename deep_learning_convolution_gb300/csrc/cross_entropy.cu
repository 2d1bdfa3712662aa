// cross_entropy.cu -- softmax cross entropy on top of a linear layer, in pieces of the
// classes (a vocabulary), so that the logits are never kept:
//
//   z[m, k] = sa[m] sb[k] sum_c x[m, c] w[k, c] + bias[k]
//   lse[m] = log sum_k exp z[m, k];  loss[m] = lse[m] - z[m, target[m]]
//   dz[m, k] = dloss[m] (exp(z[m, k] - lse[m]) - [k = target[m]])
//   dx = dz w;  dw = dz^T x;  dbias = sum_m dz        (rows without a target: 0)
//
// A row's part is kept as its largest logit t and s = sum exp(z - t); two parts are joined at the larger
// t.  loss = (t - z[target]) + log s, whose difference is exact where lse - z[target] would lose
// the digits that lse has not.
//
// Forward is one product whose epilogue leaves, for each row and 128 classes, (t, s) of its accumulators
// (gp_entropy in gemm.cu), and a kernel that joins them.  Backward works the logits out again
// in pieces of the classes, whose epilogue writes dz, and runs the two products of a linear layer's gradient on
// each piece; dx adds up in FP32.  That is 8 M V K operations for the step instead of the 6 M V K that keeping the
// logits would take.  The tensor core under the power cap bounds it: 4096 x 2048 -> 131072 1.10 ms forward (2000
// TFLOP/s) and 3.8 ms backward (1720; cuBLAS in a loop: 1725); E4M3 forward 0.57 ms (3855).  Few rows keep FP32
// logits of a piece in memory instead (fuse_fwd): 32 x 4096 -> 131072 171 us, 6.3 TB/s of filters, E4M3 102 us
// (5.3).
//
// dz enters the two products in BF16, as their other operands do: the tensor core takes both of a product's in one
// type.  One term of it, rounded once, leaves dx and dw up to 0.0017 off in norm beside FP64 whatever type they are
// kept in, more where a few rows or classes are most of it; BF16 outputs are 0.0017 off by themselves, and a
// training step's come to 0.0024.  A second term, what the rounding left, keeps 16 bits and costs the products
// twice their operations; it is taken where that is little of a call (terms_of), and is not for long products that
// the tensor core bounds (4096 x 2048 -> 131072 4.9 ms a step, some 7.2 with it).  dbias sums the values before any
// rounding.
//
// Workspace: a piece's dz takes 512 MB, but never less than 256 classes do (above 2^20 rows 512 bytes a row), and its column
// sums a 16th of that; the forward call's parts 256 MB, but never less than 1024 classes do (up to 32 of them: 256 bytes
// a row); few rows' logits 512 MB.  Beside them the FP32 sum of a BF16 dx in several pieces, and copies of operands that
// TMA cannot load.
#include <cmath>

#include "channel.cuh"
#include "gemm.h"
#include "ptx.cuh"

namespace {

using namespace dlc;

constexpr float LOG2E = 1.4426950408889634f;
constexpr int CE_THREADS = 256;
constexpr int CE_SEGMENT = 4096;  // logits of a row that a block sums up

// A part of a row's sum: exp(t) * s.  t = -inf: nothing (or only -inf) so far.
struct CePart {
    float t, s;
};

__device__ __forceinline__ CePart ce_join(CePart a, CePart b) {
    const float t = fmaxf(a.t, b.t), base = isinf(t) ? 0.f : t;
    return {t, a.s * exp2_fast((a.t - base) * LOG2E) + b.s * exp2_fast((b.t - base) * LOG2E)};
}

__device__ __forceinline__ CePart ce_join_lanes(CePart a) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) a = ce_join(a, CePart{__shfl_xor_sync(0xffffffffu, a.t, o), __shfl_xor_sync(0xffffffffu, a.s, o)});
    return a;
}

__device__ __forceinline__ long long ce_target(const IndexList &t, long long i) {
    return t.wide ? static_cast<const long long *>(t.p)[i] : static_cast<const int *>(t.p)[i];
}

// ---- logits of a piece in memory (FP32) ---------------------------------------------

struct CeParams {
    long long M;
    int V, n0, cols;           // classes in all; of this piece: the first one and how many
    const float *z;            // [M][ld]
    long long ld;
    IndexList target;
    float2 *part;              // [part][M] (t, s)
    int part0, parts;          // first part of this piece; how many there are when they are joined
    int last;                  // the rows' sums are complete, else part 0 takes what they are so far
    float *chosen;             // [M] the target's logit
    float *loss, *lse;
    const float *dloss;
    unsigned short *dz;        // [terms][M][ldz]
    long long ldz;
    int terms;
    float *sums;               // [strip][cols] or null
    int *err;
};

// A row's loss and log-sum-exp, its sum being complete.
__device__ __forceinline__ void ce_finish(const CeParams &p, long long m, CePart a, float chosen) {
    const float log_s = logf(a.s), lse = isinf(a.t) ? log_s : a.t + log_s;  // (t = +-inf: s = inf or 0)
    const long long k = ce_target(p.target, m);
    float loss = 0.f;
    if (k >= p.V) {
        record_error(p.err, DLC_DEVERR_INDEX, (int)m);
        loss = NAN;
    } else if (k >= 0) {
        loss = (a.t - chosen) + log_s;
    }
    p.lse[m] = lse;
    p.loss[m] = loss;
}

// The sum of one segment of a row of logits; of all of them, where one segment holds them.
__global__ void __launch_bounds__(CE_THREADS) ce_part_kernel(const __grid_constant__ CeParams p) {
    griddep_launch_dependents();
    __shared__ CePart warps[CE_THREADS / 32];
    constexpr int E = CE_SEGMENT / CE_THREADS;
    const int c0 = (int)blockIdx.y * CE_SEGMENT + 4 * (int)threadIdx.x;
    griddep_wait();
    const long long m = blockIdx.x;
    const float *z = p.z + m * p.ld;
    float v[E];
#pragma unroll
    for (int j = 0; j < E / 4; ++j) {
        const int c = c0 + 4 * CE_THREADS * j;
        float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (c + 4 <= p.cols) {
            q = *reinterpret_cast<const float4 *>(z + c);
        } else if (c < p.cols) {
            q.x = z[c];
            if (c + 1 < p.cols) q.y = z[c + 1];
            if (c + 2 < p.cols) q.z = z[c + 2];
        }
        v[4 * j] = q.x, v[4 * j + 1] = q.y, v[4 * j + 2] = q.z, v[4 * j + 3] = q.w;
    }
    float top = -INFINITY, s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) top = fmaxf(top, v[i]);
    const float base = isinf(top) ? 0.f : top;
#pragma unroll
    for (int i = 0; i < E; ++i) s += exp2_fast((v[i] - base) * LOG2E);
    const CePart a = ce_join_lanes(CePart{top, s});
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
        CePart t = warps[0];
        for (int i = 1; i < CE_THREADS / 32; ++i) t = ce_join(t, warps[i]);
        const long long k = ce_target(p.target, m) - p.n0;
        if (p.parts == 1) {
            ce_finish(p, m, t, k >= 0 && k < p.cols ? z[k] : 0.f);
        } else {
            p.part[(long long)(p.part0 + (int)blockIdx.y) * p.M + m] = make_float2(t.t, t.s);
            if (blockIdx.y == 0 && k >= 0 && k < p.cols) p.chosen[m] = z[k];
        }
    }
}

// Joins the parts of 32 rows a block, in a fixed order: a lane a row, the parts dealt to the warps.
// (Parts of many rows and classes would take a 32nd of what BF16 logits take: several pieces then
// share the workspace, each adding to part 0.)
__global__ void __launch_bounds__(1024) ce_loss_kernel(const __grid_constant__ CeParams p) {
    griddep_launch_dependents();
    __shared__ CePart warps[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long m = (long long)blockIdx.x * 32 + lane;
    griddep_wait();
    CePart a{-INFINITY, 0.f};
    if (m < p.M) {
#pragma unroll 4
        for (int i = warp; i < p.parts; i += 32) {
            const float2 q = p.part[(long long)i * p.M + m];
            a = ce_join(a, CePart{q.x, q.y});
        }
    }
    warps[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && m < p.M) {
        for (int i = 1; i < 32; ++i) a = ce_join(a, warps[i][lane]);
        if (p.last)
            ce_finish(p, m, a, p.chosen[m]);
        else
            p.part[m] = make_float2(a.t, a.s);
    }
}

// dz of a piece, four classes a thread, and its sums over a strip of rows.
__global__ void __launch_bounds__(CE_THREADS) ce_dz_kernel(const __grid_constant__ CeParams p) {
    griddep_launch_dependents();
    const int c = 4 * ((int)blockIdx.x * CE_THREADS + (int)threadIdx.x);
    griddep_wait();
    if (c >= p.cols) return;
    const int n = min(4, p.cols - c);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    const long long step = gridDim.y;
#pragma unroll 2
    for (long long m = blockIdx.y; m < p.M; m += step) {
        const float lse = p.lse[m];
        const long long t = ce_target(p.target, m);
        const bool counted = t >= 0 && t < p.V;
        const float d = counted ? p.dloss[m] : 0.f;
        if (t >= p.V && c == 0) record_error(p.err, DLC_DEVERR_INDEX, (int)m);
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        const float *z = p.z + m * p.ld + c;
        if (n == 4) {
            const float4 q = *reinterpret_cast<const float4 *>(z);
            v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (i < n) v[i] = z[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float e = p.n0 + c + i == t ? expm1f(v[i] - lse) : exp2_fast((v[i] - lse) * LOG2E);
            v[i] = counted ? d * e : 0.f;
            sum[i] += v[i];
        }
        unsigned short *dst = p.dz + m * p.ldz + c;  // (rows are padded to whole vectors)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        if (p.terms == 2)
            *reinterpret_cast<uint2 *>(dst + p.M * p.ldz) =
                make_uint2(pack_bf16(bf16_rest(v[0]), bf16_rest(v[1])), pack_bf16(bf16_rest(v[2]), bf16_rest(v[3])));
    }
    if (p.sums) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p.sums[(long long)blockIdx.y * p.cols + c + i] = sum[i];
    }
}

// Many strips of partial sums to CE_STRIPS of them, in a fixed order: 32 columns and one range of the strips
// a block, for column_sum's blocks to add up the rest.
constexpr int CE_STRIPS = 256;

__global__ void __launch_bounds__(1024) ce_strips_kernel(const float *sums, float *out, int cols, int strips) {
    griddep_launch_dependents();
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = (int)blockIdx.x * 32 + lane;
    const int s0 = (int)((long long)strips * blockIdx.y / CE_STRIPS), s1 = (int)((long long)strips * (blockIdx.y + 1) / CE_STRIPS);
    griddep_wait();
    float s = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int i = s0 + warp; i < s1; i += 32) s += sums[(long long)i * cols + c];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < cols) {
        for (int w = 1; w < 32; ++w) s += part[w][lane];
        out[(long long)blockIdx.y * cols + c] = s;
    }
}

// dx of the sums of dz's two terms: dx[m, c] = sum[m][c] + sum[M + m][c], four channels a thread.
struct CeTermsParams {
    const float *sum;          // [2 M][ld], rows of whole vectors
    long long M, ld, items;
    int C, pieces, vec;
    RowTensor dx;
};

__global__ void __launch_bounds__(CE_THREADS) ce_terms_kernel(const __grid_constant__ CeTermsParams p) {
    griddep_launch_dependents();
    const long long i = (long long)blockIdx.x * CE_THREADS + threadIdx.x;
    griddep_wait();
    if (i >= p.items) return;
    const long long m = i / p.pieces;
    const int c = 4 * (int)(i - m * p.pieces);
    const float4 a = *reinterpret_cast<const float4 *>(p.sum + m * p.ld + c), b = *reinterpret_cast<const float4 *>(p.sum + (p.M + m) * p.ld + c);
    const float v[4] = {a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w};
    store4(p.dx, row_off(p.dx.m, m), c, p.C - c, p.vec != 0, v);
}

// ---- dw of a few rows -------------------------------------------------------------------
//
// dw[k, c] = sum_m dz[m, k] x[m, c] for up to 16 rows, dz in two terms: little but writing dw, which the tiles of a general
// product do at 3.5 TB/s (their epilogues have one step of the product to hide behind).  A warp keeps 64
// channels of x in registers as the B operands of one step of mma.sync, and takes 16 classes of dz at a time; the
// columns of the four tiles are dealt so that a thread is left with eight neighbouring channels.  Training steps, in
// tiles and this way, with one term: 1 x 1024 -> 131072 252 and 217 us, 8 x 1024 -> 50000 132 and 120, 16 x 2048 -> 50304
// 204 and 197; two steps of it for 32 x 4096 -> 131072 850 and 1055.  With two terms 221, 124 and 198.

constexpr int CO_THREADS = 256, CO_ROWS = 16;

struct CeOuterParams {
    const unsigned short *dz;  // [2][M][ldz]
    long long ldz;
    RowTensor x;
    void *dw;                  // [cols][C]
    int M, C, cols, warps;     // warps of a block side by side along the channels (a power of two)
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T>
__global__ void __launch_bounds__(CO_THREADS, 3) ce_outer_kernel(const __grid_constant__ CeOuterParams p) {
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const int side = warp % p.warps, per = CO_THREADS / 32 / p.warps;
    const int c0 = ((int)blockIdx.x * p.warps + side) * 64;
    const int tiles = (p.cols + 15) / 16, step = (int)gridDim.y * per;
    griddep_wait();
    uint32_t b[2][4][2];  // [.. of 32 channels][tile][rows 2 q and 2 q + 8, with the next one each]
    const unsigned short *x = static_cast<const unsigned short *>(p.x.p);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int m = 8 * r + 2 * q;
        const long long r0 = m < p.M ? row_off(p.x.m, m) : 0, r1 = m + 1 < p.M ? row_off(p.x.m, m + 1) : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = c0 + 32 * h + (g >> 1) * 8 + 2 * j + (g & 1);
                const uint32_t lo = m < p.M && c < p.C ? x[r0 + c * p.x.m.cs] : 0u, hi = m + 1 < p.M && c < p.C ? x[r1 + c * p.x.m.cs] : 0u;
                b[h][j][r] = lo | hi << 16;
            }
    }
    uint32_t a[2][4], next[2][4];
    auto load = [&](int tile) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int v = tile * 16 + g + 8 * (i & 1), m = 8 * (i >> 1) + 2 * q;
                const unsigned short *dz = p.dz + (t * p.M + m) * p.ldz + v;
                const uint32_t lo = v < p.cols && m < p.M ? dz[0] : 0u, hi = v < p.cols && m + 1 < p.M ? dz[p.ldz] : 0u;
                next[t][i] = lo | hi << 16;
            }
    };
    int tile = (int)blockIdx.y * per + warp / p.warps;
    if (tile < tiles) load(tile);
    for (; tile < tiles; tile += step) {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[0][i] = next[0][i], a[1][i] = next[1][i];
        if (tile + step < tiles) load(tile + step);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float d[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.f;
                mma_16816(d[j], a[0], b[h][j][0], b[h][j][1]);
                mma_16816(d[j], a[1], b[h][j][0], b[h][j][1]);
            }
            const int c = c0 + 32 * h + 8 * q;  // (rows are whole vectors)
            if (c >= p.C) continue;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int v = tile * 16 + g + 8 * r;
                if (v >= p.cols) continue;
                T *dst = static_cast<T *>(p.dw) + (long long)v * p.C + c;
                if constexpr (sizeof(T) == 2) {
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16(d[0][2 * r], d[0][2 * r + 1]), pack_bf16(d[1][2 * r], d[1][2 * r + 1]),
                                                                 pack_bf16(d[2][2 * r], d[2][2 * r + 1]), pack_bf16(d[3][2 * r], d[3][2 * r + 1]));
                } else {
                    reinterpret_cast<float4 *>(dst)[0] = make_float4(d[0][2 * r], d[0][2 * r + 1], d[1][2 * r], d[1][2 * r + 1]);
                    reinterpret_cast<float4 *>(dst)[1] = make_float4(d[2][2 * r], d[2][2 * r + 1], d[3][2 * r], d[3][2 * r + 1]);
                }
            }
        }
    }
}

// ---- host side -------------------------------------------------------------------------

// Whether ce_outer_kernel takes dw's product.
bool outer_ok(const CrossEntropyProblem &p) { return p.M <= CO_ROWS && p.K % 8 == 0 && (uintptr_t)p.dw.p % 16 == 0; }

dlcStatus_t launch_outer(dlcContext *ctx, const CrossEntropyProblem &p, const unsigned short *dz, long long ldz, int n0, int cols) {
    CeOuterParams o;
    o.dz = dz;
    o.ldz = ldz;
    o.x = p.x;
    o.dw = static_cast<char *>(p.dw.p) + (size_t)n0 * p.K * dlc_dtype_bytes((dlcDataType_t)p.dw.dt);
    o.M = (int)p.M;
    o.C = p.K;
    o.cols = cols;
    o.warps = 1;
    while (o.warps < CO_THREADS / 32 && o.warps * 64 < p.K) o.warps *= 2;
    const int per = CO_THREADS / 32 / o.warps;
    const long long gx = (p.K + 64ll * o.warps - 1) / (64 * o.warps), need = ((cols + 15) / 16 + per - 1) / per;
    const long long gy = std::min<long long>(need, std::max<long long>(1, std::min<long long>(65535, (long long)ctx->sm_count * 12 / gx)));
    const bool bf = p.dw.dt == DLC_DATA_BFLOAT16;
    const void *kern = bf ? (const void *)ce_outer_kernel<unsigned short> : (const void *)ce_outer_kernel<float>;
    void *args[] = {&o};
    return dlc_launch(ctx, kern, dim3((unsigned)gx, (unsigned)gy), dim3(CO_THREADS), 0, args);
}

dlcStatus_t launch_terms(dlcContext *ctx, const CrossEntropyProblem &p, const RowTensor &sum) {
    CeTermsParams t;
    t.sum = static_cast<const float *>(sum.p);
    t.M = p.M;
    t.ld = sum.m.ld;
    t.C = p.K;
    t.pieces = (p.K + 3) / 4;
    t.items = p.M * t.pieces;
    t.dx = p.dx;
    t.vec = dlc_vec4_rows(p.dx);
    void *args[] = {&t};
    return dlc_launch(ctx, (const void *)ce_terms_kernel, dim3((unsigned)((t.items + CE_THREADS - 1) / CE_THREADS)), dim3(CE_THREADS), 0, args);
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// Logits (or dz) of a piece take at most about this much workspace, as far as 256 classes fit.  Backward passes of 4096 x
// 2048 -> 131072 / 8192 x 512 -> 65536 in pieces of 128 MB: 4022 / 1533 us, 256 MB 3913 / 1345,
// 512 MB 3836 / 1230, 1 GB 3893 / 1097: what a piece costs is dx's last wave and its FP32 sum.
constexpr size_t CE_PIECE_BYTES = (size_t)512 << 20;
constexpr size_t CE_PART_BYTES = (size_t)256 << 20;  // the same for the parts of fused products (1024 classes)

// Classes of a piece of `bytes`-sized elements a row and class.
int piece_of(const CrossEntropyProblem &p, int bytes) {
    const long long most = std::max<long long>(256, (long long)(CE_PIECE_BYTES / (size_t)bytes) / p.M / 256 * 256);
    return (int)std::min<long long>(p.V, most);
}

RowTensor dense(void *p, int dt, long long ld) {
    RowTensor t;
    t.p = p;
    t.dt = dt;
    t.m = RowMap{ld, 0, 0, 1, ld, 1, 1, 1};
    return t;
}

// w from class n0 on, `cols` rows of it.
RowTensor classes(const CrossEntropyProblem &p, int n0, int cols) {
    RowTensor t = p.w;
    t.p = static_cast<char *>(p.w.p) + (size_t)n0 * p.K * dlc_dtype_bytes((dlcDataType_t)p.w.dt);
    t.m.ld = cols > 1 ? p.K : (p.K + 15) / 16 * 16;  // (of one row any pitch)
    return t;
}

int segments(int cols) { return (cols + CE_SEGMENT - 1) / CE_SEGMENT; }

// How many partial sums dbias has: strips of rows, each summed up by one block or warp.
int strips(const dlcContext *ctx, const CrossEntropyProblem &p, bool fused, int cols) {
    if (fused) return (int)((p.M + 31) / 32);
    const int gx = (cols + 4 * CE_THREADS - 1) / (4 * CE_THREADS);
    return (int)std::min<long long>(p.M, std::max(1, ctx->sm_count * 8 / gx));
}

// Where a call keeps what between its kernels (ws null: sizes only).
struct CePlan {
    bool fused = false;        // the product's epilogue takes the logits from the accumulators
    int piece = 0, parts = 0;
    long long ld = 0, ldz = 0;
    int terms = 1;             // BF16 terms of dz
    bool stacked = false;      // ... whose products with w are rows of one product, added up at the end
    bool x_packed = false, w_packed = false;
    void *x_copy = nullptr, *w_copy = nullptr;
    float *z = nullptr, *chosen = nullptr, *sums = nullptr, *few_sums = nullptr;
    float2 *part = nullptr;
    unsigned short *dz = nullptr;
    RowTensor dx_sum;          // FP32, where several pieces add to a dx of another type, or two terms' rows (stacked)
    char *gemm_ws = nullptr;
    size_t bytes = 0;
    char *base;

    explicit CePlan(char *ws) : base(ws) {}
    void *take(size_t n) {
        void *at = base ? base + bytes : (void *)(uintptr_t)256;
        bytes += round256(n);
        return at;
    }
    void operands(const CrossEntropyProblem &p) {
        x_packed = dlc_pack_bytes(p.x, p.M, p.K) != 0;
        w_packed = dlc_pack_bytes(classes(p, 0, p.V), p.V, p.K) != 0;
        const long long e = dlc_dtype_bytes((dlcDataType_t)p.w.dt), row = (p.K * e + 15) / 16 * 16;
        if (x_packed) x_copy = take((size_t)p.M * row);
        if (w_packed) w_copy = take((size_t)piece * row);
    }
    RowTensor x(const CrossEntropyProblem &p) const { return x_packed ? dlc_packed(p.x, p.K, x_copy) : p.x; }
    RowTensor w(const CrossEntropyProblem &p, int n0, int cols) const {
        const RowTensor t = classes(p, n0, cols);
        return w_packed ? dlc_packed(t, p.K, w_copy) : t;
    }
    // Copies of a piece's operands, where they are wanted.
    dlcStatus_t pack(dlcContext *ctx, const CrossEntropyProblem &p, int n0, int cols) const {
        PackItem items[DLC_MAX_PACKS];
        RowTensor tx = p.x, tw = classes(p, n0, cols);
        int n = 0;
        if (x_packed && n0 == 0) items[n++] = PackItem{&tx, p.M, p.K, x_copy};
        if (w_packed) items[n++] = PackItem{&tw, cols, p.K, w_copy};
        return dlc_launch_pack(ctx, items, n);
    }
    // z = sa sb x w^T + bias of a piece
    GemmProblem logits(const CrossEntropyProblem &p, int n0, int cols) const {
        GemmProblem g;
        g.M = p.M;
        g.N = cols;
        g.K = p.K;
        g.a.t = x(p);
        g.b.t = w(p, n0, cols);
        g.sa = p.sa;
        g.sb = p.sb ? p.sb + n0 : nullptr;
        g.bias = p.bias ? p.bias + n0 : nullptr;
        g.y = dense(z, DLC_DATA_FLOAT, ld);
        g.ws = gemm_ws;
        return g;
    }
    // dx (+)= dz w of a piece; the pieces before it have left their sum in dx_sum or dx
    GemmProblem data(const CrossEntropyProblem &p, int n0, int cols) const {
        GemmProblem g;
        g.M = stacked ? 2 * p.M : p.M;
        g.N = p.K;
        g.K = cols;
        g.terms = stacked ? 1 : terms;
        g.a.t = dense(dz, DLC_DATA_BFLOAT16, ldz);
        g.b.t = w(p, n0, cols);
        g.b.trans = 1;
        const RowTensor sum = dx_sum.p ? dx_sum : p.dx;
        g.y = n0 + cols == p.V && !stacked ? p.dx : sum;
        if (n0) g.r = sum;
        g.ws = gemm_ws;
        return g;
    }
    // dw = dz^T x of a piece
    GemmProblem filters(const CrossEntropyProblem &p, int n0, int cols) const {
        GemmProblem g;
        g.M = cols;
        g.N = p.K;
        g.K = p.M;
        g.terms = terms;
        g.a.t = dense(dz, DLC_DATA_BFLOAT16, ldz);
        g.a.trans = 1;
        g.b.t = x(p);
        g.b.trans = 1;
        g.y = p.dw;
        g.y.p = static_cast<char *>(p.dw.p) + (size_t)n0 * p.K * dlc_dtype_bytes((dlcDataType_t)p.dw.dt);
        g.y.m.ld = cols > 1 ? p.K : (p.K + 15) / 16 * 16;
        g.ws = gemm_ws;
        return g;
    }
    // the same product with the loss's epilogue
    GemmProblem fused_logits(const CrossEntropyProblem &p, int mode, int n0, int cols, int part0) const {
        GemmProblem g = logits(p, n0, cols);
        g.y = mode == ENTROPY_DZ ? dense(dz, DLC_DATA_BFLOAT16, ldz) : RowTensor();
        EntropyTile &e = g.entropy;
        e.mode = mode;
        e.V = p.V;
        e.n0 = n0;
        e.target = p.target;
        e.part = part;
        e.part0 = part0;
        e.chosen = chosen;
        e.lse = p.lse;
        e.dloss = p.dloss;
        e.sums = sums;
        e.terms = terms;
        return g;
    }
    // fn(first class, how many) of every piece
    template <typename Fn>
    dlcStatus_t each(const CrossEntropyProblem &p, Fn fn) const {
        for (int n0 = 0; n0 < p.V; n0 += piece) {
            const dlcStatus_t st = fn(n0, std::min(piece, p.V - n0));
            if (st != DLC_STATUS_SUCCESS) return st;
        }
        return DLC_STATUS_SUCCESS;
    }
    int parts_of(const dlcContext *ctx, const CrossEntropyProblem &p, int n0, int cols) const {
        return fused ? dlc_entropy_parts(ctx, fused_logits(p, ENTROPY_PARTS, n0, cols, 0)) : segments(cols);
    }
};

// Whether the pair kernel's epilogue takes the logits from its accumulators.  For a few rows the
// filters' stream decides, which the few-row kernels carry better than tiles of 256 rows do,
// and FP32 logits are little beside it.  Forward, 4096 -> 131072: 1 row 162 us with logits in
// memory, 295 fused; 16 rows 169 and 179; 32 rows 176 and 179; 48 rows 184 and 182; 96 rows
// 200 and 185; more rows far apart (4096 x 2048 -> 131072 1793 and 1084 us).  Up to a segment of
// classes the rows' sums are one kernel, which moves the point: 2048 -> 1000 32 rows 7.6 and 10.2 us, 64
// rows 8.4 and 10.4, 192 rows 10.2 and 10.4; 1024 -> 4096 48 rows 8.8 and 10.1, 64 rows 8.7 and 8.2.
// Backward, with one term of dz: 8 rows 676 and 702, 16 rows 678 and 681, 32 rows 687 and 684; 2048 -> 1000: 4 rows 23.8
// and 25.0, 16 rows 24.8 and 24.6, 64 rows 26.8 and 24.7.
bool fuse_fwd(const CrossEntropyProblem &p) { return p.M > (p.V <= CE_SEGMENT ? 64 : 32); }
bool fuse_bwd(const CrossEntropyProblem &p) { return p.M > 16; }

CePlan plan_fwd(const dlcContext *ctx, const CrossEntropyProblem &p, char *ws) {
    CePlan f(ws);
    f.fused = fuse_fwd(p);
    // Where one kernel takes the rows' sums and few tiles of long rows leave most of the GPU idle, the product in
    // parts is the faster one, and the more exact one: an accumulator's additions truncate.  By parts
    // and fused, forward: 128 x 4096 -> 1000 11.1 and 15.4 us, 197 x 2992 -> 232 9.7 and 13.2 (losses 1.4e-7 and
    // 9e-7 off), 80 x 2044 -> 12 9.3 and 11.8, 2000 x 4000 -> 64 14.2 and 15.1, 512 x 4096 -> 2048 16.3 and 16.6; but 256
    // x 2048 -> 1000 11.7 and 11.0, 700 x 2048 -> 300 11.6 and 11.1, 96 x 512 -> 512 7.8 and 7.3.  Products of the
    // few-row kernel that are not in parts are neither: 3129 x 2784 -> 329 21.1 and 13.2, 622 x 2720 -> 1985 19.8 and 13.0.
    // Over 200 sizes (65 to 4000 rows, 128 to 8192 channels, 2 to 4096 classes) this is 1.5 to 2.7 % slower than the faster
    // way on average, and 1.4 to 1.6 times at worst, a few tiles of 1500 to 2500 channels (169 x 2024 -> 85 12.1 and 7.4); the
    // products' time models in its place came to 1.3 % and 1.7 times.
    if (f.fused && p.V <= CE_SEGMENT && p.K >= (p.M <= 128 ? 1024 : 2560)) {
        f.piece = p.V;
        f.ld = (p.V + 3) / 4 * 4;
        f.z = reinterpret_cast<float *>((uintptr_t)256);  // (as aligned as it will be)
        f.fused = !dlc_gemm_spread(ctx, f.logits(p, 0, p.V));
    }
    // (a part: 32 classes at least)
    f.piece = f.fused ? (int)std::min<long long>(p.V, std::max<long long>(1024, (long long)(CE_PART_BYTES / 8) / p.M * 32 / 256 * 256))
                      : piece_of(p, 4);
    // (the matrix-vector kernel takes the operands as they are)
    if (f.fused || !dlc_gemv_ok(f.logits(p, 0, f.piece))) f.operands(p);
    f.z = nullptr;
    if (!f.fused) {
        f.ld = (f.piece + 3) / 4 * 4;
        f.z = static_cast<float *>(f.take((size_t)p.M * f.ld * 4));
    }
    size_t most = 0;
    f.each(p, [&](int n0, int cols) {
        f.parts = std::max(f.parts, 1 + f.parts_of(ctx, p, n0, cols));
        most = std::max(most, dlc_gemm_workspace(ctx, f.fused ? f.fused_logits(p, ENTROPY_PARTS, n0, cols, 0) : f.logits(p, n0, cols)));
        return DLC_STATUS_SUCCESS;
    });
    f.part = static_cast<float2 *>(f.take((size_t)f.parts * p.M * 8));
    f.chosen = static_cast<float *>(f.take((size_t)p.M * 4));
    f.gemm_ws = static_cast<char *>(f.take(most));
    return f;
}

// How many BF16 terms of dz enter the products (see the top).  Two up to 128 rows, where the terms are rows of one
// tile of the product with w, added up at the end (stack_terms), and the product with x is little but writing dw; and up to
// 2^30 products of a row, class and channel, where the products are read twice as long but the call is mostly
// launches.  Backward passes with one term and two: 1 x 1024 -> 131072 181 and 186 us, 16 x 2048 -> 50304 160 and 161,
// 32 x 4096 -> 131072 685 and 701, 128 x 4096 -> 131072 708 and 748, 128 x 64 -> 131072 99 and 118; 256 x 2048 -> 1000 26.2
// and 31.4, 4096 x 256 -> 1000 34.5 and 41.3.
constexpr int CE_STACK = 128;

int terms_of(const CrossEntropyProblem &p) {
    return p.M <= CE_STACK || (p.M <= 1 << 20 && (double)p.M * p.V * p.K <= 1073741824.0) ? 2 : 1;
}

// (The sum of the terms' rows is a launch: small products are rather read twice as long.  Stacked and not: 16 x 2048 ->
// 1000 25.4 and 27.4 us, 8 x 1024 -> 50000 102 and 118, 64 x 128 -> 32768 45.8 and 50.7; 32 x 128 -> 100 19.7 and 17.9,
// 64 x 512 -> 1000 25.1 and 22.5.)
bool stack_terms(const CrossEntropyProblem &p) { return p.M <= CE_STACK && (long long)p.V * p.K > 1 << 19; }

CePlan plan_bwd(const dlcContext *ctx, const CrossEntropyProblem &p, char *ws) {
    CePlan b(ws);
    b.fused = fuse_bwd(p);
    b.terms = terms_of(p);
    b.stacked = stack_terms(p);
    b.piece = piece_of(p, b.fused ? 2 * b.terms : 4);
    b.ldz = (b.piece + 7) / 8 * 8;
    b.operands(p);
    if (!b.fused) {
        b.ld = (b.piece + 3) / 4 * 4;
        b.z = static_cast<float *>(b.take((size_t)p.M * b.ld * 4));
    }
    b.dz = static_cast<unsigned short *>(b.take((size_t)b.terms * p.M * b.ldz * 2));
    if (p.dx.p && (b.stacked || (b.piece < p.V && p.dx.dt != DLC_DATA_FLOAT))) {
        const long long ld = ((long long)p.K + 3) / 4 * 4;
        b.dx_sum = dense(b.take((size_t)(b.stacked ? 2 : 1) * p.M * ld * 4), DLC_DATA_FLOAT, ld);
    }
    size_t most = 0, sums = 0;
    b.each(p, [&](int n0, int cols) {
        sums = std::max(sums, (size_t)strips(ctx, p, b.fused, cols) * cols * 4);
        most = std::max(most, dlc_gemm_workspace(ctx, b.fused ? b.fused_logits(p, ENTROPY_DZ, n0, cols, 0) : b.logits(p, n0, cols)));
        if (p.dx.p) most = std::max(most, dlc_gemm_workspace(ctx, b.data(p, n0, cols)));
        if (p.dw.p) most = std::max(most, dlc_gemm_workspace(ctx, b.filters(p, n0, cols)));
        return DLC_STATUS_SUCCESS;
    });
    if (p.dbias) {
        b.sums = static_cast<float *>(b.take(sums));
        b.few_sums = static_cast<float *>(b.take((size_t)CE_STRIPS * b.piece * 4));
    }
    b.gemm_ws = static_cast<char *>(b.take(most));
    return b;
}

CeParams params(const dlcContext *ctx, const CrossEntropyProblem &p, const CePlan &f) {
    CeParams c = {};
    c.M = p.M;
    c.V = p.V;
    c.z = f.z;
    c.ld = f.ld;
    c.target = p.target;
    c.part = f.part;
    c.chosen = f.chosen;
    c.loss = p.loss;
    c.lse = p.lse;
    c.dloss = p.dloss;
    c.dz = f.dz;
    c.ldz = f.ldz;
    c.terms = f.terms;
    c.sums = f.sums;
    c.err = ctx->d_err;
    return c;
}

}  // namespace

size_t dlc_cross_entropy_workspace(const dlcContext *ctx, const CrossEntropyProblem &p) { return plan_fwd(ctx, p, nullptr).bytes; }

dlcStatus_t dlc_launch_cross_entropy(dlcContext *ctx, const CrossEntropyProblem &p) {
    const CePlan f = plan_fwd(ctx, p, p.ws);
    CeParams c = params(ctx, p, f);
    return f.each(p, [&](int n0, int cols) {
        dlcStatus_t s = f.pack(ctx, p, n0, cols);
        if (s != DLC_STATUS_SUCCESS) return s;
        c.part0 = n0 ? 1 : 0;
        if (f.fused) {
            s = dlc_launch_gemm(ctx, f.fused_logits(p, ENTROPY_PARTS, n0, cols, c.part0));
        } else {
            s = dlc_launch_gemm(ctx, f.logits(p, n0, cols));
            if (s != DLC_STATUS_SUCCESS) return s;
            c.n0 = n0;
            c.cols = cols;
            c.parts = cols == p.V ? segments(cols) : 0;
            void *args[] = {&c};
            s = dlc_launch(ctx, (const void *)ce_part_kernel, dim3((unsigned)p.M, (unsigned)segments(cols)), dim3(CE_THREADS), 0, args);
            if (c.parts == 1) return s;  // the rows' losses are written
        }
        if (s != DLC_STATUS_SUCCESS) return s;
        c.parts = c.part0 + f.parts_of(ctx, p, n0, cols);
        c.last = n0 + cols == p.V;
        void *args[] = {&c};
        return dlc_launch(ctx, (const void *)ce_loss_kernel, dim3((unsigned)((p.M + 31) / 32)), dim3(1024), 0, args);
    });
}

size_t dlc_cross_entropy_bwd_workspace(const dlcContext *ctx, const CrossEntropyProblem &p) { return plan_bwd(ctx, p, nullptr).bytes; }

dlcStatus_t dlc_launch_cross_entropy_bwd(dlcContext *ctx, const CrossEntropyProblem &p) {
    const CePlan b = plan_bwd(ctx, p, p.ws);
    CeParams c = params(ctx, p, b);
    return b.each(p, [&](int n0, int cols) {
        dlcStatus_t s = b.pack(ctx, p, n0, cols);
        if (s != DLC_STATUS_SUCCESS) return s;
        const int rows = strips(ctx, p, b.fused, cols);
        if (b.fused) {
            s = dlc_launch_gemm(ctx, b.fused_logits(p, ENTROPY_DZ, n0, cols, 0));
        } else {
            s = dlc_launch_gemm(ctx, b.logits(p, n0, cols));
            if (s != DLC_STATUS_SUCCESS) return s;
            c.n0 = n0;
            c.cols = cols;
            void *args[] = {&c};
            s = dlc_launch(ctx, (const void *)ce_dz_kernel,
                           dim3((unsigned)((cols + 4 * CE_THREADS - 1) / (4 * CE_THREADS)), (unsigned)rows), dim3(CE_THREADS), 0, args);
        }
        if (s == DLC_STATUS_SUCCESS && p.dbias) {
            const bool many = rows > 8 * CE_STRIPS;
            int n = cols, strips = rows;
            float *from = b.sums, *to = b.few_sums;
            void *args[] = {&from, &to, &n, &strips};
            if (many) s = dlc_launch(ctx, (const void *)ce_strips_kernel, dim3((unsigned)((cols + 31) / 32), CE_STRIPS), dim3(1024), 0, args);
            if (s == DLC_STATUS_SUCCESS) s = dlc_launch_column_sum(ctx, many ? to : from, p.dbias + n0, cols, many ? CE_STRIPS : rows);
        }
        if (s == DLC_STATUS_SUCCESS && p.dx.p) s = dlc_launch_gemm(ctx, b.data(p, n0, cols));
        if (s == DLC_STATUS_SUCCESS && p.dx.p && b.stacked && n0 + cols == p.V) s = launch_terms(ctx, p, b.dx_sum);
        if (s == DLC_STATUS_SUCCESS && p.dw.p)
            s = outer_ok(p) ? launch_outer(ctx, p, b.dz, b.ldz, n0, cols) : dlc_launch_gemm(ctx, b.filters(p, n0, cols));
        return s;
    });
}

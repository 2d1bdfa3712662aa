// gemm_rows.cu -- the products of the linear and gated layers for few rows
// (decoding, a classifier's batch): the time is that of reading the filters
// once, so every SM streams its own part of them.
//
// The operands trade places with gemm.cu: up to 128 filters are the MMA's M side,
// the rows (padded to a multiple of 16, at most 128) its N side, so a block
// moves 16 KiB of filters for 2 KiB and up of rows and pads neither much.  A
// gated tile holds the gate and the up filters of up to 64 outputs side by side.
// Where there are fewer tiles than SMs, tiles narrow to 16 filters, or a cluster of
// up to eight CTAs shares a tile, each with a range of the reduction; the partial
// sums stay in shared memory, every CTA adds up its share of the rows over the
// cluster, always in the same order, and applies the epilogue.  Nothing but the
// outputs is written to memory and there is one launch.
//
// Measured back to back: gated 64 x 4096 -> 2 x 8192 in E4M3 15.7 us, 128 x 4096 ->
// 4096 in BF16 12.6, 16 rows 10.2 (67, 34 and 34 MB of filters).  The filters stream
// at 6.5 TB/s and more once under way; the rest of a call is its start (2 to 3 us
// from the last grid's end to the first bytes) and its end (partial sums, cluster
// barriers, epilogue: 2 to 4 us).  Tried and no faster: two CTAs an SM with the
// next grid's filters prefetched into the L2 before its turn, partial sums pushed by
// bulk copies, a dry run of the epilogue that warms the instruction cache.
//
// Roles (16 warps): a thread of warp 0 loads, one of warp 1 issues the MMAs; all warps
// read the accumulators (four per quarter of the TMEM lanes) and join the partial
// sums, a thread four filters.  Every wait is bounded.
#include <cstring>

#include "channel.cuh"
#include "gemm.h"
#include "ptx.cuh"

namespace {

using namespace dlc;

constexpr int FR_M = 128;                   // the MMA's M side: a tile's filters, gate and up
constexpr int FR_LINE = 128;                // bytes of an operand row per k-block
constexpr int FR_MAX_ROWS = 128;            // of a tile
constexpr int FR_THREADS = 512;
constexpr int FR_MAX_STAGES = 24, FR_MAX_SPLITS = 8;  // (a cluster of eight is portable)
constexpr int FR_SMEM = 226 * 1024;

struct FrParams {
    long long M;
    int N, act;
    int num_kb, splits, rows;      // rows of a tile (the MMA's N)
    int filters, quads_log2;       // outputs of a tile; log2 of its quads, rounded up to a power of two
    int stages;
    uint32_t stage_bytes, idesc, tmem_cols;
    const float *sa, *sb, *bias;
    RowTensor z, r, y;
    bool z_vec, z2_vec, r_vec, y_vec;  // four-element accesses (z2: the up half of z)
    int *err;
    unsigned long long timeout_ns;
};

// Adds up the partial sums of rows j0 .. j0+count-1 of a tile over the cluster,
// in the order of their ranges, and applies the epilogue: a thread four filters,
// the same ones for all its rows.  `sums`: a CTA's partial sums, [row][filter], at
// the same address in each; `scale`: the rows' scales.  A launch runs this code once or a few times, so
// fetching it counts: it is kept short (unrolled over rows it took 2.1 us a pass
// of four rows, most of it instruction fetches).
template <bool GATED>
__device__ __forceinline__ void fr_join(const FrParams &p, uint32_t sums, const float *scale, int split, long long m0, int n, int f, int j0,
                                        int count, const float (&sb)[GATED ? 2 : 1][4],
                                        const float (&bias)[GATED ? 2 : 1][4]) {
    constexpr int HALVES = GATED ? 2 : 1, AT_ONCE = 4;  // ranges loaded before they are added
    const int cols = p.N - n;
    const uint32_t half = (uint32_t)p.filters * 4u;
#pragma unroll 1
    for (int j = (int)threadIdx.x >> p.quads_log2; j < count; j += FR_THREADS >> p.quads_log2) {
        const long long m = m0 + j0 + j;
        const float sa = scale[j0 + j];
        const uint32_t at = sums + ((uint32_t)(j0 + j) * FR_M + (uint32_t)f) * 4u;
        float v[HALVES][4];
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[h][i] = 0.f;
#pragma unroll 1
        for (int s0 = 0; s0 < p.splits; s0 += AT_ONCE) {
            float4 q[AT_ONCE][HALVES];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i)
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    const uint32_t a = at + (uint32_t)h * half;
                    if (s0 + i == split)
                        q[i][h] = ld_shared_f32x4(a);
                    else if (s0 + i < p.splits)
                        q[i][h] = ld_cluster_f32x4(mapa_shared(a, (uint32_t)(s0 + i)));
                }
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i)
#pragma unroll
                for (int h = 0; h < HALVES; ++h)
                    if (s0 + i < p.splits)
                        v[h][0] += q[i][h].x, v[h][1] += q[i][h].y, v[h][2] += q[i][h].z, v[h][3] += q[i][h].w;
        }
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[h][i] = fmaf(v[h][i], sa * sb[h][i], bias[h][i]);
        if (p.z.p) {
            const long long zo = row_off(p.z.m, m);
#pragma unroll
            for (int h = 0; h < HALVES; ++h) store4(p.z, zo, (long long)h * p.N + n, cols, h ? p.z2_vec : p.z_vec, v[h]);
        }
        float y[4] = {v[0][0], v[0][1], v[0][2], v[0][3]};
        act_dispatch(p.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < 2; ++i) set2(y, i, act_f2<decltype(act)::value>(get2(y, i)));
        });
        if (GATED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] *= v[HALVES - 1][i];
        }
        if (p.r.p) {
            float w[4];
            load4(p.r, row_off(p.r.m, m), n, cols, p.r_vec, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] += w[i];
        }
        store4(p.y, row_off(p.y.m, m), n, cols, p.y_vec, y);
    }
}

template <bool E4M3, bool GATED>
__global__ void __launch_bounds__(FR_THREADS, 1)
    gemm_rows_kernel(const __grid_constant__ FrParams p, const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmX) {
    constexpr int BK = E4M3 ? FR_LINE : FR_LINE / 2;
    constexpr int HALVES = GATED ? 2 : 1;
    griddep_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    __shared__ alignas(8) uint64_t full[FR_MAX_STAGES], empty[FR_MAX_STAGES], done;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    __shared__ float scale[FR_MAX_ROWS];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t smem = raw + ((1024u - (raw & 1023u)) & 1023u);  // same offset in every CTA
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int split = (int)cluster_ctarank();
    const int n0 = (int)(blockIdx.x / (unsigned)p.splits) * p.filters;
    const long long m0 = (long long)blockIdx.y * p.rows;
    const int kb0 = (int)((long long)p.num_kb * split / p.splits);
    const int kb1 = (int)((long long)p.num_kb * (split + 1) / p.splits);
    const uint32_t w_bytes = (uint32_t)p.filters * FR_LINE;
    auto load = [&](int kb, int stage) {
        mbar_arrive_expect_tx(&full[stage], p.stage_bytes);
        const uint32_t dst = smem + (uint32_t)stage * p.stage_bytes;
        tma_load_2d(dst, &tmW, &full[stage], kb * BK, n0);
        if (GATED) tma_load_2d(dst + w_bytes, &tmW, &full[stage], kb * BK, p.N + n0);
        tma_load_2d(dst + HALVES * w_bytes, &tmX, &full[stage], kb * BK, (int)m0);
    };
    const int first = min(kb1, kb0 + p.stages);  // the blocks that need no free stage
    if (threadIdx.x == 0) {
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmX);
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&full[i], 1u);
            mbar_init(&empty[i], 1u);
        }
        mbar_init(&done, 1u);
        abort_flag = 0;
        fence_mbar_init();
        griddep_wait();
        for (int kb = kb0; kb < first; ++kb) load(kb, kb - kb0);
    }
    if (warp == 1) {
        tmem_alloc(&tmem_slot, p.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_slot;
    const WaitCtl ctl{&abort_flag, p.err, p.timeout_ns};
    griddep_wait();

    if (warp == 0 && elect_one()) {
        int stage = first - kb0 == p.stages ? 0 : first - kb0;
        uint32_t ph = 1;
        for (int kb = first; kb < kb1; ++kb) {
            if (!mbar_wait(&empty[stage], ph ^ 1u, ctl, 31)) break;
            load(kb, stage);
            if (++stage == p.stages) stage = 0, ph ^= 1u;
        }
    } else if (warp == 1 && elect_one()) {
        int stage = 0;
        uint32_t ph = 0, acc = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait(&full[stage], ph, ctl, 32)) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            const uint32_t src = smem + (uint32_t)stage * p.stage_bytes;
            const uint64_t w = sw128_kmajor_desc(src), x = sw128_kmajor_desc(src + HALVES * w_bytes);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (E4M3)
                    umma_e4m3_nc(tmem, w + 2u * j, x + 2u * j, p.idesc, j ? 1u : acc);
                else
                    umma_bf16_nc(tmem, w + 2u * j, x + 2u * j, p.idesc, j ? 1u : acc);
            }
            acc = 1;
            umma_commit(&empty[stage]);
            if (++stage == p.stages) stage = 0, ph ^= 1u;
        }
        if (!ok) {  // loads of stages not consumed: wait briefly, so that no copy outlives the CTA
            volatile int dummy = 0;
            const WaitCtl brief{&dummy, p.err, 50000000ull};
            for (int j = 0; j < p.stages; ++j) {
                if (!mbar_wait(&full[stage], ph, brief, 92)) break;
                if (++stage == p.stages) stage = 0, ph ^= 1u;
            }
        }
        umma_commit(&done);
    }
    __syncwarp();
    // this thread's four filters in the epilogue
    const int f = 4 * ((int)threadIdx.x & ((1 << p.quads_log2) - 1)), n = n0 + f, cols = f < p.filters ? p.N - n : 0;
    float sb[HALVES][4], bias[HALVES][4];
#pragma unroll
    for (int h = 0; h < HALVES; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sb[h][i] = p.sb && i < cols ? p.sb[(long long)h * p.N + n + i] : 1.f;
            bias[h][i] = p.bias && i < cols ? p.bias[(long long)h * p.N + n + i] : 0.f;
        }
    for (int j = (int)threadIdx.x; j < p.rows; j += FR_THREADS) scale[j] = p.sa && m0 + j < p.M ? p.sa[m0 + j] : 1.f;
    bool good;
    {
        volatile int dummy = 0;  // (an abort elsewhere still commits `done`)
        const WaitCtl fin{&dummy, p.err, p.timeout_ns};
        good = mbar_wait(&done, 0u, fin, 91);
    }
    __syncwarp();
    tc_fence_after_sync();
    // partial sums to shared memory, where the operands were: [row][filter]
    {
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t mine = smem + (uint32_t)((warp & 3) * 32 + lane) * 4u;
#pragma unroll 1
        for (int c = 16 * (warp >> 2); c < p.rows; c += 4 * FR_THREADS / 32) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(lanes + (uint32_t)c, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(mine + (uint32_t)(c + i) * FR_M * 4u), "r"(v[i]) : "memory");
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (p.splits > 1) {
        cluster_arrive();
        cluster_wait();  // the cluster's partial sums are in place
    }
    good = good && abort_flag == 0;
    const int per = (p.rows + p.splits - 1) / p.splits, j0 = split * per;
    const int count = (int)min((long long)min(per, p.rows - j0), p.M - m0 - j0);
    if (good && cols > 0) fr_join<GATED>(p, smem, scale, split, m0, n, f, j0, count, sb, bias);
    __syncwarp();
    if (p.splits > 1) {
        cluster_arrive();
        cluster_wait();  // no CTA leaves while another reads its partial sums
    }
    if (warp == 1) tmem_dealloc(tmem, p.tmem_cols);
}

// Clusters of `size` CTAs (an SM each) that the device holds at once.
int resident_clusters(const dlcContext *ctx, int size) {
    static_assert(FR_MAX_SPLITS < (int)(sizeof(ctx->resident_few) / sizeof(ctx->resident_few[0])), "a count for each size");
    return dlc_resident_clusters(ctx, &ctx->resident_few[size], (const void *)gemm_rows_kernel<false, false>, size, FR_THREADS,
                                 FR_SMEM);
}

}  // namespace

FewRowsPlan dlc_few_rows_plan(const dlcContext *ctx, const GemmProblem &g) {
    FewRowsPlan p;
    const int e = dlc_dtype_bytes((dlcDataType_t)g.a.t.dt);
    p.num_kb = (int)((g.K * e + FR_LINE - 1) / FR_LINE);
    const long long row_tiles = (g.M + FR_MAX_ROWS - 1) / FR_MAX_ROWS;
    p.rows = (int)(((g.M + row_tiles - 1) / row_tiles + 15) / 16 * 16);
    p.row_tiles = (int)std::min<long long>((g.M + p.rows - 1) / p.rows, 65535);
    // Filters and CTAs a tile from a model of the time in microseconds, fitted to eleven
    // shapes from 16 x 512 -> 512 to 128 x 4096 -> 8192 (its choice is within 4 % of
    // the fastest of some twenty alternatives each), its level set against the pair
    // kernel's model on twenty more from 100 x 1024 -> 2 x 1024 to 10932 x 64 -> 320:
    // the launch; per k-block a turn of the MMA thread or the filters' bytes; the
    // partial sums' way to the epilogue and the barriers of a cluster.  The SMs of a
    // GPC that a cluster does not fill stay idle, so fewer clusters run at once than
    // the SMs suggest.
    const int halves = g.gated ? 2 : 1, most = FR_M / halves;
    p.us = 1e300;
    for (int s = 1; s <= FR_MAX_SPLITS && (s == 1 || 2 * s <= p.num_kb); ++s) {
        const int at_once = resident_clusters(ctx, s);
        for (int filters = most; filters >= 16; filters /= 2) {
            if (filters < most && filters >= g.N) continue;
            const int tiles = (g.N + filters - 1) / filters;
            const long long clusters = (long long)tiles * p.row_tiles, waves = (clusters + at_once - 1) / at_once;
            const double ctas = (double)clusters * s / (double)waves, own = p.rows * halves * filters / 16384.0;
            const double kb = std::max(0.23, halves * filters * FR_LINE * ctas / 5.8e6);
            // (a later wave starts from nothing: barriers, tensor memory, first loads)
            const double t = 2.85 + 1.4 * ctas / ctx->sm_count + 3.0 * (double)(waves - 1) +
                             waves * ((p.num_kb + s - 1) / s * kb + (s > 1 ? 0.9 : 0.) + 1.9 * own * (2.0 - 1.0 / s));
            if (t < p.us) p.us = t, p.splits = s, p.filters = filters, p.filter_tiles = tiles;
        }
    }
    if ((g.M + p.rows - 1) / p.rows > 65535) p.us = 1e300;  // more row tiles than a grid has
    return p;
}

dlcStatus_t dlc_launch_few_rows(dlcContext *ctx, const GemmProblem &g) {
    const bool e4m3 = g.a.t.dt == DLC_DATA_FLOAT8_E4M3;
    const FewRowsPlan pl = dlc_few_rows_plan(ctx, g);
    FrParams p;
    std::memset(&p, 0, sizeof(p));
    p.M = g.M;
    p.N = g.N;
    p.act = g.act;
    p.num_kb = pl.num_kb;
    p.splits = pl.splits;
    p.rows = pl.rows;
    const int halves = g.gated ? 2 : 1;
    p.filters = pl.filters;
    p.quads_log2 = 0;
    while ((4 << p.quads_log2) < pl.filters) ++p.quads_log2;
    p.stage_bytes = (uint32_t)((halves * pl.filters + pl.rows) * FR_LINE);
    // (stages carry the filters' stream: with tiles of 128 filters, one row of 2048 ->
    // 2 x 8192 took 15.4 us with six of them, 16.4 with five)
    // (the MMA reads 128 rows of filters whatever the tile holds: what lies behind them goes
    // to accumulator lanes that nothing reads)
    const int behind = std::max(0, (FR_M - halves * pl.filters - pl.rows) * FR_LINE);
    p.stages = std::min(FR_MAX_STAGES, (FR_SMEM - 1024 - behind) / (int)p.stage_bytes);
    p.stages = std::max(2, std::min(p.stages, (pl.num_kb + pl.splits - 1) / pl.splits));
    const size_t smem = 1024 + std::max((size_t)p.stages * p.stage_bytes + behind, (size_t)pl.rows * FR_M * 4);
    p.sa = g.sa;
    p.sb = g.sb;
    p.bias = g.bias;
    p.z = g.z;
    p.r = g.r;
    p.y = g.y;
    p.z_vec = dlc_vec4_rows(g.z);
    p.z2_vec = p.z_vec && g.N % 4 == 0;
    p.r_vec = dlc_vec4_rows(g.r);
    p.y_vec = dlc_vec4_rows(g.y);
    p.err = ctx->d_err;
    p.timeout_ns = ctx->timeout_ns;
    const uint32_t fmt = e4m3 ? 0u : 1u;
    p.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(pl.rows >> 3) << 17) | ((uint32_t)(FR_M >> 4) << 24);
    p.tmem_cols = 32;
    while (p.tmem_cols < (uint32_t)pl.rows) p.tmem_cols <<= 1;
    CUtensorMap tw, tx;
    const int nb = halves * g.N;
    if (!dlc_encode_operand(ctx, &tw, g.b, nb, (int)g.K, pl.filters) ||
        !dlc_encode_operand(ctx, &tx, g.a, g.M, (int)g.K, pl.rows))
        return DLC_STATUS_EXECUTION_FAILED;
    const void *kern = g.gated ? (e4m3 ? (const void *)gemm_rows_kernel<true, true> : (const void *)gemm_rows_kernel<false, true>)
                               : (e4m3 ? (const void *)gemm_rows_kernel<true, false> : (const void *)gemm_rows_kernel<false, false>);
    if (!dlc_allow_smem(ctx, kern, smem)) return DLC_STATUS_EXECUTION_FAILED;
    void *args[] = {&p, &tw, &tx};
    return dlc_launch(ctx, kern, dim3((unsigned)(pl.filter_tiles * pl.splits), (unsigned)pl.row_tiles), dim3(FR_THREADS), smem,
                      args, pl.splits);
}

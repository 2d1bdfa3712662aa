// gemm_rows.cu -- the products of the linear and gated layers for few rows
// (decoding, a classifier's batch): the time is that of reading the filters
// once, so every SM streams its own part of them.
//
// The operands trade places with gemm.cu: 128 filters are the MMA's M side,
// the rows (padded to a multiple of 16, at most 128) its N side, so a block
// moves 16 KiB of filters for 2 KiB and up of rows and pads neither much.  A
// gated tile takes 128 gate and 128 up filters into two accumulators.  Where
// there are fewer tiles than SMs, a cluster of up to eight CTAs shares a tile,
// each with a range of the reduction; the partial sums stay in shared memory
// and every CTA adds up its share of the rows over the cluster, always in the
// same order, and applies the epilogue.  Nothing but the outputs is written to
// memory and there is one launch.
//
// Roles (8 warps): warp 0 lane 0 loads, warp 1 lane 0 issues the MMAs; all warps
// read the accumulators (two per quarter of the TMEM lanes) and join the partial
// sums, a warp a row, a lane four filters.  Every wait is bounded.
#include <cstring>

#include "channel.cuh"
#include "gemm.h"
#include "ptx.cuh"

namespace {

using namespace dlc;

constexpr int FR_FILTERS = 128;
constexpr int FR_LINE = 128;                        // bytes of an operand row per k-block
constexpr int FR_W_BYTES = FR_FILTERS * FR_LINE;    // 16 KiB
constexpr int FR_THREADS = 256;
constexpr int FR_MAX_STAGES = 12, FR_MAX_SPLITS = 8;  // (a cluster of eight is portable)
constexpr int FR_SMEM = 212 * 1024, FR_BAR_AREA = 512;

struct FrParams {
    long long M;
    int N, act;
    int num_kb, splits, rows;      // rows of a tile (the MMA's N)
    int stages;
    uint32_t stage_bytes, idesc, tmem_cols;
    const float *sa, *sb, *bias;
    RowTensor z, r, y;
    bool z_vec, z2_vec, r_vec, y_vec;  // four-element accesses (z2: the up half of z)
    int *err;
    unsigned long long timeout_ns;
};

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
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t smem = raw + ((1024u - (raw & 1023u)) & 1023u);  // same offset in every CTA
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = (int)cluster_ctarank();
    const int n0 = (int)(blockIdx.x / (unsigned)p.splits) * FR_FILTERS;
    const long long m0 = (long long)blockIdx.y * p.rows;
    const int kb0 = (int)((long long)p.num_kb * split / p.splits);
    const int kb1 = (int)((long long)p.num_kb * (split + 1) / p.splits);
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&full[i], 1u);
            mbar_init(&empty[i], 1u);
        }
        mbar_init(&done, 1u);
        abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmX);
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

    if (warp == 0 && lane == 0) {
        int stage = 0;
        uint32_t ph = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait(&empty[stage], ph ^ 1u, ctl, 31)) break;
            mbar_arrive_expect_tx(&full[stage], p.stage_bytes);
            const uint32_t dst = smem + (uint32_t)stage * p.stage_bytes;
            tma_load_2d(dst, &tmW, &full[stage], kb * BK, n0);
            if (GATED) tma_load_2d(dst + FR_W_BYTES, &tmW, &full[stage], kb * BK, p.N + n0);
            tma_load_2d(dst + HALVES * FR_W_BYTES, &tmX, &full[stage], kb * BK, (int)m0);
            if (++stage == p.stages) stage = 0, ph ^= 1u;
        }
    } else if (warp == 1 && lane == 0) {
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
            const uint64_t x = sw128_kmajor_desc(src + HALVES * FR_W_BYTES);
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                const uint64_t w = sw128_kmajor_desc(src + (uint32_t)h * FR_W_BYTES);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (E4M3)
                        umma_e4m3_nc(tmem + (uint32_t)(h * p.rows), w + 2u * j, x + 2u * j, p.idesc, j ? 1u : acc);
                    else
                        umma_bf16_nc(tmem + (uint32_t)(h * p.rows), w + 2u * j, x + 2u * j, p.idesc, j ? 1u : acc);
                }
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
    // this lane's four filters in the epilogue
    const int f = lane * 4, n = n0 + f, cols = p.N - n;
    float sb[HALVES][4], bias[HALVES][4];
#pragma unroll
    for (int h = 0; h < HALVES; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sb[h][i] = p.sb && i < cols ? __ldg(p.sb + (long long)h * p.N + n + i) : 1.f;
            bias[h][i] = p.bias && i < cols ? __ldg(p.bias + (long long)h * p.N + n + i) : 0.f;
        }
    bool good;
    {
        volatile int dummy = 0;  // (an abort elsewhere still commits `done`)
        const WaitCtl fin{&dummy, p.err, p.timeout_ns};
        good = mbar_wait(&done, 0u, fin, 91);
    }
    __syncwarp();
    tc_fence_after_sync();
    // partial sums to shared memory, where the operands were: [half][row][filter]
    const uint32_t plane = (uint32_t)p.rows * FR_FILTERS * 4u;
#pragma unroll
    for (int h = 0; h < HALVES; ++h)
        for (int c = 16 * (warp >> 2); c < p.rows; c += 32) {
            const int quad = warp & 3;
            uint32_t v[16];
            tmem_ld_32x32b_x16(tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(h * p.rows + c), v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(smem + (uint32_t)h * plane +
                             ((uint32_t)(c + i) * FR_FILTERS + (uint32_t)(quad * 32 + lane)) * 4u), "r"(v[i]) : "memory");
        }
    __syncwarp();
    tc_fence_before_sync();
    cluster_sync();
    tc_fence_after_sync();
    good = good && abort_flag == 0;
    // this CTA's rows of the tile, a warp a row
    const int per = (p.rows + p.splits - 1) / p.splits;
    const int j1 = min(min(p.rows, (split + 1) * per), (int)min((long long)p.rows, p.M - m0));
    if (good && cols > 0) {
        for (int j = split * per + warp; j < j1; j += FR_THREADS / 32) {
            const long long m = m0 + j;
            const float sa = p.sa ? __ldg(p.sa + m) : 1.f;
            float v[HALVES][4];
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                const uint32_t at = smem + (uint32_t)h * plane + ((uint32_t)j * FR_FILTERS + (uint32_t)f) * 4u;
                float4 q[FR_MAX_SPLITS];
#pragma unroll
                for (int s = 0; s < FR_MAX_SPLITS; ++s)
                    if (s < p.splits) q[s] = ld_cluster_f32x4(mapa_shared(at, (uint32_t)s));
                float t[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
                for (int s = 1; s < FR_MAX_SPLITS; ++s)
                    if (s < p.splits) t[0] += q[s].x, t[1] += q[s].y, t[2] += q[s].z, t[3] += q[s].w;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[h][i] = fmaf(t[i], sa * sb[h][i], bias[h][i]);
            }
            if (p.z.p) {
                const long long zo = row_off(p.z.m, m);
#pragma unroll
                for (int h = 0; h < HALVES; ++h) store4(p.z, zo, (long long)h * p.N + n, cols, h ? p.z2_vec : p.z_vec, v[h]);
            }
            float y[4] = {v[0][0], v[0][1], v[0][2], v[0][3]};
            act_dispatch(p.act, [&](auto act) {
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = act_f<decltype(act)::value>(y[i]);
            });
            if (GATED) {
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] *= v[HALVES - 1][i];
            }
            if (p.r.p) {
                float r[4];
                load4(p.r, row_off(p.r.m, m), n, cols, p.r_vec, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] += r[i];
            }
            store4(p.y, row_off(p.y.m, m), n, cols, p.y_vec, y);
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    cluster_sync();  // no CTA leaves while another reads its partial sums
    tc_fence_after_sync();
    if (warp == 1) tmem_dealloc(tmem, p.tmem_cols);
}

}  // namespace

FewRowsPlan dlc_few_rows_plan(const dlcContext *ctx, const GemmProblem &g) {
    FewRowsPlan p;
    const int e = dlc_dtype_bytes((dlcDataType_t)g.a.t.dt);
    p.num_kb = (int)((g.K * e + FR_LINE - 1) / FR_LINE);
    p.rows = (int)std::min<long long>(FR_FILTERS, (g.M + 15) / 16 * 16);
    p.filter_tiles = (g.N + FR_FILTERS - 1) / FR_FILTERS;
    p.row_tiles = (int)((g.M + p.rows - 1) / p.rows);
    const long long tiles = (long long)p.filter_tiles * p.row_tiles;
    p.splits = 1;
    while (p.splits < FR_MAX_SPLITS && tiles * (p.splits + 1) <= ctx->sm_count && (p.splits + 1) * 2 <= p.num_kb) ++p.splits;
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
    p.stage_bytes = (uint32_t)(halves * FR_W_BYTES + pl.rows * FR_LINE);
    p.stages = std::min(FR_MAX_STAGES, (FR_SMEM - 1024) / (int)p.stage_bytes);
    p.stages = std::max(2, std::min(p.stages, (pl.num_kb + pl.splits - 1) / pl.splits));
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
    p.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(pl.rows >> 3) << 17) | ((uint32_t)(FR_FILTERS >> 4) << 24);
    p.tmem_cols = 32;
    while (p.tmem_cols < (uint32_t)(halves * pl.rows)) p.tmem_cols <<= 1;
    CUtensorMap tw, tx;
    const int nb = halves * g.N;
    if (!dlc_encode_operand(ctx, &tw, g.b, nb, (int)g.K, FR_FILTERS) ||
        !dlc_encode_operand(ctx, &tx, g.a, g.M, (int)g.K, pl.rows))
        return DLC_STATUS_EXECUTION_FAILED;
    const size_t need = std::max((size_t)p.stages * p.stage_bytes, (size_t)halves * pl.rows * FR_FILTERS * 4);
    const size_t smem = need + 1024;
    const void *kern = g.gated ? (e4m3 ? (const void *)gemm_rows_kernel<true, true> : (const void *)gemm_rows_kernel<false, true>)
                               : (e4m3 ? (const void *)gemm_rows_kernel<true, false> : (const void *)gemm_rows_kernel<false, false>);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
        cudaGetLastError();
        return DLC_STATUS_EXECUTION_FAILED;
    }
    void *args[] = {&p, &tw, &tx};
    return dlc_launch(ctx, kern, dim3((unsigned)(pl.filter_tiles * pl.splits), (unsigned)pl.row_tiles), dim3(FR_THREADS), smem,
                      args, pl.splits);
}

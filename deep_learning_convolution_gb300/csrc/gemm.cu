// gemm.cu -- the products of the linear and gated layers on pairs of SMs.
//
//   y[m, n] = act(sa[m] sb[n] sum_k a(m, k) b(n, k) + bias[n]) + r[m, n]
//   gated: y[m, n] = act(gate) * up, gate and up from rows n and N + n of b
//
// tcgen05.mma with cta_group::2: a cluster of two CTAs owns a tile of 256 rows
// and BN columns; each CTA brings its own 128 rows of a and half of the BN
// rows of b by TMA, and one MMA of M = 256, N = BN reads both CTAs' shared
// memory.  In the gated form the leader's half of b holds the gate's filters
// and the other CTA's the up filters of the same BN / 2 outputs, so gate and
// up of an output meet in one thread's accumulator row (columns j and
// BN / 2 + j) and neither projection touches memory before their product.
//
// The backward products read operands along their other axis (dx: w by
// channels; dw: both by rows): BF16 blocks of 64 x 64 with the output index
// contiguous, the tensor core's MN-major form, so nothing is transposed in
// memory.
//
// The tiles of a last wave that would leave most pairs idle (all tiles, where
// there are few) have their reduction split into ranges whose FP32 partial tiles
// go to the workspace; a second kernel adds them in a fixed order and applies the
// epilogue.
//
// Roles (11 warps a CTA): a thread of warp 0 loads a, one of warp 2 loads b, one of
// the leader's warp 1 issues the MMAs into one of two TMEM accumulators, warps
// 3-10 (two per quarter of the TMEM lanes, alternate 32-column chunks) run the
// epilogue of the other one.  Every wait is bounded.
//
// What bounds it: long reductions the tensor core under the power cap (gated 16384 x
// 4096 -> 2 x 8192 in E4M3 676 us, 3250 TFLOP/s, call after call; 16384 x 4096 -> 4096 in
// a burst of eight calls 284 us, 1940 TFLOP/s); short ones the epilogue, 2.9 us for a tile of 256
// columns in BF16 with a bias and up to 6 with GELU, residual and z, most of it
// instructions (hence the packed FP32 pairs); small ones the launch, about 5 us
// from call to call.  Loads, MMAs and bulk stores are issued by an elected thread: by
// lane 0, four MMAs took 260 cycles to issue instead of 67, and a k-block 0.32 us
// whatever its width.  Tried and slower: the epilogue's stores straight from
// registers, 64-column stores, two chunks at a time, bias and scales prefetched into
// registers (spills).
#include <cmath>
#include <cstring>

#include "channel.cuh"
#include "gemm.h"
#include "ptx.cuh"

namespace {

using namespace dlc;

constexpr int GP_ROWS = 128;                    // rows of a per CTA
constexpr int GP_LINE = 128;                    // bytes of a stage's operand rows (one swizzle span)
constexpr int GP_A_BYTES = GP_ROWS * GP_LINE;   // 16 KiB
constexpr int GP_ATOM = 64 * GP_LINE;           // MN-major: 64 indices x 64 of the reduction
constexpr int GP_EPI_WARP0 = 3, GP_EPI_WARPS = 8;
constexpr int GP_THREADS = (GP_EPI_WARP0 + GP_EPI_WARPS) * 32;
constexpr int GP_MAX_SMEM = 232448, GP_BAR_AREA = 256, GP_MAX_STAGES = 8;
constexpr int GP_COLUMNS = 2 * 256 * 4;         // scales and biases of a tile's columns

// Tiles in groups of eight row blocks (below), with the division by a group's size.
struct GpTiles {
    int m_tiles, n_tiles;
    uint32_t per, mul, shift;  // tiles of a group; t / per = (t * mul) >> (32 + shift)
};

struct GpParams {
    long long M;
    int N, act;
    int BN, nout;                 // accumulator columns of a tile, outputs of a tile (gated: BN / 2)
    int stages, num_kb;
    GpTiles tiles;
    int units;
    int full_tiles, splits;       // tiles from full_tiles on: `splits` units each, FP32 partial sums, no epilogue
    uint32_t b_stage;             // bytes of one CTA's half of b per stage
    int b_atoms;                  // MN-major b: 64-index blocks per CTA
    uint32_t idesc, tmem_cols, acc_stride;
    uint32_t epi_buf;             // bytes of one epilogue staging buffer
    const float *sa, *sb, *bias;
    RowTensor z, r, y;
    int y_tma, z_tma;
    int y_unit, z_unit;           // elements of an aligned access to y (where TMA cannot write it) and z
    int *err;
    unsigned long long timeout_ns;
};

struct GpUnit {
    long long m0;
    int nt, plane, kb0, kb1;  // plane: of the partial sums, or -1 for a whole tile
};

// Rows and column tile of tile t: groups of eight row blocks, so that the pairs
// that run together share rows of both operands in the L2.
// (Divisions are worked out without the divide where they can be: they and the
// kernel's other per-tile integer work are 1100 cycles of an epilogue otherwise.)
__device__ __forceinline__ void gp_tile(const GpTiles &g, int t, int &mt, int &nt) {
    const int grp = (int)(__umulhi((uint32_t)t, g.mul) >> g.shift), in = t - grp * (int)g.per;
    const int rows = g.m_tiles - grp * 8;
    nt = rows >= 8 ? in >> 3 : in / rows;
    mt = grp * 8 + in - nt * (rows >= 8 ? 8 : rows);
}

__device__ __forceinline__ GpUnit gp_unit(const GpParams &p, int u) {
    GpUnit w;
    int t = u, split = 0;
    w.plane = -1;
    w.kb0 = 0;
    w.kb1 = p.num_kb;
    if (u >= p.full_tiles) {
        w.plane = u - p.full_tiles;
        const int tail = w.plane / p.splits;
        split = w.plane - tail * p.splits;
        t = p.full_tiles + tail;
        w.kb0 = (int)((long long)p.num_kb * split / p.splits);
        w.kb1 = (int)((long long)p.num_kb * (split + 1) / p.splits);
    }
    int mt;
    gp_tile(p.tiles, t, mt, w.nt);
    w.m0 = (long long)mt * (2 * GP_ROWS);
    return w;
}

// One operand's loads: A's 128 rows of this CTA, or its half of B.
template <bool IS_A, bool MN, bool GATED, int BK>
__device__ void gp_produce(const GpParams &p, uint32_t rank, const CUtensorMap *tm, uint32_t smem, uint64_t *full,
                           uint64_t *empty, const WaitCtl &ctl) {
    const uint32_t bytes = IS_A ? (uint32_t)GP_A_BYTES : p.b_stage;
    const uint32_t tx = 2u * (GP_A_BYTES + p.b_stage);  // both CTAs' bytes land on the leader's barrier
    const uint32_t full0 = mapa_shared(smem_u32(full), 0);
    int stage = 0;
    uint32_t ph = 0;
    for (int u = (int)cluster_id_x(); u < p.units; u += (int)num_clusters_x()) {
        const GpUnit w = gp_unit(p, u);
        int i0;  // first index of this CTA's rows (or of its 64-index blocks)
        if (IS_A)
            i0 = (int)w.m0 + (int)rank * GP_ROWS;
        else if (GATED)
            i0 = w.nt * p.nout + (int)rank * p.N;
        else
            i0 = w.nt * p.BN + (int)rank * (p.BN / 2);
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
            if (!mbar_wait(&empty[stage], ph ^ 1u, ctl, 21)) return;
            if (IS_A && rank == 0) mbar_arrive_expect_tx(&full[stage], tx);
            const uint32_t dst = smem + (uint32_t)stage * bytes, bar = full0 + 8u * (uint32_t)stage;
            if (MN) {
                const int atoms = IS_A ? 2 : p.b_atoms;
                for (int a = 0; a < atoms; ++a) tma_load_2d_pair(dst + (uint32_t)a * GP_ATOM, tm, bar, i0 + 64 * a, kb * BK);
            } else {
                tma_load_2d_pair(dst, tm, bar, kb * BK, i0);
            }
            if (++stage == p.stages) stage = 0, ph ^= 1u;
        }
    }
}

template <bool E4M3, bool A_MN, bool B_MN>
__device__ void gp_mma(const GpParams &p, uint32_t tmem_base, uint32_t sA, uint32_t sB, uint64_t *full,
                       uint64_t *empty, uint64_t *tfull, uint64_t *tempty, uint64_t *mma_done, const WaitCtl &ctl) {
    // K-major rows advance 32 bytes per MMA; MN-major blocks 16 rows of 128 bytes
    const uint64_t a0 = A_MN ? sw128_mnmajor_desc(sA, GP_ATOM) : sw128_kmajor_desc(sA);
    const uint64_t b0 = B_MN ? sw128_mnmajor_desc(sB, GP_ATOM) : sw128_kmajor_desc(sB);
    constexpr uint64_t a_k = A_MN ? 16 * GP_LINE / 16 : 2, b_k = B_MN ? 16 * GP_LINE / 16 : 2;
    const uint64_t a_step = GP_A_BYTES >> 4, b_step = p.b_stage >> 4;
    int stage = 0, it = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int u = (int)cluster_id_x(); ok && u < p.units; u += (int)num_clusters_x(), ++it) {
        const GpUnit w = gp_unit(p, u);
        const int buf = it & 1;
        if (!mbar_wait_cluster(&tempty[buf], ((uint32_t)(it >> 1) & 1u) ^ 1u, ctl, 23)) {  // both CTAs' epilogues
            ok = false;
            break;
        }
        tc_fence_after_sync();
        const uint32_t d = tmem_base + (uint32_t)buf * p.acc_stride;
        uint32_t acc = 0;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
            if (!mbar_wait(&full[stage], ph, ctl, 24)) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            const uint64_t ad = a0 + a_step * (uint32_t)stage, bd = b0 + b_step * (uint32_t)stage;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (E4M3)
                    umma_e4m3_pair(d, ad + a_k * j, bd + b_k * j, p.idesc, acc);
                else
                    umma_bf16_pair(d, ad + a_k * j, bd + b_k * j, p.idesc, acc);
                acc = 1;
            }
            umma_commit_pair(&empty[stage], 3);  // both CTAs' slots free once these are done
            if (++stage == p.stages) stage = 0, ph ^= 1u;
        }
        if (!ok) break;
        umma_commit_pair(&tfull[buf], 3);  // both CTAs' accumulator rows are ready
    }
    if (!ok) {
        // gave up: loads issued for stages not consumed land on these barriers;
        // wait for them briefly so that no copy outlives the CTAs
        volatile int dummy = 0;
        const WaitCtl brief{&dummy, p.err, 50000000ull};
        for (int j = 0; j < p.stages; ++j) {
            if (!mbar_wait(&full[stage], ph, brief, 94)) break;
            if (++stage == p.stages) stage = 0, ph ^= 1u;
        }
    }
    umma_commit_pair(mma_done, 3);  // every MMA issued completes before tensor memory is released
}

// ---- epilogue --------------------------------------------------------------------

// The scales and biases of a tile's accumulator columns, to shared memory while
// the accumulator is on its way (from global memory where they are used, each
// 32-column chunk waited for them: 3000 x 640 -> 3008 18.2 us, 15.2 this way).
__device__ __forceinline__ void gp_columns(const GpParams &p, bool gated, int n0, float *columns) {
    const int i = (int)threadIdx.x - GP_EPI_WARP0 * 32;  // a column a thread
    if (i < p.BN) {
        const bool up = gated && i >= p.nout;
        const int n = n0 + (up ? i - p.nout : i);
        const long long k = (up ? (long long)p.N : 0) + n;
        columns[i] = p.sb && n < p.N ? p.sb[k] : 1.f;
        columns[256 + i] = p.bias && n < p.N ? p.bias[k] : 0.f;
    }
}

__device__ __forceinline__ void gp_epi_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(GP_EPI_WARPS * 32) : "memory"); }

// sa[m] sb[n] acc + bias[n] of 32 accumulator columns from `columns` on.
__device__ __forceinline__ void gp_scale_bias(const GpParams &p, float (&v)[32], float sa, const float *columns) {
    const float4 *c = reinterpret_cast<const float4 *>(columns);
    if (p.sb) {
        const float2 s = pair_of(sa);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 q = c[i];
            set2(v, 2 * i, mul2(get2(v, 2 * i), mul2(s, make_float2(q.x, q.y))));
            set2(v, 2 * i + 1, mul2(get2(v, 2 * i + 1), mul2(s, make_float2(q.z, q.w))));
        }
    }
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 q = c[64 + i];
            set2(v, 2 * i, add2(get2(v, 2 * i), make_float2(q.x, q.y)));
            set2(v, 2 * i + 1, add2(get2(v, 2 * i + 1), make_float2(q.z, q.w)));
        }
    }
}

// Where rows are written, or a residual read: by value (the kernel's parameters behind a
// reference would be loaded as memory, in the middle of the block).
struct GpRows {
    void *p;
    long long cs;
    int dt, unit;
};

// A staged 32 x 32 block (the warp's first `n` rows, `cols` columns) to rows that TMA
// cannot write: U elements a lane, U rows at a time, eight accesses in flight.
template <typename E, int U>
__device__ __forceinline__ void gp_store_units(GpRows t, uint32_t sb, int n, long long off, long long col, int cols, GpRows r,
                                               long long roff) {
    constexpr int LANES = 32 / U;  // of a row
    const int lane = threadIdx.x & 31, sub = lane / LANES, c = (lane - sub * LANES) * U;
    const long long tc = (col + c) * t.cs, rc = (col + c) * r.cs;
    const bool whole = c + U <= cols;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += 8 * U) {
        float f[8][U];
        long long o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t i = (uint32_t)(i0 + j * U + sub);
            const uint32_t at = sb + i * 128u + ((((uint32_t)c >> 2) ^ (i & 7u)) << 4) + ((uint32_t)c & 3u) * 4u;
            if constexpr (U == 4)
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(f[j][0]), "=f"(f[j][1]), "=f"(f[j][2]), "=f"(f[j][3]) : "r"(at) : "memory");
            else if constexpr (U == 2)
                asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(f[j][0]), "=f"(f[j][1]) : "r"(at) : "memory");
            else
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[j][0]) : "r"(at) : "memory");
        }
        if (r.p) {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = __shfl_sync(0xffffffffu, roff, i0 + j * U + sub) + rc;
            auto add = [&](auto *src) {
                using R = typename std::remove_const<typename std::remove_pointer<decltype(src)>::type>::type;
                R w[8][U];
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int k = 0; k < U; ++k) w[j][k] = c + k < cols && i0 + j * U + sub < n ? src[o[j] + k * r.cs] : (R)0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        if constexpr (sizeof(R) == 2)
                            f[j][k] += bf16_bits_f32(w[j][k]);
                        else
                            f[j][k] += w[j][k];
                    }
            };
            if (r.dt == DLC_DATA_BFLOAT16)
                add(static_cast<const unsigned short *>(r.p));
            else
                add(static_cast<const float *>(r.p));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = __shfl_sync(0xffffffffu, off, i0 + j * U + sub) + tc;
        E *dst = static_cast<E *>(t.p);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (i0 + j * U + sub >= n) continue;
            if (whole) {
                if constexpr (U == 1) {
                    store_elem(dst, sizeof(E) == 2 ? DLC_DATA_BFLOAT16 : DLC_DATA_FLOAT, o[j], f[j][0]);
                } else if constexpr (sizeof(E) == 2) {
                    uint32_t w[U / 2];
#pragma unroll
                    for (int k = 0; k < U / 2; ++k) w[k] = pack_bf16(f[j][2 * k], f[j][2 * k + 1]);
                    if constexpr (U == 4)
                        *reinterpret_cast<uint2 *>(dst + o[j]) = make_uint2(w[0], w[1]);
                    else
                        *reinterpret_cast<uint32_t *>(dst + o[j]) = w[0];
                } else if constexpr (U == 4) {
                    *reinterpret_cast<float4 *>(dst + o[j]) = make_float4(f[j][0], f[j][1], f[j][2], f[j][3]);
                } else {
                    *reinterpret_cast<float2 *>(dst + o[j]) = make_float2(f[j][0], f[j][1]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < U - 1; ++k)
                    if (c + k < cols) store_elem(dst, sizeof(E) == 2 ? DLC_DATA_BFLOAT16 : DLC_DATA_FLOAT, o[j] + k, f[j][k]);
            }
        }
    }
}

// Out of line: one copy for all activations, and only kernels of ROWS hold it.  It adds
// about 0.7 us a 32-column chunk to a tile's epilogue (204 x 2364 -> 1376's dw: 12.9 us,
// 10.5 with FP32 rows that TMA can write).
__device__ __noinline__ void gp_store_rows(GpRows t, uint32_t sb, int n, long long off, long long col, int cols, GpRows r,
                                           long long roff) {
    if (t.dt == DLC_DATA_BFLOAT16) {
        if (t.unit == 4) gp_store_units<unsigned short, 4>(t, sb, n, off, col, cols, r, roff);
        else if (t.unit == 2) gp_store_units<unsigned short, 2>(t, sb, n, off, col, cols, r, roff);
        else gp_store_units<unsigned short, 1>(t, sb, n, off, col, cols, r, roff);
    } else {
        if (t.unit == 4) gp_store_units<float, 4>(t, sb, n, off, col, cols, r, roff);
        else if (t.unit == 2) gp_store_units<float, 2>(t, sb, n, off, col, cols, r, roff);
        else gp_store_units<float, 1>(t, sb, n, off, col, cols, r, roff);
    }
}

// One warp's stores of 32 x 32 blocks: staged in shared memory, swizzled as the
// tensor map expects, then one bulk tensor store; or, for layouts that TMA
// cannot write, row by row with a lane per column.
struct GpStore {
    uint32_t bufs, buf_bytes;
    int nbuf, lane;
    long long row0;      // first row of the warp
    long long M;

    __device__ __forceinline__ uint32_t next() {
        const uint32_t sb = bufs + (uint32_t)(nbuf & 1) * buf_bytes;
        if (nbuf >= 2) {  // the store issued from this buffer two groups ago (the same thread is elected every time)
            if (elect_one()) bulk_wait_group_read<1>();
            __syncwarp();
        }
        ++nbuf;
        return sb;
    }

    __device__ __forceinline__ void stage_f32(uint32_t sb, const float (&v)[32]) const {
        const uint32_t rowp = sb + (uint32_t)lane * 128u;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(rowp + (((uint32_t)j ^ (lane & 7)) << 4)),
                         "f"(v[4 * j]), "f"(v[4 * j + 1]), "f"(v[4 * j + 2]), "f"(v[4 * j + 3])
                         : "memory");
    }

    __device__ __forceinline__ void tma(const CUtensorMap *tm, bool bf16, const float (&v)[32], int col, int plane) {
        if (row0 >= M) return;
        const uint32_t sb = next();
        if (bf16) {  // rows of 64 bytes, 64-byte swizzle
            const uint32_t rowp = sb + (uint32_t)lane * 64u;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 rowp + (((uint32_t)j ^ ((uint32_t)(lane >> 1) & 3u)) << 4)),
                             "r"(pack_bf16(v[8 * j], v[8 * j + 1])), "r"(pack_bf16(v[8 * j + 2], v[8 * j + 3])),
                             "r"(pack_bf16(v[8 * j + 4], v[8 * j + 5])), "r"(pack_bf16(v[8 * j + 6], v[8 * j + 7]))
                             : "memory");
        } else {
            stage_f32(sb, v);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (elect_one()) {  // rows past M and columns past N are not written
            tma_store_3d_s(tm, sb, col, (int)row0, plane);
            bulk_commit_group();
        }
    }

    // one block of a tile's partial sums
    __device__ __forceinline__ void partial(const CUtensorMap *tm, const float (&v)[32], int col, int row, int plane) {
        if (row0 >= M) return;
        const uint32_t sb = next();
        stage_f32(sb, v);
        fence_proxy_async_smem();
        __syncwarp();
        if (elect_one()) {
            tma_store_3d_s(tm, sb, col, row, plane);
            bulk_commit_group();
        }
    }

    // For layouts that TMA cannot write: a block staged (0 where the warp has no rows),
    // and then written.  `off`: this lane's row offset in t; `col`: column in t of
    // v[0], `cols` of them exist; r (or null), with `roff`: a residual added on the way.
    __device__ __forceinline__ uint32_t stage(const float (&v)[32]) {
        if (row0 >= M) return 0;
        const uint32_t sb = next();
        stage_f32(sb, v);
        __syncwarp();
        if (elect_one()) bulk_commit_group();  // an empty group keeps the buffers' turn
        return sb;
    }

    __device__ __forceinline__ void rows(const RowTensor &t, int unit, uint32_t sb, long long off, long long col, int cols,
                                         GpRows r = GpRows{nullptr, 0, 0, 1}, long long roff = 0) {
        if (!sb) return;
        gp_store_rows(GpRows{t.p, t.m.cs, t.dt, unit}, sb, (int)min(32LL, M - row0), off, col, cols, r, roff);
        __syncwarp();  // before the buffer's next turn
    }
};

// The last few values of a row (fewer than a 16-byte vector); out of line, since
// the code around them is on every tile's path.
__device__ __noinline__ uint4 gp_last_bf16(const unsigned short *src, int n) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < n) w[i >> 1] |= (uint32_t)src[i] << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __noinline__ float4 gp_last_f32(const float *src, int n) {
    return make_float4(src[0], n > 1 ? src[1] : 0.f, n > 2 ? src[2] : 0.f, 0.f);
}

// A lane's 32 residual values of a chunk (16-byte aligned rows; columns past
// `cols` are not read).  BF16 ones are loaded ahead of the chunk before, or of
// the accumulator; FP32 ones, twice the registers, where they are added.
struct GpResidual {
    uint4 q[4];
    int cols;

    __device__ __forceinline__ void load(const RowTensor &r, bool on, long long off, int columns) {
        cols = on && r.dt == DLC_DATA_BFLOAT16 ? columns : 0;
        const unsigned short *src = static_cast<const unsigned short *>(r.p) + off;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            q[j] = make_uint4(0u, 0u, 0u, 0u);
            if (8 * j + 8 <= cols) {
                q[j] = *reinterpret_cast<const uint4 *>(src + 8 * j);
            } else if (8 * j < cols) {
                q[j] = gp_last_bf16(src + 8 * j, cols - 8 * j);
            }
        }
    }

    __device__ __forceinline__ void add(const RowTensor &r, float (&v)[32], long long off, int columns) const {
        if (cols > 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t u[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    set2(v, 4 * j + i, add2(get2(v, 4 * j + i), unpack_bf16(u[i])));
                }
            }
        } else {
            const float *src = static_cast<const float *>(r.p) + off;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (4 * j + 4 <= columns) {
                    const float4 w = *reinterpret_cast<const float4 *>(src + 4 * j);
                    v[4 * j] += w.x, v[4 * j + 1] += w.y, v[4 * j + 2] += w.z, v[4 * j + 3] += w.w;
                } else if (4 * j < columns) {
                    const float4 w = gp_last_f32(src + 4 * j, columns - 4 * j);
                    v[4 * j] += w.x, v[4 * j + 1] += w.y, v[4 * j + 2] += w.z, v[4 * j + 3] += w.w;
                }
            }
        }
    }
};

template <bool GATED, bool ROWS, int ACT>
__device__ __forceinline__ void gp_epilogue(const GpParams &p, uint32_t rank, uint32_t tmem_base, uint64_t *tfull, uint64_t *tempty,
                            uint32_t epi_smem, float *columns, const CUtensorMap *tmY, const CUtensorMap *tmZ, const CUtensorMap *tmP,
                            const WaitCtl &ctl) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = warp & 3;                      // TMEM lanes 32*quad .. 32*quad+31
    const int part = (warp - GP_EPI_WARP0) >> 2;    // even or odd 32-column chunks
    const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0);
    GpStore st;
    st.bufs = epi_smem + (uint32_t)(warp - GP_EPI_WARP0) * 2u * p.epi_buf;
    st.buf_bytes = p.epi_buf;
    st.nbuf = 0;
    st.lane = lane;
    st.M = p.M;
    int it = 0;
    bool dead = false;  // a wait has given up: the rounds go on for the warps' barriers alone
    for (int u = (int)cluster_id_x(); u < p.units; u += (int)num_clusters_x(), ++it) {
        const GpUnit w = gp_unit(p, u);
        const int buf = it & 1;
        const long long m = w.m0 + (long long)rank * GP_ROWS + quad * 32 + lane;
        st.row0 = m - lane;
        const bool valid = m < p.M;
        const int n0 = w.nt * p.nout;
        // row offsets and the row's scale, worked out before the accumulator is ready
        long long zo = 0, ro = 0, yo = 0;
        float sa = 1.f;
        const bool raw = w.plane >= 0;
        if (valid && !raw) {
            if (ROWS && p.z.p) zo = row_off(p.z.m, m);
            if (p.r.p) ro = row_off(p.r.m, m);
            if (ROWS) yo = row_off(p.y.m, m);
            if (p.sa) sa = p.sa[m];
        }
        // (a gated layer has no residual; ROWS adds it where the rows are written)
        const bool res = !GATED && !ROWS && valid && !raw && p.r.p;
        GpResidual rq;
        if (!GATED && !ROWS) rq.load(p.r, res, ro + n0 + 32 * part, p.N - n0 - 32 * part);
        if (!raw && (p.sb || p.bias)) {
            gp_epi_barrier();  // the tile before has been read
            gp_columns(p, GATED, n0, columns);
            gp_epi_barrier();
        }
        int okw = 0;
        if (lane == 0 && !dead) okw = mbar_wait(&tfull[buf], (uint32_t)(it >> 1) & 1u, ctl, 25) ? 1 : 0;
        okw = __shfl_sync(0xffffffffu, okw, 0);
        dead = !okw;
        if (dead) continue;
        __syncwarp();
        tc_fence_after_sync();
        const uint32_t taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)buf * p.acc_stride;
        for (int c0 = 32 * part; c0 < p.nout && n0 + c0 < p.N; c0 += 64) {
            const int n = n0 + c0, cols = p.N - n;
            float v[32], up[GATED ? 32 : 1];
            {
                uint32_t a[32];
                tmem_ld_32x32b_x32(taddr + (uint32_t)c0, a);
                if constexpr (GATED) {
                    uint32_t b[32];
                    tmem_ld_32x32b_x32(taddr + (uint32_t)(p.nout + c0), b);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) up[i] = __uint_as_float(b[i]);
                } else {
                    tmem_ld_wait();
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(a[i]);
            }
            if (raw) {
                st.partial(tmP, v, c0, (int)rank * GP_ROWS + quad * 32, w.plane);
                if constexpr (GATED) st.partial(tmP, up, p.nout + c0, (int)rank * GP_ROWS + quad * 32, w.plane);
                continue;
            }
            gp_scale_bias(p, v, sa, columns + c0);
            if constexpr (GATED) gp_scale_bias(p, up, sa, columns + p.nout + c0);
            uint32_t z0 = 0, z1 = 0;  // blocks of z staged for rows
            if (p.z.p) {
                if (!ROWS || p.z_tma) {
                    st.tma(tmZ, p.z.dt == DLC_DATA_BFLOAT16, v, n, 0);
                    if constexpr (GATED) st.tma(tmZ, p.z.dt == DLC_DATA_BFLOAT16, up, n, 1);
                } else {
                    z0 = st.stage(v);
                    if constexpr (GATED) z1 = st.stage(up);
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float2 w = act_f2<ACT>(get2(v, i));
                if constexpr (GATED) w = mul2(w, get2(up, i));
                set2(v, i, w);
            }
            if constexpr (ROWS) {
                st.rows(p.z, p.z_unit, z0, zo, n, cols);
                st.rows(p.z, p.z_unit, z1, zo, (long long)p.N + n, cols);
            }
            if (!ROWS || (p.y_tma && !p.r.p)) {
                if (!GATED && !ROWS) {
                    if (res) rq.add(p.r, v, ro + n, cols);
                    rq.load(p.r, res && c0 + 64 < p.nout, ro + n + 64, cols - 64);
                }
                st.tma(tmY, p.y.dt == DLC_DATA_BFLOAT16, v, n, 0);
            } else if constexpr (ROWS) {
                st.rows(p.y, p.y_unit, st.stage(v), yo, n, cols, GpRows{p.r.p, p.r.m.cs, p.r.dt, 1}, ro);
            }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_tmem_free(tempty0 + 8u * (uint32_t)buf);
    }
    if (elect_one()) bulk_wait_group_read<0>();  // staged stores have read shared memory before the CTA exits
    __syncwarp();
}

// ROWS: y or z cannot be written by TMA, or the residual not be read in vectors.
template <bool E4M3, bool A_MN, bool B_MN, bool GATED, bool ROWS>
__global__ void __launch_bounds__(GP_THREADS, 1)
    gemm_pair_kernel(const __grid_constant__ GpParams p, const __grid_constant__ CUtensorMap tmA,
                     const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmY,
                     const __grid_constant__ CUtensorMap tmZ, const __grid_constant__ CUtensorMap tmP) {
    constexpr int BK = E4M3 ? GP_LINE : GP_LINE / 2;
    griddep_launch_dependents();
    extern __shared__ __align__(1024) uint8_t smem[];  // (the swizzled operands' alignment)
    const int ST = p.stages;
    uint8_t *smB = smem + (size_t)ST * GP_A_BYTES;
    uint8_t *epi = smB + (size_t)ST * p.b_stage;
    float *columns = reinterpret_cast<float *>(epi + GP_EPI_WARPS * 2 * p.epi_buf);
    uint64_t *full = reinterpret_cast<uint64_t *>(columns + 512);
    uint64_t *empty = full + ST;
    uint64_t *tfull = empty + ST;
    uint64_t *tempty = tfull + 2;
    uint64_t *mma_done = tempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
    const uint32_t rank = cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1u);   // the leader's expect-tx arrival (+ both CTAs' bytes)
            mbar_init(&empty[i], 1u);  // the leader's multicast commit
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1u);
            mbar_init(&tempty[i], 2u * GP_EPI_WARPS);  // every epilogue warp of both CTAs
        }
        mbar_init(mma_done, 1u);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == 0) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, p.tmem_cols);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any remote arrival
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    const WaitCtl ctl{abort_flag, p.err, p.timeout_ns};
    const uint32_t sA = smem_u32(smem), sB = smem_u32(smB);
    griddep_wait();  // no global memory before the grid ahead of this one is done

    if (warp == 0) {
        if (elect_one()) gp_produce<true, A_MN, GATED, BK>(p, rank, &tmA, sA, full, empty, ctl);
    } else if (warp == 2) {
        if (elect_one()) gp_produce<false, B_MN, GATED, BK>(p, rank, &tmB, sB, full, empty, ctl);
    } else if (warp == 1) {
        if (elect_one() && rank == 0)
            gp_mma<E4M3, A_MN, B_MN>(p, tmem_base, sA, sB, full, empty, tfull, tempty, mma_done, ctl);
    } else {
        // (the activation's branch out here: a block's code is straight)
        act_dispatch(p.act, [&](auto act) {
            gp_epilogue<GATED, ROWS, decltype(act)::value>(p, rank, tmem_base, tfull, tempty, smem_u32(epi), columns, &tmY, &tmZ, &tmP, ctl);
        });
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    // The leader's final commit reaches both CTAs.  Waited for here, when the tiles are
    // done: from the start of the kernel a long product would outlast a wait's limit.
    if (warp == 1) {
        if (elect_one()) {
            volatile int dummy = 0;
            const WaitCtl fin{&dummy, p.err, p.timeout_ns};
            mbar_wait(mma_done, 0u, fin, 93);
        }
        __syncwarp();
    }
    cluster_sync();  // neither CTA leaves while the pair's MMAs or loads may touch it
    tc_fence_after_sync();
    if (warp == 1) tmem_dealloc_pair(tmem_base, p.tmem_cols);
}

// ---- split reductions ----------------------------------------------------------------

struct FinishParams {
    GemmProblem g;
    const float *part;  // [tail tile][range][256][bn] FP32
    GpTiles tiles;
    int bn, nout, full_tiles, tail, splits;
    int vec;            // y, z and r take 4-element accesses
};

// Adds the partial tiles in the order of their ranges and applies the
// epilogue: four columns of a row a thread.  Bound by reading the partial sums
// from the L2, at about 5 TB/s with their writing.
__global__ void __launch_bounds__(256) gemm_finish_kernel(const __grid_constant__ FinishParams f) {
    griddep_launch_dependents();
    const GemmProblem &g = f.g;
    const int per_row = f.nout / 4, per_tile = 2 * GP_ROWS * per_row;
    const long long total = (long long)f.tail * per_tile;
    const int halves = g.gated ? 2 : 1;
    griddep_wait();
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
        const int t = (int)(i / per_tile), in = (int)(i - (long long)t * per_tile);
        const int r = in / per_row, c = (in - r * per_row) * 4;
        int mt, nt;
        gp_tile(f.tiles, f.full_tiles + t, mt, nt);
        const long long m = (long long)mt * (2 * GP_ROWS) + r;
        const int n = nt * f.nout + c, cols = g.N - n;
        if (m >= g.M || cols <= 0) continue;
        float v[2][4];
        for (int h = 0; h < halves; ++h) {
            const float *src = f.part + ((long long)t * f.splits * (2 * GP_ROWS) + r) * f.bn + h * f.nout + c;
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int sp = 0; sp < f.splits; ++sp) {
                const float4 q = *reinterpret_cast<const float4 *>(src + (long long)sp * (2 * GP_ROWS) * f.bn);
                s[0] += q.x, s[1] += q.y, s[2] += q.z, s[3] += q.w;
            }
            const float sa = g.sa ? g.sa[m] : 1.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const long long k = (long long)h * g.N + n + j;
                if (j < cols) {
                    if (g.sb) s[j] *= sa * g.sb[k];
                    if (g.bias) s[j] += g.bias[k];
                }
                v[h][j] = s[j];
            }
            if (g.z.p) store4(g.z, row_off(g.z.m, m), (long long)h * g.N + n, cols, f.vec && (h == 0 || g.N % 4 == 0), v[h]);
        }
        act_dispatch(g.act, [&](auto act) {
#pragma unroll
            for (int j = 0; j < 2; ++j) set2(v[0], j, act_f2<decltype(act)::value>(get2(v[0], j)));
        });
        if (g.gated) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[0][j] *= v[1][j];
        }
        if (g.r.p) {
            float r[4];
            load4(g.r, row_off(g.r.m, m), n, cols, f.vec, r);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[0][j] += r[j];
        }
        store4(g.y, row_off(g.y.m, m), n, cols, f.vec, v[0]);
    }
}

// ---- operands that TMA cannot load ------------------------------------------------------

// Operands copied to dense rows, each a multiple of 16 bytes long; those of a
// product, or of a backward pass's two, in one launch (blockIdx.z).  Bound by memory
// for large operands, by the launch for small ones (about 3 us in a call).
struct PackJob {
    RowTensor src;      // strides in units
    void *dst;
    long long ld, rows; // of the destination, in units
    int C, unit;        // units of a row, bytes of a unit
    int transposed;     // channels apart
    unsigned gx, gy;    // blocks of its own
};

struct PackParams {
    PackJob job[DLC_MAX_PACKS];
};

// Channels contiguous: a warp a row, eight units a lane in flight.
template <typename E>
__device__ __forceinline__ void pack_units(const PackJob &p) {
    const int lane = threadIdx.x & 31;
    const E *s = static_cast<const E *>(p.src.p);
    E *dst = static_cast<E *>(p.dst);
    for (long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); r < p.rows; r += (long long)p.gx * 8) {
        const E *from = s + row_off(p.src.m, r);
        for (int c0 = (int)blockIdx.y * 256 + lane; c0 < p.C; c0 += (int)p.gy * 256) {
            E v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c0 + 32 * i < p.C) v[i] = from[c0 + 32 * i];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c0 + 32 * i < p.C) dst[r * p.ld + c0 + 32 * i] = v[i];
        }
    }
}

// Channels apart: 32 x 32 elements through shared memory, read along the rows
// and written along the channels.
template <typename E>
__device__ __forceinline__ void pack_transposed(const PackJob &p, E (*tile)[33]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long r0 = (long long)blockIdx.x * 32;
    const E *s = static_cast<const E *>(p.src.p);
    E *dst = static_cast<E *>(p.dst);
    const long long ro = r0 + lane < p.rows ? row_off(p.src.m, r0 + lane) : 0;
    for (int c0 = (int)blockIdx.y * 32; c0 < p.C; c0 += (int)p.gy * 32) {
        __syncthreads();
#pragma unroll
        for (int i = warp; i < 32; i += 8)
            if (r0 + lane < p.rows && c0 + i < p.C) tile[lane][i] = s[ro + (long long)(c0 + i) * p.src.m.cs];
        __syncthreads();
#pragma unroll
        for (int i = warp; i < 32; i += 8)
            if (r0 + i < p.rows && c0 + lane < p.C) dst[(r0 + i) * p.ld + c0 + lane] = tile[i][lane];
    }
}

__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackParams params) {
    griddep_launch_dependents();
    __shared__ unsigned short tile[32][33];
    const PackJob &p = params.job[blockIdx.z];
    griddep_wait();
    if (blockIdx.x >= p.gx || blockIdx.y >= p.gy) return;
    if (p.transposed) {
        if (p.unit == 2)
            pack_transposed<unsigned short>(p, tile);
        else
            pack_transposed<unsigned char>(p, reinterpret_cast<unsigned char(*)[33]>(tile));
    } else if (p.unit == 8) {
        pack_units<uint2>(p);
    } else if (p.unit == 4) {
        pack_units<uint32_t>(p);
    } else if (p.unit == 2) {
        pack_units<unsigned short>(p);
    } else {
        pack_units<unsigned char>(p);
    }
}

// ---- host side ---------------------------------------------------------------------------

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// Rows of `ch` channels TMA can load: channels contiguous, one pitch (at least
// a row), 16-byte aligned.
bool tma_rows(const RowTensor &t, long long rows, long long ch) {
    const long long e = dlc_dtype_bytes((dlcDataType_t)t.dt);
    return t.m.cs == 1 && t.m.uniform && (uintptr_t)t.p % 16 == 0 &&
           (rows == 1 || ((t.m.ld * e) % 16 == 0 && t.m.ld >= ch && t.m.ld * e < (1LL << 40)));
}

// Rows of halves x `n` channels that TMA can store (each half its own plane).  A
// bulk tensor store writes whole pieces of 16 bytes: where a row ends inside one, what
// lies behind the row (a neighbour in a wider tensor, or the memory after the
// last row) would be overwritten, so rows have to be a multiple of 16 bytes long.
bool tma_store_rows(const RowTensor &t, long long rows, int n, int halves) {
    const long long e = dlc_dtype_bytes((dlcDataType_t)t.dt);
    return tma_rows(t, rows, (long long)n * halves) && ((long long)n * e) % 16 == 0;
}

bool vec16_rows(const RowTensor &t) {
    const long long e = dlc_dtype_bytes((dlcDataType_t)t.dt);
    auto mult = [&](long long s) { return (s * e) % 16 == 0; };
    return t.m.cs == 1 && (uintptr_t)t.p % 16 == 0 &&
           (t.m.uniform ? mult(t.m.ld) : (mult(t.m.s0) && mult(t.m.s2) && mult(t.m.s3)));
}

// Elements of the widest access (4, 2 or 1) that every row of t takes, and column `n` of it.
int store_unit(const RowTensor &t, long long n) {
    if (!t.p || t.m.cs != 1) return 1;
    const long long e = dlc_dtype_bytes((dlcDataType_t)t.dt);
    for (int u : {4, 2}) {
        auto mult = [&](long long s) { return s % u == 0; };
        if ((uintptr_t)t.p % (u * e) == 0 && mult(n) &&
            (t.m.uniform ? mult(t.m.ld) : (mult(t.m.s0) && mult(t.m.s2) && mult(t.m.s3))))
            return u;
    }
    return 1;
}

constexpr int GP_MAX_SPLITS = 16;

struct GemmPlan {
    int bn, nout, m_tiles, n_tiles, num_kb;
    int full_tiles, splits;     // tiles from full_tiles on are split
    long long a_rows, b_rows;
    int a_ch, b_ch;             // channels of the operands' rows
    bool pack_a, pack_b, few_rows, gemv;
    size_t a_off, b_off, part_off, bytes;
};

GemmPlan plan_gemm(const dlcContext *ctx, const GemmProblem &g) {
    GemmPlan p = {};
    const int nb = g.gated ? 2 * g.N : g.N;
    const bool e4m3 = g.a.t.dt == DLC_DATA_FLOAT8_E4M3;
    const int bk = e4m3 ? GP_LINE : GP_LINE / 2;
    p.a_rows = g.a.trans ? g.K : g.M;
    p.a_ch = (int)(g.a.trans ? g.M : g.K);
    p.b_rows = g.b.trans ? g.K : nb;
    p.b_ch = (int)(g.b.trans ? nb : g.K);
    p.gemv = dlc_gemv_ok(g);
    if (p.gemv) return p;  // operands as they are, one launch
    p.pack_a = !tma_rows(g.a.t, p.a_rows, p.a_ch);
    p.pack_b = !tma_rows(g.b.t, p.b_rows, p.b_ch);
    p.num_kb = (int)((g.K + bk - 1) / bk);
    p.m_tiles = (int)((g.M + 2 * GP_ROWS - 1) / (2 * GP_ROWS));
    // Tile width, split of the tail, and which of the two kernels, from a model of
    // the time in microseconds, fitted to 27 shapes from 128 x 1024 -> 512 to
    // 300 x 4096 -> 8192 and 12000 x 192 -> 256 and several epilogues each (its choice is
    // within 5 % of the fastest of up to ten alternatives).  A k-block takes a pair
    // 0.34 us for 256 columns and half that for 64 (the MMA thread's turn), a tile's
    // epilogue 2.9 and 1.5 us; it runs beside the next tile's k-blocks.  Pairs that a
    // last wave leaves idle are filled by splitting the reduction: that costs the
    // partial sums' way through the L2 and a launch.
    const int pairs = ctx->sm_count / 2;
    double best = 1e300;
    for (int bn : {256, 192, 128, 64}) {
        if (g.b.trans && bn % 128) continue;  // MN-major halves are whole 64-index blocks
        if (g.gated && bn % 128) continue;    // and a gated half whole 64-output chunk pairs
        const int nout = g.gated ? bn / 2 : bn, n_tiles = (g.N + nout - 1) / nout;
        const long long tiles = (long long)p.m_tiles * n_tiles;
        const double w = bn / 256.0, main = p.num_kb * std::max(0.161, 0.055 + 0.288 * w);
        const double epi = 0.97 - 0.62 * w + 2.55 * nout / 256.0, next = std::max(main, epi), fixed = 2.94;
        const long long tail = tiles % pairs, full = tiles / pairs;
        const double whole = full ? main + (double)(full - 1) * next + epi : 0.;
        for (int s = 1; s <= GP_MAX_SPLITS; ++s) {
            double t = fixed + whole;
            if (s == 1) {
                if (tail) t += full ? next : main + epi;
            } else {
                if (tail * s > pairs || 2 * s > p.num_kb) break;
                t += (double)((p.num_kb + s - 1) / s) / p.num_kb * main + 3.7 + (double)tail * s * 256 * bn * 8 / 5e6;
            }
            if (t < best) best = t, p.bn = bn, p.splits = s, p.full_tiles = (int)std::min(s == 1 ? tiles : tiles - tail, 0x7fffffffLL);
        }
    }
    // Up to 64 rows the filters' stream decides, which the few-row kernel carries
    // whatever the model says (gated 2048 -> 2 x 8192: 16 rows 14.3 us, the pair kernel 20.6,
    // 64 rows 15.1 and 16.7; at worst level, 64 x 512 -> 512 5.0 and 4.9).
    // Outputs that TMA cannot write cost the pair kernel's epilogue about another 4 us
    // for 256 columns (785 x 147 -> 1001: 12.1 us, the few-row kernel 11.0; 2842 x 848 ->
    // 114 with FP32 outputs 12.6 and 9.4).
    p.nout = g.gated ? p.bn / 2 : p.bn;
    p.n_tiles = (g.N + p.nout - 1) / p.nout;
    if (!g.a.trans && !g.b.trans) {
        const double waves = std::ceil((double)p.m_tiles * p.n_tiles / pairs);
        const double rows = tma_store_rows(g.y, g.M, g.N, 1) ? 0. : 4.0 * p.bn / 256 * waves;
        p.few_rows = g.M <= 64 || dlc_few_rows_plan(ctx, g).us < best + rows;
    } else {
        p.few_rows = false;
    }
    const long long tail = p.splits > 1 ? (long long)p.m_tiles * p.n_tiles - p.full_tiles : 0;
    size_t off = 0;
    p.a_off = off;
    if (p.pack_a) off += dlc_pack_bytes(g.a.t, p.a_rows, p.a_ch);
    p.b_off = off;
    if (p.pack_b) off += dlc_pack_bytes(g.b.t, p.b_rows, p.b_ch);
    p.part_off = off;
    if (!p.few_rows) off += round256((size_t)tail * p.splits * 2 * GP_ROWS * p.bn * 4);
    p.bytes = off;
    return p;
}

// The widest unit (bytes) that every row's address and length are multiples of.
int row_unit(const RowTensor &t, int ch) {
    const long long e = dlc_dtype_bytes((dlcDataType_t)t.dt);
    for (int u : {8, 4, 2}) {
        auto mult = [&](long long s) { return (s * e) % u == 0; };
        if ((uintptr_t)t.p % u == 0 && mult(ch) &&
            (t.m.uniform ? mult(t.m.ld) : (mult(t.m.s0) && mult(t.m.s2) && mult(t.m.s3))))
            return std::max(u, (int)e);
    }
    return (int)e;
}

// The copy of `t` ([rows][ch]) to `dst`.
PackJob pack_job(const dlcContext *ctx, const RowTensor &t, long long rows, int ch, void *dst) {
    const int e = dlc_dtype_bytes((dlcDataType_t)t.dt);
    const long long ld = (((long long)ch * e + 15) / 16 * 16) / e;
    PackJob j;
    j.src = t;
    j.dst = dst;
    j.rows = rows;
    j.transposed = t.m.cs != 1;
    j.unit = j.transposed ? e : row_unit(t, ch);
    const int per = j.unit / e;
    j.src.m.ld /= per, j.src.m.s0 /= per, j.src.m.s2 /= per, j.src.m.s3 /= per;
    j.ld = ld / per;
    j.C = ch / per;
    // enough blocks to fill the GPU: rows first, then a row's channels
    const long long most = (long long)ctx->sm_count * (j.transposed ? 16 : 8);
    const long long gx = j.transposed ? (rows + 31) / 32 : std::min<long long>((rows + 7) / 8, most);
    const long long spans = j.transposed ? (j.C + 31) / 32 : (j.C + 255) / 256;
    j.gx = (unsigned)gx;
    j.gy = (unsigned)std::min<long long>(spans, std::max<long long>(1, most / gx));
    return j;
}

bool encode(const dlcContext *ctx, CUtensorMap *tm, const RowTensor &t, int nd, const cuuint64_t *dim, long long plane,
            cuuint32_t box0, cuuint32_t box1, CUtensorMapSwizzle swz) {
    const cuuint64_t e = (cuuint64_t)dlc_dtype_bytes((dlcDataType_t)t.dt);
    const cuuint64_t str[2] = {(cuuint64_t)t.m.ld * e, (cuuint64_t)plane * e};
    const cuuint32_t box[3] = {box0, box1, 1}, ones[3] = {1, 1, 1};
    const CUtensorMapDataType dt = t.dt == DLC_DATA_FLOAT ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : t.dt == DLC_DATA_BFLOAT16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                               : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    return ctx->encode_tiled(tm, dt, (cuuint32_t)nd, t.p, dim, str, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An output's map: `halves` planes of [M][N], 32 x 32 blocks.
bool encode_output(const dlcContext *ctx, CUtensorMap *tm, const RowTensor &o, long long M, int N, int planes,
                   long long plane) {
    RowTensor t = o;
    if (M == 1) t.m.ld = ((long long)N * planes + 15) / 16 * 16;
    const cuuint64_t dim[3] = {(cuuint64_t)N, (cuuint64_t)M, (cuuint64_t)planes};
    return encode(ctx, tm, t, 3, dim, planes > 1 ? plane : t.m.ld, 32, 32,
                  t.dt == DLC_DATA_FLOAT ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

template <bool ROWS>
const void *pair_kernel(bool e4m3, bool a_mn, bool b_mn, bool gated) {
    if (gated)
        return e4m3 ? (const void *)gemm_pair_kernel<true, false, false, true, ROWS>
                    : (const void *)gemm_pair_kernel<false, false, false, true, ROWS>;
    if (e4m3) return (const void *)gemm_pair_kernel<true, false, false, false, ROWS>;
    if (a_mn) return (const void *)gemm_pair_kernel<false, true, true, false, ROWS>;
    return b_mn ? (const void *)gemm_pair_kernel<false, false, true, false, ROWS>
                : (const void *)gemm_pair_kernel<false, false, false, false, ROWS>;
}

// Pairs that the device holds at once (each CTA takes an SM's shared memory).
int resident_pairs(dlcContext *ctx) {
    return dlc_resident_clusters(ctx, &ctx->resident_pairs, (const void *)gemm_pair_kernel<false, false, false, false, false>, 2,
                                 GP_THREADS, GP_MAX_SMEM);
}

GpTiles tiles_of(const GemmPlan &pl) {
    GpTiles t;
    t.m_tiles = pl.m_tiles;
    t.n_tiles = pl.n_tiles;
    // exact for tile numbers below 2^31: mul = ceil(2^(32 + shift) / per) with
    // 2^shift >= per / 2 leaves an error below 2^31 * per / 2^(32 + shift) <= 1 ulp
    t.per = 8u * (uint32_t)pl.n_tiles;
    t.shift = 0;
    while ((2ull << t.shift) < t.per) ++t.shift;
    t.mul = (uint32_t)(((1ull << (32 + t.shift)) + t.per - 1) / t.per);
    return t;
}

dlcStatus_t launch_pair(dlcContext *ctx, const GemmProblem &g, const GemmPlan &pl) {
    const bool e4m3 = g.a.t.dt == DLC_DATA_FLOAT8_E4M3;
    GpParams p;
    std::memset(&p, 0, sizeof(p));
    p.M = g.M;
    p.N = g.N;
    p.act = g.act;
    p.BN = pl.bn;
    p.nout = pl.nout;
    p.num_kb = pl.num_kb;
    p.tiles = tiles_of(pl);
    if ((long long)pl.m_tiles * pl.n_tiles > 0x7fffffffLL) return DLC_STATUS_NOT_SUPPORTED;
    const int tail = pl.m_tiles * pl.n_tiles - pl.full_tiles;
    p.full_tiles = pl.full_tiles;
    p.splits = pl.splits;
    p.units = pl.full_tiles + tail * pl.splits;
    p.b_atoms = pl.bn / 128;
    p.b_stage = (uint32_t)(pl.bn / 2) * GP_LINE;
    p.sa = g.sa;
    p.sb = g.sb;
    p.bias = g.bias;
    p.z = g.z;
    p.r = g.r;
    p.y = g.y;
    p.err = ctx->d_err;
    p.timeout_ns = ctx->timeout_ns;
    const uint32_t fmt = e4m3 ? 0u : 1u;
    p.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)g.a.trans << 15) | ((uint32_t)g.b.trans << 16) |
              ((uint32_t)(pl.bn >> 3) << 17) | ((uint32_t)((2 * GP_ROWS) >> 4) << 24);
    p.tmem_cols = 32;
    while (p.tmem_cols < (uint32_t)(2 * pl.bn)) p.tmem_cols <<= 1;
    p.acc_stride = p.tmem_cols / 2;

    CUtensorMap ta, tb, ty, tz, tp;
    std::memset(&ty, 0, sizeof(ty));
    std::memset(&tz, 0, sizeof(tz));
    std::memset(&tp, 0, sizeof(tp));
    if (!dlc_encode_operand(ctx, &ta, g.a, pl.a_rows, pl.a_ch, GP_ROWS) ||
        !dlc_encode_operand(ctx, &tb, g.b, pl.b_rows, pl.b_ch, pl.bn / 2))
        return DLC_STATUS_EXECUTION_FAILED;
    p.y_tma = tma_store_rows(g.y, g.M, g.N, 1);
    p.z_tma = g.z.p && tma_store_rows(g.z, g.M, g.N, g.gated ? 2 : 1);
    p.y_unit = store_unit(g.y, 0);
    p.z_unit = store_unit(g.z, g.gated ? g.N : 0);
    if (p.y_tma && !encode_output(ctx, &ty, g.y, g.M, g.N, 1, 0)) return DLC_STATUS_EXECUTION_FAILED;
    if (p.z_tma && !encode_output(ctx, &tz, g.z, g.M, g.N, g.gated ? 2 : 1, g.N)) return DLC_STATUS_EXECUTION_FAILED;
    if (tail) {
        RowTensor part;
        part.p = g.ws + pl.part_off;
        part.dt = DLC_DATA_FLOAT;
        part.m.ld = pl.bn;
        if (!encode_output(ctx, &tp, part, 2 * GP_ROWS, pl.bn, tail * pl.splits, 2LL * GP_ROWS * pl.bn))
            return DLC_STATUS_EXECUTION_FAILED;
    }
    const bool rows = !p.y_tma || (g.r.p && !vec16_rows(g.r)) || (g.z.p && !p.z_tma);
    const bool f32_stage = tail || rows || g.y.dt == DLC_DATA_FLOAT || (g.z.p && g.z.dt == DLC_DATA_FLOAT);
    p.epi_buf = f32_stage ? 4096 : 2048;
    const int epi_bytes = GP_EPI_WARPS * 2 * (int)p.epi_buf;
    const int stage_bytes = GP_A_BYTES + (int)p.b_stage;
    p.stages = std::min(GP_MAX_STAGES, (GP_MAX_SMEM - GP_COLUMNS - GP_BAR_AREA - epi_bytes) / stage_bytes);
    const size_t smem = (size_t)p.stages * stage_bytes + epi_bytes + GP_COLUMNS + GP_BAR_AREA;
    const bool a_mn = g.a.trans != 0, b_mn = g.b.trans != 0, gated = g.gated != 0;
    const void *kern = rows ? pair_kernel<true>(e4m3, a_mn, b_mn, gated) : pair_kernel<false>(e4m3, a_mn, b_mn, gated);
    if (!dlc_allow_smem(ctx, kern, smem)) return DLC_STATUS_EXECUTION_FAILED;
    const int clusters = std::min(resident_pairs(ctx), p.units);
    void *args[] = {&p, &ta, &tb, &ty, &tz, &tp};
    dlcStatus_t st = dlc_launch(ctx, kern, dim3((unsigned)(2 * clusters)), dim3(GP_THREADS), smem, args, 2);
    if (st != DLC_STATUS_SUCCESS || !tail) return st;
    FinishParams f;
    f.g = g;
    f.part = reinterpret_cast<const float *>(g.ws + pl.part_off);
    f.bn = pl.bn;
    f.nout = pl.nout;
    f.tiles = p.tiles;
    f.full_tiles = pl.full_tiles;
    f.tail = tail;
    f.splits = pl.splits;
    f.vec = dlc_vec4_rows(g.y) && dlc_vec4_rows(g.z) && dlc_vec4_rows(g.r);
    const long long items = (long long)tail * 2 * GP_ROWS * (pl.nout / 4);
    const long long blocks = std::min<long long>((items + 255) / 256, (long long)ctx->sm_count * 8);
    void *fargs[] = {&f};
    return dlc_launch(ctx, (const void *)gemm_finish_kernel, dim3((unsigned)blocks), dim3(256), 0, fargs);
}

}  // namespace

// A row operand's map: K-major boxes of 128 bytes x `box_rows` rows, or
// MN-major blocks of 64 channels x 64 rows.
bool dlc_encode_operand(const dlcContext *ctx, CUtensorMap *tm, const GemmOperand &o, long long rows, int ch, int box_rows) {
    RowTensor t = o.t;
    const int e = dlc_dtype_bytes((dlcDataType_t)t.dt);
    if (rows == 1) t.m.ld = ((long long)ch * e + 15) / 16 * 16 / e;
    const cuuint64_t dim[2] = {(cuuint64_t)ch, (cuuint64_t)rows};
    return encode(ctx, tm, t, 2, dim, 0, (cuuint32_t)(GP_LINE / e), (cuuint32_t)(o.trans ? 64 : box_rows),
                  CU_TENSOR_MAP_SWIZZLE_128B);
}

size_t dlc_pack_bytes(const RowTensor &t, long long rows, int ch) {
    const long long e = dlc_dtype_bytes((dlcDataType_t)t.dt);
    return tma_rows(t, rows, ch) ? 0 : round256((size_t)rows * ((ch * e + 15) / 16 * 16));
}

RowTensor dlc_packed(const RowTensor &t, int ch, void *dst) {
    const long long e = dlc_dtype_bytes((dlcDataType_t)t.dt), ld = (ch * e + 15) / 16 * 16 / e;
    RowTensor d = t;
    d.p = dst;
    d.m = RowMap{ld, 0, 0, 1, ld, 1, 1, 1};
    return d;
}

dlcStatus_t dlc_launch_pack(dlcContext *ctx, const PackItem *items, int n) {
    if (n == 0) return DLC_STATUS_SUCCESS;
    PackParams pk;
    dim3 grid(1, 1, (unsigned)n);
    for (int i = 0; i < DLC_MAX_PACKS; ++i) {
        const PackItem &it = items[std::min(i, n - 1)];
        pk.job[i] = pack_job(ctx, *it.t, it.rows, it.ch, it.dst);
        grid.x = std::max(grid.x, pk.job[i].gx);
        grid.y = std::max(grid.y, pk.job[i].gy);
    }
    for (int i = 0; i < n; ++i) *items[i].t = dlc_packed(*items[i].t, items[i].ch, items[i].dst);
    void *args[] = {&pk};
    return dlc_launch(ctx, (const void *)pack_kernel, grid, dim3(256), 0, args);
}

dlcKernel_t dlc_gemm_variant(const dlcContext *ctx, const GemmProblem &g) {
    const GemmPlan p = plan_gemm(ctx, g);
    return p.gemv ? DLC_KERNEL_GEMV : p.few_rows ? DLC_KERNEL_FEW_ROWS : DLC_KERNEL_GEMM_PAIR;
}

size_t dlc_gemm_workspace(const dlcContext *ctx, const GemmProblem &g) { return plan_gemm(ctx, g).bytes; }

dlcStatus_t dlc_launch_gemm(dlcContext *ctx, const GemmProblem &pb) {
    GemmProblem g = pb;
    const GemmPlan pl = plan_gemm(ctx, g);
    PackItem pk[DLC_MAX_PACKS];
    int packs = 0;
    if (pl.pack_a) pk[packs++] = PackItem{&g.a.t, pl.a_rows, pl.a_ch, g.ws + pl.a_off};
    if (pl.pack_b) pk[packs++] = PackItem{&g.b.t, pl.b_rows, pl.b_ch, g.ws + pl.b_off};
    const dlcStatus_t st = dlc_launch_pack(ctx, pk, packs);
    if (st != DLC_STATUS_SUCCESS) return st;
    if (pl.gemv) return dlc_launch_gemv(ctx, g);
    return pl.few_rows ? dlc_launch_few_rows(ctx, g) : launch_pair(ctx, g, pl);
}

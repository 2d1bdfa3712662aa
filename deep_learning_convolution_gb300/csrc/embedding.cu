// embedding.cu -- rows of a table by token, and the table's gradient.
//
//   y[m] = scale * table[token[m]], 0 for a negative token
//   dtable[v] = (dtable[v]) + scale * sum over m with token[m] = v of dy[m]
//
// Forward: a copy with an address a row; bound by memory (16384 x 2048 BF16 23.3 us, 5.8 TB/s), or by the
// launch for few rows (64 x 4096 2.3 us).
//
// Backward: the tokens are sorted by a stable radix sort (so that the rows of a token stay
// in order and the FP32 sums are the same every time); blocks then take runs of 16 to
// 128 sorted positions and a slab of channels and add the rows of each token up in
// registers.  A token whose rows reach over several blocks leaves a partial sum in each,
// which a last kernel adds in order: a token that is every tenth one costs no more than
// the others.  The table is zeroed beside the sort, whose own time is latency, and the
// tokens' rows then written over.  16384 x 2048 BF16 into 65536 rows 70 us (the rows read, the table
// written: 4.8 TB/s; three launches that sort and zero are 46 us of it, at 5.8 TB/s, the sums 15, the
// join 5); zeroed beside the sums instead, by a flag a row, 120 us.  Small calls are their four
// launches: 5000 x 300 FP32 added to a table 17 us, 4000 x 300 into one 12.7.
#include "channel.cuh"
#include "ptx.cuh"

namespace {

using namespace dlc;

constexpr int EM_THREADS = 256, EM_BLOCKS = 3;  // blocks of whole vectors an SM holds

__device__ __forceinline__ long long token_at(const IndexList &t, long long i) {
    return t.wide ? static_cast<const long long *>(t.p)[i] : static_cast<const int *>(t.p)[i];
}

// W channels of a row: 8 or 4 neighbours in one or two accesses, or (APART) single ones `hop` elements apart, of
// which n exist.
template <int W, bool APART, typename T>
struct Words {
    alignas(W * sizeof(T) < 16 ? W * sizeof(T) : 16) T v[W];
    __device__ __forceinline__ void load(const T *p, long long hop, int n) {
        if constexpr (APART) {
            if (n >= W) {
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] = p[j * hop];
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] = j < n ? p[j * hop] : (T)0;
            }
        } else if constexpr (W * sizeof(T) >= 16) {
#pragma unroll
            for (int j = 0; j < W * (int)sizeof(T) / 16; ++j) reinterpret_cast<uint4 *>(v)[j] = reinterpret_cast<const uint4 *>(p)[j];
        } else {
            static_assert(W * sizeof(T) == 8, "");
            *reinterpret_cast<uint2 *>(v) = *reinterpret_cast<const uint2 *>(p);
        }
    }
    __device__ __forceinline__ float at(int j) const {
        if constexpr (sizeof(T) == 2)
            return bf16_bits_f32(v[j]);
        else
            return v[j];
    }
};

template <int W, bool APART, typename T>
__device__ __forceinline__ void store_words(T *dst, int hop, int n, const float (&f)[W]) {
    if constexpr (APART) {
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (j < n) store_elem(dst + j * hop, sizeof(T) == 2 ? DLC_DATA_BFLOAT16 : DLC_DATA_FLOAT, 0, f[j]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < W / 4; ++j)
            reinterpret_cast<float4 *>(dst)[j] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
    } else if constexpr (W == 8) {
        *reinterpret_cast<uint4 *>(dst) =
            make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    } else {
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
    }
}

// ---- forward -----------------------------------------------------------------------

struct EmParams {
    EmbeddingProblem e;
    long long items;
    int pieces;  // of a row
    int *err;
};

// BF16 to BF16, eight channels a piece in 16-byte accesses.  U pieces a thread are in flight together, and the
// tokens of the next ones.
__global__ void __launch_bounds__(EM_THREADS, EM_BLOCKS) embedding_kernel(const __grid_constant__ EmParams p) {
    griddep_launch_dependents();
    constexpr int W = 8, U = 4;
    using T = unsigned short;
    const long long step = (long long)gridDim.x * EM_THREADS;
    long long i = (long long)blockIdx.x * EM_THREADS + threadIdx.x;
    uint32_t row = (uint32_t)(i / p.pieces);  // (may run past the last one)
    int piece = (int)(i - (long long)row * p.pieces);
    const int drow = (int)(step / p.pieces), dpiece = (int)(step - (long long)drow * p.pieces);
    griddep_wait();
    long long token[U];
    int at_row[U], at_piece[U];
    // the next U pieces' places and tokens (row -1: none)
    auto next = [&]() {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            at_row[k] = i < p.items ? (int)row : -1;
            at_piece[k] = piece;
            token[k] = i < p.items ? token_at(p.e.tokens, row) : -1;
            i += step, row += drow, piece += dpiece;
            if (piece >= p.pieces) piece -= p.pieces, ++row;
        }
    };
    next();
    while (at_row[0] >= 0) {
        Words<W, false, T> v[U];
        long long at[U];
        bool there[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            there[k] = token[k] >= 0 && token[k] < p.e.V;
            at[k] = at_row[k] < 0 ? -1 : row_off(p.e.y.m, at_row[k]) + (long long)at_piece[k] * W * p.e.y.m.cs;
            if (there[k]) v[k].load(static_cast<const T *>(p.e.table.p) + token[k] * p.e.C + (long long)at_piece[k] * W, 1, W);
            if (token[k] >= p.e.V && at_piece[k] == 0) record_error(p.err, DLC_DEVERR_INDEX, at_row[k]);
        }
        next();
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (at[k] < 0) break;
            float f[W];
#pragma unroll
            for (int j = 0; j < W; ++j) f[j] = there[k] ? v[k].at(j) * p.e.scale : 0.f;
            store_words<W, false, T>(static_cast<T *>(p.e.y.p) + at[k], 1, W, f);
        }
    }
}

// FP32 on either side, rows that vectors do not reach, and any layout of y: a warp takes up to 256 channels of a
// row, single ones 32 apart a lane.  16384 x 1001 BF16 14.7 us (43.8 with a place in the rows and an address
// for each element), 16384 x 1008 FP32 14.5, in vectors of four channels 15.7, of eight 21.0.
constexpr int EM_LANE = 8, EM_ROW_BLOCKS = 6;  // channels a lane; blocks an SM holds

template <typename T, typename Y>
__global__ void __launch_bounds__(EM_THREADS, EM_ROW_BLOCKS) embedding_rows_kernel(const __grid_constant__ EmParams p) {
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long step = (long long)gridDim.x * (EM_THREADS / 32);
    long long i = (long long)blockIdx.x * (EM_THREADS / 32) + (threadIdx.x >> 5);
    long long row = i / p.pieces;
    int piece = (int)(i - row * p.pieces);
    const long long drow = step / p.pieces;
    const int dpiece = (int)(step - drow * p.pieces);
    griddep_wait();
    long long token = i < p.items ? token_at(p.e.tokens, row) : -1;
    while (i < p.items) {
        const int c = piece * 32 * EM_LANE + lane;
        const bool there = token >= 0 && token < p.e.V;
        const T *src = static_cast<const T *>(p.e.table.p) + token * p.e.C + c;
        Y *dst = static_cast<Y *>(p.e.y.p) + row_off(p.e.y.m, row) + c * p.e.y.m.cs;
        T v[EM_LANE];
#pragma unroll
        for (int j = 0; j < EM_LANE; ++j) v[j] = there && c + 32 * j < p.e.C ? src[32 * j] : (T)0;
        if (token >= p.e.V && c == 0) record_error(p.err, DLC_DEVERR_INDEX, (int)row);
        i += step, row += drow, piece += dpiece;
        if (piece >= p.pieces) piece -= p.pieces, ++row;
        if (i < p.items) token = token_at(p.e.tokens, row);
#pragma unroll
        for (int j = 0; j < EM_LANE; ++j) {
            if (c + 32 * j >= p.e.C) break;
            float f;
            if constexpr (sizeof(T) == 2)
                f = bf16_bits_f32(v[j]);
            else
                f = v[j];
            store_elem(dst + 32 * j * p.e.y.m.cs, sizeof(Y) == 2 ? DLC_DATA_BFLOAT16 : DLC_DATA_FLOAT, 0, there ? f * p.e.scale : 0.f);
        }
    }
}

// ---- the tokens in order -------------------------------------------------------------
//
// Least significant digit first, a digit at most ten bits.  A tile keeps its tokens in
// registers; the histograms of all tiles give every digit's place (the next pass's
// are counted while this one writes).  Tokens outside the table sort behind all others,
// as number V.

constexpr int SORT_MAX_BITS = 10, SORT_MAX_DIGITS = 1 << SORT_MAX_BITS;

constexpr int SORT_THREADS = 512, SORT_WARPS = SORT_THREADS / 32, SORT_EACH = 4, SORT_TILE = SORT_THREADS * SORT_EACH;
// Short lists are ranked by counting, in one launch: up to 4096 tokens where a digit would do for sorting them (300
// channels into 1003 rows: 4000 tokens 12.9 us, by digits 16.9; 5000 tokens 16.4 and 16.0; 8000 21.7 and 16.8), up
// to RANK_MOST where it takes two (64 channels into 131072 rows: 5000 tokens 19.0 us, 24.8 by digits; 8000 27.9
// and 25.6).
constexpr int RANK_ONE = 4096, RANK_MOST = 6144, RANK_THREADS = 256;
constexpr int SORT_OWN_SUMS = 64;  // tiles

struct SortParams {
    IndexList tokens;
    int rows, V, tiles;
    int bits, passes;       // of a digit; of the sort
    int *hist;              // [pass][tile][digit]; a last row for the totals
    int scanned;            // hist holds the counts of the tiles ahead, and the totals
    uint32_t *key[2], *row[2];  // pass p writes the arrays p mod 2
    int *err;
    int blocks;                 // that sort; those behind them zero this launch's part of the table
    char *fill;                 // (16-byte aligned)
    long long fill_words;       // of 16 bytes
    char *edge[2];              // bytes of the table before and behind its whole words (first launch)
    int edge_bytes[2];
};

// What the blocks behind the sorting ones do, whose time is latency: the table's rows are zeroed, all
// of them, a part in each of the sort's launches.
__device__ __forceinline__ void fill_part(const SortParams &p) {
    const long long me = (long long)((int)blockIdx.x - p.blocks) * blockDim.x + threadIdx.x;
    const long long all = (long long)((int)gridDim.x - p.blocks) * blockDim.x;
    uint4 *dst = reinterpret_cast<uint4 *>(p.fill);
    long long i = me;
    for (; i + 3 * all < p.fill_words; i += 4 * all) {
#pragma unroll
        for (int k = 0; k < 4; ++k) dst[i + k * all] = make_uint4(0u, 0u, 0u, 0u);
    }
    for (; i < p.fill_words; i += all) dst[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (me < p.edge_bytes[k]) p.edge[k][me] = 0;
}

struct SortShared {
    unsigned short count[SORT_WARPS][SORT_MAX_DIGITS];  // of a warp's tokens, then the warps before it
    int base[SORT_MAX_DIGITS];
    int sums[SORT_WARPS];
};

__device__ __forceinline__ uint32_t sort_key(const SortParams &p, int i) {
    const long long t = token_at(p.tokens, i);
    if (t >= p.V) record_error(p.err, DLC_DEVERR_INDEX, i);
    return t < 0 || t >= p.V ? (uint32_t)p.V : (uint32_t)t;
}

// base[d] = the place of this tile's first token of digit d: totals summed over smaller
// digits, and `before` of d in the tiles ahead.  Two digits a thread.
__device__ __forceinline__ void sort_places(SortShared &s, const int (&total)[2], const int (&before)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int own = total[0] + total[1];
    int sum = own;
    for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) s.sums[warp] = sum;
    __syncthreads();
    int start = sum - own;
    for (int w = 0; w < warp; ++w) start += s.sums[w];
    s.base[2 * threadIdx.x] = start + before[0];
    s.base[2 * threadIdx.x + 1] = start + total[0] + before[1];
}

// Ranks of a tile's tokens among those of the same digit; keys[k] of thread t is the tile's
// token warp * 128 + 32 k + lane.  Leaves each warp's counts in s.count.
__device__ __forceinline__ void sort_ranks(SortShared &s, const uint32_t (&keys)[SORT_EACH], const bool (&on)[SORT_EACH], int shift,
                                           uint32_t mask, int (&rank)[SORT_EACH]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < SORT_EACH; ++k) {
        const uint32_t d = on[k] ? (keys[k] >> shift) & mask : 0xffffffffu;
        const uint32_t peers = __match_any_sync(0xffffffffu, d);
        const uint32_t ahead = peers & ((1u << lane) - 1u);
        int first = 0;
        if (on[k]) first = s.count[warp][d];
        __syncwarp();
        rank[k] = first + __popc(ahead);
        if (on[k] && ahead == 0) s.count[warp][d] = (unsigned short)(first + __popc(peers));
        __syncwarp();
    }
}

// s.count: from each warp's counts to the sum of those of the warps before it.
__device__ __forceinline__ void sort_warps(SortShared &s) {
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int d = 2 * (int)threadIdx.x + h;
        int sum = 0;
        for (int w = 0; w < SORT_WARPS; ++w) {
            const int c = s.count[w][d];
            s.count[w][d] = (unsigned short)sum;
            sum += c;
        }
    }
}

// Short lists: a token's place is how many come before it, counted over all of them.  A block ranks 32
// tokens, a lane each, its warps dealing with a part of the list each; in one launch and without
// steps that wait for one another (a block that sorted 5000 tokens alone took 10 us).
__global__ void __launch_bounds__(RANK_THREADS) rank_kernel(const __grid_constant__ SortParams p) {
    griddep_launch_dependents();
    __shared__ uint4 key_s[RANK_MOST / 4];
    __shared__ int part[RANK_THREADS / 32][32];
    griddep_wait();
    if ((int)blockIdx.x >= p.blocks) {
        fill_part(p);
        return;
    }
    uint32_t *keys = reinterpret_cast<uint32_t *>(key_s);
    constexpr int U = 8;
    for (int i0 = threadIdx.x; i0 < p.rows; i0 += U * RANK_THREADS) {
        long long t[U];
#pragma unroll
        for (int k = 0; k < U; ++k) t[k] = i0 + k * RANK_THREADS < p.rows ? token_at(p.tokens, i0 + k * RANK_THREADS) : 0;
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i0 + k * RANK_THREADS < p.rows) keys[i0 + k * RANK_THREADS] = t[k] < 0 || t[k] >= p.V ? (uint32_t)p.V : (uint32_t)t[k];
    }
    const int quads = (p.rows + 3) / 4;
    if (threadIdx.x < 4 * quads - p.rows) keys[p.rows + threadIdx.x] = 0xffffffffu;  // behind all tokens
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = (int)blockIdx.x * 32, i = first + lane;
    const uint32_t mine = i < p.rows ? keys[i] : 0u;
    const int q0 = quads * warp / (RANK_THREADS / 32), q1 = quads * (warp + 1) / (RANK_THREADS / 32);
    const int b0 = min(max(first / 4, q0), q1), b1 = min(max(first / 4 + 8, q0), q1);
    int n = 0;
#pragma unroll 4
    for (int q = q0; q < b0; ++q) {  // tokens ahead of the block's: equal ones count
        const uint4 k = key_s[q];
        n += (k.x <= mine) + (k.y <= mine) + (k.z <= mine) + (k.w <= mine);
    }
    for (int q = b0; q < b1; ++q) {
        const uint4 k = key_s[q];
        const int j = 4 * q;
        n += (k.x < mine || (k.x == mine && j < i)) + (k.y < mine || (k.y == mine && j + 1 < i)) +
             (k.z < mine || (k.z == mine && j + 2 < i)) + (k.w < mine || (k.w == mine && j + 3 < i));
    }
#pragma unroll 4
    for (int q = b1; q < q1; ++q) {
        const uint4 k = key_s[q];
        n += (k.x < mine) + (k.y < mine) + (k.z < mine) + (k.w < mine);
    }
    part[warp][lane] = n;
    __syncthreads();
    if (warp == 0 && i < p.rows) {
        for (int w = 1; w < RANK_THREADS / 32; ++w) n += part[w][lane];
        p.key[0][n] = mine;
        p.row[0][n] = (uint32_t)i;
        const long long t = token_at(p.tokens, i);
        if (t >= p.V) record_error(p.err, DLC_DEVERR_INDEX, i);
    }
}

// The first pass's histograms; zeroes those of the others.
__global__ void __launch_bounds__(SORT_THREADS) sort_count_kernel(const __grid_constant__ SortParams p) {
    griddep_launch_dependents();
    __shared__ int count[SORT_MAX_DIGITS];
    const int digits = 1 << p.bits;
    for (int d = threadIdx.x; d < digits; d += SORT_THREADS) count[d] = 0;
    __syncthreads();
    griddep_wait();
    if ((int)blockIdx.x >= p.blocks) {
        fill_part(p);
        return;
    }
    const long long all = (long long)p.blocks * SORT_THREADS, me = (long long)blockIdx.x * SORT_THREADS + threadIdx.x;
    const long long per = (long long)(p.tiles + 1) * digits;
    for (long long i = per + me; i < per * p.passes; i += all) p.hist[i] = 0;
    for (int tile = blockIdx.x; tile < p.tiles; tile += p.blocks) {
#pragma unroll
        for (int k = 0; k < SORT_EACH; ++k) {
            const long long i = (long long)tile * SORT_TILE + k * SORT_THREADS + threadIdx.x;
            if (i < p.rows) atomicAdd(&count[sort_key(p, (int)i) & (uint32_t)(digits - 1)], 1);
        }
        __syncthreads();
        for (int d = threadIdx.x; d < digits; d += SORT_THREADS) {
            p.hist[(long long)tile * digits + d] = count[d];
            count[d] = 0;
        }
        __syncthreads();
    }
}

// Long lists: the tiles' counts of a pass become those of the tiles ahead, and the totals go to the last
// row.  32 digits a block; each warp takes a range of the tiles, twice.  (Otherwise a block of the
// next kernel adds up all tiles' counts itself: up to SORT_OWN_SUMS of them cost less than a launch.)
__global__ void __launch_bounds__(1024) sort_scan_kernel(const __grid_constant__ SortParams p, int pass) {
    griddep_launch_dependents();
    __shared__ int part[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, digits = 1 << p.bits, d = (int)blockIdx.x * 32 + lane;
    griddep_wait();
    int *hist = p.hist + (long long)pass * (p.tiles + 1) * digits;
    const int t0 = (int)((long long)p.tiles * warp / 32), t1 = (int)((long long)p.tiles * (warp + 1) / 32);
    int sum = 0;
    if (d < digits) {
#pragma unroll 8
        for (int t = t0; t < t1; ++t) sum += hist[(long long)t * digits + d];
    }
    part[warp][lane] = sum;
    __syncthreads();
    int ahead = 0;
    for (int w = 0; w < warp; ++w) ahead += part[w][lane];
    if (d >= digits) return;
    if (warp == 31) hist[(long long)p.tiles * digits + d] = ahead + sum;
    for (int t0b = t0; t0b < t1; t0b += 8) {
        int c[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) c[k] = t0b + k < t1 ? hist[(long long)(t0b + k) * digits + d] : 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (t0b + k < t1) hist[(long long)(t0b + k) * digits + d] = ahead;
            ahead += c[k];
        }
    }
}

__global__ void __launch_bounds__(SORT_THREADS) sort_pass_kernel(const __grid_constant__ SortParams p, int pass) {
    griddep_launch_dependents();
    __shared__ SortShared s;
    if ((int)blockIdx.x >= p.blocks) {
        griddep_wait();
        fill_part(p);
        return;
    }
    for (int i = threadIdx.x; i < SORT_WARPS * SORT_MAX_DIGITS / 2; i += SORT_THREADS) reinterpret_cast<uint32_t *>(s.count)[i] = 0u;
    __syncthreads();
    griddep_wait();
    const int tile = blockIdx.x, digits = 1 << p.bits;
    const int first = (int)(threadIdx.x >> 5) * 32 * SORT_EACH + (int)(threadIdx.x & 31);
    uint32_t key[SORT_EACH], row[SORT_EACH];
    bool on[SORT_EACH];
#pragma unroll
    for (int k = 0; k < SORT_EACH; ++k) {
        const long long i = (long long)tile * SORT_TILE + first + 32 * k;
        on[k] = i < p.rows;
        key[k] = row[k] = 0u;
        if (on[k]) {
            row[k] = pass == 0 ? (uint32_t)i : p.row[(pass - 1) & 1][i];
            key[k] = pass == 0 ? sort_key(p, (int)i) : p.key[(pass - 1) & 1][i];
        }
    }
    int rank[SORT_EACH], all[2] = {0, 0}, before[2] = {0, 0};
    const uint32_t mask = (uint32_t)digits - 1u;
    const int *hist = p.hist + (long long)pass * (p.tiles + 1) * digits + 2 * threadIdx.x;
    if (2 * (int)threadIdx.x < digits && p.scanned) {
        const int2 b = *reinterpret_cast<const int2 *>(hist + (long long)tile * digits);
        const int2 c = *reinterpret_cast<const int2 *>(hist + (long long)p.tiles * digits);
        before[0] = b.x, before[1] = b.y, all[0] = c.x, all[1] = c.y;
    } else if (2 * (int)threadIdx.x < digits) {
#pragma unroll 8
        for (int t = 0; t < p.tiles; ++t) {
            const int2 c = *reinterpret_cast<const int2 *>(hist + (long long)t * digits);
            all[0] += c.x, all[1] += c.y;
            if (t < tile) before[0] += c.x, before[1] += c.y;
        }
    }
    sort_ranks(s, key, on, pass * p.bits, mask, rank);
    sort_warps(s);
    sort_places(s, all, before);
    __syncthreads();
    const bool more = pass + 1 < p.passes;
#pragma unroll
    for (int k = 0; k < SORT_EACH; ++k)
        if (on[k]) {
            const uint32_t d = (key[k] >> (pass * p.bits)) & mask;
            const int at = s.base[d] + s.count[threadIdx.x >> 5][d] + rank[k];
            p.key[pass & 1][at] = key[k];
            p.row[pass & 1][at] = row[k];
            if (more)
                atomicAdd(p.hist + ((long long)(pass + 1) * (p.tiles + 1) + at / SORT_TILE) * digits + ((key[k] >> ((pass + 1) * p.bits)) & mask), 1);
        }
}

// ---- sums by token ---------------------------------------------------------------------

constexpr int SUM_THREADS = 128, SUM_MAX_CHUNK = 128;  // threads of a block at most
constexpr int JOIN_THREADS = 512;

struct SumParams {
    EmbeddingProblem e;        // y: dy; table: dtable
    const uint32_t *key, *row; // sorted
    float *part;               // [chunk][2][C]: of the token that comes in, of the one that goes on
    int chunk, chunks, slabs;  // sorted positions of a chunk
    int ranked;
};

// W = 8, 4: aligned vectors of dy and of the table; APART: any layout of dy, any size, a thread's channels a
// block's threads apart (16384 x 1001 BF16 into 30000 rows 45 us in all, 61 with one channel a thread).  ACC: the sums
// are added to the table's rows, which are loaded beside the rows of dy that end a token (one by
// one, where they are needed, 32 tokens took 32 memory latencies).
template <int W, bool APART, typename D, typename T, bool ACC>
__global__ void __launch_bounds__(SUM_THREADS) embedding_sum_kernel(const __grid_constant__ SumParams p) {
    griddep_launch_dependents();
    __shared__ uint32_t key_s[SUM_MAX_CHUNK + 2], row_s[SUM_MAX_CHUNK];
    const int C = p.e.C;
    griddep_wait();
    const int chunk = (int)blockIdx.x / p.slabs, slab = (int)blockIdx.x - chunk * p.slabs;
    const int n = min(p.chunk, (int)p.e.rows - chunk * p.chunk);
    const long long first = (long long)chunk * p.chunk;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        key_s[1 + i] = p.key[first + i];
        row_s[i] = p.row[first + i];
    }
    if (threadIdx.x == 0) {
        key_s[0] = chunk ? p.key[first - 1] : 0xffffffffu;
        key_s[1 + n] = first + n < p.e.rows ? p.key[first + n] : 0xffffffffu;
    }
    __syncthreads();
    const int hop = APART ? (int)blockDim.x : 1, c = slab * (int)blockDim.x * W + (int)threadIdx.x * (APART ? 1 : W);
    if (c >= C) return;
    const int there = (C - c - 1) / hop + 1;  // channels of this thread, if not W
    const long long co = c * p.e.y.m.cs, far = hop * p.e.y.m.cs;
    const uint32_t comes = key_s[0];  // the token that began in the chunk before, if it is the first here
    float acc[W];
#pragma unroll
    for (int j = 0; j < W; ++j) acc[j] = 0.f;
    constexpr int U = W * sizeof(D) > 16 || (ACC && (APART || W * sizeof(T) > 16)) ? 4 : 8;  // rows in flight
    for (int i0 = 0; i0 < n; i0 += U) {
        Words<W, APART, D> v[U];
        Words<W, APART, T> old[ACC ? U : 1];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = i0 + k;
            if (i >= n) continue;
            const uint32_t token = key_s[1 + i];
            if (token >= (uint32_t)p.e.V) continue;
            v[k].load(static_cast<const D *>(p.e.y.p) + row_off(p.e.y.m, row_s[i]) + co, far, there);
            if constexpr (ACC)
                if (key_s[2 + i] != token && token != comes) old[k].load(static_cast<const T *>(p.e.table.p) + (long long)token * C + c, hop, there);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = i0 + k;
            if (i >= n) break;
            const uint32_t token = key_s[1 + i];
            if (token >= (uint32_t)p.e.V) return;  // tokens outside the table: the last ones
#pragma unroll
            for (int j = 0; j < W; ++j) acc[j] += v[k].at(j);
            const bool ends = key_s[2 + i] != token;
            if (!ends && i + 1 < n) continue;
            if (ends && token != comes) {
                float f[W];
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    f[j] = acc[j] * p.e.scale;
                    if constexpr (ACC) f[j] += old[k].at(j);
                }
                store_words<W, APART, T>(static_cast<T *>(p.e.table.p) + (long long)token * C + c, hop, there, f);
            } else {
                store_words<W, APART, float>(p.part + ((long long)chunk * 2 + (token == comes ? 0 : 1)) * C + c, hop, there, acc);
            }
#pragma unroll
            for (int j = 0; j < W; ++j) acc[j] = 0.f;
        }
    }
}

// Tokens whose rows reach over several chunks: the block of the chunk where they begin adds up the
// partial sums, a range of them by each of its groups of `width` threads, always in the same order.
template <int W, bool APART, typename T, bool ACC>
__global__ void __launch_bounds__(JOIN_THREADS) embedding_join_kernel(const __grid_constant__ SumParams p, int width) {
    // (Among the waiting blocks of this kernel the ranking ones of a next call would be dealt to a few SMs only:
    // 4000 x 300, call after call, 27 us instead of 12.9.  Sorting by digits it gains 3 us to let the next call begin.)
    if (!p.ranked) griddep_launch_dependents();
    __shared__ float sum_s[JOIN_THREADS * W];
    griddep_wait();
    const int chunk = (int)blockIdx.x / p.slabs, slab = (int)blockIdx.x - chunk * p.slabs;
    const long long end = (long long)(chunk + 1) * p.chunk;  // (the last chunk has no block)
    const uint32_t token = p.key[end - 1], next = p.key[end], front = p.key[end - p.chunk], before = chunk ? p.key[end - p.chunk - 1] : 0xffffffffu;
    if (token >= (uint32_t)p.e.V || next != token) return;
    if (front == token && before == token) return;  // begins further ahead
    int more = 0;  // chunks after this one that the token begins
    for (;;) {
        const int k = chunk + 1 + more + (int)threadIdx.x;
        const int found = __syncthreads_count(k < p.chunks && p.key[(long long)k * p.chunk] == token);
        more += found;
        if (found < (int)blockDim.x) break;
    }
    const int groups = (int)blockDim.x / width, group = (int)threadIdx.x / width, t = (int)threadIdx.x - group * width;
    const int hop = APART ? width : 1, c = slab * width * W + t * (APART ? 1 : W), there = (p.e.C - c - 1) / hop + 1;
    const bool on = c < p.e.C;
    T *dst = static_cast<T *>(p.e.table.p) + (long long)token * p.e.C + c;
    Words<W, APART, T> old;
    if constexpr (ACC)
        if (on && group == 0) old.load(dst, hop, there);
    float acc[W];
#pragma unroll
    for (int j = 0; j < W; ++j) acc[j] = 0.f;
    // parts 0 (this chunk's second slot) and 1 .. more (the next ones' first slots)
    const int k1 = (int)((long long)(more + 1) * (group + 1) / groups);
    constexpr int U = W == 8 || APART ? 4 : 8;
    for (int k0 = (int)((long long)(more + 1) * group / groups); on && k0 < k1; k0 += U) {
        Words<W, APART, float> part[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (k0 + k < k1) part[k].load(p.part + ((long long)(chunk + k0 + k) * 2 + (k0 + k == 0 ? 1 : 0)) * p.e.C + c, hop, there);
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (k0 + k < k1) {
#pragma unroll
                for (int j = 0; j < W; ++j) acc[j] += part[k].v[j];
            }
    }
    if (groups > 1) {
#pragma unroll
        for (int j = 0; j < W; ++j) sum_s[j * JOIN_THREADS + threadIdx.x] = acc[j];
        __syncthreads();
        if (group) return;
        for (int g = 1; g < groups; ++g) {
#pragma unroll
            for (int j = 0; j < W; ++j) acc[j] += sum_s[j * JOIN_THREADS + g * width + t];
        }
    }
    if (!on) return;
#pragma unroll
    for (int j = 0; j < W; ++j) {
        acc[j] *= p.e.scale;
        if constexpr (ACC) acc[j] += old.at(j);
    }
    store_words<W, APART, T>(dst, hop, there, acc);
}

// ---- host side -----------------------------------------------------------------------

using Half = unsigned short;

template <typename T>
const void *rows_kernel(int y) {
    return y == DLC_DATA_BFLOAT16 ? (const void *)embedding_rows_kernel<T, Half> : (const void *)embedding_rows_kernel<T, float>;
}

template <int W, bool APART, typename D>
const void *sum_kernel(int t, bool acc) {
    if (t == DLC_DATA_BFLOAT16)
        return acc ? (const void *)embedding_sum_kernel<W, APART, D, Half, true> : (const void *)embedding_sum_kernel<W, APART, D, Half, false>;
    return acc ? (const void *)embedding_sum_kernel<W, APART, D, float, true> : (const void *)embedding_sum_kernel<W, APART, D, float, false>;
}

template <int W, bool APART>
const void *sum_kernel(const EmbeddingProblem &e) {
    return e.y.dt == DLC_DATA_BFLOAT16 ? sum_kernel<W, APART, Half>(e.table.dt, e.accumulate) : sum_kernel<W, APART, float>(e.table.dt, e.accumulate);
}

template <int W, bool APART>
const void *join_kernel(const EmbeddingProblem &e) {
    if (e.table.dt == DLC_DATA_BFLOAT16)
        return e.accumulate ? (const void *)embedding_join_kernel<W, APART, Half, true> : (const void *)embedding_join_kernel<W, APART, Half, false>;
    return e.accumulate ? (const void *)embedding_join_kernel<W, APART, float, true> : (const void *)embedding_join_kernel<W, APART, float, false>;
}

// Whether rows of the table and of y are whole vectors of w elements of either.
bool vectors(const EmbeddingProblem &e, int w) {
    return e.C % w == 0 && (uintptr_t)e.table.p % std::min(16, w * dlc_dtype_bytes((dlcDataType_t)e.table.dt)) == 0 && e.y.m.cs == 1 &&
           dlc_aligned_rows(e.y, std::min(16, w * dlc_dtype_bytes((dlcDataType_t)e.y.dt)));
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

struct BwdPlan {
    int bits, passes, tiles, chunk, chunks;
    bool ranked;
    size_t hist, key[2], row[2], part, bytes;
};

BwdPlan plan_bwd(long long rows, int C, int V) {
    BwdPlan b;
    int bits = 1;
    while (bits < 31 && (V >> bits) > 0) ++bits;  // tokens 0 .. V
    b.passes = (bits + SORT_MAX_BITS - 1) / SORT_MAX_BITS;
    b.bits = (bits + b.passes - 1) / b.passes;
    b.tiles = (int)((rows + SORT_TILE - 1) / SORT_TILE);
    b.ranked = rows <= (b.passes == 1 ? RANK_ONE : RANK_MOST);
    if (b.ranked) b.passes = 1;
    // Positions of a chunk: few where that gives the GPU enough to do at once, and where there are
    // more than enough many, so that a frequent token leaves fewer partial sums.
    const long long warps = rows * ((C + 255) / 256);
    b.chunk = warps <= 16 * 4096 ? 16 : warps <= 128 * 4096 ? 32 : warps <= 512 * 4096 ? 64 : SUM_MAX_CHUNK;
    b.chunks = (int)((rows + b.chunk - 1) / b.chunk);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += round256(bytes);
        return at;
    };
    b.hist = take((size_t)b.passes * (b.tiles + 1) * (1u << b.bits) * 4);
    for (int i = 0; i < 2; ++i) b.key[i] = take((size_t)rows * 4), b.row[i] = take((size_t)rows * 4);
    b.part = take((size_t)b.chunks * 2 * C * 4);
    b.bytes = off;
    return b;
}

}  // namespace

dlcStatus_t dlc_launch_embedding(dlcContext *ctx, const EmbeddingProblem &e) {
    EmParams p;
    p.e = e;
    p.err = ctx->d_err;
    const bool bf = e.table.dt == DLC_DATA_BFLOAT16, whole = bf && e.y.dt == DLC_DATA_BFLOAT16 && vectors(e, 8);
    p.pieces = whole ? e.C / 8 : (e.C + 32 * EM_LANE - 1) / (32 * EM_LANE);
    p.items = e.rows * p.pieces;
    const void *kern = whole ? (const void *)embedding_kernel : bf ? rows_kernel<Half>(e.y.dt) : rows_kernel<float>(e.y.dt);
    const int each = whole ? EM_THREADS : EM_THREADS / 32;  // pieces that a block takes at once
    const long long blocks = std::min<long long>((p.items + each - 1) / each, (long long)ctx->sm_count * (whole ? EM_BLOCKS : EM_ROW_BLOCKS));
    void *args[] = {&p};
    return dlc_launch(ctx, kern, dim3((unsigned)blocks), dim3(EM_THREADS), 0, args);
}

size_t dlc_embedding_bwd_workspace(const dlcContext *, long long rows, int C, int V) { return plan_bwd(rows, C, V).bytes; }

dlcStatus_t dlc_launch_embedding_bwd(dlcContext *ctx, const EmbeddingProblem &e) {
    const BwdPlan b = plan_bwd(e.rows, e.C, e.V);
    SortParams s;
    s.tokens = e.tokens;
    s.rows = (int)e.rows;
    s.V = e.V;
    s.tiles = b.tiles;
    s.bits = b.bits;
    s.passes = b.passes;
    s.scanned = 0;
    s.hist = reinterpret_cast<int *>(e.ws + b.hist);
    for (int i = 0; i < 2; ++i) {
        s.key[i] = reinterpret_cast<uint32_t *>(e.ws + b.key[i]);
        s.row[i] = reinterpret_cast<uint32_t *>(e.ws + b.row[i]);
    }
    s.err = ctx->d_err;
    SumParams p;
    p.e = e;
    p.key = s.key[(b.passes - 1) & 1];
    p.row = s.row[(b.passes - 1) & 1];
    p.part = reinterpret_cast<float *>(e.ws + b.part);
    p.chunk = b.chunk;
    p.chunks = b.chunks;
    p.ranked = b.ranked;
    const bool apart = !vectors(e, 4);
    const int w = !apart && vectors(e, 8) ? 8 : 4;
    const int threads = std::min(SUM_THREADS, (apart ? e.C + 31 : (e.C + w - 1) / w + 31) / 32 * 32);
    p.slabs = (e.C + threads * w - 1) / (threads * w);
    if ((long long)p.chunks * p.slabs > 0x7fffffffLL) return DLC_STATUS_NOT_SUPPORTED;
    // the table's whole 16-byte words, dealt evenly to the sort's launches
    const size_t bytes = e.accumulate ? 0 : (size_t)e.V * e.C * dlc_dtype_bytes((dlcDataType_t)e.table.dt);
    char *table = static_cast<char *>(e.table.p);
    const size_t head = std::min(bytes, (16 - (uintptr_t)table % 16) % 16), words = (bytes - head) / 16;
    const int launches = b.ranked ? 1 : 1 + b.passes;
    auto part = [&](int i) {
        const size_t w0 = words * i / launches, w1 = words * (i + 1) / launches;
        s.fill = table + head + 16 * w0;
        s.fill_words = (long long)(w1 - w0);
        s.edge[0] = table;
        s.edge[1] = table + head + 16 * words;
        s.edge_bytes[0] = i == 0 ? (int)head : 0;
        s.edge_bytes[1] = i == 0 ? (int)(bytes - head - 16 * words) : 0;
        return bytes ? (unsigned)std::min<size_t>((w1 - w0) / (SORT_THREADS * 4) + 1, (size_t)ctx->sm_count * 3) : 0u;
    };
    dlcStatus_t st;
    void *args[] = {&s};
    if (b.ranked) {
        s.blocks = (int)((e.rows + 31) / 32);
        st = dlc_launch(ctx, (const void *)rank_kernel, dim3((unsigned)s.blocks + 2 * part(0)), dim3(RANK_THREADS), 0, args);
        if (st != DLC_STATUS_SUCCESS) return st;
    } else {
        s.blocks = std::min(b.tiles, ctx->sm_count * 4);
        unsigned fill = part(0);
        st = dlc_launch(ctx, (const void *)sort_count_kernel, dim3((unsigned)s.blocks + fill), dim3(SORT_THREADS), 0, args);
        s.blocks = b.tiles;
        s.scanned = b.tiles > SORT_OWN_SUMS;
        for (int pass = 0; pass < b.passes && st == DLC_STATUS_SUCCESS; ++pass) {
            fill = part(1 + pass);
            void *pargs[] = {&s, &pass};
            if (s.scanned) st = dlc_launch(ctx, (const void *)sort_scan_kernel, dim3(((1u << b.bits) + 31) / 32), dim3(1024), 0, pargs);
            if (st != DLC_STATUS_SUCCESS) break;
            st = dlc_launch(ctx, (const void *)sort_pass_kernel, dim3((unsigned)b.tiles + fill), dim3(SORT_THREADS), 0, pargs);
        }
        if (st != DLC_STATUS_SUCCESS) return st;
    }
    void *sargs[] = {&p};
    const void *sum = w == 8 ? sum_kernel<8, false>(e) : apart ? sum_kernel<4, true>(e) : sum_kernel<4, false>(e);
    st = dlc_launch(ctx, sum, dim3((unsigned)(p.chunks * p.slabs)), dim3((unsigned)threads), 0, sargs);
    if (st != DLC_STATUS_SUCCESS || p.chunks == 1) return st;
    const void *join = w == 8 ? join_kernel<8, false>(e) : apart ? join_kernel<4, true>(e) : join_kernel<4, false>(e);
    int width = threads;
    void *jargs[] = {&p, &width};
    return dlc_launch(ctx, join, dim3((unsigned)((p.chunks - 1) * p.slabs)), dim3((unsigned)(JOIN_THREADS / width * width)), 0, jargs);
}

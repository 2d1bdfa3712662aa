// layernorm_vec.cuh -- layer norm (layernorm.cu) of rows in the usual layout: channels contiguous, every
// tensor's rows at one pitch, all inputs (and total) of one type; pitches of whole 16-byte pieces
// (layernorm_vec.cu), or (SHIFT, layernorm_shift.cu) any pitch, as far as the inputs and total begin their rows
// alike.
//
// Each input is read once and each output written once, and that should bound the kernels; with the
// general ones the instructions do (65536 x 768 BF16 to E4M3: 1278 warp instructions a row and
// 100 us in layer_rows_kernel), and then the barriers between a row's warps.  So a row takes as few
// threads as hold it, up to eight vectors of 16 bytes each (2048 channels: one warp), gamma and beta
// wait in shared memory, and only a thread's last vector can be partial or missing.  FP32 rows have
// vectors of four channels: with eight, neighbouring threads touched every other 16 bytes (8192 x 2048
// FP32 67 us, 48 this way).
//
// Measured back to back, with residual and sum: 65536 x 768 BF16 to E4M3 61.3 us (5.7 TB/s), 16384 x
// 2048 BF16 48.8 us (5.5), 8192 x 2048 FP32 48 us (5.6); backward with both sums 16384 x 2048 BF16 50.5
// us (5.3), 8192 x 2048 FP32 50 us (5.4).  A call's start and end are 7 to 10 us of it: rows beyond these
// come at 6.4 TB/s.
#pragma once

#include "norm_rows.cuh"

namespace {

using namespace dlc;

// Sums over the `tpr` threads of a row (a power of two or whole warps), as row_reduce has them; the
// usual numbers of warps without a loop, whose branches would count.  A warp has two words of the buffer in
// every reduction, of one sum too: a block's rows run ahead of one another.
template <int N, int WARPS>
__device__ __forceinline__ void join_warps(float (&a)[N], const float *row) {
    float4 q[WARPS / 2];
#pragma unroll
    for (int i = 0; i < WARPS / 2; ++i) q[i] = reinterpret_cast<const float4 *>(row)[i];
    const float *f = reinterpret_cast<const float *>(q);
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = f[i];
#pragma unroll
    for (int w = 1; w < WARPS; ++w)
#pragma unroll
        for (int i = 0; i < N; ++i) a[i] += f[w * 2 + i];
}

template <int N>
__device__ __forceinline__ void row_sums(float (&a)[N], int tpr, int slot, float (*buf)[NORM_MAX_WARPS * 2], int parity) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        if (o < 8 || o < tpr) {
#pragma unroll
            for (int i = 0; i < N; ++i) a[i] += __shfl_xor_sync(0xffffffffu, a[i], o);
        }
    }
    if (tpr > 32) {
        const int warps = tpr >> 5;
        float *mine = buf[parity] + 2 * ((int)threadIdx.x >> 5);
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) mine[i] = a[i];
        }
        asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(tpr) : "memory");
        const float *row = buf[parity] + 2 * slot * warps;
        if (warps == 2) {
            join_warps<N, 2>(a, row);
        } else if (warps == 4) {
            join_warps<N, 4>(a, row);
        } else if (warps == 8) {
            join_warps<N, 8>(a, row);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) a[i] = row[i];
            for (int w = 1; w < warps; ++w) {
#pragma unroll
                for (int i = 0; i < N; ++i) a[i] += row[w * 2 + i];
            }
        }
    }
}

// Largest |v| over a row's threads (NaN or not: such a row is NaN anyway).
__device__ __forceinline__ float row_most(float v, int tpr, int slot, float (*buf)[NORM_MAX_WARPS * 2], int parity) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
        if (o < 8 || o < tpr) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (tpr > 32) {
        const int warps = tpr >> 5;
        if ((threadIdx.x & 31) == 0) buf[parity][2 * ((int)threadIdx.x >> 5)] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(tpr) : "memory");
        const float *row = buf[parity] + 2 * slot * warps;
        v = fmaxf(row[0], row[2]);
        for (int w = 2; w < warps; ++w) v = fmaxf(v, row[2 * w]);
    }
    return v;
}

constexpr int VEC_THREADS = 256;  // of a block, or a little less (backward, long rows: TH)

// Channels of a vector: 16 bytes, so that neighbouring threads copy neighbouring words.
template <typename E>
constexpr int vec_ch() { return 16 / (int)sizeof(E); }

// Which of a thread's vectors' channels exist: n(j) first ones of vector j, but for the first skip(j).
template <int V, int CH, bool SHIFT>
struct Cover {  // only the last vector is partial or missing
    int last;
    __device__ __forceinline__ Cover(int C, int, int t, int tpr) : last(min(max(C - ((V - 1) * tpr + t) * CH, 0), CH)) {}
    __device__ __forceinline__ int n(int j) const { return j + 1 < V ? CH : last; }
    __device__ __forceinline__ int skip(int) const { return 0; }
    __device__ __forceinline__ bool whole(int j) const { return j + 1 < V || last == CH; }
    __device__ __forceinline__ void zero_front(float (&)[V * CH]) const {}
    __device__ __forceinline__ void zero_rest(float (&v)[V * CH]) const {
        if (last == 0) {
#pragma unroll
            for (int i = 0; i < CH; ++i) v[CH * (V - 1) + i] = 0.f;
        } else if (last < CH) {
#pragma unroll
            for (int i = 1; i < CH; ++i)
                if (i >= last) v[CH * (V - 1) + i] = 0.f;
        }
    }
};

// Rows that begin inside a 16-byte piece.  The vectors are the pieces; the first one begins with `lead`
// channels of what is in front of the row.  Every row of a block begins alike: its rows are a
// multiple of eight apart.
template <int V, int CH>
struct Cover<V, CH, true> {
    int front, rest, hop;
    __device__ __forceinline__ Cover(int C, int lead, int t, int tpr) : front(t == 0 ? lead : 0), rest(C + lead - CH * t), hop(CH * tpr) {}
    __device__ __forceinline__ int n(int j) const { return min(max(rest - j * hop, 0), CH); }
    __device__ __forceinline__ int skip(int j) const { return j == 0 ? front : 0; }
    __device__ __forceinline__ bool whole(int j) const { return rest - j * hop >= CH && (j > 0 || front == 0); }
    __device__ __forceinline__ void zero_front(float (&v)[V * CH]) const {
        if (front) {
#pragma unroll
            for (int i = 0; i < CH - 1; ++i)
                if (i < front) v[i] = 0.f;
        }
    }
    __device__ __forceinline__ void zero_rest(float (&v)[V * CH]) const {
        zero_front(v);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (rest - j * hop < CH) {
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    if (i >= rest - j * hop) v[CH * j + i] = 0.f;
            }
    }
};

// Centres a thread's part of a row again (far_row), or leaves it where `far` is false.
template <int V, int CH, bool SHIFT>
__device__ __forceinline__ void recentre(float (&v)[V * CH], const Cover<V, CH, SHIFT> &cover, bool far, int C, int tpr, int slot,
                                         float (*buf)[NORM_MAX_WARPS * 2], int parity) {
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < V * CH / 2; ++i) sum = add2(get2(v, i), sum);
    float off[1] = {sum.x + sum.y};
    row_sums(off, tpr, slot, buf, parity);
    const float2 mean = pair_of(far ? -off[0] / (float)C : 0.f);
#pragma unroll
    for (int i = 0; i < V * CH / 2; ++i) set2(v, i, add2(get2(v, i), mean));
    cover.zero_rest(v);
}

// A ring of S rows of T tensors in shared memory, V vectors a thread, of which a thread
// reads back only what it copied itself: no barrier, and a row's place takes the row S further
// on as soon as it has been read.  (Strides are constants: with the block's size for one, the
// addresses' instructions cost 7 %.)
template <int V, typename E, int T, int S, int TH>
struct VecRing {
    static constexpr uint32_t WORDS = (uint32_t)(T * V), WORD = 16u * TH;
    uint32_t base, row;
    __device__ __forceinline__ explicit VecRing(uint32_t smem) : base(smem + threadIdx.x * 16u), row(0) {}
    // at: this thread's first vector; hop: bytes to the next one; cover: channels of each that exist
    // (what is behind them becomes zero)
    template <typename Cover>
    __device__ __forceinline__ void fetch(int k, const char *at, uint32_t hop, const Cover &cover) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            cp_async_16(base + (row + (uint32_t)(k * V + j)) * WORD, at + (cover.n(j) > 0 ? j * hop : 0u),
                        (uint32_t)cover.n(j) * (uint32_t)sizeof(E));
    }
    __device__ __forceinline__ void next() {  // (ends the copies of a row)
        cp_async_commit();
        row = S == 1 || row == WORDS * (S - 1) ? 0u : row + WORDS;
    }
    __device__ __forceinline__ void read_vector(int k, int j, float *f) const {
        uint32_t w[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(base + (row + (uint32_t)(k * V + j)) * WORD)
                     : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(E) == 2)
                set2(f, i, unpack_bf16(w[i]));
            else
                f[i] = __uint_as_float(w[i]);
        }
    }
    __device__ __forceinline__ void read(int k, float (&f)[V * vec_ch<E>()]) const {
#pragma unroll
        for (int j = 0; j < V; ++j) read_vector(k, j, f + j * vec_ch<E>());
    }
    static constexpr size_t SMEM = (size_t)S * WORDS * WORD;
};

// A vector of a channel-wise FP32 array from shared memory: its quarters of four channels lie apart,
// so that neighbouring threads read neighbouring words.
template <int CH>
__device__ __forceinline__ void vec_param(uint32_t at, uint32_t apart, float (&g)[CH]) {
#pragma unroll
    for (int h = 0; h < CH / 4; ++h) {
        const float4 a = ld_shared_f32x4(at + (uint32_t)h * apart);
        g[4 * h] = a.x, g[4 * h + 1] = a.y, g[4 * h + 2] = a.z, g[4 * h + 3] = a.w;
    }
}

// Fills vec_param's arrays, whose vectors are dealt to `tpr` threads; zeros behind the row.  (By
// asynchronous copies ahead of the rows' a call of 65536 x 768 took 4 us more, element by element
// one of 16384 x 2048 5 us.)
template <int CH, bool SHIFT>
__device__ __forceinline__ void vec_param_fill(float *dst, const float *src, int C, int lead, int tpr, int V) {
    constexpr int H = CH / 4;
    if constexpr (SHIFT) {  // single ones, `lead` further on
        const int t = (int)threadIdx.x % tpr;
        for (int j = (int)threadIdx.x / tpr; j < V; j += (int)blockDim.x / tpr) {
            const int c = CH * (t + j * tpr) - lead;
            float g[CH];
#pragma unroll
            for (int i = 0; i < CH; ++i) g[i] = src && c + i >= 0 && c + i < C ? src[c + i] : 0.f;
#pragma unroll
            for (int h = 0; h < H; ++h)
                reinterpret_cast<float4 *>(dst)[(j * H + h) * tpr + t] = make_float4(g[4 * h], g[4 * h + 1], g[4 * h + 2], g[4 * h + 3]);
        }
        return;
    }
    const bool aligned = ((uintptr_t)src & 15u) == 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < H * tpr * V; i += blockDim.x) {
        const int vec = i / H, at = (vec / tpr * H + i % H) * tpr + vec % tpr;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (src && aligned && 4 * i + 4 <= C) {
            v = reinterpret_cast<const float4 *>(src)[i];
        } else if (src && 4 * i < C) {
            v.x = src[4 * i];
            if (4 * i + 1 < C) v.y = src[4 * i + 1];
            if (4 * i + 2 < C) v.z = src[4 * i + 2];
            if (4 * i + 3 < C) v.w = src[4 * i + 3];
        }
        reinterpret_cast<float4 *>(dst)[at] = v;
    }
}

// A vector of CH values as Y.
template <typename Y, int CH>
__device__ __forceinline__ void vec_store(char *at, const float *v) {
    if constexpr (sizeof(Y) == 4) {
#pragma unroll
        for (int i = 0; i < CH / 4; ++i) reinterpret_cast<float4 *>(at)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
        uint32_t w[CH * sizeof(Y) / 4];
        if constexpr (sizeof(Y) == 2) {
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < CH / 4; ++i) w[i] = pack_e4m3(v[4 * i], v[4 * i + 1]) | (pack_e4m3(v[4 * i + 2], v[4 * i + 3]) << 16);
        }
        if constexpr (sizeof(w) == 16)
            *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (sizeof(w) == 8)
            *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t *>(at) = w[0];
    }
}

// A vector: whole, or its channels skip .. n - 1.
template <typename Y, int CH>
__device__ __forceinline__ void vec_store_part(char *at, const float *v, bool whole, int skip, int n) {
    if (whole) {
        vec_store<Y, CH>(at, v);
    } else {
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (i >= skip && i < n) store_elem(at, sizeof(Y) == 4 ? DLC_DATA_FLOAT : sizeof(Y) == 2 ? DLC_DATA_BFLOAT16 : DLC_DATA_FLOAT8_E4M3, i, v[i]);
    }
}

// The same from a row in shared memory that begins at another place of a piece than it does in `at`: `from`
// bytes on.
template <typename Y, int CH>
__device__ __forceinline__ void vec_store_moved(char *at, const char *row, int from, bool whole, int skip, int n) {
    constexpr int WORDS = CH * (int)sizeof(Y) / 4;
    uint32_t w[WORDS + 1];
    const uint32_t *src = reinterpret_cast<const uint32_t *>(row + (from & ~3));
#pragma unroll
    for (int i = 0; i < WORDS + (sizeof(Y) < 4 ? 1 : 0); ++i) w[i] = src[i];
    if constexpr (sizeof(Y) < 4) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8u * ((uint32_t)from & 3u));
    }
    if (whole) {
        if constexpr (WORDS % 4 == 0) {
#pragma unroll
            for (int i = 0; i < WORDS / 4; ++i) reinterpret_cast<uint4 *>(at)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else if constexpr (WORDS == 2) {
            *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
        } else {
            *reinterpret_cast<uint32_t *>(at) = w[0];
        }
    } else {
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (i >= skip && i < n) {
                if constexpr (sizeof(Y) == 4)
                    reinterpret_cast<uint32_t *>(at)[i] = w[i];
                else if constexpr (sizeof(Y) == 2)
                    reinterpret_cast<unsigned short *>(at)[i] = (unsigned short)(w[i / 2] >> (16 * (i & 1)));
                else
                    reinterpret_cast<unsigned char *>(at)[i] = (unsigned char)(w[i / 4] >> (8 * (i & 3)));
            }
    }
}

// Blocks an SM holds, by the registers of V vectors a thread; rows of the rings.
template <int V, typename E>
constexpr int vec_blocks() { return V * vec_ch<E>() <= 16 ? 4 : V * vec_ch<E>() <= 32 ? 3 : 2; }
template <int V>
constexpr int vec_ring() { return V <= 2 ? 2 : 1; }
template <int V>
constexpr int vec_bwd_ring() { return V <= 2 ? 3 : 2; }

struct VecRow {  // this thread's part of a tensor's rows
    char *p;
    long long inc;
    __device__ __forceinline__ VecRow(const RowTensor &t, int e, long long row, long long step, int channel)
        : p(static_cast<char *>(t.p) + (row * t.m.ld + channel) * e), inc(step * t.m.ld * e) {}
};

// Channels in front of a block's rows in their first piece of `CH` channels (rows at pitch ld).
__device__ __forceinline__ int vec_lead(long long ld, int ch) { return (int)((long long)(blockIdx.x % ch) * (ld % ch)) % ch; }

// E: storage of x, r and t; Y: of y.  SHIFT: y may begin its rows differently; a row of it then passes through
// shared memory.
template <int V, typename E, typename Y, bool RES, bool SHIFT>
__global__ void __launch_bounds__(VEC_THREADS, vec_blocks<V, E>()) layer_vec_kernel(const __grid_constant__ LayerProblem p, int tpr) {
    griddep_launch_dependents();
    __shared__ __align__(16) float buf[2][NORM_MAX_WARPS * 2];
    extern __shared__ uint4 ring_s[];
    constexpr int CH = vec_ch<E>(), N = CH * V, S = vec_ring<V>();
    const int rpb = (int)blockDim.x / tpr, slot = (int)threadIdx.x / tpr, t = (int)threadIdx.x % tpr;
    const long long step = (long long)gridDim.x * rpb, slot0 = SHIFT ? (long long)slot * gridDim.x : slot;
    const int lead = SHIFT ? vec_lead(p.x.m.ld, CH) : 0;
    const Cover<V, CH, SHIFT> cover(p.C, lead, t, tpr);
    const int c = (V > 1 && !SHIFT) || cover.n(0) > 0 ? CH * t : 0;
    const uint32_t hop = (uint32_t)(CH * tpr), apart = 16u * (uint32_t)tpr;
    const float inv_c = 1.f / (float)p.C;
    using Ring = VecRing<V, E, RES ? 2 : 1, S, VEC_THREADS>;
    Ring ring(smem_u32(ring_s));
    float *gamma = reinterpret_cast<float *>(reinterpret_cast<char *>(ring_s) + Ring::SMEM), *beta = gamma + N * tpr;
    const uint32_t g0 = smem_u32(gamma) + 16u * (uint32_t)t, b0 = smem_u32(beta) + 16u * (uint32_t)t;
    long long row = SHIFT ? blockIdx.x + slot0 : (long long)blockIdx.x * rpb + slot, ahead = row;
    VecRow x(p.x, sizeof(E), row, step, c - lead), r(p.r, sizeof(E), row, step, c - lead), tt(p.t, sizeof(E), row, step, c - lead);
    // y's own beginning; where y's vectors come from, a row of shared memory that begins as x does
    const int y_lead = SHIFT ? vec_lead(p.y.m.ld, CH) : 0;
    const Cover<V, CH, SHIFT> y_cover(p.C, y_lead, t, tpr);
    VecRow y(p.y, sizeof(Y), row, step, CH * t - y_lead);
    char *y_row = reinterpret_cast<char *>(beta + N * tpr) + 16 + (size_t)slot * (N * sizeof(Y)) * tpr;
    griddep_wait();
    auto fetch = [&]() {
        if (ahead < p.rows) {
            ring.fetch(0, x.p, 16u * (uint32_t)tpr, cover);
            if (RES) ring.fetch(1, r.p, 16u * (uint32_t)tpr, cover);
        }
        ring.next();
        ahead += step;
        x.p += x.inc;
        r.p += r.inc;
    };
    for (int i = 0; i < S; ++i) fetch();
    vec_param_fill<CH, SHIFT>(gamma, p.gamma, p.C, lead, tpr, V);
    vec_param_fill<CH, SHIFT>(beta, p.beta, p.C, lead, tpr, V);
    __syncthreads();
    int parity = 0;
    for (; row - slot0 < p.rows; row += step) {  // (as many rounds for every thread of the block)
        const bool on = row < p.rows;
        float v[N];
        cp_async_wait<S - 1>();
        ring.read(0, v);
        if (RES) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float w[CH];
                ring.read_vector(1, j, w);
#pragma unroll
                for (int i = 0; i < CH / 2; ++i) set2(v + CH * j, i, add2(get2(v + CH * j, i), get2(w, i)));
            }
        }
        if (p.t.p && on) {
#pragma unroll
            for (int j = 0; j < V; ++j) vec_store_part<E, CH>(tt.p + j * (16u * (uint32_t)tpr), v + CH * j, cover.whole(j), cover.skip(j), cover.n(j));
        }
        cover.zero_front(v);
        tt.p += tt.inc;
        fetch();
        float2 sum = make_float2(0.f, 0.f), sq = sum;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) sum = add2(get2(v, i), sum);
        float total[1] = {sum.x + sum.y};
        row_sums(total, tpr, slot, buf, parity);
        parity ^= 1;
        const float mean = total[0] * inv_c;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) set2(v, i, add2(get2(v, i), pair_of(-mean)));
        cover.zero_rest(v);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) sq = fma2(get2(v, i), get2(v, i), sq);
        total[0] = sq.x + sq.y;
        row_sums(total, tpr, slot, buf, parity);
        parity ^= 1;
        const bool far = far_row(mean, total[0] * inv_c);
        if (__builtin_expect(__any_sync(0xffffffffu, far), 0)) {
            recentre(v, cover, far, p.C, tpr, slot, buf, parity);
            parity ^= 1;
            sq = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) sq = fma2(get2(v, i), get2(v, i), sq);
            total[0] = sq.x + sq.y;
            row_sums(total, tpr, slot, buf, parity);
            parity ^= 1;
        }
        const float2 rho = pair_of(rsqrtf(total[0] * inv_c + p.eps));
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float g[CH], b[CH];
            vec_param<CH>(g0 + (uint32_t)(j * (CH / 4)) * apart, apart, g);
            vec_param<CH>(b0 + (uint32_t)(j * (CH / 4)) * apart, apart, b);
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) set2(v + CH * j, i, fma2(mul2(get2(v + CH * j, i), rho), get2(g, i), get2(b, i)));
        }
        if constexpr (sizeof(Y) == 1) {
            float most[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < N; ++i) most[i & 1] = fmaxf(most[i & 1], fabsf(v[i]));
            const float scale = fmaxf(row_most(fmaxf(most[0], most[1]), tpr, slot, buf, parity), SCALE_FLOOR) / E4M3_MAX;
            parity ^= 1;
            if (t == 0 && on) p.scale[row] = scale;
            const float2 inv = pair_of(1.f / scale);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) set2(v, i, mul2(get2(v, i), inv));
        }
        if (SHIFT && y_lead != lead) {  // (the block's rows are alike)
#pragma unroll
            for (int j = 0; j < V; ++j) vec_store<Y, CH>(y_row + (t + j * tpr) * (CH * (int)sizeof(Y)), v + CH * j);
            if (tpr > 32)
                asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(tpr) : "memory");
            else
                __syncwarp();
            if (on) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (y_cover.n(j) > 0)
                        vec_store_moved<Y, CH>(y.p + j * (hop * (uint32_t)sizeof(Y)), y_row, ((t + j * tpr) * CH + lead - y_lead) * (int)sizeof(Y),
                                               y_cover.whole(j), y_cover.skip(j), y_cover.n(j));
            }
            if (tpr <= 32) __syncwarp();  // (else the next row's sums have a barrier)
        } else if (on) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                vec_store_part<Y, CH>(y.p + j * (hop * (uint32_t)sizeof(Y)), v + CH * j, cover.whole(j), cover.skip(j), cover.n(j));
        }
        y.p += y.inc;
    }
}

// The same for the backward pass.  128 registers a thread: 16 warps an SM.
template <int V, typename E, bool RES, int TH, bool SHIFT>
__global__ void __launch_bounds__(TH, 512 / TH) layer_bwd_vec_kernel(const __grid_constant__ LayerBwdProblem p, int tpr) {
    griddep_launch_dependents();
    __shared__ __align__(16) float buf[2][NORM_MAX_WARPS * 2];
    extern __shared__ uint4 ring_s[];
    constexpr int CH = vec_ch<E>(), N = CH * V, S = vec_bwd_ring<V>();
    const int rpb = (int)blockDim.x / tpr, slot = (int)threadIdx.x / tpr, t = (int)threadIdx.x % tpr;
    const long long step = (long long)gridDim.x * rpb, slot0 = SHIFT ? (long long)slot * gridDim.x : slot;
    const int lead = SHIFT ? vec_lead(p.t.m.ld, CH) : 0;
    const Cover<V, CH, SHIFT> cover(p.C, lead, t, tpr);
    const int c = ((V > 1 && !SHIFT) || cover.n(0) > 0 ? CH * t : 0) - lead;
    const uint32_t hop = 16u * (uint32_t)tpr;
    const float inv_c = 1.f / (float)p.C;
    using Ring = VecRing<V, E, RES ? 3 : 2, S, TH>;
    Ring ring(smem_u32(ring_s));
    float *gamma = reinterpret_cast<float *>(reinterpret_cast<char *>(ring_s) + Ring::SMEM);
    const uint32_t g0 = smem_u32(gamma) + 16u * (uint32_t)t;
    float dg[N], db[N];
#pragma unroll
    for (int i = 0; i < N; ++i) dg[i] = db[i] = 0.f;
    long long row = SHIFT ? blockIdx.x + slot0 : (long long)blockIdx.x * rpb + slot, ahead = row;
    VecRow dy(p.dy, sizeof(E), row, step, c), tt(p.t, sizeof(E), row, step, c), dt(p.dt, sizeof(E), row, step, c), dx(p.dx, sizeof(E), row, step, c);
    griddep_wait();
    auto fetch = [&]() {
        if (ahead < p.rows) {
            ring.fetch(0, dy.p, hop, cover);
            ring.fetch(1, tt.p, hop, cover);
            if (RES) ring.fetch(2, dt.p, hop, cover);
        }
        ring.next();
        ahead += step;
        dy.p += dy.inc;
        tt.p += tt.inc;
        dt.p += dt.inc;
    };
    for (int i = 0; i < S; ++i) fetch();
    vec_param_fill<CH, SHIFT>(gamma, p.gamma, p.C, lead, tpr, V);
    __syncthreads();
    for (; row - slot0 < p.rows; row += step, dx.p += dx.inc) {
        const bool on = row < p.rows;
        float d[N], v[N], g[CH];  // (gamma is read where it is used: holding it would spill)
        cp_async_wait<S - 1>();
        ring.read(0, d);
        ring.read(1, v);
        cover.zero_front(d);
        cover.zero_front(v);
        float2 sum = make_float2(0.f, 0.f), sd = sum, sq, dot;
        if (on) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) set2(db, i, add2(get2(d, i), get2(db, i)));
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            vec_param<CH>(g0 + (uint32_t)(j * (CH / 4)) * hop, hop, g);
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) {
                sum = add2(get2(v + CH * j, i), sum);
                sd = fma2(get2(d + CH * j, i), get2(g, i), sd);
            }
        }
        float means[2] = {sum.x + sum.y, sd.x + sd.y};
        row_sums(means, tpr, slot, buf, 0);
        const float mean = means[0] * inv_c;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) set2(v, i, add2(get2(v, i), pair_of(-mean)));
        cover.zero_rest(v);
        float red[2];
        auto squares = [&]() {
            sq = dot = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                vec_param<CH>(g0 + (uint32_t)(j * (CH / 4)) * hop, hop, g);
#pragma unroll
                for (int i = 0; i < CH / 2; ++i) {
                    const float2 w = get2(v + CH * j, i);
                    sq = fma2(w, w, sq);
                    dot = fma2(mul2(get2(d + CH * j, i), get2(g, i)), w, dot);
                }
            }
            red[0] = sq.x + sq.y, red[1] = dot.x + dot.y;
            row_sums(red, tpr, slot, buf, 1);
        };
        squares();
        const bool far = far_row(mean, red[0] * inv_c);
        if (__builtin_expect(__any_sync(0xffffffffu, far), 0)) {
            recentre(v, cover, far, p.C, tpr, slot, buf, 0);
            squares();
        }
        const float rho = rsqrtf(red[0] * inv_c + p.eps);
        const float2 rho2 = pair_of(rho), k2 = pair_of(-row_slope(rho, red[1] * inv_c)), m2 = pair_of(-rho * (means[1] * inv_c));
        if (on) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float s[CH];
                vec_param<CH>(g0 + (uint32_t)(j * (CH / 4)) * hop, hop, g);
                if (RES) ring.read_vector(2, j, s);
#pragma unroll
                for (int i = 0; i < CH / 2; ++i) {
                    const float2 dr = mul2(get2(d + CH * j, i), rho2), w = get2(v + CH * j, i);
                    set2(dg + CH * j, i, fma2(dr, w, get2(dg + CH * j, i)));
                    const float2 base = RES ? add2(get2(s, i), m2) : m2;
                    set2(s, i, fma2(dr, get2(g, i), fma2(w, k2, base)));
                }
                vec_store_part<E, CH>(dx.p + j * hop, s, cover.whole(j), cover.skip(j), cover.n(j));
            }
        }
        fetch();
    }
    if (!p.dgamma && !p.dbeta) return;
    float *ws0 = p.ws + 2ll * blockIdx.x * p.C;
    float *acc_s = reinterpret_cast<float *>(ring_s);  // [slot][C], in the ring's place
    cp_async_wait<0>();
    if constexpr (SHIFT) {  // in vectors as gamma has them, from where neighbouring threads take neighbouring channels
        constexpr int H = CH / 4;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float *acc = h ? db : dg;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int q = 0; q < H; ++q)
                    reinterpret_cast<float4 *>(acc_s)[(slot * V * H + j * H + q) * tpr + t] =
                        make_float4(acc[CH * j + 4 * q], acc[CH * j + 4 * q + 1], acc[CH * j + 4 * q + 2], acc[CH * j + 4 * q + 3]);
            __syncthreads();
#pragma unroll
            for (int j = 0; j < V; ++j)
                for (uint32_t i = threadIdx.x; i < (uint32_t)(CH * tpr); i += blockDim.x) {
                    const uint32_t vec = i / CH, q = i % CH;
                    const int k = j * CH * tpr + (int)i - lead;
                    if (k < 0 || k >= p.C) continue;
                    const float *at = acc_s + (((uint32_t)(j * H) + q / 4) * (uint32_t)tpr + vec) * 4 + q % 4;
                    float sum = 0.f;
                    for (int r = 0; r < rpb; ++r) sum += at[r * (N * tpr)];
                    ws0[(long long)h * p.C + k] = sum;
                }
        }
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float *acc = h ? db : dg;
        if (rpb > 1) __syncthreads();
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float *at = (rpb > 1 ? acc_s + (long long)slot * p.C : ws0 + (long long)h * p.C) + (t + j * tpr) * CH;
            const int n = cover.n(j);
            if (n == CH && p.C % 4 == 0) {
#pragma unroll
                for (int i = 0; i < CH / 4; ++i)
                    reinterpret_cast<float4 *>(at)[i] = make_float4(acc[CH * j + 4 * i], acc[CH * j + 4 * i + 1], acc[CH * j + 4 * i + 2], acc[CH * j + 4 * i + 3]);
            } else if (n > 0) {
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    if (i < n) at[i] = acc[CH * j + i];
            }
        }
        if (rpb > 1) {
            __syncthreads();
            for (int k = threadIdx.x; k < p.C; k += blockDim.x) {
                float s = 0.f;
                for (int i = 0; i < rpb; ++i) s += acc_s[(long long)i * p.C + k];
                ws0[(long long)h * p.C + k] = s;
            }
        }
    }
}

// ---- host side ---------------------------------------------------------------

// The launch: V vectors for each of a row's `tpr` threads, `rpb` rows a block.
struct VecPlan {
    int v = 0, tpr = 0, rpb = 0;
};

constexpr size_t VEC_SM_SMEM = 228 * 1024;  // of an SM

struct VecKernel {
    const void *fn;
    size_t ring;
    int threads, blocks;  // of a block; blocks an SM's registers hold
};

// The fewest threads whose `most` vectors hold a row, whole warps of them from a warp on; more, with
// fewer vectors, while the rows are too few to give every SM a block.
VecPlan plan_vec(long long rows, int C, bool fp32, int most, bool warps, bool shift, int sm_count) {
    VecPlan p;
    const int ch = fp32 ? 4 : 8, nv = (C + ch - 1 + (shift ? ch - 1 : 0)) / ch;
    p.tpr = 8;
    while (p.tpr < 32 && p.tpr * std::min(4, most) < nv) p.tpr *= 2;
    while (p.tpr * most < nv) p.tpr += warps && p.tpr >= 128 ? 32 : p.tpr;
    while (p.tpr * 2 <= VEC_THREADS && p.tpr < nv && rows * p.tpr * 2 <= (long long)VEC_THREADS * sm_count) p.tpr *= 2;
    if (p.tpr > VEC_THREADS) return VecPlan();
    p.v = (nv + p.tpr - 1) / p.tpr;
    p.rpb = VEC_THREADS / p.tpr;
    return p;
}

// `arrays`: channel-wise arrays in shared memory; `row`: bytes of a thread's vector of a row there.
// (A vector of a row that begins otherwise is read from up to 28 bytes beside its place, a word more than it has.)
size_t vec_smem(const VecKernel &k, const VecPlan &v, bool fp32, int arrays, int row) {
    return k.ring + (size_t)arrays * (fp32 ? 4 : 8) * v.v * v.tpr * sizeof(float) + (row ? (size_t)row * k.threads * v.v + 64 : 0);
}

template <typename P>
dlcStatus_t launch_vec(dlcContext *ctx, const VecKernel &k, P &p, const VecPlan &v, bool fp32, bool shift, int arrays, int row,
                       int *blocks = nullptr) {
    int tpr = v.tpr;
    const size_t smem = vec_smem(k, v, fp32, arrays, row);
    const int per_sm = std::max(1, std::min(k.blocks, (int)(VEC_SM_SMEM / (smem + 1536))));  // (static, and what the system takes)
    long long n = std::min((p.rows + v.rpb - 1) / v.rpb, (long long)ctx->sm_count * per_sm);
    if (shift) n = std::max(8ll, std::min((n + 7) / 8 * 8, (long long)ctx->sm_count * per_sm / 8 * 8));  // (Cover)
    if (blocks) *blocks = (int)n;
    void *args[] = {&p, &tpr};
    if (!dlc_allow_smem(ctx, k.fn, smem)) return DLC_STATUS_EXECUTION_FAILED;
    return dlc_launch(ctx, k.fn, dim3((unsigned)n), dim3((unsigned)k.threads), smem, args);
}

template <int V, typename E, typename Y, bool RES, bool SHIFT>
VecKernel vec_fwd() {
    return {(const void *)layer_vec_kernel<V, E, Y, RES, SHIFT>, VecRing<V, E, RES ? 2 : 1, vec_ring<V>(), VEC_THREADS>::SMEM, VEC_THREADS,
            vec_blocks<V, E>()};
}

template <int V, typename E, bool SHIFT>
VecKernel vec_fwd(const LayerProblem &p) {
    const bool res = p.r.p != nullptr;
    if (p.y.dt == DLC_DATA_BFLOAT16) return res ? vec_fwd<V, E, unsigned short, true, SHIFT>() : vec_fwd<V, E, unsigned short, false, SHIFT>();
    if (p.y.dt == DLC_DATA_FLOAT) return res ? vec_fwd<V, E, float, true, SHIFT>() : vec_fwd<V, E, float, false, SHIFT>();
    return res ? vec_fwd<V, E, unsigned char, true, SHIFT>() : vec_fwd<V, E, unsigned char, false, SHIFT>();
}

template <int V, typename E, int TH, bool SHIFT>
VecKernel vec_bwd(bool res) {
    constexpr int S = vec_bwd_ring<V>();
    return res ? VecKernel{(const void *)layer_bwd_vec_kernel<V, E, true, TH, SHIFT>, VecRing<V, E, 3, S, TH>::SMEM, TH, 512 / TH}
               : VecKernel{(const void *)layer_bwd_vec_kernel<V, E, false, TH, SHIFT>, VecRing<V, E, 2, S, TH>::SMEM, TH, 512 / TH};
}

// (a row of more than 128 threads has a block of its own: 160, 192 or 224 threads where they are enough)
template <int V, typename E, bool SHIFT>
VecKernel vec_bwd(int tpr, bool res) {
    return tpr == 160   ? vec_bwd<V, E, 160, SHIFT>(res)
           : tpr == 192 ? vec_bwd<V, E, 192, SHIFT>(res)
           : tpr == 224 ? vec_bwd<V, E, 224, SHIFT>(res)
                        : vec_bwd<V, E, 256, SHIFT>(res);
}

template <bool SHIFT>
VecKernel vec_bwd(const VecPlan &v, bool fp32, bool res) {
    using Half = unsigned short;
    if (!fp32) return v.v == 1 ? vec_bwd<1, Half, 256, SHIFT>(res) : vec_bwd<2, Half, SHIFT>(v.tpr, res);
    switch (v.v) {
        case 1: return vec_bwd<1, float, 256, SHIFT>(res);
        case 2: return vec_bwd<2, float, 256, SHIFT>(res);
        case 3: return vec_bwd<3, float, 256, SHIFT>(res);
        default: return vec_bwd<4, float, SHIFT>(v.tpr, res);
    }
}

}  // namespace

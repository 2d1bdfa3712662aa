// norm_rows.cuh -- what the norms over a row's channels share: rows in registers
// and their reductions over a row's threads, the two-pass layouts' mapping, the
// E4M3 scale of a row, and the plan of a launch.
#pragma once

#include <initializer_list>

#include "channel.cuh"
#include "ptx.cuh"
#include "row_ring.cuh"

namespace dlc {

constexpr float E4M3_MAX = 448.f;
constexpr float SCALE_FLOOR = 1e-30f;  // max |y| of an all-zero row counts as this
constexpr int NORM_THREADS = 256;
constexpr int NORM_MAX_WARPS = 32;

// A ring that a block's shared memory cannot hold (FP32 rows of 8193 to 16384 channels:
// 256 KiB forward, 384 backward) gives way to one row ahead in registers forward, and to the
// two-pass kernel backward, where the registers spill.  2730 x 12288: forward 171 us;
// backward 261 us, 433 through registers.
constexpr size_t NORM_MAX_RING = 226 * 1024;

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
__device__ __forceinline__ float2 row_reduce(float a, float b, int tpr, int slot, float2 (*buf)[NORM_MAX_WARPS], int parity) {
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

// rho^3 * mean(d t): about rho^2 for rows of any size, where rho^3 alone is out of
// FP32's range for rows of 1e-13 or 1e13.
__device__ __forceinline__ float row_slope(float rho, float mean) { return rho * (rho * (rho * mean)); }

// Whether a row lies so far from zero that its mean's rounding counts beside its deviations: its values
// are then centred a second time, by the mean of the centred ones.  Up to eight deviations the mean's chain of up
// to some 50 additions is at most 2.5e-5 of a deviation off.  A row of equal channels, whose deviations are
// all rounding, is zeros after the second time: its centred values are the same few steps in every channel, so that
// their sum and its quotient are exact.  Other rows pay for a comparison, a vote and a branch: nothing that
// shows forward, 2 to 5 % backward, where a row's reductions are what it waits for (16384 x 2048 BF16 44.2 and
// 46.4 us; with the second mean summed up for every row 47.4).
__device__ __forceinline__ bool far_row(float mean, float variance) { return mean * mean > 64.f * variance; }

// The remaining layouts, two passes over a row.  LANES (channels apart): 32
// rows a block, one per lane, the channels dealt to eight warps, so neighbouring
// rows share the loads.  Otherwise (a row too long for registers): one row a
// block, its channels dealt to the threads.  The second pass recomputes t (so t
// may overwrite x or r in place); it finds most of a row in the L1 or L2, and the
// loads' latency bounds these layouts, four a thread in flight.
constexpr int AHEAD = 4;  // channels a thread loads at once

template <bool LANES>
struct AnyMap {
    static constexpr int ROWS = LANES ? 32 : 1, STEP = LANES ? 8 : NORM_THREADS;
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
        for (int i = 0; i < NORM_THREADS / 32; ++i) {
            const float2 v = part[i][lane];
            a += v.x;
            b = MAX_B ? fmaxf(b, v.y) : b + v.y;
        }
        return make_float2(a, b);
    }
};

// ---- host side ---------------------------------------------------------------

struct RowPlan {
    int w = 0, v = 0;  // channels per vector (0: the two-pass kernels), vectors per thread
    bool lanes = false;
    int tpr = 0, threads = 0;
    long long blocks = 0;
};

// Whether every row of t can be read in 16-byte vectors of eight channels.
inline bool vec_ok(const RowTensor &t) {
    if (!t.p) return true;
    const int e = dlc_dtype_bytes((dlcDataType_t)t.dt);
    const long long b = e == 1 ? 8 : 16;
    auto mult = [&](long long s) { return (s * e) % b == 0; };
    return (uintptr_t)t.p % b == 0 &&
           (t.m.uniform ? mult(t.m.ld) : (mult(t.m.s0) && mult(t.m.s2) && mult(t.m.s3)));
}

inline bool contiguous(const RowTensor &t) { return !t.p || t.m.cs == 1; }

inline bool all_of(int dt, std::initializer_list<RowTensor> ts) {
    for (const RowTensor &t : ts)
        if (t.p && t.dt != dt) return false;
    return true;
}

inline bool ring(std::initializer_list<RowTensor> ts) { return all_of(DLC_DATA_BFLOAT16, ts) || all_of(DLC_DATA_FLOAT, ts); }

inline RowPlan plan_rows(long long rows, int C, bool cs1, bool vec, bool ring, int per_sm, int sm_count) {
    RowPlan r;
    r.threads = NORM_THREADS;
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
        if (r.w && tpr > NORM_THREADS) r.threads = tpr;
    }
    const int rpb = r.w ? r.threads / r.tpr : (r.lanes ? 32 : 1);
    const long long need = (rows + rpb - 1) / rpb;
    const long long most = (long long)sm_count * (r.w ? (r.threads > NORM_THREADS ? 1 : per_sm) : 4);
    r.blocks = need < most ? need : most;
    return r;
}

// One row a block at a time, twice over it.
inline RowPlan two_pass_rows(long long rows, int sm_count) {
    RowPlan r;
    r.threads = NORM_THREADS;
    r.blocks = std::min(rows, (long long)sm_count * 4);
    return r;
}

// Rows that may be copied in the 16-byte pieces they touch: the first row
// starts one, so no piece starts before the tensor.
inline bool pieces_ok(const RowTensor &t) {
    return !t.p || (t.dt == DLC_DATA_BFLOAT16 && t.m.uniform && (uintptr_t)t.p % 16 == 0);
}

struct RowKernel {
    const void *fn;
    size_t smem;
};

}  // namespace dlc

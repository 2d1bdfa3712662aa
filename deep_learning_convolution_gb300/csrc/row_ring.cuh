// row_ring.cuh -- how the row-wise kernels read: vectors of a row per thread,
// the next rows prefetched, addresses that step from row to row.
#pragma once

#include "channel.cuh"
#include "ptx.cuh"

namespace dlc {

// E = V * W values of one row held by a thread: V vectors of W consecutive
// channels.  W = 8 (contiguous, 16-byte aligned) or 1 (any stride).
template <int W, int V>
struct Cols {
    int c[V];   // first channel of each vector, 0 where the vector is past the row
    int n[V];   // channels of it that exist, 0 .. W
    int count;  // vectors that exist (the first ones)
    int step;   // channels from one vector to the next
    __device__ __forceinline__ Cols(int t, int tpr, int C) {
        step = tpr * W;
        count = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int at = (t + j * tpr) * W;
            n[j] = min(max(C - at, 0), W);
            c[j] = n[j] ? at : 0;
            count += n[j] ? 1 : 0;
        }
    }
};

// V vectors of a row as FP32; a partial vector is read element by element, so
// nothing past the row is touched.
template <int W, int V>
__device__ __forceinline__ void load_row(const RowTensor &t, const char *at, const Cols<W, V> &k, float (&f)[V * W]) {
    if constexpr (W == 1) {  // single elements a fixed step apart
        const long long step = k.step * t.m.cs;
        if (t.dt == DLC_DATA_BFLOAT16) {
            const unsigned short *p = reinterpret_cast<const unsigned short *>(at);
            unsigned short w[V];
#pragma unroll
            for (int j = 0; j < V; ++j, p += step) w[j] = j < k.count ? *p : (unsigned short)0;
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] = bf16_bits_f32(w[j]);
        } else {
            const float *p = reinterpret_cast<const float *>(at);
#pragma unroll
            for (int j = 0; j < V; ++j, p += step) f[j] = j < k.count ? *p : 0.f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float *v = f + j * W;
            const int d = j < k.count ? j * k.step : 0;
            if (k.n[j] == W) {
                if (t.dt == DLC_DATA_BFLOAT16) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(reinterpret_cast<const unsigned short *>(at) + d);
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int i = 0; i < W / 2; ++i) v[2 * i] = unpack_bf16(w[i]).x, v[2 * i + 1] = unpack_bf16(w[i]).y;
                } else {
                    const float4 *p = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(at) + d);
#pragma unroll
                    for (int i = 0; i < W / 4; ++i) {
                        const float4 a = p[i];
                        v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = a.z, v[4 * i + 3] = a.w;
                    }
                }
            } else {
                load_elems<W>(at, t.dt, d, 1, [&](int i) { return i < k.n[j]; }, v);
            }
        }
    }
}

// How the rows of a kernel's tensors are read: one row ahead in registers, or
// through a ring in shared memory where all of them are BF16 or all FP32.
enum { ROWS_REGS = 0, ROWS_BF16 = 1, ROWS_F32 = 2 };

// A thread's next rows of T tensors.  With W = 8 they are copied asynchronously
// into a ring of S rows in shared memory, of which a thread reads back only what
// it copied itself (no barrier), so S - 1 rows of every thread are in flight
// without holding registers; mixed types are read one row ahead into registers.
template <int W, int V, int T>
struct RowsAhead {
    float next[T][V * W];
    static constexpr int AHEAD = 1;
    __device__ __forceinline__ void start(uint32_t, int, int, int, int) {}
    __device__ __forceinline__ void fetch(const RowTensor &t, int k, const char *at, const Cols<W, V> &cols) {
        load_row<W, V>(t, at, cols, next[k]);
    }
    __device__ __forceinline__ void commit() {}
    __device__ __forceinline__ void take(float (&f)[T][V * W], const Cols<W, V> &, const uint32_t (&)[T]) {
#pragma unroll
        for (int k = 0; k < T; ++k)
#pragma unroll
            for (int i = 0; i < V * W; ++i) f[k][i] = next[k][i];
    }
    static constexpr size_t smem(int, int, int) { return 0; }
};

template <int W, int V, int KIND, int T, int S>
struct Rows : RowsAhead<W, V, T> {};

template <int V, int KIND, int T, int S>
struct Rows<8, V, KIND, T, S> {
    static constexpr int E = KIND == ROWS_BF16 ? 2 : 4, Q = E / 2;  // bytes of an element, 16-byte words of a vector
    uint32_t base, put, get, word, row;  // this thread's slot 0, the rows to fill and to read, bytes between words / rows
    static constexpr int AHEAD = S - 1;
    __device__ __forceinline__ void start(uint32_t smem, int, int, int, int) {
        base = smem + threadIdx.x * 16u;
        word = 16u * blockDim.x;
        row = (uint32_t)(T * V * Q) * word;
        put = get = 0;
    }
    __device__ __forceinline__ void fetch(const RowTensor &, int k, const char *at, const Cols<8, V> &cols) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const char *p = at + (j < cols.count ? E * j * cols.step : 0);
            const int bytes = E * cols.n[j];
#pragma unroll
            for (int q = 0; q < Q; ++q)
                cp_async_16(base + put + (uint32_t)((k * V + j) * Q + q) * word, bytes > 16 * q ? p + 16 * q : p,
                            (uint32_t)max(0, min(16, bytes - 16 * q)));
        }
    }
    __device__ __forceinline__ void commit() {
        cp_async_commit();
        put = put == row * (S - 1) ? 0 : put + row;
    }
    __device__ __forceinline__ void take(float (&f)[T][V * 8], const Cols<8, V> &, const uint32_t (&)[T]) {
        cp_async_wait<S - 2>();
#pragma unroll
        for (int k = 0; k < T; ++k)
#pragma unroll
            for (int j = 0; j < V * Q; ++j) {
                uint32_t w[4];
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                             : "r"(base + get + (uint32_t)(k * V * Q + j) * word)
                             : "memory");
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (KIND == ROWS_BF16) {
                        const float2 u = unpack_bf16(w[i]);
                        f[k][8 * j + 2 * i] = u.x, f[k][8 * j + 2 * i + 1] = u.y;
                    } else {
                        f[k][4 * j + i] = __uint_as_float(w[i]);
                    }
                }
            }
        get = get == row * (S - 1) ? 0 : get + row;
    }
    static constexpr size_t smem(int threads, int, int) { return (size_t)S * T * V * Q * 16 * threads; }
};

template <int V, int T, int S>
struct Rows<8, V, ROWS_REGS, T, S> : RowsAhead<8, V, T> {};

// BF16 rows at a pitch that is no multiple of 16 bytes, from a 16-byte aligned
// base: the 16-byte pieces that a row touches come asynchronously into a ring of
// rows, dealt to the row's threads (the first piece starts in the row before,
// the last one ends with the row), and each thread takes its elements from
// there.  `starts`: the addresses of the rows, of which the low bits count.
template <int V, int T, int S>
struct Rows<1, V, ROWS_BF16, T, S> {
    uint32_t base, put, get, row;  // this group's slot 0, the rows to fill and to read, bytes of a row of one tensor
    int t, tpr, C, group;
    static constexpr int AHEAD = S - 1;
    static __host__ __device__ uint32_t row_bytes(int C) { return ((uint32_t)C * 2u + 14u + 15u) / 16u * 16u; }
    __device__ __forceinline__ void start(uint32_t smem, int thread, int threads, int slot, int channels) {
        t = thread, tpr = threads, group = slot, C = channels;
        row = row_bytes(C);
        base = smem + (uint32_t)slot * (uint32_t)(S * T) * row;
        put = get = 0;
    }
    __device__ __forceinline__ void fetch(const RowTensor &, int k, const char *at, const Cols<1, V> &cols) {
        const char *p = at - 2 * cols.c[0];  // the row's start
        const uint32_t shift = (uint32_t)reinterpret_cast<uintptr_t>(p) & 15u, bytes = shift + 2u * (uint32_t)C;
        p -= shift;
        const uint32_t dst = base + put + (uint32_t)k * row;
        for (uint32_t i = (uint32_t)t * 16u; i < bytes; i += (uint32_t)tpr * 16u) cp_async_16(dst + i, p + i, min(16u, bytes - i));
    }
    __device__ __forceinline__ void commit() {
        cp_async_commit();
        put = put == (uint32_t)(T * (S - 1)) * row ? 0 : put + (uint32_t)T * row;
    }
    __device__ __forceinline__ void take(float (&f)[T][V], const Cols<1, V> &cols, const uint32_t (&starts)[T]) {
        cp_async_wait<S - 2>();
        // every thread's pieces have arrived, and the row before has been read
        if (tpr > 32)
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
        else
            __syncwarp();
#pragma unroll
        for (int k = 0; k < T; ++k) {
            uint32_t at = base + get + (uint32_t)k * row + (starts[k] & 15u) + 2u * (uint32_t)t;
#pragma unroll
            for (int j = 0; j < V; ++j, at += 2u * (uint32_t)tpr) {
                unsigned short w = 0;
                if (j < cols.count) asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(at) : "memory");
                f[k][j] = bf16_bits_f32(w);
            }
        }
        get = get == (uint32_t)(T * (S - 1)) * row ? 0 : get + (uint32_t)T * row;
    }
    static size_t smem(int threads, int tpr, int C) { return (size_t)S * T * row_bytes(C) * (threads / tpr); }
};

// Where a thread's part of a tensor's rows starts (its element `c` of the row),
// row after row: stepped where the rows have one pitch, worked out from n, h and
// w otherwise.
struct RowWalk {
    char *p;
    long long inc;
    __device__ __forceinline__ RowWalk(const RowTensor &t, long long row, long long step, long long c) {
        const int e = t.dt == DLC_DATA_FLOAT ? 4 : t.dt == DLC_DATA_BFLOAT16 ? 2 : 1;
        p = static_cast<char *>(t.p) + (row * t.m.ld + c) * e;
        inc = step * t.m.ld * e;
    }
    __device__ __forceinline__ char *at(const RowTensor &t, long long row, long long c) const {
        if (t.m.uniform) return p;
        const int e = t.dt == DLC_DATA_FLOAT ? 4 : t.dt == DLC_DATA_BFLOAT16 ? 2 : 1;
        return static_cast<char *>(t.p) + (row_off(t.m, row) + c) * e;
    }
    __device__ __forceinline__ void next() { p += inc; }
};

}  // namespace dlc

// dropout.cu -- dropout from a counter-based generator, with the residual's addition:
//
//   u[m, c] = word c mod 4 of Philox4x32-10 (key: the seed; counter: c / 4, m, step)
//   y[m, c] = r[m, c] + (u[m, c] >= border ? scale * x[m, c] : 0)
//
// border = floor(p 2^32), scale = 2^32 / (2^32 - border), so the mean is kept exactly.  The
// mask is a function of the element's row and channel, the seed and the step: the
// backward pass (the same with dy for x) works it out again, and nothing of it is stored.
// Philox 4x32 with ten rounds is the generator of Salmon, Moraes, Dror and Shaw, "Parallel
// random numbers: as easy as 1, 2, 3" (2011): a round multiplies two of the four words and
// crosses the halves of the products.
//
// Bound by memory: x (and r) in, y out.
#include <type_traits>

#include "channel.cuh"
#include "ptx.cuh"

namespace {

using namespace dlc;

constexpr int DO_THREADS = 256;

struct DoParams {
    DropoutProblem d;
    long long items, inner;  // pieces of a row's channels; the faster index runs over `inner` of them
    int apart;               // ... over the rows, because channels are apart
    int flat;                // dense rows all: pieces one after the other
};

struct Philox {
    uint32_t k0[10], k1[10], s0, s1;  // the rounds' keys, once a thread
    __device__ __forceinline__ explicit Philox(const unsigned long long *random) {
        const unsigned long long seed = random[0], step = random[1];
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            k0[i] = (uint32_t)seed + (uint32_t)i * 0x9E3779B9u;
            k1[i] = (uint32_t)(seed >> 32) + (uint32_t)i * 0xBB67AE85u;
        }
        s0 = (uint32_t)step, s1 = (uint32_t)(step >> 32);
    }
    __device__ __forceinline__ void words(uint32_t group, uint32_t row, uint32_t (&u)[4]) const {
        uint32_t a = group, b = row, c = s0, d = s1;
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const unsigned long long l = (unsigned long long)a * 0xD2511F53u, r = (unsigned long long)c * 0xCD9E8D57u;
            a = (uint32_t)(r >> 32) ^ b ^ k0[i];
            c = (uint32_t)(l >> 32) ^ d ^ k1[i];
            b = (uint32_t)r;
            d = (uint32_t)l;
        }
        u[0] = a, u[1] = b, u[2] = c, u[3] = d;
    }
};

// W channels of a row from memory: eight in 16-byte accesses, or up to four at any stride.
template <int W, typename E>
struct Piece {
    E v[W];
    __device__ __forceinline__ void load(const RowTensor &t, long long off, int n) {
        const E *p = static_cast<const E *>(t.p) + off;
        if constexpr (W == 8) {
            constexpr int Q = (int)sizeof(E) / 2;
#pragma unroll
            for (int i = 0; i < Q; ++i) reinterpret_cast<uint4 *>(v)[i] = reinterpret_cast<const uint4 *>(p)[i];
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] = i < n ? p[i * t.m.cs] : (E)0;
        }
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (sizeof(E) == 2)
            return bf16_bits_f32(v[i]);
        else
            return v[i];
    }
};

template <int W, typename E>
__device__ __forceinline__ void put(const RowTensor &t, long long off, int n, const float (&f)[W]) {
    E *p = static_cast<E *>(t.p) + off;
    if constexpr (W == 8 && sizeof(E) == 2) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    } else if constexpr (W == 8) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (i < n) store_elem(t.p, sizeof(E) == 2 ? DLC_DATA_BFLOAT16 : DLC_DATA_FLOAT, off + i * t.m.cs, f[i]);
    }
}

// W = 8: rows of whole aligned vectors of eight channels, fewer than 2^31 of them; W = 4: any layout.
// U pieces a thread are in flight together; a thread steps from piece to piece without dividing.
template <int W, typename X, typename R, typename Y>
__global__ void __launch_bounds__(DO_THREADS) dropout_kernel(const __grid_constant__ DoParams p) {
    griddep_launch_dependents();
    using I = typename std::conditional<W == 8, uint32_t, long long>::type;
    constexpr int U = 4;
    const I items = (I)p.items, inner = (I)p.inner, step = (I)gridDim.x * DO_THREADS;
    I i = (I)blockIdx.x * DO_THREADS + threadIdx.x;
    I out = i / inner, in = i - out * inner;
    const I dout = step / inner, din = step - dout * inner;
    griddep_wait();
    const Philox gen(p.d.random);
    const bool res = p.d.r.p != nullptr;
    while (i < items) {
        Piece<W, X> x[U];
        Piece<W, R> r[U];
        uint32_t row[U], piece[U];
        long long at[U];  // element of y
        int n[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            n[k] = 0;
            if (i < items) {
                row[k] = (uint32_t)(p.apart ? in : out);
                piece[k] = (uint32_t)(p.apart ? out : in);
                n[k] = W == 8 ? 8 : min(W, p.d.C - (int)piece[k] * W);
                if (p.flat) {
                    at[k] = (long long)i * W;
                    x[k].load(p.d.x, at[k], n[k]);
                    if (res) r[k].load(p.d.r, at[k], n[k]);
                } else {
                    const long long c = (long long)piece[k] * W;
                    at[k] = row_off(p.d.y.m, row[k]) + c * p.d.y.m.cs;
                    x[k].load(p.d.x, row_off(p.d.x.m, row[k]) + c * p.d.x.m.cs, n[k]);
                    if (res) r[k].load(p.d.r, row_off(p.d.r.m, row[k]) + c * p.d.r.m.cs, n[k]);
                }
            }
            i += step, out += dout, in += din;
            if (in >= inner) in -= inner, ++out;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (n[k] == 0) break;
            float f[W];
#pragma unroll
            for (int h = 0; h < W / 4; ++h) {
                uint32_t u[4];
                gen.words(piece[k] * (W / 4) + h, row[k], u);
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    const int e = 4 * h + j;
                    const float2 v = mul2(make_float2(x[k].at(e), x[k].at(e + 1)), pair_of(p.d.scale));
                    f[e] = u[j] >= p.d.border ? v.x : 0.f;
                    f[e + 1] = u[j + 1] >= p.d.border ? v.y : 0.f;
                }
            }
            if (res) {
#pragma unroll
                for (int j = 0; j < W; j += 2) set2(f + j, 0, add2(get2(f + j, 0), make_float2(r[k].at(j), r[k].at(j + 1))));
            }
            put<W, Y>(p.d.y, at[k], n[k], f);
        }
    }
}

using Half = unsigned short;

template <int W, typename X, typename R>
const void *do_kernel(int y) {
    return y == DLC_DATA_BFLOAT16 ? (const void *)dropout_kernel<W, X, R, Half> : (const void *)dropout_kernel<W, X, R, float>;
}

template <int W>
const void *do_kernel(const DropoutProblem &d) {
    const bool x = d.x.dt == DLC_DATA_BFLOAT16, r = d.r.p ? d.r.dt == DLC_DATA_BFLOAT16 : x;
    if (x) return r ? do_kernel<W, Half, Half>(d.y.dt) : do_kernel<W, Half, float>(d.y.dt);
    return r ? do_kernel<W, float, Half>(d.y.dt) : do_kernel<W, float, float>(d.y.dt);
}

}  // namespace

dlcStatus_t dlc_launch_dropout(dlcContext *ctx, const DropoutProblem &pb) {
    DoParams p;
    p.d = pb;
    auto vec = [&](const RowTensor &t) { return !t.p || (t.m.cs == 1 && dlc_aligned_rows(t, 16)); };
    const bool w8 = pb.C % 8 == 0 && vec(pb.x) && vec(pb.r) && vec(pb.y) && pb.rows * (pb.C / 8) < 0x60000000LL;
    const int w = w8 ? 8 : 4;
    const long long pieces = (pb.C + w - 1) / w;
    p.items = pb.rows * pieces;
    p.apart = pb.x.m.cs != 1 && pb.y.m.cs != 1;
    p.inner = p.apart ? pb.rows : pieces;
    auto flat = [&](const RowTensor &t) { return !t.p || (t.m.uniform && (t.m.ld == pb.C || pb.rows == 1)); };
    p.flat = w8 && flat(pb.x) && flat(pb.r) && flat(pb.y);
    const void *kern = w8 ? do_kernel<8>(pb) : do_kernel<4>(pb);
    const long long blocks = std::min<long long>((p.items + DO_THREADS - 1) / DO_THREADS, (long long)ctx->sm_count * 8);
    void *args[] = {&p};
    return dlc_launch(ctx, kern, dim3((unsigned)blocks), dim3(DO_THREADS), 0, args);
}

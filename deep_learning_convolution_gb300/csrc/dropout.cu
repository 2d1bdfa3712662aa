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
// x (and r) in, y out: memory bounds it with a residual, the generator close behind.  Without, no single thing does: DRAM
// 49 %, issue 55 %, integer pipe 55 %, the busiest pipe 66 % of their rates, and the five warps a scheduler has wait in
// about equal parts for loads, for the round before and for the multiplies.  16384 x 4096 BF16 63.8 us with
// residual (6.3 TB/s) and 57 us without (4.7); unaligned rows, 16384 x 1001 with
// residual, 27 us; channels apart, 128 images of 512 x 28 x 28, 172 us (1.2 TB/s).
#include "channel.cuh"
#include "ptx.cuh"

namespace {

using namespace dlc;

constexpr int DO_THREADS = 256, DO_BLOCKS = 3;  // blocks an SM holds

struct DoParams {
    DropoutProblem d;
    long long items, inner;  // pieces of a row's channels; the faster index runs over `inner` of them
    int apart;               // ... over the rows, because channels are apart
    int rows_step;           // rows that the threads of the columns kernel take at once
};

constexpr uint32_t PHILOX_M0 = 0xD2511F53u, PHILOX_M1 = 0xCD9E8D57u, PHILOX_W0 = 0x9E3779B9u, PHILOX_W1 = 0xBB67AE85u;

__device__ __forceinline__ void wide(uint32_t a, uint32_t m, uint32_t &hi, uint32_t &lo) {
    const unsigned long long p = (unsigned long long)a * m;
    hi = (uint32_t)(p >> 32);
    lo = (uint32_t)p;
}

struct Philox {
    uint32_t k0[10], k1[10], s0, s1;  // the rounds' keys, once a thread
    __device__ __forceinline__ explicit Philox(const unsigned long long *random) {
        const unsigned long long seed = random[0], step = random[1];
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            k0[i] = (uint32_t)seed + (uint32_t)i * PHILOX_W0;
            k1[i] = (uint32_t)(seed >> 32) + (uint32_t)i * PHILOX_W1;
        }
        s0 = (uint32_t)step, s1 = (uint32_t)(step >> 32);
    }
    // rounds FIRST .. 9
    template <int FIRST>
    __device__ __forceinline__ void rounds(uint32_t (&u)[4]) const {
#pragma unroll
        for (int i = FIRST; i < 10; ++i) {
            uint32_t lh, ll, rh, rl;
            wide(u[0], PHILOX_M0, lh, ll);
            wide(u[2], PHILOX_M1, rh, rl);
            u[0] = rh ^ u[1] ^ k0[i];
            u[2] = lh ^ u[3] ^ k1[i];
            u[1] = rl;
            u[3] = ll;
        }
    }
    __device__ __forceinline__ void words(uint32_t group, uint32_t row, uint32_t (&u)[4]) const {
        u[0] = group, u[1] = row, u[2] = s0, u[3] = s1;
        rounds<0>(u);
    }
};

// What the first three rounds owe to the channel alone: with the counter (g, m, s0, s1)
//   round 0   (hi(M1 s0) ^ m ^ k0,  lo(M1 s0),  hi(M0 g) ^ s1 ^ k1,  lo(M0 g))
//   round 1   (hi(M1 c) ^ lo(M1 s0) ^ k0',  lo(M1 c),  hi(M0 a) ^ lo(M0 g) ^ k1',  lo(M0 a))
// where c, round 0's third word, is the channel's and a, its first, the row's; so round 1's first
// two words are the channel's too, and of round 2's products only one is not.
struct PhiloxColumn {
    uint32_t third, product, second;  // lo(M0 g) ^ k1'; hi(M0 first) ^ k1''; lo(M1 c) ^ k0''
    uint32_t last;                    // lo(M0 first)
    __device__ __forceinline__ PhiloxColumn(const Philox &p, uint32_t group) {
        uint32_t hi, lo, h0, l0, first;
        wide(group, PHILOX_M0, hi, lo);
        third = lo ^ p.k1[1];
        wide(p.s0, PHILOX_M1, h0, l0);
        wide(hi ^ p.s1 ^ p.k1[0], PHILOX_M1, hi, second);
        first = hi ^ l0 ^ p.k0[1];
        second ^= p.k0[2];
        wide(first, PHILOX_M0, product, last);
        product ^= p.k1[2];
    }
    // hi, lo: M0 times round 0's first word
    __device__ __forceinline__ void words(const Philox &p, uint32_t hi, uint32_t lo, uint32_t (&u)[4]) const {
        uint32_t rh, rl;
        wide(hi ^ third, PHILOX_M1, rh, rl);
        u[0] = rh ^ second;
        u[1] = rl;
        u[2] = product ^ lo;
        u[3] = last;
        p.rounds<3>(u);
    }
};

// W channels of a row from memory: eight in 16-byte accesses, or up to four at any stride.
template <int W, typename E>
struct Piece {
    alignas(16) E v[W];
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
    __device__ __forceinline__ void load_some(const RowTensor &t, long long off, int n) {
        const E *p = static_cast<const E *>(t.p) + off;
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = i < n ? p[i] : (E)0;
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

// Contiguous channels, rows at one pitch: a thread keeps its W channels and steps from row to row, so
// what the generator owes to the channel is worked out once; U rows are in flight.  W = 8: aligned whole
// vectors; W = 4: single elements.  The generator takes 31 wide multiplies for eight channels
// (37 without this), a warp's at four cycles each, and some 80 other integer instructions: about half of the time of a
// call without residual each.
template <int W, typename X, typename R, typename Y>
__global__ void __launch_bounds__(DO_THREADS, DO_BLOCKS) dropout_columns_kernel(const __grid_constant__ DoParams p) {
    griddep_launch_dependents();
    constexpr int U = W == 8 && sizeof(X) + sizeof(R) > 4 ? 2 : 4, G = W / 4;
    const uint32_t pieces = (uint32_t)p.inner, i = blockIdx.x * DO_THREADS + threadIdx.x;
    const uint32_t row0 = i / pieces, piece = i - row0 * pieces;
    if (row0 >= (uint32_t)p.rows_step) return;
    const int n = min(W, p.d.C - (int)piece * W);
    griddep_wait();
    const Philox gen(p.d.random);
    const PhiloxColumn left(gen, G * piece), right(gen, G * piece + 1);
    const bool res = p.d.r.p != nullptr;
    uint32_t h0, l0;
    wide(gen.s0, PHILOX_M1, h0, l0);
    h0 ^= gen.k0[0];
    const long long c = (long long)W * piece;
    long long px = row0 * p.d.x.m.ld + c, pr = row0 * p.d.r.m.ld + c, py = row0 * p.d.y.m.ld + c;
    const long long dx = p.rows_step * p.d.x.m.ld, dr = p.rows_step * p.d.r.m.ld, dy = p.rows_step * p.d.y.m.ld;
    for (long long row = row0; row < p.d.rows; row += (long long)U * p.rows_step) {
        Piece<W, X> x[U];
        Piece<W, R> r[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (row + k * p.rows_step < p.d.rows) {
                x[k].load(p.d.x, px, n);
                if (res) r[k].load(p.d.r, pr, n);
                px += dx;
                pr += dr;
            }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (row + k * p.rows_step >= p.d.rows) break;
            uint32_t hi, lo, u[W];
            wide(h0 ^ (uint32_t)(row + k * p.rows_step), PHILOX_M0, hi, lo);
            left.words(gen, hi, lo, *reinterpret_cast<uint32_t(*)[4]>(u));
            if constexpr (G == 2) right.words(gen, hi, lo, *reinterpret_cast<uint32_t(*)[4]>(u + 4));
            float f[W];
#pragma unroll
            for (int j = 0; j < W; j += 2) {
                const float2 v = mul2(make_float2(x[k].at(j), x[k].at(j + 1)), pair_of(p.d.scale));
                f[j] = u[j] >= p.d.border ? v.x : 0.f;
                f[j + 1] = u[j + 1] >= p.d.border ? v.y : 0.f;
            }
            if (res) {
#pragma unroll
                for (int j = 0; j < W; j += 2) set2(f + j, 0, add2(get2(f + j, 0), make_float2(r[k].at(j), r[k].at(j + 1))));
            }
            put<W, Y>(p.d.y, py, n, f);
            py += dy;
        }
    }
}

// Rows that begin anywhere in a 16-byte piece, all of them alike: the pieces are vectors of eight channels, whose
// groups of four words begin `off` channels ahead, so up to three groups make a vector's words.  A thread's
// rows are a multiple of eight apart, and begin alike.  BF16: FP32 rows gain nothing from vectors, which cost them
// half as many words again (16384 x 1001 36.4 us either way, without residual 30.0 and 28.7).
__global__ void __launch_bounds__(DO_THREADS, DO_BLOCKS) dropout_shift_kernel(const __grid_constant__ DoParams p) {
    griddep_launch_dependents();
    using E = unsigned short;
    constexpr int W = 8, U = 2;
    const uint32_t pieces = (uint32_t)p.inner, i = blockIdx.x * DO_THREADS + threadIdx.x;
    const uint32_t row0 = i / pieces, piece = i - row0 * pieces;
    const int lead = (int)(row0 % 8u * (uint32_t)(p.d.x.m.ld % 8)) % 8;
    const int c = W * (int)piece - lead, skip = max(-c, 0), n = min(W, p.d.C - c);
    if (row0 >= (uint32_t)p.rows_step || n <= 0) return;
    const int off = -lead & 3;
    const uint32_t group = (uint32_t)((c - off) / 4);  // (exact)
    griddep_wait();
    const Philox gen(p.d.random);
    const PhiloxColumn first(gen, group), second(gen, group + 1), third(gen, group + 2);
    const bool res = p.d.r.p != nullptr;
    uint32_t h0, l0;
    wide(gen.s0, PHILOX_M1, h0, l0);
    h0 ^= gen.k0[0];
    long long px = row0 * p.d.x.m.ld + c, pr = row0 * p.d.r.m.ld + c, py = row0 * p.d.y.m.ld + c;
    const long long dx = p.rows_step * p.d.x.m.ld, dr = p.rows_step * p.d.r.m.ld, dy = p.rows_step * p.d.y.m.ld;
    for (long long row = row0; row < p.d.rows; row += (long long)U * p.rows_step) {
        Piece<W, E> x[U];
        Piece<W, E> r[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const long long at = row + k * p.rows_step;
            if (at < p.d.rows) {
                // (a piece that the next row begins in; the first row begins a piece)
                const bool whole = n == W || at + 1 < p.d.rows;
                if (whole)
                    x[k].load(p.d.x, px, W);
                else
                    x[k].load_some(p.d.x, px, n);
                if (res && whole) r[k].load(p.d.r, pr, W);
                if (res && !whole) r[k].load_some(p.d.r, pr, n);
                px += dx;
                pr += dr;
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (row + k * p.rows_step >= p.d.rows) break;
            uint32_t hi, lo, u[12];
            wide(h0 ^ (uint32_t)(row + k * p.rows_step), PHILOX_M0, hi, lo);
            first.words(gen, hi, lo, *reinterpret_cast<uint32_t(*)[4]>(u));
            second.words(gen, hi, lo, *reinterpret_cast<uint32_t(*)[4]>(u + 4));
            if (off) {
                third.words(gen, hi, lo, *reinterpret_cast<uint32_t(*)[4]>(u + 8));
#pragma unroll
                for (int j = 0; j < 10; ++j) u[j] = off & 2 ? u[j + 2] : u[j];
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] = off & 1 ? u[j + 1] : u[j];
            }
            float f[W];
#pragma unroll
            for (int j = 0; j < W; j += 2) {
                const float2 v = mul2(make_float2(x[k].at(j), x[k].at(j + 1)), pair_of(p.d.scale));
                f[j] = u[j] >= p.d.border ? v.x : 0.f;
                f[j + 1] = u[j + 1] >= p.d.border ? v.y : 0.f;
            }
            if (res) {
#pragma unroll
                for (int j = 0; j < W; j += 2) set2(f + j, 0, add2(get2(f + j, 0), make_float2(r[k].at(j), r[k].at(j + 1))));
            }
            if (skip == 0 && n == W) {
                put<W, E>(p.d.y, py, n, f);
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j)
                    if (j >= skip && j < n) store_elem(p.d.y.p, DLC_DATA_BFLOAT16, py + j, f[j]);
            }
            py += dy;
        }
    }
}

// Any other layout: pieces of up to four channels, U of a thread in flight together; a thread steps from
// piece to piece without dividing.
template <typename X, typename R, typename Y>
__global__ void __launch_bounds__(DO_THREADS, 2) dropout_kernel(const __grid_constant__ DoParams p) {
    griddep_launch_dependents();
    constexpr int U = 4, W = 4;
    const long long step = (long long)gridDim.x * DO_THREADS;
    long long i = (long long)blockIdx.x * DO_THREADS + threadIdx.x;
    long long out = i / p.inner, in = i - out * p.inner;
    const long long dout = step / p.inner, din = step - dout * p.inner;
    griddep_wait();
    const Philox gen(p.d.random);
    const bool res = p.d.r.p != nullptr;
    while (i < p.items) {
        Piece<W, X> x[U];
        Piece<W, R> r[U];
        uint32_t row[U], piece[U];
        int n[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            n[k] = 0;
            if (i < p.items) {
                row[k] = (uint32_t)(p.apart ? in : out);
                piece[k] = (uint32_t)(p.apart ? out : in);
                const long long c = (long long)piece[k] * W;
                n[k] = (int)min((long long)W, p.d.C - c);
                x[k].load(p.d.x, row_off(p.d.x.m, row[k]) + c * p.d.x.m.cs, n[k]);
                if (res) r[k].load(p.d.r, row_off(p.d.r.m, row[k]) + c * p.d.r.m.cs, n[k]);
            }
            i += step, out += dout, in += din;
            if (in >= p.inner) in -= p.inner, ++out;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (n[k] == 0) break;
            float f[W];
            uint32_t u[4];
            gen.words(piece[k], row[k], u);
#pragma unroll
            for (int j = 0; j < W; ++j) f[j] = u[j] >= p.d.border ? x[k].at(j) * p.d.scale : 0.f;
            if (res) {
#pragma unroll
                for (int j = 0; j < W; ++j) f[j] += r[k].at(j);
            }
            put<W, Y>(p.d.y, row_off(p.d.y.m, row[k]) + (long long)piece[k] * W * p.d.y.m.cs, n[k], f);
        }
    }
}

using Half = unsigned short;

enum { ANY, SINGLES, SHIFTED, VECTORS };

template <typename X, typename R, typename Y>
const void *do_kernel(int way) {
    return way == VECTORS   ? (const void *)dropout_columns_kernel<8, X, R, Y>
           : way == SINGLES ? (const void *)dropout_columns_kernel<4, X, R, Y>
                            : (const void *)dropout_kernel<X, R, Y>;
}

template <typename X, typename R>
const void *do_kernel(int y, int way) {
    return y == DLC_DATA_BFLOAT16 ? do_kernel<X, R, Half>(way) : do_kernel<X, R, float>(way);
}

const void *do_kernel(const DropoutProblem &d, int way) {
    if (way == SHIFTED) return (const void *)dropout_shift_kernel;
    const bool x = d.x.dt == DLC_DATA_BFLOAT16, r = d.r.p ? d.r.dt == DLC_DATA_BFLOAT16 : x;
    if (x) return r ? do_kernel<Half, Half>(d.y.dt, way) : do_kernel<Half, float>(d.y.dt, way);
    return r ? do_kernel<float, Half>(d.y.dt, way) : do_kernel<float, float>(d.y.dt, way);
}

}  // namespace

dlcStatus_t dlc_launch_dropout(dlcContext *ctx, const DropoutProblem &pb) {
    DoParams p;
    p.d = pb;
    auto columns = [&](const RowTensor &t) { return !t.p || (t.m.cs == 1 && t.m.uniform); };
    auto whole = [&](const RowTensor &t) { return !t.p || dlc_aligned_rows(t, 16); };
    // tensors that begin on a piece, and their rows in the same way; rows that do not overlap, so that what is read behind
    // one is the next one's
    auto alike = [&](const RowTensor &t) {
        return !t.p || (t.dt == DLC_DATA_BFLOAT16 && (uintptr_t)t.p % 16 == 0 && t.m.ld >= pb.C && t.m.ld % 8 == pb.x.m.ld % 8);
    };
    const long long most = (long long)ctx->sm_count * DO_BLOCKS * DO_THREADS;  // threads
    int way = ANY;
    if (columns(pb.x) && columns(pb.r) && columns(pb.y) && pb.C / 4 < most) {
        way = pb.C % 8 == 0 && whole(pb.x) && whole(pb.r) && whole(pb.y) ? VECTORS : SINGLES;
        // (with residual and without, by vectors and by single elements: 16384 x 1001 27.3 / 25.0 and 32.6 / 26.9 us, 777 x
        // 1001 3.1 / 3.0 and 3.7 / 3.4, 60000 x 250 26.0 / 23.9 and 30.1 / 24.9; 16384 x 130 5.9 / 5.6 and 6.2 / 5.4,
        // 200000 x 17 11.9 / 11.3 and 9.2 / 8.0)
        if (way == SINGLES && pb.C >= 192 && alike(pb.x) && alike(pb.r) && alike(pb.y) && (pb.C + 14) / 8 * 8 <= most) way = SHIFTED;
    }
    const int w = way == VECTORS || way == SHIFTED ? 8 : 4;
    const long long pieces = (pb.C + w - 1 + (way == SHIFTED ? 7 : 0)) / w;
    p.items = pb.rows * pieces;
    p.apart = way == ANY && pb.x.m.cs != 1 && pb.y.m.cs != 1;
    p.inner = p.apart ? pb.rows : pieces;
    p.rows_step = (int)std::min(pb.rows, most / pieces);
    if (way == SHIFTED) p.rows_step = (int)(std::min(pb.rows + 7, most / pieces) / 8 * 8);
    const long long threads = way != ANY ? p.rows_step * pieces : std::min(p.items, (long long)ctx->sm_count * 2 * DO_THREADS);
    void *args[] = {&p};
    return dlc_launch(ctx, do_kernel(pb, way), dim3((unsigned)((threads + DO_THREADS - 1) / DO_THREADS)), dim3(DO_THREADS), 0, args);
}

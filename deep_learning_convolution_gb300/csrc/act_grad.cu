// act_grad.cu -- the elementwise step of the linear and gated backward passes:
//
//   dz = dy * act'(z)                                    (linear)
//   dz = [dy * up * act'(gate), dy * act(gate)]          (gated: both halves of a row)
//   dbias = the sum of dz over the rows (of its FP32 values, before dz is rounded)
//
// It reads dy and z once and writes dz once, which bounds it: a warp handles
// 256 neighbouring channels of a row, eight a thread (16-byte accesses of
// BF16), eight rows a block at a time, the column sums staying in registers.
#include "channel.cuh"
#include "ptx.cuh"

namespace {

using namespace dlc;

constexpr int AG_WARPS = 8;

template <int W>
__device__ __forceinline__ void ag_load(const RowTensor &t, long long off, int n, float *v) {
    if (W == 8 && n >= W) {
        if (t.dt == DLC_DATA_BFLOAT16) {
            const uint4 q = *reinterpret_cast<const uint4 *>(static_cast<const unsigned short *>(t.p) + off);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(t.p) + off);
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                const float4 a = f[i];
                v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = a.z, v[4 * i + 3] = a.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = i < n ? load_elem(t.p, t.dt, off + i * t.m.cs) : 0.f;
    }
}

// dz is dense BF16 with rows of a multiple of 16 bytes, so only the vector's
// own channels decide between the two stores.
template <int W>
__device__ __forceinline__ void ag_store(const RowTensor &t, long long off, int n, const float *v) {
    if (W == 8 && n >= W) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < W / 2; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<uint4 *>(static_cast<unsigned short *>(t.p) + off) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (i < n) store_elem(t.p, t.dt, off + i, v[i]);
    }
}

// W = 8: vectors; W = 1: single elements of any strides and alignment.
template <int W, int ACT, bool GATED>
__device__ __forceinline__ void ag_rows(const ActGradProblem &p, float (&sum)[2][8]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = ((int)blockIdx.x * 32 + lane) * W, n = p.N - c;
    for (long long row = (long long)blockIdx.y * AG_WARPS + warp; row < p.rows; row += (long long)gridDim.y * AG_WARPS) {
        if (n <= 0) continue;
        float dy[W], z[W], u[W], a[W], b[W];
        ag_load<W>(p.dy, row_off(p.dy.m, row) + (long long)c * p.dy.m.cs, n, dy);
        if (p.z.p) {
            const long long zo = row_off(p.z.m, row);
            ag_load<W>(p.z, zo + (long long)c * p.z.m.cs, n, z);
            if (GATED) ag_load<W>(p.z, zo + (long long)(p.N + c) * p.z.m.cs, n, u);
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (GATED) {
                float f, df;
                act_both<ACT>(z[i], f, df);
                a[i] = dy[i] * u[i] * df;
                b[i] = dy[i] * f;
                sum[1][i] += b[i];
            } else if (ACT == DLC_ACTIVATION_IDENTITY) {
                a[i] = dy[i];
            } else {
                float f, df;
                act_both<ACT>(z[i], f, df);
                a[i] = dy[i] * df;
            }
            sum[0][i] += a[i];
        }
        if (p.dz.p) {
            const long long zo = row_off(p.dz.m, row);
            ag_store<W>(p.dz, zo + c, n, a);
            if (GATED) ag_store<W>(p.dz, zo + p.N + c, n, b);
        }
    }
}

template <int W>
__global__ void __launch_bounds__(AG_WARPS * 32) act_grad_kernel(const __grid_constant__ ActGradProblem p) {
    griddep_launch_dependents();
    __shared__ float part[AG_WARPS][32 * W];
    float sum[2][8];
    for (int h = 0; h < 2; ++h)
        for (int i = 0; i < 8; ++i) sum[h][i] = 0.f;
    griddep_wait();
    act_dispatch(p.act, [&](auto act) {
        if (p.gated)
            ag_rows<W, decltype(act)::value, true>(p, sum);
        else
            ag_rows<W, decltype(act)::value, false>(p, sum);
    });
    if (!p.dbias) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int width = p.gated ? 2 * p.N : p.N;
    for (int h = 0; h < (p.gated ? 2 : 1); ++h) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) part[warp][lane * W + i] = sum[h][i];
        __syncthreads();
        for (int j = threadIdx.x; j < 32 * W; j += AG_WARPS * 32) {
            const int c = (int)blockIdx.x * 32 * W + j;
            if (c >= p.N) continue;
            float s = 0.f;
            for (int w = 0; w < AG_WARPS; ++w) s += part[w][j];
            p.ws[(long long)blockIdx.y * width + h * p.N + c] = s;
        }
    }
}

struct AgPlan {
    int w;
    unsigned gx, gy;
};

bool ag_vec(const RowTensor &t, int n) {
    if (!t.p) return true;
    const int e = dlc_dtype_bytes((dlcDataType_t)t.dt);
    auto mult = [&](long long s) { return (s * e) % 16 == 0; };
    return t.m.cs == 1 && (uintptr_t)t.p % 16 == 0 && mult(n) &&
           (t.m.uniform ? mult(t.m.ld) : (mult(t.m.s0) && mult(t.m.s2) && mult(t.m.s3)));
}

AgPlan ag_plan(const dlcContext *ctx, const ActGradProblem &p) {
    AgPlan g;
    // a gated row's second half starts N channels in: its vectors need that aligned too
    const int n = p.gated ? p.N : 0;
    g.w = ag_vec(p.dy, 0) && ag_vec(p.z, n) && ag_vec(p.dz, n) ? 8 : 1;
    g.gx = (unsigned)((p.N + 32 * g.w - 1) / (32 * g.w));
    const long long strips = (p.rows + AG_WARPS - 1) / AG_WARPS;
    const long long want = std::max<long long>(1, (long long)ctx->sm_count * 8 / g.gx);
    g.gy = (unsigned)std::min(std::min(strips, want), 65535LL);
    return g;
}

}  // namespace

size_t dlc_act_grad_workspace(const dlcContext *ctx, const ActGradProblem &p) {
    // either vector width's number of row strips
    const long long strips = (p.rows + AG_WARPS - 1) / AG_WARPS;
    const long long want = std::max<long long>(1, (long long)ctx->sm_count * 8 / std::max(1, (p.N + 255) / 256));
    return (size_t)std::min(std::min(strips, want), 65535LL) * (p.gated ? 2 : 1) * p.N * sizeof(float);
}

dlcStatus_t dlc_launch_act_grad(dlcContext *ctx, const ActGradProblem &pb) {
    const AgPlan g = ag_plan(ctx, pb);
    ActGradProblem p = pb;
    void *args[] = {&p};
    const void *kern = g.w == 8 ? (const void *)act_grad_kernel<8> : (const void *)act_grad_kernel<1>;
    const dlcStatus_t st = dlc_launch(ctx, kern, dim3(g.gx, g.gy), dim3(AG_WARPS * 32), 0, args);
    if (st != DLC_STATUS_SUCCESS || !p.dbias) return st;
    return dlc_launch_column_sum(ctx, p.ws, p.dbias, p.gated ? 2 * p.N : p.N, (int)g.gy);
}

// gemm.cu -- the products of the linear and gated layers.
#include "channel.cuh"
#include "ptx.cuh"

namespace {

using namespace dlc;

constexpr int DT = 64, DK = 16;  // tile of 64 x 64 outputs, 16 of the reduction at a time

__device__ __forceinline__ float operand(const GemmOperand &o, long long i, long long k) {
    return o.trans ? load_elem(o.t.p, o.t.dt, row_off(o.t.m, k) + i * o.t.m.cs)
                   : load_elem(o.t.p, o.t.dt, row_off(o.t.m, i) + k * o.t.m.cs);
}

// Any types, strides and sizes: FP32 products and sums on the CUDA cores, a
// thread holding 4 x 4 outputs (and as many up projections).
template <bool GATED>
__global__ void __launch_bounds__(256) gemm_direct_kernel(const __grid_constant__ GemmProblem g) {
    griddep_launch_dependents();
    __shared__ float sa[DK][DT + 1], sb[GATED ? 2 : 1][DK][DT + 1];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const long long m0 = (long long)blockIdx.x * DT;
    const int n0 = (int)blockIdx.y * DT;
    griddep_wait();
    float acc[GATED ? 2 : 1][4][4] = {};
    for (long long k0 = 0; k0 < g.K; k0 += DK) {
        for (int i = threadIdx.x; i < DT * DK; i += 256) {
            const int r = i / DK, k = i % DK;
            const bool kin = k0 + k < g.K;
            sa[k][r] = kin && m0 + r < g.M ? operand(g.a, m0 + r, k0 + k) : 0.f;
            sb[0][k][r] = kin && n0 + r < g.N ? operand(g.b, n0 + r, k0 + k) : 0.f;
            if (GATED) sb[1][k][r] = kin && n0 + r < g.N ? operand(g.b, (long long)g.N + n0 + r, k0 + k) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < DK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[0][i][j] = fmaf(sa[k][ty * 4 + i], sb[0][k][tx * 4 + j], acc[0][i][j]);
                    if (GATED) acc[GATED][i][j] = fmaf(sa[k][ty * 4 + i], sb[GATED][k][tx * 4 + j], acc[GATED][i][j]);
                }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
        const long long m = m0 + ty * 4 + i;
        if (m >= g.M) break;
        const float s = g.sa ? g.sa[m] : 1.f;
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx * 4 + j;
            if (n >= g.N) break;
            float v = acc[0][i][j] * s * (g.sb ? g.sb[n] : 1.f) + (g.bias ? g.bias[n] : 0.f);
            const long long zo = g.z.p ? row_off(g.z.m, m) : 0;
            if (g.z.p) store_elem(g.z.p, g.z.dt, zo + n * g.z.m.cs, v);
            float u = 1.f;
            if (GATED) {
                const int n2 = g.N + n;
                u = acc[GATED][i][j] * s * (g.sb ? g.sb[n2] : 1.f) + (g.bias ? g.bias[n2] : 0.f);
                if (g.z.p) store_elem(g.z.p, g.z.dt, zo + n2 * g.z.m.cs, u);
            }
            act_dispatch(g.act, [&](auto act) { v = act_f<decltype(act)::value>(v); });
            if (GATED) v *= u;
            if (g.r.p) v += load_elem(g.r.p, g.r.dt, row_off(g.r.m, m) + n * g.r.m.cs);
            store_elem(g.y.p, g.y.dt, row_off(g.y.m, m) + n * g.y.m.cs, v);
        }
    }
}

}  // namespace

dlcKernel_t dlc_gemm_variant(const dlcContext *, const GemmProblem &) { return DLC_KERNEL_DIRECT; }

size_t dlc_gemm_workspace(const dlcContext *, const GemmProblem &) { return 0; }

dlcStatus_t dlc_launch_gemm(dlcContext *ctx, const GemmProblem &pb) {
    GemmProblem g = pb;
    void *args[] = {&g};
    return dlc_launch(ctx, g.gated ? (const void *)gemm_direct_kernel<true> : (const void *)gemm_direct_kernel<false>,
                      dim3((unsigned)((g.M + DT - 1) / DT), (unsigned)((g.N + DT - 1) / DT)), dim3(256), 0, args);
}

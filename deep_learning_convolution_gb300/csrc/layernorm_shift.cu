// layernorm_shift.cu -- the layer norm's kernels (layernorm_vec.cuh) for rows that begin anywhere in a
// 16-byte piece.
#include "layernorm_vec.cuh"

namespace {

// What these kernels take: contiguous channels, tensors that begin on a piece, so that no piece lies in front of
// one, inputs and total of one type that begin each row alike; y any pitch.
bool alike(std::initializer_list<RowTensor> ts) {
    long long ld = -1;
    if (!ring(ts)) return false;
    const int ch = all_of(DLC_DATA_FLOAT, ts) ? 4 : 8;
    for (const RowTensor &t : ts) {
        if (!t.p) continue;
        if (t.m.cs != 1 || !t.m.uniform || (uintptr_t)t.p % 16 || (ld >= 0 && t.m.ld % ch != ld)) return false;
        ld = t.m.ld % ch;
    }
    return true;
}

// Whether a row in vectors, `gain` times as fast as the general kernel's single elements where either's threads all
// have channels, is the faster way: both have a power of two of threads a row, or whole warps, and a row of 257
// vectors or of 1025 elements leaves many of them idle.  Measured against the general kernel at 16384 x 1001
// (98 % of both in use): 26.7 and 48.3 us BF16 (y with rows of its own 28.3 and 48.5), FP32 y 33.5 and 47.8 (44.0
// and 47.4), FP32 throughout 49.3 and 45.0 (57.0 and 44.9); backward 35.2 and 52.5 BF16, 54.9 and 56.0 FP32.
// 60000 x 251 backward, 49 % and 98 % in use: 45.7 and 41.3 BF16.  16384 x 515, 67 % and 50 %: 26.4 and 43.8
// FP32.  Short rows are all latency: 60000 x 25 FP32 7.8 and 11.3.
bool pays(const VecPlan &v, const RowPlan &r, int ch, int C, double gain) {
    if (!r.w) return true;  // a row longer than a block's registers
    return gain / ((double)ch * v.tpr * v.v) >= 1.0 / ((double)r.tpr * r.v) || C <= 64;
}

// (fewer numbers of vectors than for whole pieces: what a row does not need is skipped)
VecKernel shift_fwd(VecPlan &v, const LayerProblem &p) {
    using Half = unsigned short;
    const bool fp32 = p.x.dt == DLC_DATA_FLOAT;
    v.v = v.v <= 4 ? v.v : v.v <= 6 ? 6 : 8;
    switch (v.v) {
        case 1: return fp32 ? vec_fwd<1, float, true>(p) : vec_fwd<1, Half, true>(p);
        case 2: return fp32 ? vec_fwd<2, float, true>(p) : vec_fwd<2, Half, true>(p);
        case 3: return fp32 ? vec_fwd<3, float, true>(p) : vec_fwd<3, Half, true>(p);
        case 4: return fp32 ? vec_fwd<4, float, true>(p) : vec_fwd<4, Half, true>(p);
        case 6: return fp32 ? vec_fwd<6, float, true>(p) : vec_fwd<6, Half, true>(p);
        default: return fp32 ? vec_fwd<8, float, true>(p) : vec_fwd<8, Half, true>(p);
    }
}

}  // namespace

bool dlc_layer_shift(dlcContext *ctx, const LayerProblem &pb, dlcStatus_t &status) {
    LayerProblem p = pb;
    const bool fp32 = p.x.dt == DLC_DATA_FLOAT;
    const int ch = fp32 ? 4 : 8, e = dlc_dtype_bytes((dlcDataType_t)p.y.dt);
    if (!alike({p.x, p.r, p.t}) || p.y.m.cs != 1 || !p.y.m.uniform || (uintptr_t)p.y.p % std::min(16, ch * e)) return false;
    VecPlan v = plan_vec(p.rows, p.C, fp32, 8, false, true, ctx->sm_count);
    if (!v.v) return false;
    const VecKernel k = shift_fwd(v, p);
    const int row = p.y.m.ld % ch == p.x.m.ld % ch ? 0 : ch * e;
    const double gain = fp32 ? (row ? 0.85 : 0.95) : e == 4 ? (row ? 1.1 : 1.5) : 2.;
    if (vec_smem(k, v, fp32, 2, row) > NORM_MAX_RING || !pays(v, plan_rows(p.rows, p.C, true, false, true, 1, ctx->sm_count), ch, p.C, gain))
        return false;
    status = launch_vec(ctx, k, p, v, fp32, true, 2, row);
    return true;
}

bool dlc_layer_bwd_shift(dlcContext *ctx, const LayerBwdProblem &pb, dlcStatus_t &status) {
    LayerBwdProblem p = pb;
    if (!alike({p.dy, p.t, p.dt, p.dx})) return false;
    const bool fp32 = p.t.dt == DLC_DATA_FLOAT;
    const VecPlan v = plan_vec(p.rows, p.C, fp32, fp32 ? 4 : 2, true, true, ctx->sm_count);
    if (!v.v || !pays(v, plan_rows(p.rows, p.C, true, false, true, 1, ctx->sm_count), fp32 ? 4 : 8, p.C, fp32 ? 0.97 : 1.55)) return false;
    // A block's start and its sums cost more than its rows gain: by vectors and by single elements 300 x 2001 BF16 10.2 and
    // 7.3 us, 190 x 1113 BF16 8.0 and 6.7, 198 x 1383 FP32 8.3 and 7.0; but 864 x 1447 BF16 10.3 and 9.9, 904 x 2781 FP32
    // 15.9 and 17.6, 2403 x 1957 BF16 14.7 and 19.7.  Over 40 sizes of 0.03 to 2 rows a channel, 200 to 4000 channels, the
    // border at a fourth is 1 % slower than the faster way on average and 7 % at most.
    if (4 * p.rows < p.C) return false;
    int blocks = 0;
    status = launch_vec(ctx, vec_bwd<true>(v, fp32, p.dt.p != nullptr), p, v, fp32, true, 1, 0, &blocks);
    if (status == DLC_STATUS_SUCCESS && (p.dgamma || p.dbeta))
        status = dlc_launch_column_sums(ctx, p.ws, p.dgamma, p.dbeta, p.C, blocks);
    return true;
}

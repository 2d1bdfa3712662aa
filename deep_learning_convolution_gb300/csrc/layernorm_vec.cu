// layernorm_vec.cu -- the layer norm's kernels for rows of whole 16-byte pieces (layernorm_vec.cuh).
#include "layernorm_vec.cuh"

namespace {

// What these kernels take: see the top.
bool whole(std::initializer_list<RowTensor> ins, std::initializer_list<RowTensor> outs) {
    auto ok = [](const RowTensor &t, int bytes) { return !t.p || (t.m.cs == 1 && t.m.uniform && dlc_aligned_rows(t, bytes)); };
    const int ch = all_of(DLC_DATA_FLOAT, ins) ? 4 : 8;
    if (!ring(ins)) return false;
    for (const RowTensor &t : ins)
        if (!ok(t, 16)) return false;
    for (const RowTensor &t : outs)
        if (!ok(t, std::min(16, ch * dlc_dtype_bytes((dlcDataType_t)t.dt)))) return false;
    return true;
}

VecKernel vec_fwd(int v, const LayerProblem &p) {
    if (p.x.dt == DLC_DATA_FLOAT) {
        switch (v) {
            case 1: return vec_fwd<1, float, false>(p);
            case 2: return vec_fwd<2, float, false>(p);
            case 3: return vec_fwd<3, float, false>(p);
            case 4: return vec_fwd<4, float, false>(p);
            case 5: return vec_fwd<5, float, false>(p);
            case 6: return vec_fwd<6, float, false>(p);
            case 7: return vec_fwd<7, float, false>(p);
            default: return vec_fwd<8, float, false>(p);
        }
    }
    using Half = unsigned short;
    switch (v) {
        case 1: return vec_fwd<1, Half, false>(p);
        case 2: return vec_fwd<2, Half, false>(p);
        case 3: return vec_fwd<3, Half, false>(p);
        case 4: return vec_fwd<4, Half, false>(p);
        case 5: return vec_fwd<5, Half, false>(p);
        case 6: return vec_fwd<6, Half, false>(p);
        case 7: return vec_fwd<7, Half, false>(p);
        default: return vec_fwd<8, Half, false>(p);
    }
}

}  // namespace

bool dlc_layer_vec(dlcContext *ctx, const LayerProblem &pb, dlcStatus_t &status) {
    LayerProblem p = pb;
    if (!whole({p.x, p.r}, {p.t, p.y}) || (p.t.p && p.t.dt != p.x.dt)) return false;
    const bool fp32 = p.x.dt == DLC_DATA_FLOAT;
    const VecPlan v = plan_vec(p.rows, p.C, fp32, 8, false, false, ctx->sm_count);
    if (!v.v) return false;
    status = launch_vec(ctx, vec_fwd(v.v, p), p, v, fp32, false, 2, 0);
    return true;
}

bool dlc_layer_bwd_vec(dlcContext *ctx, const LayerBwdProblem &pb, dlcStatus_t &status) {
    LayerBwdProblem p = pb;
    if (!whole({p.dy, p.t, p.dt}, {p.dx}) || p.dx.dt != p.t.dt) return false;
    const bool fp32 = p.t.dt == DLC_DATA_FLOAT, res = p.dt.p != nullptr;
    const VecPlan v = plan_vec(p.rows, p.C, fp32, fp32 ? 4 : 2, true, false, ctx->sm_count);
    if (!v.v) return false;
    int blocks = 0;
    // (the rows of sums that a block joins need no more than the ring has)
    status = launch_vec(ctx, vec_bwd<false>(v, fp32, res), p, v, fp32, false, 1, 0, &blocks);
    if (status == DLC_STATUS_SUCCESS && (p.dgamma || p.dbeta))
        status = dlc_launch_column_sums(ctx, p.ws, p.dgamma, p.dbeta, p.C, blocks);
    return true;
}

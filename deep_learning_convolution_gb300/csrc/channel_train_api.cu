// channel_train_api.cu -- the C ABI of the channel operators at a network's ends and
// between its layers: layer norm, dropout, embedding, softmax cross entropy, and their
// backward passes.  Validation and workspace layout; the kernels are in
// layernorm.cu, dropout.cu, embedding.cu and cross_entropy.cu.
#include <cmath>

#include "channel_args.h"

namespace {

using namespace dlc;

// Optional pointer with its descriptor: NOT_INITIALIZED where only the pointer is there.
bool absent_or_ready(dlcTensorDescriptor_t d, const void *p) { return !p || ready(d); }

bool like(const dlcTensorStruct *d, const dlcTensorStruct *x, const void *p) { return !p || (same_rows(d, x) && d->c == x->c); }

// Channels, and rows of a table, up to which 32-bit indices with a tile's or a block's step above them hold.
constexpr int MOST_INDEX = 0x7fff0000;

dlcStatus_t index_list(dlcIndexType_t type, const void *p, long long rows, IndexList &t, Span &s) {
    if (type != DLC_INDEX_INT32 && type != DLC_INDEX_INT64) return DLC_STATUS_BAD_PARAM;
    const int e = type == DLC_INDEX_INT64 ? 8 : 4;
    if (!p || (uintptr_t)p % e) return DLC_STATUS_BAD_PARAM;
    t.p = p;
    t.wide = e == 8;
    s = span_bytes(p, (uint64_t)rows * e);
    return DLC_STATUS_SUCCESS;
}

Span vector_span(const float *p, long long n) { return p ? span_bytes(p, (uint64_t)n * 4) : Span{0, 0}; }

// ---- layer norm ------------------------------------------------------------------

dlcStatus_t layer_forward(dlcHandle_t h, double epsilon, dlcTensorDescriptor_t xd, const void *x, dlcTensorDescriptor_t rd,
                          const void *residual, const float *gamma, const float *beta, dlcTensorDescriptor_t td, void *total,
                          dlcTensorDescriptor_t yd, void *y, float *scale) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    if (!xd || !yd || !gamma || !fp32_ok(gamma) || !fp32_ok(beta) || !(epsilon >= 0.0)) return DLC_STATUS_BAD_PARAM;
    if (!xd->set || !yd->set || !absent_or_ready(rd, residual) || !absent_or_ready(td, total)) return DLC_STATUS_NOT_INITIALIZED;
    if (!like(yd, xd, yd) || !like(rd, xd, residual) || !like(td, xd, total)) return DLC_STATUS_BAD_PARAM;
    if (!is_float(xd->dtype) || (residual && !is_float(rd->dtype)) || (total && !is_float(td->dtype)) ||
        !(is_float(yd->dtype) || yd->dtype == DLC_DATA_FLOAT8_E4M3) || xd->c > MOST_INDEX)
        return DLC_STATUS_NOT_SUPPORTED;
    if ((yd->dtype == DLC_DATA_FLOAT8_E4M3) != (scale != nullptr) || !fp32_ok(scale)) return DLC_STATUS_BAD_PARAM;
    LayerProblem p;
    p.rows = rows_of(xd);
    p.C = xd->c;
    p.eps = (float)epsilon;
    Span s_x, s_y, s_r{0, 0}, s_t{0, 0};
    if (!span_of(xd, x, false, s_x) || !span_of(yd, y, true, s_y) || (residual && !span_of(rd, residual, false, s_r)) ||
        (total && !span_of(td, total, true, s_t)))
        return DLC_STATUS_BAD_PARAM;
    const Span s_g = vector_span(gamma, p.C), s_b = vector_span(beta, p.C), s_s = vector_span(scale, p.rows);
    if (overlaps(s_y, {s_x, s_r, s_t, s_g, s_b, s_s}) || (scale && overlaps(s_s, {s_x, s_r, s_t, s_g, s_b})))
        return DLC_STATUS_BAD_PARAM;
    if (total && (overlaps(s_t, {s_g, s_b}) || (overlaps(s_t, {s_x}) && !same_tensor(td, total, xd, x)) ||
                  (residual && overlaps(s_t, {s_r}) && !same_tensor(td, total, rd, residual))))
        return DLC_STATUS_BAD_PARAM;
    p.x = row_tensor(xd, x);
    if (residual) p.r = row_tensor(rd, residual);
    if (total) p.t = row_tensor(td, total);
    p.y = row_tensor(yd, y);
    if (!p.x.m.hw || !p.r.m.hw || !p.t.m.hw || !p.y.m.hw) return DLC_STATUS_NOT_SUPPORTED;
    p.gamma = gamma;
    p.beta = beta;
    p.scale = scale;
    RETURN_IF(enter(h));
    return dlc_launch_layer(h, p);
}

dlcStatus_t layer_backward(dlcHandle_t h, double epsilon, dlcTensorDescriptor_t dyd, const void *dy, dlcTensorDescriptor_t td,
                           const void *total, const float *gamma, dlcTensorDescriptor_t dtd, const void *dtotal,
                           dlcTensorDescriptor_t dxd, void *dx, float *dgamma, float *dbeta, void *ws, size_t ws_bytes) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    if (!dyd || !td || !dxd || !gamma || !fp32_ok(gamma) || !fp32_ok(dgamma) || !fp32_ok(dbeta) || !(epsilon >= 0.0))
        return DLC_STATUS_BAD_PARAM;
    if (!dyd->set || !td->set || !dxd->set || !absent_or_ready(dtd, dtotal)) return DLC_STATUS_NOT_INITIALIZED;
    if (!like(dyd, td, dyd) || !like(dxd, td, dxd) || !like(dtd, td, dtotal)) return DLC_STATUS_BAD_PARAM;
    if (!is_float(dyd->dtype) || !is_float(td->dtype) || !is_float(dxd->dtype) || (dtotal && !is_float(dtd->dtype)) ||
        td->c > MOST_INDEX)
        return DLC_STATUS_NOT_SUPPORTED;
    LayerBwdProblem p;
    p.rows = rows_of(td);
    p.C = td->c;
    p.eps = (float)epsilon;
    Span s_dy, s_t, s_dx, s_dt{0, 0};
    if (!span_of(dyd, dy, false, s_dy) || !span_of(td, total, false, s_t) || !span_of(dxd, dx, true, s_dx) ||
        (dtotal && !span_of(dtd, dtotal, false, s_dt)))
        return DLC_STATUS_BAD_PARAM;
    const Span s_g = vector_span(gamma, p.C), s_dg = vector_span(dgamma, p.C), s_db = vector_span(dbeta, p.C);
    // dx may take dtotal's place (read by the thread that writes it)
    if (overlaps(s_dx, {s_dy, s_t, s_g, s_dg, s_db}) ||
        (dtotal && overlaps(s_dx, {s_dt}) && !same_tensor(dxd, dx, dtd, dtotal)) ||
        (dgamma && overlaps(s_dg, {s_dy, s_t, s_g, s_dt, s_db})) || (dbeta && overlaps(s_db, {s_dy, s_t, s_g, s_dt})))
        return DLC_STATUS_BAD_PARAM;
    p.dy = row_tensor(dyd, dy);
    p.t = row_tensor(td, total);
    if (dtotal) p.dt = row_tensor(dtd, dtotal);
    p.dx = row_tensor(dxd, dx);
    if (!p.dy.m.hw || !p.t.m.hw || !p.dt.m.hw || !p.dx.m.hw) return DLC_STATUS_NOT_SUPPORTED;
    p.gamma = gamma;
    p.dgamma = dgamma;
    p.dbeta = dbeta;
    const size_t need = dgamma || dbeta ? ws_round(dlc_layer_bwd_workspace(h, p.rows, p.C)) : 0;
    RETURN_IF(check_workspace(ws, ws_bytes, need));
    if (need && overlaps(span_bytes(ws, need), {s_dy, s_t, s_dx, s_dt, s_g, s_dg, s_db})) return DLC_STATUS_BAD_PARAM;
    p.ws = static_cast<float *>(ws);
    RETURN_IF(enter(h));
    return dlc_launch_layer_bwd(h, p);
}

// ---- dropout ---------------------------------------------------------------------

dlcStatus_t dropout(dlcHandle_t h, double probability, const uint64_t *random, dlcTensorDescriptor_t xd, const void *x,
                    dlcTensorDescriptor_t rd, const void *residual, dlcTensorDescriptor_t yd, void *y) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    if (!xd || !yd || !random || (uintptr_t)random % 8 || !(probability >= 0.0 && probability < 1.0)) return DLC_STATUS_BAD_PARAM;
    if (!xd->set || !yd->set || !absent_or_ready(rd, residual)) return DLC_STATUS_NOT_INITIALIZED;
    if (!like(yd, xd, yd) || !like(rd, xd, residual)) return DLC_STATUS_BAD_PARAM;
    if (!is_float(xd->dtype) || !is_float(yd->dtype) || (residual && !is_float(rd->dtype)) || rows_of(xd) > 0x7fffffffLL ||
        xd->c > MOST_INDEX)
        return DLC_STATUS_NOT_SUPPORTED;
    Span s_x, s_y, s_r{0, 0};
    const Span s_s = span_bytes(random, 16);
    if (!span_of(xd, x, false, s_x) || !span_of(yd, y, true, s_y) || (residual && !span_of(rd, residual, false, s_r)))
        return DLC_STATUS_BAD_PARAM;
    if (overlaps(s_y, {s_s}) || (overlaps(s_y, {s_x}) && !same_tensor(yd, y, xd, x)) ||
        (residual && overlaps(s_y, {s_r}) && !same_tensor(yd, y, rd, residual)))
        return DLC_STATUS_BAD_PARAM;
    DropoutProblem p;
    p.rows = rows_of(xd);
    p.C = xd->c;
    const double border = std::floor(probability * 4294967296.0);  // exact: below 2^32
    p.border = (uint32_t)border;
    p.scale = (float)(4294967296.0 / (4294967296.0 - border));
    p.random = reinterpret_cast<const unsigned long long *>(random);
    p.x = row_tensor(xd, x);
    if (residual) p.r = row_tensor(rd, residual);
    p.y = row_tensor(yd, y);
    RETURN_IF(enter(h));
    return dlc_launch_dropout(h, p);
}

// ---- embedding -------------------------------------------------------------------

// A table (R = S = 1, dense) with rows of yd's channels.
dlcStatus_t table_checks(dlcFilterDescriptor_t wd, dlcTensorDescriptor_t yd) {
    if (!wd || !yd) return DLC_STATUS_BAD_PARAM;
    if (!wd->set || !yd->set) return DLC_STATUS_NOT_INITIALIZED;
    if (wd->r != 1 || wd->s != 1 || wd->c != yd->c) return DLC_STATUS_BAD_PARAM;
    if (!is_float(wd->dtype) || !is_float(yd->dtype) || rows_of(yd) > 0x7fffffffLL || wd->c > MOST_INDEX || wd->k > MOST_INDEX)
        return DLC_STATUS_NOT_SUPPORTED;
    return DLC_STATUS_SUCCESS;
}

dlcStatus_t embedding(dlcHandle_t h, bool backward, double scale, int accumulate, dlcIndexType_t type, const void *tokens,
                      dlcFilterDescriptor_t wd, const void *table, dlcTensorDescriptor_t yd, const void *y, void *ws, size_t ws_bytes) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    RETURN_IF(table_checks(wd, yd));
    EmbeddingProblem p;
    Span s_y, s_i;
    RETURN_IF(index_list(type, tokens, rows_of(yd), p.tokens, s_i));
    const int e = dlc_dtype_bytes(wd->dtype);
    if (!table || (uintptr_t)table % e || !span_of(yd, y, !backward, s_y) || !std::isfinite((float)scale)) return DLC_STATUS_BAD_PARAM;
    const Span s_w = span_bytes(table, (uint64_t)wd->k * wd->c * e);
    if (overlaps(s_w, {s_y}) || overlaps(backward ? s_w : s_y, {s_i})) return DLC_STATUS_BAD_PARAM;
    p.rows = rows_of(yd);
    p.C = yd->c;
    p.V = wd->k;
    p.scale = (float)scale;
    p.accumulate = accumulate != 0;
    p.table = filter_rows(wd, table);
    p.y = row_tensor(yd, y);
    p.ws = static_cast<char *>(ws);
    if (!backward) {
        RETURN_IF(enter(h));
        return dlc_launch_embedding(h, p);
    }
    const size_t need = ws_round(dlc_embedding_bwd_workspace(h, p.rows, p.C, p.V));
    RETURN_IF(check_workspace(ws, ws_bytes, need));
    if (overlaps(span_bytes(ws, need), {s_w, s_y, s_i})) return DLC_STATUS_BAD_PARAM;
    RETURN_IF(enter(h));
    return dlc_launch_embedding_bwd(h, p);
}

// ---- cross entropy ---------------------------------------------------------------

dlcStatus_t resolve_entropy(dlcTensorDescriptor_t xd, const void *x, dlcFilterDescriptor_t wd, const void *w, bool backward,
                            CrossEntropyProblem &p) {
    if (!xd || !wd) return DLC_STATUS_BAD_PARAM;
    if (!xd->set || !wd->set) return DLC_STATUS_NOT_INITIALIZED;
    if (wd->r != 1 || wd->s != 1 || wd->c != xd->c || wd->dtype != xd->dtype) return DLC_STATUS_BAD_PARAM;
    if (!(xd->dtype == DLC_DATA_BFLOAT16 || (!backward && xd->dtype == DLC_DATA_FLOAT8_E4M3)) || rows_of(xd) > 0x7fffffffLL ||
        wd->c > MOST_INDEX || wd->k > MOST_INDEX)
        return DLC_STATUS_NOT_SUPPORTED;
    p.M = rows_of(xd);
    p.V = wd->k;
    p.K = xd->c;
    p.x = row_tensor(xd, x);
    p.w = filter_rows(wd, w);
    return DLC_STATUS_SUCCESS;
}

dlcStatus_t entropy_forward(dlcHandle_t h, dlcTensorDescriptor_t xd, const void *x, const float *sx, dlcFilterDescriptor_t wd,
                            const void *w, const float *sw, const float *bias, dlcIndexType_t type, const void *target, float *loss,
                            float *lse, void *ws, size_t ws_bytes) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    CrossEntropyProblem p;
    RETURN_IF(resolve_entropy(xd, x, wd, w, false, p));
    const bool e4m3 = xd->dtype == DLC_DATA_FLOAT8_E4M3;
    if (e4m3 != (sx != nullptr) || e4m3 != (sw != nullptr)) return DLC_STATUS_BAD_PARAM;
    if (!loss || !lse || !fp32_ok(loss) || !fp32_ok(lse) || !fp32_ok(sx) || !fp32_ok(sw) || !fp32_ok(bias)) return DLC_STATUS_BAD_PARAM;
    const int e = dlc_dtype_bytes(wd->dtype);
    Span s_x, s_i;
    if (!w || (uintptr_t)w % e || !span_of(xd, x, false, s_x)) return DLC_STATUS_BAD_PARAM;
    RETURN_IF(index_list(type, target, p.M, p.target, s_i));
    const Span s_w = span_bytes(w, (uint64_t)wd->k * wd->c * e), s_b = vector_span(bias, p.V), s_sx = vector_span(sx, p.M),
               s_sw = vector_span(sw, p.V), s_l = vector_span(loss, p.M), s_e = vector_span(lse, p.M);
    if (overlaps(s_l, {s_x, s_w, s_b, s_sx, s_sw, s_i, s_e}) || overlaps(s_e, {s_x, s_w, s_b, s_sx, s_sw, s_i}))
        return DLC_STATUS_BAD_PARAM;
    p.sa = sx;
    p.sb = sw;
    p.bias = bias;
    p.loss = loss;
    p.lse = lse;
    const size_t need = dlc_cross_entropy_workspace(h, p);
    RETURN_IF(check_workspace(ws, ws_bytes, need));
    if (overlaps(span_bytes(ws, need), {s_x, s_w, s_b, s_sx, s_sw, s_i, s_l, s_e})) return DLC_STATUS_BAD_PARAM;
    p.ws = static_cast<char *>(ws);
    RETURN_IF(enter(h));
    return dlc_launch_cross_entropy(h, p);
}

dlcStatus_t entropy_backward(dlcHandle_t h, dlcTensorDescriptor_t xd, const void *x, dlcFilterDescriptor_t wd, const void *w,
                             const float *bias, dlcIndexType_t type, const void *target, const float *lse, const float *dloss,
                             dlcTensorDescriptor_t dxd, void *dx, dlcFilterDescriptor_t dwd, void *dw, float *dbias, void *ws,
                             size_t ws_bytes) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    CrossEntropyProblem p;
    RETURN_IF(resolve_entropy(xd, x, wd, w, true, p));
    if (!dx && !dw && !dbias) return DLC_STATUS_BAD_PARAM;
    if (!lse || !dloss || !fp32_ok(lse) || !fp32_ok(dloss) || !fp32_ok(bias) || !fp32_ok(dbias)) return DLC_STATUS_BAD_PARAM;
    Span s_x, s_i, s_dx{0, 0}, s_dw{0, 0};
    if (!w || (uintptr_t)w % 2 || !span_of(xd, x, false, s_x)) return DLC_STATUS_BAD_PARAM;
    RETURN_IF(index_list(type, target, p.M, p.target, s_i));
    if (dx) {
        if (!ready(dxd)) return DLC_STATUS_NOT_INITIALIZED;
        if (!same_rows(dxd, xd) || dxd->c != xd->c || !span_of(dxd, dx, true, s_dx)) return DLC_STATUS_BAD_PARAM;
        if (!is_float(dxd->dtype)) return DLC_STATUS_NOT_SUPPORTED;
        p.dx = row_tensor(dxd, dx);
    }
    if (dw) {
        if (!dwd || !dwd->set) return DLC_STATUS_NOT_INITIALIZED;
        if (dwd->k != wd->k || dwd->c != wd->c || dwd->r != 1 || dwd->s != 1) return DLC_STATUS_BAD_PARAM;
        if (!is_float(dwd->dtype)) return DLC_STATUS_NOT_SUPPORTED;
        const int e = dlc_dtype_bytes(dwd->dtype);
        if ((uintptr_t)dw % e) return DLC_STATUS_BAD_PARAM;
        s_dw = span_bytes(dw, (uint64_t)dwd->k * dwd->c * e);
        p.dw = filter_rows(dwd, dw);
    }
    const Span s_w = span_bytes(w, (uint64_t)wd->k * wd->c * 2), s_b = vector_span(bias, p.V), s_l = vector_span(lse, p.M),
               s_d = vector_span(dloss, p.M), s_db = vector_span(dbias, p.V);
    if ((dx && overlaps(s_dx, {s_x, s_w, s_b, s_i, s_l, s_d, s_dw, s_db})) ||
        (dw && overlaps(s_dw, {s_x, s_w, s_b, s_i, s_l, s_d, s_db})) || (dbias && overlaps(s_db, {s_x, s_w, s_b, s_i, s_l, s_d})))
        return DLC_STATUS_BAD_PARAM;
    p.bias = bias;
    p.lse = const_cast<float *>(lse);
    p.dloss = dloss;
    p.dbias = dbias;
    const size_t need = dlc_cross_entropy_bwd_workspace(h, p);
    RETURN_IF(check_workspace(ws, ws_bytes, need));
    if (overlaps(span_bytes(ws, need), {s_x, s_w, s_b, s_i, s_l, s_d, s_dx, s_dw, s_db})) return DLC_STATUS_BAD_PARAM;
    p.ws = static_cast<char *>(ws);
    RETURN_IF(enter(h));
    return dlc_launch_cross_entropy_bwd(h, p);
}

}  // namespace

extern "C" {

dlcStatus_t dlcLayerNormForward(dlcHandle_t h, double epsilon, dlcTensorDescriptor_t xd, const void *x, dlcTensorDescriptor_t rd,
                                const void *residual, const float *gamma, const float *beta, dlcTensorDescriptor_t td, void *total,
                                dlcTensorDescriptor_t yd, void *y, float *scale) {
    return layer_forward(h, epsilon, xd, x, rd, residual, gamma, beta, td, total, yd, y, scale);
}

dlcStatus_t dlcGetLayerNormBackwardWorkspaceSize(dlcHandle_t h, dlcTensorDescriptor_t td, size_t *bytes) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    if (!td || !bytes) return DLC_STATUS_BAD_PARAM;
    if (!td->set) return DLC_STATUS_NOT_INITIALIZED;
    *bytes = ws_round(dlc_layer_bwd_workspace(h, rows_of(td), td->c));
    return DLC_STATUS_SUCCESS;
}

dlcStatus_t dlcLayerNormBackward(dlcHandle_t h, double epsilon, dlcTensorDescriptor_t dyd, const void *dy, dlcTensorDescriptor_t td,
                                 const void *total, const float *gamma, dlcTensorDescriptor_t dtd, const void *dtotal,
                                 dlcTensorDescriptor_t dxd, void *dx, float *dgamma, float *dbeta, void *ws, size_t ws_bytes) {
    return layer_backward(h, epsilon, dyd, dy, td, total, gamma, dtd, dtotal, dxd, dx, dgamma, dbeta, ws, ws_bytes);
}

dlcStatus_t dlcDropoutForward(dlcHandle_t h, double probability, const uint64_t *random, dlcTensorDescriptor_t xd, const void *x,
                              dlcTensorDescriptor_t rd, const void *residual, dlcTensorDescriptor_t yd, void *y) {
    return dropout(h, probability, random, xd, x, rd, residual, yd, y);
}

dlcStatus_t dlcDropoutBackward(dlcHandle_t h, double probability, const uint64_t *random, dlcTensorDescriptor_t dyd, const void *dy,
                               dlcTensorDescriptor_t dxd, void *dx) {
    return dropout(h, probability, random, dyd, dy, nullptr, nullptr, dxd, dx);
}

dlcStatus_t dlcEmbeddingForward(dlcHandle_t h, double scale, dlcIndexType_t type, const void *tokens, dlcFilterDescriptor_t wd,
                                const void *table, dlcTensorDescriptor_t yd, void *y) {
    return embedding(h, false, scale, 0, type, tokens, wd, table, yd, y, nullptr, 0);
}

dlcStatus_t dlcGetEmbeddingBackwardWorkspaceSize(dlcHandle_t h, dlcTensorDescriptor_t dyd, dlcFilterDescriptor_t dwd, size_t *bytes) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    if (!bytes) return DLC_STATUS_BAD_PARAM;
    RETURN_IF(table_checks(dwd, dyd));
    *bytes = ws_round(dlc_embedding_bwd_workspace(h, rows_of(dyd), dyd->c, dwd->k));
    return DLC_STATUS_SUCCESS;
}

dlcStatus_t dlcEmbeddingBackward(dlcHandle_t h, double scale, dlcIndexType_t type, const void *tokens, dlcTensorDescriptor_t dyd,
                                 const void *dy, int accumulate, dlcFilterDescriptor_t dwd, void *dtable, void *ws, size_t ws_bytes) {
    return embedding(h, true, scale, accumulate, type, tokens, dwd, dtable, dyd, dy, ws, ws_bytes);
}

dlcStatus_t dlcCrossEntropyForward(dlcHandle_t h, dlcTensorDescriptor_t xd, const void *x, const float *xScale, dlcFilterDescriptor_t wd,
                                   const void *w, const float *wScale, const float *bias, dlcIndexType_t type, const void *target,
                                   float *loss, float *lse, void *ws, size_t ws_bytes) {
    return entropy_forward(h, xd, x, xScale, wd, w, wScale, bias, type, target, loss, lse, ws, ws_bytes);
}

dlcStatus_t dlcGetCrossEntropyForwardWorkspaceSize(dlcHandle_t h, dlcTensorDescriptor_t xd, const void *x, dlcFilterDescriptor_t wd,
                                                   const void *w, size_t *bytes) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    if (!bytes) return DLC_STATUS_BAD_PARAM;
    CrossEntropyProblem p;
    void *any = (void *)(uintptr_t)WS_ALIGN;
    RETURN_IF(resolve_entropy(xd, x ? x : any, wd, w ? w : any, false, p));
    *bytes = dlc_cross_entropy_workspace(h, p);
    return DLC_STATUS_SUCCESS;
}

dlcStatus_t dlcCrossEntropyBackward(dlcHandle_t h, dlcTensorDescriptor_t xd, const void *x, dlcFilterDescriptor_t wd, const void *w,
                                    const float *bias, dlcIndexType_t type, const void *target, const float *lse, const float *dloss,
                                    dlcTensorDescriptor_t dxd, void *dx, dlcFilterDescriptor_t dwd, void *dw, float *dbias, void *ws,
                                    size_t ws_bytes) {
    return entropy_backward(h, xd, x, wd, w, bias, type, target, lse, dloss, dxd, dx, dwd, dw, dbias, ws, ws_bytes);
}

// Sized for dx (BF16: its FP32 sum is kept), dw and dbias all wanted, so one workspace serves any subset.
dlcStatus_t dlcGetCrossEntropyBackwardWorkspaceSize(dlcHandle_t h, dlcTensorDescriptor_t xd, const void *x, dlcFilterDescriptor_t wd,
                                                    const void *w, size_t *bytes) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    if (!bytes) return DLC_STATUS_BAD_PARAM;
    CrossEntropyProblem p;
    void *any = (void *)(uintptr_t)WS_ALIGN;
    RETURN_IF(resolve_entropy(xd, x ? x : any, wd, w ? w : any, true, p));
    p.dx = row_tensor(xd, any);
    p.dw = filter_rows(wd, any);
    p.dbias = static_cast<float *>(any);
    *bytes = dlc_cross_entropy_bwd_workspace(h, p);
    return DLC_STATUS_SUCCESS;
}

}  // extern "C"

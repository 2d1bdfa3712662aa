// channel_api.cu -- the C ABI of the channel operators: RMS norm with the
// residual's addition, the linear layer with its epilogue, the gated
// projections, and their backward passes.  Validation, the split of a backward
// pass into its products, and workspace layout; the kernels are in rmsnorm.cu,
// act_grad.cu, gemm.cu, gemm_rows.cu and gemv.cu.
#include <atomic>
#include <climits>
#include <cstring>
#include <initializer_list>

#include "internal.h"

dlcStatus_t dlc_launch(dlcContext *ctx, const void *kernel, dim3 grid, dim3 block, size_t smem, void **args,
                       int cluster) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = dlc_pdl_enabled() ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = ctx->stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelExC(&cfg, kernel, args) != cudaSuccess) {
        cudaGetLastError();  // reported here; the next runtime call of the program is not the one to fail
        return DLC_STATUS_EXECUTION_FAILED;
    }
    ctx->launches += 1;
    return DLC_STATUS_SUCCESS;
}

bool dlc_allow_smem(const dlcContext *ctx, const void *kernel, size_t bytes) {
    // what each kernel has been allowed so far (it is a property of the kernel
    // and the device, not of a call); beyond the table's room it is set every time
    struct Entry {
        const void *kernel;
        int device;
        size_t bytes;
    };
    static Entry table[128];
    static int used = 0;
    static std::atomic_flag busy = ATOMIC_FLAG_INIT;
    if (bytes <= 47 * 1024) return true;  // (48 KiB with the static part need no leave)
    while (busy.test_and_set(std::memory_order_acquire)) {
    }
    Entry *e = nullptr;
    for (int i = 0; i < used && !e; ++i)
        if (table[i].kernel == kernel && table[i].device == ctx->device) e = &table[i];
    bool ok = e && e->bytes >= bytes;
    if (!ok) {
        ok = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
        if (!ok) {
            cudaGetLastError();
        } else if (e) {
            e->bytes = bytes;
        } else if (used < 128) {
            table[used++] = Entry{kernel, ctx->device, bytes};
        }
    }
    busy.clear(std::memory_order_release);
    return ok;
}

int dlc_resident_clusters(const dlcContext *ctx, int *known, const void *kernel, int size, int threads, size_t smem) {
    if (*known > 0) return *known;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(ctx->sm_count / size * size));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (!dlc_allow_smem(ctx, kernel, smem) || cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = std::max(1, ctx->sm_count / size);  // kept as well: the plans of a handle agree
    }
    return *known = n;
}

namespace {

constexpr size_t WS_ALIGN = 256;
size_t ws_round(size_t b) { return (b + WS_ALIGN - 1) / WS_ALIGN * WS_ALIGN; }

long long rows_of(const dlcTensorStruct *d) { return (long long)d->n * d->h * d->w; }

bool same_rows(const dlcTensorStruct *a, const dlcTensorStruct *b) {
    return a->n == b->n && a->h == b->h && a->w == b->w;
}

bool is_float(dlcDataType_t t) { return t == DLC_DATA_FLOAT || t == DLC_DATA_BFLOAT16; }

RowTensor row_tensor(const dlcTensorStruct *d, const void *p) {
    RowTensor t;
    t.p = const_cast<void *>(p);
    t.dt = d->dtype;
    RowMap &m = t.m;
    m.s0 = d->stride[0];
    m.cs = d->c > 1 ? d->stride[1] : 1;
    m.s2 = d->stride[2];
    m.s3 = d->stride[3];
    const long long hw = (long long)d->h * d->w;
    m.hw = (int)std::min(hw, (long long)INT_MAX);
    m.w = d->w;
    // one pitch for all rows, from the innermost axis longer than one
    const long long ext[3] = {d->w, d->h, d->n}, str[3] = {m.s3, m.s2, m.s0};
    long long span = 1;
    m.uniform = 1;
    m.ld = 0;
    for (int i = 0; i < 3; ++i) {
        if (ext[i] == 1) continue;
        if (span == 1)
            m.ld = str[i];
        else if (str[i] != span * m.ld)
            m.uniform = 0;
        span *= ext[i];
    }
    // Images of 2^31 pixels and more (a norm takes them) without one pitch: a group of w
    // rows for each (n, h), if those are evenly spaced; hw = 0 where they are not.
    if (!m.uniform && hw > INT_MAX) {
        m.hw = d->n == 1 || m.s0 == d->h * m.s2 ? d->w : 0;
        m.s0 = m.s2;
        m.s2 = 0;
    }
    if (span == 1) m.ld = ((long long)d->c + 15) / 16 * 16;  // a single row: any pitch
    return t;
}

// A filter bank (R = S = 1) as K rows of C channels.
RowTensor filter_rows(const dlcFilterStruct *f, const void *p) {
    RowTensor t;
    t.p = const_cast<void *>(p);
    t.dt = f->dtype;
    t.m = RowMap{f->c, 0, 0, 1, f->k > 1 ? f->c : (f->c + 15) / 16 * 16, 1, 1, 1};
    return t;
}

struct Span {
    uintptr_t lo, hi;
};

// The bytes a tensor reaches; false where its strides or pointer are unusable.
bool span_of(const dlcTensorStruct *d, const void *p, bool output, Span &s) {
    const int64_t ext[4] = {d->n, d->c, d->h, d->w};
    const int e = dlc_dtype_bytes(d->dtype);
    const int64_t last = dlc_max_offset(ext, d->stride, 4);
    if (!p || (uintptr_t)p % e || last < 0 || last >= ((int64_t)1 << 60)) return false;
    if (output && !dlc_strides_injective(ext, d->stride, 4)) return false;
    s = Span{(uintptr_t)p, (uintptr_t)p + (uintptr_t)(last + 1) * e};
    return true;
}

Span span_bytes(const void *p, uint64_t bytes) { return Span{(uintptr_t)p, (uintptr_t)p + bytes}; }

bool overlaps(const Span &a, std::initializer_list<Span> others) {
    for (const Span &o : others)
        if (dlc_ranges_overlap(a.lo, a.hi, o.lo, o.hi)) return true;
    return false;
}

// The same buffer under the same descriptor values: an elementwise in-place use.
bool same_tensor(const dlcTensorStruct *a, const void *pa, const dlcTensorStruct *b, const void *pb) {
    return pa == pb && a->dtype == b->dtype && std::memcmp(a->stride, b->stride, sizeof(a->stride)) == 0;
}

bool fp32_ok(const float *p) { return (uintptr_t)p % 4 == 0; }

bool ready(dlcTensorDescriptor_t d) { return d && d->set; }

dlcStatus_t enter(dlcContext *h) {
    const volatile int *e = h->h_err;
    if (e && e[0] != 0) return DLC_STATUS_EXECUTION_FAILED;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev != h->device) return DLC_STATUS_BAD_PARAM;
    return DLC_STATUS_SUCCESS;
}

dlcStatus_t check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return DLC_STATUS_SUCCESS;
    return ws && have >= need && (uintptr_t)ws % WS_ALIGN == 0 ? DLC_STATUS_SUCCESS : DLC_STATUS_BAD_PARAM;
}

dlcStatus_t check_act(dlcActivationMode_t act) {
    if (act < DLC_ACTIVATION_IDENTITY || act > DLC_ACTIVATION_GELU) return DLC_STATUS_BAD_PARAM;
    return act == DLC_ACTIVATION_CLIPPED_RELU ? DLC_STATUS_NOT_SUPPORTED : DLC_STATUS_SUCCESS;
}

#define RETURN_IF(expr)                                  \
    do {                                                 \
        const dlcStatus_t st_ = (expr);                  \
        if (st_ != DLC_STATUS_SUCCESS) return st_;       \
    } while (0)

// Descriptors of a forward product; y (and z) as the caller gave them.
dlcStatus_t resolve_product(bool gated, dlcTensorDescriptor_t xd, const void *x, dlcFilterDescriptor_t wd,
                            const void *w, dlcTensorDescriptor_t yd, const void *y, GemmProblem &g) {
    if (!xd || !wd || !yd) return DLC_STATUS_BAD_PARAM;
    if (!xd->set || !wd->set || !yd->set) return DLC_STATUS_NOT_INITIALIZED;
    if (wd->r != 1 || wd->s != 1 || wd->c != xd->c || !same_rows(xd, yd)) return DLC_STATUS_BAD_PARAM;
    if (gated && wd->k % 2) return DLC_STATUS_BAD_PARAM;
    const int n = gated ? wd->k / 2 : wd->k;
    if (yd->c != n || wd->dtype != xd->dtype) return DLC_STATUS_BAD_PARAM;
    if ((xd->dtype != DLC_DATA_BFLOAT16 && xd->dtype != DLC_DATA_FLOAT8_E4M3) || !is_float(yd->dtype))
        return DLC_STATUS_NOT_SUPPORTED;
    g.M = rows_of(xd);
    if (g.M > 0x7fffffffLL) return DLC_STATUS_NOT_SUPPORTED;
    g.N = n;
    g.K = xd->c;
    g.gated = gated;
    g.a.t = row_tensor(xd, x);
    g.b.t = filter_rows(wd, w);
    g.y = row_tensor(yd, y);
    return DLC_STATUS_SUCCESS;
}

dlcStatus_t product_forward(dlcHandle_t h, bool gated, dlcTensorDescriptor_t xd, const void *x, const float *sx,
                            dlcFilterDescriptor_t wd, const void *w, const float *sw, const float *bias,
                            dlcActivationMode_t act, dlcTensorDescriptor_t zd, void *z, dlcTensorDescriptor_t rd,
                            const void *r, dlcTensorDescriptor_t yd, void *y, void *ws, size_t ws_bytes) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    GemmProblem g;
    RETURN_IF(resolve_product(gated, xd, x, wd, w, yd, y, g));
    RETURN_IF(check_act(act));
    const bool e4m3 = xd->dtype == DLC_DATA_FLOAT8_E4M3;
    if (e4m3 != (sx != nullptr) || e4m3 != (sw != nullptr)) return DLC_STATUS_BAD_PARAM;
    if (!fp32_ok(sx) || !fp32_ok(sw) || !fp32_ok(bias)) return DLC_STATUS_BAD_PARAM;
    const int e = dlc_dtype_bytes(wd->dtype);
    if (!w || (uintptr_t)w % e) return DLC_STATUS_BAD_PARAM;
    Span s_x, s_y, s_z{0, 0}, s_r{0, 0};
    const Span s_w = span_bytes(w, (uint64_t)wd->k * wd->c * e);
    const Span s_b = bias ? span_bytes(bias, (uint64_t)wd->k * 4) : Span{0, 0};
    const Span s_sx = sx ? span_bytes(sx, (uint64_t)g.M * 4) : Span{0, 0};
    const Span s_sw = sw ? span_bytes(sw, (uint64_t)wd->k * 4) : Span{0, 0};
    if (!span_of(xd, x, false, s_x) || !span_of(yd, y, true, s_y)) return DLC_STATUS_BAD_PARAM;
    if (r) {
        if (!ready(rd)) return DLC_STATUS_NOT_INITIALIZED;
        if (!same_rows(rd, yd) || rd->c != yd->c || !span_of(rd, r, false, s_r)) return DLC_STATUS_BAD_PARAM;
        if (!is_float(rd->dtype)) return DLC_STATUS_NOT_SUPPORTED;
        g.r = row_tensor(rd, r);
    }
    if (z) {
        if (!ready(zd)) return DLC_STATUS_NOT_INITIALIZED;
        if (!same_rows(zd, yd) || zd->c != wd->k || !span_of(zd, z, true, s_z)) return DLC_STATUS_BAD_PARAM;
        if (!is_float(zd->dtype)) return DLC_STATUS_NOT_SUPPORTED;
        if (overlaps(s_z, {s_x, s_w, s_b, s_sx, s_sw, s_r, s_y})) return DLC_STATUS_BAD_PARAM;
        g.z = row_tensor(zd, z);
    }
    if (overlaps(s_y, {s_x, s_w, s_b, s_sx, s_sw}) || (r && overlaps(s_y, {s_r}) && !same_tensor(rd, r, yd, y)))
        return DLC_STATUS_BAD_PARAM;
    g.sa = sx;
    g.sb = sw;
    g.bias = bias;
    g.act = act;
    const size_t need = dlc_gemm_workspace(h, g);
    RETURN_IF(check_workspace(ws, ws_bytes, need));
    if (need && overlaps(span_bytes(ws, need), {s_x, s_w, s_b, s_sx, s_sw, s_r, s_y, s_z})) return DLC_STATUS_BAD_PARAM;
    g.ws = static_cast<char *>(ws);
    RETURN_IF(enter(h));
    return dlc_launch_gemm(h, g);
}

dlcStatus_t product_workspace(dlcHandle_t h, bool gated, dlcTensorDescriptor_t xd, const void *x,
                              dlcFilterDescriptor_t wd, const void *w, dlcTensorDescriptor_t yd, const void *y,
                              size_t *bytes) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    if (!bytes) return DLC_STATUS_BAD_PARAM;
    GemmProblem g;
    RETURN_IF(resolve_product(gated, xd, x, wd, w, yd, y, g));
    *bytes = dlc_gemm_workspace(h, g);
    return DLC_STATUS_SUCCESS;
}

dlcStatus_t product_kernel(dlcHandle_t h, bool gated, dlcTensorDescriptor_t xd, const void *x,
                           dlcFilterDescriptor_t wd, const void *w, dlcTensorDescriptor_t yd, const void *y,
                           dlcKernel_t *kernel) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    if (!kernel) return DLC_STATUS_BAD_PARAM;
    GemmProblem g;
    RETURN_IF(resolve_product(gated, xd, x, wd, w, yd, y, g));
    *kernel = dlc_gemm_variant(h, g);
    return DLC_STATUS_SUCCESS;
}

// The three steps of a backward pass and where each keeps its scratch.
struct BackwardPlan {
    ActGradProblem ag;
    GemmProblem gx, gw;       // dx = dz w, dw = dz^T x
    bool run_ag;
    // operands of the products that have to be copied first, all in one launch
    RowTensor source[DLC_MAX_PACKS];
    PackItem pack[DLC_MAX_PACKS];
    int packs = 0;
    size_t kept, scratch;  // dz and the copies, then one scratch area that the steps use in turn
    size_t total() const { return kept + scratch; }
};

BackwardPlan plan_backward(dlcContext *h, bool gated, const RowTensor &x, const RowTensor &w, dlcActivationMode_t act,
                           const RowTensor &z, const RowTensor &dy, const RowTensor &dx, const RowTensor &dw,
                           float *dbias, long long rows, int C, int K, char *ws) {
    BackwardPlan b;
    b.ag.rows = rows;
    b.ag.N = gated ? K / 2 : K;
    b.ag.gated = gated;
    b.ag.act = act;
    b.ag.dy = dy;
    b.ag.z = z;
    b.ag.dbias = dbias;
    // dz in BF16 with rows of a multiple of 16 bytes: the products read it
    // with TMA; rounding it is what lets them run on the tensor cores.
    // Without an activation dz is dy itself when that is BF16 already.
    RowTensor dz = dy;
    b.kept = 0;
    auto keep = [&](size_t bytes) {  // (sizing only: any aligned address)
        void *at = ws ? (void *)(ws + b.kept) : (void *)(uintptr_t)WS_ALIGN;
        b.kept += ws_round(bytes);
        return at;
    };
    const bool copy = gated || act != DLC_ACTIVATION_IDENTITY || dy.dt != DLC_DATA_BFLOAT16;
    if (copy) {
        const long long ld = ((long long)K + 7) / 8 * 8;
        dz.p = keep((size_t)rows * ld * 2);
        dz.dt = DLC_DATA_BFLOAT16;
        dz.m = RowMap{ld, 0, 0, 1, ld, 1, 1, 1};
        b.ag.dz = dz;
    }
    b.run_ag = copy || dbias;
    // (dz is read by both products: its copy serves both)
    auto packed = [&](const RowTensor &t, bool wanted, long long n, int ch) {
        const size_t bytes = wanted ? dlc_pack_bytes(t, n, ch) : 0;
        if (!bytes) return t;
        void *dst = keep(bytes);
        b.source[b.packs] = t;
        b.pack[b.packs] = PackItem{nullptr, n, ch, dst};
        ++b.packs;
        return dlc_packed(t, ch, dst);
    };
    const RowTensor dz_p = packed(dz, dx.p || dw.p, rows, K), w_p = packed(w, dx.p != nullptr, K, C),
                    x_p = packed(x, dw.p != nullptr, rows, C);
    char *scratch = ws ? ws + b.kept : nullptr;
    b.ag.ws = reinterpret_cast<float *>(scratch);
    b.gx.M = rows, b.gx.N = C, b.gx.K = K;
    b.gx.a.t = dz_p;
    b.gx.b.t = w_p;
    b.gx.b.trans = 1;
    b.gx.y = dx;
    b.gx.ws = scratch;
    b.gw.M = K, b.gw.N = C, b.gw.K = rows;
    b.gw.a.t = dz_p;
    b.gw.a.trans = 1;
    b.gw.b.t = x_p;
    b.gw.b.trans = 1;
    b.gw.y = dw;
    b.gw.ws = scratch;
    size_t s = 0;  // (the copies made, the products need none of their own)
    if (dbias) s = std::max(s, dlc_act_grad_workspace(h, b.ag));
    if (dx.p) s = std::max(s, dlc_gemm_workspace(h, b.gx));
    if (dw.p) s = std::max(s, dlc_gemm_workspace(h, b.gw));
    b.scratch = ws_round(s);
    return b;
}

dlcStatus_t resolve_backward(bool gated, dlcTensorDescriptor_t xd, dlcFilterDescriptor_t wd, dlcActivationMode_t act,
                             dlcTensorDescriptor_t zd, bool have_z, dlcTensorDescriptor_t dyd) {
    if (!xd || !wd || !dyd) return DLC_STATUS_BAD_PARAM;
    if (!xd->set || !wd->set || !dyd->set) return DLC_STATUS_NOT_INITIALIZED;
    RETURN_IF(check_act(act));
    if (wd->r != 1 || wd->s != 1 || wd->c != xd->c || !same_rows(xd, dyd) || wd->dtype != xd->dtype)
        return DLC_STATUS_BAD_PARAM;
    if ((gated && wd->k % 2) || dyd->c != (gated ? wd->k / 2 : wd->k)) return DLC_STATUS_BAD_PARAM;
    if (xd->dtype != DLC_DATA_BFLOAT16 || !is_float(dyd->dtype) || rows_of(xd) > 0x7fffffffLL)
        return DLC_STATUS_NOT_SUPPORTED;
    if (gated || act != DLC_ACTIVATION_IDENTITY) {
        if (!have_z) return DLC_STATUS_BAD_PARAM;
        if (!ready(zd)) return DLC_STATUS_NOT_INITIALIZED;
        if (!same_rows(zd, xd) || zd->c != wd->k) return DLC_STATUS_BAD_PARAM;
        if (!is_float(zd->dtype)) return DLC_STATUS_NOT_SUPPORTED;
    }
    return DLC_STATUS_SUCCESS;
}

dlcStatus_t product_backward(dlcHandle_t h, bool gated, dlcTensorDescriptor_t xd, const void *x,
                             dlcFilterDescriptor_t wd, const void *w, dlcActivationMode_t act,
                             dlcTensorDescriptor_t zd, const void *z, dlcTensorDescriptor_t dyd, const void *dy,
                             dlcTensorDescriptor_t dxd, void *dx, dlcFilterDescriptor_t dwd, void *dw, float *dbias,
                             void *ws, size_t ws_bytes) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    RETURN_IF(resolve_backward(gated, xd, wd, act, zd, z != nullptr, dyd));
    if (!dx && !dw && !dbias) return DLC_STATUS_BAD_PARAM;
    Span s_x, s_dy, s_z{0, 0}, s_dx{0, 0}, s_dw{0, 0};
    if (!w || (uintptr_t)w % 2 || !span_of(xd, x, false, s_x) || !span_of(dyd, dy, false, s_dy) || !fp32_ok(dbias))
        return DLC_STATUS_BAD_PARAM;
    const Span s_w = span_bytes(w, (uint64_t)wd->k * wd->c * 2);
    const bool need_z = gated || act != DLC_ACTIVATION_IDENTITY;
    if (need_z && !span_of(zd, z, false, s_z)) return DLC_STATUS_BAD_PARAM;
    const Span s_db = dbias ? span_bytes(dbias, (uint64_t)wd->k * 4) : Span{0, 0};
    RowTensor t_dx, t_dw;
    if (dx) {
        if (!ready(dxd)) return DLC_STATUS_NOT_INITIALIZED;
        if (!same_rows(dxd, xd) || dxd->c != xd->c || !span_of(dxd, dx, true, s_dx)) return DLC_STATUS_BAD_PARAM;
        if (!is_float(dxd->dtype)) return DLC_STATUS_NOT_SUPPORTED;
        t_dx = row_tensor(dxd, dx);
    }
    if (dw) {
        if (!dwd || !dwd->set) return DLC_STATUS_NOT_INITIALIZED;
        if (dwd->k != wd->k || dwd->c != wd->c || dwd->r != 1 || dwd->s != 1) return DLC_STATUS_BAD_PARAM;
        if (!is_float(dwd->dtype)) return DLC_STATUS_NOT_SUPPORTED;
        const int e = dlc_dtype_bytes(dwd->dtype);
        if ((uintptr_t)dw % e) return DLC_STATUS_BAD_PARAM;
        s_dw = span_bytes(dw, (uint64_t)dwd->k * dwd->c * e);
        t_dw = filter_rows(dwd, dw);
    }
    if ((dx && overlaps(s_dx, {s_x, s_w, s_dy, s_z, s_dw, s_db})) || (dw && overlaps(s_dw, {s_x, s_w, s_dy, s_z, s_db})) ||
        (dbias && overlaps(s_db, {s_x, s_w, s_dy, s_z})))
        return DLC_STATUS_BAD_PARAM;
    const BackwardPlan b =
        plan_backward(h, gated, row_tensor(xd, x), filter_rows(wd, w), act, need_z ? row_tensor(zd, z) : RowTensor(),
                      row_tensor(dyd, dy), t_dx, t_dw, dbias, rows_of(xd), xd->c, wd->k, static_cast<char *>(ws));
    RETURN_IF(check_workspace(ws, ws_bytes, b.total()));
    if (b.total() && overlaps(span_bytes(ws, b.total()), {s_x, s_w, s_dy, s_z, s_dx, s_dw, s_db}))
        return DLC_STATUS_BAD_PARAM;
    RETURN_IF(enter(h));
    PackItem packs[DLC_MAX_PACKS];
    RowTensor source[DLC_MAX_PACKS];
    for (int i = 0; i < b.packs; ++i) {
        source[i] = b.source[i];
        packs[i] = b.pack[i];
        packs[i].t = &source[i];
    }
    RETURN_IF(dlc_launch_pack(h, packs, b.packs));
    if (b.run_ag) RETURN_IF(dlc_launch_act_grad(h, b.ag));
    if (dx) RETURN_IF(dlc_launch_gemm(h, b.gx));
    if (dw) RETURN_IF(dlc_launch_gemm(h, b.gw));
    return DLC_STATUS_SUCCESS;
}

// Sized for dx, dw and dbias all wanted, so one workspace serves any subset.
dlcStatus_t product_backward_workspace(dlcHandle_t h, bool gated, dlcTensorDescriptor_t xd, const void *x,
                                       dlcFilterDescriptor_t wd, const void *w, dlcActivationMode_t act,
                                       dlcTensorDescriptor_t zd, dlcTensorDescriptor_t dyd, const void *dy,
                                       size_t *bytes) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    if (!bytes) return DLC_STATUS_BAD_PARAM;
    RETURN_IF(resolve_backward(gated, xd, wd, act, zd, true, dyd));
    void *any = (void *)(uintptr_t)WS_ALIGN;
    RowTensor dx = row_tensor(xd, any);
    const RowTensor dw = filter_rows(wd, any);
    const RowTensor z = gated || act != DLC_ACTIVATION_IDENTITY ? row_tensor(zd, any) : RowTensor();
    const BackwardPlan b = plan_backward(h, gated, row_tensor(xd, x ? x : any), filter_rows(wd, w ? w : any), act, z,
                                         row_tensor(dyd, dy ? dy : any), dx, dw, static_cast<float *>(any),
                                         rows_of(xd), xd->c, wd->k, nullptr);
    *bytes = b.total();
    return DLC_STATUS_SUCCESS;
}

}  // namespace

extern "C" {

// ---- RMS norm ------------------------------------------------------------------
dlcStatus_t dlcRmsNormForward(dlcHandle_t h, double epsilon, dlcTensorDescriptor_t xd, const void *x,
                              dlcTensorDescriptor_t rd, const void *residual, const float *gamma,
                              dlcTensorDescriptor_t td, void *total, dlcTensorDescriptor_t yd, void *y, float *scale) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    if (!xd || !yd || !gamma || !fp32_ok(gamma) || !(epsilon >= 0.0)) return DLC_STATUS_BAD_PARAM;
    if (!xd->set || !yd->set || (residual && !ready(rd)) || (total && !ready(td))) return DLC_STATUS_NOT_INITIALIZED;
    for (const dlcTensorStruct *d : {(const dlcTensorStruct *)yd, (const dlcTensorStruct *)(residual ? rd : nullptr),
                                     (const dlcTensorStruct *)(total ? td : nullptr)})
        if (d && (!same_rows(d, xd) || d->c != xd->c)) return DLC_STATUS_BAD_PARAM;
    if (!is_float(xd->dtype) || (residual && !is_float(rd->dtype)) || (total && !is_float(td->dtype)) ||
        !(is_float(yd->dtype) || yd->dtype == DLC_DATA_FLOAT8_E4M3))
        return DLC_STATUS_NOT_SUPPORTED;
    if ((yd->dtype == DLC_DATA_FLOAT8_E4M3) != (scale != nullptr) || !fp32_ok(scale)) return DLC_STATUS_BAD_PARAM;
    RmsProblem p;
    p.rows = rows_of(xd);
    p.C = xd->c;
    p.eps = (float)epsilon;
    Span s_x, s_y, s_r{0, 0}, s_t{0, 0};
    if (!span_of(xd, x, false, s_x) || !span_of(yd, y, true, s_y) || (residual && !span_of(rd, residual, false, s_r)) ||
        (total && !span_of(td, total, true, s_t)))
        return DLC_STATUS_BAD_PARAM;
    const Span s_g = span_bytes(gamma, (uint64_t)p.C * 4);
    const Span s_s = scale ? span_bytes(scale, (uint64_t)p.rows * 4) : Span{0, 0};
    if (overlaps(s_y, {s_x, s_r, s_t, s_g, s_s}) || (scale && overlaps(s_s, {s_x, s_r, s_t, s_g})))
        return DLC_STATUS_BAD_PARAM;
    if (total && (overlaps(s_t, {s_g}) || (overlaps(s_t, {s_x}) && !same_tensor(td, total, xd, x)) ||
                  (residual && overlaps(s_t, {s_r}) && !same_tensor(td, total, rd, residual))))
        return DLC_STATUS_BAD_PARAM;
    p.x = row_tensor(xd, x);
    if (residual) p.r = row_tensor(rd, residual);
    if (total) p.t = row_tensor(td, total);
    p.y = row_tensor(yd, y);
    if (!p.x.m.hw || !p.r.m.hw || !p.t.m.hw || !p.y.m.hw) return DLC_STATUS_NOT_SUPPORTED;
    p.gamma = gamma;
    p.scale = scale;
    RETURN_IF(enter(h));
    return dlc_launch_rms(h, p);
}

dlcStatus_t dlcGetRmsNormBackwardWorkspaceSize(dlcHandle_t h, dlcTensorDescriptor_t td, size_t *bytes) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    if (!td || !bytes) return DLC_STATUS_BAD_PARAM;
    if (!td->set) return DLC_STATUS_NOT_INITIALIZED;
    RmsBwdProblem p;
    p.rows = rows_of(td);
    p.C = td->c;
    *bytes = ws_round(dlc_rms_bwd_workspace(h, p));
    return DLC_STATUS_SUCCESS;
}

dlcStatus_t dlcRmsNormBackward(dlcHandle_t h, double epsilon, dlcTensorDescriptor_t dyd, const void *dy,
                               dlcTensorDescriptor_t td, const void *total, const float *gamma,
                               dlcTensorDescriptor_t dtd, const void *dtotal, dlcTensorDescriptor_t dxd, void *dx,
                               float *dgamma, void *ws, size_t ws_bytes) {
    if (!h) return DLC_STATUS_NOT_INITIALIZED;
    if (!dyd || !td || !dxd || !gamma || !fp32_ok(gamma) || !fp32_ok(dgamma) || !(epsilon >= 0.0))
        return DLC_STATUS_BAD_PARAM;
    if (!dyd->set || !td->set || !dxd->set || (dtotal && !ready(dtd))) return DLC_STATUS_NOT_INITIALIZED;
    for (const dlcTensorStruct *d : {(const dlcTensorStruct *)dyd, (const dlcTensorStruct *)dxd,
                                     (const dlcTensorStruct *)(dtotal ? dtd : nullptr)})
        if (d && (!same_rows(d, td) || d->c != td->c)) return DLC_STATUS_BAD_PARAM;
    if (!is_float(dyd->dtype) || !is_float(td->dtype) || !is_float(dxd->dtype) || (dtotal && !is_float(dtd->dtype)))
        return DLC_STATUS_NOT_SUPPORTED;
    RmsBwdProblem p;
    p.rows = rows_of(td);
    p.C = td->c;
    p.eps = (float)epsilon;
    Span s_dy, s_t, s_dx, s_dt{0, 0};
    if (!span_of(dyd, dy, false, s_dy) || !span_of(td, total, false, s_t) || !span_of(dxd, dx, true, s_dx) ||
        (dtotal && !span_of(dtd, dtotal, false, s_dt)))
        return DLC_STATUS_BAD_PARAM;
    const Span s_g = span_bytes(gamma, (uint64_t)p.C * 4);
    const Span s_dg = dgamma ? span_bytes(dgamma, (uint64_t)p.C * 4) : Span{0, 0};
    // dx may take dtotal's place (read by the thread that writes it)
    if (overlaps(s_dx, {s_dy, s_t, s_g, s_dg}) ||
        (dtotal && overlaps(s_dx, {s_dt}) && !same_tensor(dxd, dx, dtd, dtotal)) ||
        (dgamma && overlaps(s_dg, {s_dy, s_t, s_g, s_dt})))
        return DLC_STATUS_BAD_PARAM;
    p.dy = row_tensor(dyd, dy);
    p.t = row_tensor(td, total);
    if (dtotal) p.dt = row_tensor(dtd, dtotal);
    p.dx = row_tensor(dxd, dx);
    if (!p.dy.m.hw || !p.t.m.hw || !p.dt.m.hw || !p.dx.m.hw) return DLC_STATUS_NOT_SUPPORTED;
    p.gamma = gamma;
    p.dgamma = dgamma;
    const size_t need = dgamma ? ws_round(dlc_rms_bwd_workspace(h, p)) : 0;
    RETURN_IF(check_workspace(ws, ws_bytes, need));
    if (need && overlaps(span_bytes(ws, need), {s_dy, s_t, s_dx, s_dt, s_g, s_dg})) return DLC_STATUS_BAD_PARAM;
    p.ws = static_cast<float *>(ws);
    RETURN_IF(enter(h));
    return dlc_launch_rms_bwd(h, p);
}

// ---- linear layer ----------------------------------------------------------------
dlcStatus_t dlcLinearForward(dlcHandle_t h, dlcTensorDescriptor_t xd, const void *x, const float *xScale,
                             dlcFilterDescriptor_t wd, const void *w, const float *wScale, const float *bias,
                             dlcActivationMode_t act, dlcTensorDescriptor_t zd, void *z, dlcTensorDescriptor_t rd,
                             const void *residual, dlcTensorDescriptor_t yd, void *y, void *ws, size_t ws_bytes) {
    return product_forward(h, false, xd, x, xScale, wd, w, wScale, bias, act, zd, z, rd, residual, yd, y, ws, ws_bytes);
}

dlcStatus_t dlcGetLinearForwardWorkspaceSize(dlcHandle_t h, dlcTensorDescriptor_t xd, const void *x,
                                             dlcFilterDescriptor_t wd, const void *w, dlcTensorDescriptor_t yd,
                                             const void *y, size_t *bytes) {
    return product_workspace(h, false, xd, x, wd, w, yd, y, bytes);
}

dlcStatus_t dlcGetLinearForwardKernel(dlcHandle_t h, dlcTensorDescriptor_t xd, const void *x, dlcFilterDescriptor_t wd,
                                      const void *w, dlcTensorDescriptor_t yd, const void *y, dlcKernel_t *kernel) {
    return product_kernel(h, false, xd, x, wd, w, yd, y, kernel);
}

dlcStatus_t dlcLinearBackward(dlcHandle_t h, dlcTensorDescriptor_t xd, const void *x, dlcFilterDescriptor_t wd,
                              const void *w, dlcActivationMode_t act, dlcTensorDescriptor_t zd, const void *z,
                              dlcTensorDescriptor_t dyd, const void *dy, dlcTensorDescriptor_t dxd, void *dx,
                              dlcFilterDescriptor_t dwd, void *dw, float *dbias, void *ws, size_t ws_bytes) {
    return product_backward(h, false, xd, x, wd, w, act, zd, z, dyd, dy, dxd, dx, dwd, dw, dbias, ws, ws_bytes);
}

dlcStatus_t dlcGetLinearBackwardWorkspaceSize(dlcHandle_t h, dlcTensorDescriptor_t xd, const void *x,
                                              dlcFilterDescriptor_t wd, const void *w, dlcActivationMode_t act,
                                              dlcTensorDescriptor_t zd, dlcTensorDescriptor_t dyd, const void *dy,
                                              size_t *bytes) {
    return product_backward_workspace(h, false, xd, x, wd, w, act, zd, dyd, dy, bytes);
}

// ---- gated projections --------------------------------------------------------------
dlcStatus_t dlcGatedForward(dlcHandle_t h, dlcTensorDescriptor_t xd, const void *x, const float *xScale,
                            dlcFilterDescriptor_t wd, const void *w, const float *wScale, const float *bias,
                            dlcActivationMode_t act, dlcTensorDescriptor_t zd, void *z, dlcTensorDescriptor_t yd,
                            void *y, void *ws, size_t ws_bytes) {
    return product_forward(h, true, xd, x, xScale, wd, w, wScale, bias, act, zd, z, nullptr, nullptr, yd, y, ws,
                           ws_bytes);
}

dlcStatus_t dlcGetGatedForwardWorkspaceSize(dlcHandle_t h, dlcTensorDescriptor_t xd, const void *x,
                                            dlcFilterDescriptor_t wd, const void *w, dlcTensorDescriptor_t yd,
                                            const void *y, size_t *bytes) {
    return product_workspace(h, true, xd, x, wd, w, yd, y, bytes);
}

dlcStatus_t dlcGetGatedForwardKernel(dlcHandle_t h, dlcTensorDescriptor_t xd, const void *x, dlcFilterDescriptor_t wd,
                                     const void *w, dlcTensorDescriptor_t yd, const void *y, dlcKernel_t *kernel) {
    return product_kernel(h, true, xd, x, wd, w, yd, y, kernel);
}

dlcStatus_t dlcGatedBackward(dlcHandle_t h, dlcTensorDescriptor_t xd, const void *x, dlcFilterDescriptor_t wd,
                             const void *w, dlcActivationMode_t act, dlcTensorDescriptor_t zd, const void *z,
                             dlcTensorDescriptor_t dyd, const void *dy, dlcTensorDescriptor_t dxd, void *dx,
                             dlcFilterDescriptor_t dwd, void *dw, float *dbias, void *ws, size_t ws_bytes) {
    return product_backward(h, true, xd, x, wd, w, act, zd, z, dyd, dy, dxd, dx, dwd, dw, dbias, ws, ws_bytes);
}

dlcStatus_t dlcGetGatedBackwardWorkspaceSize(dlcHandle_t h, dlcTensorDescriptor_t xd, const void *x,
                                             dlcFilterDescriptor_t wd, const void *w, dlcActivationMode_t act,
                                             dlcTensorDescriptor_t zd, dlcTensorDescriptor_t dyd, const void *dy,
                                             size_t *bytes) {
    return product_backward_workspace(h, true, xd, x, wd, w, act, zd, dyd, dy, bytes);
}

}  // extern "C"

// channel_args.h -- how the C entries of the channel operators look at their
// arguments: descriptors as rows, address ranges, workspaces.
#pragma once

#include <climits>
#include <cstring>
#include <initializer_list>

#include "internal.h"

namespace dlc {

constexpr size_t WS_ALIGN = 256;
inline size_t ws_round(size_t b) { return (b + WS_ALIGN - 1) / WS_ALIGN * WS_ALIGN; }

inline long long rows_of(const dlcTensorStruct *d) { return (long long)d->n * d->h * d->w; }

inline bool same_rows(const dlcTensorStruct *a, const dlcTensorStruct *b) {
    return a->n == b->n && a->h == b->h && a->w == b->w;
}

inline bool is_float(dlcDataType_t t) { return t == DLC_DATA_FLOAT || t == DLC_DATA_BFLOAT16; }

inline RowTensor row_tensor(const dlcTensorStruct *d, const void *p) {
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
inline RowTensor filter_rows(const dlcFilterStruct *f, const void *p) {
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
inline bool span_of(const dlcTensorStruct *d, const void *p, bool output, Span &s) {
    const int64_t ext[4] = {d->n, d->c, d->h, d->w};
    const int e = dlc_dtype_bytes(d->dtype);
    const int64_t last = dlc_max_offset(ext, d->stride, 4);
    if (!p || (uintptr_t)p % e || last < 0 || last >= ((int64_t)1 << 60)) return false;
    if (output && !dlc_strides_injective(ext, d->stride, 4)) return false;
    s = Span{(uintptr_t)p, (uintptr_t)p + (uintptr_t)(last + 1) * e};
    return true;
}

inline Span span_bytes(const void *p, uint64_t bytes) { return Span{(uintptr_t)p, (uintptr_t)p + bytes}; }

inline bool overlaps(const Span &a, std::initializer_list<Span> others) {
    for (const Span &o : others)
        if (dlc_ranges_overlap(a.lo, a.hi, o.lo, o.hi)) return true;
    return false;
}

// The same buffer under the same descriptor values: an elementwise in-place use.
inline bool same_tensor(const dlcTensorStruct *a, const void *pa, const dlcTensorStruct *b, const void *pb) {
    return pa == pb && a->dtype == b->dtype && std::memcmp(a->stride, b->stride, sizeof(a->stride)) == 0;
}

inline bool fp32_ok(const float *p) { return (uintptr_t)p % 4 == 0; }

inline bool ready(dlcTensorDescriptor_t d) { return d && d->set; }

inline dlcStatus_t enter(dlcContext *h) {
    const volatile int *e = h->h_err;
    if (e && e[0] != 0) return DLC_STATUS_EXECUTION_FAILED;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev != h->device) return DLC_STATUS_BAD_PARAM;
    return DLC_STATUS_SUCCESS;
}

inline dlcStatus_t check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return DLC_STATUS_SUCCESS;
    return ws && have >= need && (uintptr_t)ws % WS_ALIGN == 0 ? DLC_STATUS_SUCCESS : DLC_STATUS_BAD_PARAM;
}

inline dlcStatus_t check_act(dlcActivationMode_t act) {
    if (act < DLC_ACTIVATION_IDENTITY || act > DLC_ACTIVATION_GELU) return DLC_STATUS_BAD_PARAM;
    return act == DLC_ACTIVATION_CLIPPED_RELU ? DLC_STATUS_NOT_SUPPORTED : DLC_STATUS_SUCCESS;
}

#define RETURN_IF(expr)                                  \
    do {                                                 \
        const dlcStatus_t st_ = (expr);                  \
        if (st_ != DLC_STATUS_SUCCESS) return st_;       \
    } while (0)

}  // namespace dlc

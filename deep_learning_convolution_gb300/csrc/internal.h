// internal.h -- host-side structures shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dlc.h"

// Largest element offset reachable through (extent, stride) pairs.
inline int64_t dlc_max_offset(const int64_t *ext, const int64_t *str, int nd) {
    int64_t m = 0;
    for (int i = 0; i < nd; ++i) m += (ext[i] - 1) * str[i];
    return m;
}

// True if distinct index tuples map to distinct offsets (no self-overlap):
// sorted by stride, each stride must reach past the span of the smaller ones.
inline bool dlc_strides_injective(const int64_t *ext, const int64_t *str, int nd) {
    int idx[4] = {0, 1, 2, 3};
    std::sort(idx, idx + nd, [&](int a, int b) { return str[a] < str[b]; });
    int64_t span = 0;  // max offset of the dims seen so far
    for (int i = 0; i < nd; ++i) {
        int d = idx[i];
        if (ext[d] == 1) continue;
        if (str[d] <= span) return false;
        span += (ext[d] - 1) * str[d];
    }
    return true;
}

inline bool dlc_ranges_overlap(uintptr_t a0, uintptr_t a1, uintptr_t b0, uintptr_t b1) {
    return a0 < b1 && b0 < a1;
}

struct dlcTensorStruct {
    int set = 0;
    dlcDataType_t dtype = DLC_DATA_FLOAT;
    int n = 0, c = 0, h = 0, w = 0;
    int64_t stride[4] = {0, 0, 0, 0};  // n, c, h, w (elements)
};

struct dlcFilterStruct {
    int set = 0;
    dlcDataType_t dtype = DLC_DATA_FLOAT;
    dlcTensorFormat_t format = DLC_TENSOR_NCHW;
    int k = 0, c = 0, r = 0, s = 0;
};

struct dlcPoolingStruct {
    int set = 0;
    dlcPoolingMode_t mode = DLC_POOLING_MAX;
    int r = 1, s = 1;
    int pad_top = 0, pad_bottom = 0, pad_left = 0, pad_right = 0;
    int u = 1, v = 1;
};

struct dlcConvolutionStruct {
    int set = 0;
    int pad_top = 0, pad_bottom = 0, pad_left = 0, pad_right = 0;
    int u = 1, v = 1, dil_h = 1, dil_w = 1;
    dlcMathType_t math = DLC_MATH_FP32;
    dlcConvolutionMode_t mode = DLC_CROSS_CORRELATION;
};

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
typedef CUresult (*EncodeIm2colFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const int *,
                                   const int *, cuuint32_t, cuuint32_t, const cuuint32_t *,
                                   CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct dlcContext {
    int device = 0;
    int sm_count = 0;
    cudaStream_t stream = nullptr;
    int *h_err = nullptr;   // mapped host words: [0] code, [1] detail
    int *d_err = nullptr;   // device alias of h_err
    uint64_t launches = 0;
    unsigned long long timeout_ns = 2000000000ull;  // pipeline wait limit
    int *sk_flags = nullptr;  // DLC_SK_FLAGS per-tile flags of split tiles (zero between launches)
    void *wpack = nullptr;    // filters repacked for the window and row-stack kernels
    size_t wpack_bytes = 0;   // its size
    int deterministic = 0;    // no split reductions whose partial sums meet in atomic adds
    EncodeTiledFn encode_tiled = nullptr;
    EncodeIm2colFn encode_im2col = nullptr;
    // What the device holds at once of the channel operators' clusters, 0 until the first
    // product asks (dlc_resident_clusters); every plan of a handle uses the same counts.
    mutable int resident_pairs = 0, resident_few[9] = {0};
};

// Split-tile flags owned by a handle: at most this many tiles per launch use them.
#define DLC_SK_FLAGS 4096
// Device bytes of the window kernel's repacked filter image (at most the
// shared memory of one CTA): the allocation-free entry point's fixed array.
#define DLC_WPACK_BYTES (256 * 1024)
// Device bytes a handle keeps for repacked filters: the window kernel's image
// or the row-stack kernel's filter slices (up to about one filter bank).
#define DLC_HANDLE_WPACK_BYTES (2 * 1024 * 1024)

inline int dlc_dtype_bytes(dlcDataType_t t) {
    return t == DLC_DATA_BFLOAT16 ? 2 : (t == DLC_DATA_DOUBLE ? 8 : (t == DLC_DATA_FLOAT8_E4M3 ? 1 : 4));
}

// A fully resolved forward problem (validated by the API layer).
struct ConvProblem {
    int N, C, H, W, K, R, S, P, Q;
    int pt, pb, pl, pr, u, v, dh, dw;
    dlcMathType_t math;
    dlcDataType_t xdt;   // storage of x and w
    dlcDataType_t ydt;   // storage of y
    dlcTensorFormat_t wfmt;
    const void *x;
    int64_t xs[4];       // n, c, h, w
    const void *w;
    int64_t ws[4];       // k, c, r, s
    void *y;
    int64_t ys[4];       // n, k, p, q
    const float *bias;
    float alpha, beta;
    int relu;
    // Filter taps read mirrored, w[k, c, R-1-r, S-1-s] (convolution mode, and
    // the data gradient's transposed filters).
    int flip = 0;
    // Filters given transposed: ws[0] is the stride of the output-channel
    // index k and must be 1 (contiguous), ws[1] that of the reduction channel
    // c.  The data gradient's problem reads the forward filters this way.
    int w_mn = 0;
};

// A fully resolved backward problem (validated by the API layer), in the
// forward problem's terms: x [N,C,H,W], w [K,C,R,S], dy [N,K,P,Q].  For the
// data gradient x is the output dx; for the filter gradient w is the output dw.
struct BwdProblem {
    int N, C, H, W, K, R, S, P, Q;
    int pt, pb, pl, pr, u, v, dh, dw;
    dlcMathType_t math;
    dlcDataType_t in_dt;   // storage of the two inputs
    dlcDataType_t out_dt;  // storage of the output
    dlcTensorFormat_t wfmt;
    int flip;              // convolution mode: the forward read w[k,c,R-1-r,S-1-s]
    const void *x;
    int64_t xs[4];         // n, c, h, w
    const void *w;
    int64_t ws[4];         // k, c, r, s
    const void *dy;
    int64_t dys[4];        // n, k, p, q
    double alpha, beta;
};

// Pooling forward (validated): x [N,C,H,W] -> y [N,C,P,Q].
struct PoolProblem {
    int N, C, H, W, R, S, P, Q;
    int pt, pl, u, v, mode;
    dlcDataType_t xdt, ydt;
    const void *x;
    int64_t xs[4];
    void *y;
    int64_t ys[4];
    double alpha, beta;
};

// Activation forward (validated): y = alpha * f(x) + beta * y, both [N,C,H,W].
struct ActProblem {
    int N, C, H, W, mode;
    dlcDataType_t xdt, ydt;
    const void *x;
    int64_t xs[4];
    void *y;
    int64_t ys[4];
    double alpha, beta, coef;
};

// pool_act.cu
dlcKernel_t dlc_pool_variant(const PoolProblem &pp);
dlcStatus_t dlc_launch_pool(dlcContext *ctx, const PoolProblem &pp);
dlcStatus_t dlc_launch_activation(dlcContext *ctx, const ActProblem &ap);

// conv_bwd.cu: data and filter gradients.
dlcKernel_t dlc_dgrad_variant(const dlcContext *ctx, const BwdProblem &bp);
dlcStatus_t dlc_launch_dgrad(dlcContext *ctx, const BwdProblem &bp);
dlcKernel_t dlc_wgrad_variant(const dlcContext *ctx, const BwdProblem &bp);
// conv_wgrad.cu: the filter gradient on the tensor cores (adds into dw).
bool dlc_wgrad_tc_ok(const BwdProblem &bp);
dlcStatus_t dlc_launch_wgrad_tc(dlcContext *ctx, const BwdProblem &bp);
dlcStatus_t dlc_launch_wgrad(dlcContext *ctx, const BwdProblem &bp);

// Kernel launchers (conv_ffma.cu, conv_tc.cu).  They return SUCCESS or an
// error status and count launches in ctx->launches.
dlcStatus_t dlc_launch_ffma(dlcContext *ctx, const ConvProblem &pb);
dlcKernel_t dlc_tc_variant(const dlcContext *ctx, const ConvProblem &pb);
dlcStatus_t dlc_launch_tc(dlcContext *ctx, const ConvProblem &pb, dlcKernel_t variant);
dlcStatus_t dlc_launch_wait_selftest(dlcContext *ctx, unsigned long long timeout_ns);
// conv_window.cu: layers with few channels per horizontal stride step.
bool dlc_window_ok(const ConvProblem &pb);
dlcStatus_t dlc_launch_window(dlcContext *ctx, const ConvProblem &pb);
// conv_pair.cu: the im2col lowering on pairs of SMs (DLC_TC_PAIR=0 turns it off).
bool dlc_pair_enabled(const dlcContext *ctx);
// Launches of the window and pair kernels overlap the tail of the grid before
// them (programmatic dependent launch) unless DLC_PDL=0.
bool dlc_pdl_enabled();
dlcStatus_t dlc_launch_pair(dlcContext *ctx, const ConvProblem &pb);
// conv_tc.cu: conditions of the TMA im2col lowering (single CTA and pairs).
bool dlc_im2col_ok(const ConvProblem &pb);
// Each loads every kernel of its translation unit into the current context
// (CUDA loads modules lazily by default, and a module load allocates device
// memory): the allocation-free entry point calls them at its per-device set-up.
dlcStatus_t dlc_preload_tc();
dlcStatus_t dlc_preload_window();
dlcStatus_t dlc_preload_pair();
dlcStatus_t dlc_preload_rowstack();
// conv_rowstack.cu: TF32 channel-planar layers with few filters and unit
// horizontal stride (filters stacked over output rows as the MMA's M side).
bool dlc_rowstack_ok(const dlcContext *ctx, const ConvProblem &pb);
dlcStatus_t dlc_launch_rowstack(dlcContext *ctx, const ConvProblem &pb);


// ---- channel operators (channel_api.cu, rmsnorm.cu, gemm.cu) -------------------
//
// A tensor as rows (pixels n, h, w in order) by channels.
struct RowMap {
    long long s0, s2, s3, cs;  // strides of n, h, w and of the channel (elements)
    long long ld;              // the rows' pitch when it is one number (uniform)
    int hw, w;                 // h * w and w (hw 0: rows that this cannot describe)
    int uniform;
};

// One tensor of a channel operator (p null: absent).
struct RowTensor {
    void *p = nullptr;
    int dt = DLC_DATA_FLOAT;
    RowMap m = {0, 0, 0, 1, 0, 1, 1, 1};
};

// Whether every row of t starts on a boundary of `bytes`.
inline bool dlc_aligned_rows(const RowTensor &t, long long bytes) {
    const long long e = dlc_dtype_bytes((dlcDataType_t)t.dt);
    auto mult = [&](long long s) { return (s * e) % bytes == 0; };
    return (uintptr_t)t.p % bytes == 0 && (t.m.uniform ? mult(t.m.ld) : (mult(t.m.s0) && mult(t.m.s2) && mult(t.m.s3)));
}

// RMS norm, forward and backward (validated by the API layer).
struct RmsProblem {
    long long rows;
    int C;
    float eps;
    RowTensor x, r, t, y;  // input, residual (or absent), their sum (or absent), output
    const float *gamma;
    float *scale;          // one per row when y is E4M3
};

struct RmsBwdProblem {
    long long rows;
    int C;
    float eps;
    RowTensor dy, t, dt, dx;  // dt: gradient arriving at the sum, or absent
    const float *gamma;
    float *dgamma;            // or null
    float *ws;                // per-block partial sums of dgamma
};

// Layer norm, forward and backward (validated by the API layer).
struct LayerProblem {
    long long rows;
    int C;
    float eps;
    RowTensor x, r, t, y;      // as in RmsProblem
    const float *gamma, *beta; // beta may be null
    float *scale;
};

struct LayerBwdProblem {
    long long rows;
    int C;
    float eps;
    RowTensor dy, t, dt, dx;
    const float *gamma;
    float *dgamma, *dbeta;     // or null
    float *ws;                 // per-block partial sums of both
};

// Dropout: y = r + keep(m, c) ? scale * x : 0 (validated by the API layer).
struct DropoutProblem {
    long long rows;
    int C;
    uint32_t border;           // words from this on keep their element
    float scale;
    RowTensor x, r, y;
    const unsigned long long *random;  // seed, step (device memory)
};

// Token or class numbers of the rows, 32 or 64 bits.
struct IndexList {
    const void *p = nullptr;
    int wide = 0;
};

// Rows of a table (validated by the API layer).  Backward: dtable (in `table`).
struct EmbeddingProblem {
    long long rows;
    int C, V;
    float scale;
    int accumulate;
    IndexList tokens;
    RowTensor table, y;
    char *ws;
};

// Softmax cross entropy on top of z = sa sb x w^T + bias (validated by the API layer).
struct CrossEntropyProblem {
    long long M = 0;
    int V = 0, K = 0;
    RowTensor x, w;                   // w: V rows of K
    const float *sa = nullptr, *sb = nullptr, *bias = nullptr;
    IndexList target;
    float *loss = nullptr, *lse = nullptr;      // backward: lse is read
    const float *dloss = nullptr;
    RowTensor dx, dw;                 // absent where not wanted
    float *dbias = nullptr;
    char *ws = nullptr;
};

// An operand of a product: element (i, k) is row i, channel k of the tensor, or
// row k, channel i where `trans` is set.
struct GemmOperand {
    RowTensor t;
    int trans = 0;
};

// What a product of a loss does with its logits instead of writing them (see gemm.cu).
enum { ENTROPY_NONE = 0, ENTROPY_PARTS = 1, ENTROPY_DZ = 2 };
struct EntropyTile {
    int mode = ENTROPY_NONE;
    int V = 0, n0 = 0;           // classes in all, and the first one of this product
    IndexList target;
    float2 *part = nullptr;      // PARTS: [part][M] (t, s), dlc_entropy_parts of them from part0 on
    int part0 = 0;
    float *chosen = nullptr;     // PARTS: [M] the target's logit
    const float *lse = nullptr, *dloss = nullptr;  // DZ; dz goes to y: BF16, rows padded to 16 bytes
    float *sums = nullptr;       // DZ: [M / 32][N] sums of dz over 32 rows, or null
    int terms = 1;               // DZ: 2 writes what y's rounding left, in M more rows
};

// y[m, n] = act(sa[m] sb[n] sum_k a(m, k) b(n, k) + bias[n]) + r[m, n], and
// z[m, n] the activation's argument; gated: b, sb, bias and z hold 2N entries
// (gate n, then up N + n) and y[m, n] = act(gate) * up.
struct GemmProblem {
    long long M = 0, K = 0;
    int N = 0, gated = 0, act = DLC_ACTIVATION_IDENTITY;
    GemmOperand a, b;
    const float *sa = nullptr, *sb = nullptr, *bias = nullptr;
    RowTensor z, r, y;
    EntropyTile entropy;
    int terms = 1;       // 2 (pair kernel): a is the sum of two operands, the second one's rows behind the first one's
    char *ws = nullptr;  // dlc_gemm_workspace bytes
};

// dz = dy * act'(z), or both halves of a gated row: dz = [dy up act'(gate), dy act(gate)];
// dbias = the sum of dz over the rows.
struct ActGradProblem {
    long long rows = 0;
    int N = 0, gated = 0, act = DLC_ACTIVATION_IDENTITY;
    RowTensor dy, z, dz;  // z absent for the identity; dz absent: only dbias
    float *dbias = nullptr;
    float *ws = nullptr;  // partial sums of dbias (dlc_act_grad_workspace bytes)
};

// gemm.cu
// An operand that TMA cannot load ([rows][ch], channels last) and where its copy goes.
struct PackItem {
    RowTensor *t;  // becomes the copy
    long long rows;
    int ch;
    void *dst;
};
constexpr int DLC_MAX_PACKS = 3;
size_t dlc_pack_bytes(const RowTensor &t, long long rows, int ch);  // 0: TMA loads it in place
RowTensor dlc_packed(const RowTensor &t, int ch, void *dst);
dlcStatus_t dlc_launch_pack(dlcContext *ctx, const PackItem *items, int n);
dlcKernel_t dlc_gemm_variant(const dlcContext *ctx, const GemmProblem &g);
size_t dlc_gemm_workspace(const dlcContext *ctx, const GemmProblem &g);
int dlc_entropy_parts(const dlcContext *ctx, const GemmProblem &g);
// Whether every output of the product is a sum of several CTAs' or warps' parts.
bool dlc_gemm_spread(const dlcContext *ctx, const GemmProblem &g);
dlcStatus_t dlc_launch_gemm(dlcContext *ctx, const GemmProblem &g);
// act_grad.cu
size_t dlc_act_grad_workspace(const dlcContext *ctx, const ActGradProblem &p);
dlcStatus_t dlc_launch_act_grad(dlcContext *ctx, const ActGradProblem &p);
// out[c] = sum_b ws[b * C + c] in a fixed order (rmsnorm.cu)
dlcStatus_t dlc_launch_column_sum(dlcContext *ctx, const float *ws, float *out, int C, int blocks);
// the same for rows of [C, C] partial sums and two outputs, each of which may be null
dlcStatus_t dlc_launch_column_sums(dlcContext *ctx, const float *ws, float *out, float *out2, int C, int blocks);
// layernorm.cu
dlcStatus_t dlc_launch_layer(dlcContext *ctx, const LayerProblem &p);
size_t dlc_layer_bwd_workspace(const dlcContext *ctx, long long rows, int C);
dlcStatus_t dlc_launch_layer_bwd(dlcContext *ctx, const LayerBwdProblem &p);
// layernorm_vec.cu, layernorm_shift.cu: false where the layout is not theirs
bool dlc_layer_vec(dlcContext *ctx, const LayerProblem &p, dlcStatus_t &status);
bool dlc_layer_bwd_vec(dlcContext *ctx, const LayerBwdProblem &p, dlcStatus_t &status);
bool dlc_layer_shift(dlcContext *ctx, const LayerProblem &p, dlcStatus_t &status);
bool dlc_layer_bwd_shift(dlcContext *ctx, const LayerBwdProblem &p, dlcStatus_t &status);
// dropout.cu
dlcStatus_t dlc_launch_dropout(dlcContext *ctx, const DropoutProblem &p);
// embedding.cu
dlcStatus_t dlc_launch_embedding(dlcContext *ctx, const EmbeddingProblem &p);
size_t dlc_embedding_bwd_workspace(const dlcContext *ctx, long long rows, int C, int V);
dlcStatus_t dlc_launch_embedding_bwd(dlcContext *ctx, const EmbeddingProblem &p);
// cross_entropy.cu
size_t dlc_cross_entropy_workspace(const dlcContext *ctx, const CrossEntropyProblem &p);
dlcStatus_t dlc_launch_cross_entropy(dlcContext *ctx, const CrossEntropyProblem &p);
size_t dlc_cross_entropy_bwd_workspace(const dlcContext *ctx, const CrossEntropyProblem &p);
dlcStatus_t dlc_launch_cross_entropy_bwd(dlcContext *ctx, const CrossEntropyProblem &p);
// rmsnorm.cu
dlcStatus_t dlc_launch_rms(dlcContext *ctx, const RmsProblem &p);
size_t dlc_rms_bwd_workspace(const dlcContext *ctx, const RmsBwdProblem &p);
dlcStatus_t dlc_launch_rms_bwd(dlcContext *ctx, const RmsBwdProblem &p);

// One launch on the context's stream that may overlap the tail of the kernel
// before it (see dlc_pdl_enabled); counts it.  Defined in channel_api.cu.
dlcStatus_t dlc_launch(dlcContext *ctx, const void *kernel, dim3 grid, dim3 block, size_t smem, void **args,
                       int cluster = 1);
// Lets a kernel of the channel operators use `bytes` of dynamic shared memory.
// False where the device refuses.  Defined in channel_api.cu.
bool dlc_allow_smem(const dlcContext *ctx, const void *kernel, size_t bytes);
// Clusters of `size` CTAs of a kernel that the context's device holds at once; asked once
// and kept in *known.  Defined in channel_api.cu.
int dlc_resident_clusters(const dlcContext *ctx, int *known, const void *kernel, int size, int threads, size_t smem);

/*
 * dlc.h -- C ABI of the GB300 (sm_103a) 2-D convolution library: the forward
 * convolution, its two backward routines, pooling and activation forward, and
 * the channel operators (RMS and layer norm, linear and gated layers, dropout,
 * embedding, softmax cross entropy) with their gradients.
 *
 * The forward (FPROP) convolution layer is
 *
 *   y[n,k,p,q] = act( alpha * sum_{c,r,s} x[n, c, p*u + r*dh - pad_top, q*v + s*dw - pad_left]
 *                                         * w[k,c,r,s]
 *                     + beta * y[n,k,p,q] + bias[k] )
 *
 * (cross-correlation; x reads as zero outside the image; act is identity or
 * ReLU), with P = floor((H + pad_top + pad_bottom - dh*(R-1) - 1) / u) + 1 and
 * Q likewise along W.
 *
 * Sources on the pages:
 *  - "cuDNN: Efficient Primitives for Deep Learning", method section: a C
 *    language API whose tensors and filters are opaque descriptors with
 *    arbitrary strides and layouts; the caller owns every device buffer and no
 *    auxiliary buffer is used; non-square inputs and asymmetric padding are
 *    supported (findings section).
 *  - "maxDNN: An Efficient Convolution Kernel for Deep Learning with Maxwell
 *    GPUs", method section: each output coordinate is the product of the input
 *    receptive field with the filter weights; efficiency counts only the
 *    direct-convolution FLOPs 2*N*K*P*Q*C*R*S.
 *  - "High-Performance Deep Learning via a Single Building Block", method
 *    section: the kernel is a batch-reduce GEMM, C += sum_i A_i * B_i, here
 *    with i running over the filter taps (r,s) and channel blocks.
 *  - "High Performance Zero-Memory Overhead Direct Convolutions", abstract and
 *    method section: no packing and no extra memory -- the workspace size is
 *    always 0.
 *
 * Conventions (all functions):
 *  - Every function returns a dlcStatus_t.  Pointers to descriptors and
 *    handles are host pointers; x, w, y and bias are device pointers owned by
 *    the caller; alpha and beta are host pointers to float.
 *  - Sizes and strides are in elements, not bytes.
 *  - Calls that launch work are asynchronous on the handle's stream.  Launch
 *    errors are reported by the call itself.  Errors that kernels detect on
 *    the device (a pipeline wait that ran out of time, a token beyond its table) are recorded in the
 *    handle and reported as DLC_STATUS_EXECUTION_FAILED by the next launching
 *    call on that handle and by dlcSynchronize(), which clears them.
 *  - The library allocates no device memory on any forward or backward call.
 *    dlcCreate allocates one small mapped host word for device error
 *    reports, the split-tile flags and a 2 MiB device buffer where calls of
 *    the few-channel kernels repack the filters before the convolution reads
 *    them (so two calls on one handle must not overlap on the GPU: use one
 *    handle per stream).  This buffer departs from the cuDNN page's "no
 *    auxiliary buffers"; the caller-visible workspace is zero.
 *  - A handle is not thread-safe; use one handle per host thread.
 */
#ifndef DLC_H_
#define DLC_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DLC_VERSION 100

typedef enum {
    DLC_STATUS_SUCCESS = 0,
    DLC_STATUS_NOT_INITIALIZED = 1,   /* handle or descriptor not created/set */
    DLC_STATUS_BAD_PARAM = 2,         /* shape, stride, pointer or size error */
    DLC_STATUS_NOT_SUPPORTED = 3,     /* valid request this library does not offer */
    DLC_STATUS_EXECUTION_FAILED = 4,  /* launch failed or a kernel reported an error */
    DLC_STATUS_INTERNAL_ERROR = 5,
    DLC_STATUS_ALLOC_FAILED = 6       /* host allocation failed */
} dlcStatus_t;

/* Storage type of x, w and y.  x and w must share it; y may be FLOAT or
 * BFLOAT16 independently (DOUBLE with DOUBLE inputs).  Bias is always FLOAT.
 * FLOAT8_E4M3 (8 bits: 4 of exponent, 3 of mantissa, largest value 448) is for
 * the channel operators; the convolution, pooling and activation calls return
 * NOT_SUPPORTED for it. */
typedef enum {
    DLC_DATA_FLOAT = 0,
    DLC_DATA_BFLOAT16 = 1,
    DLC_DATA_DOUBLE = 2,
    DLC_DATA_FLOAT8_E4M3 = 3
} dlcDataType_t;

/* Layouts.  For activations NCHW / NHWC; for filters NCHW means KCRS and NHWC
 * means KRSC. */
typedef enum {
    DLC_TENSOR_NCHW = 0,
    DLC_TENSOR_NHWC = 1
} dlcTensorFormat_t;

/* Arithmetic.  FP32: FP32 products and sums on CUDA cores (FFMA), FLOAT or
 * BFLOAT16 storage.  TF32: tensor cores, FLOAT storage read as TF32, FP32
 * accumulation.  BF16: tensor cores, BFLOAT16 storage, FP32 accumulation.
 * FP64: double-precision products and sums on CUDA cores (DFMA), DOUBLE
 * storage throughout (the cuDNN page's method section: routines in single and
 * double precision). */
typedef enum {
    DLC_MATH_FP32 = 0,
    DLC_MATH_TF32 = 1,
    DLC_MATH_BF16 = 2,
    DLC_MATH_FP64 = 3
} dlcMathType_t;

/* Filter orientation (cuDNN page, method section).  CROSS_CORRELATION sums
 * x[.., p*u + r*dh - pad_top, ..] * w[k,c,r,s] (the default, the formula at the
 * top of this file); CONVOLUTION mirrors the filter taps, w[k,c,R-1-r,S-1-s]. */
typedef enum {
    DLC_CROSS_CORRELATION = 0,
    DLC_CONVOLUTION = 1
} dlcConvolutionMode_t;

/* Activation functions (cuDNN page, summary and method section).  The fused
 * convolution epilogue takes IDENTITY and RELU; dlcActivationForward takes
 * the first five modes: f(x) = x, max(0, x), 1 / (1 + e^-x), tanh x,
 * min(max(0, x), coef).  The linear and gated layers take all but
 * CLIPPED_RELU, among them SILU, x / (1 + e^-x), and GELU, x Phi(x) with the
 * standard normal distribution function Phi. */
typedef enum {
    DLC_ACTIVATION_IDENTITY = 0,
    DLC_ACTIVATION_RELU = 1,
    DLC_ACTIVATION_SIGMOID = 2,
    DLC_ACTIVATION_TANH = 3,
    DLC_ACTIVATION_CLIPPED_RELU = 4,
    DLC_ACTIVATION_SILU = 5,
    DLC_ACTIVATION_GELU = 6
} dlcActivationMode_t;

/* Pooling (cuDNN page, summary and method section): the largest value of the
 * window's in-image elements, or their sum divided by the window size (the
 * padding counts as zeros) or by their number (the padding is excluded). */
typedef enum {
    DLC_POOLING_MAX = 0,
    DLC_POOLING_AVERAGE_COUNT_INCLUDE_PADDING = 1,
    DLC_POOLING_AVERAGE_COUNT_EXCLUDE_PADDING = 2
} dlcPoolingMode_t;

/* Which kernel a forward call launches (diagnostic). */
typedef enum {
    DLC_KERNEL_NONE = 0,
    DLC_KERNEL_FFMA = 1,          /* strict FP32 direct convolution, CUDA cores */
    DLC_KERNEL_TC_IM2COL = 2,     /* tcgen05 implicit GEMM, TMA im2col activations */
    DLC_KERNEL_TC_GATHER = 3,     /* tcgen05 implicit GEMM, element-gathered operands */
    DLC_KERNEL_TC_GATHER_RUNS = 4, /* tcgen05 implicit GEMM, operands gathered as contiguous
                                     runs: (s,c) of a filter row for NHWC + KRSC, s of a
                                     (c,r) pair for NCHW + KCRS */
    DLC_KERNEL_TC_WINDOW = 5,     /* tcgen05 implicit GEMM for few channels per stride step
                                     (v*C*element size <= 64 bytes, no horizontal dilation,
                                     K <= 256): lowered rows read in place from packed input
                                     rows in shared memory */
    DLC_KERNEL_TC_IM2COL_PAIR = 6, /* the TC_IM2COL lowering on pairs of SMs (a cluster of two
                                     CTAs shares each MMA of 256 output pixels; each CTA
                                     loads half of the filter tile) */
    DLC_KERNEL_DIRECT = 7,        /* backward routines and pooling: one output element per
                                     thread, CUDA cores, any strides */
    DLC_KERNEL_TC_WGRAD = 8,      /* filter gradient on the tensor cores: pixels as the
                                     reduction, both operands MN-major from TMA */
    DLC_KERNEL_POOL_NHWC = 9,     /* pooling with channels innermost: 16-byte vectors of
                                     channels per thread */
    DLC_KERNEL_TC_ROWSTACK = 10,  /* TF32, channel-planar (NCHW) x, unit horizontal stride,
                                     up to 64 filters: filters stacked over output rows as the
                                     MMA's M side, output pixels (per phase q mod 4) as N,
                                     read in place from shifted copies of input rows */
    DLC_KERNEL_GEMM_PAIR = 11,    /* channel operators: tcgen05 products on pairs of SMs, 256 rows
                                     a tile, operands by TMA */
    DLC_KERNEL_FEW_ROWS = 12,     /* channel operators: tcgen05 products with the filters as the
                                     MMA's M side, the reduction split over a cluster */
    DLC_KERNEL_GEMV = 13          /* channel operators: up to four rows on the CUDA cores, filters
                                     streamed by every warp */
} dlcKernel_t;

/* Storage of token and class numbers. */
typedef enum {
    DLC_INDEX_INT32 = 0,
    DLC_INDEX_INT64 = 1
} dlcIndexType_t;

/* Device error codes recorded by kernels (dlcGetLastDeviceError). */
typedef enum {
    DLC_DEVERR_NONE = 0,
    DLC_DEVERR_WAIT_TIMEOUT = 1,  /* a pipeline barrier wait ran out of time */
    DLC_DEVERR_INDEX = 2          /* a token or class number beyond the table (detail: its row) */
} dlcDeviceError_t;

typedef struct dlcContext *dlcHandle_t;
typedef struct dlcTensorStruct *dlcTensorDescriptor_t;
typedef struct dlcFilterStruct *dlcFilterDescriptor_t;
typedef struct dlcConvolutionStruct *dlcConvolutionDescriptor_t;
typedef struct dlcPoolingStruct *dlcPoolingDescriptor_t;

/* ---- library ------------------------------------------------------------ */

/* Human-readable name of a status code; never NULL. */
const char *dlcGetErrorString(dlcStatus_t status);

/* DLC_VERSION of the loaded library, written to *version. */
dlcStatus_t dlcGetVersion(int *version);

/* ---- handle ------------------------------------------------------------- */

/* Creates a handle bound to the current CUDA device and the legacy default
 * stream.  Allocates the host-side context, one mapped host word for
 * device error reports, the split-tile flags and the 2 MiB filter-repacking
 * buffer.  BAD_PARAM if handle is NULL, NOT_SUPPORTED if the
 * device is not compute capability 10.3, EXECUTION_FAILED on a CUDA error.
 * Source: cuDNN page, method section (a C library whose calls take a context
 * created once and bound to a stream). */
dlcStatus_t dlcCreate(dlcHandle_t *handle);

/* Frees the handle (does not synchronize; the caller must ensure no launched
 * work is still pending). */
dlcStatus_t dlcDestroy(dlcHandle_t handle);

/* Sets the stream (a cudaStream_t passed as void*; NULL = legacy default
 * stream) on which later calls launch.  Source: cuDNN page, method section
 * (the library runs on the caller's stream). */
dlcStatus_t dlcSetStream(dlcHandle_t handle, void *stream);
dlcStatus_t dlcGetStream(dlcHandle_t handle, void **stream);

/* Bitwise reproducibility.  By default (0) the SM-pair kernel splits the
 * output tiles of a launch's last, mostly idle wave along the reduction and
 * adds the partial sums into y with FP32 atomic adds, whose order varies from
 * run to run: those outputs can differ in their last bits between runs (each
 * run stays within the same error bound).  With deterministic = 1 every
 * kernel sums each output in a fixed order, so repeated calls give identical
 * bits, at the cost of the idle tail (a few microseconds per launch).
 * BAD_PARAM unless deterministic is 0 or 1.  No counterpart on the pages
 * (they are silent on reproducibility). */
dlcStatus_t dlcSetDeterministic(dlcHandle_t handle, int deterministic);
dlcStatus_t dlcGetDeterministic(dlcHandle_t handle, int *deterministic);

/* Synchronizes the handle's stream.  Returns EXECUTION_FAILED if a kernel
 * recorded a device error since the last call (the error is then cleared).
 * No counterpart on the pages: the bounded-wait failure report. */
dlcStatus_t dlcSynchronize(dlcHandle_t handle);

/* Synchronizes, then writes the last recorded device error code
 * (dlcDeviceError_t) and its detail word (which wait gave up, which row) and clears
 * them. */
dlcStatus_t dlcGetLastDeviceError(dlcHandle_t handle, int *code, int *detail);

/* Number of kernels this handle has launched since creation. */
dlcStatus_t dlcGetLaunchCount(dlcHandle_t handle, uint64_t *count);

/* ---- tensor descriptors (x and y) ---------------------------------------- */

dlcStatus_t dlcCreateTensorDescriptor(dlcTensorDescriptor_t *desc);
dlcStatus_t dlcDestroyTensorDescriptor(dlcTensorDescriptor_t desc);

/* Dense 4-D tensor in NCHW or NHWC order.  All sizes must be >= 1 and the
 * element count must fit in 63 bits.  Source: cuDNN page, method section
 * (opaque tensor descriptors; NCHW and NHWC both supported) and findings
 * section (non-square images). */
dlcStatus_t dlcSetTensor4dDescriptor(dlcTensorDescriptor_t desc, dlcTensorFormat_t format,
                                     dlcDataType_t dtype, int n, int c, int h, int w);

/* 4-D tensor with arbitrary non-negative strides (elements) for the logical
 * axes n, c, h, w: any layout, including sub-tensor views.  Source: cuDNN
 * page, method section (arbitrary strides along each dimension). */
dlcStatus_t dlcSetTensor4dDescriptorEx(dlcTensorDescriptor_t desc, dlcDataType_t dtype,
                                       int n, int c, int h, int w,
                                       int64_t nStride, int64_t cStride,
                                       int64_t hStride, int64_t wStride);

dlcStatus_t dlcGetTensor4dDescriptor(dlcTensorDescriptor_t desc, dlcDataType_t *dtype,
                                     int *n, int *c, int *h, int *w,
                                     int64_t *nStride, int64_t *cStride,
                                     int64_t *hStride, int64_t *wStride);

/* ---- filter descriptors (w) ---------------------------------------------- */

dlcStatus_t dlcCreateFilterDescriptor(dlcFilterDescriptor_t *desc);
dlcStatus_t dlcDestroyFilterDescriptor(dlcFilterDescriptor_t desc);

/* Dense K x C x R x S filter bank; format NCHW = KCRS, NHWC = KRSC.
 * Source: cuDNN page, method section (filter descriptors beside the tensor
 * descriptors; the filter layout follows the data layout). */
dlcStatus_t dlcSetFilter4dDescriptor(dlcFilterDescriptor_t desc, dlcDataType_t dtype,
                                     dlcTensorFormat_t format, int k, int c, int r, int s);

dlcStatus_t dlcGetFilter4dDescriptor(dlcFilterDescriptor_t desc, dlcDataType_t *dtype,
                                     dlcTensorFormat_t *format, int *k, int *c, int *r, int *s);

/* ---- convolution descriptors --------------------------------------------- */

dlcStatus_t dlcCreateConvolutionDescriptor(dlcConvolutionDescriptor_t *desc);
dlcStatus_t dlcDestroyConvolutionDescriptor(dlcConvolutionDescriptor_t desc);

/* Symmetric padding pad_h (top and bottom) and pad_w (left and right),
 * strides u (vertical) and v (horizontal), dilations, arithmetic.  Pads >= 0,
 * strides and dilations >= 1.  Source: cuDNN page, method section (padding
 * and strides of the convolution descriptor); maxDNN page, method section
 * (the arithmetic counted as direct-convolution FLOPs); dilation enters as
 * r*dh, s*dw (the pages are silent: the common convention). */
dlcStatus_t dlcSetConvolution2dDescriptor(dlcConvolutionDescriptor_t desc, int pad_h, int pad_w,
                                          int u, int v, int dilation_h, int dilation_w,
                                          dlcMathType_t math);

/* Asymmetric padding (replaces the symmetric pads).  Source: cuDNN page,
 * findings section (asymmetric padding). */
dlcStatus_t dlcSetConvolution2dPadding(dlcConvolutionDescriptor_t desc, int pad_top,
                                       int pad_bottom, int pad_left, int pad_right);

dlcStatus_t dlcGetConvolution2dDescriptor(dlcConvolutionDescriptor_t desc, int *pad_top,
                                          int *pad_bottom, int *pad_left, int *pad_right,
                                          int *u, int *v, int *dilation_h, int *dilation_w,
                                          dlcMathType_t *math);

/* Filter orientation (default CROSS_CORRELATION).  BAD_PARAM for another
 * value; NOT_INITIALIZED before dlcSetConvolution2dDescriptor.  Source: cuDNN
 * page, method section (both convolution and cross-correlation; CONVOLUTION
 * mirrors the filter taps in both axes). */
dlcStatus_t dlcSetConvolutionMode(dlcConvolutionDescriptor_t desc, dlcConvolutionMode_t mode);
dlcStatus_t dlcGetConvolutionMode(dlcConvolutionDescriptor_t desc, dlcConvolutionMode_t *mode);

/* ---- forward convolution ------------------------------------------------- */

/* Output dimensions N, K, P, Q.  BAD_PARAM if C differs between x and w or
 * if the dilated filter does not fit the padded input (P or Q < 1).  Source:
 * maxDNN page, method section (one output per receptive-field position; a
 * partial last window is dropped: the floor above). */
dlcStatus_t dlcGetConvolution2dForwardOutputDim(dlcConvolutionDescriptor_t conv,
                                                dlcTensorDescriptor_t xDesc,
                                                dlcFilterDescriptor_t wDesc,
                                                int *n, int *k, int *p, int *q);

/* Workspace needed by dlcConvolutionForward: always 0 bytes (zero memory
 * overhead).  Validates the problem like the forward call.  Source:
 * zero-memory-overhead page, abstract; cuDNN page, method section (no
 * auxiliary buffers). */
dlcStatus_t dlcGetConvolutionForwardWorkspaceSize(dlcHandle_t handle,
                                                  dlcTensorDescriptor_t xDesc,
                                                  dlcFilterDescriptor_t wDesc,
                                                  dlcConvolutionDescriptor_t conv,
                                                  dlcTensorDescriptor_t yDesc, size_t *bytes);

/* Kernel a forward call with these descriptors and pointers would launch;
 * x, w and y may be NULL (alignment is then taken as satisfied).  No
 * counterpart on the pages (a diagnostic). */
dlcStatus_t dlcGetConvolutionForwardKernel(dlcHandle_t handle,
                                           dlcTensorDescriptor_t xDesc, const void *x,
                                           dlcFilterDescriptor_t wDesc, const void *w,
                                           dlcConvolutionDescriptor_t conv,
                                           dlcTensorDescriptor_t yDesc, const void *y,
                                           dlcKernel_t *kernel);

/* y = alpha * conv(x, w) + beta * y.
 * x: device, xDesc layout; w: device, wDesc layout; y: device, yDesc layout
 * with dims (N, K, P, Q) and strides that map distinct elements to distinct
 * addresses.  beta == 0 means y is not read (NaN in y is overwritten).
 * y must not overlap x or w (BAD_PARAM).  x and w must share a storage type
 * that matches the math mode: FP32 math takes FLOAT or BFLOAT16, TF32 math
 * takes FLOAT, BF16 math takes BFLOAT16 (else NOT_SUPPORTED).
 * Non-finite inputs: x and w are expected finite.  An Inf or NaN in x reaches
 * every output whose receptive field holds it, as the sum defines; the
 * few-channel kernel (DLC_KERNEL_TC_WINDOW) also multiplies zero filter taps
 * with the input pixels just outside a window that share its packed phase
 * pixel, so there an output beside such a window can read NaN as well (same
 * image, rows whose window holds the pixel, within one stride step plus one
 * phase pixel of its column).  The row-stack kernel (DLC_KERNEL_TC_ROWSTACK)
 * likewise multiplies zero filter taps with input pixels up to 3 columns past
 * a window and with input rows of its block of output rows that a given
 * output row does not read (for one-channel layers also up to 3 input rows
 * past the block's span): there an output of the same image, within that
 * block of rows and within 4 horizontal strides of such a pixel, can read
 * NaN.  Every other kernel reads exactly each window.
 * Sources: maxDNN page, method section (each output is its receptive field
 * times the filter weights); cuDNN page, method section (C API, descriptors
 * with arbitrary strides, caller-owned buffers). */
dlcStatus_t dlcConvolutionForward(dlcHandle_t handle, const float *alpha,
                                  dlcTensorDescriptor_t xDesc, const void *x,
                                  dlcFilterDescriptor_t wDesc, const void *w,
                                  dlcConvolutionDescriptor_t conv, const float *beta,
                                  dlcTensorDescriptor_t yDesc, void *y);

/* y = act(alpha * conv(x, w) + beta * y + bias[k]); bias is a device array of
 * K floats or NULL (no bias).  Otherwise as dlcConvolutionForward.  Source:
 * the layer's epilogue (bias and activation after the sum); cuDNN page,
 * method section (activation functions beside the convolution). */
dlcStatus_t dlcConvolutionBiasActivationForward(dlcHandle_t handle, const float *alpha,
                                                dlcTensorDescriptor_t xDesc, const void *x,
                                                dlcFilterDescriptor_t wDesc, const void *w,
                                                dlcConvolutionDescriptor_t conv,
                                                const float *beta, const float *bias,
                                                dlcActivationMode_t activation,
                                                dlcTensorDescriptor_t yDesc, void *y);

/* ---- backward routines ---------------------------------------------------
 *
 * The cuDNN page's method section: beside the forward convolution the library
 * offers routines for backward propagation.  They are the derivatives of the
 * forward sum (with the descriptor's mode, pads, strides and dilations):
 *
 *   dx[n,c,h,w] = sum of dy[n,k,p,q] * w[k,c,r,s] over k, r, s and the outputs
 *                 (p, q) with p*u + r*dh - pad_top = h, q*v + s*dw - pad_left = w
 *   dw[k,c,r,s] = sum over n, p, q of dy[n,k,p,q] * x[n,c,p*u + r*dh - pad_top,
 *                 q*v + s*dw - pad_left]   (x reads as zero outside the image)
 *
 * (in convolution mode w[k,c,r,s] reads w[k,c,R-1-r,S-1-s] and dw is written
 * mirrored the same way).  The two inputs share a storage type matching the
 * math mode as for the forward call (FP32 math: FLOAT or BFLOAT16; TF32:
 * FLOAT; BF16: BFLOAT16; FP64: DOUBLE); the output is FLOAT or BFLOAT16 (DOUBLE
 * for FP64).  dy's dimensions must be the forward output's (N, K, P, Q).  The
 * output must not overlap an input (BAD_PARAM).  No workspace: the
 * workspace-size queries return 0.  Asynchronous on the handle's stream.
 */

/* dx = alpha * dgrad(w, dy) + beta * dx (beta == 0: dx is not read).
 * dxDesc gives N, C, H, W; wDesc K, C, R, S.  BF16 math with KRSC filters,
 * channels-innermost dy and dx and no dilation runs on the tensor cores (one
 * SM-pair launch per stride phase, filters read transposed); every other
 * combination runs the direct kernel (DLC_KERNEL_DIRECT).  Source: cuDNN
 * page, method section (backward routines); maxDNN page, research questions
 * (the forward techniques carry over to the backward pass). */
dlcStatus_t dlcConvolutionBackwardData(dlcHandle_t handle, const float *alpha,
                                       dlcFilterDescriptor_t wDesc, const void *w,
                                       dlcTensorDescriptor_t dyDesc, const void *dy,
                                       dlcConvolutionDescriptor_t conv, const float *beta,
                                       dlcTensorDescriptor_t dxDesc, void *dx);

/* dw = alpha * wgrad(x, dy) + beta * dw.  dwDesc gives K, C, R, S and the
 * layout of dw (KCRS or KRSC) and its storage type.  A FLOAT or DOUBLE dw may
 * be written by reductions split over CTAs whose partial sums meet in atomic
 * adds (their order varies; see dlcSetDeterministic, which turns the split
 * off).  Source: cuDNN page, method section (backward routines); batch-reduce
 * GEMM page, method section (the same building block, reducing over the
 * output pixels). */
dlcStatus_t dlcConvolutionBackwardFilter(dlcHandle_t handle, const float *alpha,
                                         dlcTensorDescriptor_t xDesc, const void *x,
                                         dlcTensorDescriptor_t dyDesc, const void *dy,
                                         dlcConvolutionDescriptor_t conv, const float *beta,
                                         dlcFilterDescriptor_t dwDesc, void *dw);

dlcStatus_t dlcGetConvolutionBackwardDataWorkspaceSize(dlcHandle_t handle,
                                                       dlcFilterDescriptor_t wDesc,
                                                       dlcTensorDescriptor_t dyDesc,
                                                       dlcConvolutionDescriptor_t conv,
                                                       dlcTensorDescriptor_t dxDesc,
                                                       size_t *bytes);
dlcStatus_t dlcGetConvolutionBackwardFilterWorkspaceSize(dlcHandle_t handle,
                                                         dlcTensorDescriptor_t xDesc,
                                                         dlcTensorDescriptor_t dyDesc,
                                                         dlcConvolutionDescriptor_t conv,
                                                         dlcFilterDescriptor_t dwDesc,
                                                         size_t *bytes);

/* Kernel the backward calls with these descriptors would launch (diagnostic;
 * pointers may be NULL, alignment is then taken as satisfied).  No
 * counterpart on the pages. */
dlcStatus_t dlcGetConvolutionBackwardDataKernel(dlcHandle_t handle, dlcFilterDescriptor_t wDesc,
                                                const void *w, dlcTensorDescriptor_t dyDesc,
                                                const void *dy, dlcConvolutionDescriptor_t conv,
                                                dlcTensorDescriptor_t dxDesc, const void *dx,
                                                dlcKernel_t *kernel);
dlcStatus_t dlcGetConvolutionBackwardFilterKernel(dlcHandle_t handle, dlcTensorDescriptor_t xDesc,
                                                  const void *x, dlcTensorDescriptor_t dyDesc,
                                                  const void *dy, dlcConvolutionDescriptor_t conv,
                                                  dlcFilterDescriptor_t dwDesc, const void *dw,
                                                  dlcKernel_t *kernel);

/* ---- pooling and activation forward ----------------------------------------
 *
 * The cuDNN page's summary and method section: pooling and activation
 * functions beside convolution, with the same tensor descriptors (any
 * strides) and caller-owned device buffers.  x and y may have different
 * layouts; storage FLOAT or BFLOAT16 (independently) or DOUBLE for both.
 * Sums and comparisons run in FP32 (FP64 for DOUBLE).  alpha and beta as for
 * the convolution (beta == 0: y is not read).  Asynchronous on the handle's
 * stream.  x and y must not overlap, except that dlcActivationForward may
 * run in place (x == y with identical descriptors).
 */

dlcStatus_t dlcCreatePoolingDescriptor(dlcPoolingDescriptor_t *desc);
dlcStatus_t dlcDestroyPoolingDescriptor(dlcPoolingDescriptor_t desc);

/* Window R x S, pads (each smaller than the window along its axis, so that
 * no window is empty), strides u, v >= 1.  BAD_PARAM otherwise.  Source:
 * cuDNN page, method section (pooling); the pad rule is this library's
 * reading (the page is silent). */
dlcStatus_t dlcSetPooling2dDescriptor(dlcPoolingDescriptor_t desc, dlcPoolingMode_t mode,
                                      int window_h, int window_w, int pad_top, int pad_bottom,
                                      int pad_left, int pad_right, int u, int v);
dlcStatus_t dlcGetPooling2dDescriptor(dlcPoolingDescriptor_t desc, dlcPoolingMode_t *mode,
                                      int *window_h, int *window_w, int *pad_top,
                                      int *pad_bottom, int *pad_left, int *pad_right, int *u,
                                      int *v);

/* Output dimensions N, C, P, Q (P = floor((H + pad_top + pad_bottom - R) / u) + 1,
 * Q likewise). */
dlcStatus_t dlcGetPooling2dForwardOutputDim(dlcPoolingDescriptor_t desc,
                                            dlcTensorDescriptor_t xDesc, int *n, int *c, int *p,
                                            int *q);

/* y[n,c,p,q] = alpha * POOL(window of x[n,c]) + beta * y[n,c,p,q].
 * POOL: the maximum, or the window sum over R*S (padding counted) or over the
 * in-image elements (padding excluded).  Source: cuDNN page, summary and
 * method section (pooling beside convolution). */
dlcStatus_t dlcPoolingForward(dlcHandle_t handle, dlcPoolingDescriptor_t desc, const float *alpha,
                              dlcTensorDescriptor_t xDesc, const void *x, const float *beta,
                              dlcTensorDescriptor_t yDesc, void *y);

/* Kernel dlcPoolingForward would launch (diagnostic; pointers may be NULL). */
dlcStatus_t dlcGetPoolingForwardKernel(dlcHandle_t handle, dlcPoolingDescriptor_t desc,
                                       dlcTensorDescriptor_t xDesc, const void *x,
                                       dlcTensorDescriptor_t yDesc, const void *y,
                                       dlcKernel_t *kernel);

/* y = alpha * f(x) + beta * y elementwise; x and y of the same dimensions.
 * coef is the ceiling of CLIPPED_RELU (ignored otherwise).  Source: cuDNN
 * page, summary and method section (activation functions; the page names no
 * list: identity, ReLU, sigmoid, tanh and clipped ReLU are this library's
 * reading). */
dlcStatus_t dlcActivationForward(dlcHandle_t handle, dlcActivationMode_t mode, double coef,
                                 const float *alpha, dlcTensorDescriptor_t xDesc, const void *x,
                                 const float *beta, dlcTensorDescriptor_t yDesc, void *y);

/* ---- channel operators -------------------------------------------------------
 *
 * What a network does with the channels of each pixel (or token) between
 * convolutions: RMS norm with the residual's addition, linear layers (products
 * over the channels) and gated projections, with their gradients.  No
 * counterpart on the pages.
 *
 * A tensor [n, c, h, w] is read as rows (n, h, w) of c channels; a matrix of
 * rows x channels is [rows, channels, 1, 1].  Any strides and alignment are
 * taken; channels contiguous, rows at one pitch and 16-byte aligned are the
 * fast layout.  Filters are [K, C, 1, 1], K rows of C channels.  Sums,
 * statistics and activations run in FP32; BFLOAT16 and FLOAT8_E4M3 results are
 * rounded once, to nearest even.  An FP8 row or filter stands for its values
 * times its FLOAT scale.  Products take up to 2^31 - 1 rows, norms more; several
 * images of 2^31 pixels and more each have to be one pitch apart (NOT_SUPPORTED).
 *
 * Pointers are device pointers; those marked optional may be NULL, and their
 * descriptor is then ignored.  Relative errors of the activations (FP32, before
 * a result is rounded to its type): GELU 4e-6 + 1e-7 z^2, SILU and SIGMOID 1e-6 +
 * 2e-7 |z|.  Outputs must not overlap other arguments
 * (BAD_PARAM; the address ranges that strides reach count) but for the in-place
 * uses named at each call.  A workspace is caller-owned, 256-byte aligned and
 * of at least the queried size (else BAD_PARAM; NULL where that is 0); its
 * contents need not be kept between calls.  The queries take pointers, which
 * may be NULL (alignment then taken as satisfied): an operand the kernels
 * cannot load in place is copied into the workspace first.  All calls are
 * bitwise reproducible, can be captured in a CUDA graph, allocate nothing and
 * are asynchronous on the handle's stream.
 */

/* total = x + residual;  y = gamma * total / sqrt(mean over channels of
 * total^2 + epsilon), from the unrounded total.  x, residual (optional), total
 * (optional output): FLOAT or BFLOAT16 independently; gamma: FLOAT, one per
 * channel.  y: FLOAT, BFLOAT16, or FLOAT8_E4M3 with scale[row] = max over
 * channels of |y| / 448 (FLOAT, one per row in order n, h, w; required then and
 * NULL otherwise; max |y| counts as at least 1e-30, so a row of zeros gives
 * zeros whatever epsilon is; FLOAT and BFLOAT16 y of a row of zeros with epsilon
 * 0 is 0 / 0, NaN).  NaN or infinity in a row makes that row NaN or zero, no other.
 * total may be x or residual in place (same descriptor values).  epsilon >= 0.
 * Squares are summed in FP32: rows whose sum of squares leaves its range (values
 * of 1e18 and more, or of 1e-18 and less beside a smaller epsilon) do not have
 * this result, nor its gradient. */
dlcStatus_t dlcRmsNormForward(dlcHandle_t handle, double epsilon, dlcTensorDescriptor_t xDesc,
                              const void *x, dlcTensorDescriptor_t residualDesc,
                              const void *residual, const float *gamma,
                              dlcTensorDescriptor_t totalDesc, void *total,
                              dlcTensorDescriptor_t yDesc, void *y, float *scale);

/* Workspace of dlcRmsNormBackward when dgamma is wanted (0 bytes otherwise). */
dlcStatus_t dlcGetRmsNormBackwardWorkspaceSize(dlcHandle_t handle,
                                               dlcTensorDescriptor_t totalDesc, size_t *bytes);

/* Gradient of the norm at total, which is also that of x and of residual:
 *   dx = dtotal + rho * dy * gamma - total * rho^3 * mean(dy * gamma * total)
 *   dgamma = sum over rows of dy * total * rho,  rho = 1 / sqrt(mean(total^2) + epsilon)
 * dtotal (optional): the gradient that reaches total by other ways (the residual
 * stream); dx may be dtotal in place.  dgamma (FLOAT) is optional.  Tensors
 * FLOAT or BFLOAT16 independently. */
dlcStatus_t dlcRmsNormBackward(dlcHandle_t handle, double epsilon, dlcTensorDescriptor_t dyDesc,
                               const void *dy, dlcTensorDescriptor_t totalDesc, const void *total,
                               const float *gamma, dlcTensorDescriptor_t dtotalDesc,
                               const void *dtotal, dlcTensorDescriptor_t dxDesc, void *dx,
                               float *dgamma, void *workspace, size_t workspaceBytes);

/* Linear layer: z[m, k] = xScale[m] * wScale[k] * sum_c x[m, c] * w[k, c] + bias[k],
 * y = act(z) + residual.
 * x and w: both BFLOAT16 (xScale and wScale NULL), or both FLOAT8_E4M3 with
 * FLOAT scales, one per row and one per filter.  bias (FLOAT), z and residual
 * are optional; z (an output, what the backward pass reads), residual and y are
 * FLOAT or BFLOAT16 independently.  residual may be y in place (same descriptor
 * values).  act: any but CLIPPED_RELU (NOT_SUPPORTED). */
dlcStatus_t dlcLinearForward(dlcHandle_t handle, dlcTensorDescriptor_t xDesc, const void *x,
                             const float *xScale, dlcFilterDescriptor_t wDesc, const void *w,
                             const float *wScale, const float *bias, dlcActivationMode_t act,
                             dlcTensorDescriptor_t zDesc, void *z,
                             dlcTensorDescriptor_t residualDesc, const void *residual,
                             dlcTensorDescriptor_t yDesc, void *y, void *workspace,
                             size_t workspaceBytes);

dlcStatus_t dlcGetLinearForwardWorkspaceSize(dlcHandle_t handle, dlcTensorDescriptor_t xDesc,
                                             const void *x, dlcFilterDescriptor_t wDesc,
                                             const void *w, dlcTensorDescriptor_t yDesc,
                                             const void *y, size_t *bytes);

/* Kernel that multiplies in dlcLinearForward (diagnostic; pointers may be NULL). */
dlcStatus_t dlcGetLinearForwardKernel(dlcHandle_t handle, dlcTensorDescriptor_t xDesc,
                                      const void *x, dlcFilterDescriptor_t wDesc, const void *w,
                                      dlcTensorDescriptor_t yDesc, const void *y,
                                      dlcKernel_t *kernel);

/* Gradients of the linear layer; that of residual is dy itself.
 *   dz = dy * act'(z);  dx = dz w;  dw = dz^T x;  dbias = sum over rows of dz
 * dz enters the products rounded to BFLOAT16; dbias sums its FP32 values.  x and
 * w: BFLOAT16; dy, dx, dw and z: FLOAT or BFLOAT16 independently; dbias: FLOAT.
 * dx, dw and dbias are each optional, one at least is wanted.  z is what the
 * forward call wrote, not read for IDENTITY (may be NULL then). */
dlcStatus_t dlcLinearBackward(dlcHandle_t handle, dlcTensorDescriptor_t xDesc, const void *x,
                              dlcFilterDescriptor_t wDesc, const void *w, dlcActivationMode_t act,
                              dlcTensorDescriptor_t zDesc, const void *z,
                              dlcTensorDescriptor_t dyDesc, const void *dy,
                              dlcTensorDescriptor_t dxDesc, void *dx, dlcFilterDescriptor_t dwDesc,
                              void *dw, float *dbias, void *workspace, size_t workspaceBytes);

/* Workspace for any subset of the three gradients. */
dlcStatus_t dlcGetLinearBackwardWorkspaceSize(dlcHandle_t handle, dlcTensorDescriptor_t xDesc,
                                              const void *x, dlcFilterDescriptor_t wDesc,
                                              const void *w, dlcActivationMode_t act,
                                              dlcTensorDescriptor_t zDesc,
                                              dlcTensorDescriptor_t dyDesc, const void *dy,
                                              size_t *bytes);

/* Gated projections: w holds 2F filters, F gates and then F ups, and so do
 * bias, wScale and z;  with z as in the linear layer,
 *   y[m, f] = act(z[m, f]) * z[m, F + f].
 * Types, optional arguments and activations as for dlcLinearForward. */
dlcStatus_t dlcGatedForward(dlcHandle_t handle, dlcTensorDescriptor_t xDesc, const void *x,
                            const float *xScale, dlcFilterDescriptor_t wDesc, const void *w,
                            const float *wScale, const float *bias, dlcActivationMode_t act,
                            dlcTensorDescriptor_t zDesc, void *z, dlcTensorDescriptor_t yDesc,
                            void *y, void *workspace, size_t workspaceBytes);

dlcStatus_t dlcGetGatedForwardWorkspaceSize(dlcHandle_t handle, dlcTensorDescriptor_t xDesc,
                                            const void *x, dlcFilterDescriptor_t wDesc,
                                            const void *w, dlcTensorDescriptor_t yDesc,
                                            const void *y, size_t *bytes);

/* Kernel that multiplies in dlcGatedForward (diagnostic; pointers may be NULL). */
dlcStatus_t dlcGetGatedForwardKernel(dlcHandle_t handle, dlcTensorDescriptor_t xDesc, const void *x,
                                     dlcFilterDescriptor_t wDesc, const void *w,
                                     dlcTensorDescriptor_t yDesc, const void *y,
                                     dlcKernel_t *kernel);

/* Gradients of the gated projections (z is required):
 *   dz = [dy * up * act'(gate), dy * act(gate)];  dx = dz w;  dw = dz^T x;
 *   dbias = sum over rows of dz
 * with types and optional arguments as for dlcLinearBackward. */
dlcStatus_t dlcGatedBackward(dlcHandle_t handle, dlcTensorDescriptor_t xDesc, const void *x,
                             dlcFilterDescriptor_t wDesc, const void *w, dlcActivationMode_t act,
                             dlcTensorDescriptor_t zDesc, const void *z,
                             dlcTensorDescriptor_t dyDesc, const void *dy,
                             dlcTensorDescriptor_t dxDesc, void *dx, dlcFilterDescriptor_t dwDesc,
                             void *dw, float *dbias, void *workspace, size_t workspaceBytes);

dlcStatus_t dlcGetGatedBackwardWorkspaceSize(dlcHandle_t handle, dlcTensorDescriptor_t xDesc,
                                             const void *x, dlcFilterDescriptor_t wDesc,
                                             const void *w, dlcActivationMode_t act,
                                             dlcTensorDescriptor_t zDesc,
                                             dlcTensorDescriptor_t dyDesc, const void *dy,
                                             size_t *bytes);

/* ---- channel operators at a network's ends and between its layers ---------------
 *
 * Layer norm, dropout, the embedding of tokens and softmax cross entropy on top
 * of a linear layer, with their gradients.  What is said above of the channel
 * operators (rows, layouts, types, workspaces, reproducibility, capture) holds
 * here too.  No counterpart on the pages.
 *
 * Tokens, and the classes that are the targets of a loss, are dense arrays of
 * one number a row in order n, h, w, 32 or 64 bits wide (dlcIndexType_t) and
 * aligned to that.  A negative one stands for none (a padded row); one beyond
 * the last row of the table counts as none as well, and the kernel records
 * DLC_DEVERR_INDEX with the row, which dlcSynchronize and the handle's next
 * call report.  These calls take up to 2^31 - 1 rows, the layer norm more, and
 * up to 2^31 - 2^16 channels and rows of a table.
 */

/* total = x + residual;  with mean and variance over the channels of a row,
 *   y = gamma * (total - mean) / sqrt(variance + epsilon) + beta
 * from the unrounded total; the variance is the mean square about the mean.
 * beta (FLOAT, one per channel) may be NULL: zeros.  Types, E4M3 rows with their
 * scale, in-place total, NaN and FP32 range as for dlcRmsNormForward (the sum of
 * squares being that about the mean).  Rows far from zero are centred twice, so that
 * a row of equal channels (up to 2^19 of them) is beta, whatever they are; with
 * epsilon 0 it is 0 / 0, NaN, in every type. */
dlcStatus_t dlcLayerNormForward(dlcHandle_t handle, double epsilon, dlcTensorDescriptor_t xDesc,
                                const void *x, dlcTensorDescriptor_t residualDesc,
                                const void *residual, const float *gamma, const float *beta,
                                dlcTensorDescriptor_t totalDesc, void *total,
                                dlcTensorDescriptor_t yDesc, void *y, float *scale);

/* Workspace of dlcLayerNormBackward when dgamma or dbeta is wanted (0 bytes
 * otherwise). */
dlcStatus_t dlcGetLayerNormBackwardWorkspaceSize(dlcHandle_t handle,
                                                 dlcTensorDescriptor_t totalDesc, size_t *bytes);

/* Gradient of the layer norm at total, which is also that of x and of residual:
 * with n = (total - mean) rho, rho = 1 / sqrt(variance + epsilon), d = dy gamma,
 *   dx = dtotal + rho * (d - mean(d) - n * mean(d n))
 *   dgamma = sum over rows of dy * n;  dbeta = sum over rows of dy
 * dtotal, dgamma and dbeta are optional; dx may be dtotal in place.  Tensors FLOAT
 * or BFLOAT16 independently. */
dlcStatus_t dlcLayerNormBackward(dlcHandle_t handle, double epsilon, dlcTensorDescriptor_t dyDesc,
                                 const void *dy, dlcTensorDescriptor_t totalDesc,
                                 const void *total, const float *gamma,
                                 dlcTensorDescriptor_t dtotalDesc, const void *dtotal,
                                 dlcTensorDescriptor_t dxDesc, void *dx, float *dgamma,
                                 float *dbeta, void *workspace, size_t workspaceBytes);

/* y = residual + (keep ? x * scale : 0): every element is dropped with the
 * probability floor(probability * 2^32) / 2^32, 0 <= probability < 1, the others
 * are scaled by the inverse of what is kept.  What is dropped counts as 0, NaN and
 * infinity too.  residual is optional; x, residual and y: FLOAT or BFLOAT16
 * independently; y may be x or residual in place (same descriptor values).
 *
 * random: two 64-bit words in device memory, a seed and a step, read when the
 * kernel runs, so that a captured graph drops anew when they are changed between its
 * replays.  Element (row m, channel c) is kept where word c mod 4 of Philox
 * 4x32-10 (Salmon et al., 2011; key: the seed's low and high word; counter: c / 4,
 * m, the step's low and high word) is at least floor(probability * 2^32).  The
 * mask depends on nothing else, not on layout or type, and is not stored: the
 * backward call works it out again from the same words. */
dlcStatus_t dlcDropoutForward(dlcHandle_t handle, double probability, const uint64_t *random,
                              dlcTensorDescriptor_t xDesc, const void *x,
                              dlcTensorDescriptor_t residualDesc, const void *residual,
                              dlcTensorDescriptor_t yDesc, void *y);

/* dx = keep ? dy * scale : 0 with the same mask (the residual's gradient is dy);
 * dx may be dy in place. */
dlcStatus_t dlcDropoutBackward(dlcHandle_t handle, double probability, const uint64_t *random,
                               dlcTensorDescriptor_t dyDesc, const void *dy,
                               dlcTensorDescriptor_t dxDesc, void *dx);

/* y[m] = scale * table[tokens[m]], zeros for a token that stands for none.  table:
 * V rows of C channels ([V, C, 1, 1]); y: rows of C channels; FLOAT or BFLOAT16
 * independently.  scale is finite (in FP32). */
dlcStatus_t dlcEmbeddingForward(dlcHandle_t handle, double scale, dlcIndexType_t indexType,
                                const void *tokens, dlcFilterDescriptor_t tableDesc,
                                const void *table, dlcTensorDescriptor_t yDesc, void *y);

dlcStatus_t dlcGetEmbeddingBackwardWorkspaceSize(dlcHandle_t handle, dlcTensorDescriptor_t dyDesc,
                                                 dlcFilterDescriptor_t dtableDesc, size_t *bytes);

/* dtable[v] = scale * (sum of dy over the rows whose token is v, in FP32 and always in
 * the same order); rows of no token become zero.  With accumulate != 0 this is added
 * to what dtable holds (a table shared with another layer, several batches), and rows
 * of no token are neither read nor written. */
dlcStatus_t dlcEmbeddingBackward(dlcHandle_t handle, double scale, dlcIndexType_t indexType,
                                 const void *tokens, dlcTensorDescriptor_t dyDesc, const void *dy,
                                 int accumulate, dlcFilterDescriptor_t dtableDesc, void *dtable,
                                 void *workspace, size_t workspaceBytes);

/* Softmax cross entropy of the classes that a linear layer rates: with z as in
 * dlcLinearForward (x and w: both BFLOAT16, or both FLOAT8_E4M3 with scales; w holds one
 * filter a class; bias optional),
 *   lse[m] = log sum_k exp z[m, k];  loss[m] = lse[m] - z[m, target[m]]
 * loss[m] is 0 for a target that stands for none, and NaN for one beyond the last
 * class.  loss and lse: FLOAT, one per row.  The logits are worked out in pieces and
 * not kept.  A class with z = -inf (a bias of -inf) has probability 0; a row of
 * nothing else has lse = -inf and no loss (NaN). */
dlcStatus_t dlcCrossEntropyForward(dlcHandle_t handle, dlcTensorDescriptor_t xDesc, const void *x,
                                   const float *xScale, dlcFilterDescriptor_t wDesc, const void *w,
                                   const float *wScale, const float *bias,
                                   dlcIndexType_t indexType, const void *target, float *loss,
                                   float *lse, void *workspace, size_t workspaceBytes);

dlcStatus_t dlcGetCrossEntropyForwardWorkspaceSize(dlcHandle_t handle, dlcTensorDescriptor_t xDesc,
                                                   const void *x, dlcFilterDescriptor_t wDesc,
                                                   const void *w, size_t *bytes);

/* Gradients of sum_m dloss[m] * loss[m] (dloss: FLOAT, one per row; the weight that
 * a mean over the rows gives each), from what the forward call wrote to lse:
 *   dz[m, k] = dloss[m] * (exp(z[m, k] - lse[m]) - (k == target[m]))
 *   dx = dz w;  dw = dz^T x;  dbias = sum over rows of dz
 * dz is 0 for rows whose target stands for none, whatever dloss is.  x and w: BFLOAT16; dz
 * enters the products in BFLOAT16: up to 128 rows, and up to 2^30 products of a row, class
 * and channel, in two terms, which keep 16 bits of it, else rounded to one; dbias sums
 * its FP32 values; dx and dw:
 * FLOAT or BFLOAT16 independently; dx, dw and dbias are each optional, one at least is
 * wanted. */
dlcStatus_t dlcCrossEntropyBackward(dlcHandle_t handle, dlcTensorDescriptor_t xDesc, const void *x,
                                    dlcFilterDescriptor_t wDesc, const void *w, const float *bias,
                                    dlcIndexType_t indexType, const void *target, const float *lse,
                                    const float *dloss, dlcTensorDescriptor_t dxDesc, void *dx,
                                    dlcFilterDescriptor_t dwDesc, void *dw, float *dbias,
                                    void *workspace, size_t workspaceBytes);

/* Workspace for any subset of the three gradients. */
dlcStatus_t dlcGetCrossEntropyBackwardWorkspaceSize(dlcHandle_t handle, dlcTensorDescriptor_t xDesc,
                                                    const void *x, dlcFilterDescriptor_t wDesc,
                                                    const void *w, size_t *bytes);

/* ---- self test of the device error path ---------------------------------- */

/* Launches one block whose pipeline wait is on a barrier nothing completes,
 * with a limit of timeout_us microseconds (1..1000000).  The kernel records
 * DLC_DEVERR_WAIT_TIMEOUT and returns; no GPU fault is involved.  Used by the
 * tests of the error path.  No counterpart on the pages. */
dlcStatus_t dlcDebugWaitTimeoutSelfTest(dlcHandle_t handle, int timeout_us);

/* ---- forward convolution that allocates nothing ---------------------------
 *
 * No counterpart on the pages: this is a service for callers that may not
 * allocate memory after start-up -- for example a serving process whose
 * memory is reserved once at start-up, or a plug-in inside a framework that
 * owns all device memory through its own allocator.  Such callers cannot
 * create a handle (dlcCreate allocates its error word, split-tile flags and
 * filter-repacking buffer).
 *
 * dlcConvolutionForwardNoAlloc computes y = alpha * conv(x, w) + beta * y like
 * dlcConvolutionForward, with tensor-core math only (TF32 or BF16; FP32 math
 * returns NOT_SUPPORTED), launched on `stream` (a cudaStream_t as void*,
 * NULL = legacy default stream) of the current device.  It allocates no host
 * or device memory and calls no allocating routine.  Besides x, w, y and
 * `status` it uses only fixed scratch arrays compiled into the library
 * (DLC_NOALLOC_MAX_TILES split-tile flags and two error words, and 256 KiB
 * where the few-channel kernel repacks the filters); every GPU that loads the
 * library holds those arrays until the process exits.
 *
 * It launches the same kernels as dlcConvolutionForward would for the
 * problem (each CTA pair or CTA works on whole output tiles or on an
 * independent part of one; no CTA waits on another CTA of the launch, so
 * other work running on the GPU at the same time cannot stall it), with the
 * few-channel kernel's repacked filters in the fixed array.  The
 * DLC_NOALLOC_MAX_TILES flags serve only the opt-in stream-K schedule
 * (environment DLC_TC_STREAMK=1), whose CTAs do wait on one another and need
 * them all resident; problems with more tiles than flags run whole tiles.
 *
 * The first call on a device sets that device up: it looks up the scratch
 * arrays' device addresses and the tensor-map encoders, and loads every
 * kernel of the library into the context (CUDA loads modules lazily, and a
 * module load allocates device memory), so later calls load nothing.  Make
 * that first call before any stream capture.  A device reset
 * (cudaDeviceReset) invalidates the set-up: calls after one are not
 * supported.  Every call reuses the same scratch arrays and clears its flags
 * on `stream` before launching, so calls whose work overlaps on the GPU (other
 * streams, other host threads) race with each other: issue them one at a
 * time.
 *
 * status: NULL, or a device-accessible array of two ints owned by the caller;
 *   the call zeroes it on `stream`, and a kernel that gives up on a pipeline
 *   wait writes dlcDeviceError_t code and detail there.  With NULL such an
 *   error goes to the scratch array and is not reported.
 * Errors: BAD_PARAM / NOT_SUPPORTED as for dlcConvolutionForward, plus the
 * above; EXECUTION_FAILED if the set-up or the launch fails.
 */
#define DLC_NOALLOC_MAX_TILES 4096

dlcStatus_t dlcConvolutionForwardNoAlloc(void *stream, const float *alpha,
                                         dlcTensorDescriptor_t xDesc, const void *x,
                                         dlcFilterDescriptor_t wDesc, const void *w,
                                         dlcConvolutionDescriptor_t conv, const float *beta,
                                         dlcTensorDescriptor_t yDesc, void *y, int *status);

#ifdef __cplusplus
}
#endif

#endif /* DLC_H_ */

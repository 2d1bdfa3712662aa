"""Descriptor marshalling for torch tensors on top of the C ABI.

Only argument marshalling: descriptor values and device pointers are read
from torch tensors and passed to the C functions in :mod:`binding`; the
convolution itself runs in ``libdlc.so``.

Axis strings name the logical meaning of a tensor's dimensions: activations
use a permutation of ``"NCHW"`` (``"NHWC"`` for channels-last storage),
filters ``"KCRS"`` or ``"KRSC"``.  Any torch strides are passed through, so
views (sub-tensors, padded rows) work where the kernel supports them.
"""
from __future__ import annotations

from typing import Optional, Sequence

from . import binding as B

MATH = {"fp32": B.DLC_MATH_FP32, "tf32": B.DLC_MATH_TF32, "bf16": B.DLC_MATH_BF16,
        "fp64": B.DLC_MATH_FP64}
MODE = {"cross_correlation": B.DLC_CROSS_CORRELATION, "convolution": B.DLC_CONVOLUTION}


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return B.DLC_DATA_FLOAT
    if t.dtype == torch.bfloat16:
        return B.DLC_DATA_BFLOAT16
    if t.dtype == torch.float64:
        return B.DLC_DATA_DOUBLE
    if t.dtype == torch.float8_e4m3fn:
        return B.DLC_DATA_FLOAT8_E4M3
    raise TypeError(f"unsupported dtype {t.dtype}")


def _logical(t, axes: str, order: str):
    """(sizes, strides) of tensor t in the logical axis order `order`."""
    if sorted(axes) != sorted(order) or t.dim() != 4:
        raise ValueError(f"axes {axes!r} do not describe a 4-D {order} tensor")
    sizes = [t.shape[axes.index(a)] for a in order]
    strides = [t.stride(axes.index(a)) for a in order]
    return sizes, strides


class Handle:
    """Owns a dlcHandle_t bound to the current device; follows torch's
    current stream unless a stream is given."""

    def __init__(self, stream=None):
        import torch
        self.h = B.dlcCreate()
        self.set_stream(stream if stream is not None else torch.cuda.current_stream())

    def set_stream(self, stream):
        self.stream = int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)
        B.dlcSetStream(self.h, self.stream)

    def synchronize(self):
        B.dlcSynchronize(self.h)

    def set_deterministic(self, on: bool = True):
        B.dlcSetDeterministic(self.h, 1 if on else 0)

    def launches(self) -> int:
        return B.dlcGetLaunchCount(self.h)

    def last_device_error(self):
        return B.dlcGetLastDeviceError(self.h)

    def close(self):
        if self.h is not None:
            B.dlcDestroy(self.h)
            self.h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


class Conv2dForward:
    """Descriptors of one forward-convolution problem built from example
    tensors; calling it launches dlcConvolution(BiasActivation)Forward."""

    def __init__(self, handle: Handle, x, w, y, *, x_axes: str = "NCHW", w_axes: str = "KCRS",
                 y_axes: str = "NCHW", pads: Sequence[int] = (0, 0, 0, 0),
                 stride: Sequence[int] = (1, 1), dilation: Sequence[int] = (1, 1),
                 math: str = "bf16", mode: str = "cross_correlation"):
        self.handle = handle
        self.x_desc = B.dlcCreateTensorDescriptor()
        self.w_desc = B.dlcCreateFilterDescriptor()
        self.y_desc = B.dlcCreateTensorDescriptor()
        self.conv = B.dlcCreateConvolutionDescriptor()
        xs, xst = _logical(x, x_axes, "NCHW")
        B.dlcSetTensor4dDescriptorEx(self.x_desc, _dtype_code(x), *xs, *xst)
        if w_axes == "KCRS":
            fmt = B.DLC_TENSOR_NCHW
        elif w_axes == "KRSC":
            fmt = B.DLC_TENSOR_NHWC
        else:
            raise ValueError("filters must be KCRS or KRSC")
        if not w.is_contiguous():
            raise ValueError("filter tensors must be dense (contiguous)")
        ws, _ = _logical(w, w_axes, "KCRS")
        B.dlcSetFilter4dDescriptor(self.w_desc, _dtype_code(w), fmt, *ws)
        ys, yst = _logical(y, y_axes, "NCHW")
        B.dlcSetTensor4dDescriptorEx(self.y_desc, _dtype_code(y), *ys, *yst)
        B.dlcSetConvolution2dDescriptor(self.conv, 0, 0, int(stride[0]), int(stride[1]),
                                        int(dilation[0]), int(dilation[1]), MATH[math])
        B.dlcSetConvolution2dPadding(self.conv, *[int(p) for p in pads])
        B.dlcSetConvolutionMode(self.conv, MODE[mode])

    def output_dim(self):
        return B.dlcGetConvolution2dForwardOutputDim(self.conv, self.x_desc, self.w_desc)

    def workspace_size(self) -> int:
        return B.dlcGetConvolutionForwardWorkspaceSize(self.handle.h, self.x_desc, self.w_desc,
                                                       self.conv, self.y_desc)

    def kernel(self, x=None, w=None, y=None) -> str:
        k = B.dlcGetConvolutionForwardKernel(
            self.handle.h, self.x_desc, x.data_ptr() if x is not None else 0, self.w_desc,
            w.data_ptr() if w is not None else 0, self.conv, self.y_desc,
            y.data_ptr() if y is not None else 0)
        return B.KERNEL_NAMES[k]

    def __call__(self, x, w, y, alpha: float = 1.0, beta: float = 0.0, bias=None,
                 relu: bool = False):
        if bias is None and not relu:
            B.dlcConvolutionForward(self.handle.h, alpha, self.x_desc, x.data_ptr(), self.w_desc,
                                    w.data_ptr(), self.conv, beta, self.y_desc, y.data_ptr())
        else:
            B.dlcConvolutionBiasActivationForward(
                self.handle.h, alpha, self.x_desc, x.data_ptr(), self.w_desc, w.data_ptr(),
                self.conv, beta, bias.data_ptr() if bias is not None else 0,
                B.DLC_ACTIVATION_RELU if relu else B.DLC_ACTIVATION_IDENTITY, self.y_desc,
                y.data_ptr())
        return y

    def close(self):
        for d, f in ((self.x_desc, B.dlcDestroyTensorDescriptor),
                     (self.y_desc, B.dlcDestroyTensorDescriptor),
                     (self.w_desc, B.dlcDestroyFilterDescriptor),
                     (self.conv, B.dlcDestroyConvolutionDescriptor)):
            if d is not None:
                f(d)
        self.x_desc = self.y_desc = self.w_desc = self.conv = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class _Descriptors:
    """Tensor, filter and convolution descriptors of one problem, in the
    forward problem's terms: activations x [N,C,H,W], filters w [K,C,R,S],
    outputs y [N,K,P,Q] (the backward routines read or write their gradients
    with the same shapes)."""

    def __init__(self, x, w, y, x_axes, w_axes, y_axes, pads, stride, dilation, math, mode):
        self.x_desc = B.dlcCreateTensorDescriptor()
        self.w_desc = B.dlcCreateFilterDescriptor()
        self.y_desc = B.dlcCreateTensorDescriptor()
        self.conv = B.dlcCreateConvolutionDescriptor()
        xs, xst = _logical(x, x_axes, "NCHW")
        B.dlcSetTensor4dDescriptorEx(self.x_desc, _dtype_code(x), *xs, *xst)
        if w_axes not in ("KCRS", "KRSC"):
            raise ValueError("filters must be KCRS or KRSC")
        if not w.is_contiguous():
            raise ValueError("filter tensors must be dense (contiguous)")
        ws, _ = _logical(w, w_axes, "KCRS")
        B.dlcSetFilter4dDescriptor(self.w_desc, _dtype_code(w),
                                   B.DLC_TENSOR_NCHW if w_axes == "KCRS" else B.DLC_TENSOR_NHWC, *ws)
        ys, yst = _logical(y, y_axes, "NCHW")
        B.dlcSetTensor4dDescriptorEx(self.y_desc, _dtype_code(y), *ys, *yst)
        B.dlcSetConvolution2dDescriptor(self.conv, 0, 0, int(stride[0]), int(stride[1]),
                                        int(dilation[0]), int(dilation[1]), MATH[math])
        B.dlcSetConvolution2dPadding(self.conv, *[int(p) for p in pads])
        B.dlcSetConvolutionMode(self.conv, MODE[mode])

    def close(self):
        for d, f in ((self.x_desc, B.dlcDestroyTensorDescriptor),
                     (self.y_desc, B.dlcDestroyTensorDescriptor),
                     (self.w_desc, B.dlcDestroyFilterDescriptor),
                     (self.conv, B.dlcDestroyConvolutionDescriptor)):
            if d is not None:
                f(d)
        self.x_desc = self.y_desc = self.w_desc = self.conv = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Conv2dBackwardData(_Descriptors):
    """dx = alpha * dgrad(w, dy) + beta * dx through dlcConvolutionBackwardData;
    built from example tensors w [K,C,R,S], dy [N,K,P,Q] and dx [N,C,H,W]."""

    def __init__(self, handle: Handle, w, dy, dx, *, w_axes="KCRS", dy_axes="NCHW",
                 dx_axes="NCHW", pads=(0, 0, 0, 0), stride=(1, 1), dilation=(1, 1),
                 math="bf16", mode="cross_correlation"):
        self.handle = handle
        super().__init__(dx, w, dy, dx_axes, w_axes, dy_axes, pads, stride, dilation, math, mode)

    def kernel(self, w=None, dy=None, dx=None) -> str:
        k = B.dlcGetConvolutionBackwardDataKernel(
            self.handle.h, self.w_desc, w.data_ptr() if w is not None else 0, self.y_desc,
            dy.data_ptr() if dy is not None else 0, self.conv, self.x_desc,
            dx.data_ptr() if dx is not None else 0)
        return B.KERNEL_NAMES[k]

    def workspace_size(self) -> int:
        return B.dlcGetConvolutionBackwardDataWorkspaceSize(self.handle.h, self.w_desc, self.y_desc,
                                                            self.conv, self.x_desc)

    def __call__(self, w, dy, dx, alpha: float = 1.0, beta: float = 0.0):
        B.dlcConvolutionBackwardData(self.handle.h, alpha, self.w_desc, w.data_ptr(), self.y_desc,
                                     dy.data_ptr(), self.conv, beta, self.x_desc, dx.data_ptr())
        return dx


class Conv2dBackwardFilter(_Descriptors):
    """dw = alpha * wgrad(x, dy) + beta * dw through dlcConvolutionBackwardFilter;
    built from example tensors x [N,C,H,W], dy [N,K,P,Q] and dw [K,C,R,S]."""

    def __init__(self, handle: Handle, x, dy, dw, *, x_axes="NCHW", dy_axes="NCHW",
                 dw_axes="KCRS", pads=(0, 0, 0, 0), stride=(1, 1), dilation=(1, 1),
                 math="bf16", mode="cross_correlation"):
        self.handle = handle
        super().__init__(x, dw, dy, x_axes, dw_axes, dy_axes, pads, stride, dilation, math, mode)

    def kernel(self, x=None, dy=None, dw=None) -> str:
        k = B.dlcGetConvolutionBackwardFilterKernel(
            self.handle.h, self.x_desc, x.data_ptr() if x is not None else 0, self.y_desc,
            dy.data_ptr() if dy is not None else 0, self.conv, self.w_desc,
            dw.data_ptr() if dw is not None else 0)
        return B.KERNEL_NAMES[k]

    def workspace_size(self) -> int:
        return B.dlcGetConvolutionBackwardFilterWorkspaceSize(self.handle.h, self.x_desc,
                                                              self.y_desc, self.conv, self.w_desc)

    def __call__(self, x, dy, dw, alpha: float = 1.0, beta: float = 0.0):
        B.dlcConvolutionBackwardFilter(self.handle.h, alpha, self.x_desc, x.data_ptr(), self.y_desc,
                                       dy.data_ptr(), self.conv, beta, self.w_desc, dw.data_ptr())
        return dw


POOL_MODES = {"max": B.DLC_POOLING_MAX, "avg_include_pad": B.DLC_POOLING_AVERAGE_COUNT_INCLUDE_PADDING,
              "avg_exclude_pad": B.DLC_POOLING_AVERAGE_COUNT_EXCLUDE_PADDING}
ACT_MODES = {"identity": B.DLC_ACTIVATION_IDENTITY, "relu": B.DLC_ACTIVATION_RELU,
             "sigmoid": B.DLC_ACTIVATION_SIGMOID, "tanh": B.DLC_ACTIVATION_TANH,
             "clipped_relu": B.DLC_ACTIVATION_CLIPPED_RELU}


class Pool2dForward:
    """y = alpha * pool(x) + beta * y through dlcPoolingForward."""

    def __init__(self, handle: Handle, x, y, *, window=(2, 2), mode="max", pads=(0, 0, 0, 0),
                 stride=(2, 2), x_axes="NCHW", y_axes="NCHW"):
        self.handle = handle
        self.pool = B.dlcCreatePoolingDescriptor()
        B.dlcSetPooling2dDescriptor(self.pool, POOL_MODES[mode], window[0], window[1], *pads,
                                    stride[0], stride[1])
        self.x_desc = B.dlcCreateTensorDescriptor()
        self.y_desc = B.dlcCreateTensorDescriptor()
        xs, xst = _logical(x, x_axes, "NCHW")
        B.dlcSetTensor4dDescriptorEx(self.x_desc, _dtype_code(x), *xs, *xst)
        ys, yst = _logical(y, y_axes, "NCHW")
        B.dlcSetTensor4dDescriptorEx(self.y_desc, _dtype_code(y), *ys, *yst)

    def output_dim(self):
        return B.dlcGetPooling2dForwardOutputDim(self.pool, self.x_desc)

    def kernel(self, x=None, y=None) -> str:
        return B.KERNEL_NAMES[B.dlcGetPoolingForwardKernel(
            self.handle.h, self.pool, self.x_desc, x.data_ptr() if x is not None else 0,
            self.y_desc, y.data_ptr() if y is not None else 0)]

    def __call__(self, x, y, alpha: float = 1.0, beta: float = 0.0):
        B.dlcPoolingForward(self.handle.h, self.pool, alpha, self.x_desc, x.data_ptr(), beta,
                            self.y_desc, y.data_ptr())
        return y

    def close(self):
        if self.pool is not None:
            B.dlcDestroyPoolingDescriptor(self.pool)
            B.dlcDestroyTensorDescriptor(self.x_desc)
            B.dlcDestroyTensorDescriptor(self.y_desc)
            self.pool = None


class ActivationForward:
    """y = alpha * f(x) + beta * y through dlcActivationForward (y may be x),
    with the tensor descriptors built once for repeated calls on the same
    shapes and layouts."""

    def __init__(self, handle: Handle, x, y, *, mode="relu", coef=0.0, x_axes="NCHW",
                 y_axes="NCHW"):
        self.handle = handle
        self.mode = ACT_MODES[mode]
        self.coef = float(coef)
        self.x_desc = B.dlcCreateTensorDescriptor()
        self.y_desc = B.dlcCreateTensorDescriptor()
        xs, xst = _logical(x, x_axes, "NCHW")
        B.dlcSetTensor4dDescriptorEx(self.x_desc, _dtype_code(x), *xs, *xst)
        ys, yst = _logical(y, y_axes, "NCHW")
        B.dlcSetTensor4dDescriptorEx(self.y_desc, _dtype_code(y), *ys, *yst)

    def __call__(self, x, y, alpha: float = 1.0, beta: float = 0.0):
        B.dlcActivationForward(self.handle.h, self.mode, self.coef, alpha, self.x_desc, x.data_ptr(),
                               beta, self.y_desc, y.data_ptr())
        return y

    def close(self):
        if self.x_desc is not None:
            B.dlcDestroyTensorDescriptor(self.x_desc)
            B.dlcDestroyTensorDescriptor(self.y_desc)
            self.x_desc = None


def activation_forward(handle: Handle, x, y, *, mode="relu", coef=0.0, alpha=1.0, beta=0.0,
                       x_axes="NCHW", y_axes="NCHW"):
    """y = alpha * f(x) + beta * y through dlcActivationForward (y may be x):
    one call of ActivationForward, its descriptors built and destroyed here."""
    op = ActivationForward(handle, x, y, mode=mode, coef=coef, x_axes=x_axes, y_axes=y_axes)
    try:
        return op(x, y, alpha=alpha, beta=beta)
    finally:
        op.close()


LINEAR_ACT_MODES = {"identity": B.DLC_ACTIVATION_IDENTITY, "relu": B.DLC_ACTIVATION_RELU,
                    "sigmoid": B.DLC_ACTIVATION_SIGMOID, "tanh": B.DLC_ACTIVATION_TANH,
                    "silu": B.DLC_ACTIVATION_SILU, "gelu": B.DLC_ACTIVATION_GELU}


def _ptr(t) -> int:
    return t.data_ptr() if t is not None else 0


_ABSENT = (None, None, None, None)  # the example of a tensor that an operator was built without


class _ChannelOp:
    """Descriptors and workspace of one channel operator, built once from
    example tensors for repeated calls on the same shapes, strides, types and
    16-byte alignment.  Activations are [rows, channels] matrices or 4-D
    tensors with ``axes`` ("NHWC" or "NCHW"); weights are [K, C] matrices or
    4-D filters with R = S = 1.  A call checks its tensors against the examples
    (shape, strides, type, device; ValueError) and vectors for dense FP32, launches
    on the handle's stream and returns no copies.  An operator has one workspace:
    calls on several streams need an operator each, or an order between them; a
    captured graph needs its operator alive."""

    _name = None  # of the C function

    def __init__(self, handle: Handle, axes: str):
        import torch
        self._fn = B.function(self._name)
        self._f32 = torch.float32
        self.handle = handle
        self.axes = axes
        self.device = None  # the examples' GPU
        self._tensors, self._filters = [], []
        self.workspace, self._ws_ptr, self._ws_bytes = None, 0, 0
        self._ws_stream = None

    def _rows(self, t):
        """(sizes, strides) of an activation tensor as n, c, h, w."""
        if t.dim() == 2:
            (rows, c), (rs, cs) = t.shape, t.stride()
            return (rows, c, 1, 1), (rs, cs, 0, 0)
        return _logical(t, self.axes, "NCHW")

    def _example(self, t):
        """What _at compares a call's tensor with."""
        if not t.is_cuda or (self.device is not None and t.get_device() != self.device):
            raise ValueError("the tensors of an operator are on one GPU")
        self.device = t.get_device()
        return t.shape, None if t.is_contiguous() else t.stride(), t.dtype

    def _act_desc(self, t):
        """Descriptor and example of an activation tensor (None and _ABSENT for none)."""
        if t is None:
            return None, _ABSENT
        sizes, strides = self._rows(t)
        example = self._example(t) + ([(n, n > 1 and s) for n, s in zip(sizes, strides)],)
        d = B.dlcCreateTensorDescriptor()
        self._tensors.append(d)
        B.dlcSetTensor4dDescriptorEx(d, _dtype_code(t), *sizes, *strides)
        return d, example

    def _weight_desc(self, t):
        """The same of a filter tensor."""
        if t is None:
            return None, _ABSENT
        if not t.is_contiguous():
            raise ValueError("filter tensors must be dense (contiguous)")
        if t.dim() not in (2, 4) or (t.dim() == 4 and t.numel() != t.shape[0] * max(t.shape[1:])):
            raise ValueError("weights are [K, C] or filters with R = S = 1")
        example = self._example(t) + (None,)
        d = B.dlcCreateFilterDescriptor()
        self._filters.append(d)
        B.dlcSetFilter4dDescriptor(d, _dtype_code(t), B.DLC_TENSOR_NCHW, t.shape[0],
                                   t.numel() // t.shape[0], 1, 1)
        return d, example

    def _at(self, t, example, what: str) -> int:
        """Pointer of a call's tensor, laid out like its example."""
        shape, strides, dtype, _ = example
        if (t.shape != shape or t.dtype is not dtype or t.get_device() != self.device
                or not (t.is_contiguous() if strides is None else t.stride() == strides)):
            self._same_elements(t, example, what)
        return t.data_ptr()

    def _same_elements(self, t, example, what: str):
        """ValueError unless t's descriptor would be that of its example (other dimensions,
        or strides of dimensions of one element)."""
        shape, strides, dtype, rows = example
        if example is _ABSENT:
            raise ValueError(f"{what} was not among the example tensors")
        same = t.dtype is dtype and t.get_device() == self.device
        if same and rows is None:
            same = t.is_contiguous() and t.shape[:1] == shape[:1] and t.numel() == shape.numel()
        elif same:
            same = t.dim() in (2, 4) and [(n, n > 1 and s) for n, s in zip(*self._rows(t))] == rows
        if not same:
            raise ValueError(f"{what} is {tuple(t.shape)} {t.dtype} with strides {t.stride()} on {t.device}, "
                             f"its example {tuple(shape)} {dtype} with strides {strides or 'of a dense one'}")

    def _set_workspace(self, nbytes: int, device):
        """Memory of the handle's stream, not of torch's current one, whose kernels
        might still write what it released last."""
        import torch
        self._ws_bytes = nbytes
        self._ws_stream = self.handle.stream
        if nbytes:
            with torch.cuda.stream(torch.cuda.ExternalStream(self._ws_stream, device=device)):
                self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
            self._ws_ptr = self.workspace.data_ptr()

    def _scratch(self) -> int:
        """The workspace's pointer for a call; a stream it comes to keeps it from being
        handed out before the kernels there are done."""
        if self._ws_stream != self.handle.stream:
            self._ws_stream = self.handle.stream
            if self.workspace is not None:
                import torch
                self.workspace.record_stream(
                    torch.cuda.ExternalStream(self._ws_stream, device=self.workspace.device))
        return self._ws_ptr

    def _vector(self, t, n: int, what: str) -> int:
        """Pointer of a dense FP32 vector of n elements."""
        if t.dtype is not self._f32 or t.numel() != n or not t.is_contiguous() or t.get_device() != self.device:
            raise ValueError(f"{what} must be a dense float32 vector of {n} elements on GPU {self.device}")
        return t.data_ptr()

    def close(self):
        for d in self._tensors:
            B.dlcDestroyTensorDescriptor(d)
        for d in self._filters:
            B.dlcDestroyFilterDescriptor(d)
        self._tensors, self._filters = [], []
        for name in [n for n in vars(self) if n.endswith("_desc")]:
            setattr(self, name, None)  # a call after this is refused by the library
        self.workspace, self._ws_ptr, self._ws_bytes = None, 0, 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class RmsNormForward(_ChannelOp):
    """total = x + residual; y = gamma * total / rms(total) through
    dlcRmsNormForward; an E4M3 y comes with one scale per row."""
    _name = "dlcRmsNormForward"

    def __init__(self, handle: Handle, x, y, *, residual=None, total=None, eps: float = 1e-6,
                 axes: str = "NHWC"):
        super().__init__(handle, axes)
        self.eps = float(eps)
        self.x_desc, self._x = self._act_desc(x)
        self.y_desc, self._y = self._act_desc(y)
        self.r_desc, self._r = self._act_desc(residual)
        self.t_desc, self._t = self._act_desc(total)
        self.channels = B.dlcGetTensor4dDescriptor(self.x_desc)[2]
        self.rows = x.numel() // self.channels

    def __call__(self, x, gamma, y, residual=None, total=None, scale=None):
        status = self._fn(self.handle.h, self.eps, self.x_desc, self._at(x, self._x, "x"),
                          self.r_desc, residual if residual is None else
                          self._at(residual, self._r, "residual"), self._vector(gamma, self.channels, "gamma"),
                          self.t_desc, total if total is None else self._at(total, self._t, "total"),
                          self.y_desc, self._at(y, self._y, "y"),
                          scale if scale is None else self._vector(scale, self.rows, "scale"))
        if status:
            B.check(self._name, status)
        return y


class RmsNormBackward(_ChannelOp):
    """dx (the gradient of x and of the residual) and dgamma of RmsNormForward
    through dlcRmsNormBackward; dtotal is the gradient that reaches the sum by
    other ways."""
    _name = "dlcRmsNormBackward"

    def __init__(self, handle: Handle, dy, total, dx, *, dtotal=None, eps: float = 1e-6,
                 axes: str = "NHWC"):
        super().__init__(handle, axes)
        self.eps = float(eps)
        self.dy_desc, self._dy = self._act_desc(dy)
        self.t_desc, self._t = self._act_desc(total)
        self.dx_desc, self._dx = self._act_desc(dx)
        self.dt_desc, self._dt = self._act_desc(dtotal)
        self.channels = B.dlcGetTensor4dDescriptor(self.t_desc)[2]
        self._set_workspace(B.dlcGetRmsNormBackwardWorkspaceSize(handle.h, self.t_desc), total.device)

    def __call__(self, dy, total, gamma, dx, dgamma=None, dtotal=None):
        status = self._fn(self.handle.h, self.eps, self.dy_desc, self._at(dy, self._dy, "dy"),
                          self.t_desc, self._at(total, self._t, "total"),
                          self._vector(gamma, self.channels, "gamma"),
                          self.dt_desc, dtotal if dtotal is None else self._at(dtotal, self._dt, "dtotal"),
                          self.dx_desc, self._at(dx, self._dx, "dx"),
                          dgamma if dgamma is None else self._vector(dgamma, self.channels, "dgamma"),
                          self._scratch(), self._ws_bytes)
        if status:
            B.check(self._name, status)
        return dx


class _Product(_ChannelOp):
    _workspace = _kernel_of = None

    def __init__(self, handle, x, w, y, act, residual, z, axes):
        super().__init__(handle, axes)
        self.act = LINEAR_ACT_MODES[act]
        self.x_desc, self._x = self._act_desc(x)
        self.w_desc, self._w = self._weight_desc(w)
        self.y_desc, self._y = self._act_desc(y)
        self.r_desc, self._r = self._act_desc(residual)
        self.z_desc, self._z = self._act_desc(z)
        self.filters = w.shape[0]
        self.rows = x.numel() // (w.numel() // w.shape[0])
        self._set_workspace(self._workspace(handle.h, self.x_desc, x.data_ptr(), self.w_desc,
                                            w.data_ptr(), self.y_desc, y.data_ptr()), x.device)

    def kernel(self, x=None, w=None, y=None) -> str:
        return B.KERNEL_NAMES[self._kernel_of(self.handle.h, self.x_desc, _ptr(x), self.w_desc,
                                              _ptr(w), self.y_desc, _ptr(y))]


class LinearForward(_Product):
    """y = act(x w^T + bias) + residual through dlcLinearForward, w being
    [K, C]; E4M3 x and w take one scale per row and per filter.  z, where
    given, receives the activation's argument for LinearBackward."""
    _name = "dlcLinearForward"
    _workspace = staticmethod(B.dlcGetLinearForwardWorkspaceSize)
    _kernel_of = staticmethod(B.dlcGetLinearForwardKernel)

    def __init__(self, handle: Handle, x, w, y, *, act: str = "identity", residual=None, z=None,
                 axes: str = "NHWC"):
        super().__init__(handle, x, w, y, act, residual, z, axes)

    def __call__(self, x, w, y, bias=None, residual=None, z=None, x_scale=None, w_scale=None):
        status = self._fn(self.handle.h, self.x_desc, self._at(x, self._x, "x"),
                          x_scale if x_scale is None else self._vector(x_scale, self.rows, "x_scale"),
                          self.w_desc, self._at(w, self._w, "w"),
                          w_scale if w_scale is None else self._vector(w_scale, self.filters, "w_scale"),
                          bias if bias is None else self._vector(bias, self.filters, "bias"), self.act,
                          self.z_desc, z if z is None else self._at(z, self._z, "z"),
                          self.r_desc, residual if residual is None else
                          self._at(residual, self._r, "residual"),
                          self.y_desc, self._at(y, self._y, "y"), self._scratch(), self._ws_bytes)
        if status:
            B.check(self._name, status)
        return y


class GatedForward(_Product):
    """y = act(gate) * up through dlcGatedForward: w is [2F, C], F gate filters
    and then F up filters, z = [gate, up] = x w^T + bias."""
    _name = "dlcGatedForward"
    _workspace = staticmethod(B.dlcGetGatedForwardWorkspaceSize)
    _kernel_of = staticmethod(B.dlcGetGatedForwardKernel)

    def __init__(self, handle: Handle, x, w, y, *, act: str = "silu", z=None, axes: str = "NHWC"):
        super().__init__(handle, x, w, y, act, None, z, axes)

    def __call__(self, x, w, y, bias=None, z=None, x_scale=None, w_scale=None):
        status = self._fn(self.handle.h, self.x_desc, self._at(x, self._x, "x"),
                          x_scale if x_scale is None else self._vector(x_scale, self.rows, "x_scale"),
                          self.w_desc, self._at(w, self._w, "w"),
                          w_scale if w_scale is None else self._vector(w_scale, self.filters, "w_scale"),
                          bias if bias is None else self._vector(bias, self.filters, "bias"), self.act,
                          self.z_desc, z if z is None else self._at(z, self._z, "z"),
                          self.y_desc, self._at(y, self._y, "y"), self._scratch(), self._ws_bytes)
        if status:
            B.check(self._name, status)
        return y


class _ProductBackward(_ChannelOp):
    _workspace = None

    def __init__(self, handle, x, w, dy, dx, dw, z, act, axes):
        super().__init__(handle, axes)
        self.act = LINEAR_ACT_MODES[act]
        self.x_desc, self._x = self._act_desc(x)
        self.w_desc, self._w = self._weight_desc(w)
        self.dy_desc, self._dy = self._act_desc(dy)
        self.dx_desc, self._dx = self._act_desc(dx)
        self.dw_desc, self._dw = self._weight_desc(dw)
        self.z_desc, self._z = self._act_desc(z)
        self.filters = w.shape[0]
        self._set_workspace(self._workspace(handle.h, self.x_desc, x.data_ptr(), self.w_desc,
                                            w.data_ptr(), self.act, self.z_desc, self.dy_desc,
                                            dy.data_ptr()), x.device)

    def __call__(self, x, w, dy, dx=None, dw=None, dbias=None, z=None):
        status = self._fn(self.handle.h, self.x_desc, self._at(x, self._x, "x"), self.w_desc,
                          self._at(w, self._w, "w"), self.act,
                          self.z_desc, z if z is None else self._at(z, self._z, "z"),
                          self.dy_desc, self._at(dy, self._dy, "dy"),
                          self.dx_desc, dx if dx is None else self._at(dx, self._dx, "dx"),
                          self.dw_desc, dw if dw is None else self._at(dw, self._dw, "dw"),
                          dbias if dbias is None else self._vector(dbias, self.filters, "dbias"),
                          self._scratch(), self._ws_bytes)
        if status:
            B.check(self._name, status)
        return dx, dw, dbias


class LinearBackward(_ProductBackward):
    """dx, dw and dbias of LinearForward through dlcLinearBackward, each where
    its tensor is given; z is what the forward call wrote (not needed for the
    identity).  The residual's gradient is dy."""
    _name = "dlcLinearBackward"
    _workspace = staticmethod(B.dlcGetLinearBackwardWorkspaceSize)

    def __init__(self, handle: Handle, x, w, dy, dx=None, dw=None, *, z=None, act: str = "identity",
                 axes: str = "NHWC"):
        super().__init__(handle, x, w, dy, dx, dw, z, act, axes)


class GatedBackward(_ProductBackward):
    """dx, dw and dbias of GatedForward through dlcGatedBackward."""
    _name = "dlcGatedBackward"
    _workspace = staticmethod(B.dlcGetGatedBackwardWorkspaceSize)

    def __init__(self, handle: Handle, x, w, dy, dx=None, dw=None, *, z=None, act: str = "silu",
                 axes: str = "NHWC"):
        super().__init__(handle, x, w, dy, dx, dw, z, act, axes)


def output_dim(x, w, *, x_axes="NCHW", w_axes="KCRS", pads=(0, 0, 0, 0), stride=(1, 1),
               dilation=(1, 1)):
    """(N, K, P, Q) from the library's descriptor call (no GPU work)."""
    xd = B.dlcCreateTensorDescriptor()
    wd = B.dlcCreateFilterDescriptor()
    cd = B.dlcCreateConvolutionDescriptor()
    try:
        xs, xst = _logical(x, x_axes, "NCHW")
        B.dlcSetTensor4dDescriptorEx(xd, _dtype_code(x), *xs, *xst)
        ws, _ = _logical(w, w_axes, "KCRS")
        B.dlcSetFilter4dDescriptor(wd, _dtype_code(w),
                                   B.DLC_TENSOR_NCHW if w_axes == "KCRS" else B.DLC_TENSOR_NHWC, *ws)
        B.dlcSetConvolution2dDescriptor(cd, 0, 0, int(stride[0]), int(stride[1]),
                                        int(dilation[0]), int(dilation[1]), B.DLC_MATH_FP32)
        B.dlcSetConvolution2dPadding(cd, *[int(p) for p in pads])
        return B.dlcGetConvolution2dForwardOutputDim(cd, xd, wd)
    finally:
        B.dlcDestroyTensorDescriptor(xd)
        B.dlcDestroyFilterDescriptor(wd)
        B.dlcDestroyConvolutionDescriptor(cd)


def layer_axes(layer):
    """(x_axes, w_axes) of a synth.Layer's storage layout."""
    return ("NHWC", "KRSC") if layer.layout == "NHWC" else ("NCHW", "KCRS")


def layer_tensors(layer, x_nchw, w_kcrs, device):
    """Device tensors x and w for a synth.Layer from logical-NCHW / KCRS numpy
    arrays (already rounded), stored in the layer's layout (dense)."""
    import numpy as np
    import torch
    from . import synth
    if layer.dtype == "bf16":
        xb = synth.round_to_bf16_bits(x_nchw).view(np.int16).reshape(x_nchw.shape)
        wb = synth.round_to_bf16_bits(w_kcrs).view(np.int16).reshape(w_kcrs.shape)
        xt = torch.from_numpy(xb).view(torch.bfloat16)
        wt = torch.from_numpy(wb).view(torch.bfloat16)
    else:
        xt = torch.from_numpy(np.ascontiguousarray(x_nchw, dtype=np.float32))
        wt = torch.from_numpy(np.ascontiguousarray(w_kcrs, dtype=np.float32))
    if layer.layout == "NHWC":
        xt = xt.permute(0, 2, 3, 1)
        wt = wt.permute(0, 2, 3, 1)
    return xt.contiguous().to(device), wt.contiguous().to(device)


def layer_problem(handle, layer, xt, wt, y_dtype=None, y_axes=None):
    """A Conv2dForward for a synth.Layer plus its freshly allocated y
    (FP32 by default, in the layer's layout unless y_axes is given)."""
    import torch
    x_axes, w_axes = layer_axes(layer)
    pads = (layer.pad_top, layer.pad_bottom, layer.pad_left, layer.pad_right)
    stride, dil = (layer.u, layer.v), (layer.dil_h, layer.dil_w)
    n, k, p, q = output_dim(xt, wt, x_axes=x_axes, w_axes=w_axes, pads=pads, stride=stride,
                            dilation=dil)
    y_axes = y_axes or x_axes
    shape = [dict(N=n, C=k, H=p, W=q)[a] for a in y_axes]
    y = torch.empty(shape, dtype=y_dtype or torch.float32, device=xt.device)
    conv = Conv2dForward(handle, xt, wt, y, x_axes=x_axes, w_axes=w_axes, y_axes=y_axes,
                         pads=pads, stride=stride, dilation=dil, math=math_of(layer))
    return conv, y


def math_of(layer) -> str:
    return {"bf16": "bf16", "tf32": "tf32", "f32": "fp32"}[layer.dtype]

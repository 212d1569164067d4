"""Channel operators of libint8conv.so: the matrix product with bias,
activation and residual (``conv_linear``), the layer norm
(``conv_layer_norm``) and their gradients, on matrices of rows (pixels of a
channels-last image, or tokens) by channels.

Argument marshalling only, like the convolution binding: every step runs in
the library's CUDA kernels, on torch tensors of any strides.  Outputs that
are not given are allocated; a workspace that is not given (or is too small)
is allocated for the call, on the stream the call runs on.
"""
from __future__ import annotations

import ctypes
import math

CONV_FLOAT32, CONV_FLOAT16, CONV_BFLOAT16 = 3, 4, 5
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = 0, 1, 2, 3, 4
ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH, "silu": ACT_SILU}

CHANNEL_SYMBOLS = (
    "conv_linear_workspace_size", "conv_linear", "conv_linear_grad_workspace_size", "conv_linear_grad",
    "conv_layer_norm", "conv_layer_norm_grad_workspace_size", "conv_layer_norm_grad",
)


class MatrixDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("row_stride", ctypes.c_int64), ("col_stride", ctypes.c_int64),
                ("capacity_bytes", ctypes.c_uint64)]


class LinearParams(ctypes.Structure):
    _fields_ = [("activation", ctypes.c_int32), ("bias_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32 * 2)]


class LayerNormParams(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_float), ("scale", ctypes.c_float), ("param_dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


def declare(L) -> None:
    """Argument types of the channel entry points of a loaded library."""
    v, sz = ctypes.c_void_p, ctypes.c_size_t
    # descriptors and parameters are passed with byref, absent ones as None
    for name, args in (
            ("conv_linear_workspace_size", [v, v, v, v, v]),
            ("conv_linear", [v, v, v, v, v, v, v, v, v, v, v, v, v, sz, v]),
            ("conv_linear_grad_workspace_size", [v, v, v, v, v, v, v, v]),
            ("conv_linear_grad", [v, v, v, v, v, v, v, v, v, v, v, v, v, v, v, sz, v]),
            ("conv_layer_norm", [v, v, v, v, v, v, v, v, v, v]),
            ("conv_layer_norm_grad_workspace_size", [v, v]),
            ("conv_layer_norm_grad", [v, v, v, v, v, v, v, v, v, v, v, v, v, v, v, sz, v])):
        f = getattr(L, name)
        f.argtypes = args
        f.restype = ctypes.c_int


_SIZES = None


def _types():
    global _SIZES
    if _SIZES is None:
        import torch
        _SIZES = {torch.int8: (1, 1), torch.int32: (2, 4), torch.float32: (CONV_FLOAT32, 4),
                  torch.float16: (CONV_FLOAT16, 2), torch.bfloat16: (CONV_BFLOAT16, 2)}
    return _SIZES


def _matrix(t, what: str):
    """Descriptor of a CUDA tensor [..., C] as a matrix of its leading dims by
    C.  The leading dims have to be walkable with one stride (a view is
    taken, nothing is copied)."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    code, size = _types().get(t.dtype, (0, 1))
    shape = t.shape
    if len(shape) != 2:
        if len(shape) == 0:
            raise ValueError(f"{what} must have at least one dimension")
        try:
            t = t.view(math.prod(shape[:-1]), shape[-1])
        except RuntimeError as e:
            raise ValueError(f"{what}: leading dimensions without a common stride; make it contiguous") from e
        shape = t.shape
    rows, cols = shape
    rs, cs = t.stride()
    # (a torch tensor always lies inside its storage: the capacity is its own extent)
    last = (rows - 1) * rs + (cols - 1) * cs + 1 if rows and cols else 0
    return MatrixDesc(code, 0, rows, cols, rs, cs, last * size)


def _vector(t, n: int, what: str):
    if t is None:
        return None
    if not t.is_cuda or t.dim() != 1 or t.shape[0] != n or not (t.is_contiguous() or n <= 1):
        raise ValueError(f"{what} must be a contiguous CUDA vector of {n} elements")
    return t.data_ptr()


def _stats(t, n: int, what: str):
    import torch
    if t is not None and t.dtype != torch.float32:
        raise ValueError(f"{what} must be float32")
    return _vector(t, n, what)


def _activation(a) -> int:
    if isinstance(a, str):
        if a not in ACTIVATIONS:
            raise ValueError(f"unknown activation {a!r}: one of {', '.join(ACTIVATIONS)}")
        return ACTIVATIONS[a]
    return int(a)


class _Call:
    """Where a call's memory comes from: the stream it runs on."""

    def __init__(self, device, stream):
        import torch
        self.torch, self.device, self.given = torch, device, stream is not None
        self.stream = stream if self.given else torch.cuda.current_stream(device)

    def empty(self, shape, dtype):
        # memory that is first used on the call's stream belongs to it, so
        # that the allocator hands it out again only behind the call
        if self.given:
            with self.torch.cuda.stream(self.stream):
                return self.torch.empty(shape, dtype=dtype, device=self.device)
        return self.torch.empty(shape, dtype=dtype, device=self.device)

    def workspace(self, need: int, given):
        if need == 0:
            return None, 0
        if given is None or given.numel() * given.element_size() < need:
            given = self.empty((need,), self.torch.uint8)
        return given, given.numel() * given.element_size()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(status: int, size, what: str) -> int:
    from . import _check
    _check(status, what)
    return int(size.value)


def conv_linear(x, w, bias=None, *, activation=ACT_NONE, residual=None, preact=None, out=None, workspace=None,
                stream=None):
    """y = act(x w^T + bias) + residual on the GPU.

    x: float16 or bfloat16 CUDA tensor [..., K] with any strides; w: [N, K] of
    x's type (a transposed view is fine); bias: optional [N], float32 or x's
    type; activation: an ACT_* code or its name; residual: optional
    [..., N] of the output's type; preact: optional tensor [..., N] of x's
    type that receives x w^T + bias (what conv_linear_grad wants); out:
    optional [..., N], x's type or float32 (default: x's type, contiguous;
    ``residual`` itself may be given).  Sums are in 32 bits.  Runs on
    ``stream`` (default: the current one).  Returns ``out``.
    """
    from . import _check, lib
    L = lib()
    c = _Call(x.device, stream)
    xd, wd = _matrix(x, "x"), _matrix(w, "w")
    if out is None:
        out = c.empty((*x.shape[:-1], wd.rows), x.dtype)
    yd = _matrix(out, "out")
    rd = None if residual is None else _matrix(residual, "residual")
    zd = None if preact is None else _matrix(preact, "preact")
    code = 0 if bias is None else _types().get(bias.dtype, (0, 1))[0]
    p = LinearParams(_activation(activation), code)
    ref = ctypes.byref
    xp, wp = x.data_ptr(), w.data_ptr()
    size = ctypes.c_size_t()
    need = _need(L.conv_linear_workspace_size(ref(xd), xp, ref(wd), wp, ref(size)), size, "linear workspace size")
    ws, have = c.workspace(need, workspace)
    _check(L.conv_linear(ref(xd), xp, ref(wd), wp, _vector(bias, wd.rows, "bias"), rd and ref(rd), _ptr(residual),
                         zd and ref(zd), _ptr(preact), ref(yd), out.data_ptr(), ref(p), _ptr(ws), have,
                         c.stream.cuda_stream), "conv_linear")
    return out


def conv_linear_grad(dy, x, w, *, preact=None, activation=ACT_NONE, dx=None, dw=None, dbias=None, workspace=None,
                     stream=None):
    """Gradients of conv_linear: fills those of dx [..., K], dw [N, K] (each
    of x's type or float32) and dbias [N] (float32 or x's type) that are
    given.  dy [..., N] is the loss gradient, preact the pre-activation of
    the forward call (needed with an activation); the residual's gradient is
    dy itself.  Returns (dx, dw, dbias)."""
    from . import _check, lib
    L = lib()
    c = _Call(x.device, stream)
    gd, xd, wd = _matrix(dy, "dy"), _matrix(x, "x"), _matrix(w, "w")
    zd = None if preact is None else _matrix(preact, "preact")
    dxd = None if dx is None else _matrix(dx, "dx")
    dwd = None if dw is None else _matrix(dw, "dw")
    code = 0 if dbias is None else _types().get(dbias.dtype, (0, 1))[0]
    p = LinearParams(_activation(activation), code)
    ref = ctypes.byref
    gp, xp, wp = dy.data_ptr(), x.data_ptr(), w.data_ptr()
    size = ctypes.c_size_t()
    need = _need(L.conv_linear_grad_workspace_size(ref(gd), gp, ref(xd), xp, ref(wd), wp, ref(p), ref(size)), size,
                 "linear gradient workspace size")
    ws, have = c.workspace(need, workspace)
    _check(L.conv_linear_grad(ref(gd), gp, ref(xd), xp, ref(wd), wp, zd and ref(zd), _ptr(preact), dxd and ref(dxd),
                              _ptr(dx), dwd and ref(dwd), _ptr(dw), _vector(dbias, wd.rows, "dbias"), ref(p),
                              _ptr(ws), have, c.stream.cuda_stream), "conv_linear_grad")
    return dx, dw, dbias


def conv_layer_norm(x, gain=None, shift=None, *, eps: float = 1e-5, scale: float = 1.0, out=None, mean=None,
                    rstd=None, stream=None):
    """Layer norm over the last dimension of x [..., C] (float32, float16,
    bfloat16, or int32 accumulators of conv_fprop taken as ``scale * x``).

    gain, shift: optional [C], both float32 or both of the output's type;
    out: optional [..., C], float32, float16 or bfloat16 (default: x's type;
    float32 for int32); mean, rstd: optional float32 vectors with one element
    per row that receive the statistics (what conv_layer_norm_grad wants).
    Returns ``out``."""
    from . import _check, lib
    L = lib()
    c = _Call(x.device, stream)
    xd = _matrix(x, "x")
    if out is None:
        out = c.empty(x.shape, x.dtype if x.dtype.is_floating_point else c.torch.float32)
    yd = _matrix(out, "out")
    p = LayerNormParams(eps, scale, _param_dtype(gain, shift), 0)
    ref = ctypes.byref
    _check(L.conv_layer_norm(ref(xd), x.data_ptr(), _vector(gain, xd.cols, "gain"), _vector(shift, xd.cols, "shift"),
                             ref(yd), out.data_ptr(), _stats(mean, xd.rows, "mean"), _stats(rstd, xd.rows, "rstd"),
                             ref(p), c.stream.cuda_stream), "conv_layer_norm")
    return out


def conv_layer_norm_grad(dy, x, gain, mean, rstd, *, residual_grad=None, dx=None, dgain=None, dshift=None,
                         workspace=None, stream=None):
    """Gradients of conv_layer_norm for the loss gradient dy [..., C] (x's
    type), with the statistics of the forward call: fills those of
    dx [..., C] (x's type; residual_grad is added to it), dgain and dshift
    [C] (float32 or x's type, gain's type when gain is given) that are
    given.  Returns (dx, dgain, dshift)."""
    from . import _check, lib
    L = lib()
    c = _Call(x.device, stream)
    gd, xd = _matrix(dy, "dy"), _matrix(x, "x")
    rd = None if residual_grad is None else _matrix(residual_grad, "residual_grad")
    dxd = None if dx is None else _matrix(dx, "dx")
    p = LayerNormParams(1e-5, 1.0, _param_dtype(gain, dgain, dshift), 0)
    ref = ctypes.byref
    size = ctypes.c_size_t()
    need = _need(L.conv_layer_norm_grad_workspace_size(ref(xd), ref(size)), size, "layer norm gradient workspace size")
    ws, have = c.workspace(need, workspace)
    _check(L.conv_layer_norm_grad(ref(gd), dy.data_ptr(), ref(xd), x.data_ptr(), _vector(gain, xd.cols, "gain"),
                                  _stats(mean, xd.rows, "mean"), _stats(rstd, xd.rows, "rstd"), rd and ref(rd),
                                  _ptr(residual_grad), dxd and ref(dxd), _ptr(dx), _vector(dgain, xd.cols, "dgain"),
                                  _vector(dshift, xd.cols, "dshift"), ref(p), _ptr(ws), have, c.stream.cuda_stream),
           "conv_layer_norm_grad")
    return dx, dgain, dshift


def _param_dtype(*tensors) -> int:
    codes = {_types().get(t.dtype, (0, 1))[0] for t in tensors if t is not None}
    if len(codes) > 1:
        raise ValueError("gain, shift and their gradients must have one type")
    return codes.pop() if codes else CONV_FLOAT32

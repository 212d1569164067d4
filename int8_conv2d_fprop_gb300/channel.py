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
from ctypes import byref as _byref

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


_lib = None        # the loaded library, its types declared
_torch = None
_types = {}        # torch dtype -> (code, element size)
_raw_stream = None  # device index -> address of its current stream
_WORKSPACE = 13    # CONV_ERR_WORKSPACE


def _load():
    global _lib, _torch, _raw_stream
    import torch

    from . import lib
    _torch = torch
    _types.update({torch.int8: (1, 1), torch.int32: (2, 4), torch.float32: (CONV_FLOAT32, 4),
                   torch.float16: (CONV_FLOAT16, 2), torch.bfloat16: (CONV_BFLOAT16, 2)})
    # the address alone costs a small part of a torch.cuda.Stream object
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)
    _lib = lib()
    return _lib


def _failed(status: int, what: str):
    from . import ConvError
    raise ConvError(status, what)


def _matrix(t, what: str):
    """Descriptor of a CUDA tensor [..., C] as a matrix of its leading dims by
    C.  The leading dims have to be walkable with one stride (a view is
    taken, nothing is copied)."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    shape = t.shape
    if len(shape) == 2:
        rows, cols = shape
        rs, cs = t.stride()
    else:
        if len(shape) == 0:
            raise ValueError(f"{what} must have at least one dimension")
        try:
            v = t.view(math.prod(shape[:-1]), shape[-1])
        except RuntimeError as e:
            raise ValueError(f"{what}: leading dimensions without a common stride; make it contiguous") from e
        rows, cols = v.shape
        rs, cs = v.stride()
    code, size = _types.get(t.dtype, (0, 1))
    # (a torch tensor always lies inside its storage: the capacity is its own extent)
    return MatrixDesc(code, 0, rows, cols, rs, cs, ((rows - 1) * rs + (cols - 1) * cs + 1) * size if rows and cols else 0)


def _vector(t, n: int, what: str):
    if t is None:
        return None
    shape = t.shape
    if not t.is_cuda or len(shape) != 1 or shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} must be a contiguous CUDA vector of {n} elements")
    return t.data_ptr()


def _stats(t, n: int, what: str):
    if t is None:
        return None
    if t.dtype != _torch.float32:
        raise ValueError(f"{what} must be float32")
    return _vector(t, n, what)


def _activation(a) -> int:
    if isinstance(a, str):
        if a not in ACTIVATIONS:
            raise ValueError(f"unknown activation {a!r}: one of {', '.join(ACTIVATIONS)}")
        return ACTIVATIONS[a]
    return int(a)


def _empty(shape, dtype, device, stream):
    """Memory for a call on `stream` (None: the current one).  Memory that is
    first used on the call's stream belongs to it, so that the allocator
    hands it out again only behind the call."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    with _torch.cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=device)


def _workspace(need: int, given, device, stream):
    """(tensor to keep until the call is queued, address, bytes)"""
    if need == 0:
        return None, None, 0
    if given is None or given.numel() * given.element_size() < need:
        given = _empty((need,), _torch.uint8, device, stream)
    return given, given.data_ptr(), given.numel() * given.element_size()


def _stream(stream, device) -> int:
    return _raw_stream(device.index) if stream is None else stream.cuda_stream


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
    L = _lib or _load()
    xd, wd = _matrix(x, "x"), _matrix(w, "w")
    device = x.device
    if out is None:
        shape = x.shape
        out = _empty((shape[0], wd.rows) if len(shape) == 2 else (*shape[:-1], wd.rows), x.dtype, device, stream)
    yd = _matrix(out, "out")
    rd = zd = rp = zp = bp = None
    code = 0
    if residual is not None:
        rd, rp = _byref(_matrix(residual, "residual")), residual.data_ptr()
    if preact is not None:
        zd, zp = _byref(_matrix(preact, "preact")), preact.data_ptr()
    if bias is not None:
        bp, code = _vector(bias, wd.rows, "bias"), _types.get(bias.dtype, (0, 1))[0]
    p = _byref(LinearParams(_activation(activation), code))
    xp, wp, yp, s = x.data_ptr(), w.data_ptr(), out.data_ptr(), _stream(stream, device)
    xd, wd, yd = _byref(xd), _byref(wd), _byref(yd)
    status = _WORKSPACE
    if workspace is None:
        # most calls need none; one that does is refused before anything runs
        status = L.conv_linear(xd, xp, wd, wp, bp, rd, rp, zd, zp, yd, yp, p, None, 0, s)
    if status == _WORKSPACE:
        size = ctypes.c_size_t()
        status = L.conv_linear_workspace_size(xd, xp, wd, wp, _byref(size))
        if status == 0:
            keep, ws, have = _workspace(size.value, workspace, device, stream)
            status = L.conv_linear(xd, xp, wd, wp, bp, rd, rp, zd, zp, yd, yp, p, ws, have, s)
    if status:
        _failed(status, "conv_linear")
    return out


def conv_linear_grad(dy, x, w, *, preact=None, activation=ACT_NONE, dx=None, dw=None, dbias=None, workspace=None,
                     stream=None):
    """Gradients of conv_linear: fills those of dx [..., K], dw [N, K] (each
    of x's type or float32) and dbias [N] (float32 or x's type) that are
    given.  dy [..., N] is the loss gradient, preact the pre-activation of
    the forward call (needed with an activation); the residual's gradient is
    dy itself.  Returns (dx, dw, dbias)."""
    L = _lib or _load()
    gd, xd, wd = _matrix(dy, "dy"), _matrix(x, "x"), _matrix(w, "w")
    device = x.device
    zd = dxd = dwd = zp = dxp = dwp = dbp = None
    code = 0
    if preact is not None:
        zd, zp = _byref(_matrix(preact, "preact")), preact.data_ptr()
    if dx is not None:
        dxd, dxp = _byref(_matrix(dx, "dx")), dx.data_ptr()
    if dw is not None:
        dwd, dwp = _byref(_matrix(dw, "dw")), dw.data_ptr()
    if dbias is not None:
        dbp, code = _vector(dbias, wd.rows, "dbias"), _types.get(dbias.dtype, (0, 1))[0]
    p = _byref(LinearParams(_activation(activation), code))
    gp, xp, wp, s = dy.data_ptr(), x.data_ptr(), w.data_ptr(), _stream(stream, device)
    gd, xd, wd = _byref(gd), _byref(xd), _byref(wd)
    size = ctypes.c_size_t()
    status = L.conv_linear_grad_workspace_size(gd, gp, xd, xp, wd, wp, p, _byref(size))
    if status == 0:
        keep, ws, have = _workspace(size.value, workspace, device, stream)
        status = L.conv_linear_grad(gd, gp, xd, xp, wd, wp, zd, zp, dxd, dxp, dwd, dwp, dbp, p, ws, have, s)
    if status:
        _failed(status, "conv_linear_grad")
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
    L = _lib or _load()
    xd = _matrix(x, "x")
    device, c, m = x.device, xd.cols, xd.rows
    if out is None:
        out = _empty(x.shape, x.dtype if x.dtype.is_floating_point else _torch.float32, device, stream)
    p = LayerNormParams(eps, scale, _param_dtype(gain, shift), 0)
    status = L.conv_layer_norm(_byref(xd), x.data_ptr(), _vector(gain, c, "gain"), _vector(shift, c, "shift"),
                               _byref(_matrix(out, "out")), out.data_ptr(), _stats(mean, m, "mean"),
                               _stats(rstd, m, "rstd"), _byref(p), _stream(stream, device))
    if status:
        _failed(status, "conv_layer_norm")
    return out


def conv_layer_norm_grad(dy, x, gain, mean, rstd, *, residual_grad=None, dx=None, dgain=None, dshift=None,
                         workspace=None, stream=None):
    """Gradients of conv_layer_norm for the loss gradient dy [..., C] (x's
    type), with the statistics of the forward call: fills those of
    dx [..., C] (x's type; residual_grad is added to it), dgain and dshift
    [C] (float32 or x's type, gain's type when gain is given) that are
    given.  Returns (dx, dgain, dshift)."""
    L = _lib or _load()
    gd, xd = _matrix(dy, "dy"), _matrix(x, "x")
    device, c, m = x.device, xd.cols, xd.rows
    rd = dxd = rp = dxp = None
    if residual_grad is not None:
        rd, rp = _byref(_matrix(residual_grad, "residual_grad")), residual_grad.data_ptr()
    if dx is not None:
        dxd, dxp = _byref(_matrix(dx, "dx")), dx.data_ptr()
    p = LayerNormParams(1e-5, 1.0, _param_dtype(gain, dgain, dshift), 0)
    xd = _byref(xd)
    size = ctypes.c_size_t()
    status = L.conv_layer_norm_grad_workspace_size(xd, _byref(size))
    if status == 0:
        keep, ws, have = _workspace(size.value, workspace, device, stream)
        status = L.conv_layer_norm_grad(_byref(gd), dy.data_ptr(), xd, x.data_ptr(), _vector(gain, c, "gain"),
                                        _stats(mean, m, "mean"), _stats(rstd, m, "rstd"), rd, rp, dxd, dxp,
                                        _vector(dgain, c, "dgain"), _vector(dshift, c, "dshift"), _byref(p), ws, have,
                                        _stream(stream, device))
    if status:
        _failed(status, "conv_layer_norm_grad")
    return dx, dgain, dshift


def _param_dtype(*tensors) -> int:
    code = 0
    for t in tensors:
        if t is not None:
            c = _types.get(t.dtype, (0, 1))[0]
            if code and c != code:
                raise ValueError("gain, shift and their gradients must have one type")
            code = c
    return code or CONV_FLOAT32

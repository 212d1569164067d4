"""Channel operators of libint8conv.so: the matrix product with bias,
activation and residual (``conv_linear``), the layer norm
(``conv_layer_norm``) and their gradients, on matrices of rows (pixels of a
channels-last image, or tokens) by channels.

Argument marshalling only, like the convolution binding: every step runs in
the library's CUDA kernels, on torch tensors of any strides.  Tensors whose
leading dimensions share no stride are refused (a view would do; nothing is
copied).  Outputs that are not given are allocated; a workspace that is not
given (or is too small) is allocated for the call, on the stream the call
runs on.  Autograd does not record these calls: a tensor that requires a
gradient is refused while gradients are recorded (detach it, or call under
``torch.no_grad()``), and outputs count as changed in place.  The marshalling
itself is compiled (csrc/python): read from Python, the tensors' attributes
take longer than the smallest kernels.
"""
from __future__ import annotations

import ctypes

CONV_FLOAT32, CONV_FLOAT16, CONV_BFLOAT16 = 3, 4, 5
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = 0, 1, 2, 3, 4
ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH, "silu": ACT_SILU}

CHANNEL_SYMBOLS = (
    "conv_linear_workspace_size", "conv_linear", "conv_linear_grad_workspace_size", "conv_linear_grad",
    "conv_layer_norm", "conv_layer_norm_grad_workspace_size", "conv_layer_norm_grad",
)


# The C ABI's structures and argument types, for callers of libint8conv.so
# through ctypes; the entry points below go through the compiled binding.
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


_binding = None


def _load():
    """The compiled binding; raises if it has not been built."""
    global _binding
    import torch  # noqa: F401  (its libraries have to be loaded first)

    from . import lib
    lib()
    try:
        from . import _channel
    except ImportError as e:
        raise RuntimeError("the channel operators' binding _channel.so is not built; run "
                           "`python -c 'import __graft_entry__ as g; g.build()'` first") from e
    _binding = _channel
    return _channel


def _failed(status: int, what: str):
    from . import ConvError
    raise ConvError(status, what)


def _activation(a) -> int:
    if isinstance(a, str):
        if a not in ACTIVATIONS:
            raise ValueError(f"unknown activation {a!r}: one of {', '.join(ACTIVATIONS)}")
        return ACTIVATIONS[a]
    return int(a)


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
    r = (_binding or _load()).linear(x, w, bias, _activation(activation), residual, preact, out, workspace,
                                     None if stream is None else stream.cuda_stream)
    if r.__class__ is int:
        _failed(r, "conv_linear")
    return r


def conv_linear_grad(dy, x, w, *, preact=None, activation=ACT_NONE, dx=None, dw=None, dbias=None, workspace=None,
                     stream=None):
    """Gradients of conv_linear: fills those of dx [..., K], dw [N, K] (each
    of x's type or float32) and dbias [N] (float32 or x's type) that are
    given.  dy [..., N] is the loss gradient, preact the pre-activation of
    the forward call (needed with an activation); the residual's gradient is
    dy itself.  Returns (dx, dw, dbias)."""
    r = (_binding or _load()).linear_grad(dy, x, w, preact, _activation(activation), dx, dw, dbias, workspace,
                                          None if stream is None else stream.cuda_stream)
    if r is not None:
        _failed(r, "conv_linear_grad")
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
    r = (_binding or _load()).layer_norm(x, gain, shift, eps, scale, out, mean, rstd,
                                         None if stream is None else stream.cuda_stream)
    if r.__class__ is int:
        _failed(r, "conv_layer_norm")
    return r


def conv_layer_norm_grad(dy, x, gain, mean, rstd, *, residual_grad=None, dx=None, dgain=None, dshift=None,
                         workspace=None, stream=None):
    """Gradients of conv_layer_norm for the loss gradient dy [..., C] (x's
    type), with the statistics of the forward call: fills those of
    dx [..., C] (x's type; residual_grad is added to it), dgain and dshift
    [C] (float32 or x's type, gain's type when gain is given) that are
    given.  Returns (dx, dgain, dshift)."""
    r = (_binding or _load()).layer_norm_grad(dy, x, gain, mean, rstd, residual_grad, dx, dgain, dshift, workspace,
                                              None if stream is None else stream.cuda_stream)
    if r is not None:
        _failed(r, "conv_layer_norm_grad")
    return dx, dgain, dshift

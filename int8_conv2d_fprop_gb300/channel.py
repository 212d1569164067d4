"""Channel operators of libint8conv.so: the matrix product with bias,
activation and residual (``conv_linear``), the layer norm
(``conv_layer_norm``) and their gradients; the same product of 8-bit floats
with a scale for each block of 128 (``conv_linear_fp8``) and what makes its
operands (``conv_quantize``); the norms before and after a residual block with
its gate and scales (``conv_block_norm``) and their gradients; all on matrices
of rows (pixels of a channels-last image, or tokens) by channels.  And the
clipping of all a model's gradients by their global norm
(``conv_clip_grads``).

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

CONV_FLOAT32, CONV_FLOAT16, CONV_BFLOAT16, CONV_FLOAT8_E4M3, CONV_FLOAT8_E5M2 = 3, 4, 5, 6, 7
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = 0, 1, 2, 3, 4
ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH, "silu": ACT_SILU}

CHANNEL_SYMBOLS = (
    "conv_linear_workspace_size", "conv_linear", "conv_linear_grad_workspace_size", "conv_linear_grad",
    "conv_layer_norm", "conv_layer_norm_grad_workspace_size", "conv_layer_norm_grad",
    "conv_quantize", "conv_linear_fp8_workspace_size", "conv_linear_fp8",
    "conv_block_norm", "conv_block_norm_grad_workspace_size", "conv_block_norm_grad",
    "conv_clip_grads_workspace_size", "conv_clip_grads",
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


class QuantizeParams(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_int32), ("activation", ctypes.c_int32), ("reserved", ctypes.c_int32 * 2)]


class BlockNormParams(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_float), ("skip_scale", ctypes.c_float), ("branch_scale", ctypes.c_float),
                ("post_norm", ctypes.c_int32), ("param_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32 * 3)]


class GradTensor(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("count", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def declare(L) -> None:
    """Argument types of the channel entry points of a loaded library."""
    v, sz, i64, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_float
    # descriptors and parameters are passed with byref, absent ones as None
    for name, args in (
            ("conv_linear_workspace_size", [v, v, v, v, v]),
            ("conv_linear", [v, v, v, v, v, v, v, v, v, v, v, v, v, sz, v]),
            ("conv_linear_grad_workspace_size", [v, v, v, v, v, v, v, v]),
            ("conv_linear_grad", [v, v, v, v, v, v, v, v, v, v, v, v, v, v, v, sz, v]),
            ("conv_layer_norm", [v, v, v, v, v, v, v, v, v, v]),
            ("conv_layer_norm_grad_workspace_size", [v, v]),
            ("conv_layer_norm_grad", [v, v, v, v, v, v, v, v, v, v, v, v, v, v, v, sz, v]),
            ("conv_quantize", [v] * 14),
            ("conv_linear_fp8_workspace_size", [v] * 5),
            ("conv_linear_fp8", [v] * 17 + [sz, v]),
            ("conv_block_norm", [v] * 18),
            ("conv_block_norm_grad_workspace_size", [v, i64, v]),
            ("conv_block_norm_grad", [v] * 24 + [sz, v]),
            ("conv_clip_grads_workspace_size", [v, i64, v]),
            ("conv_clip_grads", [v, i64, f32, f32, v, v, sz, v])):
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


_types = None


def _type_code(dtype) -> int:
    """The code of a torch dtype (or a CONV_* code as it is)."""
    global _types
    if _types is None:
        import torch
        _types = {torch.float32: CONV_FLOAT32, torch.float16: CONV_FLOAT16, torch.bfloat16: CONV_BFLOAT16,
                  torch.float8_e4m3fn: CONV_FLOAT8_E4M3, torch.float8_e5m2: CONV_FLOAT8_E5M2}
    code = _types.get(dtype, dtype)
    if code.__class__ is not int:
        raise ValueError(f"no output of {dtype} is made")
    return code


def conv_quantize(x, *, dtype=CONV_FLOAT8_E4M3, tile: int = 1, rows: bool = True, columns: bool = False, preact=None,
                  activation=ACT_NONE, out=None, scale=None, out_t=None, scale_t=None, stream=None):
    """8-bit floats with a float32 scale for each block of 128, of
    x [..., C] (float32, float16 or bfloat16, any strides) or, with an
    activation, of x times its slope at preact [..., C] (a loss gradient on
    its way back through the activation).

    dtype: torch.float8_e4m3fn or torch.float8_e5m2; tile: rows that share a
    scale, 1 (activations, gradients) or 128 (weights).  rows: gives
    out [..., C] and scale [..., ceil(C / 128)] (tile 128: [ceil(M / 128),
    ceil(C / 128)] for M rows); columns: the same of x transposed, out_t
    [C, M] and scale_t, for products over the rows; both are made from one
    reading.  A value is about out * scale.  Outputs that are not given are
    allocated with 16-byte aligned rows, as conv_linear_fp8 reads them in
    place.  Returns (out, scale), (out_t, scale_t) or all four."""
    r = (_binding or _load()).quantize(x, preact, _activation(activation), tile, _type_code(dtype), rows, columns, out,
                                       scale, out_t, scale_t, None if stream is None else stream.cuda_stream)
    if r.__class__ is int:
        _failed(r, "conv_quantize")
    return r


def conv_linear_fp8(x, x_scale, w, w_scale, bias=None, *, activation=ACT_NONE, residual=None, preact=None, out=None,
                    dtype=CONV_BFLOAT16, workspace=None, stream=None):
    """y = act(x w^T + bias) + residual of 8-bit operands with block scales, as
    conv_quantize makes them.

    x [..., K] and w [N, K]: float8_e4m3fn or float8_e5m2, each its own, with
    adjacent columns; x_scale: float32 [..., ceil(K / 128)], a scale for each
    row, or [ceil(M / 128), ceil(K / 128)] for squares of 128; w_scale: the
    same with N.  bias: [N], float32 or the output's type; residual [..., N]
    of the output's type; preact: float16 or bfloat16 [..., N] that receives
    x w^T + bias; out: optional [..., N], float32, float16 or bfloat16 (else
    allocated, of ``dtype``).  Sums are in 32 bits.  Runs on ``stream``
    (default: the current one).  Returns ``out``.

    Gradients are calls of the same kind: with the loss gradient dz quantised
    both ways and w and x in columns, dx = conv_linear_fp8(dz, dz_scale, wt,
    wt_scale) and dw = conv_linear_fp8(dzt, dzt_scale, xt, xt_scale)."""
    r = (_binding or _load()).linear_fp8(x, x_scale, w, w_scale, bias, _activation(activation), residual, preact, out,
                                         _type_code(dtype), workspace, None if stream is None else stream.cuda_stream)
    if r.__class__ is int:
        _failed(r, "conv_linear_fp8")
    return r


def conv_block_norm(x, skip=None, *, post_norm: bool = False, post_gain=None, gate=None, skip_scale: float = 1.0,
                    branch_scale: float = 1.0, gain=None, norm: bool = True, eps: float = 1e-6, sum=None, out=None,
                    out_scale=None, dtype=None, post_rstd=None, rstd=None, stream=None):
    """The end of a residual block and the beginning of the next, for the
    block's output x [..., C] and the stream skip [..., C] around it:

        n   = x / rms(x) * post_gain            (post_norm; else x)
        sum = skip_scale * skip + branch_scale * gate * n
        out = sum / rms(sum) * gain             (norm)

    with rms(v) = sqrt(mean(v^2) + eps) over the last dimension.  x: float32,
    float16 or bfloat16; skip and sum: of x's type or float32; post_gain and
    gain: optional [C], both float32 or both of x's type; gate: optional [C]
    or [G, C] (leading dims count together), float32 or x's type, G dividing
    the rows, each serving as many rows in turn.  out is of x's type, or with
    dtype=torch.float8_e4m3fn quantised with out_scale [..., ceil(C / 128)] as
    by conv_quantize.  post_rstd, rstd: optional float32 vectors, an element
    per row, that receive 1 / rms (what conv_block_norm_grad wants).  Outputs
    that are not given are allocated; sum may be skip or x, and out x.  With
    x and gain alone this is the root-mean-square norm.  Returns (sum, out),
    or (sum, out, out_scale) with an 8-bit out; sum is None where it is x
    itself (no skip, gate, post norm or branch_scale) and not given, out
    without a norm."""
    r = (_binding or _load()).block_norm(x, skip, post_norm, post_gain, gate, skip_scale, branch_scale, gain, norm, eps,
                                         sum, out, out_scale, None if dtype is None else _type_code(dtype), post_rstd,
                                         rstd, None if stream is None else stream.cuda_stream)
    if r.__class__ is int:
        _failed(r, "conv_block_norm")
    return r


def conv_block_norm_grad(dy, dsum, x, sum, *, post_norm: bool = False, post_gain=None, gate=None,
                         skip_scale: float = 1.0, branch_scale: float = 1.0, gain=None, post_rstd=None, rstd=None,
                         dx=None, dskip=None, dgate=None, dgain=None, dpost_gain=None, workspace=None, stream=None):
    """Gradients of conv_block_norm for the loss gradients dy of out (x's type)
    and dsum of sum (sum's type), either of which may be None, with x, sum and
    the statistics of the forward call: fills those of dx [..., C] (x's type),
    dskip [..., C] (sum's type), dgate (gate's shape, or any [G, C] without a
    gate; float32 or x's type), dgain and dpost_gain [C] (of the gains' type)
    that are given.  x is wanted for a post norm and for dgate, sum and rstd
    with dy.  dskip may be dsum, and dx may be dy.  Returns (dx, dskip, dgate,
    dgain, dpost_gain)."""
    r = (_binding or _load()).block_norm_grad(dy, dsum, x, sum, post_norm, post_gain, gate, skip_scale, branch_scale,
                                              gain, post_rstd, rstd, dx, dskip, dgate, dgain, dpost_gain, workspace,
                                              None if stream is None else stream.cuda_stream)
    if r is not None:
        _failed(r, "conv_block_norm_grad")
    return dx, dskip, dgate, dgain, dpost_gain


def conv_clip_grads(grads, max_norm=None, *, eps: float = 1e-6, out=None, norm=None, workspace=None, stream=None):
    """The global norm of the tensors in grads (float32, float16 or bfloat16,
    without gaps between their elements), and, with a max_norm, the tensors
    times min(1, max_norm / (norm + eps)): in place, or to the tensors in out
    (of the same types, shapes and strides).  An infinite max_norm is none:
    nothing is written then, and out is refused.  norm: optional float32 tensor of
    one element that receives the norm.  Nothing waits for the GPU.  Returns
    norm."""
    r = (_binding or _load()).clip_grads(grads, float("inf") if max_norm is None else max_norm, eps, out, norm, workspace,
                                         None if stream is None else stream.cuda_stream)
    if r.__class__ is int:
        _failed(r, "conv_clip_grads")
    return r

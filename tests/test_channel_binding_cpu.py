"""What the channel operators' compiled binding refuses before anything touches
a device.  The tensors are CUDA tensors by their descriptors only: their
addresses point at nothing, so a call that is not refused ends, on a machine
without a GPU, in the error of the missing driver.  Where there is a GPU the
tests do not run."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


class _DLTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("device_type", ctypes.c_int32), ("device_id", ctypes.c_int32),
                ("ndim", ctypes.c_int32), ("code", ctypes.c_uint8), ("bits", ctypes.c_uint8), ("lanes", ctypes.c_uint16),
                ("shape", ctypes.c_void_p), ("strides", ctypes.c_void_p), ("byte_offset", ctypes.c_uint64)]


class _Managed(ctypes.Structure):
    _fields_ = [("tensor", _DLTensor), ("context", ctypes.c_void_p), ("deleter", ctypes.c_void_p)]


_CODES = {torch.int8: (0, 8), torch.int16: (0, 16), torch.int32: (0, 32), torch.int64: (0, 64), torch.uint8: (1, 8),
          torch.bool: (6, 8), torch.float16: (2, 16), torch.float32: (2, 32), torch.float64: (2, 64),
          torch.bfloat16: (4, 16)}
_kept = []
_next = [0x10000000]


def described(*shape, dtype=torch.bfloat16, device=0):
    """A contiguous CUDA tensor of this shape without memory behind it."""
    sizes = (ctypes.c_int64 * len(shape))(*shape)
    code, bits = _CODES[dtype]
    _next[0] += 1 << 20
    m = _Managed(_DLTensor(_next[0], 2, device, len(shape), code, bits, 1, ctypes.addressof(sizes), None, 0), None, None)
    _kept.append((m, sizes))
    capsule = ctypes.pythonapi.PyCapsule_New
    capsule.restype, capsule.argtypes = ctypes.py_object, [ctypes.c_void_p, ctypes.c_char_p, ctypes.c_void_p]
    return torch._C._from_dlpack(capsule(ctypes.addressof(m), b"dltensor", None))


@pytest.fixture
def ic(monkeypatch):
    if torch.cuda.is_available():
        pytest.skip("these addresses are not to reach a GPU")
    monkeypatch.setattr(torch.cuda, "_lazy_init", lambda: None)
    import __graft_entry__
    __graft_entry__.build_library()
    import int8_conv2d_fprop_gb300 as m
    return m


BF16, F32 = torch.bfloat16, torch.float32
NOT_FLOATS = [torch.float64, torch.int64, torch.int32, torch.int16, torch.int8, torch.uint8, torch.bool]


def refused(ic, name, call):
    with pytest.raises(ic.ConvError) as e:
        call()
    assert e.value.name == name


@pytest.mark.parametrize("dtype", NOT_FLOATS)
@pytest.mark.parametrize("which", ["gain", "shift"])
def test_layer_norm_takes_float_parameters_only(ic, which, dtype):
    x = described(4, 16)
    refused(ic, "CONV_ERR_DTYPE", lambda: ic.conv_layer_norm(x, **{which: described(16, dtype=dtype)}))
    # ... and not with a float vector beside it
    both = {"gain": described(16, dtype=F32), "shift": described(16, dtype=F32)}
    both[which] = described(16, dtype=dtype)
    refused(ic, "CONV_ERR_DTYPE", lambda: ic.conv_layer_norm(x, **both))


@pytest.mark.parametrize("dtype", NOT_FLOATS)
@pytest.mark.parametrize("which", ["gain", "dgain", "dshift"])
def test_layer_norm_grad_takes_float_parameters_only(ic, which, dtype):
    x, dy, dx = described(4, 16), described(4, 16), described(4, 16)
    mean, rstd = described(4, dtype=F32), described(4, dtype=F32)

    def call(**vectors):
        gain = vectors.pop("gain", None)
        return lambda: ic.conv_layer_norm_grad(dy, x, gain, mean, rstd, dx=dx, **vectors)

    refused(ic, "CONV_ERR_DTYPE", call(**{which: described(16, dtype=dtype)}))
    every = {k: described(16, dtype=F32) for k in ("gain", "dgain", "dshift")}
    every[which] = described(16, dtype=dtype)
    refused(ic, "CONV_ERR_DTYPE", call(**every))


def test_parameters_of_two_float_types(ic):
    x = described(4, 16)
    with pytest.raises(ValueError, match="one type"):
        ic.conv_layer_norm(x, described(16, dtype=F32), described(16))


# every tensor argument of the four calls: builds it, given the device of one of them
def _linear_arguments(at):
    return ("conv_linear", [described(4, 16, device=at("x")), described(8, 16, device=at("w"))],
            {"bias": described(8, device=at("bias")), "residual": described(4, 8, device=at("residual")),
             "preact": described(4, 8, device=at("preact")), "out": described(4, 8, device=at("out")),
             "workspace": described(1 << 16, dtype=torch.uint8, device=at("workspace"))})


def _linear_grad_arguments(at):
    return ("conv_linear_grad", [described(4, 8, device=at("dy")), described(4, 16, device=at("x")),
                                 described(8, 16, device=at("w"))],
            {"preact": described(4, 8, device=at("preact")), "activation": "gelu",
             "dx": described(4, 16, device=at("dx")), "dw": described(8, 16, device=at("dw")),
             "dbias": described(8, dtype=F32, device=at("dbias")),
             "workspace": described(1 << 16, dtype=torch.uint8, device=at("workspace"))})


def _norm_arguments(at):
    return ("conv_layer_norm", [described(4, 16, device=at("x")), described(16, dtype=F32, device=at("gain")),
                                described(16, dtype=F32, device=at("shift"))],
            {"out": described(4, 16, device=at("out")), "mean": described(4, dtype=F32, device=at("mean")),
             "rstd": described(4, dtype=F32, device=at("rstd"))})


def _norm_grad_arguments(at):
    return ("conv_layer_norm_grad", [described(4, 16, device=at("dy")), described(4, 16, device=at("x")),
                                     described(16, dtype=F32, device=at("gain")),
                                     described(4, dtype=F32, device=at("mean")), described(4, dtype=F32, device=at("rstd"))],
            {"residual_grad": described(4, 16, device=at("residual_grad")), "dx": described(4, 16, device=at("dx")),
             "dgain": described(16, dtype=F32, device=at("dgain")), "dshift": described(16, dtype=F32, device=at("dshift")),
             "workspace": described(1 << 16, dtype=torch.uint8, device=at("workspace"))})


_TENSORS = [(_linear_arguments, "x w bias residual preact out workspace"),
            (_linear_grad_arguments, "dy x w preact dx dw dbias workspace"),
            (_norm_arguments, "x gain shift out mean rstd"),
            (_norm_grad_arguments, "dy x gain mean rstd residual_grad dx dgain dshift workspace")]


@pytest.mark.parametrize("arguments,which", [(a, w) for a, names in _TENSORS for w in names.split()])
def test_tensors_of_two_devices(ic, arguments, which):
    name, args, kwargs = arguments(lambda n: 1 if n == which else 0)
    with pytest.raises(ValueError, match="device"):
        getattr(ic, name)(*args, **kwargs)


@pytest.mark.parametrize("code", [-1, 5, 1 << 32, (1 << 32) + 2, -(1 << 32), 1 << 70])
def test_activation_codes_are_not_cut_to_32_bits(ic, code):
    x, w, dy = described(4, 16), described(8, 16), described(4, 8)
    refused(ic, "CONV_ERR_BAD_PARAM", lambda: ic.conv_linear(x, w, activation=code))
    refused(ic, "CONV_ERR_BAD_PARAM", lambda: ic.conv_linear_grad(dy, x, w, preact=dy, activation=code, dx=x))


@pytest.mark.parametrize("arguments,which", [(a, w) for a, names in _TENSORS for w in names.split() if w != "workspace"])
def test_tensors_that_require_a_gradient(ic, arguments, which):
    """Refused while gradients are recorded, which the call would not be; with
    recording off such a call is like any other (here it gets as far as the
    missing driver)."""
    name, args, kwargs = arguments(lambda n: 0)
    order = dict(_TENSORS)[arguments].split()
    target = args[order.index(which)] if order.index(which) < len(args) else kwargs[which]
    target.requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        getattr(ic, name)(*args, **kwargs)
    with torch.no_grad(), pytest.raises(RuntimeError, match="CUDA"):
        getattr(ic, name)(*args, **kwargs)


@pytest.mark.parametrize("arguments,which", [(a, w) for a, names in _TENSORS for w in names.split() if w != "workspace"])
def test_lazily_negated_views(ic, arguments, which):
    """The imaginary part of a conjugate, say: its memory holds the opposite."""
    name, args, kwargs = arguments(lambda n: 0)
    order = dict(_TENSORS)[arguments].split()
    i = order.index(which)
    where, key = (args, i) if i < len(args) else (kwargs, which)
    where[key] = torch._neg_view(where[key])
    with pytest.raises(ValueError, match="lazy"):
        getattr(ic, name)(*args, **kwargs)

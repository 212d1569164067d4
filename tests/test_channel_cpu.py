"""Host side of the channel operators: the refusals of every entry point
(made before anything touches a device), workspace sizes, and the 64-bit
definitions the GPU tests compare with, pinned to differences."""
import ctypes

import numpy as np
import pytest

from oracle import channel as oc

A = 0x10000000  # addresses that are never dereferenced
B, C, D, E, F, G, W = (A + i * 0x1000000 for i in range(1, 8))


@pytest.fixture(scope="module")
def ic():
    import __graft_entry__
    __graft_entry__.build_library()
    import int8_conv2d_fprop_gb300 as m
    m.lib()
    return m


def mat(ic, rows, cols, dtype=None, rs=None, cs=1, cap=None, reserved=0):
    dtype = ic.CONV_FLOAT16 if dtype is None else dtype
    rs = cols if rs is None else rs
    size = {1: 1, 4: 2, 5: 2}.get(dtype, 4)
    need = ((rows - 1) * rs + (cols - 1) * cs + 1) * size if rows > 0 and cols > 0 else 0
    return ic.MatrixDesc(dtype, reserved, rows, cols, rs, cs, max(need, 0) if cap is None else cap)


def linear(ic, x, w, y, xp=A, wp=B, yp=C, bias=None, res=None, resp=None, pre=None, prep=None, act=0, bias_dtype=3,
           ws=None, ws_bytes=0, reserved=0):
    p = ic.LinearParams(act, bias_dtype)
    p.reserved[1] = reserved
    r = ctypes.byref
    st = ic.lib().conv_linear(r(x), xp, r(w), wp, bias, res and r(res), resp, pre and r(pre), prep, r(y), yp, r(p), ws,
                              ws_bytes, None)
    return ic.STATUS[st]


def test_linear_refusals(ic):
    h, b, f, i8 = ic.CONV_FLOAT16, ic.CONV_BFLOAT16, ic.CONV_FLOAT32, ic.CONV_INT8
    x, w, y = mat(ic, 5, 16), mat(ic, 7, 16), mat(ic, 5, 7)
    p = ic.LinearParams(0, 3)
    assert ic.STATUS[ic.lib().conv_linear(None, A, None, B, None, None, None, None, None, None, C, ctypes.byref(p),
                                          None, 0, None)] == "CONV_ERR_NULL_PTR"
    assert linear(ic, x, w, y, xp=None) == "CONV_ERR_NULL_PTR"
    assert linear(ic, x, w, y, yp=None) == "CONV_ERR_NULL_PTR"
    assert linear(ic, x, mat(ic, 7, 16, b), y) == "CONV_ERR_DTYPE"
    assert linear(ic, mat(ic, 5, 16, f), mat(ic, 7, 16, f), y) == "CONV_ERR_DTYPE"
    assert linear(ic, mat(ic, 5, 16, i8), mat(ic, 7, 16, i8), y) == "CONV_ERR_DTYPE"
    assert linear(ic, mat(ic, 5, 16, 9), w, y) == "CONV_ERR_DTYPE"
    assert linear(ic, x, w, mat(ic, 5, 7, b)) == "CONV_ERR_DTYPE"
    assert linear(ic, x, w, y, bias=D, bias_dtype=b) == "CONV_ERR_DTYPE"
    assert linear(ic, x, w, y, res=mat(ic, 5, 7, f), resp=D) == "CONV_ERR_DTYPE"
    assert linear(ic, x, w, mat(ic, 5, 7, f), pre=mat(ic, 5, 7, f), prep=D) == "CONV_ERR_DTYPE"
    assert linear(ic, x, mat(ic, 7, 17), y) == "CONV_ERR_SHAPE_MISMATCH"
    assert linear(ic, x, w, mat(ic, 5, 8)) == "CONV_ERR_SHAPE_MISMATCH"
    assert linear(ic, x, w, y, res=mat(ic, 4, 7), resp=D) == "CONV_ERR_SHAPE_MISMATCH"
    assert linear(ic, x, w, y, act=5) == "CONV_ERR_BAD_PARAM"
    assert linear(ic, x, w, y, reserved=1) == "CONV_ERR_BAD_PARAM"
    assert linear(ic, mat(ic, 5, 16, reserved=2), w, y) == "CONV_ERR_BAD_PARAM"
    assert linear(ic, mat(ic, -1, 16), w, y) == "CONV_ERR_BAD_PARAM"
    assert linear(ic, mat(ic, 5, 16, rs=0), w, y) == "CONV_ERR_BAD_STRIDES"
    assert linear(ic, x, w, mat(ic, 5, 7, rs=6)) == "CONV_ERR_BAD_STRIDES"
    assert linear(ic, mat(ic, 5, 16, rs=-16, cap=1 << 20), w, y) == "CONV_ERR_BAD_STRIDES"
    assert linear(ic, mat(ic, 5, 16, cap=159), w, y) == "CONV_ERR_BUFFER_TOO_SMALL"
    assert linear(ic, x, w, y, xp=A + 1) == "CONV_ERR_ALIGNMENT"
    assert linear(ic, x, w, y, bias=D + 2, bias_dtype=3) == "CONV_ERR_ALIGNMENT"
    assert linear(ic, mat(ic, 1 << 31, 16, cap=1 << 40), w, y) == "CONV_ERR_TOO_LARGE"
    assert linear(ic, mat(ic, 5, 16, rs=1 << 40, cap=1 << 62), w, y) == "CONV_ERR_TOO_LARGE"
    assert linear(ic, x, w, y, yp=A + 64) == "CONV_ERR_OVERLAP"
    assert linear(ic, x, w, y, bias=C, bias_dtype=3) == "CONV_ERR_OVERLAP"
    assert linear(ic, x, w, y, res=mat(ic, 5, 7, rs=8), resp=C) == "CONV_ERR_OVERLAP"
    assert linear(ic, x, w, y, pre=mat(ic, 5, 7), prep=C) == "CONV_ERR_OVERLAP"
    # odd row strides are packed: a workspace is needed, apart from the rest
    xo = mat(ic, 5, 16, rs=17)
    assert linear(ic, xo, w, y) == "CONV_ERR_WORKSPACE"
    assert linear(ic, xo, w, y, ws=W, ws_bytes=255) == "CONV_ERR_WORKSPACE"
    assert linear(ic, xo, w, y, ws=W + 16, ws_bytes=4096) == "CONV_ERR_WORKSPACE"
    assert linear(ic, xo, w, y, ws=C - 256, ws_bytes=1 << 20, yp=C - 256) == "CONV_ERR_OVERLAP"
    # empty results ask for nothing
    assert linear(ic, mat(ic, 0, 16), w, mat(ic, 0, 7), xp=None, yp=None) == "CONV_OK"
    assert linear(ic, x, mat(ic, 0, 16), mat(ic, 5, 0), wp=None, yp=None) == "CONV_OK"


def test_linear_workspace(ic):
    def size(x, w, xp=0, wp=0):
        out = ctypes.c_size_t()
        r = ctypes.byref
        st = ic.lib().conv_linear_workspace_size(r(x), xp, r(w), wp, r(out))
        assert ic.STATUS[st] == "CONV_OK"
        return out.value

    w = mat(ic, 7, 16)
    assert size(mat(ic, 5, 16), w) == 0
    assert size(mat(ic, 5, 16, rs=24), w) == 0
    assert size(mat(ic, 5, 16, rs=1, cs=8), w) == 0       # columns contiguous
    assert size(mat(ic, 1, 13), mat(ic, 7, 13, rs=16)) == 0  # one row has no stride
    assert size(mat(ic, 5, 16), w, xp=A + 2) == 256       # misaligned address
    assert size(mat(ic, 5, 16, rs=17), w) == 256
    assert size(mat(ic, 5, 16, rs=64, cs=2), w) == 256    # no contiguous dim
    assert size(mat(ic, 100, 13, rs=13), mat(ic, 7, 13, rs=13)) == 3200 + 128 + 256
    assert size(mat(ic, 0, 13), mat(ic, 7, 13, rs=16)) == 0


def test_interleaved_matrices_do_not_overlap(ic):
    # y beside x in one buffer of 64 columns; one column too wide touches it
    # (w has an odd row stride: a call that passes the overlap check is then
    # refused for its missing workspace, before anything runs)
    x, w = mat(ic, 8, 32, rs=64), mat(ic, 24, 32, rs=33)
    assert linear(ic, x, w, mat(ic, 8, 24, rs=64), yp=A + 64) == "CONV_ERR_WORKSPACE"
    assert linear(ic, x, w, mat(ic, 8, 24, rs=64), yp=A + 62) == "CONV_ERR_OVERLAP"
    assert linear(ic, x, mat(ic, 33, 32, rs=33), mat(ic, 8, 33, rs=64), yp=A + 64) == "CONV_ERR_OVERLAP"
    assert linear(ic, x, w, mat(ic, 8, 24, rs=72), yp=A + 64) == "CONV_ERR_OVERLAP"


def grad(ic, dy, x, w, dx=None, dw=None, db=None, pre=None, act=0, bias_dtype=3, ws=W, ws_bytes=1 << 20, dyp=A, xp=B,
         wp=C, dxp=D, dwp=E, prep=F):
    r = ctypes.byref
    p = ic.LinearParams(act, bias_dtype)
    st = ic.lib().conv_linear_grad(r(dy), dyp, r(x), xp, r(w), wp, pre and r(pre), prep, dx and r(dx), dxp,
                                   dw and r(dw), dwp, db, r(p), ws, ws_bytes, None)
    return ic.STATUS[st]


def test_linear_grad_refusals(ic):
    b, f = ic.CONV_BFLOAT16, ic.CONV_FLOAT32
    dy, x, w = mat(ic, 5, 7, rs=8), mat(ic, 5, 16), mat(ic, 7, 16)
    dx, dw = mat(ic, 5, 16), mat(ic, 7, 16)
    assert grad(ic, dy, x, w) == "CONV_ERR_NULL_PTR"
    assert grad(ic, dy, x, w, dx, act=2) == "CONV_ERR_NULL_PTR"  # no pre-activation
    assert grad(ic, dy, x, w, dx, dxp=None) == "CONV_ERR_NULL_PTR"
    assert grad(ic, mat(ic, 5, 7, b), x, w, dx) == "CONV_ERR_DTYPE"
    assert grad(ic, dy, x, w, mat(ic, 5, 16, b)) == "CONV_ERR_DTYPE"
    assert grad(ic, dy, x, w, dx, pre=mat(ic, 5, 7, f), act=1) == "CONV_ERR_DTYPE"
    assert grad(ic, dy, x, w, db=G, bias_dtype=b) == "CONV_ERR_DTYPE"
    assert grad(ic, mat(ic, 5, 8), x, w, dx) == "CONV_ERR_SHAPE_MISMATCH"
    assert grad(ic, dy, x, w, dw=mat(ic, 16, 7)) == "CONV_ERR_SHAPE_MISMATCH"
    assert grad(ic, dy, x, w, dx, pre=mat(ic, 5, 8), act=1) == "CONV_ERR_SHAPE_MISMATCH"
    assert grad(ic, dy, x, w, dx, act=7) == "CONV_ERR_BAD_PARAM"
    assert grad(ic, dy, x, w, dx, dxp=B) == "CONV_ERR_OVERLAP"
    assert grad(ic, dy, x, w, dx, dw, dwp=D) == "CONV_ERR_OVERLAP"
    assert grad(ic, dy, x, w, db=A) == "CONV_ERR_OVERLAP"
    assert grad(ic, dy, x, w, dx, pre=mat(ic, 5, 7), act=1, ws=None, ws_bytes=0) == "CONV_ERR_WORKSPACE"
    assert grad(ic, dy, x, w, dx, pre=mat(ic, 5, 7), act=1, ws=D, ws_bytes=1 << 20) == "CONV_ERR_OVERLAP"


def norm(ic, x, y, xp=A, yp=B, gain=C, shift=D, mean=None, rstd=None, eps=1e-5, scale=1.0, pd=3, reserved=0):
    p = ic.LayerNormParams(eps, scale, pd, reserved)
    r = ctypes.byref
    return ic.STATUS[ic.lib().conv_layer_norm(r(x), xp, gain, shift, r(y), yp, mean, rstd, r(p), None)]


def test_layer_norm_refusals(ic):
    h, b, f, i32 = ic.CONV_FLOAT16, ic.CONV_BFLOAT16, ic.CONV_FLOAT32, ic.CONV_INT32
    x, y = mat(ic, 5, 16), mat(ic, 5, 16)
    assert norm(ic, x, y, xp=None) == "CONV_ERR_NULL_PTR"
    assert norm(ic, mat(ic, 5, 16, ic.CONV_INT8), y) == "CONV_ERR_DTYPE"
    assert norm(ic, x, mat(ic, 5, 16, i32)) == "CONV_ERR_DTYPE"
    assert norm(ic, x, y, pd=b) == "CONV_ERR_DTYPE"
    assert norm(ic, x, mat(ic, 5, 15)) == "CONV_ERR_SHAPE_MISMATCH"
    assert norm(ic, mat(ic, 5, 0), mat(ic, 5, 0)) == "CONV_ERR_BAD_PARAM"
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert norm(ic, x, y, eps=eps) == "CONV_ERR_BAD_PARAM"
    for scale in (0.0, float("nan"), float("inf")):
        assert norm(ic, x, y, scale=scale) == "CONV_ERR_BAD_PARAM"
    assert norm(ic, x, y, reserved=1) == "CONV_ERR_BAD_PARAM"
    assert norm(ic, x, mat(ic, 5, 16, rs=15)) == "CONV_ERR_BAD_STRIDES"
    assert norm(ic, x, y, gain=C + 2) == "CONV_ERR_ALIGNMENT"
    assert norm(ic, x, y, yp=A + 2) == "CONV_ERR_OVERLAP"
    assert norm(ic, x, mat(ic, 5, 16, f), yp=A) == "CONV_ERR_OVERLAP"  # in place wants one size
    assert norm(ic, x, y, gain=B) == "CONV_ERR_OVERLAP"
    assert norm(ic, x, y, mean=A) == "CONV_ERR_OVERLAP"
    assert norm(ic, x, y, mean=E, rstd=E + 16) == "CONV_ERR_OVERLAP"
    assert norm(ic, x, y, rstd=C) == "CONV_ERR_OVERLAP"
    assert norm(ic, mat(ic, 0, 16), mat(ic, 0, 16), xp=None, yp=None) == "CONV_OK"


def norm_grad(ic, dy, x, dx=None, dg=None, db=None, res=None, dyp=A, xp=B, gain=C, mean=D, rstd=D + 4096, dxp=E,
              resp=F, scale=1.0, pd=3, ws=W, ws_bytes=1 << 20):
    p = ic.LayerNormParams(1e-5, scale, pd, 0)
    r = ctypes.byref
    return ic.STATUS[ic.lib().conv_layer_norm_grad(r(dy), dyp, r(x), xp, gain, mean, rstd, res and r(res), resp,
                                                   dx and r(dx), dxp, dg, db, r(p), ws, ws_bytes, None)]


def test_layer_norm_grad_refusals(ic):
    x, dy, dx = mat(ic, 5, 16), mat(ic, 5, 16), mat(ic, 5, 16)
    assert norm_grad(ic, dy, x) == "CONV_ERR_NULL_PTR"
    assert norm_grad(ic, dy, x, dx, mean=None) == "CONV_ERR_NULL_PTR"
    assert norm_grad(ic, dy, x, dx, dxp=None) == "CONV_ERR_NULL_PTR"
    i = mat(ic, 5, 16, ic.CONV_INT32)
    assert norm_grad(ic, i, i, i) == "CONV_ERR_DTYPE"
    assert norm_grad(ic, mat(ic, 5, 16, ic.CONV_BFLOAT16), x, dx) == "CONV_ERR_DTYPE"
    assert norm_grad(ic, dy, x, dx, pd=ic.CONV_BFLOAT16) == "CONV_ERR_DTYPE"
    assert norm_grad(ic, mat(ic, 4, 16), x, dx) == "CONV_ERR_SHAPE_MISMATCH"
    assert norm_grad(ic, dy, x, dx, res=mat(ic, 5, 17)) == "CONV_ERR_SHAPE_MISMATCH"
    assert norm_grad(ic, dy, x, dx, scale=2.0) == "CONV_ERR_BAD_PARAM"
    assert norm_grad(ic, dy, x, dx, dxp=A) == "CONV_ERR_OVERLAP"
    assert norm_grad(ic, dy, x, dx, dxp=B + 4) == "CONV_ERR_OVERLAP"
    assert norm_grad(ic, dy, x, dx, dg=G, db=G + 32) == "CONV_ERR_OVERLAP"
    assert norm_grad(ic, dy, x, dx, dg=C) == "CONV_ERR_OVERLAP"
    assert norm_grad(ic, dy, x, dx, dg=E) == "CONV_ERR_OVERLAP"
    assert norm_grad(ic, dy, x, dx, dg=G, ws=None) == "CONV_ERR_WORKSPACE"
    assert norm_grad(ic, dy, x, dx, dg=G, ws_bytes=16) == "CONV_ERR_WORKSPACE"
    assert norm_grad(ic, dy, x, dx, dg=G, ws=E) == "CONV_ERR_OVERLAP"
    assert norm_grad(ic, dy, x, dx, res=dx, resp=E, ws=None) == "CONV_ERR_WORKSPACE"  # in place: allowed


# ------------------------------------------------------- the 64-bit definitions
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


@pytest.mark.parametrize("act", ACTS)
def test_slope_is_the_difference_quotient(act):
    # away from ReLU's corner; |f'''| <= 2, so the quotient is within h^2/3 + rounding
    z = np.concatenate([np.linspace(-9, -0.01, 200), np.linspace(0.01, 9, 200)])
    h = 1e-5
    q = (oc.activate(z + h, act) - oc.activate(z - h, act)) / (2 * h)
    assert np.max(np.abs(q - oc.activation_slope(z, act))) < 1e-9 + h * h


@pytest.mark.parametrize("act", ACTS)
def test_linear_gradients_are_difference_quotients(act):
    g = np.random.default_rng(3)
    x, w, b, dy = g.standard_normal((4, 6)), g.standard_normal((5, 6)), g.standard_normal(5), g.standard_normal((4, 5))
    _, z = oc.linear(x, w, b, act)
    dx, dw, db, _ = oc.linear_grad(dy, x, w, z, act)
    h = 1e-6
    for arr, grad_ in ((x, dx), (w, dw), (b, db)):
        q = np.empty_like(arr)
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + h
            up = (dy * oc.linear(x, w, b, act)[0]).sum()
            arr[i] = keep - h
            q[i] = (up - (dy * oc.linear(x, w, b, act)[0]).sum()) / (2 * h)
            arr[i] = keep
        assert np.max(np.abs(q - grad_)) < 1e-7


def test_layer_norm_gradients_are_difference_quotients():
    g = np.random.default_rng(4)
    x, dy, gain, shift = g.standard_normal((3, 7)) + 2, g.standard_normal((3, 7)), g.standard_normal(7), g.standard_normal(7)
    _, mean, rstd = oc.layer_norm(x, gain, shift)
    dx, dg, db = oc.layer_norm_grad(dy, x, gain, mean, rstd)
    h = 1e-6
    for arr, grad_ in ((x, dx), (gain, dg), (shift, db)):
        q = np.empty_like(arr)
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + h
            up = (dy * oc.layer_norm(x, gain, shift)[0]).sum()
            arr[i] = keep - h
            q[i] = (up - (dy * oc.layer_norm(x, gain, shift)[0]).sum()) / (2 * h)
            arr[i] = keep
        assert np.max(np.abs(q - grad_)) < 1e-7


def test_binding_refuses_what_no_descriptor_can_say(ic):
    torch = pytest.importorskip("torch")
    x, w = torch.ones(2, 8, dtype=torch.float16), torch.ones(4, 8, dtype=torch.float16)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        ic.conv_linear(x, w)
    with pytest.raises(TypeError):
        ic.conv_linear([1.0], w)
    with pytest.raises(ValueError, match="x is required"):
        ic.conv_layer_norm(None)
    with pytest.raises(ValueError, match="unknown activation"):
        ic.conv_linear(x, w, activation="tanh")
    with pytest.raises(ValueError):
        ic.conv_layer_norm_grad(x, x, None, None, None, dx=x)

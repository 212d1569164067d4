"""Host side of the 8-bit product, its quantisation, the block norms and the
clipping: the refusals of every entry point (made before anything touches a
device), workspace sizes, and the 64-bit definitions that the GPU tests compare
with, pinned to differences."""
import ctypes
import math

import pytest

A = 0x10000000  # addresses that are never dereferenced
B, C, D, E, F, G, H, I, J, W = (A + i * 0x1000000 for i in range(1, 11))
F32, F16, BF16, E4, E5 = 3, 4, 5, 6, 7


@pytest.fixture(scope="module")
def ic():
    import __graft_entry__
    __graft_entry__.build_library()
    import int8_conv2d_fprop_gb300 as m
    m.lib()
    return m


def mat(ic, rows, cols, dtype=BF16, rs=None, cs=1, cap=None, reserved=0):
    rs = cols if rs is None else rs
    size = {1: 1, F16: 2, BF16: 2, E4: 1, E5: 1}.get(dtype, 4)
    need = ((rows - 1) * rs + (cols - 1) * cs + 1) * size if rows > 0 and cols > 0 else 0
    return ic.MatrixDesc(dtype, reserved, rows, cols, rs, cs, max(need, 0) if cap is None else cap)


def ref(d):
    return None if d is None else ctypes.byref(d)


def quantize(ic, x, q=None, s=None, qt=None, st=None, z=None, xp=A, zp=B, qp=C, sp=D, qtp=E, stp=F, tile=1, act=0, reserved=0):
    p = ic.QuantizeParams(tile, act)
    p.reserved[0] = reserved
    return ic.STATUS[ic.lib().conv_quantize(ref(x), xp, ref(z), zp, ref(q), qp, ref(s), sp, ref(qt), qtp, ref(st), stp, ref(p), None)]


def test_quantize_refusals(ic):
    x, q, s = mat(ic, 5, 200), mat(ic, 5, 200, E4), mat(ic, 5, 2, F32)
    qt, st = mat(ic, 200, 5, E4), mat(ic, 200, 1, F32)
    assert quantize(ic, None, q, s) == "CONV_ERR_NULL_PTR"
    assert quantize(ic, x) == "CONV_ERR_NULL_PTR"
    assert quantize(ic, x, q) == "CONV_ERR_NULL_PTR"
    assert quantize(ic, x, q, s, st=st) == "CONV_ERR_NULL_PTR"
    assert quantize(ic, x, q, s, xp=None) == "CONV_ERR_NULL_PTR"
    assert quantize(ic, x, q, s, act=2) == "CONV_ERR_NULL_PTR"
    assert quantize(ic, mat(ic, 5, 200, 2), q, s) == "CONV_ERR_DTYPE"
    assert quantize(ic, mat(ic, 5, 200, E4), q, s) == "CONV_ERR_DTYPE"
    assert quantize(ic, x, mat(ic, 5, 200, 1), s) == "CONV_ERR_DTYPE"
    assert quantize(ic, x, q, mat(ic, 5, 2, F16)) == "CONV_ERR_DTYPE"
    assert quantize(ic, x, q, s, mat(ic, 200, 5, E5), st) == "CONV_ERR_DTYPE"
    assert quantize(ic, x, q, s, z=mat(ic, 5, 200, F32), act=2) == "CONV_ERR_DTYPE"
    assert quantize(ic, x, q, s, tile=64) == "CONV_ERR_BAD_PARAM"
    assert quantize(ic, x, q, s, act=5) == "CONV_ERR_BAD_PARAM"
    assert quantize(ic, x, q, s, reserved=1) == "CONV_ERR_BAD_PARAM"
    assert quantize(ic, x, mat(ic, 5, 201, E4), s) == "CONV_ERR_SHAPE_MISMATCH"
    assert quantize(ic, x, q, mat(ic, 5, 3, F32)) == "CONV_ERR_SHAPE_MISMATCH"
    assert quantize(ic, x, q, s, tile=128) == "CONV_ERR_SHAPE_MISMATCH"
    assert quantize(ic, x, q, s, z=mat(ic, 5, 199), act=2) == "CONV_ERR_SHAPE_MISMATCH"
    assert quantize(ic, x, q, s, sp=D + 2) == "CONV_ERR_ALIGNMENT"
    assert quantize(ic, x, mat(ic, 5, 200, E4, rs=100), s) == "CONV_ERR_BAD_STRIDES"
    assert quantize(ic, x, q, s, qp=A + 64) == "CONV_ERR_OVERLAP"
    assert quantize(ic, x, q, s, sp=C) == "CONV_ERR_OVERLAP"
    assert quantize(ic, x, q, s, qt, st, qtp=C) == "CONV_ERR_OVERLAP"
    assert quantize(ic, mat(ic, 0, 200), mat(ic, 0, 200, E4), mat(ic, 0, 2, F32), xp=None, qp=None, sp=None) == "CONV_OK"


def linear(ic, x, xs, w, ws, y, r=None, z=None, bias=None, bias_dtype=F32, act=0, xp=A, xsp=B, wp=C, wsp=D, yp=E, rp=F, zp=G, work=None,
           work_bytes=0):
    p = ic.LinearParams(act, bias_dtype)
    return ic.STATUS[ic.lib().conv_linear_fp8(ref(x), xp, ref(xs), xsp, ref(w), wp, ref(ws), wsp, bias, ref(r), rp, ref(z), zp, ref(y), yp,
                                              ref(p), work, work_bytes, None)]


def test_linear_fp8_refusals(ic):
    x, xs, w, ws, y = mat(ic, 40, 256, E4), mat(ic, 40, 2, F32), mat(ic, 300, 256, E5), mat(ic, 3, 2, F32), mat(ic, 40, 300)
    assert linear(ic, x, None, w, ws, y) == "CONV_ERR_NULL_PTR"
    assert linear(ic, x, xs, w, ws, y, wsp=None) == "CONV_ERR_NULL_PTR"
    assert linear(ic, mat(ic, 40, 256), xs, w, ws, y) == "CONV_ERR_DTYPE"
    assert linear(ic, x, mat(ic, 40, 2, F16), w, ws, y) == "CONV_ERR_DTYPE"
    assert linear(ic, x, xs, w, ws, mat(ic, 40, 300, E4)) == "CONV_ERR_DTYPE"
    assert linear(ic, x, xs, w, ws, y, r=mat(ic, 40, 300, F32)) == "CONV_ERR_DTYPE"
    assert linear(ic, x, xs, w, ws, y, z=mat(ic, 40, 300, F32)) == "CONV_ERR_DTYPE"
    assert linear(ic, x, xs, w, ws, y, bias=H, bias_dtype=F16) == "CONV_ERR_DTYPE"
    assert linear(ic, x, mat(ic, 40, 3, F32), w, ws, y) == "CONV_ERR_SHAPE_MISMATCH"
    assert linear(ic, x, mat(ic, 2, 2, F32), w, ws, y) == "CONV_ERR_SHAPE_MISMATCH"
    assert linear(ic, x, xs, mat(ic, 300, 255, E5), ws, y) == "CONV_ERR_SHAPE_MISMATCH"
    assert linear(ic, x, xs, w, ws, mat(ic, 40, 301)) == "CONV_ERR_SHAPE_MISMATCH"
    assert linear(ic, mat(ic, 40, 256, E4, rs=1, cs=40), xs, w, ws, y) == "CONV_ERR_BAD_STRIDES"
    assert linear(ic, x, xs, w, ws, y, act=9) == "CONV_ERR_BAD_PARAM"
    assert linear(ic, x, xs, w, ws, y, yp=A) == "CONV_ERR_OVERLAP"
    assert linear(ic, x, xs, w, ws, y, yp=B) == "CONV_ERR_OVERLAP"
    assert linear(ic, x, xs, w, ws, y, z=mat(ic, 40, 300), zp=E) == "CONV_ERR_OVERLAP"
    assert linear(ic, x, xs, w, ws, y, bias=E) == "CONV_ERR_OVERLAP"
    # rows that are not 16-byte aligned are packed
    xo = mat(ic, 40, 256, E4, rs=257)
    assert linear(ic, xo, xs, w, ws, y) == "CONV_ERR_WORKSPACE"
    assert linear(ic, xo, xs, w, ws, y, work=W + 16, work_bytes=1 << 24) == "CONV_ERR_WORKSPACE"
    assert linear(ic, xo, xs, w, ws, y, work=E - 256, work_bytes=1 << 24) == "CONV_ERR_OVERLAP"
    assert linear(ic, mat(ic, 0, 256, E4), mat(ic, 0, 2, F32), w, ws, mat(ic, 0, 300), xp=None, xsp=None, yp=None) == "CONV_OK"


def test_linear_fp8_workspace(ic):
    def size(x, w, xp=0, wp=0):
        out = ctypes.c_size_t()
        assert ic.STATUS[ic.lib().conv_linear_fp8_workspace_size(ref(x), xp, ref(w), wp, ref(out))] == "CONV_OK"
        return out.value

    w = mat(ic, 256, 256, E4)
    assert size(mat(ic, 8, 256, E4), w) == 0
    assert size(mat(ic, 8, 250, E4), mat(ic, 256, 250, E4, rs=256)) == 2048      # 8 rows of 256 bytes
    assert size(mat(ic, 8, 256, E4), w, xp=A + 4) == 2048
    assert size(mat(ic, 1, 250, E4), mat(ic, 256, 250, E4, rs=256)) == 0          # one row has no stride
    assert size(mat(ic, 200, 1 << 14, E4), mat(ic, 256, 1 << 14, E4)) % 256 == 0  # sums cut into runs
    assert size(mat(ic, 200, 1 << 14, E4), mat(ic, 256, 1 << 14, E4)) > 0


def norm(ic, x, skip=None, gate=None, s=None, y=None, ys=None, pg=None, g=None, prstd=None, rstd=None, xp=A, skp=B, gp=C, sp=D, yp=E,
         ysp=F, eps=1e-6, ss=1.0, bs=1.0, post=0, par=F32, reserved=0):
    p = ic.BlockNormParams(eps, ss, bs, post, par)
    p.reserved[1] = reserved
    return ic.STATUS[ic.lib().conv_block_norm(ref(x), xp, ref(skip), skp, ref(gate), gp, pg, g, ref(s), sp, ref(y), yp, ref(ys), ysp, prstd,
                                              rstd, ref(p), None)]


def test_block_norm_refusals(ic):
    x = mat(ic, 6, 200)
    y, s, skip = x, x, x
    assert norm(ic, x) == "CONV_ERR_NULL_PTR"
    assert norm(ic, x, y=y, xp=None) == "CONV_ERR_NULL_PTR"
    assert norm(ic, x, y=mat(ic, 6, 200, E4)) == "CONV_ERR_NULL_PTR"
    assert norm(ic, mat(ic, 6, 200, 2), y=y) == "CONV_ERR_DTYPE"
    assert norm(ic, x, y=mat(ic, 6, 200, F16)) == "CONV_ERR_DTYPE"
    assert norm(ic, x, mat(ic, 6, 200, F16), y=y) == "CONV_ERR_DTYPE"
    assert norm(ic, x, mat(ic, 6, 200, F32), s=s) == "CONV_ERR_DTYPE"
    assert norm(ic, x, gate=mat(ic, 1, 200, F16), s=s) == "CONV_ERR_DTYPE"
    assert norm(ic, x, y=y, par=F16) == "CONV_ERR_DTYPE"
    assert norm(ic, x, y=mat(ic, 6, 200, E4), ys=mat(ic, 6, 2, F16)) == "CONV_ERR_DTYPE"
    assert norm(ic, x, y=mat(ic, 6, 200, E4), ys=mat(ic, 6, 3, F32)) == "CONV_ERR_SHAPE_MISMATCH"
    assert norm(ic, x, gate=mat(ic, 4, 200), s=s) == "CONV_ERR_SHAPE_MISMATCH"
    assert norm(ic, x, gate=mat(ic, 0, 200), s=s) == "CONV_ERR_SHAPE_MISMATCH"
    assert norm(ic, x, gate=mat(ic, 3, 199), s=s) == "CONV_ERR_SHAPE_MISMATCH"
    for bad in (dict(eps=0.0), dict(eps=math.nan), dict(ss=math.inf), dict(bs=math.nan), dict(post=2), dict(reserved=1)):
        assert norm(ic, x, y=y, **bad) == "CONV_ERR_BAD_PARAM"
    assert norm(ic, mat(ic, 6, 0), y=mat(ic, 6, 0)) == "CONV_ERR_BAD_PARAM"
    assert norm(ic, mat(ic, 6, 49153), y=mat(ic, 6, 49153)) == "CONV_ERR_TOO_LARGE"
    assert norm(ic, x, y=y, g=G + 2) == "CONV_ERR_ALIGNMENT"
    assert norm(ic, x, y=y, rstd=G + 1) == "CONV_ERR_ALIGNMENT"
    assert norm(ic, x, skip, s=s, y=y, yp=B) == "CONV_ERR_OVERLAP"      # y is not made in skip's place
    assert norm(ic, x, s=s, y=y, yp=D) == "CONV_ERR_OVERLAP"
    assert norm(ic, x, s=s, sp=A + 2) == "CONV_ERR_OVERLAP"
    assert norm(ic, x, y=y, rstd=A) == "CONV_ERR_OVERLAP"
    assert norm(ic, mat(ic, 0, 200), y=mat(ic, 0, 200), xp=None, yp=None) == "CONV_OK"


def grad(ic, dy=None, ds=None, x=None, s=None, gate=None, dx=None, dskip=None, dgate=None, dpg=None, dg=None, pg=None, g=None, prstd=None,
         rstd=None, post=0, par=F32, work=W, work_bytes=1 << 24, dyp=A, dsp=B, xp=C, sp=D, gp=E, dxp=F, dskp=G, dgp=H):
    p = ic.BlockNormParams(1e-6, 1.0, 1.0, post, par)
    return ic.STATUS[ic.lib().conv_block_norm_grad(ref(dy), dyp, ref(ds), dsp, ref(x), xp, ref(s), sp, ref(gate), gp, pg, g, prstd, rstd,
                                                   ref(dx), dxp, ref(dskip), dskp, ref(dgate), dgp, dpg, dg, ref(p), work, work_bytes, None)]


def test_block_norm_grad_refusals(ic):
    m = mat(ic, 6, 200)
    ok = dict(dy=m, s=m, rstd=I, dx=m)
    assert grad(ic, dx=m) == "CONV_ERR_NULL_PTR"
    assert grad(ic, dy=m, s=m, rstd=I) == "CONV_ERR_NULL_PTR"
    assert grad(ic, dy=m, rstd=I, dx=m) == "CONV_ERR_NULL_PTR"
    assert grad(ic, dy=m, s=m, dx=m) == "CONV_ERR_NULL_PTR"
    assert grad(ic, **ok, post=1) == "CONV_ERR_NULL_PTR"
    assert grad(ic, **ok, x=m, post=1) == "CONV_ERR_NULL_PTR"
    assert grad(ic, **ok, dgate=mat(ic, 1, 200)) == "CONV_ERR_NULL_PTR"
    assert grad(ic, **ok, dpg=J) == "CONV_ERR_BAD_PARAM"
    assert grad(ic, ds=m, dskip=m, dg=J) == "CONV_ERR_BAD_PARAM"
    assert grad(ic, dy=m, s=mat(ic, 6, 200, F16), rstd=I, dx=m) == "CONV_ERR_DTYPE"
    assert grad(ic, dy=m, s=m, ds=mat(ic, 6, 200, F32), rstd=I, dx=m) == "CONV_ERR_DTYPE"
    assert grad(ic, dy=m, s=m, rstd=I, dx=mat(ic, 6, 201)) == "CONV_ERR_SHAPE_MISMATCH"
    assert grad(ic, **ok, x=m, gate=mat(ic, 2, 200), dgate=mat(ic, 3, 200)) == "CONV_ERR_SHAPE_MISMATCH"
    big = mat(ic, 6, 24577)
    assert grad(ic, dy=big, s=big, rstd=I, dx=big) == "CONV_ERR_TOO_LARGE"
    assert grad(ic, **ok, work=None) == "CONV_ERR_WORKSPACE"
    assert grad(ic, **ok, work_bytes=256) == "CONV_ERR_WORKSPACE"
    assert grad(ic, **ok, dxp=D) == "CONV_ERR_OVERLAP"
    assert grad(ic, **ok, dskip=m, dskp=F) == "CONV_ERR_OVERLAP"
    assert grad(ic, **ok, dg=I) == "CONV_ERR_OVERLAP"


def clip(ic, tensors, most=1.0, eps=1e-6, norm_at=I, work=W, work_bytes=1 << 24):
    t = (ic.GradTensor * max(1, len(tensors)))(*[ic.GradTensor(*v) for v in tensors])
    return ic.STATUS[ic.lib().conv_clip_grads(t, len(tensors), most, eps, norm_at, work, work_bytes, None)]


def test_clip_grads_refusals(ic):
    one = (A, None, 100, F32, 0)
    assert clip(ic, [one], norm_at=None) == "CONV_ERR_NULL_PTR"
    assert clip(ic, [(None, None, 100, F32, 0)]) == "CONV_ERR_NULL_PTR"
    assert clip(ic, [(A, None, 100, 2, 0)]) == "CONV_ERR_DTYPE"
    assert clip(ic, [(A, None, 100, E4, 0)]) == "CONV_ERR_DTYPE"
    assert clip(ic, [(A, None, -1, F32, 0)]) == "CONV_ERR_BAD_PARAM"
    assert clip(ic, [(A, None, 100, F32, 1)]) == "CONV_ERR_BAD_PARAM"
    for bad in (dict(most=-1.0), dict(most=math.nan), dict(eps=-1.0), dict(eps=math.inf), dict(eps=math.nan)):
        assert clip(ic, [one], **bad) == "CONV_ERR_BAD_PARAM"
    assert clip(ic, [(A + 2, None, 100, F32, 0)]) == "CONV_ERR_ALIGNMENT"
    assert clip(ic, [one], norm_at=I + 2) == "CONV_ERR_ALIGNMENT"
    assert clip(ic, [(A, None, 1 << 45, F16, 0)]) == "CONV_ERR_TOO_LARGE"
    assert clip(ic, [one], work=None) == "CONV_ERR_WORKSPACE"
    assert clip(ic, [one], work_bytes=1024) == "CONV_ERR_WORKSPACE"
    assert clip(ic, [one, one]) == "CONV_ERR_OVERLAP"                                  # given twice
    assert clip(ic, [one, (A + 396, None, 10, F32, 0)]) == "CONV_ERR_OVERLAP"
    assert clip(ic, [(A, B, 100, F32, 0), (C, B + 64, 100, F32, 0)]) == "CONV_ERR_OVERLAP"
    assert clip(ic, [one], norm_at=A + 40) == "CONV_ERR_OVERLAP"
    assert clip(ic, [one] + [(B + 4096 * i, None, 4, F32, 0) for i in range(100)] + [one]) == "CONV_ERR_OVERLAP"


def test_definitions_against_differences():
    torch = pytest.importorskip("torch")
    from oracle import blocks as ob
    g = torch.Generator().manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float64)

    m, c, groups = 12, 20, 3
    x, skip, gate, pg, gn = normal(m, c), normal(m, c), normal(groups, c), 1 + normal(c) / 4, 1 + normal(c) / 4
    wy, ws = normal(m, c), normal(m, c)

    def loss(x, skip, gate, pg, gn):
        out = ob.block_norm(x, skip, True, pg, gate, 0.7, 0.6, gn, 1e-6)
        return float((out["y"][0] * wy).sum() + (out["sum"][0] * ws).sum())

    out = ob.block_norm(x, skip, True, pg, gate, 0.7, 0.6, gn, 1e-6)
    got = ob.block_norm_grad(wy, ws, x, out["sum"][0], True, pg, gate, groups, 0.7, 0.6, gn, out["post_rstd"][0], out["rstd"][0])
    inputs, e = [x, skip, gate, pg, gn], 1e-5
    for i, k in enumerate(("dx", "dskip", "dgate", "dpost_gain", "dgain")):
        d = normal(*inputs[i].shape)
        at = [loss(*[v + s * e * d if j == i else v for j, v in enumerate(inputs)]) for s in (1, -1)]
        assert abs((at[0] - at[1]) / (2 * e) - float((got[k][0] * d).sum())) < 1e-6, k
    q = torch.tensor([[448.0, 1.0, -3.3, 0.0]], dtype=torch.float64)
    assert ob.check_quantized(q.float().to(torch.float8_e4m3fn), torch.ones(1, 1), q, 1) is None
    wrong = q.clone()
    wrong[0, 2] = -3.0  # a step beside -3.25
    assert ob.check_quantized(wrong.float().to(torch.float8_e4m3fn), torch.ones(1, 1), q, 1) is not None
    assert ob.check_quantized(q.float().to(torch.float8_e4m3fn), torch.full((1, 1), 1.001), q, 1) is not None

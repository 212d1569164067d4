"""The channel operators on the GPU against their 64-bit definitions: sizes
from one row or channel to several tiles, odd sizes, strides, offsets and
orders, every type, activation and optional operand, empty extents, infinities
and NaN, memory on another stream, repeatability, and gradients against
differences of the operators themselves."""
import itertools

import numpy as np
import pytest

from oracle import channel as oc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
NAME = {torch.float16: "float16", torch.bfloat16: "bfloat16", torch.float32: "float32"}
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ic():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import int8_conv2d_fprop_gb300 as m
    torch.cuda.set_device(0)
    yield m
    torch.cuda.synchronize()
    assert m.device_status() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def place(v, dtype, layout="rows"):
    """The values of a float32 matrix in dtype, laid out as named; the memory
    around the elements holds NaN."""
    m, n = v.shape
    nan = float("nan")
    if layout == "rows":
        t = torch.empty(m, n, device="cuda", dtype=dtype)
    elif layout == "padded":      # rows 16-byte aligned, further apart than they are long
        t = torch.full((m, (n + 7) // 8 * 8 + 8), nan, device="cuda", dtype=dtype)[:, :n]
    elif layout == "odd":         # odd row stride
        t = torch.full((m, n + 1 + n % 2), nan, device="cuda", dtype=dtype)[:, :n]
    elif layout == "shifted":     # aligned row stride, address one element past alignment
        t = torch.full((m, (n + 7) // 8 * 8 + 8), nan, device="cuda", dtype=dtype)[:, 1:n + 1]
    elif layout == "cols":        # columns contiguous, aligned
        t = torch.full((n, (m + 7) // 8 * 8), nan, device="cuda", dtype=dtype)[:, :m].t()
    elif layout == "cols_odd":
        t = torch.full((n, m + 1 + m % 2), nan, device="cuda", dtype=dtype)[:, :m].t()
    else:                         # "spread": no contiguous dim
        t = torch.full((m, 2 * n), nan, device="cuda", dtype=dtype)[:, ::2]
    return t.copy_(v)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def check(got, want, bound, what):
    got = f64(got)
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside the bound, first at "
                           f"{tuple(int(i[0]) for i in np.nonzero(bad))}, worst {np.nanmax(np.abs(got - want) / bound):.3g}")


def run_linear(ic, m, k, n, dt=BF16, act="none", bias=True, bias_dt=None, residual=False, preact=False, out_dt=None,
               lx="rows", lw="rows", ly="rows", seed=0, scale=1.0):
    g = gen(seed + 1)
    out_dt = out_dt or dt
    x, w = place(randn(g, m, k) * scale, dt, lx), place(randn(g, n, k) / max(k, 1) ** 0.5, dt, lw)
    b = randn(g, n).to(bias_dt or dt) if bias else None
    r = place(randn(g, m, n), out_dt, ly) if residual else None
    z = place(torch.zeros(m, n, device="cuda"), dt, ly) if preact else None
    y = place(torch.zeros(m, n, device="cuda"), out_dt, ly)
    assert ic.conv_linear(x, w, b, activation=act, residual=r, preact=z, out=y) is y
    fx, fw, fb, fr = f64(x), f64(w), f64(b), f64(r)
    wy, wz = oc.linear(fx, fw, fb, act, fr)
    by, bz = oc.linear_bounds(fx, fw, fb, act, fr, wy, wz, NAME[out_dt], NAME[dt])
    check(y, wy, by, "y")
    if z is not None:
        check(z, wz, bz, "preact")
    return x, w, b, r, y


SIZES = [(1, 1, 1), (1, 8, 16), (1, 64, 128), (1, 1000, 257), (1, 4096, 512), (2, 65, 3), (7, 256, 128), (16, 512, 384),
         (17, 129, 130), (33, 64, 1), (64, 1024, 200), (100, 40, 1000), (127, 64, 64), (128, 128, 128), (129, 192, 255),
         (200, 16, 24), (255, 2048, 96), (256, 256, 256), (257, 72, 264), (300, 1, 300), (513, 520, 777),
         (1000, 333, 70), (2048, 64, 512), (5000, 96, 48),
         # few tiles and a long k: summed in runs and joined
         (300, 20488, 520), (257, 30001, 130),
         # up to four rows
         (1, 72, 64), (2, 67, 65), (3, 4096, 300), (4, 1003, 1000), (1, 8200, 67), (4, 64, 64), (5, 64, 64)]


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dt", [BF16, F16])
def test_linear_sizes(ic, m, k, n, dt):
    run_linear(ic, m, k, n, dt, "gelu", residual=True, preact=True, seed=m + k + n)


@pytest.mark.parametrize("act,dt,out", list(itertools.product(ACTS, (BF16, F16), (None, F32))))
def test_linear_activations_and_types(ic, act, dt, out):
    for m in (3, 7, 150):
        run_linear(ic, m, 200, 136, dt, act, bias_dt=F32, residual=True, preact=True, out_dt=out)
        run_linear(ic, m, 64, 40, dt, act, bias=False, out_dt=out, scale=20.0)


@pytest.mark.parametrize("bias,residual,preact", list(itertools.product((False, True), repeat=3)))
def test_linear_optional_operands(ic, bias, residual, preact):
    for m, n in ((5, 96), (260, 520)):
        run_linear(ic, m, 128, n, BF16, "silu", bias=bias, residual=residual, preact=preact)


LAYOUTS = ("rows", "padded", "odd", "shifted", "cols", "cols_odd", "spread")


@pytest.mark.parametrize("lx,lw", list(itertools.product(LAYOUTS, LAYOUTS)))
def test_linear_operand_layouts(ic, lx, lw):
    for m, k, n in ((2, 72, 136), (3, 67, 77), (5, 72, 136), (140, 136, 300), (9, 67, 45), (131, 70, 139), (260, 131, 261)):
        run_linear(ic, m, k, n, F16, "relu", lx=lx, lw=lw)


@pytest.mark.parametrize("ly", LAYOUTS)
@pytest.mark.parametrize("out", [BF16, F32])
def test_linear_output_layouts(ic, ly, out):
    for m, k, n in ((1, 64, 33), (2, 72, 133), (9, 72, 137), (140, 136, 301), (300, 64, 520)):
        run_linear(ic, m, k, n, BF16, "silu", residual=True, preact=True, ly=ly, out_dt=out)


def test_linear_writes_nothing_else(ic):
    g = gen(9)
    for m, n, ld in ((3, 30, 40), (130, 70, 72), (257, 300, 304), (257, 301, 303)):
        x, w = randn(g, m, 64).to(BF16), randn(g, n, 64).to(BF16)
        buf = torch.full((m + 2, ld), 7.0, device="cuda", dtype=BF16)
        ic.conv_linear(x, w, out=buf[1:m + 1, :n])
        keep = buf.clone()
        keep[1:m + 1, :n] = 7.0
        assert (keep == 7.0).all()
        assert not (buf[1:m + 1, :n] == 7.0).all()


def test_linear_residual_in_place_and_column_blocks(ic):
    g = gen(10)
    for m, k, n in ((4, 64, 64), (300, 128, 264)):
        x, w = randn(g, m, k).to(BF16), (randn(g, n, k) / 8).to(BF16)
        r = randn(g, m, n).to(BF16)
        want = ic.conv_linear(x, w, residual=r)
        got = r.clone()
        ic.conv_linear(x, w, residual=got, out=got)
        assert torch.equal(got, want)
        buf = torch.zeros(m, k + n, device="cuda", dtype=BF16)
        buf[:, :k] = x
        ic.conv_linear(buf[:, :k], w, residual=r, out=buf[:, k:])
        assert torch.equal(buf[:, k:], want) and torch.equal(buf[:, :k], x)


def test_linear_empty_extents(ic):
    w, b = torch.ones(5, 8, device="cuda", dtype=F16), torch.arange(5, device="cuda", dtype=F16) - 2
    assert ic.conv_linear(torch.empty(0, 8, device="cuda", dtype=F16), w, b).shape == (0, 5)
    assert ic.conv_linear(torch.ones(3, 8, device="cuda", dtype=F16), w[:0]).shape == (3, 0)
    # no products: the bias alone
    for m in (1, 3, 200):
        y = ic.conv_linear(torch.empty(m, 0, device="cuda", dtype=F16), torch.empty(5, 0, device="cuda", dtype=F16), b,
                           activation="relu")
        assert torch.equal(y, torch.relu(b).expand(m, 5))
        y = ic.conv_linear(torch.empty(m, 0, device="cuda", dtype=F16), torch.empty(5, 0, device="cuda", dtype=F16))
        assert torch.equal(y, torch.zeros(m, 5, device="cuda", dtype=F16))


def test_linear_leading_dimensions(ic):
    g = gen(11)
    x, w = randn(g, 2, 3, 5, 24).to(F16), randn(g, 10, 24).to(F16)
    y = ic.conv_linear(x, w)
    assert y.shape == (2, 3, 5, 10)
    assert torch.equal(y.view(30, 10), ic.conv_linear(x.view(30, 24), w))
    assert torch.equal(ic.conv_linear(x[0, 0, 0], w), y[0, 0, 0])
    with pytest.raises(ValueError):
        ic.conv_linear(x.transpose(0, 1), w)


def test_linear_infinities_and_nan_stay_in_their_rows(ic):
    g = gen(12)
    for m in (3, 200):
        x, w = randn(g, m, 100).to(BF16), randn(g, 140, 100).to(BF16)
        clean = ic.conv_linear(x, w, activation="relu")
        x[1, 5], x[m - 1, 99] = float("nan"), float("inf")
        y = ic.conv_linear(x, w, activation="relu")
        assert torch.isnan(y[1]).all()
        assert torch.equal(y[2:m - 1], clean[2:m - 1]) and torch.equal(y[0], clean[0])
        assert torch.equal(y[m - 1], torch.where(w[:, 99] > 0, float("inf"), 0.0).to(BF16))
        # a weight's infinity stays in its column
        x[1, 5], x[m - 1, 99] = 0.5, 0.5
        base = ic.conv_linear(x, w)
        w[7, 3] = float("inf")
        y = ic.conv_linear(x, w)
        assert torch.isinf(y[x[:, 3] != 0, 7]).all()
        y[:, 7] = base[:, 7]
        assert torch.equal(y, base)


def test_linear_f16_overflow_is_infinity(ic):
    x, w = torch.full((2, 64), 200.0, device="cuda", dtype=F16), torch.full((64, 64), 200.0, device="cuda", dtype=F16)
    assert torch.isinf(ic.conv_linear(x, w)).all()
    out = torch.empty(2, 64, device="cuda", dtype=F32)
    assert (ic.conv_linear(x, w, out=out) == 64 * 40000.0).all()


def test_linear_repeats_bit_for_bit_and_on_other_streams(ic):
    g = gen(13)
    side = torch.cuda.Stream()
    for m, k, n, ld in ((1, 4096, 512, 0), (64, 2048, 640, 1), (700, 1024, 900, 0), (512, 8192, 256, 3)):
        x, w = randn(g, m, k + ld).to(BF16)[:, :k], randn(g, n, k).to(BF16)
        first = ic.conv_linear(x, w, activation="silu")
        for _ in range(3):
            assert torch.equal(ic.conv_linear(x, w, activation="silu"), first)
        torch.cuda.synchronize()
        outs = [ic.conv_linear(x, w, activation="silu", stream=side) for _ in range(4)]
        # memory of the current stream that the side stream's calls must not be given
        junk = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(4)]
        side.synchronize()
        assert all(torch.equal(o, first) for o in outs) and len(junk) == 4


def test_linear_graph_capture(ic):
    g = gen(14)
    x, w = randn(g, 96, 512).to(BF16), randn(g, 384, 512).to(BF16)
    y = torch.empty(96, 384, device="cuda", dtype=BF16)
    want = ic.conv_linear(x, w, activation="gelu").clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ic.conv_linear(x, w, activation="gelu", out=y)
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


# ------------------------------------------------------------ linear, backward
def run_linear_grad(ic, m, k, n, dt=BF16, act="none", types=(None, None, F32), layouts=("rows",) * 4, seed=0):
    g = gen(seed + 2)
    x, w = place(randn(g, m, k), dt, layouts[0]), place(randn(g, n, k) / k ** 0.5, dt, layouts[1])
    dy = place(randn(g, m, n) / 8, dt, layouts[2])
    z = None if act == "none" else place(randn(g, m, n) * 2, dt, layouts[2])
    dx = place(torch.zeros(m, k, device="cuda"), types[0] or dt, layouts[3])
    dw = place(torch.zeros(n, k, device="cuda"), types[1] or dt, layouts[3])
    db = torch.zeros(n, device="cuda", dtype=types[2] or dt)
    ic.conv_linear_grad(dy, x, w, preact=z, activation=act, dx=dx, dw=dw, dbias=db)
    fdy, fx, fw = f64(dy), f64(x), f64(w)
    *want, fdz = oc.linear_grad(fdy, fx, fw, f64(z), act)
    bounds = oc.linear_grad_bounds(fdz, fx, fw, fdy, act, want, [NAME[t.dtype] for t in (dx, dw, db)], NAME[dt])
    for got, v, b, what in zip((dx, dw, db), want, bounds, ("dx", "dw", "dbias")):
        check(got, v, b, what)


GRAD_SIZES = [(1, 1, 1), (1, 64, 40), (2, 200, 8), (9, 8, 9), (31, 65, 33), (64, 64, 64), (128, 256, 128),
              (130, 70, 257), (333, 192, 257), (512, 24, 520), (1000, 128, 64), (4099, 64, 72), (700, 600, 500), (20011, 512, 520),
              # a last round of tiles cut into runs
              (5130, 2100, 2568)]


@pytest.mark.parametrize("m,k,n", GRAD_SIZES)
@pytest.mark.parametrize("dt,act", [(BF16, "none"), (F16, "none"), (BF16, "gelu"), (F16, "relu")])
def test_linear_grad_sizes(ic, m, k, n, dt, act):
    run_linear_grad(ic, m, k, n, dt, act, seed=m * 3 + k + n)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("types", [(None, None, None), (F32, F32, F32)])
def test_linear_grad_activations_and_types(ic, act, types):
    for dt in (BF16, F16):
        run_linear_grad(ic, 150, 136, 200, dt, act, types)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("which", range(4))
def test_linear_grad_layouts(ic, layout, which):
    layouts = ["rows"] * 4
    layouts[which] = layout
    for act in ("none", "silu"):
        run_linear_grad(ic, 75, 72, 137, F16, act, layouts=layouts)
        run_linear_grad(ic, 133, 139, 69, F16, act, layouts=layouts)
        run_linear_grad(ic, 264, 136, 144, BF16, act, layouts=layouts)


@pytest.mark.parametrize("want", [w for w in itertools.product((False, True), repeat=3) if any(w)])
def test_linear_grad_any_subset(ic, want):
    g = gen(20)
    x, w, dy, z = randn(g, 70, 96).to(BF16), randn(g, 50, 96).to(BF16), randn(g, 70, 50).to(BF16), randn(g, 70, 50).to(BF16)
    full = [torch.empty_like(x), torch.empty_like(w), torch.empty(50, device="cuda")]
    ic.conv_linear_grad(dy, x, w, preact=z, activation="gelu", dx=full[0], dw=full[1], dbias=full[2])
    part = [torch.empty_like(t) if k else None for t, k in zip(full, want)]
    ic.conv_linear_grad(dy, x, w, preact=z, activation="gelu", dx=part[0], dw=part[1], dbias=part[2])
    for a, b in zip(full, part):
        assert b is None or torch.equal(a, b)


def test_linear_grad_empty_extents(ic):
    x, w, dy = (torch.ones(s, device="cuda", dtype=F16) for s in ((0, 24), (10, 24), (0, 10)))
    dw, db = torch.full((10, 24), 5.0, device="cuda", dtype=F16), torch.full((10,), 5.0, device="cuda")
    ic.conv_linear_grad(dy, x, w, dx=torch.empty_like(x), dw=dw, dbias=db)
    assert not dw.any() and not db.any()
    x, w, dy = (torch.ones(s, device="cuda", dtype=F16) for s in ((30, 24), (0, 24), (30, 0)))
    dx = torch.full((30, 24), 5.0, device="cuda", dtype=F16)
    ic.conv_linear_grad(dy, x, w, dx=dx, dw=torch.empty_like(w), dbias=torch.empty(0, device="cuda"))
    assert not dx.any()


@pytest.mark.parametrize("act", ACTS)
def test_linear_grad_is_the_difference_quotient(ic, act):
    """The operator's own forward, with float32 outputs, moved by h along a
    direction v of 0 and +-1 in x and in w (all values multiples of 2^-6, so
    that x +- h v is exact): the central difference is off by h^2/6 times the
    third derivative along v (|act'''| <= 2 by |dy| |dz|^3) and by the
    forward's 32-bit rounding over h; the gradients by their bounds.  ReLU's
    corner is kept out by an odd multiple of 2^-13 in the bias, with only one
    input moved at a time."""
    g = gen(30)
    m, k, n, h = 24, 16, 20, 2.0 ** -6
    x, w = ((randn(g, *s) * 16).round() / 64 for s in ((m, k), (n, k)))
    b = (randn(g, n) * 64).round() / 64 + 2.0 ** -13
    dy = (randn(g, m, n) * 16).round() / 64
    f = lambda a, c: ic.conv_linear(a.to(F16), c.to(F16), b, activation=act, out=torch.empty(m, n, device="cuda"))  # noqa: E731
    z = torch.empty(m, n, device="cuda", dtype=F16)
    ic.conv_linear(x.to(F16), w.to(F16), b, activation=act, preact=z, out=torch.empty(m, n, device="cuda"))
    dx, dw = torch.empty(m, k, device="cuda"), torch.empty(n, k, device="cuda")
    ic.conv_linear_grad(dy.to(F16), x.to(F16), w.to(F16), preact=z, activation=act, dx=dx, dw=dw)
    for i in range(6):
        for which in (0, 1):
            v = torch.zeros_like((x, w)[which])
            col = (5 * i + 3) % k
            v[:, col] = torch.randint(-1, 2, (v.shape[0],), generator=g, device="cuda").float()
            if act == "relu":
                # keep the pieces linear: only outputs whose sign is the same on both sides
                up, dn = (f(x + s * v, w) if which == 0 else f(x, w + s * v) for s in (h, -h))
                same = (up > 0) == (dn > 0)
                c = torch.where(same, dy, 0)
                gx, gw = torch.empty_like(dx), torch.empty_like(dw)
                ic.conv_linear_grad(c.to(F16), x.to(F16), w.to(F16), preact=z, activation=act, dx=gx, dw=gw)
            else:
                up, dn = (f(x + s * v, w) if which == 0 else f(x, w + s * v) for s in (h, -h))
                c, gx, gw = dy, dx, dw
            quotient = float((c.double() * (up.double() - dn.double())).sum() / (2 * h))
            gradient = float(((gx, gw)[which].double() * v.double()).sum())
            # |dz| along v: |w| (or |x|) of the moved column
            step = (w[:, col].abs().double()[None, :].expand(m, n) if which == 0
                    else x[:, col].abs().double()[:, None].expand(m, n))
            third = 0.0 if act in ("none", "relu") else float((c.abs().double() * step ** 3).sum()) * 2 * h * h / 6
            rounding = float((c.abs().double() * (up.abs() + dn.abs() + 1).double()).sum()) * 2.0 ** -19 / (2 * h)
            # z and dz are held in 16 bits: |act''| <= 1.2
            stored = float((c.abs().double() * step).sum()) * (2.0 ** -10 + 1.2 * 2.0 ** -11 * float(z.abs().max()))
            assert abs(quotient - gradient) <= third + rounding + stored, (i, which, quotient, gradient)


# ------------------------------------------------------------------ layer norm
def norm_input(g, m, c, dt, layout="rows"):
    v = randn(g, m, c) * (0.5 + torch.rand(m, 1, generator=g, device="cuda")) + randn(g, m, 1)
    if dt == torch.int32:
        v = (v * 40000).round()
        if layout != "rows":
            t = torch.full((m, c + 3), 12345, device="cuda", dtype=dt)[:, :c]
            return t.copy_(v)
        return v.to(dt)
    return place(v, dt, layout)


def run_norm(ic, m, c, dt, out=None, affine=True, p_dt=F32, layout="rows", seed=0, eps=1e-5):
    g = gen(seed + 3)
    out = out or (F32 if dt == torch.int32 else dt)
    x = norm_input(g, m, c, dt, layout)
    gain, shift = ((1 + 0.2 * randn(g, c)).to(p_dt), randn(g, c).to(p_dt)) if affine else (None, None)
    scale = 2.0 ** -14 if dt == torch.int32 else 1.0
    y = place(torch.zeros(m, c, device="cuda"), out, layout)
    mean, rstd = torch.zeros(m, device="cuda"), torch.zeros(m, device="cuda")
    ic.conv_layer_norm(x, gain, shift, eps=eps, scale=scale, out=y, mean=mean, rstd=rstd)
    fx, fg, fs = f64(x), f64(gain), f64(shift)
    eps = float(np.float32(eps))
    want = oc.layer_norm(fx, fg, fs, eps, scale)
    bounds = oc.layer_norm_bounds(fx, fg, fs, eps, scale, *want, NAME[out])
    for got, v, b, what in zip((y, mean, rstd), want, bounds, ("y", "mean", "rstd")):
        check(got, v, b, what)


NORM_SIZES = [(1, 1), (1, 2), (3, 7), (1, 64), (5, 32), (2, 33), (17, 100), (4, 256), (9, 257), (300, 192), (2, 511),
              (33, 512), (3, 1000), (2, 1024), (3, 1025), (5, 2047), (2, 4096), (3, 5001), (2, 8192), (1, 16384),
              (2, 16391), (1, 65536), (1, 70001), (5000, 64)]


@pytest.mark.parametrize("m,c", NORM_SIZES)
@pytest.mark.parametrize("dt,out", [(BF16, None), (F16, None), (F32, None), (torch.int32, BF16), (BF16, F32)])
def test_layer_norm_sizes(ic, m, c, dt, out):
    run_norm(ic, m, c, dt, out, seed=m + c)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dt", [BF16, F32, torch.int32])
def test_layer_norm_layouts(ic, layout, dt):
    for m, c in ((5, 40), (130, 257), (3, 1032), (2, 4104)):
        run_norm(ic, m, c, dt, layout=layout)
        run_norm(ic, m, c, dt, affine=False, layout=layout)


@pytest.mark.parametrize("dt,out", [(BF16, BF16), (F16, F16), (F16, F32), (F32, F16), (torch.int32, F16)])
def test_layer_norm_parameters_in_the_output_type(ic, dt, out):
    for c in (96, 101, 3000):
        run_norm(ic, 6, c, dt, out, p_dt=out)


def test_layer_norm_constant_rows_and_non_finite_rows(ic):
    for c in (1, 40, 513, 9000):
        x = torch.randn(4, c, device="cuda")
        x[0], x[3] = 3.0, 0.0
        clean = ic.conv_layer_norm(x)
        assert not clean[0].any() and not clean[3].any()  # no deviation: the shift, here 0
        x[1, c - 1], x[2, 0] = float("inf"), float("nan")
        y = ic.conv_layer_norm(x)
        assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
        assert torch.equal(y[0], clean[0]) and torch.equal(y[3], clean[3])


def test_layer_norm_far_from_zero(ic):
    # a mean of 1000 deviations: the variance comes from differences, not squares
    g = gen(40)
    for c in (64, 768, 6000):
        x = randn(g, 4, c) + 1000
        y = torch.empty_like(x)
        ic.conv_layer_norm(x, out=y)
        want = oc.layer_norm(f64(x))
        check(y, want[0], oc.layer_norm_bounds(f64(x), None, None, 1e-5, 1.0, *want, "float32")[0], "y")


def test_layer_norm_in_place_and_empty(ic):
    g = gen(41)
    for c in (96, 1027, 20000):
        x = randn(g, 5, c)
        want = ic.conv_layer_norm(x)
        ic.conv_layer_norm(x, out=x)
        assert torch.equal(x, want)
    assert ic.conv_layer_norm(torch.empty(0, 8, device="cuda")).shape == (0, 8)
    with pytest.raises(ic.ConvError):
        ic.conv_layer_norm(torch.empty(3, 0, device="cuda"))


def test_layer_norm_takes_the_convolutions_accumulators(ic):
    import synth
    cfg = synth.ConvConfig("norm_link", 2, 64, 10, 9, 48, 3, 3, pre=(1, 1), post=(1, 1), seed=5)
    x, w, _ = synth.make_inputs(cfg)
    xt = torch.from_numpy(x).cuda().contiguous(memory_format=torch.channels_last)
    wt = torch.from_numpy(w).cuda().contiguous(memory_format=torch.channels_last)
    acc = ic.conv_fprop(xt, wt, pre_padding=(1, 1), post_padding=(1, 1))  # channels last
    rows = acc.permute(0, 2, 3, 1)
    y = ic.conv_layer_norm(rows, scale=2.0 ** -12, out=torch.empty(rows.shape, device="cuda", dtype=BF16))
    f = f64(rows.reshape(-1, 48))
    want = oc.layer_norm(f, scale=2.0 ** -12, eps=float(np.float32(1e-5)))
    check(y.reshape(-1, 48), want[0], oc.layer_norm_bounds(f, None, None, 1e-5, 2.0 ** -12, *want, "bfloat16")[0], "y")


def run_norm_grad(ic, m, c, dt, p_dt=F32, gain=True, residual=False, layout="rows", seed=0):
    g = gen(seed + 4)
    x, dy = norm_input(g, m, c, dt, layout), place(randn(g, m, c) / 4, dt, layout)
    ga = (1 + 0.3 * randn(g, c)).to(p_dt) if gain else None
    r = place(randn(g, m, c) / 4, dt, layout) if residual else None
    _, mean, rstd = oc.layer_norm(f64(x))
    mean, rstd = (torch.from_numpy(v.astype(np.float32)).cuda() for v in (mean, rstd))
    dx = place(torch.zeros(m, c, device="cuda"), dt, layout)
    dg, db = torch.zeros(c, device="cuda", dtype=p_dt), torch.zeros(c, device="cuda", dtype=p_dt)
    ic.conv_layer_norm_grad(dy, x, ga, mean, rstd, residual_grad=r, dx=dx, dgain=dg, dshift=db)
    args = [f64(v) for v in (dy, x, ga, mean, rstd, r)]
    want = oc.layer_norm_grad(*args)
    bounds = oc.layer_norm_grad_bounds(*args, want, NAME[dt], NAME[p_dt])
    for got, v, b, what in zip((dx, dg, db), want, bounds, ("dx", "dgain", "dshift")):
        check(got, v, b, what)


@pytest.mark.parametrize("m,c", NORM_SIZES)
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_layer_norm_grad_sizes(ic, m, c, dt):
    run_norm_grad(ic, m, c, dt, residual=bool(c % 2), seed=m + c)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dt", [F16, F32])
def test_layer_norm_grad_layouts(ic, layout, dt):
    for m, c in ((5, 40), (130, 257), (3, 1032), (2, 4104)):
        run_norm_grad(ic, m, c, dt, layout=layout, residual=True)
        run_norm_grad(ic, m, c, dt, layout=layout, gain=False)


@pytest.mark.parametrize("dt", [BF16, F16])
def test_layer_norm_grad_parameters_in_the_rows_type(ic, dt):
    for c in (96, 101, 3000):
        run_norm_grad(ic, 40, c, dt, p_dt=dt)


@pytest.mark.parametrize("want", [w for w in itertools.product((False, True), repeat=3) if any(w)])
def test_layer_norm_grad_any_subset(ic, want):
    g = gen(50)
    for m, c in ((70, 96), (9, 3000), (3, 40000)):
        x, dy, gain = randn(g, m, c), randn(g, m, c), randn(g, c)
        mean, rstd = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
        ic.conv_layer_norm(x, mean=mean, rstd=rstd)
        full = [torch.empty_like(x), torch.empty_like(gain), torch.empty_like(gain)]
        ic.conv_layer_norm_grad(dy, x, gain, mean, rstd, dx=full[0], dgain=full[1], dshift=full[2])
        part = [torch.empty_like(t) if k else None for t, k in zip(full, want)]
        ic.conv_layer_norm_grad(dy, x, gain, mean, rstd, dx=part[0], dgain=part[1], dshift=part[2])
        for a, b in zip(full, part):
            assert b is None or torch.equal(a, b)


def test_layer_norm_grad_in_place_empty_and_repeated(ic):
    g = gen(51)
    for m, c in ((2000, 128), (50, 2000), (3, 30000)):
        x, dy, gain, r = randn(g, m, c), randn(g, m, c), randn(g, c), randn(g, m, c)
        mean, rstd = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
        ic.conv_layer_norm(x, mean=mean, rstd=rstd)
        outs = []
        for _ in range(3):
            dx, dg, db = torch.empty_like(x), torch.empty_like(gain), torch.empty_like(gain)
            ic.conv_layer_norm_grad(dy, x, gain, mean, rstd, residual_grad=r, dx=dx, dgain=dg, dshift=db)
            outs.append((dx, dg, db))
        for o in outs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
        ic.conv_layer_norm_grad(dy, x, gain, mean, rstd, residual_grad=r, dx=r)
        assert torch.equal(r, outs[0][0])
    e = torch.empty(0, 16, device="cuda")
    dg, db = torch.ones(16, device="cuda"), torch.ones(16, device="cuda")
    s = torch.empty(0, device="cuda")
    ic.conv_layer_norm_grad(e, e, None, s, s, dx=torch.empty_like(e), dgain=dg, dshift=db)
    assert not dg.any() and not db.any()


def test_layer_norm_grad_is_the_difference_quotient(ic):
    """Central differences of the forward operator in float32 along random
    directions of x, gain and shift: off by h^2 times the third derivative
    along v (below 64 |dy| |v|^3 rstd^3 C for these well-scaled rows) and by
    the forward's rounding over h."""
    g = gen(52)
    m, c, h = 6, 48, 2.0 ** -7
    x, dy, gain, shift = randn(g, m, c), randn(g, m, c), 1 + 0.2 * randn(g, c), randn(g, c)
    mean, rstd = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    ic.conv_layer_norm(x, gain, shift, mean=mean, rstd=rstd)
    grads = [torch.empty_like(t) for t in (x, gain, shift)]
    ic.conv_layer_norm_grad(dy, x, gain, mean, rstd, dx=grads[0], dgain=grads[1], dshift=grads[2])
    at = [x, gain, shift]
    for which in range(3):
        for _ in range(4):
            v = torch.zeros_like(at[which]).view(-1)
            v[torch.randint(0, v.numel(), (3,), generator=g, device="cuda")] = 1.0
            v = v.view_as(at[which])
            f = []
            for s in (h, -h):
                moved = list(at)
                moved[which] = at[which] + s * v
                f.append(ic.conv_layer_norm(*moved).double())
            quotient = float((dy.double() * (f[0] - f[1])).sum() / (2 * h))
            gradient = float((grads[which].double() * v.double()).sum())
            cut = 64 * h * h * float(dy.abs().sum(1).max() * rstd.max() ** 3) if which == 0 else 0.0
            rounding = float((dy.abs().double() * (f[0].abs() + 4)).sum()) * 2.0 ** -20 / (2 * h)
            assert abs(quotient - gradient) <= cut + rounding + 2.0 ** -18 * abs(gradient)


# ---------------------------------------------------------------- together
def test_convolution_and_channel_block(ic):
    """The example's block against float32 autograd: every stored tensor on the
    way is rounded to bfloat16 (2^-9 of its norm at random), and a gradient has
    at most six such tensors behind it."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import channel_block
    for shape in ((2, 64, 14, 96, 384), (1, 32, 9, 40, 136)):
        for name, far in channel_block.compare(*shape).items():
            assert far < 6 * 2.0 ** -8, (name, far)


def test_offsets_beyond_32_bits(ic):
    """Rows 2^31 + 16 elements apart: byte offsets pass 32 bits and element
    offsets pass 31."""
    ld, m, c = (1 << 31) + 16, 3, 72
    buf = torch.empty((m - 1) * ld + 4096, device="cuda", dtype=BF16)
    x = buf.as_strided((m, c), (ld, 1))
    out = torch.empty((m - 1) * ld + 4096, device="cuda", dtype=BF16).as_strided((m, 104), (ld, 1))
    g = gen(60)
    v, w = randn(g, m, c).to(BF16), randn(g, 104, c).to(BF16)
    x.copy_(v)
    assert torch.equal(ic.conv_linear(x, w, out=out), ic.conv_linear(v, w))
    many = torch.empty(200, c, device="cuda", dtype=BF16)
    many[:] = v[1]
    assert torch.equal(ic.conv_linear(many, w)[0], ic.conv_linear(torch.cat([v, many]), w)[1])
    y = out[:, :c]
    assert torch.equal(ic.conv_layer_norm(x, out=y), ic.conv_layer_norm(v))
    mean, rstd = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    ic.conv_layer_norm(v, mean=mean, rstd=rstd)
    dy = randn(g, m, c).to(BF16)
    a, b = [torch.empty_like(v)] + [torch.empty(c, device="cuda") for _ in range(2)], torch.empty(c, device="cuda")
    ic.conv_layer_norm_grad(dy, v, None, mean, rstd, dx=a[0], dgain=a[1], dshift=a[2])
    ic.conv_layer_norm_grad(dy, x, None, mean, rstd, dx=y, dgain=b)
    assert torch.equal(y, a[0]) and torch.equal(b, a[1])
    dx, dw = out[:, :c], torch.empty_like(w)
    dz = randn(g, m, 104).to(BF16)
    ic.conv_linear_grad(dz, x, w, dx=dx, dw=dw)
    want = torch.empty_like(v), torch.empty_like(w)
    ic.conv_linear_grad(dz, v, w, dx=want[0], dw=want[1])
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])

"""The forms of the channel operators' kernels that a size selects, each with
every epilogue: products on tiles of CTA pairs and on wide single tiles, sums
cut into runs and shared by clusters, norms whose blocks take several rows."""
import itertools
import math

import channel_sizes as sizes
import numpy as np
import pytest

from oracle import channel as oc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
NAME = {F16: "float16", BF16: "bfloat16", F32: "float32"}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


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
    """The values in dtype, in rows as long as they are ("rows"), a multiple of 8
    elements apart ("padded"), an odd number apart ("odd"), one element past
    alignment ("shifted"), or in columns ("cols")."""
    m, n = v.shape
    nan = float("nan")
    if layout == "padded":
        t = torch.full((m, (n + 7) // 8 * 8 + 8), nan, device="cuda", dtype=dtype)[:, :n]
    elif layout == "odd":
        t = torch.full((m, n + 1 + n % 2), nan, device="cuda", dtype=dtype)[:, :n]
    elif layout == "shifted":
        t = torch.full((m, (n + 7) // 8 * 8 + 8), nan, device="cuda", dtype=dtype)[:, 1:n + 1]
    elif layout == "cols":
        t = torch.full((n, (m + 7) // 8 * 8), nan, device="cuda", dtype=dtype)[:, :m].t()
    else:
        t = torch.empty(m, n, device="cuda", dtype=dtype)
    return t.copy_(v)


def check(got, want, bound, what):
    far = (got.double() - want).abs()
    bad = ~(far <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, worst {float((far / bound).max()):.3g}"


# ------------------------------------------------------- products, every epilogue
def activate64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def run_linear(ic, m, k, n, dt, act, out, residual, preact, ly, lx="rows", lw="rows"):
    g = gen(m + n)
    x, w = place(randn(g, m, k), dt, lx), place(randn(g, n, k) / k ** 0.5, dt, lw)
    b = randn(g, n)
    r = place(randn(g, m, n), out, ly) if residual else None
    z = place(torch.zeros(m, n, device="cuda"), dt, ly) if preact else None
    y = place(torch.zeros(m, n, device="cuda"), out, ly)
    ic.conv_linear(x, w, b, activation=act, residual=r, preact=z, out=y)
    fz = x.double() @ w.double().t() + b.double()
    fy = activate64(fz, act)
    # the oracle's bounds (oracle/channel.py: linear_bounds), for these short sums
    ez = (k + 2) * 2.0 ** -23 * (x.double().abs() @ w.double().abs().t() + b.double().abs())
    ey = ez if act == "none" else 1.2 * ez + 2.0 ** -20 * fz.abs()
    if residual:
        fy, ey = fy + r.double(), ey + 2.0 ** -23 * r.double().abs()
    check(y, fy, ey + oc.UNIT[NAME[out]] * (fy.abs() + ey) + oc.TINY[NAME[out]], "y")
    if preact:
        check(z, fz, ez + oc.UNIT[NAME[dt]] * (fz.abs() + ez) + oc.TINY[NAME[dt]], "preact")


WIDE = sizes.PAIR_TILES + sizes.WIDE_SINGLE_TILES


@pytest.mark.parametrize("size", WIDE)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt,out", [(BF16, BF16), (F16, F16), (BF16, F32)])
def test_wide_tiles_every_activation(ic, size, act, dt, out):
    run_linear(ic, *size, dt, act, out, True, True, "rows")


@pytest.mark.parametrize("size", WIDE)
@pytest.mark.parametrize("ly", ["padded", "odd", "shifted", "cols"])
@pytest.mark.parametrize("out", [F16, F32])
def test_wide_tiles_output_layouts(ic, size, ly, out):
    run_linear(ic, *size, F16, "silu", out, True, True, ly)


@pytest.mark.parametrize("size", WIDE)
@pytest.mark.parametrize("residual,preact", list(itertools.product((False, True), repeat=2)))
def test_wide_tiles_optional_operands(ic, size, residual, preact):
    run_linear(ic, *size, BF16, "gelu", BF16, residual, preact, "rows")


@pytest.mark.parametrize("size", WIDE)
@pytest.mark.parametrize("lx,lw", [("cols", "rows"), ("rows", "cols"), ("odd", "cols"), ("cols", "odd")])
def test_wide_tiles_operand_orders(ic, size, lx, lw):
    run_linear(ic, *size, F16, "relu", F16, True, False, "rows", lx, lw)


def test_wide_tiles_write_nothing_else(ic):
    g = gen(3)
    for m, k, n in WIDE:
        x, w, r = randn(g, m, k).to(BF16), randn(g, n, k).to(BF16), randn(g, m, n).to(BF16)
        buf = torch.full((m + 2, (n + 7) // 8 * 8 + 16), 7.0, device="cuda", dtype=BF16)
        out = buf[1:m + 1, 8:n + 8]
        ic.conv_linear(x, w, residual=r, out=out)
        assert torch.equal(out, ic.conv_linear(x, w, residual=r))
        out.fill_(7.0)
        assert bool((buf == 7.0).all())


# ------------------------------------------------ sums: no term lost, none twice
def whole(g, *shape, dtype=BF16):
    return torch.randint(-3, 4, shape, generator=g, device="cuda").to(dtype)


SUMS = sizes.JOINED_RUNS + sizes.CUT_LAST_ROUND + [s for _, s in sizes.CLUSTERS] + sizes.FEW_ROWS + WIDE


@pytest.mark.parametrize("size", SUMS)
@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("lx,lw", [("rows", "rows"), ("cols", "cols"), ("odd", "shifted")])
def test_sums_of_integers_are_exact(ic, size, dt, lx, lw):
    """Whole numbers up to 3: every partial sum is below 2^24, so 32-bit sums in
    any order are exact, and one term lost or taken twice is seen."""
    m, k, n = size
    g = gen(m + k + n)
    x, w, b = place(whole(g, m, k), dt, lx), place(whole(g, n, k), dt, lw), whole(g, n)
    r, z, y = whole(g, m, n, dtype=F32), torch.empty(m, n, device="cuda", dtype=dt), torch.empty(m, n, device="cuda")
    ic.conv_linear(x, w, b.to(dt), activation="relu", residual=r, preact=z, out=y)
    want = x.double() @ w.double().t() + b.double()
    assert float(want.abs().max()) > 8  # (the sums are no handful of zeros)
    assert torch.equal(y.double(), want.clamp(min=0) + r.double())
    assert torch.equal(z, want.to(dt))
    assert torch.equal(ic.conv_linear(x, w, out=y).double(), want - b.double())


@pytest.mark.parametrize("m,k,n", [(20011, 512, 520), (50176, 256, 1024), (30008, 130, 300), (5130, 2100, 2568),
                                   (333, 192, 257), (4097, 64, 64), (20000, 40, 72), (3, 2000, 3000), (700, 8, 16400),
                                   # extents of one
                                   (1, 1, 1), (1, 70, 1), (1, 1, 70), (700, 1, 1), (700, 70, 1), (700, 1, 70), (2, 1, 3)])
@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("layout", ["rows", "odd", "cols"])
def test_gradient_sums_of_integers_are_exact(ic, m, k, n, act, layout):
    g = gen(m + k + n)
    x, w, dy = place(whole(g, m, k), BF16, layout), place(whole(g, n, k), BF16, layout), place(whole(g, m, n), BF16, layout)
    z = place(whole(g, m, n), BF16, layout) if act == "relu" else None
    dx, dw, db = torch.empty(m, k, device="cuda"), torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    ic.conv_linear_grad(dy, x, w, preact=z, activation=act, dx=dx, dw=dw, dbias=db)
    dz = dy.double() if z is None else dy.double() * (z > 0)
    assert torch.equal(dx.double(), dz @ w.double())
    assert torch.equal(dw.double(), dz.t() @ x.double())
    assert torch.equal(db.double(), dz.sum(0))


# ------------------------------------------- norms: several rows to a block or warp
ROWS = [(5003, 200), (3001, 505), (3001, 1032), (1201, 1500), (1001, 5001), (650, 8192), (650, 10001)]


def norm_rows(g, m, c):
    return randn(g, m, c) * (0.5 + torch.rand(m, 1, generator=g, device="cuda")) + randn(g, m, 1)


@pytest.mark.parametrize("m,c", ROWS)
@pytest.mark.parametrize("dt,out", [(F16, F16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("lx,ly", [("rows", "rows"), ("odd", "odd"), ("odd", "padded"), ("padded", "shifted")])
def test_layer_norm_rows_one_after_another(ic, m, c, dt, out, lx, ly):
    g = gen(m + c)
    x, gain, shift = place(norm_rows(g, m, c), dt, lx), 1 + 0.2 * randn(g, c), randn(g, c)
    y, mean, rstd = place(torch.zeros(m, c, device="cuda"), out, ly), torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    ic.conv_layer_norm(x, gain, shift, out=y, mean=mean, rstd=rstd)
    eps = float(np.float32(1e-5))
    fx, fg, fs = (t.double().cpu().numpy() for t in (x, gain, shift))
    want = oc.layer_norm(fx, fg, fs, eps)
    bounds = oc.layer_norm_bounds(fx, fg, fs, eps, 1.0, *want, NAME[out])
    for got, v, b, what in zip((y, mean, rstd), want, bounds, ("y", "mean", "rstd")):
        check(got, torch.from_numpy(v).cuda(), torch.from_numpy(b).cuda(), what)


@pytest.mark.parametrize("m,c", ROWS)
@pytest.mark.parametrize("dt", [F16, F32])
# of x, dy, residual, dx: alike; odd; dx turned (its rows at another lead); the rows read at several leads
@pytest.mark.parametrize("layouts", [("rows",) * 4, ("odd",) * 4, ("padded", "padded", "padded", "odd"),
                                     ("odd", "odd", None, "rows"), ("odd", "padded", "rows", "shifted"),
                                     ("padded", "shifted", None, "padded")])
def test_layer_norm_grad_rows_one_after_another(ic, m, c, dt, layouts):
    g = gen(m + c)
    lx, ly, lr, ld = layouts
    x, dy = place(norm_rows(g, m, c), dt, lx), place(randn(g, m, c) / 4, dt, ly)
    r = place(randn(g, m, c) / 4, dt, lr) if lr else None
    gain, dx = 1 + 0.3 * randn(g, c), place(torch.zeros(m, c, device="cuda"), dt, ld)
    f = x.double()
    mean, rstd = f.mean(1).float(), (f.var(1, unbiased=False) + 1e-5).rsqrt().float()
    dg, db = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    ic.conv_layer_norm_grad(dy, x, gain, mean, rstd, residual_grad=r, dx=dx, dgain=dg, dshift=db)
    args = [None if t is None else t.double().cpu().numpy() for t in (dy, x, gain, mean, rstd, r)]
    want = oc.layer_norm_grad(*args)
    bounds = oc.layer_norm_grad_bounds(*args, want, NAME[dt], "float32", centred=True)
    for got, v, b, what in zip((dx, dg, db), want, bounds, ("dx", "dgain", "dshift")):
        check(got, torch.from_numpy(v).cuda(), torch.from_numpy(b).cuda(), what)


@pytest.mark.parametrize("m,c", ROWS)
def test_layer_norm_grad_sums_of_integers_are_exact(ic, m, c):
    """Whole x and dy, mean 0 and rstd 1: dgain and dshift are exact in 32 bits,
    and a row lost or taken twice is seen."""
    g = gen(m)
    for layout in ("rows", "odd"):
        x, dy = place(whole(g, m, c), F16, layout), place(whole(g, m, c), F16, layout)
        mean, rstd = torch.zeros(m, device="cuda"), torch.ones(m, device="cuda")
        dg, db = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
        ic.conv_layer_norm_grad(dy, x, None, mean, rstd, dx=torch.empty_like(x), dgain=dg, dshift=db)
        assert torch.equal(dg.double(), (dy.double() * x.double()).sum(0))
        assert torch.equal(db.double(), dy.double().sum(0))

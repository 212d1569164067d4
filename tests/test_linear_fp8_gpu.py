"""conv_linear_fp8 on the GPU against its definition in 64 bits: sizes from one
row to several tiles and cut sums, types, scale kinds and strides, epilogues,
layouts, exact sums, NaN, empty extents, graphs, repeatability, and the
gradients of a layer by products of the same kind."""
import itertools

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import blocks as ob  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
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


def operand(seed, rows, k, dtype=E4, tile=1, layout="aligned", scales="columns"):
    """8-bit values and positive scales as they come, not from a quantisation."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = (torch.randn(rows, k, generator=g, device="cuda") * 40).clamp(-448, 448).to(dtype)
    s = torch.exp(torch.randn(-(-rows // tile), ob.blocks(k), generator=g, device="cuda")) / 100
    pad = {"aligned": (k + 15) // 16 * 16, "wide": (k + 15) // 16 * 16 + 32, "odd": k + 1 + k % 2, "tight": k}[layout]
    t = torch.full((rows * pad + 16,), 0x7f, dtype=torch.uint8, device="cuda").view(dtype)  # NaN around the values
    t = t[1 if layout == "odd" else 0:][:rows * pad].view(rows, pad)[:, :k]
    t.copy_(v)
    if scales == "columns":
        s = s.t().contiguous().t()
    elif scales == "spread":
        s = s.repeat_interleave(3, 0).repeat_interleave(2, 1)[::3, ::2]
    return t, s


def check(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at "
                                 f"{bad.nonzero()[0].tolist()}, worst {float(((got.double() - want).abs() / bound).nan_to_num().max()):.3g}")


def run(ic, m, k, n, out=BF16, act="none", bias=False, residual=False, preact=False, x8=E4, w8=E4, x_tile=1, w_tile=128,
        lx="aligned", lw="aligned", scales="columns", ly="rows", z_dt=BF16, bias_dt=F32, seed=0):
    x, xs = operand(seed + 1, m, k, x8, x_tile, lx, scales)
    w, ws = operand(seed + 2, n, k, w8, w_tile, lw, scales)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def result(dtype):
        v = torch.randn(m, n, generator=g, device="cuda")
        if ly == "rows":
            return v.to(dtype)
        if ly == "odd":
            return torch.empty(m, n + 1 + n % 2, dtype=dtype, device="cuda")[:, :n].copy_(v)
        return torch.empty(n, m + 1, dtype=dtype, device="cuda")[:, :m].t().copy_(v)

    b = torch.randn(n, generator=g, device="cuda").to(bias_dt) if bias else None
    r = result(out) if residual else None
    z = result(z_dt) if preact else None
    y = result(out)
    assert ic.conv_linear_fp8(x, xs, w, ws, b, activation=act, residual=r, preact=z, out=y) is y
    wy, wz, size = ob.linear_fp8(x, xs, w, ws, b, act, r)
    by, bz = ob.linear_fp8_bounds(k, wy, wz, size, act, r, out, z_dt)
    check(y, wy, by, "y")
    if z is not None:
        check(z, wz, bz, "preact")
    return x, xs, w, ws, y


SIZES = [(1, 1, 1), (1, 128, 64), (1, 4096, 257), (2, 127, 16), (3, 129, 40), (8, 1000, 130), (9, 256, 128), (13, 4096, 512),
         (16, 640, 1000), (17, 128, 17), (32, 384, 96), (33, 200, 300), (48, 4096, 520), (64, 1024, 200), (100, 515, 129),
         (127, 64, 64), (128, 128, 128), (129, 192, 255), (200, 16, 24), (255, 2048, 96), (256, 256, 256), (257, 72, 264),
         (300, 16400, 520), (257, 30001, 130), (513, 520, 777), (1000, 333, 70), (2048, 64, 512), (5000, 96, 48),
         (700, 1024, 2300), (1100, 520, 4000), (19712, 128, 520), (2500, 2504, 1030)]


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("w_tile", [128, 1])
def test_sizes(ic, m, k, n, w_tile):
    run(ic, m, k, n, act="gelu", bias=True, residual=True, preact=True, w_tile=w_tile, seed=m + k + n)


@pytest.mark.parametrize("x8,w8,out", list(itertools.product((E4, E5), (E4, E5), (BF16, F16, F32))))
@pytest.mark.parametrize("m", [5, 150, 600])
def test_types(ic, x8, w8, out, m):
    run(ic, m, 700, 300, out, x8=x8, w8=w8, residual=True)
    run(ic, m, 256, 136, out, "silu", x8=x8, w8=w8, bias=True, bias_dt=out, preact=True, z_dt=F16)


@pytest.mark.parametrize("act,residual,preact", list(itertools.product(ACTS, (False, True), (False, True))))
@pytest.mark.parametrize("m", [3, 140, 520])
def test_epilogues(ic, act, residual, preact, m):
    for out in (BF16, F32):
        run(ic, m, 264, 392, out, act, bias=True, residual=residual, preact=preact)


@pytest.mark.parametrize("x_tile,w_tile,scales", list(itertools.product((1, 128), (1, 128), ("columns", "rows", "spread"))))
@pytest.mark.parametrize("m", [20, 300])
def test_scales(ic, x_tile, w_tile, scales, m):
    run(ic, m, 900, 390, F32, x_tile=x_tile, w_tile=w_tile, scales=scales)


@pytest.mark.parametrize("lx,lw,ly", [("wide", "odd", "rows"), ("odd", "wide", "odd"), ("tight", "tight", "cols"), ("aligned", "aligned", "cols")])
@pytest.mark.parametrize("m,k,n", [(5, 333, 200), (140, 333, 200), (600, 1001, 260)])
def test_layouts(ic, lx, lw, ly, m, k, n):
    for out in (BF16, F32):
        run(ic, m, k, n, out, "silu", lx=lx, lw=lw, ly=ly, bias=True, residual=True, preact=True)


@pytest.mark.parametrize("m,k,n", [(1, 4096, 64), (40, 1024, 256), (300, 4096, 512), (1024, 2048, 1024), (256, 16384, 256)])
@pytest.mark.parametrize("w_tile", [128, 1])
def test_exact_sums(ic, m, k, n, w_tile):
    """Small integers with scales of powers of two: every partial sum is an
    integer below 2^24, so the 32-bit result has to be the exact one.  One
    product in each block is 2^17: a sum that dropped bits against the largest
    term would lose the ones beside it."""
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randint(-2, 3, (m, k), generator=g, device="cuda").float()
    w = torch.randint(-1, 2, (n, k), generator=g, device="cuda").float()
    x[:, ::128], w[:, ::128] = 256.0, 256.0
    if k > 8192:  # (128 blocks of 2^16 + 254 stay below 2^24)
        x[:, ::128] = 128.0
    s = torch.ones(m, ob.blocks(k), device="cuda")
    t = torch.full((-(-n // w_tile), ob.blocks(k)), 2.0 ** -3, device="cuda")
    y = ic.conv_linear_fp8(x.to(E4), s, w.to(E4), t, dtype=F32)
    assert torch.equal(y.double(), x.double() @ w.double().t() / 8)


@pytest.mark.parametrize("m", [4, 130, 600])
def test_nan_and_infinity_stay_in_their_rows(ic, m):
    x, xs = operand(1, m, 512)
    w, ws = operand(2, 260, 512)
    clean = ic.conv_linear_fp8(x, xs, w, ws)
    x2, xs2, w2 = x.clone(), xs.clone(), w.clone()
    x2.view(torch.uint8)[1, 300] = 0x7f
    w2.view(torch.uint8)[7, 3] = 0xff
    xs2[3, 2] = float("inf")
    y = ic.conv_linear_fp8(x2, xs2, w2, ws)
    assert torch.isnan(y[1]).all() and torch.isnan(y[:, 7]).all() and not torch.isfinite(y[3]).any()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[1], keep[3], keep[:, 7] = False, False, False
    assert torch.equal(y[keep], clean[keep])


def test_empty_extents(ic):
    def make(rows, k):
        return torch.zeros(rows, k, device="cuda").to(E4), torch.ones(rows, ob.blocks(k), device="cuda")

    for m in (5, 40):
        b, r = torch.randn(24, device="cuda"), torch.randn(m, 24, device="cuda").to(BF16)
        y = ic.conv_linear_fp8(*make(m, 0), *make(24, 0), b, activation="silu", residual=r)
        want = ob.activate(b.double(), "silu") + r.double()
        check(y, want, 2.0 ** -8 * want.abs() + 2.0 ** -20, "y")
    assert ic.conv_linear_fp8(*make(0, 64), *make(24, 64)).shape == (0, 24)
    assert ic.conv_linear_fp8(*make(5, 64), *make(0, 64)).shape == (5, 0)


def test_in_place_residual_leading_dims_and_neighbours(ic):
    x, xs = operand(3, 6, 300)
    w, ws = operand(4, 130, 300, tile=128)
    big = torch.randn(2, 3, 140, device="cuda").to(BF16)
    before = big.clone()
    out = big[..., 5:135]
    want, _, size = ob.linear_fp8(x, xs, w, ws, None, "none", before[..., 5:135].reshape(6, 130))
    ic.conv_linear_fp8(x.reshape(2, 3, 300) if x.is_contiguous() else x.contiguous().view(2, 3, 300), xs.contiguous().view(2, 3, 3), w, ws,
                       residual=out, out=out)
    by, _ = ob.linear_fp8_bounds(300, want, want, size, "none", before[..., 5:135].reshape(6, 130), BF16)
    check(out.reshape(6, 130), want, by, "y")
    assert torch.equal(big[..., :5], before[..., :5]) and torch.equal(big[..., 135:], before[..., 135:])


@pytest.mark.parametrize("m,k,n", [(13, 1024, 512), (200, 8192, 256), (1024, 1024, 1024)])
def test_repeats_in_graphs_and_on_streams(ic, m, k, n):
    x, xs = operand(5, m, k)
    w, ws = operand(6, n, k, tile=128)
    first = ic.conv_linear_fp8(x, xs, w, ws, dtype=F32)
    for _ in range(3):
        assert torch.equal(ic.conv_linear_fp8(x, xs, w, ws, dtype=F32), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = ic.conv_linear_fp8(x, xs, w, ws, dtype=F32)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = ic.conv_linear_fp8(x, xs, w, ws, dtype=F32)
    xs.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(z, 2 * first)


@pytest.mark.parametrize("m,k,n", [(70, 200, 300), (1000, 384, 512)])
def test_layer_forward_and_gradients(ic, m, k, n):
    """A layer y = gelu(x w^T + b) with 8-bit products: the forward pass, and
    dx and dw from the gradient quantised both ways, against the definition on
    the quantised values; and those against the unquantised layer to the 8-bit
    steps."""
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(m, k, generator=g, device="cuda").to(BF16)
    w = (torch.randn(n, k, generator=g, device="cuda") / k ** 0.5).to(BF16)
    b, dy = torch.randn(n, generator=g, device="cuda") / 8, torch.randn(m, n, generator=g, device="cuda").to(BF16)
    xq, xs, xt, xts = ic.conv_quantize(x, columns=True)
    wq, ws, wt, wts = ic.conv_quantize(w, tile=128, columns=True)
    z = torch.empty(m, n, dtype=BF16, device="cuda")
    y = ic.conv_linear_fp8(xq, xs, wq, ws, b, activation="gelu", preact=z)
    dq, ds, dt, dts = ic.conv_quantize(dy, preact=z, activation="gelu", columns=True, dtype=E5)
    dx = ic.conv_linear_fp8(dq, ds, wt, wts, dtype=F32)
    dw = ic.conv_linear_fp8(dt, dts, xt, xts, dtype=F32)
    for got, (a, sa, c, sc) in ((dx, (dq, ds, wt, wts)), (dw, (dt, dts, xt, xts))):
        want, _, size = ob.linear_fp8(a, sa, c, sc)
        check(got, want, ob.linear_fp8_bounds(a.shape[1], want, want, size, "none", None, F32)[0], "gradient")
    # unquantised: errors of the values are at most 2^-4 (e4m3) and 2^-3 (e5m2) of them or of the block's smallest step,
    # independent, so the 2-norms are off by less than those shares of the products' sizes
    zf = x.double() @ w.double().t() + b.double()
    dz = dy.double() * ob.slope(z.double(), "gelu")
    for got, want, size, far in ((y, ob.activate(zf, "gelu"), 1.2 * (x.double().abs() @ w.double().abs().t()), 2 * 2.0 ** -4),
                                 (dx, dz @ w.double(), dz.abs() @ w.double().abs(), 2.0 ** -3 + 2.0 ** -4 + 2.0 ** -6),
                                 (dw, dz.t() @ x.double(), dz.t().abs() @ x.double().abs(), 2.0 ** -3 + 2.0 ** -4 + 2.0 ** -6)):
        assert float((got.double() - want).norm()) < far * float(size.norm())

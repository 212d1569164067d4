"""Edges of the channel operators on the GPU."""
import numpy as np
import pytest

from oracle import channel as oc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

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


# ------------------------------------------------------------------- autograd
def test_outputs_count_as_changed_in_place(ic):
    g = gen(1)
    x, w, dy = randn(g, 6, 16).to(F16), randn(g, 8, 16).to(F16), randn(g, 6, 8).to(F16)
    z, y = torch.empty_like(dy), torch.empty_like(dy)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(8, device="cuda")
    mean, rstd = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    n, dn, dg, dh = torch.empty_like(x), torch.empty_like(x), torch.empty(16, device="cuda"), torch.empty(16, device="cuda")

    def counts(outputs, call):
        before = [t._version for t in outputs]
        call()
        assert [t._version - b for t, b in zip(outputs, before)] == [1] * len(outputs)

    counts([y, z], lambda: ic.conv_linear(x, w, activation="silu", preact=z, out=y))
    counts([dx, dw, db], lambda: ic.conv_linear_grad(dy, x, w, preact=z, activation="silu", dx=dx, dw=dw, dbias=db))
    counts([n, mean, rstd], lambda: ic.conv_layer_norm(x, out=n, mean=mean, rstd=rstd))
    counts([dn, dg, dh], lambda: ic.conv_layer_norm_grad(x, x, None, mean, rstd, dx=dn, dgain=dg, dshift=dh))
    # a graph that saved the tensor refuses to go back
    a, p = randn(g, 6, 16), torch.ones(16, device="cuda", requires_grad=True)
    s = (a * p).sum()
    ic.conv_layer_norm(a, out=a)
    with pytest.raises(RuntimeError, match="in-?place|modified"):
        s.backward()
    # an inference tensor has no version to count
    with torch.inference_mode():
        frozen = randn(g, 6, 16)
    ic.conv_layer_norm(frozen, out=frozen)


# ----------------------------------------------------------- norm, far from zero
def f64(t):
    return None if t is None else t.double().cpu().numpy()


def check(got, want, bound, what):
    got = f64(got)
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside the bound, first at "
                           f"{tuple(int(i[0]) for i in np.nonzero(bad))}, worst {np.nanmax(np.abs(got - want) / bound):.3g}")


def strided(v, dtype, lead):
    """The values in rows that start `lead` elements past a boundary of 8 and are
    a multiple of 8 apart; lead None: columns two elements apart."""
    m, c = v.shape
    if lead is None:
        return torch.full((m, 2 * c), float("nan"), device="cuda", dtype=dtype)[:, ::2].copy_(v)
    return torch.full((m, (c + 15) // 8 * 8), float("nan"), device="cuda", dtype=dtype)[:, lead:lead + c].copy_(v)


# every way a row is held: by a warp (two widths), by a block (three), read again for each pass
HELD = [(40, 200), (40, 512), (700, 1000), (700, 4097), (330, 8192), (6, 17000)]


@pytest.mark.parametrize("m,c", HELD)
@pytest.mark.parametrize("mean", [1000.0, -30000.0])
# x, dy alike; x and dy at different leads; columns apart
@pytest.mark.parametrize("leads", [(0, 0), (3, 3), (1, 2), (None, 0)])
def test_layer_norm_grad_far_from_zero(ic, m, c, mean, leads):
    """Rows whose mean is many deviations: n = (x - mean) rstd is only off by
    its own rounding, whatever the mean."""
    g = gen(m + c)
    x, dy = strided(randn(g, m, c) + mean, F32, leads[0]), strided(randn(g, m, c) / 4, F32, leads[1])
    gain = 1 + 0.3 * randn(g, c)
    _, mu, rstd = oc.layer_norm(f64(x))
    mu, rstd = (torch.from_numpy(v.astype(np.float32)).cuda() for v in (mu, rstd))
    dx, dg, db = torch.empty(m, c, device="cuda"), torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    ic.conv_layer_norm_grad(dy, x, gain, mu, rstd, dx=dx, dgain=dg, dshift=db)
    args = [f64(v) for v in (dy, x, gain, mu, rstd)] + [None]
    want = oc.layer_norm_grad(*args)
    bounds = oc.layer_norm_grad_bounds(*args, want, "float32", "float32", centred=True)
    for got, v, b, what in zip((dx, dg, db), want, bounds, ("dx", "dgain", "dshift")):
        check(got, v, b, what)


@pytest.mark.parametrize("m,c", HELD)
def test_layer_norm_grad_of_constant_rows(ic, m, c):
    """No deviation: n is 0, and so is dgain, whatever the rows' value."""
    g = gen(c)
    dy = randn(g, m, c)
    mean, rstd = torch.randn(m, generator=g, device="cuda") * 1e6, torch.full((m,), 1e-5 ** -0.5, device="cuda")
    x = mean[:, None].expand(m, c).contiguous()
    dx, dg = torch.empty_like(x), torch.full((c,), 5.0, device="cuda")
    ic.conv_layer_norm_grad(dy, x, None, mean, rstd, dx=dx, dgain=dg)
    assert not dg.any()
    want = f64(rstd)[:, None] * (f64(dy) - f64(dy).mean(1, keepdims=True))
    d = np.abs(f64(dy))
    check(dx, want, f64(rstd)[:, None] * ((c / 32 + 16) * 2.0 ** -23 * d.mean(1, keepdims=True) + 2.0 ** -21 * (d + 1)), "dx")


# ------------------------------------------------------- non-finite pre-activations
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dt", [F16, BF16])
# the gradient's passes over dy: few rows; rows of aligned vectors, of any alignment; columns contiguous
@pytest.mark.parametrize("m,n,cols", [(3, 24, False), (600, 24, False), (600, 25, False), (600, 24, True)])
def test_slopes_at_infinite_and_nan_preactivations(ic, act, dt, m, n, cols):
    """1 at plus infinity, 0 at minus infinity (the slopes' limits; 0 where dy is
    0), NaN at a NaN, but ReLU's 0."""
    g = gen(n)
    z, dy = randn(g, m, n).to(dt), torch.zeros(m, n, device="cuda", dtype=dt)
    inf, nan = float("inf"), float("nan")
    z[1, 0], z[m - 1, 1], z[1, 2] = inf, -inf, nan
    z[0, 3], z[1, 4] = inf, -inf
    dy[1, 0], dy[m - 1, 1], dy[1, 2] = 2.0, 2.0, 2.0
    x, w = randn(g, m, 8).to(dt), randn(g, n, 8).to(dt)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(n, device="cuda")
    if cols:
        z, dy = z.t().contiguous().t(), dy.t().contiguous().t()
    ic.conv_linear_grad(dy, x, w, preact=z, activation=act, dx=dx, dw=dw, dbias=db)
    assert db[0] == 2 and db[1] == 0 and not db[3:].any()
    assert db[2] == 0 if act == "relu" else torch.isnan(db[2])
    assert torch.equal(dw[0], 2 * x[1]) and not dw[1].any() and not dw[3:].any()
    assert not dx[0].any() and not dx[m - 1].any()
    if act == "relu":
        assert torch.equal(dx[1], 2 * w[0]) and not dw[2].any()
    else:
        assert torch.isnan(dx[1]).all() and torch.isnan(dw[2]).all()


# --------------------------------------------------------------------- GELU
@pytest.mark.parametrize("m", [1, 100, 3000])
def test_gelu_is_as_exact_as_stated(ic, m):
    """Phi off by 1.4e-7 by its fit and 2^-23 by its exponential (2^-22.5 of a
    value of at most a half), then one rounding; the slope's second term, at
    most a quarter, by a few 2^-22 of itself."""
    n = 1040
    z = torch.linspace(-16.5, 16.5, n, device="cuda").to(BF16)
    x, w = torch.zeros(m, 8, device="cuda", dtype=BF16), torch.zeros(n, 8, device="cuda", dtype=BF16)
    x[:, 0], w[:, 0] = 1.0, z
    y = ic.conv_linear(x, w, activation="gelu", out=torch.empty(m, n, device="cuda"))
    f = f64(z)
    want = oc.activate(f, "gelu")
    check(y, np.broadcast_to(want, (m, n)), (1.4e-7 + 2.0 ** -23) * np.abs(f) + 2.0 ** -23 * np.abs(want) + 2.0 ** -126, "y")
    # the bias gradient of one row is dy times the slope, in 32 bits
    one, db = torch.ones(1, n, device="cuda", dtype=BF16), torch.empty(n, device="cuda")
    ic.conv_linear_grad(one, x[:1], w, preact=z[None], activation="gelu", dbias=db)
    check(db, oc.activation_slope(f, "gelu"), np.full(n, 2.0 ** -21), "slope")

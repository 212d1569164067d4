"""conv_quantize on the GPU against its definition in 64 bits: sizes from one
element to several tiles, every type, both forms, tiles, layouts, slopes, zeros,
infinities and NaN, and the neighbourhood of what it writes."""
import itertools

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import blocks as ob  # noqa: E402
from oracle import channel as oc  # noqa: E402

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


def values(seed, m, c):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(m, c, generator=g, device="cuda") * torch.exp(torch.randn(c, generator=g, device="cuda"))


def place(v, dtype, layout):
    m, n = v.shape
    nan = float("nan")
    if layout == "rows":
        t = torch.empty(m, n, device="cuda", dtype=dtype)
    elif layout == "odd":
        t = torch.full((m, n + 1 + n % 2), nan, device="cuda", dtype=dtype)[:, :n]
    elif layout == "shifted":
        t = torch.full((m, (n + 7) // 8 * 8 + 8), nan, device="cuda", dtype=dtype)[:, 1:n + 1]
    elif layout == "cols":
        t = torch.full((n, (m + 7) // 8 * 8), nan, device="cuda", dtype=dtype)[:, :m].t()
    else:
        t = torch.full((m, 2 * n), nan, device="cuda", dtype=dtype)[:, ::2]
    return t.copy_(v)


def run(ic, m, c, dt=BF16, to=E4, tile=1, rows=True, columns=True, act="none", layout="rows", z_dt=None, seed=0):
    x = place(values(seed, m, c), dt, layout)
    z = place(values(seed + 1, m, c), z_dt or BF16, layout) if act != "none" else None
    got = ic.conv_quantize(x, dtype=to, tile=tile, rows=rows, columns=columns, preact=z, activation=act)
    v, ev = x.double(), None
    if z is not None:
        v, ev = v * ob.slope(z.double(), act), 2.0 ** -19 * v.abs()
    assert len(got) == 2 * (rows + columns)
    got = list(got)
    if rows:
        q, s = got.pop(0), got.pop(0)
        assert q.shape == x.shape and q.dtype == to and q.stride(0) % 16 == 0
        assert ob.check_quantized(q, s, v, tile, ev) is None, ob.check_quantized(q, s, v, tile, ev)
    if columns:
        q, s = got
        assert q.shape == (c, m) and q.dtype == to
        e = None if ev is None else ev.t()
        assert ob.check_quantized(q, s, v.t(), tile, e) is None, ob.check_quantized(q, s, v.t(), tile, e)


SIZES = [(1, 1), (1, 128), (1, 4096), (2, 127), (5, 129), (7, 8), (16, 640), (33, 200), (127, 1), (128, 128), (129, 257),
         (130, 384), (300, 1000), (1000, 72), (513, 515), (1, 16385), (4097, 3)]


@pytest.mark.parametrize("m,c", SIZES)
@pytest.mark.parametrize("tile", [1, 128])
def test_sizes(ic, m, c, tile):
    run(ic, m, c, tile=tile, seed=m + c)


@pytest.mark.parametrize("dt,to,act", list(itertools.product((BF16, F16, F32), (E4, E5), ACTS)))
def test_types_and_slopes(ic, dt, to, act):
    run(ic, 150, 200, dt, to, act=act)
    run(ic, 131, 261, dt, to, tile=128, act=act, z_dt=F16)
    run(ic, 9, 40, dt, to, columns=False, act=act, z_dt=dt)
    run(ic, 9, 40, dt, to, rows=False, act=act, z_dt=dt)


@pytest.mark.parametrize("layout", ["rows", "odd", "shifted", "cols", "spread"])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_layouts(ic, layout, dt):
    run(ic, 140, 270, dt, layout=layout)
    run(ic, 140, 272, dt, act="silu", layout=layout, tile=128)


def test_exact_ties_and_range(ic):
    # a block whose largest value is L: its scale is 1, and every value is rounded to nearest even
    u = torch.linspace(-448, 448, 128 * 64, device="cuda").to(BF16).view(64, 128).clone()
    u[:, 0] = 448
    q, s = ic.conv_quantize(u)
    assert torch.equal(s, torch.ones_like(s))
    assert torch.equal(q.float(), u.float().to(E4).float())
    q, s = ic.conv_quantize(u * 128, dtype=E5)   # largest 57344
    assert torch.equal(s, torch.ones_like(s))
    assert torch.equal(q.float(), (u.float() * 128).to(E5).float())


def test_zeros_and_small_values(ic):
    x = torch.zeros(130, 260, device="cuda", dtype=F32)
    x[1, 5] = 1e-44         # far below 448 * 2^-126
    x[2, 200] = 448 * 2.0 ** -126
    x[3, 7] = 3e38
    q, s, qt, st = ic.conv_quantize(x, columns=True)
    assert ob.check_quantized(q, s, x.double(), 1) is None
    assert ob.check_quantized(qt, st, x.t().double(), 1) is None
    assert float(s[0, 0]) == 2.0 ** -126 and not q[0].float().any()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_infinities_and_nan_stay_in_their_block(ic, bad):
    x = values(3, 200, 300).to(BF16)
    x[130, 140] = bad
    clean = x.clone()
    clean[130, 140] = 0
    for tile in (1, 128):
        q, s, qt, st = ic.conv_quantize(x, tile=tile, columns=True)
        for a, b, hit in ((q, s, (130 // tile, 1)), (qt, st, (140 // tile, 1))):
            assert not torch.isfinite(b[hit])
            finite = torch.isfinite(b)
            assert int((~finite).sum()) == 1
        whole = q.float() * ob.per_element(s, 200, 300).float()
        block = torch.zeros(200, 300, dtype=torch.bool, device="cuda")
        r0 = 130 // tile * tile
        block[r0:r0 + tile, 128:256] = True
        assert torch.isnan(whole[block]).all() and torch.isfinite(whole[~block]).all()


def test_given_outputs_and_their_neighbours(ic):
    m, c = 133, 261
    x = values(5, m, c).to(BF16)
    want = ic.conv_quantize(x, columns=True)
    # strided 8-bit outputs, scales row by row; what lies between stays
    q = torch.full((m, c + 7), 77, dtype=torch.uint8, device="cuda")
    qt = torch.full((c, m + 3), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((m, 5), -1.0, device="cuda")
    st = torch.full((c, 5), -1.0, device="cuda")
    got = ic.conv_quantize(x, columns=True, out=q.view(E4)[:, :c], scale=s[:, :3], out_t=qt.view(E4)[:, 1:m + 1], scale_t=st[:, 1:3])
    for a, b in zip(got, want):
        assert torch.equal(a.float(), b.float())
    assert (q[:, c:] == 77).all() and (qt[:, 0] == 77).all() and (qt[:, m + 1:] == 77).all()
    assert (s[:, 3:] == -1).all() and (st[:, 0] == -1).all() and (st[:, 3:] == -1).all()


def test_leading_dims_empty_and_other_stream(ic):
    x = values(6, 6 * 35, 96).to(F16).view(2, 3, 35, 96)
    q, s = ic.conv_quantize(x)
    assert q.shape == x.shape and s.shape == (2, 3, 35, 1)
    assert ob.check_quantized(q.reshape(-1, 96), s.reshape(-1, 1), x.reshape(-1, 96).double(), 1) is None
    q, s = ic.conv_quantize(x, tile=128)
    assert s.shape == (2, 1)
    for shape in ((0, 40), (40, 0)):
        q, s, qt, st = ic.conv_quantize(torch.empty(shape, device="cuda", dtype=BF16), columns=True)
        assert q.shape == shape and qt.shape == shape[::-1]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    a = ic.conv_quantize(x, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    b = ic.conv_quantize(x)
    assert torch.equal(a[0].float(), b[0].float()) and torch.equal(a[1], b[1])

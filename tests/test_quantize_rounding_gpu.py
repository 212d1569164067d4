"""conv_quantize rounds to the nearest 8-bit value and to the even one of two
that are equally near, bit for bit.

The quotient of a 16-bit value v by a scale a / L (L = 7 * 2^k) is 7 v / a: it
lies on the middle between two 8-bit values, which has 5 bits M at most, where
7 v = M a, or else is away from it by 1 part in M a at least, that is by 2^-16
(a has 11 bits or fewer).  So any quotient that is exact where 32 bits hold it
and within 2^-20 elsewhere gives the same 8 bits as the exact one."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import blocks as ob  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


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


def exact(v, dtype, tile):
    """8-bit values (as float64) and scales (float32) of v (float64)."""
    m, c = v.shape
    most = ob.block_largest(v, tile)
    scale = (most / ob.LARGEST[dtype]).float().clamp(min=ob.LEAST_SCALE)
    a = ob.per_element(most.clamp(min=ob.LEAST_SCALE * ob.LARGEST[dtype]), m, c)
    u = v * ob.LARGEST[dtype] / a
    # the step between 8-bit values at u, a power of two that is made of its bits: pow need not give it exactly
    bits, least = ob.BITS[dtype]
    e = (u.abs().view(torch.int64) >> 52).clamp(min=least + 1023)
    step = ((e - bits) << 52).view(torch.float64)
    return torch.round(u / step) * step, scale  # (to even)


def check(got, v, dtype, tile):
    q, s = exact(v, dtype, tile)
    assert torch.equal(got[1], s)
    wrong = int((got[0].double() != q).sum())
    assert wrong == 0


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("to", [E4, E5])
@pytest.mark.parametrize("tile", [1, 128])
@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("wide", [False, True])
def test_nearest_and_even(ic, dt, to, tile, act, wide):
    """wide: the same values as 32-bit floats; relu: the slopes are 0 and 1."""
    g = torch.Generator(device="cuda").manual_seed(2)
    m, c = 640, 1024
    x = (torch.randn(m, c, generator=g, device="cuda") * torch.exp(torch.randn(c, generator=g, device="cuda"))).to(dt)
    z = torch.randn(m, c, generator=g, device="cuda").to(dt) if act == "relu" else None
    v = x.double() if z is None else x.double() * (z > 0)
    given = x.float() if wide else x
    got = ic.conv_quantize(given, dtype=to, tile=tile, columns=True, preact=z, activation=act)
    check(got[:2], v, to, tile)
    check(got[2:], v.t(), to, tile)


def test_every_middle(ic):
    """Blocks whose values are the middles themselves, times a: q is the even neighbour.  (a of up to 6 bits, so that
    bf16 holds M a / 7.)"""
    rows = []
    for e4 in (True, False):
        dtype, L = (E4, 448.0) if e4 else (E5, 57344.0)
        for a in range(7, 57, 7):
            u = torch.arange(0, 256, device="cuda", dtype=torch.uint8)
            v = u.view(dtype).float()
            v = v[torch.isfinite(v) & (v >= 0)].unique()
            mid = (v[1:] + v[:-1]) / 2
            x = mid.double() * a / L
            keep = x.to(BF16).double() == x
            x = torch.cat([x[keep], x.new_tensor([float(a)])])
            x = torch.nn.functional.pad(x, (0, 128 - x.numel())).to(BF16)[None]
            rows.append((dtype, x))
    for dtype in (E4, E5):
        x = torch.cat([r for d, r in rows if d is dtype])
        assert x.count_nonzero() > 8 * 20
        check(ic.conv_quantize(x, dtype=dtype), x.double(), dtype, 1)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("m,c,pad", [(1, 5, 0), (1, 131, 0), (1, 203, 0), (7, 100, 4), (130, 261, 3)])
def test_preactivation_that_ends_with_its_buffer(ic, dt, m, c, pad):
    """Rows from 16-byte boundaries whose last one ends inside a vector, at the end of the memory: nothing is read past it.
    (ReLU's slopes of the wrong elements, or of NaN beside them, would show in q.)"""
    g = torch.Generator(device="cuda").manual_seed(m + c)
    x = torch.randn(m, c, generator=g, device="cuda").to(dt)
    flat = torch.full(((m - 1) * (c + pad) + c,), float("nan"), device="cuda", dtype=dt)
    z = flat.as_strided((m, c), (c + pad, 1))
    z.copy_(torch.randn(m, c, generator=g, device="cuda"))
    assert z.data_ptr() % 16 == 0 and (m == 1 or (c + pad) % 8 == 0)
    got = ic.conv_quantize(x, columns=True, preact=z, activation="relu")
    v = x.double() * (z > 0)
    check(got[:2], v, E4, 1)
    check(got[2:], v.t(), E4, 1)

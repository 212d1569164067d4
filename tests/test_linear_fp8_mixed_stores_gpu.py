"""conv_linear_fp8 where the output and the pre-activation are stored in unlike
ways (rows by TMA, rows of other alignment, columns, chunks at the edge), which
take turns on the staging slots of a warp.  Without activation, bias and
residual both are roundings of one sum, so that they have to agree bit for bit;
and they are held to the 64-bit definition."""
import itertools

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import blocks as ob  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E4 = torch.float8_e4m3fn


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


def place(m, n, dtype, layout):
    """A matrix between values that have to stay, and all of its memory."""
    if layout == "cols":
        whole = torch.full((n, m + 1), 7.0, dtype=dtype, device="cuda")
        return whole[:, :m].t(), whole
    pad = {"rows": 0, "wide": (-n) % 8 + 8, "odd": 1 + n % 2}[layout]
    whole = torch.full((m, n + pad), 7.0, dtype=dtype, device="cuda")
    return whole[:, :n], whole


# tiles of 64, 128 and 256 columns, several to a CTA, and few tiles
SIZES = [(33000, 60), (20000, 124), (4000, 2100), (2500, 1032), (300, 264), (257, 100), (40, 520)]
LAYOUTS = [p for p in itertools.product(("rows", "wide", "odd", "cols"), repeat=2)]


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("out", [BF16, F32])
def test_output_and_preactivation_agree(ic, m, n, out):
    k = 256
    g = torch.Generator(device="cuda").manual_seed(m + n)
    x = (torch.randn(m, k, generator=g, device="cuda") * 40).clamp(-448, 448).to(E4)
    w = (torch.randn(n, k, generator=g, device="cuda") * 40).clamp(-448, 448).to(E4)
    xs = torch.exp(torch.randn(m, 2, generator=g, device="cuda")) / 100
    ws = torch.exp(torch.randn(n, 2, generator=g, device="cuda")) / 100
    want, _, size = ob.linear_fp8(x, xs, w, ws)
    by, bz = ob.linear_fp8_bounds(k, want, want, size, "none", None, out, BF16)
    for ly, lz in LAYOUTS:
        y, y_whole = place(m, n, out, ly)
        z, z_whole = place(m, n, BF16, lz)
        for _ in range(2):
            y.fill_(7.0)
            z.fill_(7.0)
            ic.conv_linear_fp8(x, xs, w, ws, preact=z, out=y)
            assert torch.equal(y.to(BF16), z), (ly, lz)
            assert bool(((y.double() - want).abs() <= by).all()) and bool(((z.double() - want).abs() <= bz).all()), (ly, lz)
        for part, whole in ((y, y_whole), (z, z_whole)):
            part.fill_(7.0)
            assert bool((whole == 7.0).all()), (ly, lz)

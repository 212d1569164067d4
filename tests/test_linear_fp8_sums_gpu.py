"""The block sums of conv_linear_fp8 keep 24 bits: sums of integers below 2^24
that hold a product near their top come out exactly, wherever it lies.  The
scales are powers of two, so that nothing else is rounded."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import blocks as ob  # noqa: E402

F32 = torch.float32
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


def exact(ic, x, w, dtype, w_tile):
    s = torch.ones(x.shape[0], ob.blocks(x.shape[1]), device="cuda")
    t = torch.full((-(-w.shape[0] // w_tile), ob.blocks(x.shape[1])), 2.0 ** -3, device="cuda")
    y = ic.conv_linear_fp8(x.to(dtype), s, w.to(dtype), t, dtype=F32)
    want = x.double() @ w.double().t()
    assert float((x.double().abs() @ w.double().abs().t()).max()) < 2.0 ** 24
    assert torch.equal(y.double(), want / 8)


def small(seed, rows, k):
    return torch.randint(-1, 2, (rows, k), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").float()


@pytest.mark.parametrize("m,n", [(1, 64), (13, 200), (40, 256), (300, 130), (2100, 1100)])
@pytest.mark.parametrize("w_tile", [128, 1])
def test_one_product_of_2_to_the_23(ic, m, n, w_tile):
    """Of E5M2; the products beside it are 0, 1 or -1, the last of 24 bits."""
    for where in (0, 17, 64, 127):
        x, w = small(m, m, 128), small(n + 1, n, 128)
        x[:, where], w[:, where] = 2.0 ** 11, 2.0 ** 12
        exact(ic, x, w, E5, w_tile)


@pytest.mark.parametrize("m,n", [(1, 64), (13, 200), (40, 256), (300, 130)])
@pytest.mark.parametrize("w_tile", [128, 1])
def test_the_largest_products_of_e4m3(ic, m, n, w_tile):
    """448 * 448 = 200704 in each of 64 blocks of 128: below 2^24 with what lies beside them (64 * (200704 + 127))."""
    x, w = small(m, m, 8192), small(n + 1, n, 8192)
    x[:, 5::128], w[:, 5::128] = 448.0, 448.0
    exact(ic, x, w, E4, w_tile)

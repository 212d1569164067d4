"""conv_block_norm and its gradients without a post norm, where the branch is x
itself: what of the results depends on x and what does not."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32


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


# rows held by warps (of whole groups and not), by blocks, and in shared memory
@pytest.mark.parametrize("c", [200, 203, 512, 1100, 2003, 9000])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_dx_does_not_depend_on_x(ic, c, groups, bad):
    """dx = branch_scale * gate * dh, with h and its statistics as given."""
    m = 20
    g = torch.Generator(device="cuda").manual_seed(c)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x, h, dy, ds = (normal(m, c).to(BF16) for _ in range(4))
    rs = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    gate = normal(groups, c).to(BF16)

    def grads(x, dy, ds):
        dx, dskip, dgate = torch.empty_like(h), torch.empty_like(h), torch.empty(groups, c, device="cuda")
        ic.conv_block_norm_grad(dy, ds, x, h if dy is not None else None, gate=gate, branch_scale=0.5,
                                rstd=rs if dy is not None else None, dx=dx, dskip=dskip, dgate=dgate)
        return dx, dskip, dgate

    broken = x.clone()
    broken[7, 5] = bad
    for a, b in ((dy, ds), (None, ds), (dy, None)):
        clean, got = grads(x, a, b), grads(broken, a, b)
        assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
        hit = torch.zeros_like(clean[2], dtype=torch.bool)
        hit[7 // (m // groups), 5] = True
        assert not bool(torch.isfinite(got[2][hit]).any()) and torch.equal(got[2][~hit], clean[2][~hit])


@pytest.mark.parametrize("c", [200, 2003])
def test_scaled_branch_alone_has_a_sum(ic, c):
    """The sum is left out only where it is x itself: not where the branch is scaled."""
    x = torch.randn(9, c, device="cuda").to(BF16)
    s, y = ic.conv_block_norm(x)
    assert s is None
    for scale in (0.5, -1.0, 0.0):
        s, y = ic.conv_block_norm(x, branch_scale=scale)
        given, out = torch.empty_like(x), torch.empty_like(x)
        ic.conv_block_norm(x, branch_scale=scale, sum=given, out=out)
        assert s is not None and torch.equal(s, given) and torch.equal(s, (scale * x.float()).to(BF16))
        assert torch.equal(y, out)
        # (the statistics belong to this sum: |y| has a mean square of 1, where the sum has one)
        if scale:
            assert float((y.double().square().mean(1) - 1).abs().max()) < 2.0 ** -7

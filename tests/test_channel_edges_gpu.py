"""Edges of the channel operators on the GPU."""
import pytest

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

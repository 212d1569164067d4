"""conv_clip_grads without a limit writes no tensors, so that it is not given any
to write; and numbers beyond 32 bits are not taken as infinite ones."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


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


def test_outputs_need_a_finite_limit(ic):
    grads = [torch.randn(100, device="cuda"), torch.randn(7, device="cuda").bfloat16()]
    before, out = [g.clone() for g in grads], [torch.full_like(g, 5) for g in grads]
    for most in (None, math.inf):
        with pytest.raises(ValueError, match="out"):
            ic.conv_clip_grads(grads, most, out=out)
        assert float(ic.conv_clip_grads(grads, most)) > 0
    for most in (1e39, 1e300):
        for given in (None, out):
            with pytest.raises(ValueError, match="32-bit"):
                ic.conv_clip_grads(grads, most, out=given)
    assert all(torch.equal(a, b) for a, b in zip(grads, before)) and all(bool((t == 5).all()) for t in out)
    ic.conv_clip_grads(grads, 3e38, out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, before))

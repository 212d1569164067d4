"""conv_clip_grads on the GPU against 64 bits: counts, types, odd sizes and
addresses, many tensors, the ends of the range, in place and apart, norm alone,
streams and graphs.  A sum of 32 squares in 32 bits is off by 2^-19 of itself
at most, its root by half that, and the stored norm by one rounding more."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import blocks as ob  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
NORM = 2.0 ** -20 + 2.0 ** -23


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


def tensors(sizes, types=(F32, BF16, F16), scale=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(types[i % len(types)]) for i, n in enumerate(sizes)]


def check(norm, outs, want_norm, want):
    assert abs(float(norm) - want_norm) <= NORM * want_norm
    for i, (a, b) in enumerate(zip(outs, want)):
        bound = ob.rounded((NORM + 2.0 ** -23) * b.abs(), b, a.dtype)
        assert bool(((a.double() - b).abs() <= bound).all()), i


SETS = [[1], [5], [0, 3], [4096], [16384], [16385], [100003], [1, 2, 3, 7, 8, 9, 127, 0, 2048, 16383], [5000000, 11, 700001],
        list(range(1, 64)), [1000 + i for i in range(65)], [300] * 961, [17, 40000] * 1100]


@pytest.mark.parametrize("k", range(len(SETS)))
def test_sets(ic, k):
    grads = tensors(SETS[k], seed=k)
    for most in (0.5, 1e6, 0.0):
        norm, want = ob.clip(grads, most, 1e-6)
        apart = [torch.empty_like(g) for g in grads]
        before = [g.clone() for g in grads]
        check(ic.conv_clip_grads(grads, most, out=apart), apart, norm, want)
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
        check(ic.conv_clip_grads(before, most), before, norm, want)
    norm, want = ob.clip(grads, math.inf, 0)
    before = [g.clone() for g in grads]
    given = torch.zeros(1, device="cuda")
    assert ic.conv_clip_grads(grads, norm=given) is given
    check(given, grads, norm, before)


def test_views_and_addresses(ic):
    flat = torch.randn(100000, device="cuda").to(BF16)
    parts = [flat[1:1001], flat[1001:20000], flat[20001:20002], flat[30000:60000].view(100, 300).t(), flat[60003:99999]]
    rest = torch.ones_like(flat, dtype=torch.bool)
    for a, b in ((1, 20000), (20001, 20002), (30000, 60000), (60003, 99999)):
        rest[a:b] = False
    before = flat.clone()
    norm, want = ob.clip(parts, 1.0, 1e-6)
    check(ic.conv_clip_grads(parts, 1.0), parts, norm, want)
    assert torch.equal(flat[rest], before[rest])


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-18, 1e15, 1e19, 1e30])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_ends_of_the_range(ic, scale, dt):
    grads = tensors([5000, 37], (dt,), scale)
    norm, want = ob.clip(grads, scale, 0.0)
    apart = [torch.empty_like(g) for g in grads]
    check(ic.conv_clip_grads(grads, scale, eps=0.0, out=apart), apart, norm, want)


def test_mixed_sizes_of_values(ic):
    grads = tensors([1000], (F32,), 1e25) + tensors([1000], (F32,), 1e-25, 1) + [torch.zeros(100000, device="cuda")]
    norm, want = ob.clip(grads, 1.0, 1e-6)
    got = ic.conv_clip_grads([g.clone() for g in grads])
    assert abs(float(got) - norm) <= NORM * norm
    grads = [torch.full((33,), 2.0 ** -149, device="cuda")]
    assert abs(float(ic.conv_clip_grads(grads)) - math.sqrt(33) * 2.0 ** -149) <= 2.0 ** -149


def test_infinite_and_nan_norms(ic):
    for bad in (math.inf, math.nan):
        grads = tensors([1000, 2000], (F32, BF16))
        grads[0][500] = bad
        norm = ic.conv_clip_grads(grads, 1.0)
        assert math.isnan(float(norm)) if math.isnan(bad) else math.isinf(float(norm))
        assert torch.isnan(grads[0][500])
        assert torch.isnan(grads[1]).all() if math.isnan(bad) else not grads[1].any()


def test_factor_of_one_in_place_keeps_the_bits(ic):
    grads = tensors([3000, 41])
    before = [g.clone() for g in grads]
    ic.conv_clip_grads(grads, 1e9)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))


def test_no_tensors(ic):
    norm = torch.ones(1, device="cuda")
    assert float(ic.conv_clip_grads([torch.empty(0, device="cuda")], 1.0, norm=norm)) == 0.0


def test_repeats_in_graphs_and_on_streams(ic):
    grads = tensors([200000, 7, 90001])
    apart = [torch.empty_like(g) for g in grads]
    first = ic.conv_clip_grads(grads, 1.0, out=apart).clone()
    want = [t.clone() for t in apart]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n = ic.conv_clip_grads(grads, 1.0, out=apart, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(n, first) and all(torch.equal(a, b) for a, b in zip(apart, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = ic.conv_clip_grads(grads, 1.0, out=apart)
    for t in apart:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(n, first) and all(torch.equal(a, b) for a, b in zip(apart, want))

"""The 8-bit operators together, as a residual block uses them: block norm with
8-bit rows, expansion, quantisation, projection, block norm; backward through
quantised gradients; all gradients clipped.  Every result against its
definition on the values the operator was given."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import blocks as ob  # noqa: E402

BF16, F32, E4, E5 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e5m2


@pytest.mark.parametrize("m,c,hidden,groups", [(13, 256, 512, 1), (392, 136, 520, 8)])
def test_block_forward_backward_and_clipping(m, c, hidden, groups):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import int8_conv2d_fprop_gb300 as ic
    g = torch.Generator(device="cuda").manual_seed(m)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def check(got, want, bound):
        assert bool(((got.double() - want).abs() <= bound).all())

    stream, before = normal(m, c).to(BF16), normal(m, c).to(BF16)
    gain, pg, gate = 1 + normal(c) / 8, 1 + normal(c) / 8, (1 + normal(groups, c) / 4).to(BF16)
    w1, w2 = (normal(hidden, c) / c ** 0.5).to(BF16), (normal(c, hidden) / hidden ** 0.5).to(BF16)
    prstd, rstd, prstd2, rstd2 = (torch.empty(m, device="cuda") for _ in range(4))
    # the end of the block before, and this one's rows in 8 bits
    h, xq, xs = ic.conv_block_norm(before, stream, post_norm=True, post_gain=pg, gate=gate, gain=gain, dtype=E4, post_rstd=prstd, rstd=rstd)
    want = ob.block_norm(before, stream, True, pg, gate, 1.0, 1.0, gain, 1e-6)
    assert ob.check_quantized(xq, xs, want["y"][0], 1, want["y"][1]) is None
    q1, s1, q1t, s1t = ic.conv_quantize(w1, tile=128, columns=True)
    q2, s2, q2t, s2t = ic.conv_quantize(w2, tile=128, columns=True)
    z = torch.empty(m, hidden, dtype=BF16, device="cuda")
    a = ic.conv_linear_fp8(xq, xs, q1, s1, activation="silu", preact=z)
    wy, wz, size = ob.linear_fp8(xq, xs, q1, s1, None, "silu")
    by, bz = ob.linear_fp8_bounds(c, wy, wz, size, "silu", None, BF16)
    check(a, wy, by)
    check(z, wz, bz)
    aq, as_, at, ats = ic.conv_quantize(a, columns=True)
    b = ic.conv_linear_fp8(aq, as_, q2, s2)
    h2, y = ic.conv_block_norm(b, h, post_norm=True, post_gain=pg, gate=gate, gain=gain, post_rstd=prstd2, rstd=rstd2)
    want = ob.block_norm(b, h, True, pg, gate, 1.0, 1.0, gain, 1e-6)
    check(y, want["y"][0], ob.rounded(want["y"][1], want["y"][0], BF16))
    # backward
    dy = normal(m, c).to(BF16)
    db, dh = torch.empty_like(b), torch.empty_like(h)
    grads = {"gate": torch.empty(groups, c, device="cuda"), "pg": torch.empty_like(pg), "gain": torch.empty_like(gain)}
    ic.conv_block_norm_grad(dy, None, b, h2, post_norm=True, post_gain=pg, gate=gate, gain=gain, post_rstd=prstd2, rstd=rstd2, dx=db,
                            dskip=dh, dgate=grads["gate"], dpost_gain=grads["pg"], dgain=grads["gain"])
    ref = ob.block_norm_grad(dy, None, b, h2, True, pg, gate, groups, 1.0, 1.0, gain, prstd2, rstd2)
    for got, k, d in ((db, "dx", BF16), (dh, "dskip", BF16), (grads["gate"], "dgate", F32), (grads["pg"], "dpost_gain", F32),
                      (grads["gain"], "dgain", F32)):
        check(got, ref[k][0], ob.rounded(ref[k][1], ref[k][0], d))
    dq, ds, dt, dts = ic.conv_quantize(db, columns=True, dtype=E5)
    da = ic.conv_linear_fp8(dq, ds, q2t, s2t)
    grads["w2"] = ic.conv_linear_fp8(dt, dts, at, ats, dtype=F32)
    eq, es, et, ets = ic.conv_quantize(da, preact=z, activation="silu", columns=True, dtype=E5)
    xt, xts = ic.conv_quantize((xq.float() * ob.per_element(xs, m, c).float()).to(BF16), rows=False, columns=True)
    grads["w1"] = ic.conv_linear_fp8(et, ets, xt, xts, dtype=F32)
    for got, (p, ps, r, rs) in ((grads["w2"], (dt, dts, at, ats)), (grads["w1"], (et, ets, xt, xts))):
        want, _, size = ob.linear_fp8(p, ps, r, rs)
        check(got, want, ob.linear_fp8_bounds(m, want, want, size, "none", None, F32)[0])
    dn = ic.conv_linear_fp8(eq, es, q1t, s1t)
    dstream = torch.empty_like(stream)
    ic.conv_block_norm_grad(dn, dh, before, h, post_norm=True, post_gain=pg, gate=gate, gain=gain, post_rstd=prstd, rstd=rstd, dskip=dstream)
    ref = ob.block_norm_grad(dn, dh, before, h, True, pg, gate, groups, 1.0, 1.0, gain, prstd, rstd)
    check(dstream, ref["dskip"][0], ob.rounded(ref["dskip"][1], ref["dskip"][0], BF16))
    # all gradients by their norm
    all_grads = list(grads.values())
    norm, want = ob.clip(all_grads, 0.1, 1e-6)
    got = ic.conv_clip_grads(all_grads, 0.1)
    assert abs(float(got) - norm) <= 2.0 ** -19 * norm
    for t, w in zip(all_grads, want):
        check(t, w, 2.0 ** -19 * w.abs() + 2.0 ** -126)
    assert ic.device_status() == 0

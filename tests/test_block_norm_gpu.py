"""conv_block_norm and its gradients on the GPU against their definitions in 64
bits and against differences: widths held by warps, blocks and shared memory,
types, gates, optional parts, layouts, in-place outputs, 8-bit outputs,
infinities, empty extents, streams and graphs."""
import itertools

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import blocks as ob  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E4 = torch.float8_e4m3fn
EPS = 1e-6


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


def place(v, dtype, layout="rows"):
    m, n = v.shape
    nan = float("nan")
    if layout == "rows":
        t = torch.empty(m, n, device="cuda", dtype=dtype)
    elif layout == "padded":
        t = torch.full((m, (n + 7) // 8 * 8 + 8), nan, device="cuda", dtype=dtype)[:, :n]
    elif layout == "odd":
        t = torch.full((m, n + 1 + n % 2), nan, device="cuda", dtype=dtype)[:, :n]
    elif layout == "shifted":
        t = torch.full((m, (n + 7) // 8 * 8 + 8), nan, device="cuda", dtype=dtype)[:, 1:n + 1]
    elif layout == "cols":
        t = torch.full((n, (m + 7) // 8 * 8), nan, device="cuda", dtype=dtype)[:, :m].t()
    else:
        t = torch.full((m, 2 * n), nan, device="cuda", dtype=dtype)[:, ::2]
    return t.copy_(v)


def check(got, want, dtype, what):
    value, bound = want
    bound = ob.rounded(bound, value, dtype)
    bad = ~((got.double().reshape(value.shape) - value).abs() <= bound)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at {bad.nonzero()[0].tolist()}, "
                                 f"worst {float(((got.double().reshape(value.shape) - value).abs() / bound).nan_to_num().max()):.3g}")


class Case:
    """Inputs of one call and its expected results."""

    def __init__(self, m, c, dt=BF16, stream=None, groups=1, post=True, skip=True, gate=True, gains=True, par=F32, gate_dt=None,
                 layout="rows", skip_layout=None, seed=0, skip_scale=0.75, branch_scale=-1.5):
        g = torch.Generator(device="cuda").manual_seed(seed + m + c)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        self.m, self.c, self.dt, self.stream, self.groups, self.post, self.par = m, c, dt, stream or dt, groups, post, par
        self.x = place(normal(m, c) * (0.5 + torch.rand(m, 1, generator=g, device="cuda")), dt, layout)
        self.skip = place(2 * normal(m, c), self.stream, skip_layout or layout) if skip else None
        self.gate = (1 + 0.5 * normal(groups, c)).to(gate_dt or dt) if gate else None
        self.pg = (1 + 0.2 * normal(c)).to(par) if gains and post else None
        self.g = (1 + 0.2 * normal(c)).to(par) if gains else None
        self.ss, self.bs = skip_scale, branch_scale
        self.layout, self.normal = layout, normal

    def forward(self, ic, **given):
        prstd = torch.zeros(self.m, device="cuda") if self.post else None
        rstd = torch.zeros(self.m, device="cuda")
        out = ic.conv_block_norm(self.x, self.skip, post_norm=self.post, post_gain=self.pg, gate=self.gate, skip_scale=self.ss,
                                 branch_scale=self.bs, gain=self.g, eps=EPS, post_rstd=prstd, rstd=rstd, **given)
        return out, prstd, rstd

    def want(self):
        return ob.block_norm(self.x, self.skip, self.post, self.pg, self.gate, self.ss, self.bs, self.g, EPS)

    def check_forward(self, ic, **given):
        want = self.want()
        (s, y, *scale), prstd, rstd = self.forward(ic, **given)
        if s is not None:
            check(s, want["sum"], self.stream, "sum")
        if scale:
            v, ev = want["y"]
            assert ob.check_quantized(y, scale[0], v, 1, ev) is None, ob.check_quantized(y, scale[0], v, 1, ev)
        else:
            check(y, want["y"], self.dt, "y")
        check(rstd, want["rstd"], F32, "rstd")
        if self.post:
            check(prstd, want["post_rstd"], F32, "post_rstd")
        return s, y

    def check_grad(self, ic, dy=True, ds=True, wanted=("dx", "dskip", "dgate", "dgain", "dpost_gain"), out_layout=None, dgate_dt=F32,
                   in_place=False):
        want = self.want()
        h = place(want["sum"][0], self.stream, self.layout)
        rs = ((h.double() ** 2).mean(1) + EPS).rsqrt().float()
        rx = want["post_rstd"][0].float() if self.post else None
        a = place(self.normal(self.m, self.c) / 4, self.dt, self.layout) if dy else None
        b = place(self.normal(self.m, self.c) / 4, self.stream, self.layout) if ds else None
        need_x = self.post or "dgate" in wanted
        ref = ob.block_norm_grad(a, b, self.x if need_x else None, h, self.post, self.pg, self.gate, self.groups, self.ss, self.bs,
                                 self.g, rx, rs)
        out = {"dx": (self.m, self.c, self.dt), "dskip": (self.m, self.c, self.stream)}
        lay = out_layout or self.layout
        given = {k: place(torch.zeros(m, c, device="cuda"), d, lay) for k, (m, c, d) in out.items() if k in wanted}
        if in_place:
            given["dx"], given["dskip"] = a, b
        if "dgate" in wanted:
            given["dgate"] = torch.full((self.groups, self.c), float("nan"), dtype=dgate_dt, device="cuda")
        for k in ("dgain", "dpost_gain"):
            if k in wanted and k in ref:
                given[k] = torch.full((self.c,), float("nan"), dtype=self.par, device="cuda")
        ic.conv_block_norm_grad(a, b, self.x if need_x else None, h if dy else None, post_norm=self.post, post_gain=self.pg,
                                gate=self.gate, skip_scale=self.ss, branch_scale=self.bs, gain=self.g, post_rstd=rx, rstd=rs if dy else None,
                                **given)
        types = {"dx": self.dt, "dskip": self.stream, "dgate": dgate_dt, "dgain": self.par, "dpost_gain": self.par}
        for k, v in given.items():
            check(v, ref[k], types[k], k)


WIDTHS = [(1, 1), (3, 7), (9, 8), (20, 64), (33, 200), (17, 256), (25, 264), (40, 512), (13, 520), (7, 1000), (64, 1024), (5, 2056),
          (13, 4096), (6, 4104), (3, 8192), (3, 8200), (2, 16384), (2, 20001), (2000, 96), (1500, 520), (700, 2048)]


@pytest.mark.parametrize("m,c", WIDTHS)
def test_forward_widths(ic, m, c):
    for stream in (BF16, F32):
        Case(m, c, BF16, stream).check_forward(ic)
    Case(m, c, BF16, post=False, skip=False, gate=False, branch_scale=1.0).check_forward(ic)
    Case(m, c, BF16).check_forward(ic, dtype=E4)


@pytest.mark.parametrize("m,c", WIDTHS)
def test_gradient_widths(ic, m, c):
    for stream in (BF16, F32):
        Case(m, c, BF16, stream).check_grad(ic)
    Case(m, c, BF16, post=False).check_grad(ic)


@pytest.mark.parametrize("dt,stream,par,gate_dt", [(F16, F16, F32, F16), (F16, F32, F16, F32), (BF16, BF16, BF16, F32), (F32, F32, F32, F32)])
@pytest.mark.parametrize("c", [72, 384, 1504, 5000, 9000])
def test_types(ic, dt, stream, par, gate_dt, c):
    Case(11, c, dt, stream, par=par, gate_dt=gate_dt).check_forward(ic)
    Case(11, c, dt, stream, par=par, gate_dt=gate_dt).check_forward(ic, dtype=E4)
    Case(11, c, dt, stream, par=par, gate_dt=gate_dt).check_grad(ic, dgate_dt=gate_dt)


@pytest.mark.parametrize("m,groups", [(12, 12), (12, 3), (64, 2), (3000, 3000), (3000, 750), (1300, 650), (6000, 3), (2432, 608), (4000, 8)])
@pytest.mark.parametrize("c", [136, 600])
def test_gates(ic, m, groups, c):
    Case(m, c, groups=groups).check_forward(ic)
    Case(m, c, groups=groups).check_grad(ic)
    Case(m, c, groups=groups, post=False).check_grad(ic, dgate_dt=BF16)


def test_gate_rows_apart(ic):
    # gates as one of several vectors that a projection made
    case = Case(60, 200, groups=5)
    whole = torch.randn(5, 6 * 200, device="cuda").to(BF16)
    case.gate = whole[:, 400:600]
    case.check_forward(ic)
    case.check_grad(ic)


@pytest.mark.parametrize("layout,other", [("padded", "padded"), ("odd", "odd"), ("shifted", "shifted"), ("odd", "rows"), ("cols", "cols"),
                                          ("spread", "rows"), ("rows", "shifted")])
@pytest.mark.parametrize("m,c", [(30, 133), (19, 515), (300, 2001), (9, 5001), (40, 256)])
def test_layouts(ic, layout, other, m, c):
    case = Case(m, c, F16, F32, layout=layout, skip_layout=other)
    case.check_forward(ic)
    case.check_forward(ic, dtype=E4)
    s, y = place(torch.zeros(m, c, device="cuda"), F32, other), place(torch.zeros(m, c, device="cuda"), F16, other)
    case.check_forward(ic, sum=s, out=y)
    case.check_grad(ic, out_layout=other)
    Case(m, c, BF16, layout=layout, groups=m if m < 50 else 1).check_grad(ic, out_layout=other)


@pytest.mark.parametrize("skip,gate,gains,post", list(itertools.product((False, True), repeat=4)))
@pytest.mark.parametrize("c", [200, 1100])
def test_optional_parts(ic, skip, gate, gains, post, c):
    Case(21, c, skip=skip, gate=gate, gains=gains, post=post).check_forward(ic)
    Case(21, c, skip=skip, gate=gate, gains=gains, post=post).check_grad(ic)


@pytest.mark.parametrize("c", [200, 1100, 9001])
def test_gradients_wanted(ic, c):
    for dy, ds in ((True, False), (False, True)):
        for post in (True, False):
            wanted = ["dx", "dskip", "dgate"] + (["dgain"] if dy else []) + (["dpost_gain"] if post else [])
            Case(19, c, post=post).check_grad(ic, dy, ds, wanted)
            for k in wanted:
                Case(19, c, post=post, seed=1).check_grad(ic, dy, ds, (k,))


def test_sum_alone_and_norm_alone(ic):
    case = Case(40, 320)
    want = case.want()
    s, y = ic.conv_block_norm(case.x, case.skip, post_norm=True, post_gain=case.pg, gate=case.gate, skip_scale=case.ss,
                              branch_scale=case.bs, norm=False, eps=EPS)
    assert y is None
    check(s, want["sum"], BF16, "sum")
    s, y = ic.conv_block_norm(case.x, gain=case.g, eps=EPS)
    assert s is None
    check(y, ob.block_norm(case.x, None, False, None, None, 1.0, 1.0, case.g, EPS)["y"], BF16, "y")


@pytest.mark.parametrize("c", [200, 1100, 9000])
def test_in_place(ic, c):
    case = Case(25, c)
    want = case.want()
    x, skip = case.x.clone(), case.skip.clone()
    ic.conv_block_norm(x, skip, post_norm=True, post_gain=case.pg, gate=case.gate, skip_scale=case.ss, branch_scale=case.bs, gain=case.g,
                       eps=EPS, sum=skip, out=x)
    check(skip, want["sum"], BF16, "sum")
    check(x, want["y"], BF16, "y")
    x = case.x.clone()
    ic.conv_block_norm(x, case.skip, post_norm=True, post_gain=case.pg, gate=case.gate, skip_scale=case.ss, branch_scale=case.bs, norm=False,
                       eps=EPS, sum=x)
    check(x, want["sum"], BF16, "sum")


@pytest.mark.parametrize("c", [200, 1100, 8200])
def test_gradients_in_place(ic, c):
    case = Case(25, c)
    want = case.want()
    h = place(want["sum"][0], BF16)
    rs, rx = ((h.double() ** 2).mean(1) + EPS).rsqrt().float(), want["post_rstd"][0].float()
    dy, ds = case.normal(25, c).to(BF16), case.normal(25, c).to(BF16)
    ref = ob.block_norm_grad(dy, ds, case.x, h, True, case.pg, case.gate, 1, case.ss, case.bs, case.g, rx, rs)
    ic.conv_block_norm_grad(dy, ds, case.x, h, post_norm=True, post_gain=case.pg, gate=case.gate, skip_scale=case.ss, branch_scale=case.bs,
                            gain=case.g, post_rstd=rx, rstd=rs, dx=dy, dskip=ds)
    check(dy, ref["dx"], BF16, "dx")
    check(ds, ref["dskip"], BF16, "dskip")


def test_neighbours_stay(ic):
    m, c = 21, 203
    case = Case(m, c, F16, F32)
    bufs = {k: torch.full((m, c + 5), 7.0, dtype=d, device="cuda") for k, d in (("sum", F32), ("out", F16), ("dx", F16), ("dskip", F32))}
    case.check_forward(ic, sum=bufs["sum"][:, 2:c + 2], out=bufs["out"][:, 2:c + 2])
    want = case.want()
    h = place(want["sum"][0], F32)
    rs, rx = ((h.double() ** 2).mean(1) + EPS).rsqrt().float(), want["post_rstd"][0].float()
    ic.conv_block_norm_grad(case.normal(m, c).to(F16), None, case.x, h, post_norm=True, post_gain=case.pg, gate=case.gate, gain=case.g,
                            post_rstd=rx, rstd=rs, dx=bufs["dx"][:, 2:c + 2], dskip=bufs["dskip"][:, 2:c + 2])
    for b in bufs.values():
        assert (b[:, :2] == 7).all() and (b[:, c + 2:] == 7).all() and not (b[:, 2:c + 2] == 7).all()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("c", [200, 1100, 9000])
def test_infinities_and_nan_stay_in_their_row(ic, bad, c):
    case = Case(19, c)
    case.x[4, 5] = bad
    case.skip[7, c - 1] = bad
    (s, y), _, _ = case.forward(ic)
    assert torch.isnan(y[4]).all() and torch.isnan(y[7]).all() and torch.isnan(s[4]).all()
    keep = [i for i in range(19) if i not in (4, 7)]
    clean = Case(19, c)
    (s2, y2), _, _ = clean.forward(ic)
    assert torch.equal(y[keep], y2[keep]) and torch.equal(s[keep], s2[keep])


def test_empty_extents(ic):
    x = torch.empty(0, 40, device="cuda", dtype=BF16)
    s, y = ic.conv_block_norm(x, x, post_norm=True, gate=torch.ones(40, device="cuda"))
    assert s.shape == y.shape == (0, 40)
    dg, dpg, dgate = (torch.ones(40, device="cuda"), torch.ones(40, device="cuda"), torch.ones(3, 40, device="cuda"))
    none = torch.empty(0, device="cuda")
    ic.conv_block_norm_grad(x, x, x, x, post_norm=True, post_rstd=none, rstd=none, dgain=dg, dpost_gain=dpg, dgate=dgate)
    assert not dg.any() and not dpg.any() and not dgate.any()


@pytest.mark.parametrize("m,c,groups", [(40, 48, 4), (33, 600, 33)])
def test_gradients_against_differences(ic, m, c, groups):
    """Central differences of the forward call in 32 bits along a random
    direction of each input.  A difference of step e is off by e^2 times the
    third derivative (some units here) and by the forward call's rounding,
    2^-22 of the loss's terms (about 500 in 2-norm), over e."""
    case = Case(m, c, F32, groups=groups, gate_dt=F32, skip_scale=0.75, branch_scale=0.5)
    wy, ws = case.normal(m, c) / 8, case.normal(m, c) / 8

    def loss(x, skip, gate, pg, g):
        s, y = ic.conv_block_norm(x, skip, post_norm=True, post_gain=pg, gate=gate, skip_scale=case.ss, branch_scale=case.bs, gain=g, eps=EPS)
        return float((y.double() * wy.double()).sum() + (s.double() * ws.double()).sum())

    (s, y), prstd, rstd = case.forward(ic)
    grads = {k: torch.empty_like(v) for k, v in (("dx", case.x), ("dskip", case.skip), ("dgate", case.gate), ("dpost_gain", case.pg),
                                                 ("dgain", case.g))}
    ic.conv_block_norm_grad(wy, ws, case.x, s, post_norm=True, post_gain=case.pg, gate=case.gate, skip_scale=case.ss,
                            branch_scale=case.bs, gain=case.g, post_rstd=prstd, rstd=rstd, **grads)
    inputs = [case.x, case.skip, case.gate, case.pg, case.g]
    e = 2.0 ** -7
    for i, k in enumerate(grads):
        d = case.normal(*inputs[i].shape)
        d /= d.norm()
        at = [[v + sign * e * d if j == i else v for j, v in enumerate(inputs)] for sign in (1, -1)]
        slope = (loss(*at[0]) - loss(*at[1])) / (2 * e)
        want = float((grads[k].double() * d.double()).sum())
        assert abs(slope - want) < 20 * e * e + 2.0 ** -22 * 500 / e, k


@pytest.mark.parametrize("c,groups", [(264, 1), (2048, 4)])
def test_repeats_in_graphs_and_on_streams(ic, c, groups):
    case = Case(600, c, groups=groups)
    dy, ds = case.normal(600, c).to(BF16), case.normal(600, c).to(BF16)

    def step():
        (s, y), prstd, rstd = case.forward(ic)
        out = {"dx": torch.empty_like(case.x), "dskip": torch.empty_like(case.x), "dgate": torch.empty(groups, c, device="cuda"),
               "dgain": torch.empty(c, device="cuda"), "dpost_gain": torch.empty(c, device="cuda")}
        ic.conv_block_norm_grad(dy, ds, case.x, s, post_norm=True, post_gain=case.pg, gate=case.gate, skip_scale=case.ss,
                                branch_scale=case.bs, gain=case.g, post_rstd=prstd, rstd=rstd, **out)
        return [s, y] + list(out.values())

    first = step()
    for a, b in zip(first, step()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        inside = step()
    for t in inside:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, inside):
        assert torch.equal(a, b)

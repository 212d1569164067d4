"""The channel-mixing operators as measured cases: the matrix product with
bias, activation and residual (forward and gradients) and the layer norm over
channels (forward and gradients), each in a plain form and as the library's
own calls.

Rows are tokens or the pixels of a channels-last image, columns are channels.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "i32": torch.int32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _linear(name, m, k, n, dt, act, bias=True, residual=False, preact=False, pad=0, wt=False):
    return {"name": name, "op": "linear", "m": m, "k": k, "n": n, "dt": dt, "act": act, "bias": bias,
            "residual": residual, "preact": preact, "pad": pad, "wt": wt}


def _linear_grad(name, m, k, n, dt, act, bias=True, pad=0, wt=False):
    return {"name": name, "op": "linear_grad", "m": m, "k": k, "n": n, "dt": dt, "act": act, "bias": bias,
            "pad": pad, "wt": wt}


def _norm(name, m, c, dt, out, stats=False, pad=0):
    return {"name": name, "op": "norm", "m": m, "c": c, "dt": dt, "out": out, "stats": stats, "pad": pad}


def _norm_grad(name, m, c, dt, residual=False, pad=0):
    return {"name": name, "op": "norm_grad", "m": m, "c": c, "dt": dt, "residual": residual, "pad": pad}


def listed():
    return [
        # one token through a square projection with its residual: a call's latency
        _linear("linear_one_token", 1, 1024, 1024, "bf16", "none", residual=True),
        # a small decoding batch through an expansion: streaming 134 MB of weights
        _linear("linear_decode_16", 16, 4096, 16384, "bf16", "silu"),
        # odd sizes, odd row strides and a weight kept input-major, in f16
        _linear("linear_ragged", 1777, 1003, 515, "f16", "relu", residual=True, pad=3, wt=True),
        # the pixels of 64 images of 28 x 28 through a channel expansion, training forward
        _linear("linear_pixels", 50176, 512, 2048, "bf16", "gelu", preact=True),
        # a long prompt or a training batch: a large expansion
        _linear("linear_large", 8192, 4096, 16384, "bf16", "gelu_tanh"),
        # a few hundred rows through a narrow layer: many launches for little work
        _linear_grad("linear_grad_small", 333, 192, 257, "f16", "relu", pad=1),
        # the pixels again, backward: a weight gradient over 50176 rows with few output tiles
        _linear_grad("linear_grad_pixels", 50176, 256, 1024, "bf16", "gelu"),
        # a training batch, backward
        _linear_grad("linear_grad_large", 8192, 4096, 4096, "bf16", "silu"),
        # one row of each request while decoding
        _norm("norm_rows_16", 16, 4096, "bf16", "bf16"),
        # the int32 accumulators of 32 x 256 x 56 x 56 convolution outputs, channels last
        _norm("norm_accumulators", 100352, 256, "i32", "bf16", stats=True),
        # the 64 x 28 x 28 pixels of 512 channels, backward with the skip's gradient
        _norm_grad("norm_grad_pixels", 50176, 512, "bf16", residual=True),
        # odd width and odd row stride, in f16
        _norm_grad("norm_grad_ragged", 2047, 5001, "f16", pad=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size between lo and hi, spread over the logarithm; two in three are multiples of 8."""
    v = _log(rng, lo, hi)
    if v >= 16 and rng.random() < 0.67:
        v = v // 8 * 8
    return v


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_grad", "norm", "norm_grad"))
    dt = rng.choice(("bf16", "f16"))
    pad = rng.choice((0, 0, 0, 8, 1))
    while True:
        if op in ("linear", "linear_grad"):
            m, k, n = _size(rng, 1, 65536), _size(rng, 64, 8192), _size(rng, 64, 16384)
            if m * k * n > 8192 * 4096 * (16384 if op == "linear" else 4096) or m * (k + n) > 50176 * 4608:
                continue
        else:
            m, k = _size(rng, 1, 131072), _size(rng, 64, 16384)
            if m * k > 50176 * 512:
                continue
        break
    if op == "linear":
        c = _linear("", m, k, n, dt, rng.choice(ACTS), rng.random() < 0.8, rng.random() < 0.4, rng.random() < 0.3, pad,
                    rng.random() < 0.25)
    elif op == "linear_grad":
        c = _linear_grad("", m, k, n, dt, rng.choice(ACTS), rng.random() < 0.8, pad, rng.random() < 0.25)
    elif op == "norm":
        x = rng.choice((dt, dt, "f32", "i32"))
        c = _norm("", m, k, x, "f32" if x == "f32" else dt, rng.random() < 0.5, pad)
    else:
        c = _norm_grad("", m, k, rng.choice((dt, dt, "f32")), rng.random() < 0.5, pad)
    del c["name"]
    return c


def _matrix(values, dtype, pad):
    """`values` rounded to dtype, in rows of `pad` more elements than they use."""
    rows, cols = values.shape
    t = torch.empty(rows, cols + pad, dtype=dtype, device=values.device)[:, :cols]
    return t.copy_(values)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case)
    dt, pad, m = DTYPES[case["dt"]], case["pad"], case["m"]
    if case["op"] in ("linear", "linear_grad"):
        k, n = case["k"], case["n"]
        s["x"] = _matrix(normal(m, k), dt, pad)
        w = normal(n, k) / math.sqrt(k)
        s["w"] = _matrix(w.t(), dt, pad).t() if case["wt"] else _matrix(w, dt, pad)
        s["b"] = (0.2 * normal(n)).to(dt) if case["bias"] and case["op"] == "linear" else None
        if case["op"] == "linear":
            s["r"] = _matrix(normal(m, n), dt, pad) if case["residual"] else None
        else:
            s["dy"] = _matrix(normal(m, n) / 16, dt, pad)
            s["z"] = None if case["act"] == "none" else _matrix(normal(m, n), dt, pad)
        return s
    c = case["c"]
    if case["dt"] == "i32":
        # sums of a convolution's products: some channels larger, and off centre
        x = torch.round((normal(m, c) + 0.5 * normal(c)) * torch.exp(normal(c) + 9))
        s["scale"] = 2.0 ** -13
    else:
        x = normal(m, c) * (0.5 + torch.rand(m, 1, generator=g, device="cuda")) + 0.5 * normal(c)
        s["scale"] = 1.0
    s["x"] = _matrix(x, dt, pad)
    s["g"] = 1 + 0.2 * normal(c)
    s["h"] = 0.2 * normal(c)
    s["eps"] = 1e-5
    if case["op"] == "norm_grad":
        s["dy"] = _matrix(normal(m, c) / 16, dt, pad)
        s["dr"] = _matrix(normal(m, c) / 16, dt, pad) if case["residual"] else None
        # the statistics that the forward pass kept
        f = s["x"].double()
        s["mean"] = f.mean(1).float()
        s["rstd"] = (f.var(1, unbiased=False) + s["eps"]).rsqrt().float()
    return s


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        u = math.sqrt(2 / math.pi)
        t = torch.tanh(u * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * u * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _plain(s):
    op = s["op"]
    if op == "linear":
        dt = s["x"].dtype
        z = s["x"].float() @ s["w"].float().t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(z, s["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return (y.to(dt), z.to(dt)) if s["preact"] else y.to(dt)
    if op == "linear_grad":
        dt = s["x"].dtype
        dz = s["dy"].float()
        if s["z"] is not None:
            dz = dz * _act_slope(s["z"].float(), s["act"])
        out = [(dz @ s["w"].float()).to(dt), (dz.t() @ s["x"].float()).to(dt)]
        return out + [dz.sum(0)] if s["bias"] else out
    x = s["x"].float() * s["scale"]
    if op == "norm":
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + s["eps"])
        y = (d * rstd * s["g"] + s["h"]).to(DTYPES[s["out"]])
        return (y, mean[:, 0], rstd[:, 0]) if s["stats"] else y
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    t = dy * s["g"]
    dx = rstd * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
    if s["dr"] is not None:
        dx = dx + s["dr"].float()
    return dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)


def _own(s):
    import int8_conv2d_fprop_gb300 as ic
    op, x = s["op"], s["x"]
    if op == "linear":
        z = torch.empty(s["m"], s["n"], dtype=x.dtype, device=x.device) if s["preact"] else None
        y = ic.conv_linear(x, s["w"], s["b"], activation=s["act"], residual=s["r"], preact=z)
        return (y, z) if s["preact"] else y
    if op == "linear_grad":
        dx, dw = torch.empty(x.shape, dtype=x.dtype, device=x.device), torch.empty(s["w"].shape, dtype=x.dtype, device=x.device)
        db = torch.empty(s["n"], dtype=torch.float32, device=x.device) if s["bias"] else None
        ic.conv_linear_grad(s["dy"], x, s["w"], preact=s["z"], activation=s["act"], dx=dx, dw=dw, dbias=db)
        return [dx, dw, db] if s["bias"] else [dx, dw]
    if op == "norm":
        y = torch.empty(x.shape, dtype=DTYPES[s["out"]], device=x.device)
        mean = torch.empty(s["m"], dtype=torch.float32, device=x.device) if s["stats"] else None
        rstd = torch.empty(s["m"], dtype=torch.float32, device=x.device) if s["stats"] else None
        ic.conv_layer_norm(x, s["g"], s["h"], eps=s["eps"], scale=s["scale"], out=y, mean=mean, rstd=rstd)
        return (y, mean, rstd) if s["stats"] else y
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dg, dh = torch.empty_like(s["g"]), torch.empty_like(s["g"])
    ic.conv_layer_norm_grad(s["dy"], x, s["g"], s["mean"], s["rstd"], residual_grad=s["dr"], dx=dx, dgain=dg, dshift=dh)
    return dx, dg, dh


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    m = case["m"]
    if case["op"] in ("linear", "linear_grad"):
        k, n = case["k"], case["n"]
        if case["op"] == "linear":
            values = m * k + n * k + m * n * (1 + case["residual"] + case["preact"]) + n * case["bias"]
            return {"bytes": 2 * values, "flops": 2 * m * n * k}
        values = m * n * (1 + (case["act"] != "none")) + 2 * m * k + 2 * n * k
        return {"bytes": 2 * values + 4 * n * case["bias"], "flops": 4 * m * n * k}
    c, size = case["c"], {"bf16": 2, "f16": 2, "f32": 4, "i32": 4}
    if case["op"] == "norm":
        return {"bytes": m * c * (size[case["dt"]] + size[case["out"]]) + 8 * c + 8 * m * case["stats"], "flops": 8 * m * c}
    return {"bytes": m * c * size[case["dt"]] * (3 + case["residual"]) + 8 * m + 12 * c, "flops": 14 * m * c}


def exact(case, seed):
    """The operators' definitions in 64 bits: the Gaussian's distribution
    function through erfc, the logistic function through torch.sigmoid, and
    the layer norm's gradient through the normalised rows."""
    s = prepare(case, seed)
    x = s["x"].double()

    def phi(v):
        return 0.5 * torch.special.erfc(-v / math.sqrt(2.0))

    def tanh_arg(v):
        return 2 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)

    if case["op"] == "linear":
        z = torch.mm(x, s["w"].double().t())
        if s["b"] is not None:
            z += s["b"].double()
        act = case["act"]
        y = (z.clamp(min=0) if act == "relu" else z * phi(z) if act == "gelu" else
             z * torch.sigmoid(tanh_arg(z)) if act == "gelu_tanh" else z * torch.sigmoid(z) if act == "silu" else z)
        if s["r"] is not None:
            y = y + s["r"].double()
        return (y, z) if case["preact"] else y
    if case["op"] == "linear_grad":
        d, act = s["dy"].double(), case["act"]
        if s["z"] is not None:
            z = s["z"].double()
            if act == "relu":
                d = d.masked_fill(z <= 0, 0)
            elif act == "gelu":
                d = d * (phi(z) + z * torch.exp(-z * z / 2) * (2 * math.pi) ** -0.5)
            elif act == "gelu_tanh":
                p = torch.sigmoid(tanh_arg(z))
                d = d * (p + z * p * (1 - p) * 2 * math.sqrt(2.0 / math.pi) * (1 + 0.134145 * z * z))
            else:
                p = torch.sigmoid(z)
                d = d * (p + z * p * (1 - p))
        out = [torch.mm(d, s["w"].double()), torch.mm(d.t(), x)]
        return out + [d.sum(0)] if case["bias"] else out
    x = x * s["scale"]
    if case["op"] == "norm":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + s["eps"]).rsqrt()
        y = (x - mean[:, None]) * rstd[:, None] * s["g"].double() + s["h"].double()
        return (y, mean, rstd) if case["stats"] else y
    d, c = s["dy"].double(), x.shape[1]
    r = s["rstd"].double()[:, None]
    n = (x - s["mean"].double()[:, None]) * r
    t = d * s["g"].double()
    dx = r / c * (c * t - t.sum(1, keepdim=True) - n * (t * n).sum(1, keepdim=True))
    if s["dr"] is not None:
        dx = dx + s["dr"].double()
    return dx, (d * n).sum(0), d.sum(0)

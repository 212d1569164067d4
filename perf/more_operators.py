"""The 8-bit channel product and what stands around it as measured cases: the
quantisation to 8-bit floats with a scale for each block of 128, the matrix
product of such operands, the norms before and after a residual block fused
with its gate and scales (forward and gradients), and the clipping of many
gradient tensors by their global norm; each in a plain form and as the
library's own calls.

Rows are tokens or the pixels of a channels-last image, columns are channels.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1, "e5m2": 1}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
LEAST_SCALE = 2.0 ** -126
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
BLOCK = 128


def _quantize(name, m, c, dt, to="e4m3", tile=1, rows=True, columns=False, act="none", pad=0):
    return {"name": name, "op": "quantize", "m": m, "c": c, "dt": dt, "to": to, "tile": tile, "rows": rows,
            "columns": columns, "act": act, "pad": pad}


def _linear(name, m, k, n, out, act="none", x8="e4m3", w_tile=128, bias=False, residual=False, preact=False):
    return {"name": name, "op": "linear", "m": m, "k": k, "n": n, "out": out, "act": act, "x8": x8, "w_tile": w_tile,
            "bias": bias, "residual": residual, "preact": preact}


def _norm(name, m, c, dt, stream, groups, post=True, stats=False, out8=False, pad=0):
    return {"name": name, "op": "block_norm", "m": m, "c": c, "dt": dt, "stream": stream, "groups": groups, "post": post,
            "stats": stats, "out8": out8, "pad": pad}


def _norm_grad(name, m, c, dt, stream, groups, post=True, pad=0):
    return {"name": name, "op": "block_norm_grad", "m": m, "c": c, "dt": dt, "stream": stream, "groups": groups,
            "post": post, "pad": pad}


def _clip(name, dt, layers, width, hidden):
    return {"name": name, "op": "clip", "dt": dt, "layers": layers, "width": width, "hidden": hidden}


def listed():
    return [
        # the activations of a long prompt before an 8-bit product
        _quantize("quantize_prompt", 16384, 4096, "bf16"),
        # an expansion's loss gradient in training: through GELU's slope, in rows for one product and in columns for
        # the other; odd width, odd row stride
        _quantize("quantize_gradient_ragged", 2047, 5001, "f16", "e5m2", columns=True, act="gelu", pad=2),
        # one token through a square projection with its residual: latency and 17 MB of weights
        _linear("linear_fp8_one_token", 1, 4096, 4096, "bf16", residual=True),
        # thirteen requests decoding through an expansion: streaming 67 MB of weights
        _linear("linear_fp8_decode_13", 13, 4096, 16384, "bf16", "silu", bias=True),
        # a long prompt or a training batch: a large expansion
        _linear("linear_fp8_large", 8192, 4096, 16384, "bf16", "gelu_tanh"),
        # the weight gradient of a square projection: both operands quantised along the tokens, summed to 32 bits
        _linear("linear_fp8_weight_grad", 4096, 8192, 4096, "f32", x8="e5m2", w_tile=1),
        # thirteen requests decoding: the next product's input comes out in 8 bits
        _norm("block_norm_decode_13", 13, 4096, "bf16", "bf16", 1, out8=True),
        # the pixels of 64 images of 28 x 28 in training, a gate for each image
        _norm("block_norm_pixels", 50176, 512, "bf16", "bf16", 64, stats=True),
        # the same, backward
        _norm_grad("block_norm_grad_pixels", 50176, 512, "bf16", "bf16", 64),
        # odd width and row stride, a residual stream in 32 bits, one gate for all rows
        _norm_grad("block_norm_grad_ragged", 2047, 5001, "f16", "f32", 1, pad=2),
        # the gradients of one narrow block: six small tensors
        _clip("clip_block", "f32", 1, 257, 1028),
        # the gradients of a stack of blocks: 268 million values in 48 tensors of two types
        _clip("clip_stack", "bf16", 8, 2048, 8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, of=8):
    """A size between lo and hi, spread over the logarithm; two in three are multiples of `of`."""
    v = _log(rng, lo, hi)
    if v >= 2 * of and rng.random() < 0.67:
        v = v // of * of
    return v


def _divisor(rng, m):
    """How many gates m rows have: one, one each, or a divisor of them."""
    return rng.choice([1, m] + [d for d in (2, 4, 8, 16, 64) if m % d == 0])


def draw(rng):
    op = rng.choice(("quantize", "linear", "linear", "block_norm", "block_norm_grad", "clip"))
    dt = rng.choice(("bf16", "f16"))
    pad = rng.choice((0, 0, 0, 8, 1))
    if op == "clip":
        while True:
            layers, width = _log(rng, 1, 8), _log(rng, 32, 2048)
            hidden = _log(rng, 2, 4) * width
            if layers * width * hidden <= 8 * 2048 * 8192:
                break
        c = _clip("", rng.choice(("bf16", "f16", "f32")), layers, width, hidden)
    elif op == "linear":
        while True:
            m, k, n = _size(rng, 1, 16384), _size(rng, 64, 8192, 128), _size(rng, 64, 16384, 128)
            if m * k * n <= 8192 * 4096 * 16384 and m * n <= 8192 * 16384:
                break
        if rng.random() < 0.7:
            c = _linear("", m, k, n, rng.choice((dt, dt, "f32")), rng.choice(ACTS), bias=rng.random() < 0.6,
                        residual=rng.random() < 0.4, preact=rng.random() < 0.3)
        else:
            c = _linear("", m, k, n, "f32", x8=rng.choice(("e4m3", "e5m2")), w_tile=1)
    else:
        while True:
            m, k = _size(rng, 1, 131072), _size(rng, 64, 16384)
            if m * k <= 50176 * 512:
                break
        if op == "quantize":
            rows, columns = rng.choice(((True, False), (True, True), (False, True)))
            c = _quantize("", m, k, rng.choice((dt, dt, "f32")), rng.choice(("e4m3", "e4m3", "e5m2")),
                          rng.choice((1, 1, 128)), rows, columns, rng.choice(("none", "none") + ACTS[1:]), pad)
        elif op == "block_norm":
            c = _norm("", m, k, dt, rng.choice((dt, dt, "f32")), _divisor(rng, m), rng.random() < 0.7, rng.random() < 0.5,
                      rng.random() < 0.3, pad)
        else:
            c = _norm_grad("", m, k, dt, rng.choice((dt, dt, "f32")), _divisor(rng, m), rng.random() < 0.7, pad)
    del c["name"]
    return c


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _matrix(values, dtype, pad):
    """`values` rounded to dtype, in rows of `pad` more elements than they use."""
    rows, cols = values.shape
    t = torch.empty(rows, cols + pad, dtype=dtype, device=values.device)[:, :cols]
    return t.copy_(values)


def _eight_bits(v, to, tile):
    """(8-bit values, scales) of a matrix of floats: a scale for each 128
    elements of a row (tile 1) or each square of 128 (tile 128), the block's
    largest magnitude over the type's."""
    m, c = v.shape
    mb, cb = -(-m // tile), _blocks(c)
    full = torch.zeros(mb * tile, cb * BLOCK, device=v.device, dtype=v.dtype)
    full[:m, :c] = v
    full = full.view(mb, tile, cb, BLOCK)
    most = full.abs().amax((1, 3))
    scale = torch.clamp((most.double() / LARGEST[to]).float(), min=LEAST_SCALE)
    # (the quotient in 64 bits: a value that lies halfway between two of the type's has to be seen to)
    step = torch.clamp(most.double(), min=LEAST_SCALE * LARGEST[to])[:, None, :, None]
    q = (full.double() * LARGEST[to] / step).to(DTYPES[to])
    return q.view(mb * tile, cb * BLOCK)[:m, :c], scale


def _in_hand(values, to, tile):
    """An operand as the quantisation leaves it: rows of a multiple of 16
    bytes, the scales of neighbouring rows next to one another."""
    q, scale = _eight_bits(values, to, tile)
    rows, cols = q.shape
    t = torch.empty(rows, (cols + 15) // 16 * 16, dtype=q.dtype, device=q.device)[:, :cols]
    s = torch.empty(scale.shape[1], scale.shape[0], device=q.device).t()
    return t.copy_(q), s.copy_(scale)


def _shapes(case):
    """The gradients of a stack of blocks: two products, their biases, a norm's gain and a gate's."""
    w, h = case["width"], case["hidden"]
    one = [((h, w), case["dt"]), ((w, h), case["dt"]), ((h,), "f32"), ((w,), "f32"), ((w,), "f32"), ((w,), "f32")]
    return one * case["layers"]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case)
    if case["op"] == "clip":
        # a quarter of the tensors have gradients a hundred times smaller
        s["grads"] = [(normal(*shape) * (0.0002 if i % 4 == 3 else 0.02)).to(DTYPES[dt])
                      for i, (shape, dt) in enumerate(_shapes(case))]
        s["clipped"] = [torch.empty_like(t) for t in s["grads"]]
        s["most"] = 1.0
        return s
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        # channels of unlike size, as activations have them
        s["x"], s["xs"] = _in_hand(normal(m, k) * torch.exp(0.5 * normal(k)), case["x8"], 1)
        s["w"], s["ws"] = _in_hand(normal(n, k) / math.sqrt(k), "e4m3", case["w_tile"])
        out = DTYPES[case["out"]]
        s["b"] = 0.2 * normal(n) if case["bias"] else None
        s["r"] = normal(m, n).to(out) if case["residual"] else None
        return s
    m, c, dt, pad = case["m"], case["c"], DTYPES[case["dt"]], case["pad"]
    if case["op"] == "quantize":
        s["x"] = _matrix(normal(m, c) * torch.exp(0.5 * normal(c)), dt, pad)
        s["z"] = None if case["act"] == "none" else _matrix(normal(m, c), dt, pad)
        return s
    stream = DTYPES[case["stream"]]
    s["eps"], s["skip_scale"], s["branch_scale"] = 1e-6, 1.0, 0.5
    s["x"] = _matrix(normal(m, c) * (0.5 + torch.rand(m, 1, generator=g, device="cuda")), dt, pad)
    s["skip"] = _matrix(2 * normal(m, c), stream, pad)
    s["gate"] = (1 + 0.5 * normal(case["groups"], c)).to(dt)
    s["pg"], s["g"] = 1 + 0.2 * normal(c), 1 + 0.2 * normal(c)
    if case["op"] == "block_norm_grad":
        s["dy"] = _matrix(normal(m, c) / 16, dt, pad)
        s["ds"] = _matrix(normal(m, c) / 16, stream, pad)
        # what the forward pass kept: the stream behind the block and the two norms' statistics
        x = s["x"].double()
        s["prstd"] = ((x * x).mean(1) + s["eps"]).rsqrt().float() if case["post"] else None
        branch = x * s["prstd"].double()[:, None] * s["pg"].double() if case["post"] else x
        gate = s["gate"].double().repeat_interleave(m // case["groups"], 0)
        h = s["skip_scale"] * s["skip"].double() + s["branch_scale"] * gate * branch
        s["h"] = _matrix(h, stream, pad)
        h = s["h"].double()
        s["rstd"] = ((h * h).mean(1) + s["eps"]).rsqrt().float()
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


def _whole(q, scale):
    """The 32-bit values of an 8-bit operand."""
    m, k = q.shape
    scale = scale.repeat_interleave(BLOCK, 1)[:, :k]
    if scale.shape[0] != m:
        scale = scale.repeat_interleave(BLOCK, 0)[:m]
    return q.float() * scale


def _plain(s):
    op = s["op"]
    if op == "clip":
        norm = torch.sqrt(sum(t.double().square().sum() for t in s["grads"]))
        factor = torch.clamp(s["most"] / (norm + 1e-6), max=1.0).float()
        return [norm.float()] + [(t.float() * factor).to(t.dtype) for t in s["grads"]]
    if op == "quantize":
        v = s["x"].float()
        if s["z"] is not None:
            v = v * _act_slope(s["z"].float(), s["act"])
        out = list(_eight_bits(v, s["to"], s["tile"])) if s["rows"] else []
        return out + list(_eight_bits(v.t(), s["to"], s["tile"])) if s["columns"] else out
    if op == "linear":
        out = DTYPES[s["out"]]
        z = _whole(s["x"], s["xs"]) @ _whole(s["w"], s["ws"]).t()
        if s["b"] is not None:
            z = z + s["b"]
        y = _act(z, s["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return (y.to(out), z.to(torch.bfloat16)) if s["preact"] else y.to(out)
    x, m = s["x"].float(), s["m"]
    gate = s["gate"].float().repeat_interleave(m // s["groups"], 0)
    if op == "block_norm":
        stats = []
        if s["post"]:
            prstd = 1 / torch.sqrt((x * x).mean(1) + s["eps"])
            x = x * prstd[:, None] * s["pg"]
            stats = [prstd]
        h = s["skip_scale"] * s["skip"].float() + s["branch_scale"] * gate * x
        rstd = 1 / torch.sqrt((h * h).mean(1) + s["eps"])
        y = h * rstd[:, None] * s["g"]
        out = [h.to(DTYPES[s["stream"]])] + (list(_eight_bits(y, "e4m3", 1)) if s["out8"] else [y.to(DTYPES[s["dt"]])])
        return out + stats + [rstd] if s["stats"] else out
    h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    n = h * rstd
    t = dy * s["g"]
    dh = rstd * (t - n * (t * n).mean(1, keepdim=True)) + s["ds"].float()
    dg = (dy * n).sum(0)
    b = x * s["prstd"][:, None] if s["post"] else x
    normed = b * s["pg"] if s["post"] else b
    dgate = s["branch_scale"] * (dh * normed).view(s["groups"], -1, s["c"]).sum(1)
    db = s["branch_scale"] * dh * gate
    dskip = (s["skip_scale"] * dh).to(s["ds"].dtype)
    if not s["post"]:
        return db.to(s["x"].dtype), dskip, dgate, dg
    dpg = (db * b).sum(0)
    t = db * s["pg"]
    dx = s["prstd"][:, None] * (t - b * (t * b).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), dskip, dgate, dg, dpg


def _own(s):
    import int8_conv2d_fprop_gb300 as ic
    op = s["op"]
    if op == "clip":
        return [ic.conv_clip_grads(s["grads"], s["most"], out=s["clipped"])] + s["clipped"]
    x = s["x"]
    if op == "quantize":
        return ic.conv_quantize(x, dtype=DTYPES[s["to"]], tile=s["tile"], rows=s["rows"], columns=s["columns"],
                                preact=s["z"], activation=s["act"])
    if op == "linear":
        z = torch.empty(s["m"], s["n"], dtype=torch.bfloat16, device=x.device) if s["preact"] else None
        y = ic.conv_linear_fp8(x, s["xs"], s["w"], s["ws"], s["b"], activation=s["act"], residual=s["r"], preact=z,
                               dtype=DTYPES[s["out"]])
        return (y, z) if s["preact"] else y
    m, f32 = s["m"], torch.float32
    scales = {"skip_scale": s["skip_scale"], "branch_scale": s["branch_scale"]}
    if op == "block_norm":
        prstd = torch.empty(m, dtype=f32, device=x.device) if s["stats"] and s["post"] else None
        rstd = torch.empty(m, dtype=f32, device=x.device) if s["stats"] else None
        out = ic.conv_block_norm(x, s["skip"], post_norm=s["post"], post_gain=s["pg"] if s["post"] else None,
                                 gate=s["gate"], gain=s["g"], eps=s["eps"], post_rstd=prstd, rstd=rstd,
                                 dtype=torch.float8_e4m3fn if s["out8"] else None, **scales)
        return list(out) + ([prstd] if prstd is not None else []) + ([rstd] if rstd is not None else [])
    dx, dskip = torch.empty(x.shape, dtype=x.dtype, device=x.device), torch.empty(x.shape, dtype=s["ds"].dtype, device=x.device)
    dgate = torch.empty(s["gate"].shape, dtype=f32, device=x.device)
    dg = torch.empty_like(s["g"])
    dpg = torch.empty_like(s["pg"]) if s["post"] else None
    ic.conv_block_norm_grad(s["dy"], s["ds"], x, s["h"], post_norm=s["post"], post_gain=s["pg"] if s["post"] else None,
                            gate=s["gate"], gain=s["g"], post_rstd=s["prstd"], rstd=s["rstd"], dx=dx, dskip=dskip,
                            dgate=dgate, dgain=dg, dpost_gain=dpg, **scales)
    return (dx, dskip, dgate, dg, dpg) if s["post"] else (dx, dskip, dgate, dg)


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op = case["op"]
    if op == "clip":
        values = [(math.prod(shape), SIZE[dt]) for shape, dt in _shapes(case)]
        return {"bytes": 2 * sum(n * size for n, size in values), "flops": 3 * sum(n for n, size in values)}
    if op == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        scales = m * _blocks(k) + -(-n // case["w_tile"]) * _blocks(k)
        out = m * n * (SIZE[case["out"]] * (1 + case["residual"]) + 2 * case["preact"])
        return {"bytes": m * k + n * k + 4 * scales + out + 4 * n * case["bias"], "flops": 2 * m * n * k}
    m, c = case["m"], case["c"]
    if op == "quantize":
        scales = case["rows"] * -(-m // case["tile"]) * _blocks(c) + case["columns"] * -(-c // case["tile"]) * _blocks(m)
        return {"bytes": m * c * (SIZE[case["dt"]] * (1 + (case["act"] != "none")) + case["rows"] + case["columns"]) + 4 * scales,
                "flops": 4 * m * c}
    size, stream, gates = SIZE[case["dt"]], SIZE[case["stream"]], case["groups"] * c
    if op == "block_norm":
        out = m * c + 4 * m * _blocks(c) if case["out8"] else m * c * size
        return {"bytes": m * c * (size + 2 * stream) + out + gates * size + 8 * c + 4 * m * case["stats"] * (1 + case["post"]),
                "flops": 10 * m * c}
    return {"bytes": m * c * (3 * size + 3 * stream) + gates * (size + 4) + 4 * m * (1 + case["post"]) + 8 * c * (1 + case["post"]),
            "flops": 20 * m * c}


def exact(case, seed):
    """The operators' definitions in 64 bits: 8-bit values as the quotients
    before they are rounded, products by blocks of 128, the norms through
    the rows' lengths, and their gradients through projections."""
    s = prepare(case, seed)
    op = case["op"]

    def phi(v):
        return 0.5 * torch.special.erfc(-v / math.sqrt(2.0))

    def tanh_arg(v):
        return 2 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)

    def quotients(v, tile):
        """Of every element by its block's scale, and the scales: block after block of columns."""
        values, scales = [], []
        for part in v.split(BLOCK, 1):
            most = part.abs().amax(1)
            if tile == BLOCK:
                most = torch.stack([p.amax() for p in most.split(BLOCK)])
            step = (most / LARGEST[case.get("to", "e4m3")]).clamp(min=LEAST_SCALE)
            scales.append(step)
            values.append(part / (step if tile == 1 else step.repeat_interleave(BLOCK)[:len(part)])[:, None])
        return [torch.cat(values, 1), torch.stack(scales, 1)]

    if op == "clip":
        norm = math.sqrt(sum(float(torch.linalg.vector_norm(t.double())) ** 2 for t in s["grads"]))
        factor = min(1.0, s["most"] / (norm + 1e-6))
        return [torch.tensor(norm, dtype=torch.float64)] + [t.double() * factor for t in s["grads"]]
    x = s["x"].double()
    if op == "quantize":
        if s["z"] is not None:
            z, act = s["z"].double(), case["act"]
            if act == "relu":
                x = x.masked_fill(z <= 0, 0)
            elif act == "gelu":
                x = x * (phi(z) + z * torch.exp(-z * z / 2) * (2 * math.pi) ** -0.5)
            elif act == "gelu_tanh":
                p = torch.sigmoid(tanh_arg(z))
                x = x * (p + z * p * (1 - p) * 2 * math.sqrt(2.0 / math.pi) * (1 + 0.134145 * z * z))
            else:
                p = torch.sigmoid(z)
                x = x * (p + z * p * (1 - p))
        out = quotients(x, case["tile"]) if case["rows"] else []
        return out + quotients(x.t(), case["tile"]) if case["columns"] else out
    if op == "linear":
        w, z = s["w"].double(), 0
        xs, ws = s["xs"].double(), s["ws"].double()
        if case["w_tile"] == BLOCK:
            ws = ws.repeat_interleave(BLOCK, 0)[:case["n"]]
        for b in range(_blocks(case["k"])):
            k = slice(b * BLOCK, (b + 1) * BLOCK)
            z = torch.addmm(z, x[:, k] * xs[:, b:b + 1], (w[:, k] * ws[:, b:b + 1]).t()) if b else \
                (x[:, k] * xs[:, b:b + 1]) @ (w[:, k] * ws[:, b:b + 1]).t()
        if s["b"] is not None:
            z = z + s["b"].double()
        act = case["act"]
        y = (z.clamp(min=0) if act == "relu" else z * phi(z) if act == "gelu" else
             z * torch.sigmoid(tanh_arg(z)) if act == "gelu_tanh" else z * torch.sigmoid(z) if act == "silu" else z)
        if s["r"] is not None:
            y = y + s["r"].double()
        return (y, z) if case["preact"] else y
    m, c, groups = case["m"], case["c"], case["groups"]
    gate = s["gate"].double()[:, None, :].expand(groups, m // groups, c).reshape(m, c) * s["branch_scale"]
    if op == "block_norm":
        stats = []
        if case["post"]:
            stats = [(torch.linalg.vector_norm(x, dim=1).square() / c + s["eps"]).pow(-0.5)]
            x = x * (stats[0][:, None] * s["pg"].double())
        h = torch.addcmul(s["skip"].double() * s["skip_scale"], gate, x)
        stats.append((torch.linalg.vector_norm(h, dim=1).square() / c + s["eps"]).pow(-0.5))
        y = h * (stats[-1][:, None] * s["g"].double())
        return [h] + (quotients(y, 1) if case["out8"] else [y]) + (stats if case["stats"] else [])
    h, dy, r = s["h"].double(), s["dy"].double(), s["rstd"].double()[:, None]
    t = dy * s["g"].double()
    dh = s["ds"].double() + r * t - h * (r ** 3 * torch.einsum("mc,mc->m", t, h)[:, None] / c)
    dg = torch.einsum("mc,mc->c", dy, h * r)
    grown = dh * gate
    if not case["post"]:
        dgate = torch.einsum("grc,grc->gc", dh.view(groups, -1, c), x.view(groups, -1, c)) * s["branch_scale"]
        return grown, dh * s["skip_scale"], dgate, dg
    p, pg = s["prstd"].double()[:, None], s["pg"].double()
    dgate = torch.einsum("grc,grc->gc", dh.view(groups, -1, c), (x * p).view(groups, -1, c)) * pg * s["branch_scale"]
    dpg = torch.einsum("mc,mc->c", grown, x * p)
    t = grown * pg
    dx = p * t - x * (p ** 3 * torch.einsum("mc,mc->m", t, x)[:, None] / c)
    return dx, dh * s["skip_scale"], dgate, dg, dpg

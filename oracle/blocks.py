"""Plain 64-bit definitions (torch, any device) of the 8-bit product with block
scales and its quantisation, the block norm and its gradients, and the clipping
of gradients, each with the bound on a 32-bit computation's distance from it
that the tests use."""
from __future__ import annotations

import math

import torch

from .channel import TINY, UNIT

BLOCK = 128
LARGEST = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
# mantissa bits and least normal exponent
BITS = {torch.float8_e4m3fn: (3, -6), torch.float8_e5m2: (2, -14)}
LEAST_SCALE = 2.0 ** -126


def unit(dtype):
    return UNIT[str(dtype).replace("torch.", "")]


def tiny(dtype):
    return TINY[str(dtype).replace("torch.", "")]


def blocks(n):
    return -(-n // BLOCK)


def per_element(scale, rows, cols):
    """Block scales [rows or ceil(rows / 128), ceil(cols / 128)] as a matrix of elements."""
    s = scale.double().repeat_interleave(BLOCK, 1)[:, :cols]
    return s if s.shape[0] == rows else s.repeat_interleave(BLOCK, 0)[:rows]


def block_largest(v, tile):
    """Largest magnitude of each block of [M, C]."""
    m, c = v.shape
    full = torch.zeros(-(-m // tile) * tile, blocks(c) * BLOCK, dtype=v.dtype, device=v.device)
    full[:m, :c] = v.abs()
    return full.view(-1, tile, blocks(c), BLOCK).amax((1, 3))


def half_step(u, dtype):
    """Half the distance between neighbouring 8-bit values at magnitude u."""
    bits, least = BITS[dtype]
    e = torch.floor(torch.log2(u.clamp(min=2.0 ** least)))
    return 2.0 ** (e - bits - 1)


def check_quantized(q, scale, v, tile, ev=None):
    """None, or what is wrong with q and scale as the 8-bit form of v (float64,
    known to ev).  The scale is one rounding away from largest / L; a value is
    rounded by half a step at most, after a factor that is off by 2^-22."""
    dtype, (m, c) = q.dtype, v.shape
    ev = torch.zeros_like(v) if ev is None else ev
    most = block_largest(v, tile)
    want = (most / LARGEST[dtype]).clamp(min=LEAST_SCALE)
    far = (scale.double() - want).abs() > 2.0 ** -23 * want + block_largest(ev, tile) / LARGEST[dtype]
    if bool(far.any()):
        return f"{int(far.sum())} of {far.numel()} scales"
    s = per_element(scale, m, c)
    u = v.abs() / s
    bound = s * half_step(u * (1 + 2.0 ** -21) + ev / s, dtype) + 2.0 ** -22 * v.abs() + ev
    bad = ~((q.double() * s - v).abs() <= bound)
    if bool(bad.any()):
        return f"{int(bad.sum())} of {bad.numel()} values, first at {bad.nonzero()[0].tolist()}"
    return None


def phi(v):
    return 0.5 * torch.special.erfc(-v / math.sqrt(2.0))


def activate(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * phi(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        p = torch.sigmoid(2 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
        return p + z * p * (1 - p) * 2 * math.sqrt(2.0 / math.pi) * (1 + 0.134145 * z * z)
    if act == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    return torch.ones_like(z)


def linear_fp8(x, xs, w, ws, bias=None, act="none", residual=None):
    """(y, z, size): size is the sum of absolute values behind z."""
    x = x.double() * per_element(xs, *x.shape)
    w = w.double() * per_element(ws, *w.shape)
    z, size = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, size = z + bias.double(), size + bias.double().abs()
    y = activate(z, act)
    return (y if residual is None else y + residual.double()), z, size


def linear_fp8_bounds(k, y, z, size, act, residual, y_type, z_type=torch.bfloat16):
    """Every 32-bit addition of the K products and the blocks' sums, and every
    product of scales, is off by 2^-23 of the sum of absolute values at most;
    the activations as in the 16-bit product."""
    ez = (k + 4 * blocks(k) + 4) * 2.0 ** -23 * size
    ey = ez if act == "none" else 1.2 * ez + 2.0 ** -20 * z.abs()
    if residual is not None:
        ey = ey + 2.0 ** -23 * residual.double().abs()
    return (ey + unit(y_type) * (y.abs() + ey) + tiny(y_type), ez + unit(z_type) * (z.abs() + ez) + tiny(z_type))


def rounded(e, v, dtype):
    """Bound e of an unrounded value with one rounding to dtype behind it."""
    return e + unit(dtype) * (v.abs() + e) + tiny(dtype)


def sum_error(c):
    """Relative error of a 32-bit sum of c positive values by lanes and tree."""
    return (c / 32 + 16) * 2.0 ** -23


def gate_rows(gate, rows):
    return None if gate is None else gate.double().reshape(-1, gate.shape[-1]).repeat_interleave(
        rows // max(1, gate.numel() // gate.shape[-1]), 0)


def block_norm(x, skip, post, post_gain, gate, skip_scale, branch_scale, gain, eps):
    """{name: (value, bound before rounding)} of sum, y, post_rstd and rstd."""
    x = x.double()
    rows, c = x.shape
    n, en, out = x, torch.zeros_like(x), {}
    if post:
        rx = ((x * x).mean(1) + eps) ** -0.5
        er = (0.5 * sum_error(c) + 2.0 ** -21) * rx
        out["post_rstd"] = (rx, er)
        n = x * rx[:, None] * (1 if post_gain is None else post_gain.double())
        en = n.abs() * (er / rx)[:, None] + 2.0 ** -22 * n.abs()
    g = gate_rows(gate, rows)
    g = branch_scale * (1 if g is None else g)
    h = g * n
    eh = (g.abs() if torch.is_tensor(g) else abs(g)) * en + 2.0 ** -22 * h.abs()
    if skip is not None:
        eh = eh + 2.0 ** -23 * (skip_scale * skip.double()).abs()
        h = h + skip_scale * skip.double()
        eh = eh + 2.0 ** -23 * h.abs()
    out["sum"] = (h, eh)
    var = (h * h).mean(1) + eps
    rs = var ** -0.5
    ev = sum_error(c) + ((2 * h.abs() * eh + eh * eh).mean(1)) / var
    er = rs * (0.5 * ev + ev * ev + 2.0 ** -21)
    out["rstd"] = (rs, er)
    a = 1 if gain is None else gain.double()
    y = h * rs[:, None] * a
    ey = (eh * (rs + er)[:, None] + h.abs() * er[:, None]) * (1 if gain is None else a.abs()) + 2.0 ** -22 * y.abs()
    out["y"] = (y, ey)
    return out


def block_norm_grad(dy, dsum, x, h, post, post_gain, gate, groups, skip_scale, branch_scale, gain, rx, rs):
    """{name: (value, bound before rounding)} of dx, dskip, dgate, dgain and
    dpost_gain, with the statistics rx and rs as given."""
    like = dy if dy is not None else dsum
    rows, c = like.shape
    t_err, s_err, out = 2.0 ** -21, sum_error(c), {}
    dh = torch.zeros(rows, c, dtype=torch.float64, device=like.device)
    edh = torch.zeros_like(dh)
    if dy is not None:
        dy, r = dy.double(), rs.double()[:, None]
        t, u = dy * (1 if gain is None else gain.double()), h.double() * r
        s, size = (t * u).mean(1, keepdim=True), (t * u).abs().mean(1, keepdim=True)
        dh = r * (t - u * s)
        edh = r * (t_err * t.abs() + u.abs() * (s_err + 2 * t_err) * size) + t_err * dh.abs()
        out["dgain"] = ((dy * u).sum(0), ((rows + 8) * 2.0 ** -23 + t_err) * (dy * u).abs().sum(0))
    if dsum is not None:
        dh = dh + dsum.double()
        edh = edh + 2.0 ** -23 * (dsum.double().abs() + dh.abs())
    out["dskip"] = (skip_scale * dh, abs(skip_scale) * edh + 2.0 ** -23 * (skip_scale * dh).abs())
    g = gate_rows(gate, rows)
    g = branch_scale * (torch.ones(rows, c, dtype=torch.float64, device=like.device) if g is None else g)
    db, edb = g * dh, g.abs() * edh + t_err * (g * dh).abs()
    p = 1 if post_gain is None else post_gain.double()
    if x is not None:
        r = rx.double()[:, None] if post else 1
        v = x.double() * r
        gs, es = dh * v, edh * v.abs() + t_err * (dh * v).abs()
        k = branch_scale * (p if post else 1)
        sums = lambda m: m.view(groups, -1, c).sum(1)  # noqa: E731
        out["dgate"] = (k * sums(gs), (abs(k) if not torch.is_tensor(k) else k.abs()) * (
            sums(es) + ((rows // groups + 8) * 2.0 ** -23 + t_err) * sums(gs.abs())))
        if post:
            # (through the gates' sums: each of them, times its gate, then their sum)
            out["dpost_gain"] = ((db * v).sum(0), (edb * v.abs()).sum(0) + ((rows + 8) * 2.0 ** -23 + 2 * t_err) * (db * v).abs().sum(0))
            dn, edn = db * p, edb * (p.abs() if torch.is_tensor(p) else p) + t_err * (db * p).abs()
            s, size = (dn * v).mean(1, keepdim=True), (dn * v).abs().mean(1, keepdim=True)
            out["dx"] = (r * (dn - v * s), r * (edn + v.abs() * ((edn * v.abs()).mean(1, keepdim=True) + (s_err + 2 * t_err) * size)
                                                + t_err * dn.abs()))
    if not post:
        out["dx"] = (db, edb)
    return out


def clip(grads, max_norm, eps):
    """(norm, tensors) in 64 bits."""
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    f = 1.0 if math.isinf(max_norm) else min(1.0, max_norm / (norm + eps))
    return norm, [g.double() * f for g in grads]

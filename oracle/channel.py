"""Plain 64-bit definitions of the channel operators (numpy): the matrix
product with bias, activation and residual, the layer norm, and their
gradients, each with the bound on a 32-bit computation's distance from it
that the tests use."""
from __future__ import annotations

import math

import numpy as np

# unit roundoffs of the stored types
UNIT = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11, "float32": 2.0 ** -24}
TINY = {"bfloat16": 2.0 ** -133, "float16": 2.0 ** -24, "float32": 2.0 ** -149}  # least positive value

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def normal_cdf(z):
    return 0.5 * _erfc(-np.asarray(z, np.float64) / math.sqrt(2))


def logistic(z):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-z))


def activate(z, act):
    if act == "relu":
        return np.where(z < 0, 0.0, z)
    if act == "gelu":
        return z * normal_cdf(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * logistic(z)
    return z


def activation_slope(z, act):
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "gelu":
        return normal_cdf(z) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        u = math.sqrt(2 / math.pi)
        t = np.tanh(u * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * u * (1 + 0.134145 * z * z)
    if act == "silu":
        s = logistic(z)
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def linear(x, w, bias=None, act="none", residual=None):
    """(y, z) of float64 arrays."""
    z = x @ w.T
    if bias is not None:
        z = z + bias
    y = activate(z, act)
    return (y if residual is None else y + residual), z


def linear_bounds(x, w, bias, act, residual, y, z, y_type, z_type):
    """How far stored y and z may be from linear()'s: every 32-bit addition of
    the K products (and the bias) is off by at most 2^-23 of the sum of
    absolute values; the activations' slopes are at most 1.2, and their own
    32-bit evaluation is off by at most 2^-20 of |z|; one more rounding to the
    stored type."""
    size = np.abs(x) @ np.abs(w).T + (0 if bias is None else np.abs(bias))
    ez = (x.shape[1] + 2) * 2.0 ** -23 * size
    ey = ez if act == "none" else 1.2 * ez + 2.0 ** -20 * np.abs(z)
    if residual is not None:
        ey = ey + 2.0 ** -23 * np.abs(residual)
    return (ey + UNIT[y_type] * (np.abs(y) + ey) + TINY[y_type],
            ez + UNIT[z_type] * (np.abs(z) + ez) + TINY[z_type])


def linear_grad(dy, x, w, z=None, act="none"):
    """(dx, dw, dbias, dz) of float64 arrays."""
    dz = dy if act == "none" else dy * activation_slope(z, act)
    return dz @ w, dz.T @ x, dz.sum(0), dz


def linear_grad_bounds(dz, x, w, dy, act, outs, types, in_type):
    """dz is off by 2^-19 of |dy| (the slope's evaluation) and, with an
    activation, by one rounding to the stored type; the sums as in
    linear_bounds."""
    dx, dw, db = outs
    edz = 0 if act == "none" else 2.0 ** -19 * np.abs(dy)
    rdz = edz if act == "none" else edz + UNIT[in_type] * np.abs(dz) + TINY[in_type]
    a, m, n = np.abs(dz) + rdz, dz.shape[0], dz.shape[1]
    ex = (n + 2) * 2.0 ** -23 * (a @ np.abs(w)) + (rdz @ np.abs(w) if act != "none" else 0)
    ew = (m + 2) * 2.0 ** -23 * (a.T @ np.abs(x)) + (rdz.T @ np.abs(x) if act != "none" else 0)
    eb = (m + 2) * 2.0 ** -23 * a.sum(0) + (edz.sum(0) if act != "none" else 0)
    return [e + UNIT[t] * (np.abs(v) + e) + TINY[t] for e, v, t in ((ex, dx, types[0]), (ew, dw, types[1]),
                                                                   (eb, db, types[2]))]


def layer_norm(x, gain=None, shift=None, eps=1e-5, scale=1.0):
    """(y, mean, rstd) of float64 arrays."""
    v = scale * x
    mean = v.mean(1)
    d = v - mean[:, None]
    rstd = 1 / np.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    if gain is not None:
        y = y * gain
    return (y if shift is None else y + shift), mean, rstd


def layer_norm_bounds(x, gain, shift, eps, scale, y, mean, rstd, y_type):
    """A 32-bit sum of C values by lanes and tree is off by at most
    (C/32 + 16) 2^-23 of the sum of absolute values; that moves the mean, the
    differences to it and (by half its relative error) rstd."""
    c = x.shape[1]
    v = scale * x
    terms = (c / 32 + 16) * 2.0 ** -23
    em = (terms + 2.0 ** -22) * np.abs(v).mean(1)
    d = np.abs(v - mean[:, None])
    ed = em[:, None] + 2.0 ** -22 * (np.abs(v) + np.abs(mean)[:, None])
    var = (d * d).mean(1) + eps
    ev = terms * var + (2 * d * ed + ed * ed).mean(1)
    er = rstd * (0.5 * ev / var + (ev / var) ** 2 + 2.0 ** -21)
    g = np.ones(c) if gain is None else np.abs(gain)
    ey = (ed * (rstd + er)[:, None] + d * er[:, None]) * g + 2.0 ** -21 * (np.abs(y) + (0 if shift is None else np.abs(shift)))
    return ey + UNIT[y_type] * (np.abs(y) + ey) + TINY[y_type], em + 2.0 ** -24 * np.abs(mean), er


def layer_norm_grad(dy, x, gain, mean, rstd, residual=None):
    """(dx, dgain, dshift) of float64 arrays."""
    n = (x - mean[:, None]) * rstd[:, None]
    t = dy if gain is None else dy * gain
    dx = rstd[:, None] * (t - t.mean(1, keepdims=True) - n * (t * n).mean(1, keepdims=True))
    return (dx if residual is None else dx + residual), (dy * n).sum(0), dy.sum(0)


def layer_norm_grad_bounds(dy, x, gain, mean, rstd, residual, outs, x_type, p_type, centred=False):
    """Sums as in layer_norm_bounds; the normalised value n is off by 2^-22 of
    (|x| + |mean|) rstd + |n|, or with `centred` of |n| alone, as the product of
    a rounded difference x - mean is."""
    dx, dg, db = outs
    m, c = x.shape
    terms = (c / 32 + 16) * 2.0 ** -23
    r = rstd[:, None]
    n = (x - mean[:, None]) * r
    en = 2.0 ** -22 * ((0 if centred else (np.abs(x) + np.abs(mean)[:, None]) * r) + np.abs(n))
    t = np.abs(dy if gain is None else dy * gain)
    s1, s2 = t.mean(1, keepdims=True), (t * np.abs(n)).mean(1, keepdims=True)
    e2 = (terms + 2.0 ** -21) * s2 + (t * en).mean(1, keepdims=True)
    ex = r * (terms * s1 + np.abs(n) * e2 + en * (s2 + e2) + 2.0 ** -21 * (t + s1 + np.abs(n) * s2))
    if residual is not None:
        ex = ex + 2.0 ** -23 * (np.abs(residual) + np.abs(dx))
    ex = ex + UNIT[x_type] * (np.abs(dx) + ex) + TINY[x_type]
    eg = (m + 4) * 2.0 ** -23 * (np.abs(dy * n)).sum(0) + (np.abs(dy) * en).sum(0)
    eb = (m + 4) * 2.0 ** -23 * np.abs(dy).sum(0)
    return ex, eg + UNIT[p_type] * (np.abs(dg) + eg) + TINY[p_type], eb + UNIT[p_type] * (np.abs(db) + eb) + TINY[p_type]

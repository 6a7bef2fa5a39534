"""Orthogonalization by Newton-Schulz steps and the Muon step in fp64 (test infrastructure only).

    X_0 = U / max(|U|, eps),  A = X X^T,  X <- a X + (b A + c A^2) X   (U's shorter side as rows)

``rounded_newton_schulz`` is the same with the roundings that the library's products make, in
fp64 otherwise: what its results may be off by is judged against that. ``single_newton_schulz`` is
the same in fp32 throughout.
"""
from __future__ import annotations

import math

import numpy as np

from .optimizers import round_bf16

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
LIFT = 2.0 ** 12  # the library holds the iterate times this in fp16


def per_step(coefficients, steps):
    c = np.asarray(coefficients, np.float64)
    return [tuple(c)] * steps if c.ndim == 1 else [tuple(r) for r in c]


def start(u, eps):
    """X_0, and whether it is transposed."""
    u = np.asarray(u, np.float64)
    norm = math.sqrt(float(np.sum(u * u)))
    top = max(norm, eps)
    x = u / top if top > 0 else u * 0.0
    tall = u.shape[0] > u.shape[1]
    return (x.T if tall else x), tall


def newton_schulz(u, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    """One matrix."""
    if not np.all(np.isfinite(u)):
        return np.full(np.shape(u), np.nan)
    x, tall = start(u, eps)
    for a, b, c in per_step(coefficients, steps):
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if tall else x


def _half(v, scale):
    return np.asarray(v * scale, np.float32).astype(np.float16).astype(np.float64) / scale


def rounded_newton_schulz(u, steps=5, coefficients=COEFFICIENTS, eps=1e-7, parts=1):
    """``parts``: of fp16 that the products' operands have (2: matrices with few rows)."""
    x, tall = start(u, eps)
    if parts == 2:
        x = _rounded_in_two_parts(x, per_step(coefficients, steps))
        return x.T if tall else x

    def parts(v):
        hi = _half(v, LIFT)
        return hi, _half(v - hi, LIFT)

    hi, lo = parts(x)
    for a, b, c in per_step(coefficients, steps):
        g = hi @ hi.T
        d = (np.diag(g) + np.sum(lo * (2 * hi + lo), axis=1)).astype(np.float32).astype(np.float64)
        o = _half(g - np.diag(np.diag(g)), 256.0)
        sq = o @ o
        p = o * (b + c * (d[:, None] + d[None, :])) + c * sq
        q = (a + b * d + c * (d * d + np.diag(sq))).astype(np.float32).astype(np.float64)
        p = _half(p - np.diag(np.diag(p)), 256.0)
        t = a + (q - a) * np.minimum(1.0, d * d)
        x = q[:, None] * hi + t[:, None] * lo + p @ hi
        hi, lo = parts(x)
    return x.T if tall else x


def _rounded_in_two_parts(x, coefficients):
    """Every operand as hi + lo, products without lo lo."""
    def parts(v, lift):
        hi = _half(v, lift)
        return hi, _half(v - hi, lift)

    def mul(p, q):
        return p[0] @ q[0] + p[0] @ q[1] + p[1] @ q[0]

    for a, b, c in coefficients:
        x = parts(x, LIFT)
        g = mul(x, (x[0].T, x[1].T))
        d = np.diag(g).astype(np.float32).astype(np.float64)
        o = parts(g - np.diag(np.diag(g)), 256.0)
        sq = mul(o, o)
        p = (o[0] + o[1]) * (b + c * (d[:, None] + d[None, :])) + c * sq
        q = (a + b * d + c * (d * d + np.diag(sq))).astype(np.float32).astype(np.float64)
        p = parts(p - np.diag(np.diag(p)), 256.0)
        x = q[:, None] * (x[0] + x[1]) + mul(p, x)
    return x


def single_newton_schulz(u, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    x, tall = start(u, eps)
    x = x.astype(np.float32)
    for a, b, c in np.asarray(per_step(coefficients, steps), np.float32):
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return (x.T if tall else x).astype(np.float64)


def bound_of_one_step(u, coefficients=COEFFICIENTS, eps=1e-7):
    """How far one step's result may be off, element by element: every rounding counted at its
    most (fp16 2^-11 of the value, sums in fp32 2^-23 of the terms' magnitudes per term)."""
    a, b, c = per_step(coefficients, 1)[0]
    x, tall = start(u, eps)
    m, n = x.shape
    h, s, tiny = 2.0 ** -11, (n + m + 8) * 2.0 ** -23, 2.0 ** -24 / 256  # (smallest fp16 step of O and B)
    ax = np.abs(x)
    ex = h * ax + 2.0 ** -24 / LIFT  # of an operand
    ag = ax @ ax.T
    eg = ex @ ax.T + ax @ ex.T + ex @ ex.T + s * ag
    eo = eg + h * (ag + eg) + tiny  # (the diagonal is not rounded: more than it needs)
    ag2 = ag + eo
    ep = abs(b) * eo + abs(c) * (ag2 @ eo + eo @ ag2) + s * (abs(b) * ag2 + abs(c) * (ag2 @ ag2))
    ap = abs(b) * ag2 + abs(c) * (ag2 @ ag2)
    ep = ep + h * (ap + ep) + tiny
    ey = ep @ ax + ap @ ex + ep @ ex + (s + 2.0 ** -21) * (abs(a) * ax + ap @ ax) + abs(a) * 2.0 ** -25 / LIFT
    return ey.T if tall else ey


def shape_scale(adjust_lr, rows, cols):
    return math.sqrt(max(1.0, rows / cols)) if adjust_lr == "original" else 0.2 * math.sqrt(max(rows, cols))


def quantize(m):
    """The momentum's 8-bit form: scale max|m| times fp32 1/127 per 128 values, codes to nearest even."""
    v = np.asarray(m, np.float32).reshape(-1)
    n = v.size
    v = np.concatenate([v, np.zeros(-n % 128, np.float32)]).reshape(-1, 128)
    with np.errstate(all="ignore"):
        scale = np.max(np.abs(v), axis=1) * (np.float32(1.0) / np.float32(127.0))
        ok = np.isfinite(scale) & (scale > 0)
        codes = np.where(ok[:, None], np.rint(v / np.where(ok, scale, np.float32(1.0))[:, None]), np.float32(0.0))
    scale = np.where(np.isfinite(scale), scale, np.float32(np.nan)).astype(np.float32)
    return np.clip(codes, -128, 127).astype(np.int8).reshape(-1)[:n].reshape(np.shape(m)), scale


def dequantize(codes, scale):
    c = np.asarray(codes, np.float32).reshape(-1)
    return (c * np.repeat(scale, 128)[:c.size]).reshape(np.shape(codes))


def momentum(m, g, beta, kind):
    """The stored momentum, bit for bit (float32 arithmetic): float32 values, and (8-bit) codes and scales."""
    b, omb = np.float32(beta), np.float32(1.0 - beta)
    new = np.asarray(m, np.float32) * b + np.asarray(g, np.float32) * omb
    if kind == "bfloat16":
        return np.float32(round_bf16(new)), None
    if kind == "int8":
        q = quantize(new)
        return dequantize(*q), q
    return new, None


def direction(m, g, beta, nesterov):
    b, omb = np.float32(beta), np.float32(1.0 - beta)
    return np.asarray(g, np.float32) * omb + m * b if nesterov else m


def muon_step_tensor(x, g, m, *, kind="float32", lr=1e-3, momentum_=0.95, weight_decay=0.1, nesterov=True,
                     adjust_lr="original", steps=5, coefficients=COEFFICIENTS, eps=1e-7, ns=newton_schulz):
    """(param, stored momentum as float32, its 8-bit form or None); x [..., rows, cols] in fp64."""
    new, q = momentum(m, g, momentum_, kind)
    u = direction(new, g, momentum_, nesterov)
    rows, cols = x.shape[-2:]
    o = np.stack([ns(v, steps, coefficients, eps) for v in u.reshape(-1, rows, cols)]).reshape(x.shape)
    return x * (1.0 - lr * weight_decay) - lr * shape_scale(adjust_lr, rows, cols) * o, new, q

"""Float64 reference of the norms with gate and residual between retention
cores, their gradients, and the 8-bit form of kept activations.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Plain numpy; each
function states its definition.  Pages: [RN-zh] sections "門控多尺度
Retention" (per-head GroupNorm, swish gate) and "Retention 網路總體結構"
(LayerNorm, residual connections), titles in ``oracle.retention``.

Beside each value the functions give its *size*: the same expression with
every term replaced by a bound on its magnitude ((|h| + mean|h|) r for the
normalised (h - mu) r; (|h| + |mu|) r where mu is given).  A float32 evaluation is off by at most a small
multiple of 2^-24 times that size, however much the terms cancel.
"""
from __future__ import annotations

import numpy as np

F64 = np.float64
GROUP = 32
Q_TOP = {"e4m3": 448.0, "i8": 127.0}


def _f64(x):
    return np.asarray(x, dtype=F64)


# ------------------------------------------------------------- 8-bit form --
def e4m3_values():
    """The 256 e4m3 codes' values (sign, 4 exponent bits of bias 7, 3 of the
    significand; no infinities, S.1111.111 is NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where(c & 128, -v, v)
    return np.where((c & 127) == 127, np.nan, v)


def q_exponent(amax, fmt):
    """The smallest e >= -127 with amax <= top 2^e (0 for amax = 0: -127)."""
    amax = _f64(amax)
    e = np.full(amax.shape, -127)
    for k in range(-127, 129):
        e = np.where(amax > Q_TOP[fmt] * 2.0 ** k, k + 1, e)
    return e


def q_pack(x, fmt):
    """x [..., cols] to (codes as values q, scale bytes e + 127): q is x 2^-e
    rounded to the nearest code, ties to the even one; a group with an
    infinity or a NaN gets q = 0 and the byte 255."""
    x = _f64(x)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    bad = ~np.all(np.isfinite(g), axis=-1)
    g = np.where(bad[..., None], 0.0, g)
    e = q_exponent(np.max(np.abs(g), axis=-1), fmt)
    v = np.ldexp(g, -e[..., None])
    if fmt == "i8":
        q = np.rint(v)
    else:
        _, ex = np.frexp(np.maximum(np.abs(v), 2.0 ** -6))
        step = np.ldexp(1.0, ex - 4)                  # 3 bits behind the leading one
        q = np.rint(v / step) * step
    return q.reshape(x.shape), np.where(bad, 255, e + 127).astype(np.uint8)


def q_unpack(q, qs):
    """q 2^e; NaN where the byte is 255."""
    q, e = _f64(q), np.asarray(qs).astype(int) - 127
    g = q.reshape(*q.shape[:-1], -1, GROUP)
    v = np.where((e == 128)[..., None], np.nan, np.ldexp(g, np.where(e == 128, 0, e)[..., None]))
    return v.reshape(q.shape)


# ------------------------------------------------------------------ norms --
def norm_stats(h, layer, eps):
    """mu (0 unless layer) and r = 1 / sqrt(mean((h - mu)^2) + eps) over the last dimension."""
    h = _f64(h)
    mu = h.mean(-1) if layer else np.zeros(h.shape[:-1])
    return mu, 1.0 / np.sqrt(((h - mu[..., None]) ** 2).mean(-1) + eps)


def normalised(h, mu, r, mu_size=None):
    """((h - mu) r, its size).  mu_size: the size of mu where it is formed from h -- the mean of d values is off by
    roundings of its partial sums, up to mean|h| each, however small mu itself is (given: |mu|)."""
    h, mu, r = _f64(h), _f64(mu)[..., None], _f64(r)[..., None]
    ms = np.abs(mu) if mu_size is None else _f64(mu_size)[..., None]
    return (h - mu) * r, (np.abs(h) + ms) * r


def resid_norm(h, layer, eps, weight=1.0, bias=0.0):
    """(y, size of y, mu, r) of y = (h - mu) r weight + bias."""
    mu, r = norm_stats(h, layer, eps)
    xh, size = normalised(h, mu, r, np.abs(_f64(h)).mean(-1) if layer else None)
    w, c = _f64(weight), _f64(bias)
    return xh * w + c, size * np.abs(w) + np.abs(c), mu, r


def _norm_grad(g, gs, xh, xs, r, layer):
    """r (g - [layer] mean(g) - xh mean(g xh)) and its size."""
    r = r[..., None]
    mean = lambda x: x.mean(-1, keepdims=True)
    v = g - xh * mean(g * xh) - (mean(g) if layer else 0.0)
    return r * v, r * (gs + xs * mean(gs * xs) + (mean(gs) if layer else 0.0))


def resid_norm_grad(dy, h, mu, r, layer, dh_in=0.0, weight=1.0, b=None):
    """{name: (value, size)} of dh, dweight, dbias and (with b) dscale; rows are the first dimension."""
    dy, r, dh_in, w = _f64(dy), _f64(r), _f64(dh_in), _f64(weight)
    xh, xs = normalised(h, mu, r)
    v, size = _norm_grad(dy * w, np.abs(dy * w), xh, xs, r, layer)
    dh, dhs = dh_in + v, np.abs(dh_in) + size
    out = {"dh": (dh, dhs), "dweight": ((dy * xh).sum(0), (np.abs(dy) * xs).sum(0)),
           "dbias": (dy.sum(0), np.abs(dy).sum(0))}
    if b is not None:
        out["dscale"] = ((dh * _f64(b)).sum(0), (dhs * np.abs(_f64(b))).sum(0))
    return out


def gated_norm(o, g, layer, eps, weight=1.0, bias=0.0):
    """(z, size of z, mu, r) of z = swish(g) ((o - mu) r weight + bias), the norm over the last dimension."""
    n, size, mu, r = resid_norm(o, layer, eps, weight, bias)
    g = _f64(g)
    sw = g / (1.0 + np.exp(-g))
    return sw * n, np.abs(sw) * size, mu, r


def gated_norm_grad(dz, o, g, mu, r, layer, weight=1.0, bias=0.0):
    """{name: (value, size)} of do, dg, dweight, dbias and z; rows are the first dimension."""
    dz, g, w, c, r = _f64(dz), _f64(g), _f64(weight), _f64(bias), _f64(r)
    xh, xs = normalised(o, mu, r)
    n, ns = xh * w + c, xs * np.abs(w) + np.abs(c)
    sg = 1.0 / (1.0 + np.exp(-g))
    sw = g * sg
    dn, dns = dz * sw, np.abs(dz * sw)
    do = _norm_grad(dn * w, dns * np.abs(w), xh, xs, r, layer)
    slope = sg * (1.0 + g * (1.0 - sg))               # of swish; its size: sg (1 + |g| (1 - sg))
    return {"do": do, "dg": (dz * n * slope, np.abs(dz) * ns * sg * (1.0 + np.abs(g) * (1.0 - sg))),
            "dweight": ((dn * xh).sum(0), (dns * xs).sum(0)), "dbias": (dn.sum(0), dns.sum(0)),
            "z": (sw * n, np.abs(sw) * ns)}

"""Oracle for the RMS norm, the 8-bit rows and their product (CPU).

TEST INFRASTRUCTURE ONLY: imported by ``tests/``; never by the product
package, which shares no code with it.

fp64, but for the 8-bit rows, whose definition names its fp32 roundings and is
followed literally in numpy's float32. Beside a result stands ``S``, the same
expression with every term taken positive: what the rounding errors of its
fp32 evaluation are proportional to.

Parity: pinned (tests/test_rows8_cpu.py): autograd and explicit sums.
"""
import numpy as np

from .conv import _f64


def rows8(x):
    """(q, scale) of rows [..., C] of float32 values."""
    x = np.asarray(_f64(x), np.float32)
    with np.errstate(all="ignore"):
        top = np.abs(x).max(axis=-1, keepdims=True)
        bad = ~np.isfinite(x).all(axis=-1, keepdims=True)
        small = top < np.float32(2.0 ** -100)
        inv = np.where(small | bad, np.float32(0), np.float32(127) / top).astype(np.float32)
        q = np.where(bad, 0, np.clip(np.rint(x * inv), -127, 127))
        scale = np.where(small, np.float32(0), top / np.float32(127)).astype(np.float32)
    q = np.where(np.isfinite(q), q, 0).astype(np.int64)
    return q, np.where(bad, np.float32(np.nan), scale)[..., 0]


def rms_norm(h, w, eps):
    """out and rstd of rows h [R, C]."""
    h = _f64(h)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=-1) + eps)
    out = h * rstd[..., None]
    return (out if w is None else out * _f64(w)), rstd


def rms_norm_bwd(dout, h, rstd, w, dsum):
    """(dx, S), (dw, S); rstd is a value of the forward pass."""
    dout, h, rstd = _f64(dout), _f64(h), _f64(rstd)[:, None]
    ds = np.zeros_like(h) if dsum is None else _f64(dsum)
    g = dout if w is None else dout * _f64(w)
    xh = h * rstd
    dx = rstd * (g - xh * (g * xh).mean(axis=1, keepdims=True)) + ds
    A, X = np.abs(g), np.abs(xh)
    S = rstd * (A + X * (A * X).mean(axis=1, keepdims=True)) + np.abs(ds)
    return (dx, S), ((dout * xh).sum(axis=0), np.abs(dout * xh).sum(axis=0))


def linear8(xq, xs, wq, ws, bias):
    """(out, S): whole-number sums, scaled."""
    acc = np.asarray(xq, np.int64) @ np.asarray(wq, np.int64).T
    v = acc.astype(np.float64) * _f64(xs)[:, None] * _f64(ws)
    b = 0.0 if bias is None else _f64(bias)
    return v + b, np.abs(v) + np.abs(b)

"""Oracle for the training steps around the scan (fp64, CPU).

TEST INFRASTRUCTURE ONLY: imported by ``tests/``; never by the product
package, which shares no code with it.

Layer norm with its residual add, the gradients of the layer norm, of the
gated RMS norm (``epilogue.py``) and of the short convolution (``conv.py``),
and the 8-bit checkpoint's code. Beside each result stands ``S``, the same
expression with every term taken positive: what the rounding errors of its
fp32 evaluation are proportional to.

Parity: pinned (tests/test_train_cpu.py): autograd through plain torch
forwards in fp64 and central differences.
"""
import numpy as np

from .conv import _f64


def act8(x):
    """(q, E) of an array [..., C]: blocks of 32 channels, E the largest fp32
    exponent field, q = clamp(round(v 2^(133-E)), -127, 127)."""
    x = _f64(x)
    C = x.shape[-1]
    nb = (C + 31) // 32
    q = np.zeros(x.shape, np.int64)
    E = np.zeros(x.shape[:-1] + (nb,), np.int64)
    for i in range(nb):
        v = x[..., 32 * i:32 * i + 32]
        bad = ~np.isfinite(v).all(axis=-1)
        top = np.where(np.isfinite(v), np.abs(v), 0.0).max(axis=-1)
        # floor(log2 top) + 127, at least 0 (frexp: top = m 2^e, 1/2 <= m < 1)
        e = np.where(top > 0, np.frexp(top)[1] - 1 + 127, 0)
        e = np.maximum(e, 0)
        with np.errstate(invalid="ignore"):
            m = np.clip(np.round(np.ldexp(np.where(np.isfinite(v), v, 0.0), 133 - e[..., None])), -127, 127)
        q[..., 32 * i:32 * i + 32] = np.where(bad[..., None], 0, m).astype(np.int64)
        E[..., i] = np.where(bad, 255, e)
    return q, E


def act8_values(q, E):
    q, E = np.asarray(q, np.int64), np.asarray(E, np.int64)
    e = np.repeat(E, 32, axis=-1)[..., :q.shape[-1]]
    v = np.ldexp(q.astype(np.float64), e - 133)
    return np.where(e == 255, np.nan, v)


def layer_norm(h, w, b, eps):
    """out, S, mean, rstd of rows h [R, C]."""
    h = _f64(h)
    w = np.ones(h.shape[1]) if w is None else _f64(w)
    b = np.zeros(h.shape[1]) if b is None else _f64(b)
    mean = h.mean(axis=1)
    d = h - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    out = d * rstd[:, None] * w + b
    S = (np.abs(h) + np.abs(mean)[:, None] + np.abs(h).mean(axis=1)[:, None]) * rstd[:, None] * np.abs(w) + np.abs(b)
    return out, S, mean, rstd


def layer_norm_bwd(dout, h, mean, rstd, w, dsum):
    """dx, dw, db and their S."""
    dout, h, mean, rstd = _f64(dout), _f64(h), _f64(mean)[:, None], _f64(rstd)[:, None]
    w = np.ones(h.shape[1]) if w is None else _f64(w)
    ds = np.zeros_like(h) if dsum is None else _f64(dsum)
    xh = (h - mean) * rstd
    g = dout * w
    dx = rstd * (g - g.mean(axis=1, keepdims=True) - xh * (g * xh).mean(axis=1, keepdims=True)) + ds
    X = (np.abs(h) + np.abs(mean)) * rstd
    A = np.abs(g)
    S = rstd * (A + A.mean(axis=1, keepdims=True) + X * (A * X).mean(axis=1, keepdims=True)) + np.abs(ds)
    return (dx, S), ((dout * xh).sum(axis=0), (np.abs(dout) * X).sum(axis=0)), \
        (dout.sum(axis=0), np.abs(dout).sum(axis=0))


def _sig(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def gated_norm_bwd(dout, y, z, w, group, eps):
    """dy, dz, dw and their S."""
    dout, y, z, w = _f64(dout), _f64(y), _f64(z), _f64(w)
    R, C = y.shape
    s = _sig(z)
    v = y * z * s

    def mean(a):
        return np.repeat(a.reshape(R, C // group, group).mean(axis=2), group, axis=1)

    r = 1.0 / np.sqrt(mean(v * v) + eps)
    g = dout * w
    dv = r * (g - v * r * r * mean(g * v))
    Sv = r * (np.abs(g) + np.abs(v) * r * r * mean(np.abs(g * v)))
    slope = s * (1.0 + z * (1.0 - s))
    top = s * (1.0 + np.abs(z) * (1.0 - s))
    return (dv * z * s, Sv * np.abs(z) * s), (dv * y * slope, Sv * np.abs(y) * top), \
        ((dout * v * r).sum(axis=0), np.abs(dout * v * r).sum(axis=0))


def _shift(a, n, starts):
    """Rows of a [T, ch] n later within each sequence [starts[i], starts[i+1])."""
    o = np.zeros_like(a)
    for s, e in zip(starts, starts[1:]):
        if n >= 0 and e - s > n:
            o[s + n:e] = a[s:e - n]
        elif n < 0 and e - s > -n:
            o[s:e + n] = a[s - n:e]
    return o


def conv1d_bwd(xbc, w, b, dout, reverse=False, cu_seqlens=None, activation="silu"):
    """din [B, L, ch], dw [ch, W], db [ch] and their S, of one direction;
    dout [B, L, ch] is the gradient of x | B | C."""
    xbc, w, dout = _f64(xbc), _f64(w), _f64(dout)
    B, L, ch = xbc.shape
    W = w.shape[1]
    b = np.zeros(ch) if b is None else _f64(b)
    sg = -1 if reverse else 1
    starts = [0, L] if cu_seqlens is None else list(cu_seqlens)
    din, Sin = np.zeros_like(xbc), np.zeros_like(xbc)
    dw, Sw = np.zeros((ch, W)), np.zeros((ch, W))
    db, Sb = np.zeros(ch), np.zeros(ch)
    for i in range(B):
        x, g = xbc[i], dout[i]
        u = b + sum(w[:, k] * _shift(x, sg * (W - 1 - k), starts) for k in range(W))
        U = np.abs(b) + sum(np.abs(w[:, k] * _shift(x, sg * (W - 1 - k), starts)) for k in range(W))
        if activation == "silu":
            s = _sig(u)
            du = g * s * (1.0 + u * (1.0 - s))
        else:
            du = g
        # a rounding of u moves the slope by at most half as much
        D = np.abs(g) * (1.0 + U)
        for k in range(W):
            n = sg * (W - 1 - k)
            din[i] += w[:, k] * _shift(du, -n, starts)
            Sin[i] += np.abs(w[:, k]) * _shift(D, -n, starts)
            t = _shift(x, n, starts)
            dw[:, k] += (du * t).sum(axis=0)
            Sw[:, k] += (D * np.abs(t)).sum(axis=0)
        db += du.sum(axis=0)
        Sb += D.sum(axis=0)
    return (din, Sin), (dw, Sw), (db, Sb)

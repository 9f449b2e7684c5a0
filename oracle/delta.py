"""Oracle for the gated delta rule and its gradient (fp64, CPU).

TEST INFRASTRUCTURE ONLY: imported by ``tests/``; never by the product
package, which shares no code with it.

The recurrence token by token, vectorized over heads, and its adjoint. States
are [sequences, H, P, N] as the library's.

Parity: pinned (tests/test_delta_cpu.py): autograd through a plain torch
recurrence, central differences, hand-worked tokens, block by block against
whole, packed against separate, reversal.
"""
import numpy as np

from .conv import _f64

KEYS = ("q", "k", "v", "g", "beta")


def _units(batch, L, cu):
    """(row, first token, one past the last) of each unit."""
    if cu is None:
        return [(b, 0, L) for b in range(batch)]
    return [(0, a, b) for a, b in zip(cu, cu[1:])]


def _heads(d, b, order):
    """A unit's tokens in order, queries and keys by value head."""
    x = {n: _f64(d[n])[b][order] for n in KEYS}
    rep = x["v"].shape[1] // x["k"].shape[1]
    x["q"], x["k"] = np.repeat(x["q"], rep, axis=1), np.repeat(x["k"], rep, axis=1)
    return x


def _forward(x, S, scale, keep=False):
    """y [L,H,P], the last state [H,N,P] and, with keep, each token's decayed
    state before its write and the error e."""
    L, H, P = x["v"].shape
    y, kept, errs = np.zeros((L, H, P)), [], []
    for t in range(L):
        k = x["k"][t][:, :, None]
        with np.errstate(under="ignore"):
            S = np.exp(x["g"][t])[:, None, None] * S
        e = x["v"][t] - (S * k).sum(axis=1)
        if keep:
            kept.append(S)
            errs.append(e)
        S = S + k * (x["beta"][t][:, None] * e)[:, None, :]
        y[t] = scale * (S * x["q"][t][:, :, None]).sum(axis=1)
    return y, S, kept, errs


def fwd(dirs, scale, cu=None, init=None):
    """(y [b,L,H,P] summed over the directions, the forward's last states)."""
    batch, L, H, P = dirs[0]["v"].shape
    N = dirs[0]["k"].shape[-1]
    units = _units(batch, L, cu)
    y, last = np.zeros((batch, L, H, P)), np.zeros((len(units), H, P, N))
    for i, d in enumerate(dirs):
        for u, (b, lo, hi) in enumerate(units):
            order = np.arange(lo, hi)[::-1] if i else np.arange(lo, hi)
            S = np.zeros((H, N, P)) if i or init is None else _f64(init)[u].transpose(0, 2, 1)
            part, S, _, _ = _forward(_heads(d, b, order), S, scale)
            y[b, order] += part
            if i == 0:
                last[u] = S.transpose(0, 2, 1)
    return y, last


def _back(x, S0, dy, dS, scale):
    L, H, P = x["v"].shape
    _, _, kept, errs = _forward(x, S0, scale, keep=True)
    got = {n: np.zeros_like(x[n]) for n in KEYS}
    mag = np.zeros_like(x["g"])
    for t in reversed(range(L)):
        S, e, b = kept[t], errs[t], x["beta"][t][:, None]
        k, q = x["k"][t][:, :, None], x["q"][t][:, :, None]
        do = scale * dy[t][:, None, :]
        u = (b * e)[:, None, :]
        got["q"][t] = ((S + k * u) * do).sum(axis=2)
        dS = dS + q * do
        z = (dS * k).sum(axis=1)
        f = b * z
        got["beta"][t] = (z * e).sum(axis=1)
        got["v"][t] = f
        got["k"][t] = (dS * u).sum(axis=2) - (S * f[:, None, :]).sum(axis=2)
        dS = dS - k * f[:, None, :]
        got["g"][t] = (dS * S).sum(axis=(1, 2))
        # what the chunked sum for dg adds up: a product for the token's query
        # and each of its key's three parts
        mag[t] = np.abs(x["q"][t] * got["q"][t]).sum(axis=1) + np.abs(x["k"][t]).max(axis=1) * (
            np.abs((dS * u).sum(axis=2)).sum(axis=1) + 2 * np.abs((S * f[:, None, :]).sum(axis=2)).sum(axis=1))
        dS = np.exp(x["g"][t])[:, None, None] * dS
    got["mag"] = mag
    return got, dS


def bwd(dirs, dy, scale, cu=None, init=None, dfinal=None):
    """([gradients of each direction], dinit). Beside g's gradient stands
    "gS", the size of the terms that a chunk of 64 adds up for it."""
    batch, L, H, P = dirs[0]["v"].shape
    G, N = dirs[0]["k"].shape[2:]
    units = _units(batch, L, cu)
    dy = _f64(dy)
    dinit, out = np.zeros((len(units), H, P, N)), []
    for i, d in enumerate(dirs):
        res = {n: np.zeros(tuple(d[n].shape)) for n in KEYS}
        res["gS"] = np.zeros(tuple(d["g"].shape))
        for u, (b, lo, hi) in enumerate(units):
            order = np.arange(lo, hi)[::-1] if i else np.arange(lo, hi)
            S = np.zeros((H, N, P)) if i or init is None else _f64(init)[u].transpose(0, 2, 1)
            dS = np.zeros((H, N, P)) if i or dfinal is None else _f64(dfinal)[u].transpose(0, 2, 1)
            got, dS = _back(_heads(d, b, order), S, dy[b][order], dS, scale)
            for n in ("q", "k"):
                got[n] = got[n].reshape(got[n].shape[0], G, H // G, N).sum(axis=2)
            mag = got.pop("mag")
            for c in range(0, len(order), 64):
                res["gS"][b, order[c:c + 64]] = np.abs(got["g"][c:c + 64]) + mag[c:c + 64].sum(axis=0)
            for n in KEYS:
                res[n][b, order] = got[n]
            if i == 0:
                dinit[u] = dS.transpose(0, 2, 1)
        out.append(res)
    return out, dinit

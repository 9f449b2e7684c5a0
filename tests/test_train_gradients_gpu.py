"""Gradients of the training steps against differences, in directions that a
missing term of the formula would show in, and a layer's backward pass from
8-bit checkpoints at an fp32 bar.

The differences are central ones of the definition in 64 bits (step 2^-17:
what they leave out is step^2/6 = 2^-37 of the third derivative, below every
bar here), so each bar is the kernel's rounding alone: along a direction d,
sum |d| * rel * S over the elements, with S the expression with every term
taken positive. rel: 2^-16 for the gated norm, as for its elements. The layer
norm's elements are within 2^-17 S for given statistics; here the statistics
are the forward pass's, each within 2^-18, and enter every term at most three
times (rstd) and twice (mean): 2^-17 + 5 * 2^-18 < 2^-15."""
import numpy as np
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
import oracle
from oracle import conv as oconv
from oracle import epilogue as oepi
from oracle import train as otrain

pytestmark = pytest.mark.gpu

DEV = "cuda"
LN_REL, GATE_REL = 2.0 ** -15, 2.0 ** -16
STEP = 2.0 ** -17


def _np(t):
    return t.detach().double().cpu().numpy()


def _slope(f, x, d):
    """Derivative of f (an array, summed exactly enough in 64 bits) along d."""
    return float((f(x + STEP * d) - f(x - STEP * d)).sum() / (2 * STEP))


def _along(name, got, S, d, want, rel):
    """The kernel's gradient along d; what a term of the gradient would be
    worth there is for the caller to hold against the bar returned."""
    have, bar = float((_np(got) * d).sum()), float((np.abs(d) * S).sum() * rel)
    print(f"  {name}: {have:.6f}, differences {want:.6f}, bar {bar:.1e}", flush=True)
    assert abs(have - want) <= bar + 2.0 ** -30 * abs(want), name
    return bar


@pytest.mark.parametrize("rows,C", [(6, 200), (5, 777), (3, 2500)])
@pytest.mark.parametrize("weight", [False, True])
def test_layer_norm_gradient_along_its_terms(rows, C, weight):
    g = torch.Generator(device=DEV).manual_seed(C)
    x = torch.randn(rows, C, generator=g, device=DEV) + 0.3
    dout = torch.randn(rows, C, generator=g, device=DEV)
    w = torch.rand(C, generator=g, device=DEV) + 0.5 if weight else None
    o = bm.layer_norm(x, w)
    dx, dw, db = bm.layer_norm_bwd(dout, x, o["mean"], o["rstd"], w)
    h, do = _np(x), _np(dout)
    (_, S), (_, Sw), _ = otrain.layer_norm_bwd(dout, x, o["mean"], o["rstd"], w, None)
    gw = do * (np.ones(C) if w is None else _np(w))
    mean, rstd = h.mean(axis=1, keepdims=True), 1.0 / np.sqrt(h.var(axis=1, keepdims=True) + 1e-5)
    xh = (h - mean) * rstd

    def loss(v):
        return do * otrain.layer_norm(v, w, None, 1e-5)[0]
    r = np.random.default_rng(C)
    # a constant of each row moves nothing: what a missing mean(g) would leave
    # (the signs are such that the rows' shares of it add up)
    c = np.sign(gw.sum(axis=1, keepdims=True)) * r.uniform(0.5, 1.5, (rows, 1))
    bar = _along("constants", dx, S, c * np.ones_like(h), _slope(loss, h, c * np.ones_like(h)), LN_REL)
    assert abs((c * rstd * gw.sum(axis=1, keepdims=True)).sum()) > 20 * bar
    # nor (but for eps) does a multiple of the normalized row
    c = np.sign((gw * xh).sum(axis=1, keepdims=True)) * r.uniform(0.5, 1.5, (rows, 1))
    bar = _along("scales", dx, S, c * xh, _slope(loss, h, c * xh), LN_REL)
    assert abs((c * rstd * (gw * xh).sum(axis=1, keepdims=True)).sum()) > 20 * bar
    d = r.normal(size=h.shape)
    _along("any", dx, S, d, _slope(loss, h, d), LN_REL)
    if weight:
        d = r.normal(size=C)
        _along("weight", dw, Sw, d, _slope(lambda v: do * otrain.layer_norm(h, v, None, 1e-5)[0], _np(w), d), LN_REL)


@pytest.mark.parametrize("rows,C,group", [(3, 512, 256), (4, 1280, 1280), (2, 8192, 1024)])
def test_gated_norm_gradient_along_its_terms(rows, C, group):
    g = torch.Generator(device=DEV).manual_seed(C)
    y, z, dout = (torch.randn(rows, C, generator=g, device=DEV) for _ in range(3))
    w = torch.rand(C, generator=g, device=DEV) + 0.5
    got = bm.gated_norm_bwd(dout, y, z, w, group_size=group)
    Sy, Sz, Sw = (s for _, s in otrain.gated_norm_bwd(dout, y, z, w, group, 1e-5))
    a, b, wd, do = _np(y), _np(z), _np(w), _np(dout)
    r = np.random.default_rng(C)

    def by_y(v):
        return do * oepi.gated_rmsnorm(v, b, wd, group)

    def by_z(v):
        return do * oepi.gated_rmsnorm(a, v, wd, group)
    # a factor of each group moves nothing but for eps: what a gradient
    # without its projection term would leave
    v = a * oepi.silu(b)
    c = np.sign((do * wd * v).reshape(rows, -1, group).sum(axis=2)) * r.uniform(0.5, 1.5, (rows, C // group))
    c = np.repeat(c, group, axis=1)
    bar = _along("scales", got[0], Sy, c * a, _slope(by_y, a, c * a), GATE_REL)
    rg = 1.0 / np.sqrt(np.repeat((v * v).reshape(rows, -1, group).mean(axis=2), group, axis=1) + 1e-5)
    assert abs((c * do * wd * v * rg).sum()) > 20 * bar
    # the same factor through the gate: silu'(z) dz = silu(z) c
    s = 1.0 / (1.0 + np.exp(-b))
    slope = s * (1.0 + b * (1.0 - s))
    d = np.where(np.abs(slope) > 0.2, c * b * s / slope, 0.0)
    _along("gates", got[1], Sz, d, _slope(by_z, b, d), GATE_REL)
    d = r.normal(size=a.shape)
    _along("y", got[0], Sy, d, _slope(by_y, a, d), GATE_REL)
    _along("z", got[1], Sz, d, _slope(by_z, b, d), GATE_REL)
    d = r.normal(size=C)
    _along("weight", got[2], Sw, d, _slope(lambda u: do * oepi.gated_rmsnorm(a, b, u, group), wd, d), GATE_REL)


# ---- a layer's backward pass from what it kept ---------------------------------------------

def _rms(got, ref):
    return float(np.sqrt(np.mean((_np(got).reshape(ref.shape) - ref) ** 2) / np.mean(ref ** 2)))


def test_backward_pass_from_checkpoints():
    """norm with the residual -> projections -> convolution -> scan -> gated
    norm, and back from 8-bit checkpoints of x, xbc, y and z. The oracle runs
    the same backward pass step by step in 64 bits on the values that the
    checkpoints hold, with the forward pass's mean and rstd, so what is left
    is the kernels' rounding.

    Bars: each step's element is within 2^-16 S of its formula (this file's
    head; 2^-17 the norm, 2^-18 the convolution), and S is some 4 times the
    RMS of the results at these sizes (terms of random signs: a result of n
    terms has the RMS of sqrt(n) of them where S has all n, but the rounding
    errors' signs are as random). Five steps follow one another:
    5 * 2^-16 = 7.6e-5, and 1e-4 is the bar, as for full activations; a step
    that took one of the kept arrays elsewhere, or from the unrounded values
    (0.7 % RMS each), is far outside it."""
    batch, L, H, P, N, C = 2, 150, 16, 16, 16, 64
    ch, D = H * P + 2 * N, H * P
    r = np.random.default_rng(15)

    def dev(a):
        return torch.tensor(a, dtype=torch.float32, device=DEV).contiguous()
    nw, nb, gw = dev(r.uniform(0.5, 1.5, C)), dev(0.1 * r.normal(size=C)), dev(r.uniform(0.5, 1.5, D))
    par = [dict(win=dev(r.normal(size=(C, ch)) / 8), cw=dev(r.uniform(-0.5, 0.5, (ch, 4))),
                cb=dev(r.uniform(-0.5, 0.5, ch)), A=dev(-np.exp(r.uniform(0, 1, H))), D=dev(r.normal(size=H)),
                dt=dev(np.log1p(np.exp(r.normal(size=(batch, L, H)) - 2)))) for _ in range(2)]
    x, res, dres = (dev(r.normal(size=(batch, L, C))) for _ in range(3))
    z, dout = dev(r.normal(size=(batch, L, D))), dev(r.normal(size=(batch, L, D)))

    # forward, and what it keeps
    o = bm.layer_norm(x, nw, nb, residual=res, checkpoint=True)
    raw = [dict(xbc=(o["out"] @ p["win"]).contiguous(), weight=p["cw"], bias=p["cb"]) for p in par]
    conv = bm.conv1d(raw[0], raw[1], H, P, 1, N)
    scan = [dict(c, A=p["A"], D=p["D"], dt=p["dt"]) for c, p in zip(conv, par)]
    y = bm.ssd_fwd(scan[0], scan[1], chunk=64).view(batch, L, D)
    out = bm.gated_norm(y, z, gw)
    ref = oepi.gated_rmsnorm(y, z, gw, D)
    assert _rms(out, ref) < 2.0 ** -18
    y8, z8 = bm.act8_pack(y), bm.act8_pack(z)
    kept = [dict(d, xbc=bm.act8_pack(d["xbc"])) for d in raw]

    # backward from it
    dy, dz, dgw = bm.gated_norm_bwd(dout, y8, z8, gw)
    again = bm.conv1d(kept[0], kept[1], H, P, 1, N, dtype=torch.float32)
    scan = [dict(s, **c) for s, c in zip(scan, again)]
    gs = bm.ssd_bwd(scan[0], scan[1], dy.view(batch, L, H, P))
    gc = bm.conv1d_bwd(kept[0], kept[1], gs[0], gs[1], H, P, 1, N, dtype=torch.float32)
    dn = sum(g["xbc"].double() @ p["win"].double().t() for g, p in zip(gc, par)).float().contiguous()
    dx, dnw, dnb = bm.layer_norm_bwd(dn, o["ckpt"], o["mean"], o["rstd"], nw, dsum=dres)

    # the same in 64 bits, each step on the oracle's own results
    def val(a):
        return otrain.act8_values(a.q.cpu().numpy(), a.scale.cpu().numpy())
    (ry, _), (rz, _), (rgw, _) = otrain.gated_norm_bwd(_np(dout).reshape(-1, D), val(y8).reshape(-1, D),
                                                       val(z8).reshape(-1, D), gw, D, 1e-5)
    want = dict(dz=rz, dgw=rgw)
    rdn, adj = 0.0, []
    for p, k, rev in zip(par, kept, (False, True)):
        c = oconv.conv1d(val(k["xbc"]), p["cw"], p["cb"], reverse=rev)
        xs, B, Cc = oconv.split_xbc(c, H, P, 1, N)
        adj.append(dict(x=xs, B=B, C=Cc, A=_np(p["A"]), D=_np(p["D"]), dt=_np(p["dt"])))
    grads = oracle.bissd_bwd(adj[0], adj[1], ry.reshape(batch, L, H, P))
    for i, (p, k, rev) in enumerate(zip(par, kept, (False, True))):
        gr = np.concatenate([np.asarray(grads[i][n]).reshape(batch, L, -1) for n in ("x", "B", "C")], axis=2)
        (gx, _), (gcw, _), (gcb, _) = otrain.conv1d_bwd(val(k["xbc"]), p["cw"], p["cb"], gr, rev)
        want[f"cw{i}"], want[f"cb{i}"], want[f"dA{i}"] = gcw, gcb, np.asarray(grads[i]["A"])
        rdn = rdn + gx @ _np(p["win"]).T
    (rx, _), (rnw, _), (rnb, _) = otrain.layer_norm_bwd(rdn.reshape(-1, C), val(o["ckpt"]).reshape(-1, C),
                                                        _np(o["mean"]).ravel(), _np(o["rstd"]).ravel(), nw,
                                                        _np(dres).reshape(-1, C))
    want.update(dx=rx, dnw=rnw, dnb=rnb)
    have = dict(dz=dz, dgw=dgw, dx=dx, dnw=dnw, dnb=dnb)
    for i in range(2):
        have.update({f"cw{i}": gc[i]["weight"], f"cb{i}": gc[i]["bias"], f"dA{i}": gs[i]["A"]})
    for k in sorted(want):
        e = _rms(have[k], want[k])
        print(f"  {k}: {e:.1e}", flush=True)
        assert e < 1e-4, k

"""GPU parity of the training steps around the scan (layer norm and its
gradient, the gradients of the gated norm and of the short convolution, 8-bit
checkpoints) against the fp64 oracle in oracle/train.py.

Tolerances. Each result is an fp32 evaluation of a short expression with sums
in it; its error is bounded by (number of roundings on the longest path) x
2^-24 x S, S the same expression with every term taken positive. Longest
paths: a row's sum has at most 32 serial terms in a lane, 6 levels over the
wave and 8 waves (46 roundings); two such sums and some ten roundings of
factors make less than 128 = 2^7 roundings for the layer norm (2^-17 S). The
gated norm adds exp's error, 1.5 |z| 2^-24 relative, in each of the factors of
the gate (twice in dz): with |z| <= 8 less than 256 roundings (2^-16 S). The
convolution's gradient has the filter (5), the slope (exp as above, the
filter's error times the slope's derivative: within the factor 1 + U of S)
and the filter again: 2^-18 S; its weights' gradient adds a run's 64 serial
terms and 4 joins: 2^-17 S. bf16 results are one rounding more: they must lie
between the roundings of ref - delta and ref + delta. Checkpoints are exact.
"""
import numpy as np
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
import oracle
from metrics import bf16_rne
from oracle import conv as oconv
from oracle import epilogue as oepi
from oracle import train as otrain

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LN_REL, GATE_REL, CONV_REL, CONVW_REL = 2.0 ** -17, 2.0 ** -16, 2.0 ** -18, 2.0 ** -17


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(name, got, ref, S, rel, dtype="f32"):
    got = _np(got).reshape(ref.shape)
    delta = rel * S
    lo, hi = ref - delta, ref + delta
    if dtype == "bf16":
        lo, hi = bf16_rne(lo), bf16_rne(hi)
    bad = ~((got >= lo) & (got <= hi))
    worst = np.max(np.abs(got - ref) / np.maximum(S, 1e-300)) if got.size else 0.0
    print(f"  {name}: worst {worst:.2e} of S, {int(bad.sum())} outside", flush=True)
    assert not bad.any(), (name, np.argwhere(bad)[:3].tolist(), float(worst))


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def _values(t):
    return otrain.act8_values(t.q.cpu().numpy(), t.scale.cpu().numpy()) if isinstance(t, bm.Act8) else _np(t)


# ---- checkpoints ------------------------------------------------------------------

@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (2, 31), (5, 32), (4, 33), (7, 8), (9, 100), (64, 256),
                                   (3, 5, 4352), (1000, 65), (2, 70001)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_act8_exact(shape, dtype):
    g = _gen(len(shape) * 1000 + shape[-1])
    x = _randn(g, *shape) * torch.exp(2 * _randn(g, *shape))
    x = torch.where(torch.rand(*shape, generator=g, device=DEV) < 0.1, torch.zeros_like(x), x).to(DT[dtype])
    a = bm.act8_pack(x)
    back = bm.act8_unpack(a, dtype=DT[dtype])
    torch.cuda.synchronize()
    q, E = otrain.act8(x)
    assert np.array_equal(a.q.cpu().numpy(), q)
    assert np.array_equal(a.scale.cpu().numpy(), E)
    for d in ("bf16", "f32"):
        assert np.array_equal(_np(bm.act8_unpack(a, dtype=DT[d])), otrain.act8_values(q, E)), d
    assert np.array_equal(_np(back), otrain.act8_values(q, E))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_act8_extremes(dtype):
    """Subnormals, the largest numbers, infinities, NaN, zeros, halves that go
    to even, and a block of them in a row's short tail."""
    one = torch.zeros(8, 40)
    one[0, :4] = torch.tensor([2.0 ** -126, -2.0 ** -130, 2.0 ** -133, 0.0])
    one[1, :3] = torch.tensor([3.3e38, -1.0, 3.0e38])
    one[2, 5] = float("inf")
    one[3, 33] = float("nan")
    one[4, :6] = torch.tensor([1.0, 2.0 ** -7, 3 * 2.0 ** -7, -(2.0 ** -7), 5 * 2.0 ** -7, 1.9921875])
    one[5, 39] = -float("inf")
    one[6, :2] = torch.tensor([2.0 ** -127, 2.0 ** -128])
    x = one.to(DT[dtype]).to(DEV)
    a = bm.act8_pack(x)
    torch.cuda.synchronize()
    q, E = otrain.act8(x)
    assert np.array_equal(a.scale.cpu().numpy(), E)
    assert np.array_equal(a.q.cpu().numpy(), q)
    for d in ("bf16", "f32"):
        got = _np(bm.act8_unpack(a, dtype=DT[d]))
        want = otrain.act8_values(q, E)
        assert np.array_equal(got, want, equal_nan=True), d


def test_act8_unaligned_rows_and_out():
    """Arrays that start inside an allocation, at one element's alignment, and
    what lies around them."""
    g = _gen(5)
    buf = _randn(g, 10 * 65 + 3, dtype=torch.bfloat16)
    x = buf[1:1 + 10 * 65].view(10, 65)
    qb = torch.full((10 * 65 + 6,), 77, dtype=torch.int8, device=DEV)
    sb = torch.full((10 * 3 + 6,), 78, dtype=torch.uint8, device=DEV)
    a = bm.Act8(qb[3:3 + 650].view(10, 65), sb[3:33].view(10, 3))
    assert bm.act8_pack(x, out=a) is a
    ob = torch.full((653,), 9.0, dtype=torch.bfloat16, device=DEV)
    bm.act8_unpack(a, out=ob[1:651].view(10, 65))
    torch.cuda.synchronize()
    q, E = otrain.act8(x)
    assert np.array_equal(a.q.cpu().numpy(), q) and np.array_equal(a.scale.cpu().numpy(), E)
    assert np.array_equal(_np(ob[1:651]).reshape(10, 65), otrain.act8_values(q, E))
    assert (qb[:3] == 77).all() and (qb[653:] == 77).all() and (sb[:3] == 78).all() and (sb[33:] == 78).all()
    assert (ob[0] == 9.0) and (ob[651:] == 9.0).all()


def test_act8_empty():
    for shape in ((0, 64), (0, 3, 7)):
        a = bm.act8_pack(torch.empty(*shape, dtype=torch.bfloat16, device=DEV))
        assert bm.act8_unpack(a).shape == shape


# ---- layer norm ----------------------------------------------------------------------

LN_CASES = [
    # rows, channels, dtype, residual, checkpoint, weight, bias
    (1, 8, "bf16", False, False, True, True),
    (3, 9, "f32", True, True, True, False),
    (5, 33, "bf16", True, True, False, True),
    (64, 2560, "bf16", True, False, True, False),
    (2, 512, "f32", False, True, True, True),
    (70, 513, "bf16", False, True, True, True),
    (37, 777, "f32", True, True, True, True),
    (33, 2048, "bf16", True, True, True, True),
    (9, 2049, "f32", False, True, True, True),
    (9, 4097, "bf16", True, True, True, False),
    (5, 8191, "bf16", False, True, True, True),
    (4, 16384, "f32", True, True, True, True),
    (3, 16383, "bf16", True, False, False, False),
    (5000, 96, "bf16", True, True, True, True),
    (9001, 40, "f32", False, False, True, True),
    (4097, 16, "bf16", True, True, True, True),
    (3001, 130, "f32", True, True, False, True),
    (2000, 200, "bf16", False, True, True, False),
    (1500, 256, "f32", True, False, True, True),
    (129, 257, "bf16", True, True, True, True),
]


def _ln_inputs(rows, C, dtype, residual, weight, bias, seed):
    g = _gen(seed)
    x = (_randn(g, rows, C) * torch.exp(0.5 * _randn(g, C)) + 0.3).to(DT[dtype])
    r = _randn(g, rows, C, dtype=DT[dtype]) if residual else None
    w = torch.rand(C, generator=g, device=DEV) + 0.5 if weight else None
    b = _randn(g, C) if bias else None
    return g, x, r, w, b


@pytest.mark.parametrize("case", LN_CASES, ids=[f"{c[0]}x{c[1]}-{c[2]}-r{c[3]:d}c{c[4]:d}w{c[5]:d}b{c[6]:d}"
                                                for c in LN_CASES])
def test_layer_norm(case):
    rows, C, dtype, residual, ckpt, weight, bias = case
    print(f"case {case}", flush=True)
    g, x, r, w, b = _ln_inputs(rows, C, dtype, residual, weight, bias, 7 + C)
    o = bm.layer_norm(x, w, b, residual=r, eps=1e-5, checkpoint=ckpt)
    torch.cuda.synchronize()
    h = (x.float() + r.float()).to(DT[dtype]) if residual else x
    assert torch.equal(o["sum"], h)
    ref, S, mean, rstd = otrain.layer_norm(h, w, b, 1e-5)
    _close("out", o["out"], ref, S, LN_REL, dtype)
    H = np.abs(_np(h)).mean(axis=1)
    _close("mean", o["mean"], mean, H, 2.0 ** -18)
    # the mean's error shifts the variance by its square
    _close("rstd", o["rstd"], rstd, rstd * (1 + 2.0 ** -18 * (H * rstd) ** 2), 2.0 ** -18)
    if ckpt:
        q, E = otrain.act8(h)
        assert np.array_equal(o["ckpt"].q.cpu().numpy(), q)
        assert np.array_equal(o["ckpt"].scale.cpu().numpy(), E)
    else:
        assert o["ckpt"] is None
    # its gradient, from h and from the checkpoint
    dout = _randn(g, rows, C, dtype=DT[dtype])
    dsum = _randn(g, rows, C, dtype=DT[dtype]) if residual else None
    for kept in [o["sum"]] + ([o["ckpt"]] if ckpt else []):
        dx, dw, db = bm.layer_norm_bwd(dout, kept, o["mean"], o["rstd"], w, dsum=dsum)
        torch.cuda.synchronize()
        v = _values(kept)
        gx, gw, gb = otrain.layer_norm_bwd(dout, v, o["mean"], o["rstd"], w, dsum)
        _close("dx", dx, *gx, LN_REL, dtype)
        _close("dweight", dw, *gw, LN_REL)
        _close("dbias", db, *gb, LN_REL)
        dx2, none_w, none_b = bm.layer_norm_bwd(dout, kept, o["mean"], o["rstd"], w, dsum=dsum, wgrad=False)
        assert none_w is None and none_b is None and torch.equal(dx, dx2)
        again = bm.layer_norm_bwd(dout, kept, o["mean"], o["rstd"], w, dsum=dsum)
        assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))


def test_layer_norm_far_mean():
    """A large common offset: the two-pass variance keeps the small spread."""
    g = _gen(3)
    x = _randn(g, 16, 1000) + 3000.0
    o = bm.layer_norm(x, eps=1e-5)
    ref, S, mean, rstd = otrain.layer_norm(x, None, None, 1e-5)
    H = np.abs(_np(x)).mean(axis=1)
    _close("out", o["out"], ref, S, LN_REL)
    _close("rstd", o["rstd"], rstd, rstd * (1 + 2.0 ** -18 * (H * rstd) ** 2), 2.0 ** -18)


def test_layer_norm_constant_rows_and_zeros():
    x = torch.zeros(4, 100, device=DEV)
    x[1] = 5.0
    o = bm.layer_norm(x, eps=1e-5, checkpoint=True)
    assert torch.equal(o["out"], torch.zeros_like(x))
    assert torch.equal(o["mean"], torch.tensor([0.0, 5.0, 0.0, 0.0], device=DEV))


def test_layer_norm_nan_row_stays_in_its_row():
    g = _gen(4)
    x = _randn(g, 300, 129, dtype=torch.bfloat16)
    clean = bm.layer_norm(x, checkpoint=True)
    bad = x.clone()
    bad[7, 128] = float("nan")
    bad[200, 0] = float("inf")
    o = bm.layer_norm(bad, checkpoint=True)
    keep = torch.ones(300, dtype=torch.bool, device=DEV)
    keep[[7, 200]] = False
    assert torch.equal(o["out"][keep], clean["out"][keep])
    assert o["out"][7].isnan().all() and o["out"][200].isnan().all()
    assert o["ckpt"].scale[7, 4] == 255 and o["ckpt"].scale[200, 0] == 255
    assert torch.equal(o["ckpt"].scale[7, :4], clean["ckpt"].scale[7, :4])


def test_layer_norm_in_place_stream():
    """sum_out may be the residual or x; dx may be dsum."""
    g, x, r, w, b = _ln_inputs(50, 2500, "bf16", True, True, True, 11)
    want = bm.layer_norm(x, w, b, residual=r)
    r2, x2 = r.clone(), x.clone()
    o = bm.layer_norm(x, w, b, residual=r2, sum_out=r2)
    assert o["sum"] is r2 and torch.equal(r2, want["sum"]) and torch.equal(o["out"], want["out"])
    o = bm.layer_norm(x2, w, b, residual=r, sum_out=x2)
    assert torch.equal(x2, want["sum"]) and torch.equal(o["out"], want["out"])
    dout, ds = _randn(g, 50, 2500, dtype=torch.bfloat16), _randn(g, 50, 2500, dtype=torch.bfloat16)
    dx = bm.layer_norm_bwd(dout, want["sum"], want["mean"], want["rstd"], w, dsum=ds)[0]
    ds2 = ds.clone()
    got = bm.layer_norm_bwd(dout, want["sum"], want["mean"], want["rstd"], w, dsum=ds2, dx=ds2)[0]
    assert got is ds2 and torch.equal(got, dx)


def test_layer_norm_unaligned_and_guards():
    """Rows at one element's alignment; nothing around the outputs changes."""
    g = _gen(12)
    rows, C = 7, 101
    n = rows * C

    def at(off, fill=None, dtype=torch.bfloat16):
        buf = torch.full((n + 16,), 3.0, dtype=dtype, device=DEV)
        v = buf[off:off + n].view(rows, C)
        if fill is not None:
            v.copy_(fill)
        return buf, v
    _, x = at(1, _randn(g, rows, C))
    _, r = at(3, _randn(g, rows, C))
    ob, out = at(5)
    sb, s = at(7)
    qb = torch.full((n + 9,), 5, dtype=torch.int8, device=DEV)
    cb = torch.full((rows * 4 + 9,), 6, dtype=torch.uint8, device=DEV)
    ck = bm.Act8(qb[3:3 + n].view(rows, C), cb[1:1 + rows * 4].view(rows, 4))
    o = bm.layer_norm(x, residual=r, out=out, sum_out=s, checkpoint=ck)
    want = bm.layer_norm(x.clone(), residual=r.clone(), checkpoint=True)
    assert torch.equal(out, want["out"]) and torch.equal(s, want["sum"]) and torch.equal(ck.q, want["ckpt"].q)
    assert torch.equal(ck.scale, want["ckpt"].scale)
    db, dx = at(9)
    _, dout = at(11, _randn(g, rows, C))
    bm.layer_norm_bwd(dout, ck, o["mean"], o["rstd"], dx=dx)
    assert torch.equal(dx, bm.layer_norm_bwd(dout.clone(), want["ckpt"], o["mean"], o["rstd"])[0])
    for buf, off in ((ob, 5), (sb, 7), (db, 9)):
        assert (buf[:off] == 3.0).all() and (buf[off + n:] == 3.0).all()
    assert (qb[:3] == 5).all() and (qb[3 + n:] == 5).all() and (cb[:1] == 6).all() and (cb[1 + rows * 4:] == 6).all()


def test_layer_norm_empty():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    o = bm.layer_norm(x, checkpoint=True)
    assert o["out"].shape == (0, 64)
    dx, dw, db = bm.layer_norm_bwd(x, o["ckpt"], o["mean"], o["rstd"])
    assert torch.equal(dw, torch.zeros(64, device=DEV)) and torch.equal(db, torch.zeros(64, device=DEV))


def test_layer_norm_bwd_differences():
    """Directional derivative by central differences of the forward call."""
    g, x, _, w, b = _ln_inputs(6, 200, "f32", False, True, True, 13)
    dout, dirx = _randn(g, 6, 200), _randn(g, 6, 200)
    o = bm.layer_norm(x, w, b)
    dx, dw, db = bm.layer_norm_bwd(dout, x, o["mean"], o["rstd"], w)

    def loss(xx, ww, bb):
        return (bm.layer_norm(xx, ww, bb)["out"].double() * dout.double()).sum().item()
    eps = 2.0 ** -6
    # h^2/6 times the third derivative of order 1 a row, and the calls'
    # rounding 2^-17 S over 2 h: far below a hundredth of the gradient's size
    for got, up, down in ((dx, loss(x + eps * dirx, w, b), loss(x - eps * dirx, w, b)),):
        want = (up - down) / (2 * eps)
        have = (got.double() * dirx.double()).sum().item()
        assert abs(want - have) < 0.01 * got.double().norm().item() * dirx.double().norm().item() / 10
    dirw = _randn(g, 200)
    want = (loss(x, w + eps * dirw, b) - loss(x, w - eps * dirw, b)) / (2 * eps)
    assert abs(want - (dw.double() * dirw.double()).sum().item()) < 1e-3 * dw.double().norm().item() * dirw.norm().item()
    want = (loss(x, w, b + eps * dirw) - loss(x, w, b - eps * dirw)) / (2 * eps)
    assert abs(want - (db.double() * dirw.double()).sum().item()) < 1e-3 * db.double().norm().item() * dirw.norm().item()


# ---- the gated norm's gradient ------------------------------------------------------------

GATE_CASES = [
    # rows, channels, group, dtype, y kept in 8 bits, z kept
    (1, 256, 256, "bf16", False, False),
    (3, 256, 256, "f32", True, True),
    (17, 1280, 256, "bf16", True, False),
    (5, 1536, 768, "f32", False, True),
    (33, 4096, 4096, "bf16", True, True),
    (12, 5120, 1280, "bf16", False, True),
    (7, 8192, 256, "f32", False, False),
    (6, 8192, 8192, "bf16", True, True),
    (2500, 768, 768, "bf16", False, False),
    (1100, 2048, 1024, "f32", True, False),
]


@pytest.mark.parametrize("case", GATE_CASES, ids=lambda c: "x".join(map(str, c)))
def test_gated_norm_bwd(case):
    rows, C, gs, dtype, y8, z8 = case
    print(f"case {case}", flush=True)
    g = _gen(C + rows)
    y = _randn(g, rows, C) * torch.exp(0.5 * _randn(g, C))
    z = (2 * _randn(g, rows, C)).clamp(-8, 8).to(DT[dtype])
    w = torch.rand(C, generator=g, device=DEV) + 0.5
    dout = _randn(g, rows, C, dtype=DT[dtype])
    yk, zk = bm.act8_pack(y) if y8 else y, bm.act8_pack(z) if z8 else z
    dy, dz, dw = bm.gated_norm_bwd(dout, yk, zk, w, group_size=gs, eps=1e-5)
    torch.cuda.synchronize()
    ry, rz, rw = otrain.gated_norm_bwd(dout, _values(yk), _values(zk), w, gs, 1e-5)
    _close("dy", dy, *ry, GATE_REL)
    _close("dz", dz, *rz, GATE_REL, dtype)
    _close("dweight", dw, *rw, GATE_REL)
    again = bm.gated_norm_bwd(dout, yk, zk, w, group_size=gs, eps=1e-5)
    assert all(torch.equal(a, b) for a, b in zip(again, (dy, dz, dw)))
    part = bm.gated_norm_bwd(dout, yk, zk, w, group_size=gs, eps=1e-5, wgrad=False)
    assert part[2] is None and torch.equal(part[0], dy) and torch.equal(part[1], dz)


def test_gated_norm_bwd_far_gates_and_zero_groups():
    """Gates of any size give finite gradients; a group of zeros has the norm
    1/sqrt(eps)."""
    rows, C = 4, 512
    g = _gen(21)
    y, z, w = _randn(g, rows, C), 200 * _randn(g, rows, C), torch.ones(C, device=DEV)
    y[1, :256] = 0
    dout = _randn(g, rows, C)
    dy, dz, dw = bm.gated_norm_bwd(dout, y, z, w, group_size=256)
    for t in (dy, dz, dw):
        assert t.isfinite().all()
    s = z.double() * torch.sigmoid(z.double())
    assert torch.allclose(dy[1, :256].double(), (dout.double() * s)[1, :256] / 1e-5 ** 0.5, rtol=1e-4, atol=1e-30)
    assert (dz[1, :256] == 0).all()


def test_gated_norm_bwd_matches_forward_differences():
    rows, C = 3, 512
    g = _gen(22)
    y, z, w = _randn(g, rows, C), _randn(g, rows, C), torch.rand(C, generator=g, device=DEV) + 0.5
    dout = _randn(g, rows, C)
    got = bm.gated_norm_bwd(dout, y, z, w, group_size=256)

    def loss(a, b, c):
        return (bm.gated_norm(a, b, c, group_size=256).double() * dout.double()).sum().item()
    eps = 2.0 ** -6
    for i, t in enumerate((y, z, w)):
        d = _randn(g, *t.shape)
        args = [y, z, w]
        args[i] = t + eps * d
        up = loss(*args)
        args[i] = t - eps * d
        want = (up - loss(*args)) / (2 * eps)
        have = (got[i].double() * d.double()).sum().item()
        assert abs(want - have) < 1e-3 * got[i].double().norm().item() * d.double().norm().item(), i


def test_gated_norm_bwd_empty():
    e = torch.empty(0, 512, device=DEV)
    dy, dz, dw = bm.gated_norm_bwd(e, e, e, torch.ones(512, device=DEV))
    assert dy.shape == (0, 512) and torch.equal(dw, torch.zeros(512, device=DEV))


# ---- the convolution ---------------------------------------------------------------------------

CONV_CASES = [
    # batch, L, H, P, G, N, width, dtype, act, both, bias, checkpoint, packed lengths
    (1, 1, 1, 16, 1, 16, 4, "bf16", "silu", True, True, False, None),
    (2, 3, 2, 16, 1, 16, 4, "f32", "silu", True, True, False, None),
    (1, 2, 1, 16, 1, 16, 3, "f32", "none", True, False, True, None),
    (3, 65, 3, 16, 1, 16, 2, "bf16", "silu", True, True, True, None),
    (1, 300, 5, 7, 1, 3, 4, "bf16", "silu", True, True, True, None),
    (1, 77, 3, 5, 1, 3, 3, "f32", "silu", False, True, False, None),
    (2, 130, 4, 64, 2, 64, 4, "bf16", "silu", True, True, True, None),
    (1, 1000, 2, 64, 1, 128, 4, "f32", "silu", True, True, True, None),
    (1, None, 4, 16, 1, 16, 4, "bf16", "silu", True, True, False, (300, 0, 1, 2, 3, 4, 77, 0, 60, 5)),
    (1, None, 3, 7, 1, 3, 4, "f32", "silu", True, True, True, (1, 1, 1, 63, 2, 64, 128)),
    (1, None, 2, 16, 1, 16, 2, "f32", "none", True, True, False, (0, 5, 0)),
    (1, None, 8, 64, 1, 128, 3, "bf16", "silu", True, False, True, (700, 33, 512, 260)),
    (1, None, 2, 16, 1, 16, 4, "f32", "silu", True, True, True, (3, 0, 5, 1, 30, 64) * 21),
    (1, None, 2, 16, 1, 16, 4, "bf16", "silu", True, True, True, (1, 2, 0, 70) * 33),
    (1, None, 2, 16, 1, 16, 3, "f32", "silu", True, True, False, (1,) * 300),
]


def _conv_inputs(case, seed):
    batch, L, H, P, G, N, W, dtype, act, both, bias, ckpt, lens = case
    cu = None
    if lens is not None:
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        L = cu[-1]
    ch = H * P + 2 * G * N
    g = _gen(seed)
    dirs, grads = [], []
    for _ in range(2 if both else 1):
        x = _randn(g, batch, L, ch, dtype=DT[dtype])
        dirs.append(dict(xbc=bm.act8_pack(x) if ckpt else x, weight=_randn(g, ch, W) * 0.5,
                         bias=_randn(g, ch) * 0.5 if bias else None))
        grads.append(dict(x=_randn(g, batch, L, H, P), B=_randn(g, batch, L, G, N), C=_randn(g, batch, L, G, N)))
    if not both:
        dirs.append(None)
        grads.append(None)
    return dirs, grads, cu, L, ch


@pytest.mark.parametrize("case", CONV_CASES, ids=lambda c: "-".join(str(v).replace(" ", "")[:32] for v in c))
def test_conv1d_bwd(case):
    batch, _, H, P, G, N, W, dtype, act, both, bias, ckpt, lens = case
    print(f"case {case}", flush=True)
    dirs, grads, cu, L, ch = _conv_inputs(case, 31)
    kw = dict(activation=act, cu_seqlens=cu, dtype=DT[dtype])
    res = bm.conv1d_bwd(dirs[0], dirs[1], grads[0], grads[1], H, P, G, N, **kw)
    torch.cuda.synchronize()
    for d, gr, o, rev in zip(dirs, grads, res, (False, True)):
        if d is None:
            assert o is None
            continue
        dout = torch.cat([gr[k].reshape(batch, L, -1) for k in ("x", "B", "C")], dim=2)
        rx, rw, rb = otrain.conv1d_bwd(_values(d["xbc"]), d["weight"], d["bias"], dout, rev, cu, act)
        _close("dxbc", o["xbc"], *rx, CONV_REL, dtype)
        _close("dweight", o["weight"], *rw, CONVW_REL)
        if bias:
            _close("dbias", o["bias"], *rb, CONVW_REL)
        else:
            assert o["bias"] is None
    again = bm.conv1d_bwd(dirs[0], dirs[1], grads[0], grads[1], H, P, G, N, **kw)
    for o, p in zip(res, again):
        assert o is None or all(o[k] is None or torch.equal(o[k], p[k]) for k in o)
    if ckpt:
        # the outputs rebuilt from the checkpoint are those of its values
        full = [None if d is None else dict(d, xbc=bm.act8_unpack(d["xbc"], dtype=DT[dtype])) for d in dirs]
        a = bm.conv1d(dirs[0], dirs[1], H, P, G, N, **kw)
        b = bm.conv1d(full[0], full[1], H, P, G, N, **kw)
        for o, p in zip(a, b):
            assert o is None or all(torch.equal(o[k], p[k]) for k in ("x", "B", "C"))


def test_conv1d_bwd_layer():
    """The training layer's size in one direction each, against the oracle on
    a slab of channels (channels are independent), and what a NaN reaches."""
    case = (8, 1024, 64, 64, 1, 128, 4, "bf16", "silu", True, True, True, None)
    dirs, grads, cu, L, ch = _conv_inputs(case, 32)
    res = bm.conv1d_bwd(dirs[0], dirs[1], grads[0], grads[1], 64, 64, 1, 128)
    torch.cuda.synchronize()
    for d, gr, o, rev in zip(dirs, grads, res, (False, True)):
        dout = torch.cat([gr[k].reshape(8, L, -1) for k in ("x", "B", "C")], dim=2)
        for lo, hi in ((0, 40), (4090, 4130), (4320, 4352)):
            sl = slice(lo, hi)
            rx, rw, rb = otrain.conv1d_bwd(_values(d["xbc"])[..., sl], d["weight"][sl], d["bias"][sl], dout[..., sl],
                                           rev, cu, "silu")
            _close("dxbc", o["xbc"][..., sl], *rx, CONV_REL, "bf16")
            _close("dweight", o["weight"][sl], *rw, CONVW_REL)
            _close("dbias", o["bias"][sl], *rb, CONVW_REL)


def test_conv1d_bwd_nan_stays_in_its_sequence():
    case = (1, None, 2, 16, 1, 16, 4, "f32", "silu", True, True, False, (40, 50, 60))
    dirs, grads, cu, L, ch = _conv_inputs(case, 33)
    clean = bm.conv1d_bwd(dirs[0], dirs[1], grads[0], grads[1], 2, 16, 1, 16, cu_seqlens=cu)
    for d in dirs:
        d["xbc"][0, 40, 3] = float("nan")
        d["xbc"][0, 89, 4] = float("inf")
    res = bm.conv1d_bwd(dirs[0], dirs[1], grads[0], grads[1], 2, 16, 1, 16, cu_seqlens=cu)
    for o, p in zip(res, clean):
        for sl in (slice(0, 40), slice(90, 150)):
            assert torch.equal(o["xbc"][:, sl], p["xbc"][:, sl])
        keep = [c for c in range(ch) if c not in (3, 4)]
        assert torch.equal(o["xbc"][..., keep], p["xbc"][..., keep])
        assert torch.equal(o["weight"][keep], p["weight"][keep])
        assert o["xbc"][0, 40, 3].isnan()


def test_conv1d_bwd_empty():
    case = (2, 0, 2, 16, 1, 16, 4, "bf16", "silu", True, True, False, None)
    dirs, grads, cu, L, ch = _conv_inputs(case, 34)
    for o in bm.conv1d_bwd(dirs[0], dirs[1], grads[0], grads[1], 2, 16, 1, 16):
        assert o["xbc"].shape == (2, 0, ch)
        assert torch.equal(o["weight"], torch.zeros(ch, 4, device=DEV))
        assert torch.equal(o["bias"], torch.zeros(ch, device=DEV))


def test_binding_refusals():
    x = torch.zeros(2, 4, 64, device=DEV)
    w = torch.zeros(64, 4, device=DEV)
    d, a = dict(xbc=x, weight=w), dict(xbc=bm.act8_pack(x), weight=w)
    gr = dict(x=torch.zeros(2, 4, 2, 16, device=DEV), B=torch.zeros(2, 4, 1, 16, device=DEV),
              C=torch.zeros(2, 4, 1, 16, device=DEV))
    dims = (2, 16, 1, 16)
    with pytest.raises(TypeError, match="Act8"):
        bm.conv1d_bwd(d, a, gr, gr, *dims)
    with pytest.raises(TypeError, match="Act8"):
        bm.conv1d(a, d, *dims)
    with pytest.raises(ValueError, match="contexts"):
        bm.conv1d(a, None, *dims, init_ctx=torch.zeros(2, 3, 64, device=DEV))
    with pytest.raises(TypeError, match="dtype"):
        bm.conv1d(d, None, *dims, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="together"):
        bm.conv1d_bwd(d, None, gr, gr, *dims)
    with pytest.raises(TypeError, match="dtype"):
        bm.layer_norm(torch.zeros(2, 64, dtype=torch.float16, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        bm.layer_norm(torch.zeros(64, 16, device=DEV).t())
    with pytest.raises(bm.BimambaError):
        bm.layer_norm(torch.zeros(2, 7, device=DEV))
    with pytest.raises(ValueError, match="residual"):
        bm.layer_norm(x, sum_out=x)
    with pytest.raises(ValueError, match="mean"):
        bm.layer_norm_bwd(x, x, torch.zeros(2, device=DEV), torch.zeros(2, 4, device=DEV))
    with pytest.raises(bm.BimambaError):
        bm.gated_norm_bwd(x, x, x, torch.zeros(64, device=DEV))


# ---- together -------------------------------------------------------------------------------------

def _layer(seed, batch=2, L=150, H=4, P=16, N=16):
    """A mixer layer's parameters and input, fp32 on the host in fp64."""
    r = np.random.default_rng(seed)
    C, ch = 64, H * P + 2 * N
    p = dict(nw=r.uniform(0.5, 1.5, C), nb=0.1 * r.normal(size=C), gw=r.uniform(0.5, 1.5, 256))
    for s in "fr":
        p[s] = dict(win=r.normal(size=(C, ch)) / 8, cw=r.uniform(-0.5, 0.5, (ch, 4)), cb=r.uniform(-0.5, 0.5, ch),
                    A=-np.exp(r.uniform(0, 1, H)), D=r.normal(size=H),
                    dt=np.log1p(np.exp(r.normal(size=(batch, L, H)) - 2)))
    x, res = r.normal(size=(batch, L, C)), r.normal(size=(batch, L, C))
    return p, x, res


def test_training_step_of_a_layer():
    """norm with the residual -> projections -> convolution -> scan -> gated
    norm, and back, through the framework's calls and from 8-bit checkpoints,
    against autograd in fp64 of the same layer evaluated at the checkpointed
    values' points: gradients agree to the checkpoints' error. From full
    activations they agree to fp32."""
    batch, L, H, P, N = 2, 150, 16, 16, 16
    ch, C = H * P + 2 * N, 64
    p, x, res = _layer(5, batch, L, H, P, N)
    r = np.random.default_rng(6)
    z = r.normal(size=(batch, L, H * P))
    dout = r.normal(size=(batch, L, H * P))
    dres = r.normal(size=(batch, L, C))

    def dev(a):
        return torch.tensor(a, dtype=torch.float32, device=DEV).contiguous()

    def step(kept):
        o = bm.layer_norm(dev(x), dev(p["nw"]), dev(p["nb"]), residual=dev(res), checkpoint=kept)
        conv, raw = [], []
        for s in "fr":
            xbc = (o["out"] @ dev(p[s]["win"])).contiguous()
            raw.append(dict(xbc=xbc, weight=dev(p[s]["cw"]), bias=dev(p[s]["cb"])))
        conv = bm.conv1d(raw[0], raw[1], H, P, 1, N)
        scan = [dict(c, A=dev(p[s]["A"]), D=dev(p[s]["D"]), dt=dev(p[s]["dt"])) for c, s in zip(conv, "fr")]
        y = bm.ssd_fwd(scan[0], scan[1], chunk=64)
        zz, gw = dev(z), dev(p["gw"])
        bm.gated_norm(y.view(batch, L, H * P), zz, gw)
        # what the backward keeps
        if kept:
            xk, yk, zk = o["ckpt"], bm.act8_pack(y.view(batch, L, H * P)), bm.act8_pack(zz)
            raw = [dict(d, xbc=bm.act8_pack(d["xbc"])) for d in raw]
            conv = bm.conv1d(raw[0], raw[1], H, P, 1, N, dtype=torch.float32)
            scan = [dict(s, **c) for s, c in zip(scan, conv)]
        else:
            xk, yk, zk = o["sum"], y.view(batch, L, H * P), zz
        dy, dz, dgw = bm.gated_norm_bwd(dev(dout), yk, zk, gw)
        gs = bm.ssd_bwd(scan[0], scan[1], dy.view(batch, L, H, P))
        gc = bm.conv1d_bwd(raw[0], raw[1], gs[0], gs[1], H, P, 1, N, dtype=torch.float32)
        dn = sum(g["xbc"] @ dev(p[s]["win"]).t() for g, s in zip(gc, "fr")).contiguous()
        dx, dnw, dnb = bm.layer_norm_bwd(dn, xk, o["mean"], o["rstd"], dev(p["nw"]), dsum=dev(dres))
        return dict(dx=dx, dnw=dnw, dnb=dnb, dz=dz, dgw=dgw, dcw=gc[0]["weight"], dcb=gc[1]["bias"])

    # fp64 autograd of the same layer
    def leaf(a):
        return torch.tensor(a, dtype=torch.float64, requires_grad=True)
    tx, tnw, tnb, tz, tgw = leaf(x), leaf(p["nw"]), leaf(p["nb"]), leaf(z), leaf(p["gw"])
    h = tx + torch.tensor(res)
    nrm = torch.nn.functional.layer_norm(h, (C,), tnw, tnb, 1e-5)
    cws, cbs, ys = [], [], []
    for s in "fr":
        cw, cb = leaf(p[s]["cw"]), leaf(p[s]["cb"])
        cws.append(cw)
        cbs.append(cb)
        xbc = (nrm @ torch.tensor(p[s]["win"])).transpose(1, 2)
        dt = torch.tensor(p[s]["dt"])
        if s == "r":
            xbc, dt = xbc.flip(2), dt.flip(1)
        u = torch.nn.functional.silu(torch.nn.functional.conv1d(torch.nn.functional.pad(xbc, (3, 0)), cw[:, None], cb,
                                                                groups=ch)).transpose(1, 2)
        xs = u[..., :H * P].reshape(batch, L, H, P)
        B, Cc = u[..., H * P:H * P + N], u[..., H * P + N:]
        A, D = torch.tensor(p[s]["A"]), torch.tensor(p[s]["D"])
        st, out = torch.zeros(batch, H, P, N, dtype=torch.float64), []
        for t in range(L):
            st = torch.exp(dt[:, t] * A)[..., None, None] * st + \
                (dt[:, t, :, None] * xs[:, t])[..., None] * B[:, t, None, None, :]
            out.append((st * Cc[:, t, None, None, :]).sum(-1) + D[:, None] * xs[:, t])
        y = torch.stack(out, dim=1)
        ys.append(y.flip(1) if s == "r" else y)
    v = (ys[0] + ys[1]).reshape(batch, L, H * P) * torch.nn.functional.silu(tz)
    o = v * torch.rsqrt((v * v).mean(dim=2, keepdim=True) + 1e-5) * tgw
    ((o * torch.tensor(dout)).sum() + (h * torch.tensor(dres)).sum()).backward()
    want = dict(dx=tx.grad, dnw=tnw.grad, dnb=tnb.grad, dz=tz.grad, dgw=tgw.grad, dcw=cws[0].grad, dcb=cbs[1].grad)
    full, kept = step(False), step(True)
    for k, ref in want.items():
        ref = ref.numpy()
        scale = np.sqrt(np.mean(ref ** 2))
        e_full = np.sqrt(np.mean((_np(full[k]).reshape(ref.shape) - ref) ** 2)) / scale
        e_kept = np.sqrt(np.mean((_np(kept[k]).reshape(ref.shape) - ref) ** 2)) / scale
        print(f"  {k}: full {e_full:.1e} 8-bit {e_kept:.1e}", flush=True)
        # fp32: a chain of five operators, each within 2^-16 of its terms'
        # sizes, amplified by cancellation in the sums over tokens
        assert e_full < 1e-4, k
        # a kept value is off by a uniform error of at most 2^-7 of its
        # block's largest magnitude, about 3 times the RMS of its 32 values:
        # 3 * 2^-7 / sqrt(3) / 2 = 0.7 % RMS each for x, xbc, y and z, through
        # slopes of order one
        assert e_kept < 0.1, k


def test_graph_replays_and_streams():
    """Captured once, replayed on new inputs with eager work between; two
    graphs alive; a call on a stream of its own."""
    rows, C, H, P, N = 300, 512, 4, 16, 16
    ch = H * P + 2 * N
    g = _gen(41)
    x, r, dout = (torch.empty(rows, C, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    w, b = torch.rand(C, generator=g, device=DEV), _randn(g, C)
    y, gz, gd = torch.empty(rows, C, device=DEV), torch.empty_like(x), torch.empty_like(x)
    conv = [dict(xbc=torch.empty(1, rows, ch, dtype=torch.bfloat16, device=DEV), weight=_randn(g, ch, 4),
                 bias=_randn(g, ch)) for _ in range(2)]
    grads = [dict(x=torch.empty(1, rows, H, P, device=DEV), B=torch.empty(1, rows, 1, N, device=DEV),
                  C=torch.empty(1, rows, 1, N, device=DEV)) for _ in range(2)]
    cu = [0, 100, 130, rows]

    def fill(seed):
        q = _gen(seed)
        for t in [x, r, dout, y, gz, gd] + [d["xbc"] for d in conv] + [v for d in grads for v in d.values()]:
            t.copy_(torch.randn(t.shape, generator=q, device=DEV))

    def norms():
        o = bm.layer_norm(x, w, b, residual=r, checkpoint=True)
        return list(bm.layer_norm_bwd(dout, o["ckpt"], o["mean"], o["rstd"], w, dsum=dout)) + \
            [o["out"], o["sum"], o["ckpt"].q] + list(bm.gated_norm_bwd(gd, bm.act8_pack(y), gz, w, group_size=256))

    def convs():
        k = [dict(d, xbc=bm.act8_pack(d["xbc"])) for d in conv]
        o = bm.conv1d_bwd(k[0], k[1], grads[0], grads[1], H, P, 1, N, cu_seqlens=cu)
        f = bm.conv1d(k[0], k[1], H, P, 1, N, cu_seqlens=cu)
        return [v for d in o + f for v in d.values()]
    fill(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        norms(), convs()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for f in (norms, convs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = f()
        graphs.append((gr, out, f))
    for seed in (2, 3, 4):
        fill(seed)
        for gr, out, f in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for gr, out, f in graphs:
            for a, e in zip(out, f()):
                assert torch.equal(a, e)
    # the stream argument: inputs ready on it, results taken after it
    side = torch.cuda.Stream()
    want = bm.layer_norm(x, w, b, residual=r)
    torch.cuda.synchronize()
    o = bm.layer_norm(x, w, b, residual=r, stream=side)
    d = bm.layer_norm_bwd(dout, o["sum"], o["mean"], o["rstd"], w, stream=side)
    side.synchronize()
    assert torch.equal(o["out"], want["out"])
    assert all(torch.equal(a, e) for a, e in zip(d, bm.layer_norm_bwd(dout, want["sum"], want["mean"], want["rstd"], w)))


def test_two_streams_at_once():
    """Calls on two streams have workspaces of their own."""
    g = _gen(42)
    rows, C = 2000, 1024
    ins = [(_randn(g, rows, C, dtype=torch.bfloat16), _randn(g, rows, C, dtype=torch.bfloat16)) for _ in range(2)]
    stats = [bm.layer_norm(x) for x, _ in ins]
    want = [bm.layer_norm_bwd(d, x, s["mean"], s["rstd"]) for (x, d), s in zip(ins, stats)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [bm.layer_norm_bwd(d, x, s["mean"], s["rstd"], stream=q)
               for (x, d), s, q in zip(ins, stats, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("C", [100, 600, 2500])
def test_layer_norm_overflowing_variance(C):
    """Where the variance passes fp32's range rstd is 0, and so is the output
    (plus the bias); lanes past the row's end add nothing to that."""
    x = torch.zeros(3, C, device=DEV)
    x[1, C - 1] = 1e30
    x[2, 0] = -1e30
    b = torch.full((C,), 0.5, device=DEV)
    o = bm.layer_norm(x, None, b)
    assert torch.equal(o["out"], torch.full_like(x, 0.5))
    assert torch.equal(o["rstd"][1:], torch.zeros(2, device=DEV))


# ---- offsets past 32 bits --------------------------------------------------------------------------
# Arrays of more than 2^31 elements: their last rows must come out as they do
# alone (rows, or a filter's width of them, are all that a result depends on).

BIG_ROWS, BIG_C, TAIL = 263000, 8192, 5   # 2.15e9 elements


def test_norms_past_32_bits():
    g = _gen(51)
    x = torch.empty(BIG_ROWS, BIG_C, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    tail = x[-TAIL:].clone()
    o, s = bm.layer_norm(x, checkpoint=True), bm.layer_norm(tail, checkpoint=True)
    assert torch.equal(o["out"][-TAIL:], s["out"]) and torch.equal(o["ckpt"].q[-TAIL:], s["ckpt"].q)
    assert torch.equal(o["ckpt"].scale[-TAIL:], s["ckpt"].scale) and torch.equal(o["rstd"][-TAIL:], s["rstd"])
    back = bm.act8_unpack(o["ckpt"])
    assert torch.equal(back[-TAIL:], bm.act8_unpack(s["ckpt"]))
    del back
    a = bm.act8_pack(x)
    assert torch.equal(a.q[-TAIL:], s["ckpt"].q) and torch.equal(a.scale[-TAIL:], s["ckpt"].scale)
    # x serves as the gradient, too
    dx = bm.layer_norm_bwd(x, a, o["mean"], o["rstd"], dsum=x)[0]
    ds = bm.layer_norm_bwd(tail, s["ckpt"], s["mean"], s["rstd"], dsum=tail)[0]
    assert torch.equal(dx[-TAIL:], ds)
    del dx, o
    w = torch.ones(BIG_C, device=DEV)
    dy, dz, _ = bm.gated_norm_bwd(x, a, a, w)
    ey, ez, _ = bm.gated_norm_bwd(tail, s["ckpt"], s["ckpt"], w)
    assert torch.equal(dy[-TAIL:], ey) and torch.equal(dz[-TAIL:], ez)


def test_convolution_past_32_bits():
    g = _gen(52)
    L, H, P, G, N = 525000, 64, 64, 1, 16
    ch, tail = H * P + 2 * N, 200
    d = dict(xbc=torch.empty(1, L, ch, dtype=torch.bfloat16, device=DEV).normal_(generator=g),
             weight=_randn(g, ch, 4) * 0.5, bias=_randn(g, ch))
    gr = dict(x=torch.empty(1, L, H, P, device=DEV).normal_(generator=g), B=_randn(g, 1, L, G, N),
              C=_randn(g, 1, L, G, N))
    d["xbc"] = bm.act8_pack(d["xbc"])

    def cut(v):
        return v[:, -tail:].contiguous()
    sd = dict(d, xbc=bm.Act8(cut(d["xbc"].q), cut(d["xbc"].scale)))
    sg = {k: cut(v) for k, v in gr.items()}
    for big, small in zip(bm.conv1d_bwd(d, d, gr, gr, H, P, G, N), bm.conv1d_bwd(sd, sd, sg, sg, H, P, G, N)):
        assert torch.equal(big["xbc"][:, -100:], small["xbc"][:, -100:])
    for big, small in zip(bm.conv1d(d, d, H, P, G, N), bm.conv1d(sd, sd, H, P, G, N)):
        for k in ("x", "B", "C"):
            assert torch.equal(big[k][:, -100:], small[k][:, -100:]), k

"""GPU parity of the RMS norm, its gradient, the 8-bit rows and their product
against oracle/rows8.py.

Tolerances. A row's sum has at most 32 serial terms in a lane, 6 levels over
the wave and 8 waves; two such sums and some ten roundings of factors make
less than 128 = 2^7 roundings of 2^-24 each: 2^-17 of S, as for the layer norm.
bf16 results are one rounding more: they must lie between the roundings of
ref - delta and ref + delta. 8-bit rows of given values are exact; rows of a
norm's result are off by half a unit and what the result is off by, in the
unit's own error too: 127 (2^-17 + 2^-17) < 0.002 units. The product is one
conversion (exact below 2^24), two products and one fma: 4 roundings, 2^-22 S.
"""
import numpy as np
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
from metrics import bf16_rne
from oracle import rows8 as orows
from oracle import train as otrain

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
REL, PROD = 2.0 ** -17, 2.0 ** -22


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(name, got, ref, S, rel, dtype="f32"):
    got = _np(got).reshape(ref.shape)
    lo, hi = ref - rel * S, ref + rel * S
    if dtype == "bf16":
        lo, hi = bf16_rne(lo), bf16_rne(hi)
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), (name, np.argwhere(bad)[:3].tolist(), float(np.max(np.abs(got - ref) / (S + 1e-300))))


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


# rows, channels (each way a row is held, and lengths that end inside a vector), dtype
SHAPES = [(1, 8, "bf16"), (3, 9, "f32"), (70, 64, "bf16"), (33, 65, "bf16"), (19, 128, "f32"), (300, 200, "bf16"),
          (5, 256, "f32"), (11, 257, "bf16"), (7, 512, "bf16"), (9, 1000, "f32"), (64, 2560, "bf16"),
          (6, 4099, "bf16"), (4, 8192, "f32"), (3, 16384, "bf16"), (2, 16383, "f32"), (5001, 777, "bf16")]


# ---- 8-bit rows -----------------------------------------------------------------

@pytest.mark.parametrize("rows, C, dtype", SHAPES)
def test_rows8_exact(rows, C, dtype):
    g = _gen(rows + C)
    x = (_randn(g, rows, C) * torch.exp(2 * _randn(g, rows, 1))).to(DT[dtype])
    a = bm.rows8_pack(x)
    q, s = orows.rows8(x)
    assert np.array_equal(a.q.cpu().numpy(), q) and np.array_equal(a.scale.cpu().numpy(), s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows8_extremes(dtype):
    x = torch.zeros(12, 40)
    x[1, 3] = float("inf")
    x[2, 39] = float("nan")
    x[3, :3] = torch.tensor([3.3e38, -3.3e38, 1e38])
    x[4, 0], x[5, 0], x[6, 0] = 2.0 ** -100, 2.0 ** -101, 2.0 ** -149
    x[7, :4] = torch.tensor([127.0, 0.5, 1.5, -2.5])
    x[8, 5] = -float("inf")
    x[9] = -1.0
    x[10, :2] = torch.tensor([2.0 ** -99, -2.0 ** -100])
    x[11, 7] = -0.0
    x = x.to(DT[dtype]).to(DEV)
    a = bm.rows8_pack(x)
    q, s = orows.rows8(x)
    assert np.array_equal(a.q.cpu().numpy(), q)
    assert np.array_equal(a.scale.cpu().numpy(), s, equal_nan=True)


def test_rows8_inside_an_allocation():
    """Arrays at one element's alignment, and what lies around them."""
    g = _gen(5)
    x = _randn(g, 10 * 65 + 3, dtype=torch.bfloat16)[1:651].view(10, 65)
    qb = torch.full((656,), 77, dtype=torch.int8, device=DEV)
    sb = torch.full((14,), 78.0, device=DEV)
    a = bm.Rows8(qb[3:653].view(10, 65), sb[2:12])
    assert bm.rows8_pack(x, out=a) is a
    q, s = orows.rows8(x)
    assert np.array_equal(a.q.cpu().numpy(), q) and np.array_equal(a.scale.cpu().numpy(), s)
    assert (qb[:3] == 77).all() and (qb[653:] == 77).all() and (sb[:2] == 78).all() and (sb[12:] == 78).all()


# ---- the norm -------------------------------------------------------------------

@pytest.mark.parametrize("rows, C, dtype", SHAPES)
@pytest.mark.parametrize("res, w, rows8, dense", [(True, True, True, False), (False, True, False, True),
                                                  (True, False, True, True), (False, False, True, False)])
def test_rms_norm(rows, C, dtype, res, w, rows8, dense):
    g = _gen(rows * 7 + C)
    dt = DT[dtype]
    x, r = _randn(g, rows, C, dtype=dt), _randn(g, rows, C, dtype=dt) * 3
    wt = _randn(g, C) if w else None
    o = bm.rms_norm(x, wt, residual=r if res else None, eps=1e-4, rows8=rows8, dense=dense)
    h = (x.float() + r.float()).to(dt) if res else x
    assert torch.equal(o["sum"], h) and (res or o["sum"] is x)
    ref, rstd = orows.rms_norm(h, wt, 1e-4)
    _close("rstd", o["rstd"], rstd, rstd, REL)
    assert (o["out"] is None) == (not dense) and (o["rows8"] is None) == (not rows8)
    if dense:
        _close("out", o["out"], ref, np.abs(ref), REL, dtype)
    if rows8:
        top = np.abs(ref).max(axis=1)
        _close("scale", o["rows8"].scale, top / 127, top / 127, REL)
        q, s = _np(o["rows8"].q), _np(o["rows8"].scale)[:, None]
        assert np.all(np.abs(q - ref / s) <= 0.502)
        assert np.all(np.abs(q).max(axis=1) == 127)


def test_rms_norm_rows_of_zeros_and_no_number():
    x = torch.ones(6, 300, device=DEV, dtype=torch.bfloat16)
    x[1] = 0
    x[2, 17] = float("nan")
    x[3, 299] = float("inf")
    o = bm.rms_norm(x, rows8=True, dense=True, eps=0.0)
    s, q = o["rows8"].scale, o["rows8"].q
    # a row of zeros without eps is 0 / 0
    assert torch.isnan(s[1:4]).all() and (q[1:4] == 0).all() and torch.isfinite(s[[0, 4, 5]]).all()
    assert torch.isnan(o["out"][1:3]).all() and (q[[0, 4, 5]] == 127).all()
    o = bm.rms_norm(x[1:2], rows8=True)
    assert o["rows8"].scale.item() == 0 and (o["rows8"].q == 0).all() and o["out"] is None


@pytest.mark.parametrize("C", [40, 777, 2560])
def test_rms_norm_in_place(C):
    g = _gen(C)
    x, r, w = _randn(g, 33, C, dtype=torch.bfloat16), _randn(g, 33, C, dtype=torch.bfloat16), _randn(g, C)
    want = bm.rms_norm(x, w, residual=r, rows8=True, dense=True)
    for out, sm in (("x", "r"), ("r", "x"), (None, "r"), ("x", None)):
        t = dict(x=x.clone(), r=r.clone())
        got = bm.rms_norm(t["x"], w, residual=t["r"], rows8=True, dense=True, out=t.get(out), sum_out=t.get(sm))
        for k in ("out", "sum", "rstd"):
            assert torch.equal(got[k], want[k]), (out, sm, k)
        assert torch.equal(got["rows8"].q, want["rows8"].q)


@pytest.mark.parametrize("rows, C, dtype", SHAPES)
@pytest.mark.parametrize("ckpt, dsum, w", [(False, True, True), (True, False, True), (True, True, False)])
def test_rms_norm_bwd(rows, C, dtype, ckpt, dsum, w):
    g = _gen(rows + 3 * C)
    dt = DT[dtype]
    x, do = _randn(g, rows, C, dtype=dt), _randn(g, rows, C, dtype=dt)
    ds = _randn(g, rows, C, dtype=dt) if dsum else None
    wt = _randn(g, C) if w else None
    rstd = bm.rms_norm(x, wt)["rstd"]
    kept = bm.act8_pack(x) if ckpt else x
    dx, dw = bm.rms_norm_bwd(do, kept, rstd, wt, dsum=ds)
    h = otrain.act8_values(kept.q.cpu().numpy(), kept.scale.cpu().numpy()) if ckpt else x
    (rx, Sx), (rw, Sw) = orows.rms_norm_bwd(do, h, rstd, wt, ds)
    _close("dx", dx, rx, Sx, REL, dtype)
    # a workgroup's rows are added in a lane: at most 5001 / 4 of them in a row
    _close("dw", dw, rw, Sw, REL + (rows / 4) * 2.0 ** -24)
    dx2, none = bm.rms_norm_bwd(do, kept, rstd, wt, dsum=ds, wgrad=False)
    assert none is None and torch.equal(dx, dx2)
    if not ckpt:
        for t in (do.clone(), ds.clone() if dsum else do.clone(), x.clone()):
            src = dict(dout=do, x=x, dsum=ds)
            for k in src:
                if src[k] is not None and torch.equal(src[k], t):
                    src[k] = t
            got, gw = bm.rms_norm_bwd(src["dout"], src["x"], rstd, wt, dsum=src["dsum"], dx=t)
            assert got is t and torch.equal(got, dx) and torch.equal(gw, dw)


def test_rms_norm_gradient_by_differences():
    """Along random directions, against differences of the forward in 64 bits."""
    g = _gen(3)
    x, w, do = _randn(g, 7, 100), _randn(g, 100), _randn(g, 7, 100)
    dx, dw = bm.rms_norm_bwd(do, x, bm.rms_norm(x, w, eps=1e-3)["rstd"], w)
    xn, wn, dn = _np(x), _np(w), _np(do)

    def loss(a, b):
        return float((orows.rms_norm(a, b, 1e-3)[0] * dn).sum())
    r = np.random.default_rng(1)
    for _ in range(5):
        u, v, h = r.normal(size=xn.shape), r.normal(size=wn.shape), 1e-5
        num = (loss(xn + h * u, wn + h * v) - loss(xn - h * u, wn - h * v)) / (2 * h)
        assert abs(num - (_np(dx) * u).sum() - (_np(dw) * v).sum()) <= 1e-4 * (np.abs(_np(dx) * u).sum() + np.abs(_np(dw) * v).sum())


def test_no_rows():
    x = torch.empty(0, 3, 64, dtype=torch.bfloat16, device=DEV)
    o = bm.rms_norm(x, residual=x, rows8=True, dense=True)
    assert o["out"].shape == x.shape and o["rows8"].q.shape == x.shape and o["rstd"].shape == (0, 3)
    assert bm.rows8_pack(x).scale.shape == (0, 3)
    dx, dw = bm.rms_norm_bwd(x, x, o["rstd"])
    assert dx.shape == x.shape and (dw == 0).all()
    assert bm.linear8(o["rows8"], bm.rows8_pack(torch.ones(5, 64, device=DEV))).shape == (0, 3, 5)


# ---- the product ----------------------------------------------------------------

def _int8(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, device=DEV).to(torch.int8)


# rows, cin, cout: every tile, ends inside tiles and steps, lengths that are no multiple of 16
PRODUCTS = [(1, 16, 16), (1, 1, 1), (3, 5, 2), (16, 64, 48), (17, 80, 33), (33, 2064, 17), (64, 4096, 2048),
            (64, 100, 130), (65, 128, 64), (100, 1000, 70), (128, 144, 257), (300, 272, 515), (129, 4112, 129),
            (513, 777, 640), (2100, 1023, 2100), (2050, 256, 2200), (5000, 384, 4100), (4099, 400, 4100)]


@pytest.mark.parametrize("rows, cin, cout", PRODUCTS)
@pytest.mark.parametrize("dtype, bias", [("bf16", False), ("f32", True)])
def test_linear8(rows, cin, cout, dtype, bias):
    g = _gen(rows + cin + cout)
    x = bm.Rows8(_int8(g, rows, cin), torch.rand(rows, generator=g, device=DEV))
    w = bm.Rows8(_int8(g, cout, cin), torch.rand(cout, generator=g, device=DEV))
    b = _randn(g, cout) * 100 if bias else None
    buf = torch.full((rows * cout + 8,), 5.0, dtype=DT[dtype], device=DEV)
    out = bm.linear8(x, w, b, out=buf[4:-4].view(rows, cout))
    torch.cuda.synchronize()
    assert (buf[:4] == 5).all() and (buf[-4:] == 5).all()
    ref, S = orows.linear8(x.q.double().cpu().numpy(), x.scale, w.q.double().cpu().numpy(), w.scale, b) \
        if rows * cin * cout < 1e8 else _fast(x, w, b)
    _close("out", out, ref, S, PROD, dtype)


def _fast(x, w, b):
    """The same in torch's fp64 (whole numbers: exact)."""
    v = (x.q.double() @ w.q.double().t()) * x.scale.double()[:, None] * w.scale.double()
    bb = b.double() if b is not None else torch.zeros_like(w.scale.double())
    return _np(v + bb), _np(v.abs() + bb.abs())


def test_linear8_largest_sums():
    """The longest rows of the most negative number: sums of 2^31 - 2^14, above
    what a float holds exactly."""
    n = 131071
    x = bm.Rows8(torch.full((3, n), -128, dtype=torch.int8, device=DEV), torch.ones(3, device=DEV))
    w = bm.Rows8(torch.full((20, n), -128, dtype=torch.int8, device=DEV), torch.ones(20, device=DEV))
    assert (bm.linear8(x, w, dtype=torch.float32).double() == float(np.float32(128 * 128 * n))).all()
    n = 131056   # a multiple of 16: the other path
    x = bm.Rows8(x.q[:, :n].contiguous(), x.scale)
    w = bm.Rows8(w.q[:, :n].contiguous(), w.scale)
    assert (bm.linear8(x, w, dtype=torch.float32).double() == float(np.float32(128 * 128 * n))).all()


@pytest.mark.parametrize("off", [0, 1, 3, 8])
def test_linear8_unaligned(off):
    """Operands that start at any byte."""
    g = _gen(off)
    xb, wb = _int8(g, 40 * 64 + 16), _int8(g, 90 * 64 + 16)
    x = bm.Rows8(xb[off:off + 2560].view(40, 64), torch.rand(40, generator=g, device=DEV))
    w = bm.Rows8(wb[off:off + 5760].view(90, 64), torch.rand(90, generator=g, device=DEV))
    ref, S = _fast(x, w, None)
    _close("out", bm.linear8(x, w), ref, S, PROD, "bf16")


def test_linear8_of_rows_without_a_number():
    """A row whose scale is NaN gives NaNs in its own row of out alone."""
    x = torch.ones(70, 64, device=DEV)
    x[3, 3] = float("inf")
    o = bm.linear8(bm.rows8_pack(x), bm.rows8_pack(torch.ones(9, 64, device=DEV)), dtype=torch.float32)
    assert torch.isnan(o[3]).all() and torch.isfinite(o[:3]).all() and torch.isfinite(o[4:]).all()


# ---- together, captured, on streams ------------------------------------------------

def _serve(x, r, w, wi, wo):
    n = bm.rms_norm(x, w, residual=r, rows8=True)
    h = bm.linear8(n["rows8"], wi)
    return bm.linear8(bm.rows8_pack(h), wo, dtype=torch.float32), n["sum"]


def test_norm_to_product_graph_and_streams():
    """A norm, a projection from it and one back: against the values that the
    8-bit rows stand for, captured and replayed, and on another stream."""
    g = _gen(9)
    x, r, w = _randn(g, 2, 50, 512, dtype=torch.bfloat16), _randn(g, 2, 50, 512, dtype=torch.bfloat16), _randn(g, 512)
    wi, wo = bm.rows8_pack(_randn(g, 1100, 512)), bm.rows8_pack(_randn(g, 512, 1100))
    out, sm = _serve(x, r, w, wi, wo)
    n = bm.rms_norm(x, w, residual=r, rows8=True)["rows8"]
    h = ((n.q.double() * n.scale.double()[..., None]) @ (wi.q.double() * wi.scale.double()[:, None]).t()).to(torch.bfloat16)
    h8 = bm.rows8_pack(h)
    ref = (h8.q.double() * h8.scale.double()[..., None]) @ (wo.q.double() * wo.scale.double()[:, None]).t()
    # h may round to the other bf16 where it lies at a tie (2^-22 of it): one
    # unit of 2^-8 in few of 1100 elements
    assert ((out.double() - ref).norm() / ref.norm()).item() < 2.0 ** -10
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _serve(x, r, w, wi, wo)
    torch.cuda.current_stream().wait_stream(side)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        go, gs = _serve(x, r, w, wi, wo)
    for i in range(4):
        x.copy_(_randn(_gen(100 + i), 2, 50, 512, dtype=torch.bfloat16))
        gr.replay()
        torch.cuda.synchronize()
        eo, es = _serve(x, r, w, wi, wo)
        assert torch.equal(go, eo) and torch.equal(gs, es)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = bm.rms_norm(x, w, residual=r, rows8=True, stream=s)
    b = bm.linear8(a["rows8"], wi, stream=s)
    c = bm.rows8_pack(b, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(bm.linear8(c, wo, dtype=torch.float32), eo)

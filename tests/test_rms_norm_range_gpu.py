"""RMS norm of rows whose squares, or their sum, leave fp32's range while the norm
does not. Against oracle/rows8.py; tolerances as in test_rows8_gpu.py (scaling a
row by a power of two rounds nothing), and half a step of fp32's subnormals,
2^-150, where rstd lies among them."""
import numpy as np
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
from oracle import rows8 as orows
from test_rows8_gpu import DT, REL, _close, _gen, _np, _randn

pytestmark = pytest.mark.gpu

DEV = "cuda"
# each way a row is held, and lengths that end inside a vector
WIDTHS = [8, 9, 64, 65, 128, 200, 257, 512, 1000, 2560, 4099, 16384]
# a row's size (powers of two), in turn with ordinary rows: squares beyond fp32;
# squares inside, their sum not; squares among the subnormals; squares that are zero
SIZES = [0, 123, 0, 64, 63, 61, 0, -62, -70, -90, 0, 100, -110, 0]


def _rows(g, C, dtype, n=70):
    k = torch.tensor([SIZES[i % len(SIZES)] for i in range(n)], device=DEV, dtype=torch.float64)
    x = _randn(g, n, C).double().clamp(-4, 4) * torch.exp2(k)[:, None]
    return x.to(DT[dtype]), k


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("res, rows8, dense", [(False, False, True), (True, True, False), (False, True, True)])
@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-5])
def test_rms_norm_of_any_size(C, dtype, res, rows8, dense, eps):
    g = _gen(C + 5)
    x, k = _rows(g, C, dtype)
    w = _randn(g, C)
    o = bm.rms_norm(x, w, residual=x if res else None, eps=eps, rows8=rows8, dense=dense)
    h = o["sum"]
    assert torch.isfinite(h).all()
    # the call takes eps as a float: 1e-42 is 714 x 2^-149, 5.3e-4 more
    ref, rstd = orows.rms_norm(h, w, float(np.float32(eps)))
    _close("rstd", o["rstd"], rstd, rstd + 2.0 ** -150 / REL, REL)
    if dense:
        _close("out", o["out"], ref, np.abs(ref) + 2.0 ** -133 / REL, REL, dtype)
    if rows8:
        top = np.abs(ref).max(axis=1)
        live = top > 2.0 ** -99
        q, s = _np(o["rows8"].q), _np(o["rows8"].scale)
        _close("scale", o["rows8"].scale[torch.tensor(live, device=DEV)], top[live] / 127, top[live] / 127, REL)
        assert np.all(np.abs(q[live] - ref[live] / s[live, None]) <= 0.502) and np.all(np.abs(q[live]).max(axis=1) == 127)
        assert (q[top < 2.0 ** -101] == 0).all() and (s[top < 2.0 ** -101] == 0).all()
    # a row is what it is beside any others
    plain = np.flatnonzero(_np(k) == 0)
    alone = bm.rms_norm(x[plain], w, residual=x[plain] if res else None, eps=eps, rows8=rows8, dense=dense)
    assert torch.equal(alone["rstd"], o["rstd"][plain])
    assert not dense or torch.equal(alone["out"], o["out"][plain])
    assert not rows8 or torch.equal(alone["rows8"].q, o["rows8"].q[plain])


@pytest.mark.parametrize("C", [65, 1000, 4099])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_of_large_rows(C, dtype):
    """The gradient takes such a row's rstd as any other's."""
    g = _gen(C)
    x, _ = _rows(g, C, dtype)
    x = x[[1, 3, 4, 5, 7, 11]].contiguous()
    w, do = _randn(g, C), _randn(g, *x.shape, dtype=DT[dtype])
    rstd = bm.rms_norm(x, w)["rstd"]
    dx, dw = bm.rms_norm_bwd(do, x, rstd, w)
    (rx, Sx), (rw, Sw) = orows.rms_norm_bwd(do, x, rstd, w, None)
    _close("dx", dx, rx, Sx + (2.0 ** -133 if dtype == "bf16" else 2.0 ** -148) / REL, REL, dtype)
    _close("dw", dw, rw, Sw, REL + x.shape[0] * 2.0 ** -24)


@pytest.mark.parametrize("C", [40, 777, 2560])
def test_infinities_and_nan_stay_what_they_were(C):
    x = torch.ones(6, C, device=DEV) * 1e25
    x[1, 3], x[2, C - 1], x[3, 7] = float("inf"), float("nan"), -float("inf")
    o = bm.rms_norm(x, rows8=True, dense=True)
    s, q = o["rows8"].scale, o["rows8"].q
    assert torch.isnan(s[1:4]).all() and (q[1:4] == 0).all() and (q[[0, 4, 5]] == 127).all()
    assert (o["rstd"][[1, 3]] == 0).all() and torch.isnan(o["rstd"][2])
    assert torch.isnan(o["out"][1, 3]) and torch.isnan(o["out"][2]).all() and (o["out"][0] == 1).all()


@pytest.mark.parametrize("C, rows", [(64, 70000), (300, 17000), (1500, 6300), (9000, 4200)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_turns(C, rows, dtype):
    """Such rows in a workgroup's several turns, one after the other and between
    ordinary ones: what each is in a short batch."""
    g = _gen(rows)
    k = torch.randint(0, 3, (rows, 1), generator=g, device=DEV)
    x = _randn(g, rows, C) * torch.tensor([1.0, 1e25, 1e-25], device=DEV)[k]
    x, w = x.to(DT[dtype]), _randn(g, C)
    o = bm.rms_norm(x, w, eps=0.0, rows8=True, dense=True)
    for a in range(0, rows, 1500):
        b = bm.rms_norm(x[a:a + 1500], w, eps=0.0, rows8=True, dense=True)
        for n in ("out", "rstd"):
            assert torch.equal(o[n][a:a + 1500], b[n]), (a, n)
        assert torch.equal(o["rows8"].q[a:a + 1500], b["rows8"].q)
        assert torch.equal(o["rows8"].scale[a:a + 1500], b["rows8"].scale)
    _, rstd = orows.rms_norm(x[-500:], w, 0.0)
    _close("rstd", o["rstd"][-500:], rstd, rstd, REL)

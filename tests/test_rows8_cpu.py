"""Pins of the oracle of the 8-bit rows, the RMS norm and the integer product
(oracle/rows8.py), and these entry points' refusals; all on the CPU: every
rejected call is refused before any HIP call."""
import ctypes
import os

import numpy as np
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
from bidirectional_mamba_ssm_amd import _abi
from oracle import rows8 as orows

STEP = 1 << 24   # further apart than any array here is long


# ---- the oracle ---------------------------------------------------------------

def test_rms_norm_pins():
    r = np.random.default_rng(1)
    h, w, g, ds = (torch.tensor(r.normal(size=s)) for s in ((5, 33), (33,), (5, 33), (5, 33)))
    h.requires_grad_(), w.requires_grad_()
    out = torch.nn.functional.rms_norm(h, (33,), w, 1e-3)
    ((out * g).sum() + (h * ds).sum()).backward()
    got, rstd = orows.rms_norm(h, w, 1e-3)
    assert np.allclose(got, out.detach().numpy(), rtol=1e-12, atol=1e-14)
    for (v, S), want in zip(orows.rms_norm_bwd(g, h, rstd, w, ds), (h.grad, w.grad)):
        assert np.allclose(v, want.numpy(), rtol=1e-10, atol=1e-12)
        assert np.all(S >= np.abs(v) - 1e-12)


def test_rows8_pins():
    x = np.array([[127.0, -63.5, 0.5, 1.5, -0.25], [0, 0, 0, 0, 0], [2.0 ** -101, 0, 0, 0, 0],
                  [1, np.inf, 0, 0, 0], [np.nan, 1, 0, 0, 0], [-3e38, 3e38, 1e38, 0, 1]])
    q, s = orows.rows8(x)
    assert q.tolist()[:5] == [[127, -64, 0, 2, 0]] + [[0] * 5] * 4 and q[5].tolist() == [-127, 127, 42, 0, 0]
    assert s[0] == 1.0 and s[1] == 0 and s[2] == 0 and np.isnan(s[3]) and np.isnan(s[4])
    r = np.random.default_rng(2).normal(size=(50, 40)).astype(np.float32)
    q, s = orows.rows8(r)
    assert np.all(np.abs(q * s[:, None].astype(np.float64) - r) <= 0.50001 * s[:, None])
    assert np.all(np.abs(q).max(axis=1) == 127)


def test_linear8_pins():
    r = np.random.default_rng(3)
    xq, wq = r.integers(-127, 128, (3, 17)), r.integers(-127, 128, (4, 17))
    xs, ws, b = r.random(3), r.random(4), r.normal(size=4)
    got, S = orows.linear8(xq, xs, wq, ws, b)
    for i in range(3):
        for j in range(4):
            v = sum(int(xq[i, c]) * int(wq[j, c]) for c in range(17)) * xs[i] * ws[j]
            assert abs(got[i, j] - v - b[j]) <= 1e-12 * S[i, j] and S[i, j] >= abs(got[i, j]) - 1e-12


# ---- refusals -----------------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_abi.LIB_PATH):
        from bidirectional_mamba_ssm_amd import build
        build.build()
    return _abi.load()


def _places(*names):
    return {n: STEP * (i + 1) for i, n in enumerate(names)}


def _rows8(q, s):
    return ctypes.byref(_abi.Rows8Ptrs(q, s))


def _code(lib, rc, code, word=""):
    assert rc == code, (rc, lib.bimamba_last_error())
    assert word in lib.bimamba_last_error().decode(), lib.bimamba_last_error()


ROWS, C = 8, 64


def _norm(lib, at, rows=ROWS, C=C, dtype=_abi.BF16, eps=1e-5):
    o8 = _rows8(at["q"], at["scale"]) if "q" in at else None
    return lib.bimamba_rms_norm(rows, C, dtype, at["x"], at["res"], at["w"], eps, at["out"], at["sum"], at["rstd"], o8,
                                None)


NORM = ("x", "res", "w", "out", "sum", "rstd", "q", "scale")


@pytest.mark.parametrize("kw, code", [
    (dict(rows=-1), _abi.EINVAL), (dict(rows=2 ** 31), _abi.EUNSUPPORTED), (dict(C=7), _abi.EUNSUPPORTED),
    (dict(C=16385), _abi.EUNSUPPORTED), (dict(dtype=2), _abi.EINVAL), (dict(eps=-1.0), _abi.EINVAL),
    (dict(eps=float("nan")), _abi.EINVAL), (dict(eps=float("inf")), _abi.EINVAL)])
def test_rms_norm_arguments(lib, kw, code):
    _code(lib, _norm(lib, _places(*NORM), **kw), code)


@pytest.mark.parametrize("change, word", [
    (dict(x=None), "x is required"), (dict(sum=None), "residual and sum"), (dict(res=None), "residual and sum"),
    (dict(scale=None), "q and scale"), (dict(x=STEP + 1), "aligned"), (dict(w=STEP * 3 + 2), "aligned"),
    (dict(scale=STEP * 9 + 2), "aligned"), (dict(rstd=STEP * 9 + 1), "aligned")])
def test_rms_norm_pointers(lib, change, word):
    at = _places(*NORM)
    at.update(change)
    _code(lib, _norm(lib, at), _abi.EINVAL, word)


def test_rms_norm_no_output(lib):
    at = _places(*NORM[:-2])
    at["out"] = None
    _code(lib, _norm(lib, at), _abi.EINVAL, "out8")


@pytest.mark.parametrize("out", ["out", "sum", "rstd", "q", "scale"])
@pytest.mark.parametrize("other", ["x", "res", "w", "out", "sum", "rstd", "q", "scale"])
def test_rms_norm_overlaps(lib, out, other):
    if out == other:
        return
    for shift in (0, 4, -4):
        if shift == 0 and out in ("out", "sum") and other in ("x", "res"):
            continue   # in place
        at = _places(*NORM)
        at[out] = at[other] + shift
        _code(lib, _norm(lib, at), _abi.EINVAL, "overlaps")


def _norm_bwd(lib, at, q8=False, rows=ROWS, ws=1 << 20, dtype=_abi.BF16):
    return lib.bimamba_rms_norm_bwd(rows, C, dtype, at["x"], at["scale"] if q8 else None, at["rstd"], at["w"],
                                    at["dout"], at["dsum"], at["dx"], at["dw"], at["ws"], ws, None)


BWD = ("x", "scale", "rstd", "w", "dout", "dsum", "dx", "dw", "ws")


@pytest.mark.parametrize("change, code", [
    (dict(x=None), _abi.EINVAL), (dict(rstd=None), _abi.EINVAL), (dict(dout=None), _abi.EINVAL),
    (dict(dx=None), _abi.EINVAL), (dict(ws=None), _abi.EWORKSPACE), (dict(ws=STEP * 9 + 16), _abi.EINVAL),
    (dict(dx=STEP + 1), _abi.EINVAL), (dict(rstd=STEP * 3 + 1), _abi.EINVAL), (dict(dw=STEP * 8 + 2), _abi.EINVAL)])
def test_rms_norm_bwd_pointers(lib, change, code):
    at = _places(*BWD)
    at.update(change)
    _code(lib, _norm_bwd(lib, at), code)


def test_rms_norm_bwd_workspace(lib):
    n = ctypes.c_size_t(0)
    assert lib.bimamba_rms_norm_bwd_workspace_size(ROWS, C, 1, ctypes.byref(n)) == 0 and n.value > 0
    _code(lib, _norm_bwd(lib, _places(*BWD), ws=n.value - 1), _abi.EWORKSPACE)
    assert lib.bimamba_rms_norm_bwd_workspace_size(ROWS, C, 1, None) == _abi.EINVAL
    assert lib.bimamba_rms_norm_bwd_workspace_size(ROWS, 4, 1, ctypes.byref(n)) == _abi.EUNSUPPORTED


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("out", ["dx", "dw", "ws"])
def test_rms_norm_bwd_overlaps(lib, out, q8):
    for other in BWD:
        if other == out or (other == "scale" and not q8):
            continue
        # dx may be dout, dsum or the array x
        for shift in ([256] if out == "dx" and other in ("dout", "dsum", "x") and not (other == "x" and q8) else [0]):
            at = _places(*BWD)
            at[out] = at[other] + shift
            _code(lib, _norm_bwd(lib, at, q8), _abi.EINVAL, "overlaps")


def test_rows8_pack_refusals(lib):
    def call(x=STEP, q=2 * STEP, s=3 * STEP, rows=ROWS, c=C, dtype=1):
        return lib.bimamba_rows8_pack(rows, c, dtype, x, _rows8(q, s), None)
    for kw in (dict(x=None), dict(q=None), dict(s=None), dict(x=STEP + 1), dict(s=3 * STEP + 2), dict(dtype=7),
               dict(rows=-1), dict(q=STEP), dict(s=STEP + 4), dict(s=2 * STEP)):
        _code(lib, call(**kw), _abi.EINVAL)
    for kw in (dict(c=4), dict(c=20000), dict(rows=2 ** 31)):
        _code(lib, call(**kw), _abi.EUNSUPPORTED)
    _code(lib, lib.bimamba_rows8_pack(ROWS, C, 1, STEP, None, None), _abi.EINVAL)


def test_linear8_refusals(lib):
    def call(xq=STEP, xs=2 * STEP, wq=3 * STEP, ws=4 * STEP, b=5 * STEP, o=6 * STEP, rows=ROWS, ci=C, co=32, dtype=1):
        return lib.bimamba_linear8(rows, ci, co, dtype, _rows8(xq, xs), _rows8(wq, ws), b, o, None)
    for kw in (dict(xq=None), dict(xs=None), dict(wq=None), dict(ws=None), dict(o=None), dict(xs=2 * STEP + 1),
               dict(ws=4 * STEP + 2), dict(b=5 * STEP + 2), dict(o=6 * STEP + 1), dict(dtype=-1), dict(rows=-1),
               dict(o=STEP + 2), dict(o=2 * STEP), dict(o=3 * STEP - 2), dict(o=4 * STEP), dict(o=5 * STEP)):
        _code(lib, call(**kw), _abi.EINVAL)
    for kw in (dict(ci=0), dict(ci=131072), dict(co=0), dict(co=2 ** 24 + 1), dict(rows=2 ** 31),
               dict(rows=2 ** 31 - 1, co=2 ** 20)):
        _code(lib, call(**kw), _abi.EUNSUPPORTED)
    _code(lib, lib.bimamba_linear8(ROWS, C, 32, 1, None, _rows8(1, 1), None, STEP, None), _abi.EINVAL)
    # nothing to do
    assert lib.bimamba_linear8(0, C, 32, 1, _rows8(None, None), _rows8(None, None), None, None, None) == 0


def test_binding_refusals():
    x = torch.zeros(4, 16)
    for call in (lambda: bm.rows8_pack(x), lambda: bm.rms_norm(x), lambda: bm.rms_norm_bwd(x, x, x[:, 0]),
                 lambda: bm.linear8(bm.Rows8(x, x), bm.Rows8(x, x))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError, match="Rows8"):
        bm.linear8(x, x)

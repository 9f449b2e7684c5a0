"""Pins of the gated delta rule's oracle (oracle/delta.py), and its entry
points' refusals; all on the CPU: every rejected call is refused before any
HIP call."""
import ctypes
import os

import numpy as np
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
from bidirectional_mamba_ssm_amd import _abi
from delta_inputs import direction
from oracle import delta as od

STEP = 1 << 26


# ---- the oracle ---------------------------------------------------------------

def _dirs(seed, n, *a, **kw):
    g = torch.Generator().manual_seed(seed)
    return [direction(g, *a, **kw) for _ in range(n)], g


def test_first_tokens_by_hand():
    """Keys along the axes: the second token reads and corrects the first's entry."""
    one = lambda *v: torch.tensor(v, dtype=torch.float64).reshape(1, -1, 1)
    k = torch.zeros(1, 3, 1, 2, dtype=torch.float64)
    k[0, 0, 0, 0] = k[0, 1, 0, 0] = k[0, 2, 0, 1] = 1.0
    d = dict(q=k.clone(), k=k, v=one(2.0, 5.0, 7.0).unsqueeze(-1), g=one(0.0, np.log(0.5), 0.0), beta=one(0.5, 1.0, 0.25))
    y, last = od.fwd([d], 1.0)
    # S = [1, 0]; decays to 0.5, its error is 4.5, written whole: 5; then 7 / 4 at the other key
    assert np.allclose(y.ravel(), [1.0, 5.0, 1.75], atol=1e-15) and np.allclose(last.ravel(), [5.0, 1.75], atol=1e-15)


def _torch(d, init, scale, reverse, spans):
    """The definition as a plain torch recurrence."""
    H, G = d["v"].shape[2], d["k"].shape[2]
    q, k = (d[n].repeat_interleave(H // G, dim=2) for n in ("q", "k"))
    y, last = torch.zeros_like(d["v"]), []
    for u, (b, lo, hi) in enumerate(spans):
        S = init[u].transpose(1, 2) if init is not None else torch.zeros(H, k.shape[3], d["v"].shape[3], dtype=y.dtype)
        for t in (range(hi - 1, lo - 1, -1) if reverse else range(lo, hi)):
            S = torch.exp(d["g"][b, t])[:, None, None] * S
            e = d["v"][b, t] - torch.einsum("hnp,hn->hp", S, k[b, t])
            S = S + torch.einsum("hn,hp->hnp", k[b, t], d["beta"][b, t][:, None] * e)
            out = torch.zeros_like(y)
            out[b, t] = scale * torch.einsum("hnp,hn->hp", S, q[b, t])
            y = y + out
        last.append(S.transpose(1, 2))
    return y, torch.stack(last)


@pytest.mark.parametrize("cu", [None, [0, 4, 4, 5, 11]])
def test_against_autograd(cu):
    batch, L, H, P, G, N = (2, 7, 4, 3, 2, 5) if cu is None else (1, 11, 4, 3, 2, 5)
    dirs, g = _dirs(1, 2, batch, L, H, P, G, N, "f32")
    dirs = [{n: t.double().requires_grad_() for n, t in d.items()} for d in dirs]
    spans = od._units(batch, L, cu)
    init = torch.randn(len(spans), H, P, N, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(batch, L, H, P, generator=g, dtype=torch.float64)
    df = torch.randn(len(spans), H, P, N, generator=g, dtype=torch.float64)
    yf, last = _torch(dirs[0], init, 0.7, False, spans)
    yb, _ = _torch(dirs[1], None, 0.7, True, spans)
    y, mine = od.fwd(dirs, 0.7, cu, init)
    assert np.allclose(y, (yf + yb).detach().numpy(), atol=1e-13) and np.allclose(mine, last.detach().numpy(), atol=1e-13)
    ((yf + yb) * dy).sum().add((last * df).sum()).backward()
    grads, dinit = od.bwd(dirs, dy, 0.7, cu, init, df)
    for d, got in zip(dirs, grads):
        for n in od.KEYS:
            assert np.allclose(got[n], d[n].grad.numpy(), rtol=1e-9, atol=1e-12), n
        assert np.all(got["gS"] >= np.abs(got["g"]))
    assert np.allclose(dinit, init.grad.numpy(), rtol=1e-9, atol=1e-12)


def test_differences():
    dirs, g = _dirs(2, 1, 1, 9, 2, 4, 1, 3, "f32")
    d = {n: t.double() for n, t in dirs[0].items()}
    dy = torch.randn(1, 9, 2, 4, generator=g, dtype=torch.float64)
    grads, _ = od.bwd([d], dy, 0.5)
    r = np.random.default_rng(0)
    for n in od.KEYS:
        u = torch.tensor(r.normal(size=tuple(d[n].shape)))
        up, dn = (float((od.fwd([dict(d, **{n: d[n] + h * u})], 0.5)[0] * dy.numpy()).sum()) for h in (1e-6, -1e-6))
        assert abs((up - dn) / 2e-6 - float((grads[0][n] * u.numpy()).sum())) < 1e-7, n


def test_blocks_packing_and_reversal():
    dirs, g = _dirs(3, 1, 1, 20, 2, 4, 1, 3, "f32")
    d = dirs[0]
    y, last = od.fwd([d], 1.0)
    cut = {n: t[:, :13] for n, t in d.items()}, {n: t[:, 13:] for n, t in d.items()}
    ya, mid = od.fwd([cut[0]], 1.0)
    yb, end = od.fwd([cut[1]], 1.0, init=torch.tensor(mid))
    assert np.array_equal(np.concatenate([ya, yb], axis=1), y) and np.array_equal(end, last)
    yp, lp = od.fwd([d], 1.0, cu=[0, 13, 13, 20])
    y2, l2 = od.fwd([cut[1]], 1.0)
    assert np.array_equal(yp[:, :13], ya) and np.array_equal(yp[:, 13:], y2)
    assert np.array_equal(lp[0], mid[0]) and (lp[1] == 0).all() and np.array_equal(lp[2], l2[0])
    zero = {n: torch.zeros_like(t) for n, t in d.items()}
    back, _ = od.fwd([zero, {n: t.flip(1) for n, t in d.items()}], 1.0)
    assert np.array_equal(back[:, ::-1], y)


# ---- refusals -----------------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_abi.LIB_PATH):
        from bidirectional_mamba_ssm_amd import build
        build.build()
    return _abi.load()


SHAPE = dict(batch=2, seqlen=100, nheads=4, headdim=40, d_state=32, ngroups=2, chunk=64, dtype=1, flags=0)
NAMES = ["fq", "fk", "fv", "fg", "fb", "rq", "rk", "rv", "rg", "rb", "init", "final", "y", "ws"]
GRADS = [r + "d" + n for r in "fr" for n in ("q", "k", "v", "g", "b")]


def _shape(**kw):
    return ctypes.byref(_abi.Shape(*dict(SHAPE, **kw).values()))


def _places(names):
    return {n: STEP * (i + 1) for i, n in enumerate(names)}


def _dir(at, r):
    return ctypes.byref(_abi.DeltaDir(*(at[r + n] for n in "qkvgb")))


def _cu(cu):
    return (ctypes.c_int32 * len(cu))(*cu) if cu is not None else None


def _fwd(lib, at, shape=None, both=True, scale=1.0, cu=None, nseq=None, ws=1 << 30):
    nseq = nseq if nseq is not None else len(cu) - 1 if cu is not None else 0
    return lib.bimamba_delta_fwd(shape or _shape(), _dir(at, "f"), _dir(at, "r") if both else None, scale, _cu(cu), nseq,
                                 at["init"], at["final"], at["y"], at["ws"], ws, None)


def _code(lib, rc, code, word=""):
    assert rc == code, (rc, lib.bimamba_last_error())
    assert word in lib.bimamba_last_error().decode(), lib.bimamba_last_error()


BAD_SHAPES = [
    (dict(batch=0), _abi.EINVAL), (dict(seqlen=-1), _abi.EINVAL), (dict(ngroups=3), _abi.EINVAL),
    (dict(headdim=129), _abi.EUNSUPPORTED), (dict(d_state=48), _abi.EUNSUPPORTED), (dict(d_state=256), _abi.EUNSUPPORTED),
    (dict(chunk=128), _abi.EUNSUPPORTED), (dict(chunk=1), _abi.EUNSUPPORTED), (dict(flags=1), _abi.EINVAL),
    (dict(dtype=5), _abi.EINVAL), (dict(batch=1 << 20, nheads=64, headdim=16, seqlen=1), _abi.EUNSUPPORTED),
    (dict(batch=1, nheads=32770, headdim=16, seqlen=1), _abi.EUNSUPPORTED),
    (dict(batch=1 << 22, nheads=2, seqlen=4, headdim=16, ngroups=2), _abi.EUNSUPPORTED),
    (dict(batch=1 << 16, seqlen=1 << 16), _abi.EUNSUPPORTED)]


@pytest.mark.parametrize("kw, code", BAD_SHAPES)
def test_shapes(lib, kw, code):
    at = _places(NAMES + GRADS)
    _code(lib, _fwd(lib, at, _shape(**kw)), code)
    _code(lib, _bwd(lib, at, _shape(**kw)), code)
    n = ctypes.c_size_t(0)
    for query, both in ((lib.bimamba_delta_workspace_size, (1,)), (lib.bimamba_delta_bwd_workspace_size, ())):
        _code(lib, query(_shape(**kw), *both, 0, ctypes.byref(n)), code)
    rc = lib.bimamba_delta_step(_shape(**kw), STEP * 40, _dir(at, "f"), None, 1.0, 1, at["y"], None, 0, None)
    _code(lib, rc, code if kw.get("seqlen", 0) <= 256 else _abi.EINVAL)


def test_queries(lib):
    n = ctypes.c_size_t(0)
    for query, both in ((lib.bimamba_delta_workspace_size, (1,)), (lib.bimamba_delta_bwd_workspace_size, ())):
        assert query(_shape(), *both, 0, ctypes.byref(n)) == 0
        assert query(_shape(), *both, 0, None) == _abi.EINVAL
        assert query(_shape(), *both, -1, ctypes.byref(n)) == _abi.EINVAL
        assert query(None, *both, 0, ctypes.byref(n)) == _abi.EINVAL


@pytest.mark.parametrize("name", ["fq", "fk", "fv", "fg", "fb", "rq", "rv", "rb", "y"])
def test_fwd_missing_and_unaligned(lib, name):
    at = _places(NAMES)
    at[name] = None
    _code(lib, _fwd(lib, at), _abi.EINVAL)
    at = _places(NAMES)
    at[name] += 2 if name[1:] in ("g", "b") else 8
    _code(lib, _fwd(lib, at), _abi.EINVAL, "aligned")


@pytest.mark.parametrize("cu, nseq", [([0, 50, 40, 100], 3), ([0, 99], 1), ([1, 100], 1), ([0, 101], 1), (None, 2)])
def test_offsets(lib, cu, nseq):
    _code(lib, _fwd(lib, _places(NAMES), _shape(batch=1), cu=cu, nseq=nseq), _abi.EINVAL)
    _code(lib, _bwd(lib, _places(NAMES + GRADS), _shape(batch=1), cu=cu, nseq=nseq), _abi.EINVAL)


def test_fwd_other(lib):
    at = _places(NAMES)
    _code(lib, _fwd(lib, at, cu=[0, 100]), _abi.EINVAL, "batch == 1")
    for s in (float("nan"), float("inf")):
        _code(lib, _fwd(lib, at, scale=s), _abi.EINVAL, "scale")
    _code(lib, _fwd(lib, at, _shape(batch=1), cu=[0, 40, 100], ws=8), _abi.EWORKSPACE)
    at["ws"] += 16
    _code(lib, _fwd(lib, at, _shape(batch=1), cu=[0, 40, 100]), _abi.EINVAL, "256")


@pytest.mark.parametrize("out", ["y", "final", "ws"])
@pytest.mark.parametrize("other", [n for n in NAMES])
def test_fwd_overlaps(lib, out, other):
    if out == other:
        return
    for shift in (0, 256):
        if out == "final" and other == "init" and shift == 0:
            continue   # in place
        at = _places(NAMES)
        at[out] = at[other] + shift
        if "ws" in (out, other):
            rc = _fwd(lib, at, _shape(batch=1, seqlen=100), cu=list(range(101)))
        else:
            rc = _fwd(lib, at)
        _code(lib, rc, _abi.EINVAL, "overlaps")


def test_step(lib):
    at = _places(NAMES)

    def call(state=STEP * 40, f=_dir(at, "f"), r=None, y=at["y"], **kw):
        return lib.bimamba_delta_step(_shape(**dict(dict(seqlen=1), **kw)), state, f, r, 1.0, 1, y, at["ws"], 1 << 30, None)
    _code(lib, call(state=None), _abi.EINVAL, "state")
    _code(lib, call(state=STEP * 40 + 4), _abi.EINVAL, "aligned")
    _code(lib, call(seqlen=257), _abi.EINVAL, "256")
    _code(lib, call(seqlen=0), _abi.EINVAL)
    _code(lib, call(y=None), _abi.EINVAL)
    _code(lib, call(f=None), _abi.EINVAL)
    _code(lib, call(state=at["y"]), _abi.EINVAL, "overlaps")
    _code(lib, call(state=at["fv"]), _abi.EINVAL, "overlaps")


def _grad(at, r):
    return ctypes.byref(_abi.DeltaGrad(*(at[r + "d" + n] for n in "qkvgb")))


def _bwd(lib, at, shape=None, both=True, cu=None, nseq=None, ws=1 << 40, scale=1.0, gb=True):
    nseq = nseq if nseq is not None else len(cu) - 1 if cu is not None else 0
    at = dict(dict(dy=STEP * 60, df=STEP * 61, di=STEP * 62), **at)
    return lib.bimamba_delta_bwd(shape or _shape(), _dir(at, "f"), _dir(at, "r") if both else None, scale, _cu(cu), nseq,
                                 at["init"], at["df"], at["dy"], _grad(at, "f"), _grad(at, "r") if gb else None,
                                 at["di"], at["ws"], ws, None)


def test_bwd_missing_and_unaligned(lib):
    for name in GRADS + ["dy", "fq", "rb"]:
        at = dict(_places(NAMES + GRADS), dy=STEP * 60)
        at[name] = None
        _code(lib, _bwd(lib, at), _abi.EINVAL)
    for name in GRADS + ["dy", "init", "rk"]:
        at = dict(_places(NAMES + GRADS), dy=STEP * 60)
        at[name] += 2
        _code(lib, _bwd(lib, at), _abi.EINVAL, "aligned")
    at = _places(NAMES + GRADS)
    _code(lib, _bwd(lib, at, gb=False), _abi.EINVAL, "NULL")
    _code(lib, _bwd(lib, at, both=False), _abi.EINVAL, "without the reverse")
    n = ctypes.c_size_t(0)
    assert lib.bimamba_delta_bwd_workspace_size(_shape(), 0, ctypes.byref(n)) == 0
    _code(lib, _bwd(lib, at, ws=n.value - 1), _abi.EWORKSPACE)
    _code(lib, _bwd(lib, dict(at, ws=None)), _abi.EWORKSPACE)
    _code(lib, _bwd(lib, at, scale=float("nan")), _abi.EINVAL, "scale")


@pytest.mark.parametrize("out", GRADS + ["di", "ws"])
def test_bwd_overlaps(lib, out):
    for other in NAMES + GRADS + ["dy", "df", "di"]:
        if other in (out, "y", "final"):
            continue
        at = dict(_places(NAMES + GRADS), dy=STEP * 60, df=STEP * 61, di=STEP * 62)
        at[out] = at[other]
        _code(lib, _bwd(lib, at), _abi.EINVAL, "overlaps")


def test_binding():
    d = _dirs(4, 1, 1, 4, 2, 4, 1, 16, "f32")[0][0]
    for call in (lambda: bm.delta_fwd(d), lambda: bm.delta_step(torch.zeros(1, 2, 4, 16), d),
                 lambda: bm.delta_bwd(d, None, d["v"])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    assert bm.delta_workspace_size(d) >= 0 and bm.delta_bwd_workspace_size(d) > 0
    with pytest.raises(ValueError, match="32 bits"):
        far = torch.empty(1, device="meta").expand(1, 2 ** 32 + 8, 1, 16)
        bm.delta_workspace_size(dict(q=far, v=far.to(torch.bfloat16)))

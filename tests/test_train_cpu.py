"""Pins of the training oracle (oracle/train.py) and the refusals of the
training entry points, all on the CPU: every rejected call is refused before
any HIP call."""
import ctypes
import os

import numpy as np
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
from bidirectional_mamba_ssm_amd import _abi
from oracle import conv as oconv
from oracle import train as otrain


# ---- the oracle ---------------------------------------------------------------

def _rng(seed):
    return np.random.default_rng(seed)


def _auto(f, *arrays):
    ts = [torch.tensor(a, dtype=torch.float64, requires_grad=True) for a in arrays]
    f(*ts).backward()
    return [t.grad.numpy() for t in ts]


def test_layer_norm_pins():
    r = _rng(1)
    h, w, b, g, ds = r.normal(size=(5, 33)), r.normal(size=33), r.normal(size=33), r.normal(size=(5, 33)), \
        r.normal(size=(5, 33))
    out, _, mean, rstd = otrain.layer_norm(h, w, b, 1e-3)
    ref = torch.nn.functional.layer_norm(torch.tensor(h), (33,), torch.tensor(w), torch.tensor(b), 1e-3).numpy()
    assert np.allclose(out, ref, rtol=1e-12, atol=1e-12)

    def f(x, wt, bt):
        y = torch.nn.functional.layer_norm(x, (33,), wt, bt, 1e-3)
        return (y * torch.tensor(g)).sum() + (x * torch.tensor(ds)).sum()
    for got, want in zip(otrain.layer_norm_bwd(g, h, mean, rstd, w, ds), _auto(f, h, w, b)):
        assert np.allclose(got[0], want, rtol=1e-10, atol=1e-12)
        assert np.all(got[1] >= np.abs(got[0]) - 1e-12)


@pytest.mark.parametrize("group", [8, 24])
def test_gated_norm_pins(group):
    r = _rng(2)
    y, z, w, g = r.normal(size=(4, 24)), 3 * r.normal(size=(4, 24)), r.normal(size=24), r.normal(size=(4, 24))

    def f(yt, zt, wt):
        v = yt * torch.nn.functional.silu(zt)
        q = v.reshape(4, 24 // group, group)
        o = (q * torch.rsqrt((q * q).mean(dim=2, keepdim=True) + 1e-4)).reshape(4, 24) * wt
        return (o * torch.tensor(g)).sum()
    for got, want in zip(otrain.gated_norm_bwd(g, y, z, w, group, 1e-4), _auto(f, y, z, w)):
        assert np.allclose(got[0], want, rtol=1e-9, atol=1e-12)
        assert np.all(got[1] >= np.abs(got[0]) - 1e-12)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("cu", [None, [0, 3, 3, 4, 11]])
def test_conv_bwd_pins(reverse, act, cu):
    """Central differences of the forward oracle, and autograd through torch's
    depthwise convolution sequence by sequence."""
    r = _rng(3)
    B, L, ch, W = (2 if cu is None else 1), 11, 3, 4
    x, w, b, g = r.normal(size=(B, L, ch)), r.normal(size=(ch, W)), r.normal(size=ch), r.normal(size=(B, L, ch))
    got = otrain.conv1d_bwd(x, w, b, g, reverse, cu, act)

    def loss(xx, ww, bb):
        o = oconv.conv1d(xx, ww, bb, reverse=reverse, cu_seqlens=cu, activation=act)
        return float((o * g).sum())
    h = 1e-6
    for a, (grad, S) in zip((x, w, b), got):
        assert np.all(S >= np.abs(grad) - 1e-9)
        for idx in np.ndindex(a.shape):
            keep = a[idx]
            a[idx] = keep + h
            up = loss(x, w, b)
            a[idx] = keep - h
            down = loss(x, w, b)
            a[idx] = keep
            assert abs((up - down) / (2 * h) - grad[idx]) < 1e-7 * (1 + S[idx])

    def f(xt, wt, bt):
        total = 0.0
        starts = [0, L] if cu is None else cu
        for s, e in zip(starts, starts[1:]):
            if e == s:
                continue
            seg = xt[:, s:e].transpose(1, 2)
            if reverse:
                seg = seg.flip(2)
            o = torch.nn.functional.conv1d(torch.nn.functional.pad(seg, (W - 1, 0)), wt[:, None], bt, groups=ch)
            if act == "silu":
                o = torch.nn.functional.silu(o)
            if reverse:
                o = o.flip(2)
            total = total + (o.transpose(1, 2) * torch.tensor(g[:, s:e])).sum()
        return total
    for want, (grad, _) in zip(_auto(f, x, w, b), got):
        assert np.allclose(grad, want, rtol=1e-10, atol=1e-12)


def test_act8_pins():
    # worked by hand: top 1.5 has exponent field 127, unit 2^-6
    v = np.zeros((1, 33))
    v[0, :5] = [1.5, -1.0, 0.25 + 2.0 ** -7, 0.25 + 3 * 2.0 ** -7, 1e-9]
    v[0, 32] = -3.0
    q, E = otrain.act8(v)
    assert E.tolist() == [[127, 128]]
    assert q[0, :5].tolist() == [96, -64, 16, 18, 0]      # the halves go to even
    assert q[0, 32] == -96
    assert otrain.act8_values(q, E)[0, 32] == -3.0
    # values of up to 7 bits below the block's top come back as they were
    r = _rng(4)
    m = r.integers(-127, 128, size=(3, 64)).astype(np.float64)
    m[:, ::32] = 127.0
    x = m * 2.0 ** r.integers(-30, 30, size=(3, 1))
    assert np.array_equal(otrain.act8_values(*otrain.act8(x)), x)
    # the bound, the clamp (the largest mantissas), zeros, subnormals, NaN
    x = r.normal(size=(4, 320))
    err = np.abs(otrain.act8_values(*otrain.act8(x)) - x).reshape(4, 10, 32).max(axis=2)
    assert np.all(err <= np.abs(x).reshape(4, 10, 32).max(axis=2) * 2.0 ** -7)
    q, E = otrain.act8(np.array([[2.0 - 2.0 ** -20] + [0.0] * 31]))
    assert q[0, 0] == 127 and E[0, 0] == 127
    assert otrain.act8(np.zeros((1, 32)))[1][0, 0] == 0
    q, E = otrain.act8(np.array([[2.0 ** -127, 2.0 ** -134, 3 * 2.0 ** -134]]))
    assert E[0, 0] == 0 and q[0].tolist() == [64, 0, 2]
    q, E = otrain.act8(np.array([[1.0, np.inf] + [2.0] * 30 + [5.0]]))
    assert E.tolist() == [[255, 129]] and np.isnan(otrain.act8_values(q, E)[0, :32]).all()


def test_a_mistake_in_the_oracle_is_seen():
    """The pins' comparisons fail for a gradient with a term missing."""
    r = _rng(5)
    h, g = r.normal(size=(3, 16)), r.normal(size=(3, 16))
    _, _, mean, rstd = otrain.layer_norm(h, None, None, 1e-5)
    good = otrain.layer_norm_bwd(g, h, mean, rstd, None, None)[0][0]
    bad = (g - g.mean(axis=1, keepdims=True)) * rstd[:, None]
    assert np.abs(good - bad).max() > 1e-2


# ---- refusals: the C ABI ------------------------------------------------------------

FAKE = 0x10000   # aligned, never dereferenced: every call below fails validation


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_abi.LIB_PATH):
        from bidirectional_mamba_ssm_amd import build
        build.build()
    return _abi.load()


def _ln(lib, rows=4, C=64, dt=_abi.BF16, x=FAKE, res=None, w=None, b=None, eps=1e-5, out=FAKE, s=None, mean=None,
        rstd=None, ck=None):
    return lib.bimamba_layer_norm(rows, C, dt, x, res, w, b, eps, out, s, mean, rstd,
                                  ctypes.byref(ck) if ck is not None else None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), _abi.EINVAL), (dict(rows=1 << 31), _abi.EUNSUPPORTED), (dict(dt=3), _abi.EINVAL),
    (dict(C=7), _abi.EUNSUPPORTED), (dict(C=16385), _abi.EUNSUPPORTED), (dict(C=0), _abi.EUNSUPPORTED),
    (dict(eps=-1.0), _abi.EINVAL), (dict(eps=float("nan")), _abi.EINVAL), (dict(eps=float("inf")), _abi.EINVAL),
    (dict(x=None), _abi.EINVAL), (dict(out=None), _abi.EINVAL), (dict(x=FAKE + 1), _abi.EINVAL),
    (dict(dt=_abi.F32, out=FAKE + 2), _abi.EINVAL), (dict(w=FAKE + 2), _abi.EINVAL), (dict(mean=FAKE + 1), _abi.EINVAL),
    (dict(res=FAKE), _abi.EINVAL), (dict(s=FAKE), _abi.EINVAL), (dict(ck=_abi.Act8Ptrs(FAKE, None)), _abi.EINVAL),
])
def test_layer_norm_refused(lib, kw, code):
    assert _ln(lib, **kw) == code and lib.bimamba_last_error()


def test_layer_norm_no_rows(lib):
    assert _ln(lib, rows=0, x=None, out=None) == 0


def _lnb(lib, rows=4, C=64, dt=_abi.BF16, x=FAKE, xs=None, mean=FAKE, rstd=FAKE, w=None, dout=FAKE, dsum=None,
         dx=FAKE, dw=FAKE, db=FAKE, ws=None, wsb=0):
    return lib.bimamba_layer_norm_bwd(rows, C, dt, x, xs, mean, rstd, w, dout, dsum, dx, dw, db, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(), _abi.EWORKSPACE), (dict(ws=FAKE, wsb=16), _abi.EWORKSPACE), (dict(ws=FAKE + 16, wsb=1 << 30), _abi.EINVAL),
    (dict(C=4), _abi.EUNSUPPORTED), (dict(rows=-2), _abi.EINVAL), (dict(dt=-1), _abi.EINVAL),
    (dict(mean=None), _abi.EINVAL), (dict(dout=None), _abi.EINVAL), (dict(dx=FAKE + 1), _abi.EINVAL),
    (dict(dsum=FAKE + 1), _abi.EINVAL), (dict(dw=FAKE + 1), _abi.EINVAL), (dict(rstd=FAKE + 2), _abi.EINVAL),
])
def test_layer_norm_bwd_refused(lib, kw, code):
    assert _lnb(lib, **kw) == code and lib.bimamba_last_error()


def test_layer_norm_bwd_no_rows(lib):
    # without weight gradients there is nothing to do for no row
    assert _lnb(lib, rows=0, dw=None, db=None) == 0


def _gnb(lib, rows=4, C=512, gs=256, dt=_abi.BF16, y=FAKE, ys=None, z=FAKE, zs=None, w=FAKE, eps=1e-5, dout=FAKE,
         dy=FAKE, dz=FAKE, dw=FAKE, ws=None, wsb=0):
    return lib.bimamba_gated_norm_bwd(rows, C, gs, dt, y, ys, z, zs, w, eps, dout, dy, dz, dw, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(), _abi.EWORKSPACE), (dict(C=500), _abi.EUNSUPPORTED), (dict(C=8448), _abi.EUNSUPPORTED),
    (dict(gs=128), _abi.EINVAL), (dict(C=1024, gs=768), _abi.EINVAL), (dict(eps=-1e-9), _abi.EINVAL),
    (dict(y=None), _abi.EINVAL), (dict(dz=None), _abi.EINVAL), (dict(dy=FAKE + 8), _abi.EINVAL),
    (dict(y=FAKE + 4, ys=FAKE), _abi.EINVAL), (dict(dw=FAKE + 2), _abi.EINVAL), (dict(dt=9), _abi.EINVAL),
    (dict(rows=1 << 31), _abi.EUNSUPPORTED),
])
def test_gated_norm_bwd_refused(lib, kw, code):
    assert _gnb(lib, **kw) == code and lib.bimamba_last_error()


def _cshape(**kw):
    d = dict(batch=1, seqlen=8, nheads=2, headdim=16, d_state=16, ngroups=1, width=4, dtype=_abi.BF16, activation=1,
             flags=0)
    d.update(kw)
    return _abi.ConvShape(**d)


def _cgrad(**kw):
    d = dict(xbc=FAKE, xbc_scale=None, weight=FAKE, bias=FAKE, dx=FAKE, dB=FAKE, dC=FAKE, dxbc=FAKE, dweight=FAKE,
             dbias=FAKE)
    d.update(kw)
    return _abi.ConvGrad(**d)


def _cb(lib, s=None, f=None, b=None, cu=None, nseq=0, ws=None, wsb=0):
    arr = (ctypes.c_int32 * len(cu))(*cu) if cu is not None else None
    s, f = s or _cshape(), f or _cgrad()
    return lib.bimamba_conv1d_bwd(ctypes.byref(s), ctypes.byref(f), ctypes.byref(b) if b is not None else None, arr,
                                  nseq, ws, wsb, None)


def test_conv_bwd_refused(lib):
    E, U, K = _abi.EINVAL, _abi.EUNSUPPORTED, _abi.EWORKSPACE
    assert lib.bimamba_conv1d_bwd(None, None, None, None, 0, None, 0, None) == E
    assert _cb(lib) == K
    assert _cb(lib, ws=FAKE, wsb=16) == K
    assert _cb(lib, ws=FAKE + 16, wsb=1 << 30) == E
    assert _cb(lib, s=_cshape(width=5)) == U
    assert _cb(lib, s=_cshape(width=1)) == U
    assert _cb(lib, s=_cshape(flags=1)) == E
    assert _cb(lib, s=_cshape(seqlen=(1 << 30) + 1)) == U
    assert _cb(lib, s=_cshape(batch=20000, seqlen=100000, nheads=512, headdim=128)) == U
    for name in ("xbc", "weight", "dx", "dB", "dC", "dxbc", "dweight"):
        assert _cb(lib, f=_cgrad(**{name: None})) == E, name
    for name in ("xbc", "dx", "dB", "dC", "dxbc"):
        assert _cb(lib, f=_cgrad(**{name: FAKE + 8})) == E, name
    for name in ("weight", "bias", "dweight", "dbias"):
        assert _cb(lib, f=_cgrad(**{name: FAKE + 2})) == E, name
    assert _cb(lib, f=_cgrad(xbc_scale=FAKE), b=_cgrad()) == U
    assert _cb(lib, b=_cgrad(dC=None)) == E
    other = dict(dxbc=FAKE * 2, dweight=FAKE * 2, dbias=FAKE * 2)
    assert _cb(lib, b=_cgrad(**other)) == K
    for name in other:   # one array for both directions
        assert _cb(lib, b=_cgrad(**dict(other, **{name: FAKE}))) == E, name
    assert _cb(lib, f=_cgrad(dbias=None), b=_cgrad(**dict(other, dbias=None))) == K
    assert _cb(lib, nseq=2) == E
    assert _cb(lib, cu=[0, 3, 7], nseq=2) == E
    assert _cb(lib, cu=[0, 5, 4, 8], nseq=3) == E
    assert _cb(lib, s=_cshape(batch=2), cu=[0, 8], nseq=1) == E
    n = ctypes.c_size_t(0)
    s = _cshape()
    assert lib.bimamba_conv1d_bwd_workspace_size(ctypes.byref(s), 1, 0, None) == E
    assert lib.bimamba_conv1d_bwd_workspace_size(ctypes.byref(s), 1, -1, ctypes.byref(n)) == E
    assert lib.bimamba_conv1d_bwd_workspace_size(ctypes.byref(s), 1, 2, ctypes.byref(n)) == 0
    assert _cb(lib, b=_cgrad(**other), cu=[0, 3, 8], nseq=2, ws=FAKE, wsb=n.value - 1) == K


def test_conv_act8_refused(lib):
    E = _abi.EINVAL
    s = _cshape()

    def call(d, a, rd=None, ra=None, cu=None, nseq=0, sh=s):
        arr = (ctypes.c_int32 * len(cu))(*cu) if cu is not None else None
        return lib.bimamba_conv1d_act8(ctypes.byref(sh), d and ctypes.byref(d), a and ctypes.byref(a),
                                       rd and ctypes.byref(rd), ra and ctypes.byref(ra), arr, nseq, None, 0, None)
    d = _abi.ConvDir(None, FAKE, FAKE, FAKE, FAKE, FAKE)
    a = _abi.Act8Ptrs(FAKE, FAKE)
    assert call(None, a) == E
    assert call(d, None) == E
    assert call(d, _abi.Act8Ptrs(None, FAKE)) == E
    assert call(d, _abi.Act8Ptrs(FAKE, None)) == E
    assert call(d, _abi.Act8Ptrs(FAKE + 4, FAKE)) == E
    assert call(_abi.ConvDir(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE), a) == E
    assert call(_abi.ConvDir(None, FAKE, FAKE, FAKE + 2, FAKE, FAKE), a) == E
    assert call(d, a, d, None) == E
    assert call(d, a, None, a) == E
    assert call(d, a, nseq=1) == E
    many = [0] * 129 + [8]   # beyond what goes by value: a table in the workspace
    assert call(d, a, cu=many, nseq=129) == _abi.EWORKSPACE
    n = ctypes.c_size_t(0)
    assert lib.bimamba_conv1d_act8_workspace_size(ctypes.byref(s), 129, ctypes.byref(n)) == 0 and n.value >= 32
    assert lib.bimamba_conv1d_act8_workspace_size(ctypes.byref(s), 128, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.bimamba_conv1d_act8_workspace_size(ctypes.byref(s), -1, ctypes.byref(n)) == E


def test_act8_refused(lib):
    a = _abi.Act8Ptrs(FAKE, FAKE)
    for f, args in ((lib.bimamba_act8_pack, lambda x, p: (x, p)), (lib.bimamba_act8_unpack, lambda x, p: (p, x))):
        def call(rows=1, C=32, dt=_abi.BF16, x=FAKE, p=ctypes.byref(a)):
            return f(rows, C, dt, *args(x, p), None)
        assert call(rows=-1) == _abi.EINVAL
        assert call(rows=1 << 31) == _abi.EUNSUPPORTED
        assert call(C=0) == _abi.EUNSUPPORTED
        assert call(C=1 << 31) == _abi.EUNSUPPORTED
        assert call(dt=2) == _abi.EINVAL
        assert call(x=None) == _abi.EINVAL
        assert call(x=FAKE + 1) == _abi.EINVAL
        assert call(p=None) == _abi.EINVAL
        assert call(p=ctypes.byref(_abi.Act8Ptrs(FAKE, None))) == _abi.EINVAL
        assert call(rows=0, x=None, p=None) == 0


# ---- refusals: the binding ------------------------------------------------------------

def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64)
    st = torch.zeros(2)
    a = bm.Act8.empty((2, 64), "cpu")
    for f in (lambda: bm.act8_pack(x), lambda: bm.act8_unpack(a), lambda: bm.layer_norm(x),
              lambda: bm.layer_norm_bwd(x, x, st, st),
              lambda: bm.gated_norm_bwd(x, x, x, torch.zeros(64)),
              lambda: bm.conv1d_bwd(dict(xbc=torch.zeros(1, 2, 64), weight=torch.zeros(64, 4)), None, {}, None, 2, 16,
                                    1, 16),
              lambda: bm.conv1d(dict(xbc=bm.Act8.empty((1, 2, 64), "cpu"), weight=torch.zeros(64, 4)), None, 2, 16, 1,
                                16)):
        with pytest.raises(ValueError, match="CUDA"):
            f()


def test_act8_shapes_checked():
    dev = torch.device("cpu")
    a = bm.Act8.empty((3, 5, 33), "cpu")
    assert a.q.shape == (3, 5, 33) and a.scale.shape == (3, 5, 2) and a.shape == (3, 5, 33)
    a._ptrs("a", (3, 5, 33), dev)
    with pytest.raises(ValueError, match="shape"):
        a._ptrs("a", (3, 5, 34), dev)
    with pytest.raises(ValueError, match="scale"):
        bm.Act8(a.q, a.scale[..., :1].contiguous())._ptrs("a", (3, 5, 33), dev)
    with pytest.raises(TypeError, match="dtype"):
        bm.Act8(a.q.view(torch.uint8), a.scale)._ptrs("a", (3, 5, 33), dev)
    with pytest.raises(ValueError, match="contiguous"):
        bm.Act8(a.q.transpose(0, 1), a.scale)._ptrs("a", (5, 3, 33), dev)

"""Arrays of the training steps that overlap where a result would depend on
the order of reads and writes: such calls are refused before any HIP call.
CPU only, on addresses that are never dereferenced."""
import ctypes
import os

import pytest

from bidirectional_mamba_ssm_amd import _abi

STEP = 1 << 24   # further apart than any array here is long


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_abi.LIB_PATH):
        from bidirectional_mamba_ssm_amd import build
        build.build()
    return _abi.load()


class Places:
    """Addresses of named arrays, each in a place of its own."""

    def __init__(self):
        self.used = {}

    def __call__(self, name):
        return self.used.setdefault(name, STEP * (len(self.used) + 1))


def _refused(lib, rc, *names):
    assert rc == _abi.EINVAL, (rc, lib.bimamba_last_error())
    msg = lib.bimamba_last_error().decode()
    assert "overlaps" in msg and all(n in msg for n in names), msg


# ---- the convolution's gradient ---------------------------------------------------

B_, L_, H_, P_, N_, G_, W_ = 2, 50, 2, 16, 16, 1, 4
CH = H_ * P_ + 2 * G_ * N_
TOK = B_ * L_
# bytes of each array (bf16) and whether the call writes it
CONV = dict(xbc=(TOK * CH * 2, False), weight=(CH * W_ * 4, False), bias=(CH * 4, False),
            dx=(TOK * H_ * P_ * 4, False), dB=(TOK * N_ * 4, False), dC=(TOK * N_ * 4, False),
            dxbc=(TOK * CH * 2, True), dweight=(CH * W_ * 4, True), dbias=(CH * 4, True))


def _conv_bwd(lib, at, q8=False):
    s = _abi.ConvShape(B_, L_, H_, P_, N_, G_, W_, _abi.BF16, 1, 0)
    n = ctypes.c_size_t(0)
    assert lib.bimamba_conv1d_bwd_workspace_size(ctypes.byref(s), 1, 0, ctypes.byref(n)) == 0
    dirs = [_abi.ConvGrad(at[r + "xbc"], at[r + "scale"] if q8 else None, at[r + "weight"], at[r + "bias"],
                          at[r + "dx"], at[r + "dB"], at[r + "dC"], at[r + "dxbc"], at[r + "dweight"],
                          at[r + "dbias"]) for r in "fr"]
    return lib.bimamba_conv1d_bwd(ctypes.byref(s), ctypes.byref(dirs[0]), ctypes.byref(dirs[1]), None, 0, at["ws"],
                                  n.value, None)


def _conv_places():
    p = Places()
    at = {r + k: p(r + k) for r in "fr" for k in list(CONV) + ["scale"]}
    at["ws"] = p("ws")
    return at


@pytest.mark.parametrize("out", ["fdxbc", "rdxbc"])
@pytest.mark.parametrize("src", ["fxbc", "rxbc"])
def test_conv_bwd_onto_its_input(lib, out, src):
    at = _conv_places()
    at[out] = at[src]
    _refused(lib, _conv_bwd(lib, at), "dxbc", "xbc")


@pytest.mark.parametrize("src", sorted(CONV))
def test_conv_bwd_partial_overlaps(lib, src):
    """An output that begins inside another array's last bytes, and one that
    ends in another's first ones."""
    nbytes = CONV[src][0]
    for r in "fr":
        at = _conv_places()
        if r + src != "fdxbc":
            at["fdxbc"] = at[r + src] + (nbytes - 1) // 16 * 16
            _refused(lib, _conv_bwd(lib, at), "the forward dxbc")
            at = _conv_places()
            at["fdxbc"] = at[r + src] - (CONV["dxbc"][0] - 16)
            _refused(lib, _conv_bwd(lib, at), "the forward dxbc")
        if r + src != "rdweight":
            at = _conv_places()
            at["rdweight"] = at[r + src] + nbytes - 4
            _refused(lib, _conv_bwd(lib, at), "the reverse dweight")


def test_conv_bwd_checkpoints_and_workspace(lib):
    for out, size in (("fdxbc", 16), ("rdxbc", 16), ("fdweight", 4), ("rdbias", 4)):
        at = _conv_places()
        at[out] = at["rscale"] + (TOK * 2 - 1) // size * size
        _refused(lib, _conv_bwd(lib, at, q8=True), "the reverse xbc_scale")
        at = _conv_places()
        at[out] = at["fxbc"] + TOK * CH - size   # a byte an element
        _refused(lib, _conv_bwd(lib, at, q8=True), "the forward xbc")
        at = _conv_places()
        at[out] = at["ws"]
        _refused(lib, _conv_bwd(lib, at), "the workspace")
    at = _conv_places()
    at["rdC"] = at["ws"]
    _refused(lib, _conv_bwd(lib, at), "the workspace", "the reverse dC")


# ---- the convolution from checkpoints ----------------------------------------------

C8_OUT = dict(x=TOK * H_ * P_ * 2, B=TOK * N_ * 2, C=TOK * N_ * 2)
C8_IN = dict(q=TOK * CH, scale=TOK * 2, weight=CH * W_ * 4, bias=CH * 4)


def _conv_act8(lib, at):
    s = _abi.ConvShape(B_, L_, H_, P_, N_, G_, W_, _abi.BF16, 1, 0)
    dirs = [_abi.ConvDir(None, at[r + "weight"], at[r + "bias"], at[r + "x"], at[r + "B"], at[r + "C"]) for r in "fr"]
    kept = [_abi.Act8Ptrs(at[r + "q"], at[r + "scale"]) for r in "fr"]
    return lib.bimamba_conv1d_act8(ctypes.byref(s), ctypes.byref(dirs[0]), ctypes.byref(kept[0]), ctypes.byref(dirs[1]),
                                   ctypes.byref(kept[1]), None, 0, None, 0, None)


@pytest.mark.parametrize("out", [r + k for r in "fr" for k in C8_OUT])
def test_conv_from_checkpoint_overlaps(lib, out):
    p = Places()
    places = {r + k: p(r + k) for r in "fr" for k in list(C8_OUT) + list(C8_IN)}
    for other, place in places.items():
        if other == out:
            continue
        nbytes = (C8_OUT | C8_IN)[other[1:]]
        for at in (place, place + (nbytes - 1) // 16 * 16, place - C8_OUT[out[1:]] + 16):
            _refused(lib, _conv_act8(lib, dict(places, **{out: at})))


def test_conv_from_checkpoint_onto_its_sequence_table(lib):
    s = _abi.ConvShape(1, L_, H_, P_, N_, G_, W_, _abi.BF16, 1, 0)
    p = Places()
    d = _abi.ConvDir(None, p("weight"), p("bias"), p("x"), p("B"), p("C"))
    kept = _abi.Act8Ptrs(p("q"), p("scale"))
    cu = (ctypes.c_int32 * 201)(*[min(i, L_) for i in range(201)])
    n = ctypes.c_size_t(0)
    assert lib.bimamba_conv1d_act8_workspace_size(ctypes.byref(s), 200, ctypes.byref(n)) == 0
    rc = lib.bimamba_conv1d_act8(ctypes.byref(s), ctypes.byref(d), ctypes.byref(kept), None, None, cu, 200, p("C"),
                                 n.value, None)
    _refused(lib, rc, "the forward C", "the workspace")


# ---- layer norm -------------------------------------------------------------------------

ROWS, CHS = 9, 72
LN_OUT = dict(out=ROWS * CHS * 2, sum=ROWS * CHS * 2, mean=ROWS * 4, rstd=ROWS * 4, q=ROWS * CHS, scale=ROWS * 3)
LN_IN = dict(x=ROWS * CHS * 2, residual=ROWS * CHS * 2, weight=CHS * 4, bias=CHS * 4)


def _ln_places():
    p = Places()
    return {k: p(k) for k in list(LN_OUT) + list(LN_IN)}


def _layer_norm(lib, at):
    ck = _abi.Act8Ptrs(at["q"], at["scale"])
    return lib.bimamba_layer_norm(ROWS, CHS, _abi.BF16, at["x"], at["residual"], at["weight"], at["bias"], 1e-5,
                                  at["out"], at["sum"], at["mean"], at["rstd"], ctypes.byref(ck), None)


@pytest.mark.parametrize("out", sorted(LN_OUT))
def test_layer_norm_overlaps(lib, out):
    for other, nbytes in (LN_OUT | LN_IN).items():
        if other == out:
            continue
        places = _ln_places()
        whole = (out in ("out", "sum") and other in ("x", "residual"))   # in place, see below
        for at in ([] if whole else [places[other]]) + [places[other] + (nbytes - 1) // 4 * 4,
                                                        places[other] - LN_OUT[out] + 4]:
            _refused(lib, _layer_norm(lib, dict(places, **{out: at})))


@pytest.mark.parametrize("src", ["x", "residual"])
def test_layer_norm_sum_is_not_out(lib, src):
    """One array for both results, a place of its own or an input's."""
    places = _ln_places()
    _refused(lib, _layer_norm(lib, dict(places, sum=places["out"])), "out", "sum")
    _refused(lib, _layer_norm(lib, dict(places, sum=places[src], out=places[src])), "out", "sum")
    # an input that is an output keeps the other outputs away, too
    for out in ("out", "sum"):
        for k in ("mean", "q"):
            _refused(lib, _layer_norm(lib, dict(places, **{out: places[src], k: places[src] + 64})), k)


# ---- layer norm's gradient ---------------------------------------------------------------

LNB_IN = dict(x=ROWS * CHS * 2, mean=ROWS * 4, rstd=ROWS * 4, weight=CHS * 4, dout=ROWS * CHS * 2, dsum=ROWS * CHS * 2)
LNB_OUT = dict(dx=ROWS * CHS * 2, dweight=CHS * 4, dbias=CHS * 4)


def _lnb_places():
    p = Places()
    return {k: p(k) for k in list(LNB_OUT) + list(LNB_IN) + ["scale", "ws"]}


def _layer_norm_bwd(lib, at, q8=False):
    n = ctypes.c_size_t(0)
    assert lib.bimamba_layer_norm_bwd_workspace_size(ROWS, CHS, _abi.BF16, ctypes.byref(n)) == 0
    return lib.bimamba_layer_norm_bwd(ROWS, CHS, _abi.BF16, at["x"], at["scale"] if q8 else None, at["mean"], at["rstd"],
                                      at["weight"], at["dout"], at["dsum"], at["dx"], at["dweight"], at["dbias"],
                                      at["ws"], n.value, None)


@pytest.mark.parametrize("out", sorted(LNB_OUT))
def test_layer_norm_bwd_overlaps(lib, out):
    for other, nbytes in (LNB_OUT | LNB_IN).items():
        if other == out:
            continue
        places = _lnb_places()
        whole = out == "dx" and other in ("x", "dout", "dsum")   # in place
        for at in ([] if whole else [places[other]]) + [places[other] + (nbytes - 1) // 4 * 4,
                                                        places[other] - LNB_OUT[out] + 4]:
            _refused(lib, _layer_norm_bwd(lib, dict(places, **{out: at})))
    places = _lnb_places()
    _refused(lib, _layer_norm_bwd(lib, dict(places, **{out: places["ws"]})), "the workspace")
    for k in ("x", "scale"):
        _refused(lib, _layer_norm_bwd(lib, dict(places, **{out: places[k]}), q8=True), "x")


@pytest.mark.parametrize("src", ["dout", "dsum", "x"])
def test_layer_norm_bwd_in_place_keeps_others_away(lib, src):
    places = _lnb_places()
    places["dx"] = places[src]
    _refused(lib, _layer_norm_bwd(lib, dict(places, dweight=places[src] + 8)), "dweight")
    _refused(lib, _layer_norm_bwd(lib, dict(places, rstd=places[src] + 8)), "rstd")


# ---- the gated norm's gradient -----------------------------------------------------------

GC = 512
GN_IN = dict(y=ROWS * GC * 4, z=ROWS * GC * 2, weight=GC * 4, dout=ROWS * GC * 2)
GN_OUT = dict(dy=ROWS * GC * 4, dz=ROWS * GC * 2, dweight=GC * 4)


def _gn_places():
    p = Places()
    return {k: p(k) for k in list(GN_OUT) + list(GN_IN) + ["ys", "zs", "ws"]}


def _gated_norm_bwd(lib, at, q8=False):
    n = ctypes.c_size_t(0)
    assert lib.bimamba_gated_norm_bwd_workspace_size(ROWS, GC, 256, _abi.BF16, ctypes.byref(n)) == 0
    return lib.bimamba_gated_norm_bwd(ROWS, GC, 256, _abi.BF16, at["y"], at["ys"] if q8 else None, at["z"],
                                      at["zs"] if q8 else None, at["weight"], 1e-5, at["dout"], at["dy"], at["dz"],
                                      at["dweight"], at["ws"], n.value, None)


@pytest.mark.parametrize("out", sorted(GN_OUT))
def test_gated_norm_bwd_overlaps(lib, out):
    for other, nbytes in (GN_OUT | GN_IN).items():
        if other == out:
            continue
        places = _gn_places()
        whole = (out, other) in (("dy", "y"), ("dz", "z"), ("dz", "dout"))   # in place
        for at in ([] if whole else [places[other]]) + [places[other] + (nbytes - 1) // 16 * 16,
                                                        places[other] - GN_OUT[out] + 16]:
            _refused(lib, _gated_norm_bwd(lib, dict(places, **{out: at})))
    places = _gn_places()
    for k in ("y", "z", "ys", "zs"):
        _refused(lib, _gated_norm_bwd(lib, dict(places, **{out: places[k]}), q8=True), k[0])
    _refused(lib, _gated_norm_bwd(lib, dict(places, **{out: places["ws"]})), "the workspace")


# ---- 8-bit checkpoints ---------------------------------------------------------------------

def test_act8_overlaps(lib):
    nbytes = dict(x=ROWS * 33 * 4, q=ROWS * 33, scale=ROWS * 2)
    p = Places()
    places = {k: p(k) for k in nbytes}
    for pack in (True, False):
        for a in nbytes:
            for b in nbytes:
                if a == b or (not pack and "x" not in (a, b)):
                    continue   # an array read may overlap another that is read
                for at in (places[b], places[b] + (nbytes[b] - 1) // 4 * 4, places[b] - nbytes[a] // 4 * 4 + 4):
                    q = dict(places, **{a: at})
                    ck = _abi.Act8Ptrs(q["q"], q["scale"])
                    if pack:
                        rc = lib.bimamba_act8_pack(ROWS, 33, _abi.F32, q["x"], ctypes.byref(ck), None)
                    else:
                        rc = lib.bimamba_act8_unpack(ROWS, 33, _abi.F32, ctypes.byref(ck), q["x"], None)
                    _refused(lib, rc)

"""The convolution's gradient where runs, rows and sequences end: infinities
near a run's end, and rows shorter than a run in a batch of many."""
import numpy as np
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
from metrics import bf16_rne
from oracle import train as otrain

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
H, P, G, N = 4, 16, 1, 16
CH = H * P + 2 * G * N


def _direction(g, batch, L, W, dtype):
    d = dict(xbc=torch.randn(batch, L, CH, generator=g, device=DEV).to(DT[dtype]),
             weight=torch.randn(CH, W, generator=g, device=DEV) * 0.5,
             bias=torch.randn(CH, generator=g, device=DEV) * 0.5)
    gr = dict(x=torch.randn(batch, L, H, P, generator=g, device=DEV),
              B=torch.randn(batch, L, G, N, generator=g, device=DEV),
              C=torch.randn(batch, L, G, N, generator=g, device=DEV))
    return d, gr


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cu", [None, [0, 1, 17, 17, 40, 72, 96]], ids=["row", "packed"])
def test_one_infinity_a_channel(W, dtype, cu):
    """Without an activation the filter is linear: an infinite input at token
    c of channel c (so at every distance from a run's end) leaves xbc's and
    the bias's gradient as they are, and makes the gradient of each weight
    that meets it infinite, with the sign of that position's gradient; of no
    other weight."""
    L = CH
    print(f"W {W} {dtype} {cu}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(W)
    (f, gf), (r, gr) = _direction(g, 1, L, W, dtype), _direction(g, 1, L, W, dtype)
    call = dict(activation="none", cu_seqlens=cu)
    clean = bm.conv1d_bwd(f, r, gf, gr, H, P, G, N, **call)
    for d in (f, r):
        i = torch.arange(CH, device=DEV)
        d["xbc"] = d["xbc"].clone()
        d["xbc"][0, i, i] = float("inf")
    got = bm.conv1d_bwd(f, r, gf, gr, H, P, G, N, **call)
    starts = [0, L] if cu is None else cu
    for o, c, grad, sign in zip(got, clean, (gf, gr), (1, -1)):
        assert torch.equal(o["xbc"], c["xbc"]) and torch.equal(o["bias"], c["bias"])
        dout = torch.cat([grad[k].reshape(L, -1) for k in ("x", "B", "C")], dim=1).cpu().numpy()
        want = np.full((CH, W), np.nan)
        for ch in range(CH):
            lo = max(s for s in starts if s <= ch)
            hi = min(s for s in starts if s > ch)
            for k in range(W):
                t = ch + sign * (W - 1 - k)   # the token whose tap k is the infinite input
                want[ch, k] = np.inf * np.sign(dout[t, ch]) if lo <= t < hi else np.nan
        w = o["weight"].cpu().numpy()
        meets = ~np.isnan(want)
        assert np.array_equal(w[meets], want[meets])
        assert np.isfinite(w[~meets]).all()


def _close(name, got, ref, S, rel, dtype):
    """As in the parity tests: within rel * S, bf16 between the roundings of
    that interval's ends."""
    got, delta = got.double().cpu().numpy().reshape(ref.shape), rel * S
    lo, hi = ref - delta, ref + delta
    if dtype == "bf16":
        lo, hi = bf16_rne(lo), bf16_rne(hi)
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), (name, np.argwhere(bad)[:3].tolist())


@pytest.mark.parametrize("batch,L", [(1000, 1), (400, 2), (300, 5), (257, 8), (130, 33), (96, 64), (40, 129)])
@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("kept", [False, True], ids=["array", "ckpt"])
def test_rows_shorter_than_a_workgroups_runs(batch, L, W, kept):
    """A workgroup never crosses a row, so in short ones some of its waves (or
    of a wave's positions) have nothing to do. Bars as for one long row: 2^-18
    S, 2^-17 S for the weights' gradient (a run's 32 serial terms and 4 joins,
    the rest in 64 bits)."""
    dtype = "bf16" if W == 4 else "f32"
    print(f"{batch} x {L}, W {W} {dtype} {kept}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(batch + L)
    pairs = [_direction(g, batch, L, W, dtype) for _ in range(2)]
    dirs = [dict(d, xbc=bm.act8_pack(d["xbc"])) if kept else d for d, _ in pairs]
    res = bm.conv1d_bwd(dirs[0], dirs[1], pairs[0][1], pairs[1][1], H, P, G, N, dtype=DT[dtype])
    plain = [dict(d, xbc=bm.act8_unpack(d["xbc"], dtype=DT[dtype])) if kept else d for d in dirs]
    for d, (_, gr), o, rev in zip(plain, pairs, res, (False, True)):
        dout = torch.cat([gr[k].reshape(batch, L, -1) for k in ("x", "B", "C")], dim=2)
        rx, rw, rb = otrain.conv1d_bwd(d["xbc"], d["weight"], d["bias"], dout, rev, None, "silu")
        _close("dxbc", o["xbc"], *rx, 2.0 ** -18, dtype)
        _close("dweight", o["weight"], *rw, 2.0 ** -17, "f32")
        _close("dbias", o["bias"], *rb, 2.0 ** -17, "f32")
    if kept:
        for o, p in zip(bm.conv1d(dirs[0], dirs[1], H, P, G, N, dtype=DT[dtype]),
                        bm.conv1d(plain[0], plain[1], H, P, G, N)):
            assert all(torch.equal(o[k], p[k]) for k in ("x", "B", "C"))

"""The convolution's gradient where runs, rows and sequences end: infinities
near a run's end, and rows shorter than a run in a batch of many."""
import numpy as np
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm

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

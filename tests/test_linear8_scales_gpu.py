"""The 8-bit product where the product of its two scales leaves fp32's normal
numbers while the result does not, in each of its kernels.

Tolerances as in test_rows8_gpu.py: 2^-22 of the magnitudes, and half a step of
fp32's subnormals, 2^-150, where a result lies among them. A result beyond
fp32's largest number is an infinity."""
import numpy as np
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
from test_rows8_gpu import DT, PROD, _close, _fast, _gen, _int8

pytestmark = pytest.mark.gpu

DEV = "cuda"
# rows, cin, cout: few rows (each number of tiles), 64 and 128 wide tiles, the wide
# ones; rows that are no multiple of 16 bytes in both tiles
FORMS = [(7, 64, 40), (30, 80, 33), (64, 128, 100), (64, 64, 5000), (130, 48, 70), (2100, 64, 2100), (3700, 16, 3800),
         (20, 33, 50), (2100, 17, 2200)]


def _scales(g, n, low, high):
    """Magnitudes of 2^low to 2^high."""
    return torch.exp2(low + (high - low) * torch.rand(n, generator=g, device=DEV, dtype=torch.float64)).float()


def _pair(g, rows, cin, cout, xr, wr):
    x = bm.Rows8(_int8(g, rows, cin), _scales(g, rows, *xr))
    w = bm.Rows8(_int8(g, cout, cin), _scales(g, cout, *wr))
    x.q[::3] = 0   # whole rows of zeros among them
    return x, w


@pytest.mark.parametrize("rows, cin, cout", FORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_small_scales(rows, cin, cout, dtype):
    """Products of scales from 2^-145 to 2^-120, sums of up to 2^20 and more: ordinary
    results, which 4 to 24 bits of the scales' product would have to make."""
    g = _gen(rows + cout)
    x, w = _pair(g, rows, cin, cout, (-72, -60), (-73, -60))
    ref, S = _fast(x, w, None)
    got = bm.linear8(x, w, dtype=DT[dtype])
    # bf16 results among bf16's subnormals, in steps of 2^-133, are half a step off
    ref, S = ref, S + 2.0 ** ((-134 if dtype == "bf16" else -150) + 22)
    _close("out", got, ref, S, PROD, dtype)


@pytest.mark.parametrize("rows, cin, cout", FORMS)
def test_large_scales(rows, cin, cout):
    """Products of scales beyond 2^128: an empty sum leaves the bias, another one is
    an infinity with the sum's sign."""
    g = _gen(rows + cout + 1)
    x, w = _pair(g, rows, cin, cout, (90, 110), (60, 90))
    b = torch.randn(cout, generator=g, device=DEV)
    ref, _ = _fast(x, w, b)
    with np.errstate(over="ignore"):
        want = ref.astype(np.float32)
    got = bm.linear8(x, w, b, dtype=torch.float32).cpu().numpy()
    assert np.isinf(want).any() and (got[::3] == b.cpu().numpy()).all()
    inf = np.isinf(want)
    assert (got[inf] == want[inf]).all()
    assert np.all(np.abs(got[~inf].astype(np.float64) - ref[~inf]) <= PROD * np.abs(ref[~inf]) + 2.0 ** -150)


def test_scales_of_zero_and_no_number():
    """A scale of zero, as an empty row has it, leaves the bias; a NaN or an infinity
    makes its own row or channel what the definition says, and nothing else."""
    g = _gen(3)
    x = bm.Rows8(_int8(g, 200, 64), torch.rand(200, generator=g, device=DEV) + 0.5)
    w = bm.Rows8(_int8(g, 150, 64), torch.rand(150, generator=g, device=DEV) + 0.5)
    b = torch.randn(150, generator=g, device=DEV)
    clean = bm.linear8(x, w, b, dtype=torch.float32)
    x.scale[5], x.scale[77], x.scale[130] = 0.0, float("nan"), float("inf")
    w.scale[9] = 0.0
    x.q[130, :] = 0
    x.q[130, 0] = 1
    w.q[4, 0] = 0
    got = bm.linear8(x, w, b, dtype=torch.float32)
    rows = [r for r in range(200) if r not in (5, 77, 130)]
    cols = [c for c in range(150) if c not in (4, 9)]
    assert torch.equal(got[rows][:, cols], clean[rows][:, cols])
    assert torch.equal(got[5], b) and torch.equal(got[rows][:, 9], b[9].expand(len(rows)))
    assert torch.isnan(got[77]).all()
    # inf * 0 is no number, inf * q one of q's sign
    s = w.q[:, 0].double()
    s[9] = 0
    assert torch.isnan(got[130][s == 0]).all()
    assert torch.equal(got[130][s != 0], torch.sign(s[s != 0]).float() * float("inf"))


@pytest.mark.parametrize("rows, cin, cout", FORMS)
@pytest.mark.parametrize("bits", [0x7fc00000, 0x7fffffff, 0xffffffff, 0x7f800001, 0xffff8000])
def test_no_number_of_any_bits(rows, cin, cout, bits):
    """A NaN in a bias or a scale, whatever its bits, is a NaN in bf16, too."""
    g = _gen(rows + cin)
    x, w = _pair(g, rows, cin, cout, (-1, 0), (-1, 0))
    b = torch.randn(cout, generator=g, device=DEV)
    clean = bm.linear8(x, w, b)
    nan = torch.tensor(np.array([bits], dtype=np.uint32).view(np.float32), device=DEV)
    b[cout // 2], w.scale[1], x.scale[rows // 3] = nan[0], nan[0], nan[0]
    got = bm.linear8(x, w, b)
    bad = torch.zeros(rows, cout, dtype=torch.bool, device=DEV)
    bad[:, cout // 2], bad[:, 1], bad[rows // 3] = True, True, True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], clean[~bad])

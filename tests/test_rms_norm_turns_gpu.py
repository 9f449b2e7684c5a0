"""RMS norm and 8-bit rows where a workgroup takes several turns of rows, the next
ones fetched ahead, in each way that a row is held; and rows past 2^31 elements
against the oracle. Tolerances as in test_rows8_gpu.py."""
import numpy as np
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
from oracle import rows8 as orows
from test_rows8_gpu import DT, REL, _close, _gen, _np, _randn

pytestmark = pytest.mark.gpu

DEV = "cuda"
# more rows than 2048 workgroups hold at once: 32, 16, 8, 4 and 1 of them a workgroup
MANY = [(140001, 24), (66000, 64), (33001, 65), (33333, 128), (17001, 200), (16500, 256), (8300, 300), (8200, 512),
        (8201, 1000), (4099, 1500), (2500, 2560), (2100, 9000)]


@pytest.mark.parametrize("rows, C", MANY)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("res, rows8, dense", [(False, False, True), (True, True, False), (False, True, True), (True, False, True)])
def test_many_rows(rows, C, dtype, res, rows8, dense):
    g = _gen(rows)
    dt = DT[dtype]
    x, w = _randn(g, rows, C, dtype=dt), _randn(g, C)
    x *= torch.exp(_randn(g, rows, 1)).to(dt)
    r = _randn(g, rows, C, dtype=dt) if res else None
    o = bm.rms_norm(x, w, residual=r, rows8=rows8, dense=dense)
    h = (x.float() + r.float()).to(dt) if res else x
    assert torch.equal(o["sum"], h)
    ref, rstd = orows.rms_norm(h, w, 1e-5)
    _close("rstd", o["rstd"], rstd, rstd, REL)
    if dense:
        _close("out", o["out"], ref, np.abs(ref), REL, dtype)
    if rows8:
        top = np.abs(ref).max(axis=1)
        _close("scale", o["rows8"].scale, top / 127, top / 127, REL)
        q, s = _np(o["rows8"].q), _np(o["rows8"].scale)[:, None]
        assert np.all(np.abs(q - ref / s) <= 0.502) and np.all(np.abs(q).max(axis=1) == 127)
    if rows8 and not res:
        a = bm.rows8_pack(x)
        q, s = orows.rows8(x)
        assert np.array_equal(a.q.cpu().numpy(), q) and np.array_equal(a.scale.cpu().numpy(), s)


@pytest.mark.parametrize("C", [64, 2048])
def test_rows_past_31_bits(C):
    """2^31 elements and more: rows around the ends and around the 2^31st element."""
    rows = (2 ** 31 + 2 ** 22) // C
    x = torch.empty(rows, C, dtype=torch.bfloat16, device=DEV)
    x.normal_(generator=_gen(C))
    w = _randn(_gen(1), C)
    o = bm.rms_norm(x, w, rows8=True, dense=True)
    a = bm.rows8_pack(x)
    mid = 2 ** 31 // C
    at = sorted(set(list(range(70)) + list(range(mid - 70, mid + 70)) + list(range(rows - 70, rows)) + list(range(0, rows, rows // 97))))
    at = torch.tensor(at, device=DEV)
    ref, rstd = orows.rms_norm(x[at], w, 1e-5)
    _close("out", o["out"][at], ref, np.abs(ref), REL, "bf16")
    _close("rstd", o["rstd"][at], rstd, rstd, REL)
    q, s = _np(o["rows8"].q[at]), _np(o["rows8"].scale[at])[:, None]
    assert np.all(np.abs(q - ref / s) <= 0.502)
    q, s = orows.rows8(x[at])
    assert np.array_equal(a.q[at].cpu().numpy(), q) and np.array_equal(a.scale[at].cpu().numpy(), s)

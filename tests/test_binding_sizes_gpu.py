"""Numbers beyond 32 bits are refused by every entry point that takes them
(the low 32 bits of each make a valid call, which is not the one asked for)."""
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm

pytestmark = pytest.mark.gpu

DEV = "cuda"
FAR = 2 ** 32
L, H, P, G, N = 40, 2, 16, 1, 16
CH = H * P + 2 * G * N


def _z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype, device=DEV)


def _scan():
    return dict(x=_z(1, L, H, P), dt=_z(1, L, H), A=_z(H), B=_z(1, L, G, N), C=_z(1, L, G, N), D=_z(H))


def _conv(kept=False):
    x = _z(1, L, CH)
    return dict(xbc=bm.act8_pack(x) if kept else x, weight=_z(CH, 4))


@pytest.mark.parametrize("cu", [[0, FAR + 7, L], [0, 7, FAR + L]], ids=["inner", "last"])
def test_offsets(cu):
    s, c, k, dims = _scan(), _conv(), _conv(True), (H, P, G, N)
    calls = dict(
        ssd_fwd=lambda cu: bm.ssd_fwd(s, s, chunk=64, cu_seqlens=cu),
        ssd_fwd_noalloc=lambda cu: bm.ssd_fwd_noalloc(s, s, _z(1, L, H, P), chunk=64, cu_seqlens=cu),
        ssd_fwd_streams=lambda cu: bm.ssd_fwd_streams(s, s, chunk=64, cu_seqlens=cu),
        conv1d=lambda cu: bm.conv1d(c, c, *dims, cu_seqlens=cu),
        conv1d_act8=lambda cu: bm.conv1d(k, k, *dims, cu_seqlens=cu),
        conv1d_bwd=lambda cu: bm.conv1d_bwd(c, c, s, s, *dims, cu_seqlens=cu),
        seq_index=lambda cu: bm.seq_index(cu))
    for name, call in calls.items():
        print(name, flush=True)
        call([v % FAR for v in cu])
        with pytest.raises(ValueError, match="cu_seqlens.*32 bits"):
            call(cu)


def test_group_size():
    y, w = _z(4, 512), torch.ones(512, device=DEV)
    bm.gated_norm(y, y, w, group_size=256)
    bm.gated_norm_bwd(y, y, y, w, group_size=256)
    for gs in (FAR + 256, 256 - FAR):
        with pytest.raises(ValueError, match="group_size.*32 bits"):
            bm.gated_norm(y, y, w, group_size=gs)
        with pytest.raises(ValueError, match="group_size.*32 bits"):
            bm.gated_norm_bwd(y, y, y, w, group_size=gs)


def test_other_sizes():
    s, c, k = _scan(), _conv(), _conv(True)
    for chunk in (FAR + 64, 64 - FAR):
        for call in (lambda: bm.ssd_fwd(s, s, chunk=chunk), lambda: bm.ssd_fwd_streams(s, s, chunk=chunk),
                     lambda: bm.ssd_fwd_noalloc(s, s, _z(1, L, H, P), chunk=chunk)):
            with pytest.raises(ValueError, match="32 bits"):
                call()
    # head and state sizes that come out at the same number of channels
    far = (2 - FAR, 16, 1, 2 ** 35 + 16)
    assert bm.conv_channels(*far) == CH
    for call in (lambda: bm.conv1d(c, None, *far, out=({k: v for k, v in s.items()}, None)),
                 lambda: bm.conv1d(k, None, *far), lambda: bm.conv1d_bwd(c, None, s, None, *far)):
        with pytest.raises((ValueError, RuntimeError)):
            call()
    st = bm.State(2, H, P, N)
    try:
        st.tensor().fill_(1.0)
        with pytest.raises(ValueError, match="slots.*32 bits"):
            st.reset([FAR + 1])
        st.reset([])
        assert (st.tensor() == 1.0).all()
        st.reset([1])
        torch.cuda.synchronize()
        assert (st.tensor()[0] == 1.0).all() and (st.tensor()[1] == 0.0).all()
    finally:
        st.free()

"""The delta rule's gradient where a workgroup walks several heads of a group, one
after the other: what it loads ahead for the next head's columns of the states
is the next head's, at every width of a head. Against the fp64 oracle; tolerances
as in test_delta_gpu.py."""
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
from oracle import delta as od
from test_delta_gpu import _case, _close, _pair

pytestmark = pytest.mark.gpu

# batch, L, H, P, G, N, dtype, both. With 256 chunks and groups or more all heads of
# a group go to one workgroup, with fewer to as many as have work; heads of one, two,
# three and four times 32 columns (64 of which are a slice where d_state is 128)
FORMS = [(130, 65, 2, 65, 1, 128, "bf16", True), (130, 65, 2, 80, 1, 128, "f32", False),
         (130, 65, 3, 96, 1, 128, "bf16", False), (130, 65, 3, 96, 1, 128, "f32", False),
         (50, 65, 5, 80, 1, 128, "f32", True), (26, 66, 8, 72, 2, 128, "bf16", False),
         (130, 65, 2, 33, 1, 128, "f32", False), (130, 65, 3, 64, 1, 128, "bf16", False),
         (130, 65, 2, 97, 1, 128, "bf16", False), (130, 65, 3, 1, 1, 128, "f32", False),
         (130, 65, 3, 65, 1, 64, "bf16", False), (130, 65, 2, 96, 1, 32, "f32", False),
         (130, 65, 3, 33, 1, 16, "bf16", False)]


@pytest.mark.parametrize("case", FORMS, ids=lambda c: "-".join(map(str, c)))
def test_heads_of_a_group_in_turn(case):
    batch, L, H, P, G, N, dtype, both = case
    dirs, init, df, dy = _case(L * 41 + P + N, *case)
    f, b = _pair(dirs)
    dinit = torch.empty_like(init)
    gf, gb = bm.delta_bwd(f, b, dy, init_state=init, dfinal=df, dinit=dinit)
    ref, rd = od.bwd(dirs, dy, N ** -0.5, None, init, df)
    for got, want, name in zip((gf, gb), ref, ("fwd", "bwd")):
        for n in od.KEYS:
            _close(f"{name} d{n}", got[n], want[n], 2.0, want["gS"] if n == "g" else None)
    _close("dinit", dinit, rd, 2.0)


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("case", [(1, 300, 8, 40, 1, 128, "bf16", True), (2, 130, 12, 33, 2, 32, "f32", True),
                                  (130, 65, 2, 80, 1, 128, "f32", False)], ids=lambda c: "-".join(map(str, c)))
def test_gradients_at_any_element(case, off):
    """Gradient arrays that start at any element, a group's heads in parts and not:
    the bits of aligned ones, and nothing around them."""
    dirs, init, df, dy = _case(case[1] + off, *case)
    f, b = _pair(dirs)
    want = bm.delta_bwd(f, b, dy, init_state=init, dfinal=df)
    bufs, grads = [], []
    for d in dirs:
        one = {}
        for n, t in d.items():
            bufs.append(torch.full((t.numel() + 8,), 7.0, device="cuda"))
            one[n] = bufs[-1][off:off + t.numel()].view(t.shape)
        grads.append(one)
    got = bm.delta_bwd(f, b, dy, init_state=init, dfinal=df, grads=(grads + [None])[:2])
    for g, w in zip(got, want):
        assert w is None or all(torch.equal(g[n], w[n]) for n in od.KEYS)
    for buf in bufs:
        assert (buf[:off] == 7).all() and (buf[off - 8:] == 7).all()

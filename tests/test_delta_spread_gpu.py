"""How far an infinity or a NaN goes in the delta rule's gradient, and one long
sequence against the fp64 oracle (tolerances as in test_delta_gpu.py)."""
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
from oracle import delta as od
from test_delta_gpu import _case, _close, _pair

pytestmark = pytest.mark.gpu

CU = [0, 200, 300]
OWN = ("v", "g", "beta")   # gradients that no other head adds to


def _grads(d, init, df, dy, both):
    dinit = torch.empty_like(init)
    gf, gb = bm.delta_bwd(d[0], d[1] if both else None, dy, cu_seqlens=CU, init_state=init, dfinal=df, dinit=dinit)
    return [gf, gb] if both else [gf], dinit


def _elsewhere(got, want, heads, groups, what):
    """Other heads' and groups' gradients, and the other sequence's."""
    for g, w in zip(got, want):
        for n in od.KEYS:
            a, b = g[n], w[n]
            assert torch.equal(a[:, 200:], b[:, 200:]), (what, n, "the other sequence")
            keep = heads if n in OWN else groups
            assert torch.equal(a[:, :, keep], b[:, :, keep]), (what, n)


@pytest.mark.parametrize("dtype, N, P", [("bf16", 128, 64), ("f32", 64, 40), ("bf16", 16, 128)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_no_number_in_an_input(dtype, N, P, bad):
    """Of 4 heads in 2 groups, head 1's inputs at token 100 of 200."""
    dirs, init, df, dy = _case(31, 1, 300, 4, P, 2, N, dtype, True, 2)
    want, dinit = _grads(dirs, init, df, dy, True)
    for n in od.KEYS:
        for i in range(2):
            d = [dict(x) for x in dirs]
            d[i][n] = d[i][n].clone()
            at = (0, 100, 0, 3) if n in "qk" else (0, 100, 1, 5) if n == "v" else (0, 100, 1)
            d[i][n][at] = bad
            if n == "g" and bad == -float("inf"):
                continue   # a reset, which is a number
            got, di = _grads(d, init, df, dy, True)
            # a query or key is its group's, the rest one head's; the other direction knows nothing of it
            heads = [2, 3] if n in "qk" else [0, 2, 3]
            _elsewhere([got[i]], [want[i]], heads, [1], n)
            assert all(torch.equal(got[1 - i][m], want[1 - i][m]) for m in od.KEYS), n
            assert torch.equal(di[1], dinit[1]) and torch.equal(di[:, heads], dinit[:, heads])
            if i == 1:
                assert torch.equal(di, dinit)
            if n == "v":
                # what reaches a write does not know what is written
                assert torch.equal(got[i]["v"], want[i]["v"]) and torch.equal(di, dinit)
                # nor do the chunks that come before it in the direction's order
                past = slice(0, 64) if i == 0 else slice(136, 200)
                for m in od.KEYS:
                    assert torch.equal(got[i][m][:, past], want[i][m][:, past]), m
            if n == "q":
                # a query's own token alone in dv's and dbeta's past: later tokens' writes are not asked by it
                later = slice(128, 200) if i == 0 else slice(0, 72)
                for m in ("v", "beta"):
                    assert torch.equal(got[i][m][:, later], want[i][m][:, later]), m


@pytest.mark.parametrize("dtype, N, P", [("bf16", 128, 64), ("f32", 64, 40), ("bf16", 16, 128)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_no_number_in_a_gradient(dtype, N, P, bad):
    """dy of head 1, column 5, at token 100: the forward direction's later chunks and
    the reverse one's earlier chunks do not see it."""
    dirs, init, df, dy = _case(32, 1, 300, 4, P, 2, N, dtype, True, 2)
    want, dinit = _grads(dirs, init, df, dy, True)
    e = dy.clone()
    e[0, 100, 1, 5] = bad
    got, di = _grads(dirs, init, df, e, True)
    _elsewhere(got, want, [0, 2, 3], [1], "dy")
    for i, unseen in enumerate((slice(128, 200), slice(0, 72))):
        for m in od.KEYS:
            assert torch.equal(got[i][m][:, unseen], want[i][m][:, unseen]), (i, m)
        cols = [p for p in range(P) if p != 5]
        assert torch.equal(got[i]["v"][..., cols], want[i]["v"][..., cols])
    assert torch.equal(di[1], dinit[1]) and torch.equal(di[:, [0, 2, 3]], dinit[:, [0, 2, 3]])
    f = df.clone()
    f[0, 1, 5, 3] = bad
    got, di = _grads(dirs, init, f, dy, True)
    _elsewhere(got[:1], want[:1], [0, 2, 3], [1], "dfinal")
    assert all(torch.equal(got[1][m], want[1][m]) for m in od.KEYS)


@pytest.mark.parametrize("case", [(1, 12345, 2, 64, 1, 128, "bf16", True), (1, 9000, 1, 40, 1, 32, "f32", False),
                                  (1, 6400, 2, 128, 2, 128, "f32", False)], ids=lambda c: "-".join(map(str, c)))
def test_one_long_sequence(case):
    batch, L, H, P, G, N, dtype, both = case
    dirs, init, df, dy = _case(33, *case)
    f, b = _pair(dirs)
    last, dinit = torch.empty_like(init), torch.empty_like(init)
    y = bm.delta_fwd(f, b, init_state=init, final_state=last)
    ry, rl = od.fwd(dirs, N ** -0.5, None, init)
    _close("y", y, ry)
    _close("last", last, rl)
    gf, gb = bm.delta_bwd(f, b, dy, init_state=init, dfinal=df, dinit=dinit)
    ref, rd = od.bwd(dirs, dy, N ** -0.5, None, init, df)
    for got, want in zip((gf, gb), ref):
        for n in od.KEYS:
            _close("d" + n, got[n], want[n], 2.0, want["gS"] if n == "g" else None)
    _close("dinit", dinit, rd, 2.0)

"""GPU parity of the gated delta rule, its cached step and its gradient against
the fp64 oracle (oracle/delta.py).

Tolerances. fp32 inputs are computed in fp32. A token's step is a product over
N / 8 terms in a lane, three levels over lanes and some ten more roundings: less
than 32 of 2^-24. The transition does not lengthen an error (e^g <= 1, beta
|k|^2 <= 1), so errors add up over the tokens that a state remembers; roundings
are independent, so over T tokens they come to sqrt(32 T) 2^-24 / sqrt(3) of
the magnitudes: with T <= 1024 (the slowest decay here) 105 x 2^-24, bounded by
2^-17 in the 2-norm, and twice as much for a gradient, whose walk back adds its
own: 2^-16. A single element may be off by 2^-11 of the RMS: 64 times more than
the norm's bound, as much as extreme elements and small divisors take.

Operands of the matrix cores are three bf16 terms each, which hold an fp32 whole
(8 bits a term, the rest of a term's rounding going to the next); of the nine
products of two such the three left out are below 3 x 2^-24 of the whole, which
is a rounding more to each of the thirty: the same bars hold with bf16 inputs,
whose single term is exact.

g's gradient is the difference of sums over a chunk (the oracle gives their
size); its error is measured against that size.
"""
import numpy as np
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
from delta_inputs import DT, direction
from oracle import delta as od

pytestmark = pytest.mark.gpu

DEV = "cuda"
NORM, ELEM = 2.0 ** -17, 2.0 ** -11


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(name, got, ref, more=1.0, size=None):
    got = _np(got)
    assert got.shape == ref.shape, name
    if not ref.size:
        return
    size = ref if size is None else size
    norm, rms = np.linalg.norm(size), np.sqrt(np.mean(size ** 2))
    rel, top = np.linalg.norm(got - ref) / max(norm, 1e-300), np.max(np.abs(got - ref)) / max(rms, 1e-300)
    print(f"  {name}: {rel:.2e} of the norm, {top:.2e} of the RMS", flush=True)
    assert rel <= more * NORM and top <= more * ELEM, (name, rel, top)


def _case(seed, batch, L, H, P, G, N, dtype, both, units=None, **kw):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dirs = [direction(g, batch, L, H, P, G, N, dtype, DEV, **kw) for _ in range(2 if both else 1)]
    u = units if units is not None else batch
    init, df = (torch.randn(u, H, P, N, generator=g, device=DEV) for _ in range(2))
    return dirs, init, df, torch.randn(batch, L, H, P, generator=g, device=DEV)


def _pair(dirs):
    return dirs[0], dirs[1] if len(dirs) > 1 else None


# batch, L, H, P, G, N, dtype, both, cu: every head size, lengths around tiles and chunks, shared
# and single groups, odd head widths
CASES = [
    (1, 1, 1, 1, 1, 16, "f32", False, None), (2, 2, 2, 3, 1, 16, "bf16", True, None),
    (1, 15, 3, 16, 3, 32, "f32", True, None), (3, 17, 4, 17, 2, 64, "bf16", False, None),
    (1, 63, 2, 64, 1, 128, "bf16", True, None), (1, 64, 2, 64, 2, 128, "bf16", False, None),
    (2, 65, 4, 40, 2, 32, "f32", True, None), (1, 129, 2, 128, 1, 128, "bf16", True, None),
    (1, 200, 3, 100, 1, 64, "f32", False, None), (2, 300, 2, 33, 1, 16, "bf16", True, None),
    (1, 700, 2, 64, 1, 128, "bf16", False, None), (1, 513, 4, 128, 2, 128, "f32", False, None),
    (1, 90, 2, 24, 1, 32, "bf16", True, [0, 1, 1, 30, 90]), (1, 260, 4, 64, 2, 128, "bf16", True, [0, 64, 129, 130, 260]),
    (1, 333, 2, 40, 1, 64, "f32", True, [0, 0, 63, 127, 333, 333]), (1, 600, 2, 128, 2, 128, "bf16", False, [0, 599, 600]),
    (16, 70, 8, 64, 4, 32, "bf16", False, None), (130, 3, 4, 48, 1, 16, "f32", True, None),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:8])) + ("-packed" if c[8] else ""))
def test_fwd_and_bwd(case):
    batch, L, H, P, G, N, dtype, both, cu = case
    units = len(cu) - 1 if cu else batch
    dirs, init, df, dy = _case(L * 31 + P, batch, L, H, P, G, N, dtype, both, units)
    f, b = _pair(dirs)
    scale = N ** -0.5
    last = torch.full_like(init, 9.0)
    y = bm.delta_fwd(f, b, cu_seqlens=cu, init_state=init, final_state=last)
    ry, rl = od.fwd(dirs, scale, cu, init)
    _close("y", y, ry)
    _close("last", last, rl)
    # without states; in place
    y0 = bm.delta_fwd(f, b, cu_seqlens=cu)
    _close("y from zeros", y0, od.fwd(dirs, scale, cu)[0])
    state = init.clone()
    assert torch.equal(bm.delta_fwd(f, b, cu_seqlens=cu, init_state=state, final_state=state), y)
    assert torch.equal(state, last)
    dinit = torch.full_like(init, 9.0)
    gf, gb = bm.delta_bwd(f, b, dy, cu_seqlens=cu, init_state=init, dfinal=df, dinit=dinit)
    ref, rd = od.bwd(dirs, dy, scale, cu, init, df)
    assert (gb is None) == (b is None)
    for got, want, name in zip((gf, gb), ref, ("fwd", "bwd")):
        for n in od.KEYS:
            _close(f"{name} d{n}", got[n], want[n], 2.0, want["gS"] if n == "g" else None)
    _close("dinit", dinit, rd, 2.0)
    if L > 1:
        # without states: again the same bits as with zeros
        zero = torch.zeros_like(init)
        g0 = bm.delta_bwd(f, b, dy, cu_seqlens=cu)
        g1 = bm.delta_bwd(f, b, dy, cu_seqlens=cu, init_state=zero, dfinal=zero)
        for a, c in zip(g0, g1):
            assert a is None or all(torch.equal(a[n], c[n]) for n in od.KEYS)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H, P, G, N", [(4, 64, 2, 128), (2, 128, 1, 64), (3, 20, 3, 16), (8, 128, 4, 128)])
def test_step_by_step_is_the_whole(dtype, H, P, G, N):
    """Tokens, then blocks, from a cached state, against the whole sequence."""
    L = 150
    dirs, init, _, _ = _case(5, 2, L, H, P, G, N, dtype, False)
    f = dirs[0]
    ry, rl = od.fwd(dirs, N ** -0.5, None, init)
    st = bm.State(3, H, P, N)
    try:
        st.tensor().zero_()
        st.tensor()[:2].copy_(init)
        at, ys = 0, []
        for n in [1, 1, 1, 5, 16, 64, 1, 33, 28]:
            cut = {k: t[:, at:at + n].contiguous() for k, t in f.items()}
            before = st.tensor().clone()
            y0 = bm.delta_step(st, cut, commit=False)
            assert torch.equal(st.tensor(), before)
            ys.append(bm.delta_step(st, cut))
            assert torch.equal(ys[-1], y0)
            at += n
        assert at == L
        _close("y", torch.cat(ys, dim=1), ry)
        _close("state", st.tensor()[:2], rl)
        assert (st.tensor()[2] == 0).all()
    finally:
        st.free()


@pytest.mark.parametrize("L", [1, 30, 64, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_step_both_directions(L, dtype):
    dirs, init, _, _ = _case(6, 2, L, 4, 64, 2, 128, dtype, True)
    state = init.clone()
    y = bm.delta_step(state, *dirs, commit=False, scale=0.25)
    ry, rl = od.fwd(dirs, 0.25, None, init)
    _close("y", y, ry)
    assert torch.equal(state, init)
    assert torch.equal(bm.delta_step(state, *dirs, scale=0.25), y)
    _close("state", state, rl)


# ---- values at the edges -----------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_resets_and_closed_gates(dtype):
    """Decays that reset the state (-inf, far below what fp32 tells from it),
    tokens that do nothing, long runs without decay."""
    batch, L, H, P, G, N = 1, 400, 4, 64, 2, 128
    dirs, init, df, dy = _case(7, batch, L, H, P, G, N, dtype, False)
    d = dirs[0]
    d["g"][0, 70, 0] = -float("inf")
    d["g"][0, 71, 1] = -1e30
    d["g"][0, 130:140, 2] = -300.0
    d["g"][0, :, 3] = 0.0
    d["beta"][0, 200:330, 1] = 0.0
    d["beta"][0, 150, 0] = 0.0
    last = torch.empty_like(init)
    y = bm.delta_fwd(d, init_state=init, final_state=last)
    ry, rl = od.fwd(dirs, N ** -0.5, None, init)
    _close("y", y, ry)
    _close("last", last, rl)
    gf, _ = bm.delta_bwd(d, None, dy, init_state=init, dfinal=df)
    # the oracle's e^-inf times a finite state is the zero it should be
    ref, _ = od.bwd(dirs, dy, N ** -0.5, None, init, df)
    for n in od.KEYS:
        _close("d" + n, gf[n], ref[0][n], 2.0, ref[0]["gS"] if n == "g" else None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_values_and_equal_keys(dtype):
    """Values beyond what half precision holds, states and errors of 1e30, and a
    chunk whose keys are all the same (every entry of its triangle large)."""
    dirs, init, _, _ = _case(8, 1, 200, 4, 64, 2, 128, dtype, False, alike=30.0)
    d = dirs[0]
    d["v"][..., 0, :] *= 1e30
    d["v"][..., 1, :] *= 1e5
    d["v"][..., 2, :] *= 1e-30
    init = init * torch.tensor([1e30, 1e5, 1e-30, 1.0], device=DEV).reshape(1, 4, 1, 1)
    last = torch.empty_like(init)
    y = bm.delta_fwd(d, init_state=init, final_state=last)
    ry, rl = od.fwd(dirs, 128 ** -0.5, None, init)
    for h in range(4):
        _close(f"y {h}", y[:, :, h], ry[:, :, h])
        _close(f"last {h}", last[:, h], rl[:, h])


def test_no_number_stays_in_its_head_and_future():
    """A NaN or an infinity in a value spoils its column from its token on, and
    no other column, head, sequence or earlier chunk."""
    dirs, init, _, _ = _case(9, 1, 300, 4, 64, 2, 128, "bf16", False, 2)
    d, cu = dirs[0], [0, 200, 300]
    clean = bm.delta_fwd(d, cu_seqlens=cu, init_state=init)
    for bad in (float("nan"), float("inf")):
        e = dict(d, v=d["v"].clone())
        e["v"][0, 100, 1, 5] = bad
        y = bm.delta_fwd(e, cu_seqlens=cu, init_state=init)
        other = [0, 2, 3]
        assert torch.equal(y[:, :, other], clean[:, :, other]) and torch.equal(y[:, 200:], clean[:, 200:])
        col = [p for p in range(64) if p != 5]
        assert torch.equal(y[:, :, 1][:, :, col], clean[:, :, 1][:, :, col])
        assert torch.equal(y[:, :64], clean[:, :64])   # the chunks before
        assert not torch.isfinite(y[0, 100:200, 1, 5]).any()


def test_no_token():
    dirs, init, df, _ = _case(10, 2, 0, 2, 16, 1, 16, "bf16", False)
    d = dirs[0]
    last = torch.empty_like(init)
    assert bm.delta_fwd(d, init_state=init, final_state=last).shape == (2, 0, 2, 16)
    assert torch.equal(last, init)
    bm.delta_fwd(d, final_state=last)
    assert (last == 0).all()
    dinit = torch.empty_like(init)
    gf, _ = bm.delta_bwd(d, None, torch.empty(2, 0, 2, 16, device=DEV), dfinal=df, dinit=dinit)
    assert torch.equal(dinit, df) and gf["q"].shape == (2, 0, 1, 16)
    y = bm.delta_fwd({n: t[:1] for n, t in d.items()}, cu_seqlens=[0, 0, 0], init_state=init, final_state=last)
    assert y.shape == (1, 0, 2, 16) and torch.equal(last, init)


def test_what_lies_around():
    """Nothing but the results is written."""
    batch, L, H, P, G, N = 1, 150, 2, 40, 1, 32
    dirs, init, df, dy = _case(11, batch, L, H, P, G, N, "bf16", False)
    n = L * H * P
    buf = torch.full((n + 8,), 7.0, device=DEV)
    bm.delta_fwd(dirs[0], y=buf[4:-4].view(batch, L, H, P))
    grads, bufs = {}, []
    for k, t in dirs[0].items():
        b = torch.full((t.numel() + 8,), 7.0, device=DEV)
        bufs.append(b)
        grads[k] = b[4:-4].view(t.shape)
    for size in (bm.delta_bwd_workspace_size(dirs[0]),):
        ws = torch.full((size + 256,), 55, dtype=torch.uint8, device=DEV)
        bm.delta_bwd(dirs[0], None, dy, grads=(grads, None), workspace=ws[:size])
        assert (ws[size:] == 55).all()
    for b in bufs + [buf]:
        assert (b[:4] == 7).all() and (b[-4:] == 7).all() and torch.isfinite(b).all()


def test_gradient_by_differences():
    """Along random directions, against differences of the oracle's forward."""
    dirs, init, df, dy = _case(12, 1, 100, 2, 20, 1, 16, "f32", False)
    d = dirs[0]
    dinit = torch.empty_like(init)
    gf, _ = bm.delta_bwd(d, None, dy, scale=0.3, init_state=init, dfinal=df, dinit=dinit)
    x = {n: _np(t) for n, t in dict(d, init=init).items()}

    def loss(v):
        e = {n: torch.tensor(v[n]) for n in od.KEYS}
        y, last = od.fwd([e], 0.3, None, torch.tensor(v["init"]))
        return (y * _np(dy)).sum() + (last * _np(df)).sum()
    r = np.random.default_rng(2)
    for n, got in list(gf.items()) + [("init", dinit)]:
        u = r.normal(size=x[n].shape)
        h = 1e-5
        num = (loss(dict(x, **{n: x[n] + h * u})) - loss(dict(x, **{n: x[n] - h * u}))) / (2 * h)
        terms = _np(got) * u
        assert abs(num - terms.sum()) <= 1e-4 * np.sqrt((terms ** 2).sum()), n


# ---- together, captured, on streams ------------------------------------------------

def _layer(x, p, cu=None):
    """A delta-rule mixer in 8 bits: norm, projection, convolution, delta rule both
    ways, gated norm, projection back."""
    H, P, G, N = p["dims"]
    n = bm.rms_norm(x, p["norm"], rows8=True)
    wide = bm.linear8(n["rows8"], p["wi"])
    xbc = wide[..., :H * P + 2 * G * N].contiguous()
    conv = dict(xbc=xbc, weight=p["conv"], bias=None)
    fo, bo = bm.conv1d(conv, conv, H, P, G, N, cu_seqlens=cu)
    gates = wide[..., H * P + 2 * G * N:].float()
    dirs = []
    for o in (fo, bo):
        q, k = (torch.nn.functional.normalize(o[c].float(), dim=-1).to(x.dtype) for c in "CB")
        dirs.append(dict(q=q, k=k, v=o["x"], g=-torch.nn.functional.softplus(gates[..., :H]) * 0.1,
                         beta=torch.sigmoid(gates[..., H:2 * H].contiguous())))
    y = bm.delta_fwd(*dirs, cu_seqlens=cu)
    z = wide[..., :H * P].contiguous()
    out = bm.gated_norm(y.flatten(2).contiguous(), z, p["gate"])
    return bm.linear8(bm.rows8_pack(out), p["wo"]), dirs, y


def test_a_mixer_layer():
    g = torch.Generator(device=DEV).manual_seed(20)
    H, P, G, N, D = 4, 64, 2, 128, 256
    ch = H * P + 2 * G * N

    def r(*shape):
        return torch.randn(*shape, generator=g, device=DEV)
    p = dict(dims=(H, P, G, N), norm=r(D), wi=bm.rows8_pack(r(ch + 2 * H, D) / 16), conv=r(ch, 4), gate=r(H * P),
             wo=bm.rows8_pack(r(D, H * P)))
    x = r(1, 210, D).to(torch.bfloat16)
    cu = [0, 100, 210]
    out, dirs, y = _layer(x, p, cu)
    assert out.shape == (1, 210, D) and torch.isfinite(out).all()
    _close("y", y, od.fwd(dirs, N ** -0.5, cu)[0])
    dy = r(1, 210, H, P)
    gf, gb = bm.delta_bwd(*dirs, dy, cu_seqlens=cu)
    ref, _ = od.bwd(dirs, dy, N ** -0.5, cu)
    for got, want in zip((gf, gb), ref):
        for n in od.KEYS:
            _close("d" + n, got[n], want[n], 2.0, want["gS"] if n == "g" else None)
    # what the convolution's gradient takes, as it is
    conv = dict(xbc=r(1, 210, ch).to(torch.bfloat16), weight=p["conv"], bias=None)
    grads = [dict(x=t["v"], B=t["k"], C=t["q"]) for t in (gf, gb)]
    cf, cb = bm.conv1d_bwd(conv, dict(conv), *grads, H, P, G, N, cu_seqlens=cu)
    assert torch.isfinite(cf["xbc"]).all() and torch.isfinite(cb["xbc"]).all()


@pytest.mark.parametrize("cu", [None, [0, 70, 140]])
def test_graph_replays_and_streams(cu):
    """Captured twice, replayed in turn with eager work between; on a stream of
    its own; two streams at once."""
    shape = (1, 140, 4, 64, 2, 128, "bf16", True)
    dirs, init, df, dy = _case(13, *shape, units=2 if cu else 1)
    state = init.clone()

    def call():
        last = torch.empty_like(init)
        y = bm.delta_fwd(*dirs, cu_seqlens=cu, init_state=init, final_state=last)
        gf, gb = bm.delta_bwd(*dirs, dy, cu_seqlens=cu, init_state=init, dfinal=df)
        return [y, last] + [t for d in (gf, gb) for t in d.values()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = call()
        graphs.append((gr, out))
    for i in range(3):
        fresh = _case(50 + i, *shape, units=2 if cu else 1)[0]
        for d, f in zip(dirs, fresh):
            for n in d:
                d[n].copy_(f[n])
        want = call()
        for gr, out in graphs:
            gr.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))
        torch.ones(1000, device=DEV).sum().item()
    want = [t.clone() for t in want]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    res = [(bm.delta_fwd(*dirs, cu_seqlens=cu, init_state=init, stream=s),
            bm.delta_bwd(*dirs, dy, cu_seqlens=cu, init_state=init, dfinal=df, stream=s)) for s in streams * 2]
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for y, (gf, gb) in res:
        assert all(torch.equal(a, b) for a, b in zip([y] + [t for d in (gf, gb) for t in d.values()], [want[0]] + want[2:]))
    if cu is None:
        s = streams[0]
        y = bm.delta_step(state, *dirs, commit=True, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(y, want[0]) and torch.equal(state, want[1])


def test_wrong_calls():
    dirs, init, df, dy = _case(14, 2, 10, 2, 16, 1, 16, "bf16", True)
    f, b = dirs
    for kw, err in ((dict(init_state=init[:1]), ValueError), (dict(final_state=init.double()), TypeError),
                    (dict(y=dy.double()), TypeError), (dict(init_state=init.cpu()), ValueError)):
        with pytest.raises(err):
            bm.delta_fwd(f, b, **kw)
    for name, t in (("q", f["q"].float()), ("v", f["v"][:, :9]), ("g", f["g"].to(torch.bfloat16)),
                    ("beta", f["beta"][..., :1]), ("k", f["k"].expand(2, 10, 1, 16)[:, ::1].transpose(0, 1))):
        with pytest.raises((TypeError, ValueError)):
            bm.delta_fwd(dict(f, **{name: t}), b)
    with pytest.raises(ValueError):
        bm.delta_step(init[:1], f)
    with pytest.raises(bm.BimambaError, match="batch == 1"):
        bm.delta_fwd(f, b, cu_seqlens=[0, 10])
    with pytest.raises(bm.BimambaError, match="overlaps"):
        bm.delta_bwd(f, b, dy, init_state=init, dinit=init)
    with pytest.raises(TypeError):
        bm.delta_fwd({k: t.half() if t.dtype == torch.bfloat16 else t for k, t in f.items()})

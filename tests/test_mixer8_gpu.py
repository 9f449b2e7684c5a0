"""The delta rule and the 8-bit product over the forms that a call's sizes choose
(widths of tiles, directions side by side or one after the other, a head's
columns in one workgroup or two, a group's heads in parts), from several threads
at once, and on arrays of more than 2^31 elements. Tolerances as in
test_delta_gpu.py and test_rows8_gpu.py: a form changes the order of additions
alone, of parts of a group's heads, within what is counted there."""
import threading

import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
from delta_inputs import direction
from oracle import delta as od
from test_delta_gpu import _case, _close, _pair
from test_rows8_gpu import PROD, _close as _close8, _fast, _gen, _int8

pytestmark = pytest.mark.gpu

DEV = "cuda"

# rows, cout: tiles 224, 256, 160 and 192 channels wide, then two and three times
# 16 channels a workgroup of few rows
WIDE = [(7213, 1558), (7213, 1817), (7213, 2076), (8718, 1299)]
FEW = [(33, 5000), (64, 8203), (40, 9001), (64, 12289), (48, 4096), (64, 4097)]


@pytest.mark.parametrize("rows, cout", WIDE + FEW)
@pytest.mark.parametrize("cin, dtype", [(16, torch.float32), (64, torch.bfloat16), (208, torch.float32),
                                        (336, torch.bfloat16), (1040, torch.bfloat16)])
def test_linear8_widths(rows, cout, cin, dtype):
    g = _gen(rows + cin + cout)
    x = bm.Rows8(_int8(g, rows, cin), torch.rand(rows, generator=g, device=DEV))
    w = bm.Rows8(_int8(g, cout, cin), torch.rand(cout, generator=g, device=DEV))
    b = torch.randn(cout, generator=g, device=DEV)
    buf = torch.full((rows * cout + 8,), 5.0, dtype=dtype, device=DEV)
    out = bm.linear8(x, w, b, out=buf[4:-4].view(rows, cout))
    torch.cuda.synchronize()
    assert (buf[:4] == 5).all() and (buf[-4:] == 5).all()
    ref, S = _fast(x, w, b)
    _close8("out", out, ref, S, PROD, "bf16" if dtype == torch.bfloat16 else "f32")


# batch, L, H, P, G, N, dtype, both, cu: more heads and rows than half the CUs (a
# workgroup to a wide head, one direction after the other), then groups whose heads
# go to parts, evenly and not, and to one
FORMS = [(70, 70, 2, 128, 1, 128, "bf16", True, None), (70, 70, 2, 100, 1, 128, "f32", True, None),
         (44, 130, 3, 128, 1, 64, "bf16", False, None), (44, 66, 3, 72, 3, 16, "f32", True, None),
         (44, 66, 3, 97, 1, 32, "bf16", True, None), (33, 200, 4, 127, 2, 128, "bf16", True, None),
         (130, 65, 2, 40, 2, 128, "bf16", False, None), (130, 65, 1, 64, 1, 128, "f32", True, None),
         (8, 300, 20, 16, 1, 16, "f32", True, None), (1, 300, 7, 64, 1, 128, "bf16", True, None),
         (2, 130, 12, 48, 2, 32, "bf16", True, None), (1, 64, 40, 8, 1, 64, "bf16", False, None),
         (64, 200, 2, 128, 1, 128, "bf16", True, None), (64, 70, 2, 128, 2, 32, "f32", True, None)]


@pytest.mark.parametrize("case", FORMS, ids=lambda c: "-".join(map(str, c[:8])))
def test_delta_forms(case):
    batch, L, H, P, G, N, dtype, both, cu = case
    dirs, init, df, dy = _case(L * 37 + P, batch, L, H, P, G, N, dtype, both)
    f, b = _pair(dirs)
    scale = N ** -0.5
    last, dinit = torch.empty_like(init), torch.empty_like(init)
    y = bm.delta_fwd(f, b, init_state=init, final_state=last)
    ry, rl = od.fwd(dirs, scale, cu, init)
    _close("y", y, ry)
    _close("last", last, rl)
    gf, gb = bm.delta_bwd(f, b, dy, init_state=init, dfinal=df, dinit=dinit)
    ref, rd = od.bwd(dirs, dy, scale, cu, init, df)
    for got, want, name in zip((gf, gb), ref, ("fwd", "bwd")):
        for n in od.KEYS:
            _close(f"{name} d{n}", got[n], want[n], 2.0, want["gS"] if n == "g" else None)
    _close("dinit", dinit, rd, 2.0)
    # a direction alone, whichever form it takes, and the same bits again
    again = bm.delta_bwd(f, b, dy, init_state=init, dfinal=df)
    for a, c in zip((gf, gb), again):
        assert a is None or all(torch.equal(a[n], c[n]) for n in od.KEYS)
    if both:
        alone = bm.delta_bwd(f, None, dy, init_state=init, dfinal=df)[0]
        assert all(torch.equal(alone[n], gf[n]) for n in od.KEYS)


@pytest.mark.parametrize("each", [1, 20, 40])
def test_hundreds_of_sequences(each):
    """Offsets beyond one launch's table, empty sequences among them: against the
    same rows as a batch."""
    S, H, P, N = 600, 2, 24, 32
    g = torch.Generator(device=DEV).manual_seed(each)
    dirs = [direction(g, S, each, H, P, 1, N, "bf16", DEV) for _ in range(2)]
    init, df = (torch.randn(S + 50, H, P, N, generator=g, device=DEV) for _ in range(2))
    dy = torch.randn(S, each, H, P, generator=g, device=DEV)
    cu, full = [0], []
    for s in range(S + 50):
        empty = s % 13 == 12
        cu.append(cu[-1] + (0 if empty else each))
        if not empty:
            full.append(s)
    assert cu[-1] == S * each and len(full) == S
    flat = [{n: t.flatten(0, 1)[None].contiguous() for n, t in d.items()} for d in dirs]
    last, dinit = torch.empty_like(init), torch.empty_like(init)
    blast = torch.empty_like(init[full])
    bdinit = torch.empty_like(blast)
    y = bm.delta_fwd(*flat, cu_seqlens=cu, init_state=init, final_state=last)
    gf, gb = bm.delta_bwd(*flat, dy.flatten(0, 1)[None].contiguous(), cu_seqlens=cu, init_state=init, dfinal=df, dinit=dinit)
    ry, rl = od.fwd(dirs, N ** -0.5, None, init[full])
    _close("y", y.view(dy.shape), ry)
    _close("last", last[full], rl)
    bf, bb = bm.delta_bwd(*dirs, dy, init_state=init[full].contiguous(), dfinal=df[full].contiguous(), dinit=bdinit)
    for got, want in zip((gf, gb), (bf, bb)):
        for n in od.KEYS:
            assert torch.equal(got[n].view(want[n].shape), want[n]), n
    assert torch.equal(dinit[full], bdinit)
    empty = [s for s in range(S + 50) if s not in set(full)]
    assert torch.equal(last[empty], init[empty]) and torch.equal(dinit[empty], df[empty])


# ---- several threads at once ---------------------------------------------------------

THREADS, TURNS = 4, 10


def _thread_inputs(i):
    """Other sizes in every thread."""
    g = torch.Generator(device=DEV).manual_seed(300 + i)
    L, H, P, N, C = 100 + 61 * i, 2 + i, 16 * (1 + i), 32, 128 * (1 + i)
    dirs = [direction(g, 1, L, H, P, 1, N, "bf16", DEV) for _ in range(2)]
    x, w = torch.randn(L, C, generator=g, device=DEV).bfloat16(), torch.randn(C, generator=g, device=DEV)
    wide = bm.rows8_pack(torch.randn(300 + i, C, generator=g, device=DEV))
    state = torch.randn(1, H, P, N, generator=g, device=DEV)
    dy = torch.randn(1, L, H, P, generator=g, device=DEV)
    return x, w, wide, dirs, state, dy, [0, 31, 31, L] if i % 2 else None


def _thread_step(x, w, wide, dirs, state, dy, cu):
    n = bm.rms_norm(x, w, residual=x, rows8=True)
    out = [n["sum"], n["rstd"], n["rows8"].q, n["rows8"].scale, bm.linear8(n["rows8"], wide)]
    out += list(bm.rms_norm_bwd(x, n["sum"], n["rstd"], w, dsum=x))
    cached = state.clone()
    out += [bm.delta_step(cached, {k: t[:, :9].contiguous() for k, t in dirs[0].items()}), cached]
    out.append(bm.delta_fwd(*dirs, cu_seqlens=cu))
    for d in bm.delta_bwd(*dirs, dy, cu_seqlens=cu):
        out += list(d.values())
    return out


def test_threads():
    ins = [_thread_inputs(i) for i in range(THREADS)]
    want = [_thread_step(*a) for a in ins]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(THREADS, timeout=60)

    def work(i):
        try:
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                start.wait()
                for turn in range(TURNS):
                    got = _thread_step(*ins[i])
                    try:   # the library's message is this thread's own
                        bm.rms_norm(torch.zeros(2, 4 + i, device=DEV))
                        bad.append((i, "not refused"))
                    except bm.BimambaError as e:
                        if f"channels {4 + i} " not in str(e):
                            bad.append((i, str(e)))
                    side.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        bad.append((i, turn))
        except Exception as e:   # a failure in a thread is the test's
            bad.append((i, repr(e)))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(THREADS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(100)
        assert not t.is_alive()
    assert not bad, bad[:5]


def test_state_elsewhere_or_freed():
    """A State of another device, or one that was freed, is refused."""
    d = direction(torch.Generator(device=DEV).manual_seed(0), 1, 1, 2, 16, 1, 16, "f32", DEV)
    st = bm.State(1, 2, 16, 16)
    st.reset()
    bm.delta_step(st, d)
    here, st.device = st.device, torch.device("cuda", 7)
    with pytest.raises(ValueError, match="state is on cuda:7"):
        bm.delta_step(st, d)
    st.device = here
    st.free()
    with pytest.raises(bm.BimambaError, match="state is NULL"):
        bm.delta_step(st, d)


def test_no_number_in_queries_and_gates():
    """Spoils the group's or head's chunk and what follows it; nothing else."""
    dirs, init, _, _ = _case(61, 1, 300, 4, 32, 2, 64, "f32", False, 2)
    d, cu = dirs[0], [0, 210, 300]
    clean = bm.delta_fwd(d, cu_seqlens=cu, init_state=init)
    for name, heads in (("q", [0, 1]), ("k", [0, 1]), ("g", [0]), ("beta", [0])):
        for bad in (float("nan"), float("inf")):
            e = dict(d, **{name: d[name].clone()})
            e[name][0, 100, 0] = bad
            y = bm.delta_fwd(e, cu_seqlens=cu, init_state=init)
            others = [h for h in range(4) if h not in heads]
            assert torch.equal(y[:, :, others], clean[:, :, others]), name
            assert torch.equal(y[:, 210:], clean[:, 210:]) and torch.equal(y[:, :64], clean[:, :64]), name
            assert not torch.isfinite(y[0, 100, heads]).all(), name


# ---- arrays beyond 32 bits of elements --------------------------------------------------

def test_rows_beyond_31_bits():
    """The last rows of a long array are what they are alone."""
    C, rows = 4096, 2 ** 19 + 1000
    x = torch.empty(rows, C, dtype=torch.bfloat16, device=DEV)
    g = _gen(1)
    x[:3], x[3:-700] = 1.0, 0.5
    x[-700:] = torch.randn(700, C, generator=g, device=DEV).bfloat16()
    w = torch.randn(C, generator=g, device=DEV)
    o = bm.rms_norm(x, w, rows8=True, dense=True)
    tail = x[-700:].clone()
    t = bm.rms_norm(tail, w, rows8=True, dense=True)
    assert torch.equal(o["out"][-700:], t["out"]) and torch.equal(o["rstd"][-700:], t["rstd"])
    assert torch.equal(o["rows8"].q[-700:], t["rows8"].q) and torch.equal(o["rows8"].scale[-700:], t["rows8"].scale)
    p = bm.rows8_pack(x)
    assert torch.equal(p.q[-700:], bm.rows8_pack(tail).q)
    dx, _ = bm.rms_norm_bwd(o["out"], x, o["rstd"], w)
    assert torch.equal(dx[-700:], bm.rms_norm_bwd(t["out"], tail, t["rstd"], w)[0])
    few = bm.rows8_pack(torch.randn(4200, 64, generator=g, device=DEV))
    x8 = bm.Rows8(p.q.view(-1)[-64 * rows:].view(rows, 64), p.scale)
    y = bm.linear8(x8, few)
    assert y.numel() > 2 ** 31
    assert torch.equal(y[-300:], bm.linear8(bm.Rows8(x8.q[-300:].clone(), x8.scale[-300:].clone()), few))
    assert torch.equal(y[:300], bm.linear8(bm.Rows8(x8.q[:300].clone(), x8.scale[:300].clone()), few))


def test_states_beyond_31_bits():
    batch, H, P, N = 4100, 32, 128, 128
    g = torch.Generator(device=DEV).manual_seed(3)
    state = torch.zeros(batch, H, P, N, device=DEV)
    assert state.numel() > 2 ** 31
    state[-3:] = torch.randn(3, H, P, N, generator=g, device=DEV)
    few = state[-3:].clone()
    for L in (1, 20):
        d = direction(g, batch, L, H, P, 4, N, "bf16", DEV)
        y = bm.delta_step(state, d)
        ty = bm.delta_step(few, {n: t[-3:].clone() for n, t in d.items()})
        assert torch.equal(y[-3:], ty) and torch.equal(state[-3:], few), L


def test_tokens_beyond_31_bits():
    """Forward and back; the kept states and their gradients are beyond it too."""
    batch, L, H, P, G, N = 9, 60000, 32, 128, 2, 128
    g = torch.Generator(device=DEV).manual_seed(4)
    d = {n: t.expand(batch, *t.shape[1:]).contiguous() for n, t in direction(g, 1, L, H, P, G, N, "bf16", DEV).items()}
    d["v"][-1] *= 2.0
    assert d["v"].numel() > 2 ** 31
    y = bm.delta_fwd(d)
    one = {n: t[-1:].clone() for n, t in d.items()}
    assert torch.equal(y[-1:], bm.delta_fwd(one))
    gf, _ = bm.delta_bwd(d, None, y)
    last = y[-1:].clone()
    del y
    ref, _ = bm.delta_bwd(one, None, last)
    for n in od.KEYS:
        assert torch.equal(gf[n][-1:], ref[n]), n

"""The stream argument: whatever a call allocates, results and workspaces,
belongs to the stream it runs on (a workspace of the current stream would be
given to that stream's next allocation while the other stream still uses it),
and results stay safe to use on the caller's stream."""
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm

pytestmark = pytest.mark.gpu

DEV = "cuda"
BATCH, L, H, P, G, N = 1, 300, 4, 16, 1, 16
CH = H * P + 2 * G * N
CU = [0, 40, 40, 211, L]


def _inputs():
    g = torch.Generator(device=DEV).manual_seed(1)

    def r(*shape):
        return torch.randn(*shape, generator=g, device=DEV)
    scan = [dict(x=r(BATCH, L, H, P), dt=r(BATCH, L, H).abs() * 0.1, A=-r(H).abs(), B=r(BATCH, L, G, N),
                 C=r(BATCH, L, G, N), D=r(H)) for _ in range(2)]
    conv = [dict(xbc=r(BATCH, L, CH), weight=r(CH, 4), bias=r(CH)) for _ in range(2)]
    x, res, z = r(L, 512), r(L, 512), r(L, 512)
    return scan, conv, x, res, z, torch.ones(512, device=DEV), r(BATCH, L, H, P), \
        r(32, 1024).to(torch.bfloat16)


def _calls():
    (f, b), (cf, cb), x, res, z, w, dy, mw = _inputs()
    dims = (H, P, G, N)
    kept = [dict(d, xbc=bm.act8_pack(d["xbc"])) for d in (cf, cb)]
    n = bm.layer_norm(x, w, residual=res, checkpoint=True)
    x8, z8 = bm.act8_pack(x), bm.act8_pack(z)
    y = torch.zeros(BATCH, L, H, P, device=DEV)
    many = list(range(0, 200)) + [L]   # more sequences than go by value: a table in the workspace
    return dict(
        ssd_fwd=lambda s: bm.ssd_fwd(f, b, chunk=64, cu_seqlens=CU, stream=s),
        ssd_fwd_noalloc=lambda s: bm.ssd_fwd_noalloc(f, b, y, chunk=64, cu_seqlens=CU, stream=s),
        ssd_fwd_streams=lambda s: bm.ssd_fwd_streams(f, b, chunk=64, cu_seqlens=CU, stream=s),
        ssd_bwd=lambda s: bm.ssd_bwd(f, b, dy, stream=s),
        merge_linear=lambda s: bm.merge_linear(x, res, mw, stream=s),
        conv1d=lambda s: bm.conv1d(cf, cb, *dims, cu_seqlens=CU, stream=s),
        conv1d_act8=lambda s: bm.conv1d(kept[0], kept[1], *dims, cu_seqlens=many, stream=s),
        conv1d_bwd=lambda s: bm.conv1d_bwd(cf, cb, f, b, *dims, cu_seqlens=many, stream=s),
        gated_norm=lambda s: bm.gated_norm(x, z, w, stream=s),
        gated_norm_bwd=lambda s: bm.gated_norm_bwd(x, x8, z8, w, stream=s),
        act8_pack=lambda s: bm.act8_pack(x, stream=s),
        act8_unpack=lambda s: bm.act8_unpack(x8, stream=s),
        layer_norm=lambda s: bm.layer_norm(x, w, residual=res, checkpoint=True, stream=s),
        layer_norm_bwd=lambda s: bm.layer_norm_bwd(x, n["ckpt"], n["mean"], n["rstd"], w, stream=s),
        seq_index=lambda s: bm.seq_index(CU, stream=s),
    )


@pytest.mark.parametrize("name", sorted(["ssd_fwd", "ssd_fwd_noalloc", "ssd_fwd_streams", "ssd_bwd", "merge_linear",
                                         "conv1d", "conv1d_act8", "conv1d_bwd", "gated_norm", "gated_norm_bwd",
                                         "act8_pack", "act8_unpack", "layer_norm", "layer_norm_bwd", "seq_index"]))
def test_allocations_belong_to_the_stream(name, monkeypatch):
    print(name, flush=True)
    call = _calls()[name]
    want = bm._tensors(call(None))
    want = [t.clone() for t in want]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    streams = []
    for f in ("empty", "empty_like"):
        make = getattr(torch, f)

        def spy(*a, make=make, **kw):
            streams.append(torch.cuda.current_stream().cuda_stream)
            return make(*a, **kw)
        monkeypatch.setattr(torch, f, spy)
    got = bm._tensors(call(side))
    monkeypatch.undo()
    assert torch.cuda.current_stream() != side
    assert all(s == side.cuda_stream for s in streams)
    assert streams or name == "ssd_fwd_noalloc"
    side.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_block_steps_on_a_stream():
    (f, b), (cf, cb), *_ = _inputs()
    f, b = [dict(d, **{k: d[k][:, :64].contiguous() for k in ("x", "dt", "B", "C")}) for d in (f, b)]
    cf, cb = [dict(d, xbc=d["xbc"][:, :64].contiguous()) for d in (cf, cb)]
    side = torch.cuda.Stream()
    st = bm.State(BATCH, H, P, N)
    sc = bm.State(BATCH, H, P, N, conv=(G, 4, torch.float32))
    try:
        st.tensor().normal_()
        sc.tensor().copy_(st.tensor())
        sc.ctx_tensor().zero_()
        want = bm.block_step(st, f, b), bm.block_step_conv(sc, f, b, cf, cb)
        torch.cuda.synchronize()
        plan = bm.BlockStepPlan(st, f, b, stream=side)
        got = [bm.block_step(st, f, b, stream=side), bm.block_step_conv(sc, f, b, cf, cb, stream=side), plan.run()]
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[0])
    finally:
        torch.cuda.synchronize()
        st.free()
        sc.free()


def test_results_outlive_their_use_on_the_callers_stream():
    """A result dropped while the caller's stream still reads it: its memory is
    not the side stream's next allocation."""
    *_, x, res, z, w, dy, mw = _inputs()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = bm.gated_norm(x, z, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(20_000_000)
    read = y.clone()
    at, want = y.data_ptr(), bm.gated_norm(x, z, w)
    del y
    with torch.cuda.stream(side):
        other = [torch.full((L, 512), 7.0, device=DEV) for _ in range(3)]
    assert all(t.data_ptr() != at for t in other)
    torch.cuda.synchronize()
    assert torch.equal(read, want)


def test_stream_of_another_device_is_refused():
    class Elsewhere:
        device, cuda_stream = torch.device("cuda", 7), 0
    *_, x, res, z, w, dy, mw = _inputs()
    with pytest.raises(ValueError, match="stream is on"):
        bm.gated_norm(x, z, w, stream=Elsewhere())
    with pytest.raises(ValueError, match="stream is on"):
        bm.layer_norm(x, stream=Elsewhere())

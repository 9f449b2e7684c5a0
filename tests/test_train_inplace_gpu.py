"""Training steps whose results go into one of their own inputs: what the
documentation allows gives the bits of separate arrays, and what it does not
allow is refused. Widths at which a row's last vector overlaps a vector of
another wave are among them."""
import ctypes

import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
from bidirectional_mamba_ssm_amd import _abi

pytestmark = pytest.mark.gpu

DEV = "cuda"
# 2500: neighbours in one wave; the others: in two (bf16 and fp32, forward and gradient)
WIDTHS = [100, 257, 513, 1025, 1537, 2049, 2500, 4097, 8193]
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _arrays(rows, C, dtype, seed, n):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(rows, C, generator=g, device=DEV).to(DT[dtype]) for _ in range(n)]


def _same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_norm_into_its_inputs(C, dtype):
    rows = 700
    print(f"rows {rows} C {C} {dtype}", flush=True)
    x, r = _arrays(rows, C, dtype, C, 2)
    want = bm.layer_norm(x, residual=r, checkpoint=True)
    for into in ((0, None), (1, None), (None, 0), (None, 1), (0, 1), (1, 0)):
        a = [x.clone(), r.clone()]
        out, s = (None if i is None else a[i] for i in into)
        o = bm.layer_norm(a[0], residual=a[1], out=out, sum_out=s, checkpoint=True)
        assert out is None or o["out"] is out
        assert s is None or o["sum"] is s
        assert _same([o["out"], o["sum"], o["mean"], o["rstd"], o["ckpt"].q, o["ckpt"].scale],
                     [want["out"], want["sum"], want["mean"], want["rstd"], want["ckpt"].q, want["ckpt"].scale]), into


def test_layer_norm_refusals():
    x, r, t = _arrays(6, 200, "bf16", 1, 3)
    with pytest.raises(bm.BimambaError, match="overlaps"):
        bm.layer_norm(x, residual=r, out=t, sum_out=t)
    with pytest.raises(bm.BimambaError, match="overlaps"):
        bm.layer_norm(x, residual=r, out=x, sum_out=x)
    with pytest.raises(ValueError, match="overlaps"):
        bm.layer_norm(x, out=x)
    buf = torch.zeros(7, 200, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(bm.BimambaError, match="overlaps"):
        bm.layer_norm(buf[:6], out=buf[1:])
    bm.layer_norm(x[:0], out=x[:0])   # no row, nothing to overlap


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_norm_bwd_into_its_inputs(C, dtype):
    rows = 700
    print(f"rows {rows} C {C} {dtype}", flush=True)
    x, dout, dsum = _arrays(rows, C, dtype, C, 3)
    o = bm.layer_norm(x, checkpoint=True)
    for kept in (x, o["ckpt"]):
        want = bm.layer_norm_bwd(dout, kept, o["mean"], o["rstd"], dsum=dsum)
        for into in ("dout", "dsum") + (("x",) if kept is x else ()):
            a = dict(dout=dout.clone(), dsum=dsum.clone(), x=x.clone())
            got = bm.layer_norm_bwd(a["dout"], a["x"] if kept is x else kept, o["mean"], o["rstd"], dsum=a["dsum"],
                                    dx=a[into])
            assert got[0] is a[into] and _same(got, want), into


def test_layer_norm_bwd_refusals():
    x, dout = _arrays(6, 256, "bf16", 2, 2)
    o = bm.layer_norm(x, checkpoint=True)
    buf = torch.zeros(7, 256, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(bm.BimambaError, match="overlaps"):
        bm.layer_norm_bwd(buf[:6], x, o["mean"], o["rstd"], dx=buf[1:])
    with pytest.raises(bm.BimambaError, match="overlaps"):
        bm.layer_norm_bwd(dout, x, o["mean"], o["rstd"], weight=buf.flatten()[:512].view(torch.float32), dx=buf[:6])


@pytest.mark.parametrize("C,group", [(256, 256), (1280, 256), (2048, 2048), (5120, 1280), (8192, 8192)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gated_norm_bwd_into_its_inputs(C, group, dtype):
    rows = 1500
    print(f"rows {rows} C {C} group {group} {dtype}", flush=True)
    z, dout = _arrays(rows, C, dtype, C, 2)
    y, = _arrays(rows, C, "f32", C + 1, 1)
    w = torch.rand(C, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV) + 0.5
    want = bm.gated_norm_bwd(dout, y, z, w, group_size=group)
    names = (None, "y", "z", "dout")
    for into_y in names if dtype == "f32" else (None, "y"):
        for into_z in names if dtype == "f32" else (None, "z", "dout"):
            if into_y == into_z and into_y is not None:
                continue
            a = dict(y=y.clone(), z=z.clone(), dout=dout.clone())
            got = bm.gated_norm_bwd(a["dout"], a["y"], a["z"], w, group_size=group, dy=a.get(into_y), dz=a.get(into_z))
            assert _same(got, want), (into_y, into_z)


def test_gated_norm_bwd_refusals():
    y, z, dout = _arrays(6, 256, "f32", 4, 3)
    w, buf = torch.ones(256, device=DEV), torch.zeros(7, 256, device=DEV)
    t = torch.zeros_like(y)
    for kw in (dict(dy=t, dz=t), dict(dy=y, dz=y), dict(dy=buf[1:], dz=buf[:6])):
        with pytest.raises(bm.BimambaError, match="overlaps"):
            bm.gated_norm_bwd(dout, y, z, w, **kw)
    for kw in (dict(dy=buf[1:]), dict(dz=buf[1:])):
        for a in ((buf[:6], y, z), (dout, buf[:6], z), (dout, y, buf[:6])):
            with pytest.raises(bm.BimambaError, match="overlaps"):
                bm.gated_norm_bwd(*a, w, **kw)


def test_act8_refusals():
    buf = torch.zeros(4, 128, device=DEV)
    a = bm.Act8(buf.view(torch.int8)[:, 128:256].contiguous(), torch.zeros(4, 4, dtype=torch.uint8, device=DEV))
    bm.act8_pack(buf, out=a)
    over = bm.Act8(buf.view(torch.int8).flatten()[:512].view(4, 128), a.scale)
    with pytest.raises(bm.BimambaError, match="overlaps"):
        bm.act8_pack(buf, out=over)
    with pytest.raises(bm.BimambaError, match="overlaps"):
        bm.act8_unpack(over, dtype=torch.float32, out=buf)


def test_conv1d_refusals():
    """The convolution's gradient onto its input, and outputs of one array."""
    batch, L, H, P, G, N = 1, 200, 2, 16, 1, 16
    ch = H * P + 2 * G * N
    x = [torch.zeros(batch, L, ch, device=DEV) for _ in range(2)]
    dirs = [dict(xbc=t, weight=torch.zeros(ch, 4, device=DEV)) for t in x]
    g = dict(x=torch.zeros(batch, L, H, P, device=DEV), B=torch.zeros(batch, L, G, N, device=DEV),
             C=torch.zeros(batch, L, G, N, device=DEV))
    t = torch.zeros_like(x[0])
    for out in ((x[0], None), (x[1], None), (None, x[0]), (None, x[1]), (t, t)):
        with pytest.raises(bm.BimambaError, match="overlaps|different arrays"):
            bm.conv1d_bwd(dirs[0], dirs[1], g, g, H, P, G, N, out=out)
    kept = [dict(d, xbc=bm.act8_pack(d["xbc"])) for d in dirs]
    o = dict(x=torch.zeros_like(g["x"]), B=torch.zeros_like(g["B"]), C=torch.zeros_like(g["C"]))
    for out in ((o, o), (dict(o, C=o["B"]), None)):
        with pytest.raises(bm.BimambaError, match="overlaps"):
            bm.conv1d(kept[0], kept[1], H, P, G, N, out=out, dtype=torch.float32)
    # the same input, weights or gradients for both directions are no overlap
    want = bm.conv1d_bwd(dirs[0], dict(dirs[0]), g, g, H, P, G, N, out=(t, torch.zeros_like(t)))
    assert want[0]["xbc"] is t


@pytest.mark.parametrize("C", [100, 513, 1025, 2049, 8193])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_norm_onto_x_through_the_library(C, dtype):
    """Without a residual the library takes out = x (the binding, which returns
    x as the sum, does not)."""
    rows = 700
    print(f"rows {rows} C {C} {dtype}", flush=True)
    x, = _arrays(rows, C, dtype, C, 1)
    want = bm.layer_norm(x, checkpoint=True)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    ck = bm.Act8.empty((rows, C), torch.device(DEV))
    p = _abi.Act8Ptrs(ck.q.data_ptr(), ck.scale.data_ptr())
    rc = bm.lib().bimamba_layer_norm(rows, C, bm.DTYPES[x.dtype], x.data_ptr(), None, None, None, 1e-5, x.data_ptr(),
                                     None, mean.data_ptr(), rstd.data_ptr(), ctypes.byref(p),
                                     torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert _same([x, mean, rstd, ck.q, ck.scale],
                 [want["out"], want["mean"], want["rstd"], want["ckpt"].q, want["ckpt"].scale])

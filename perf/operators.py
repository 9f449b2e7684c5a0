"""Workloads of the training operators around the scan, with plain forms.

Layer norm (with the residual add and an 8-bit checkpoint of its input) and
its gradient, the gated norm's gradient, the short convolution's gradient, the
convolution recomputed from an 8-bit checkpoint, and the checkpoints
themselves (blocks of 32 channels that share a power of two, 8-bit integers).

``run`` computes an operator with elementary torch operations in 32 bits, or,
with ``own`` set, through the framework's entry points. ``exact`` writes the
same results in 64 bits, from the definitions.
"""
import math

import torch

own = False

EPS = 1e-5
BLOCK = 32
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # the norm in front of one denoising step: a block of 64 tokens of the
        # 80-head model (d_inner 5120, d_model 2560), one sequence: latency
        dict(name="ln_block_step", op="layer_norm", rows=64, channels=2560, dtype="bf16",
             residual=True, ckpt=False, weight=True, bias=False),
        # a 131 072-token training row of the 64-head model (d_model 2048),
        # residual stream updated and the input kept in 8 bits: the largest
        dict(name="ln_long_row_ckpt", op="layer_norm", rows=131072, channels=2048, dtype="bf16",
             residual=True, ckpt=True, weight=True, bias=True),
        # the training layer's 8 x 1024 tokens, gradient from the checkpoint,
        # the residual stream's gradient added
        dict(name="ln_bwd_layer_ckpt", op="layer_norm_bwd", rows=8192, channels=2048, dtype="bf16",
             dsum=True, ckpt=True, weight=True),
        # a small fp32 model of an odd width, as for checking gradients
        dict(name="ln_bwd_odd_f32", op="layer_norm_bwd", rows=1000, channels=777, dtype="f32",
             dsum=False, ckpt=False, weight=True),
        # the training layer's output stage: 64 heads x 64, one group
        dict(name="gated_bwd_layer", op="gated_norm_bwd", rows=8192, channels=4096, group=4096,
             dtype="bf16", ckpt=False),
        # a ragged number of tokens of the 80-head model, four groups, scan
        # output and gate kept in 8 bits
        dict(name="gated_bwd_groups_ckpt", op="gated_norm_bwd", rows=3001, channels=5120, group=1280,
             dtype="bf16", ckpt=True),
        # the training layer's convolution: 8 x 1024 tokens, 4352 channels,
        # both streams
        dict(name="conv_bwd_layer", op="conv1d_bwd", batch=8, length=1024, nseq=0, nheads=64,
             headdim=64, ngroups=1, d_state=128, width=4, dtype="bf16", silu=True, both=True,
             bias=True, ckpt=False),
        # packed sequences of uneven lengths, small heads, fp32
        dict(name="conv_bwd_packed_small_f32", op="conv1d_bwd", batch=1, length=2500, nseq=11, nheads=4,
             headdim=16, ngroups=1, d_state=16, width=4, dtype="f32", silu=True, both=True,
             bias=True, ckpt=False),
        # the scan's inputs rebuilt from the checkpoint before its gradient:
        # the training layer
        dict(name="conv_from_ckpt_layer", op="conv1d_ckpt", batch=8, length=1024, nseq=0, nheads=64,
             headdim=64, ngroups=1, d_state=128, width=4, dtype="bf16", silu=True, both=True, bias=True),
        # the same for a short ragged row of a small model, forward stream only
        dict(name="conv_from_ckpt_small", op="conv1d_ckpt", batch=2, length=333, nseq=0, nheads=5,
             headdim=16, ngroups=1, d_state=16, width=3, dtype="bf16", silu=True, both=False, bias=True),
        # the training layer's convolution input stored in 8 bits and read back
        dict(name="act8_layer", op="act8", rows=8192, channels=4352, dtype="bf16"),
        # rows that end inside a block, fp32
        dict(name="act8_odd_f32", op="act8", rows=333, channels=1001, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm_bwd", "gated_norm_bwd", "conv1d_bwd", "conv1d_ckpt", "act8"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("layer_norm", "layer_norm_bwd", "act8"):
        channels = _log_int(rng, 16, 8192)
        if rng.random() < 0.6:
            channels = max(64, channels // 64 * 64)
        rows = _log_int(rng, 1, min(65536, 40_000_000 // channels))
        case = dict(op=op, rows=rows, channels=channels, dtype=dtype)
        if op == "layer_norm":
            case.update(residual=rng.random() < 0.6, ckpt=rng.random() < 0.5, weight=rng.random() < 0.8,
                        bias=rng.random() < 0.5)
        elif op == "layer_norm_bwd":
            case.update(dsum=rng.random() < 0.6, ckpt=rng.random() < 0.5, weight=rng.random() < 0.8)
        return case
    if op == "gated_norm_bwd":
        group = 256 * rng.randint(1, 8)
        channels = group * rng.randint(1, 8192 // group)
        rows = _log_int(rng, 1, min(32768, 40_000_000 // channels))
        return dict(op=op, rows=rows, channels=channels, group=group, dtype=dtype, ckpt=rng.random() < 0.5)
    headdim = rng.choice([16, 32, 64])
    d_state = rng.choice([16, 64, 128])
    ngroups = rng.choice([1, 1, 2])
    nheads = ngroups * rng.randint(1, 40 // ngroups)
    ch = nheads * headdim + 2 * ngroups * d_state
    nseq = rng.choice([0, 0, rng.randint(1, 24)])
    tokens = _log_int(rng, 8, min(16384, 30_000_000 // ch))
    batch = 1 if nseq else min(rng.randint(1, 8), tokens)
    case = dict(op=op, batch=batch, length=max(1, tokens // batch), nseq=nseq, nheads=nheads, headdim=headdim,
                ngroups=ngroups, d_state=d_state, width=rng.randint(2, 4), dtype=dtype,
                silu=rng.random() < 0.8, both=rng.random() < 0.7, bias=rng.random() < 0.7)
    if op == "conv1d_bwd":
        case["ckpt"] = rng.random() < 0.5
    return case


def _channels(case):
    if "nheads" in case:
        return case["nheads"] * case["headdim"] + 2 * case["ngroups"] * case["d_state"]
    return case["channels"]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    ch = _channels(case)
    c8 = 1.0 + 1.0 / BLOCK
    if "nheads" in case:
        n = case["batch"] * case["length"] * ch * (2 if case["both"] else 1)
        taps = ch * (case["width"] + 1) * 4 * (2 if case["both"] else 1)
        if case["op"] == "conv1d_ckpt":
            return {"bytes": int(n * (c8 + e) + taps), "flops": n * (2 * case["width"] + 6)}
        per = (c8 if case["ckpt"] else e) + 4 + e
        return {"bytes": int(n * per + 2 * taps), "flops": n * (6 * case["width"] + 14)}
    n = case["rows"] * ch
    if case["op"] == "layer_norm":
        per = 2 * e + (2 * e if case["residual"] else 0) + (c8 if case["ckpt"] else 0)
        return {"bytes": int(n * per + case["rows"] * 8 + ch * 8), "flops": n * 9}
    if case["op"] == "layer_norm_bwd":
        per = 2 * e + (e if case["dsum"] else 0) + (c8 if case["ckpt"] else e)
        return {"bytes": int(n * per + case["rows"] * 8 + ch * 12), "flops": n * 14}
    if case["op"] == "gated_norm_bwd":
        per = (2 * c8 if case["ckpt"] else 4 + e) + e + 4 + e
        return {"bytes": int(n * per + ch * 8), "flops": n * 30}
    return {"bytes": int(n * (2 * e + 2 * c8)), "flops": n * 6}


# ---- inputs -----------------------------------------------------------------

def _activations(g, shape, dtype):
    """Gaussian activations whose channels differ in scale, a few of them by
    far, as in a residual stream."""
    ch = shape[-1]
    scale = torch.exp(0.5 * torch.randn(ch, generator=g, device="cuda"))
    big = torch.rand(ch, generator=g, device="cuda") < 0.01
    scale = torch.where(big, scale * 20.0, scale)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype).contiguous()


def _gradient(g, shape, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * 0.01).to(dtype).contiguous()


def _pow2(k):
    """2^k for whole numbers k in [-126, 127], from the exponent's bits."""
    return ((k + 127) << 23).view(torch.float32)


def _pack(x):
    """8-bit checkpoint of x along its last dimension: (q int8, scale uint8)."""
    ch = x.shape[-1]
    v = x.float().reshape(-1, ch)
    pad = -ch % BLOCK
    if pad:
        v = torch.cat([v, torch.zeros(v.shape[0], pad, device=v.device)], dim=1)
    v = v.reshape(v.shape[0], -1, BLOCK)
    scale = ((v.view(torch.int32) & 0x7fffffff) >> 23).amax(dim=2)
    ok = (scale < 255).unsqueeze(2)
    # times 2^(133 - scale) in two steps, each an exact power of two
    k = 133 - scale
    h = torch.div(k, 2, rounding_mode="floor")
    m = v * _pow2(h).unsqueeze(2) * _pow2(k - h).unsqueeze(2)
    q = torch.where(ok, torch.clamp(torch.round(m), -127, 127), torch.zeros_like(m)).to(torch.int8)
    q = q.reshape(q.shape[0], -1)[:, :ch].reshape(x.shape).contiguous()
    return q, scale.to(torch.uint8).reshape(x.shape[:-1] + (scale.shape[1],)).contiguous()


def _unpack(q, scale):
    """The values an 8-bit checkpoint stands for, fp32."""
    ch = q.shape[-1]
    s = scale.to(torch.int32)
    k = s - 133
    h = torch.div(k, 2, rounding_mode="floor")
    a, b = _pow2(h), _pow2(k - h)
    a = torch.where(s == 255, torch.full_like(a, float("nan")), a)
    a = a.repeat_interleave(BLOCK, dim=-1)[..., :ch]
    b = b.repeat_interleave(BLOCK, dim=-1)[..., :ch]
    return q.float() * a * b


def _kept(x, ckpt):
    return _pack(x) if ckpt else x


def _offsets(case, seed):
    if not case["nseq"]:
        return None
    g = torch.Generator().manual_seed(seed + 1)
    cuts = torch.randint(0, case["length"] + 1, (case["nseq"] - 1,), generator=g)
    return [0] + sorted(int(c) for c in cuts) + [case["length"]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    st = {"case": case, "dtype": dt}
    if "nheads" in case:
        ch, w = _channels(case), case["width"]
        shape = (case["batch"], case["length"], ch)
        hp, gn = case["nheads"] * case["headdim"], case["ngroups"] * case["d_state"]
        bound = 1.0 / math.sqrt(w)
        st["dirs"] = []
        for _ in range(2 if case["both"] else 1):
            d = {"xbc": _kept(_activations(g, shape, dt), case.get("ckpt", True))}
            d["weight"] = (torch.rand(ch, w, generator=g, device="cuda") * 2 - 1) * bound
            d["bias"] = (torch.rand(ch, generator=g, device="cuda") * 2 - 1) * bound if case["bias"] else None
            if case["op"] == "conv1d_bwd":
                lead = shape[:2]
                d["dout"] = {
                    "x": _gradient(g, lead + (case["nheads"], case["headdim"]), torch.float32),
                    "B": _gradient(g, lead + (case["ngroups"], case["d_state"]), torch.float32),
                    "C": _gradient(g, lead + (case["ngroups"], case["d_state"]), torch.float32)}
            st["dirs"].append(d)
        st["cu"] = _offsets(case, seed)
        st["seq"] = None
        if st["cu"] is not None:
            lens = torch.tensor([b - a for a, b in zip(st["cu"], st["cu"][1:])])
            st["seq"] = torch.repeat_interleave(torch.arange(len(lens)), lens).to("cuda")
        st["split"] = (hp, gn)
        return st
    rows, ch = case["rows"], case["channels"]
    if case["op"] == "act8":
        st["x"] = _activations(g, (rows, ch), dt)
        return st
    if case["op"] == "gated_norm_bwd":
        st["y"] = _kept(_activations(g, (rows, ch), torch.float32), case["ckpt"])
        st["z"] = _kept(torch.randn(rows, ch, generator=g, device="cuda").to(dt), case["ckpt"])
        st["weight"] = torch.rand(ch, generator=g, device="cuda") + 0.5
        st["dout"] = _gradient(g, (rows, ch), dt)
        return st
    x = _activations(g, (rows, ch), dt)
    st["weight"] = torch.rand(ch, generator=g, device="cuda") + 0.5 if case["weight"] else None
    if case["op"] == "layer_norm":
        st["x"] = x
        st["residual"] = _activations(g, (rows, ch), dt) if case["residual"] else None
        st["bias"] = torch.randn(ch, generator=g, device="cuda") * 0.1 if case["bias"] else None
        return st
    xd = x.double()
    mean = xd.mean(dim=1)
    st["mean"] = mean.float()
    st["rstd"] = torch.rsqrt(((xd - mean.unsqueeze(1)) ** 2).mean(dim=1) + EPS).float()
    st["x"] = _kept(x, case["ckpt"])
    st["dout"] = _gradient(g, (rows, ch), dt)
    st["dsum"] = _gradient(g, (rows, ch), dt) if case["dsum"] else None
    return st


# ---- plain forms ------------------------------------------------------------

def _value(t):
    return _unpack(*t) if isinstance(t, tuple) else t.float()


def _plain_layer_norm(st):
    case, dt = st["case"], st["dtype"]
    h = st["x"]
    if st["residual"] is not None:
        h = (h.float() + st["residual"].float()).to(dt)
    v = h.float()
    mean = v.mean(dim=1)
    c = v - mean.unsqueeze(1)
    rstd = torch.rsqrt((c * c).mean(dim=1) + EPS)
    o = c * rstd.unsqueeze(1)
    if st["weight"] is not None:
        o = o * st["weight"]
    if st["bias"] is not None:
        o = o + st["bias"]
    res = {"out": o.to(dt), "sum": h, "mean": mean, "rstd": rstd}
    if case["ckpt"]:
        res["ckpt"] = _unpack(*_pack(h)).to(dt)
    return res


def _plain_layer_norm_bwd(st):
    xh = (_value(st["x"]) - st["mean"].unsqueeze(1)) * st["rstd"].unsqueeze(1)
    do = st["dout"].float()
    g = do * st["weight"] if st["weight"] is not None else do
    dx = (g - g.mean(dim=1, keepdim=True) - xh * (g * xh).mean(dim=1, keepdim=True)) * st["rstd"].unsqueeze(1)
    if st["dsum"] is not None:
        dx = dx + st["dsum"].float()
    return {"dx": dx.to(st["dtype"]), "dweight": (do * xh).sum(dim=0), "dbias": do.sum(dim=0)}


def _plain_gated_norm_bwd(st):
    case = st["case"]
    rows, ch, gs = case["rows"], case["channels"], case["group"]
    y, z, do = _value(st["y"]), _value(st["z"]), st["dout"].float()
    sig = 1.0 / (1.0 + torch.exp(-z))
    s = z * sig
    v = (y * s).reshape(rows, ch // gs, gs)
    r = torch.rsqrt((v * v).mean(dim=2, keepdim=True) + EPS)
    vn = v * r
    g = (do * st["weight"]).reshape(v.shape)
    dv = ((g - vn * (g * vn).mean(dim=2, keepdim=True)) * r).reshape(rows, ch)
    dz = dv * y * sig * (1.0 + z * (1.0 - sig))
    return {"dy": dv * s, "dz": dz.to(st["dtype"]), "dweight": (do * vn.reshape(rows, ch)).sum(dim=0)}


def _shift(v, n, seq):
    """v moved n tokens later (n < 0: earlier) along dim 1, zeros where a row
    or a packed sequence has no such token."""
    if n == 0:
        return v
    L = v.shape[1]
    o = torch.zeros_like(v)
    if abs(n) < L:
        if n > 0:
            o[:, n:] = v[:, :-n]
        else:
            o[:, :n] = v[:, -n:]
        if seq is not None:
            same = torch.zeros(L, dtype=torch.bool, device=v.device)
            if n > 0:
                same[n:] = seq[n:] == seq[:-n]
            else:
                same[:n] = seq[:n] == seq[-n:]
            o = o * same.reshape(1, L, 1)
    return o


def _plain_filter(v, d, width, sign, seq):
    u = torch.zeros_like(v)
    for k in range(width):
        u = u + d["weight"][:, k] * _shift(v, sign * (width - 1 - k), seq)
    return u if d["bias"] is None else u + d["bias"]


def _plain_conv1d_ckpt(st):
    case = st["case"]
    hp, gn = st["split"]
    outs = []
    for d, sign in zip(st["dirs"], (1, -1)):
        u = _plain_filter(_value(d["xbc"]), d, case["width"], sign, st["seq"])
        if case["silu"]:
            u = u / (1.0 + torch.exp(-u))
        u = u.to(st["dtype"])
        lead = u.shape[:2]
        outs.append({"x": u[..., :hp].reshape(lead + (case["nheads"], case["headdim"])).contiguous(),
                     "B": u[..., hp:hp + gn].reshape(lead + (case["ngroups"], case["d_state"])).contiguous(),
                     "C": u[..., hp + gn:].reshape(lead + (case["ngroups"], case["d_state"])).contiguous()})
    return outs


def _plain_conv1d_bwd(st):
    case = st["case"]
    w = case["width"]
    outs = []
    for d, sign in zip(st["dirs"], (1, -1)):
        v = _value(d["xbc"])
        du = torch.cat([d["dout"][k].reshape(v.shape[:2] + (-1,)) for k in ("x", "B", "C")], dim=2)
        if case["silu"]:
            u = _plain_filter(v, d, w, sign, st["seq"])
            sig = 1.0 / (1.0 + torch.exp(-u))
            du = du * sig * (1.0 + u * (1.0 - sig))
        dv = torch.zeros_like(v)
        dw = []
        for k in range(w):
            n = sign * (w - 1 - k)
            dv = dv + d["weight"][:, k] * _shift(du, -n, st["seq"])
            dw.append((du * _shift(v, n, st["seq"])).sum(dim=(0, 1)))
        o = {"xbc": dv.to(st["dtype"]), "weight": torch.stack(dw, dim=1)}
        if d["bias"] is not None:
            o["bias"] = du.sum(dim=(0, 1))
        outs.append(o)
    return outs


def _plain(st):
    op = st["case"]["op"]
    if op == "act8":
        return _unpack(*_pack(st["x"])).to(st["dtype"])
    return {"layer_norm": _plain_layer_norm, "layer_norm_bwd": _plain_layer_norm_bwd,
            "gated_norm_bwd": _plain_gated_norm_bwd, "conv1d_bwd": _plain_conv1d_bwd,
            "conv1d_ckpt": _plain_conv1d_ckpt}[op](st)


# ---- the framework's calls ---------------------------------------------------

def _framework(st):
    import bidirectional_mamba_ssm_amd as bm

    def kept(t):
        return bm.Act8(*t) if isinstance(t, tuple) else t

    case, dt = st["case"], st["dtype"]
    op = case["op"]
    if op == "act8":
        return bm.act8_unpack(bm.act8_pack(st["x"]), dtype=dt)
    if op == "layer_norm":
        r = bm.layer_norm(st["x"], st["weight"], st["bias"], residual=st["residual"], eps=EPS,
                          checkpoint=case["ckpt"])
        res = {k: r[k] for k in ("out", "sum", "mean", "rstd")}
        if case["ckpt"]:
            res["ckpt"] = bm.act8_unpack(r["ckpt"], dtype=dt)
        return res
    if op == "layer_norm_bwd":
        dx, dw, db = bm.layer_norm_bwd(st["dout"], kept(st["x"]), st["mean"], st["rstd"], st["weight"],
                                       dsum=st["dsum"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    if op == "gated_norm_bwd":
        dy, dz, dw = bm.gated_norm_bwd(st["dout"], kept(st["y"]), kept(st["z"]), st["weight"],
                                       group_size=case["group"], eps=EPS)
        return {"dy": dy, "dz": dz, "dweight": dw}
    dirs = [dict(xbc=kept(d["xbc"]), weight=d["weight"], bias=d["bias"]) for d in st["dirs"]] + [None]
    dims = (case["nheads"], case["headdim"], case["ngroups"], case["d_state"])
    act = "silu" if case["silu"] else "none"
    if op == "conv1d_ckpt":
        return [o for o in bm.conv1d(dirs[0], dirs[1], *dims, activation=act, cu_seqlens=st["cu"], dtype=dt)
                if o is not None]
    douts = [d["dout"] for d in st["dirs"]] + [None]
    gs = bm.conv1d_bwd(dirs[0], dirs[1], douts[0], douts[1], *dims, activation=act, cu_seqlens=st["cu"],
                       dtype=dt)
    return [{k: v for k, v in o.items() if v is not None} for o in gs if o is not None]


def run(state):
    return _framework(state) if own else _plain(state)


# ---- 64-bit results ----------------------------------------------------------

def _double_pow2(k):
    """2^k in 64 bits, exactly, for whole numbers k."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_value(t):
    if not isinstance(t, tuple):
        return t.double()
    q, s = t
    ch = torch.arange(q.shape[-1], device=q.device) // BLOCK
    s = s.to(torch.int64)[..., ch]
    v = q.double() * _double_pow2(s - 133)
    return torch.where(s == 255, torch.full_like(v, float("nan")), v)


def _exact_round_trip(x):
    """Each block of 32 in units of 2^-6 of the power of two at or below its
    largest magnitude (2^-127 at least), as whole numbers of at most 127."""
    out = torch.empty_like(x, dtype=torch.float64)
    for c0 in range(0, x.shape[-1], BLOCK):
        v = x[..., c0:c0 + BLOCK].double()
        top = v.abs().amax(dim=-1, keepdim=True)
        # frexp: top = m 2^e with m in [1/2, 1)
        e = torch.frexp(top).exponent - 1
        unit = _double_pow2(torch.where(top > 0, e, torch.full_like(e, -127)).clamp(min=-127) - 6)
        out[..., c0:c0 + BLOCK] = torch.clamp(torch.round(v / unit), -127.0, 127.0) * unit
    return out


def _sources(case, st, sign):
    """idx[k][t]: the token that tap k of token t reads, -1 where there is none."""
    L, w = case["length"], case["width"]
    t = torch.arange(L, device="cuda")
    first, last = torch.zeros_like(t), torch.full_like(t, L - 1)
    if st["cu"] is not None:
        for a, b in zip(st["cu"], st["cu"][1:]):
            first[a:b], last[a:b] = a, b - 1
    idx = []
    for k in range(w):
        j = t - sign * (w - 1 - k)
        idx.append(torch.where((j >= first) & (j <= last), j, torch.full_like(j, -1)))
    return idx


def _exact_conv(case, st):
    hp, gn = st["split"]
    outs = []
    for d, sign in zip(st["dirs"], (1, -1)):
        xin = _exact_value(d["xbc"])
        W = d["weight"].double()
        taps = []
        for j in _sources(case, st, sign):
            taps.append(xin.index_select(1, j.clamp(min=0)) * (j >= 0).reshape(1, -1, 1).double())
        u = sum(W[:, k] * taps[k] for k in range(case["width"]))
        if d["bias"] is not None:
            u = u + d["bias"].double()
        sig = torch.sigmoid(u)
        if case["op"] == "conv1d_ckpt":
            o = u * sig if case["silu"] else u
            lead = o.shape[:2]
            x, B, C = torch.split(o, [hp, gn, gn], dim=2)
            outs.append({"x": x.reshape(lead + (case["nheads"], case["headdim"])),
                         "B": B.reshape(lead + (case["ngroups"], case["d_state"])),
                         "C": C.reshape(lead + (case["ngroups"], case["d_state"]))})
            continue
        du = torch.cat([d["dout"][k].double().flatten(2) for k in ("x", "B", "C")], dim=2)
        if case["silu"]:
            du = du * (sig + u * sig * torch.sigmoid(-u))
        dxbc = torch.zeros_like(xin)
        dw = torch.empty_like(W)
        for k, j in enumerate(_sources(case, st, sign)):
            ok = j >= 0
            dxbc.index_add_(1, j[ok], W[:, k] * du[:, ok])
            dw[:, k] = (du * taps[k]).sum(dim=1).sum(dim=0)
        o = {"xbc": dxbc, "weight": dw}
        if d["bias"] is not None:
            o["bias"] = du.sum(dim=1).sum(dim=0)
        outs.append(o)
    return outs


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "act8":
        return _exact_round_trip(st["x"])
    if op in ("conv1d_bwd", "conv1d_ckpt"):
        return _exact_conv(case, st)
    if op == "layer_norm":
        h = st["x"]
        if st["residual"] is not None:
            h = (h.double() + st["residual"].double()).to(st["dtype"])
        v = h.double()
        mean = v.mean(dim=1)
        var = torch.var(v, dim=1, correction=0)
        out = (v - mean[:, None]) / torch.sqrt(var + EPS)[:, None]
        if st["weight"] is not None:
            out = out * st["weight"].double()
        if st["bias"] is not None:
            out = out + st["bias"].double()
        res = {"out": out, "sum": v, "mean": mean, "rstd": 1.0 / torch.sqrt(var + EPS)}
        if case["ckpt"]:
            res["ckpt"] = _exact_round_trip(h)
        return res
    do = st["dout"].double()
    if op == "layer_norm_bwd":
        rstd = st["rstd"].double()[:, None]
        xh = (_exact_value(st["x"]) - st["mean"].double()[:, None]) * rstd
        g = do if st["weight"] is None else do * st["weight"].double()
        n = case["channels"]
        dx = rstd / n * (n * g - g.sum(dim=1, keepdim=True) - xh * (g * xh).sum(dim=1, keepdim=True))
        if st["dsum"] is not None:
            dx = dx + st["dsum"].double()
        return {"dx": dx, "dweight": (do * xh).sum(dim=0), "dbias": do.sum(dim=0)}
    y, z, w = _exact_value(st["y"]), _exact_value(st["z"]), st["weight"].double()
    gate = z * torch.sigmoid(z)
    v = y * gate
    parts = case["channels"] // case["group"]
    q = (v ** 2).unflatten(1, (parts, -1)).mean(dim=2) + EPS            # mean square of each group
    gv = (do * w * v).unflatten(1, (parts, -1)).mean(dim=2)
    q = q.repeat_interleave(case["group"], dim=1)
    gv = gv.repeat_interleave(case["group"], dim=1)
    dv = do * w / torch.sqrt(q) - v * gv / q ** 1.5
    slope = torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
    return {"dy": dv * gate, "dz": dv * y * slope, "dweight": (do * v / torch.sqrt(q)).sum(dim=0)}

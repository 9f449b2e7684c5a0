"""Workloads of a delta-rule mixer layer, with plain forms.

The gated delta rule over whole sequences, its gradient and its cached step
(a recurrence on a matrix state, beside the selective scan); the RMS norm with
the residual add, its output in 8-bit integers with a scale for each row, and
its gradient; the product of 8-bit integers with a scale for each token and
channel, which reads that output.

``run`` computes an operator with elementary torch operations in 32 bits, or,
with ``own`` set, through the framework's entry points. ``exact`` writes the
same results in 64 bits, from the definitions.
"""
import math

import torch

own = False

EPS = 1e-5
CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # the norm in front of one denoising step: 64 tokens of a block, one
        # sequence, d_model 2560, straight to 8 bits for the projection: latency
        dict(name="rms_block_step_8bit", op="rms_norm", rows=64, channels=2560, dtype="bf16",
             residual=True, weight=True, rows8=True, dense=False),
        # a 131 072-token row of a model with d_model 2048, residual stream
        # updated, output in 8 bits
        dict(name="rms_long_row_8bit", op="rms_norm", rows=131072, channels=2048, dtype="bf16",
             residual=True, weight=True, rows8=True, dense=False),
        # the training layer's 8 x 1024 tokens, the residual stream's gradient added
        dict(name="rms_bwd_layer", op="rms_norm_bwd", rows=8192, channels=2048, dtype="bf16",
             dsum=True, ckpt=False, weight=True),
        # a small fp32 model of an odd width, gradient from the 8-bit checkpoint
        dict(name="rms_bwd_odd_f32", op="rms_norm_bwd", rows=1000, channels=777, dtype="f32",
             dsum=False, ckpt=True, weight=True),
        # the output projection of one denoising step (d_inner 4096 to d_model
        # 2048, 64 tokens), its input quantized in the call: latency
        dict(name="linear8_block_step", op="linear8", rows=64, cin=4096, cout=2048, dtype="bf16",
             bias=False, pack=True),
        # the input projection of the training layer's 8 x 1024 tokens (gate,
        # value, key, query and step channels of the 64-head model): the largest
        dict(name="linear8_layer", op="linear8", rows=8192, cin=2048, cout=8512, dtype="bf16",
             bias=False, pack=False),
        # the training layer: 8 x 1024 tokens, 32 heads of 128 x 128 states,
        # two of them to a query and key
        dict(name="delta_fwd_layer", op="delta_fwd", batch=8, length=1024, nseq=0, nheads=32, headdim=128,
             ngroups=16, d_state=128, dtype="bf16", both=False, state=True),
        # packed sequences of uneven lengths, both streams, small odd heads, fp32
        dict(name="delta_fwd_packed_f32", op="delta_fwd", batch=1, length=2500, nseq=11, nheads=6, headdim=40,
             ngroups=3, d_state=32, dtype="f32", both=True, state=True),
        # one token of 64 sequences: every state read and written
        dict(name="delta_step_token", op="delta_step", batch=64, length=1, nheads=32, headdim=128, ngroups=16,
             d_state=128, dtype="bf16", both=False, commit=True),
        # one denoising step: a block of 64 tokens, both streams, state kept
        dict(name="delta_step_block", op="delta_step", batch=1, length=64, nheads=64, headdim=64, ngroups=16,
             d_state=128, dtype="bf16", both=True, commit=False),
        # the training layer's gradient
        dict(name="delta_bwd_layer", op="delta_bwd", batch=8, length=1024, nseq=0, nheads=32, headdim=128,
             ngroups=16, d_state=128, dtype="bf16", both=False, state=False),
        # packed sequences, both streams, from and to a state, fp32
        dict(name="delta_bwd_packed_f32", op="delta_bwd", batch=1, length=1300, nseq=7, nheads=6, headdim=40,
             ngroups=3, d_state=32, dtype="f32", both=True, state=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rms_norm", "rms_norm_bwd", "linear8", "linear8", "delta_fwd", "delta_fwd", "delta_step",
                     "delta_bwd", "delta_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("rms_norm", "rms_norm_bwd"):
        channels = _log_int(rng, 16, 16384)
        if rng.random() < 0.6:
            channels = max(64, channels // 64 * 64)
        rows = _log_int(rng, 1, min(65536, 60_000_000 // channels))
        case = dict(op=op, rows=rows, channels=channels, dtype=dtype, weight=rng.random() < 0.8)
        if op == "rms_norm":
            rows8 = rng.random() < 0.7
            case.update(residual=rng.random() < 0.6, rows8=rows8, dense=not rows8 or rng.random() < 0.3)
        else:
            case.update(dsum=rng.random() < 0.6, ckpt=rng.random() < 0.4)
        return case
    if op == "linear8":
        cin, cout = _log_int(rng, 16, 8192), _log_int(rng, 16, 8192)
        if rng.random() < 0.7:
            cin, cout = max(64, cin // 64 * 64), max(64, cout // 64 * 64)
        rows = _log_int(rng, 1, min(8192, 130_000_000_000 // (cin * cout)))
        return dict(op=op, rows=rows, cin=cin, cout=cout, dtype=dtype, bias=rng.random() < 0.5,
                    pack=rng.random() < 0.4)
    d_state = rng.choice([16, 32, 64, 128, 128])
    headdim = rng.choice([16, 40, 64, 64, 128, 128, rng.randint(1, 128)])
    ngroups = rng.choice([1, 2, 4, 8])
    nheads = ngroups * rng.randint(1, 32 // ngroups)
    case = dict(op=op, nheads=nheads, headdim=headdim, ngroups=ngroups, d_state=d_state, dtype=dtype,
                both=rng.random() < 0.4)
    if op == "delta_step":
        length = rng.choice([1, 1, 2, 16, 64, rng.randint(1, 256)])
        case.update(batch=_log_int(rng, 1, max(1, min(128, 2048 // length))), length=length, commit=rng.random() < 0.6)
        return case
    most = 4096 if op == "delta_fwd" else 2048
    nseq = rng.choice([0, 0, rng.randint(1, 12)])
    tokens = _log_int(rng, 16, most)
    batch = 1 if nseq else min(rng.randint(1, 8), tokens)
    case.update(batch=batch, length=max(1, tokens // batch), nseq=nseq, state=rng.random() < 0.5)
    return case


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "rms_norm":
        n = case["rows"] * case["channels"]
        per = e + (2 * e if case["residual"] else 0) + (1 if case["rows8"] else 0) + (e if case["dense"] else 0)
        return {"bytes": n * per + case["rows"] * 8 + case["channels"] * 4, "flops": n * 7}
    if op == "rms_norm_bwd":
        n = case["rows"] * case["channels"]
        per = 2 * e + (e if case["dsum"] else 0) + (1 + 1 / 32 if case["ckpt"] else e)
        return {"bytes": int(n * per) + case["rows"] * 4 + case["channels"] * 8, "flops": n * 11}
    if op == "linear8":
        r, ci, co = case["rows"], case["cin"], case["cout"]
        return {"bytes": r * ci * (e if case["pack"] else 1) + ci * co + r * co * e + (r + co) * 4,
                "flops": 2 * r * ci * co}
    tok, nh, p = case["batch"] * case["length"], case["nheads"], case["headdim"]
    g, n = case["ngroups"], case["d_state"]
    dirs = 2 if case["both"] else 1
    inputs = dirs * tok * ((nh * p + 2 * g * n) * e + nh * 8)
    states = (case["nseq"] if case.get("nseq") else case["batch"]) * nh * p * n * 4
    if op == "delta_bwd":
        grads = dirs * tok * ((nh * p + 2 * g * n) * 4 + nh * 8)
        return {"bytes": inputs + grads + tok * nh * p * 4 + (3 * states if case["state"] else 0),
                "flops": dirs * tok * nh * p * n * 18}
    moved = states * (2 if case["commit"] else 1) if op == "delta_step" else 2 * states if case["state"] else 0
    return {"bytes": inputs + tok * nh * p * 4 + moved, "flops": dirs * tok * nh * p * n * 6}


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


def _unit(g, shape, dtype):
    """Queries and keys: SiLU of Gaussians (the convolution's output), each of
    length one."""
    v = torch.randn(shape, generator=g, device="cuda")
    v = v / (1.0 + torch.exp(-v))
    return (v / (v * v).sum(dim=-1, keepdim=True).sqrt()).to(dtype).contiguous()


def _quantize(v):
    """Rows in 8 bits: (q int8 [rows, C], scale float32 [rows])."""
    top = v.abs().amax(dim=1, keepdim=True)
    inv = torch.where(top >= 2.0 ** -100, 127.0 / top, torch.zeros_like(top))
    scale = torch.where(top >= 2.0 ** -100, top / 127.0, torch.zeros_like(top))
    return torch.round(v * inv).to(torch.int8).contiguous(), scale.squeeze(1).contiguous()


def _pow2(k):
    """2^k for whole numbers k in [-126, 127], from the exponent's bits."""
    return ((k + 127) << 23).view(torch.float32)


def _block8(x):
    """The 8-bit checkpoint of x: 32 consecutive channels share a power of two
    (q int8 [rows, C], scale uint8 [rows, blocks]). All values are ordinary."""
    rows, ch = x.shape
    v = torch.cat([x.float(), torch.zeros(rows, -ch % 32, device=x.device)], dim=1).reshape(rows, -1, 32)
    scale = ((v.view(torch.int32) & 0x7fffffff) >> 23).amax(dim=2)
    q = torch.clamp(torch.round(v * _pow2(133 - scale).unsqueeze(2)), -127, 127).to(torch.int8)
    return q.reshape(rows, -1)[:, :ch].contiguous(), scale.to(torch.uint8).contiguous()


def _offsets(case, seed):
    if not case.get("nseq"):
        return None
    g = torch.Generator().manual_seed(seed + 1)
    cuts = torch.randint(0, case["length"] + 1, (case["nseq"] - 1,), generator=g)
    return [0] + sorted(int(c) for c in cuts) + [case["length"]]


def _places(case, cu):
    """For each sequence and each position the token's place in the flattened
    batch, -1 past the end, in forward and in reverse order."""
    L = case["length"]
    spans = [(a, b) for a, b in zip(cu, cu[1:])] if cu else [(i * L, i * L + L) for i in range(case["batch"])]
    longest = max(1, max(b - a for a, b in spans))
    at = torch.arange(longest)
    start = torch.tensor([a for a, _ in spans]).unsqueeze(1)
    count = torch.tensor([b - a for a, b in spans]).unsqueeze(1)
    none = torch.full((1, 1), -1)
    fwd = torch.where(at < count, start + at, none)
    rev = torch.where(at < count, start + count - 1 - at, none)
    return [fwd.to("cuda"), rev.to("cuda")]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = DTYPES[case["dtype"]], case["op"]
    st = {"case": case, "dtype": dt}
    if op in ("rms_norm", "rms_norm_bwd"):
        shape = (case["rows"], case["channels"])
        x = _activations(g, shape, dt)
        st["weight"] = torch.rand(shape[1], generator=g, device="cuda") + 0.5 if case["weight"] else None
        if op == "rms_norm":
            st["x"] = x
            st["residual"] = _activations(g, shape, dt) if case["residual"] else None
            return st
        st["rstd"] = torch.rsqrt((x.double() ** 2).mean(dim=1) + EPS).float()
        st["x"] = _block8(x) if case["ckpt"] else x
        st["dout"] = _gradient(g, shape, dt)
        st["dsum"] = _gradient(g, shape, dt) if case["dsum"] else None
        return st
    if op == "linear8":
        x = _activations(g, (case["rows"], case["cin"]), dt)
        w = torch.randn(case["cout"], case["cin"], generator=g, device="cuda") / math.sqrt(case["cin"])
        st["x"] = x if case["pack"] else _quantize(x.float())
        st["weight"] = _quantize(w)
        st["bias"] = torch.randn(case["cout"], generator=g, device="cuda") * 0.1 if case["bias"] else None
        return st
    b, L, H, P = case["batch"], case["length"], case["nheads"], case["headdim"]
    G, N = case["ngroups"], case["d_state"]
    st["dirs"] = []
    for _ in range(2 if case["both"] else 1):
        # decay rates and step sizes as the scan's: A in [-16, -1], dt from
        # 0.001 to 0.1 on a logarithmic scale
        A = 1.0 + 15.0 * torch.rand(H, generator=g, device="cuda")
        step = torch.exp(math.log(1e-3) + math.log(1e2) * torch.rand(b, L, H, generator=g, device="cuda"))
        st["dirs"].append(dict(
            q=_unit(g, (b, L, G, N), dt), k=_unit(g, (b, L, G, N), dt),
            v=torch.randn(b, L, H, P, generator=g, device="cuda").to(dt),
            g=(-step * A).contiguous(),
            beta=1.0 / (1.0 + torch.exp(-torch.randn(b, L, H, generator=g, device="cuda")))))
    st["cu"] = _offsets(case, seed)
    st["places"] = _places(case, st["cu"])
    units = case["nseq"] if case.get("nseq") else b
    st["state"] = st["dfinal"] = None
    if op == "delta_step" or case["state"]:
        st["state"] = torch.randn(units, H, P, N, generator=g, device="cuda") * 0.3
    if op == "delta_bwd":
        st["dy"] = _gradient(g, (b, L, H, P), torch.float32)
        if case["state"]:
            st["dfinal"] = _gradient(g, (units, H, P, N), torch.float32)
    return st


# ---- plain forms: norm and product ------------------------------------------

def _plain_rms_norm(st):
    case, dt = st["case"], st["dtype"]
    h = st["x"]
    if st["residual"] is not None:
        h = (h.float() + st["residual"].float()).to(dt)
    v = h.float()
    rstd = torch.rsqrt((v * v).mean(dim=1) + EPS)
    o = v * rstd.unsqueeze(1)
    if st["weight"] is not None:
        o = o * st["weight"]
    res = {"sum": h, "rstd": rstd}
    if case["dense"]:
        res["out"] = o.to(dt)
    if case["rows8"]:
        q, scale = _quantize(o)
        res["values"], res["scale"] = (q.float() * scale.unsqueeze(1)).to(torch.bfloat16), scale
    return res


def _block8_values(q, scale):
    unit = _pow2(scale.to(torch.int32) - 133).repeat_interleave(32, dim=1)[:, :q.shape[1]]
    return q.float() * unit


def _plain_rms_norm_bwd(st):
    x = _block8_values(*st["x"]) if st["case"]["ckpt"] else st["x"].float()
    r = st["rstd"].unsqueeze(1)
    xh = x * r
    do = st["dout"].float()
    g = do * st["weight"] if st["weight"] is not None else do
    dx = (g - xh * (g * xh).mean(dim=1, keepdim=True)) * r
    if st["dsum"] is not None:
        dx = dx + st["dsum"].float()
    return {"dx": dx.to(st["dtype"]), "dweight": (do * xh).sum(dim=0)}


def _plain_linear8(st):
    xq, xs = _quantize(st["x"].float()) if st["case"]["pack"] else st["x"]
    wq, ws = st["weight"]
    # whole numbers whose sums stay under 2^24 for these inputs: exact in fp32
    out = (xq.float() @ wq.float().t()) * xs.unsqueeze(1) * ws
    if st["bias"] is not None:
        out = out + st["bias"]
    return out.to(st["dtype"])


# ---- plain forms: the delta rule by chunks ----------------------------------

def _take(t, at, n):
    """Tokens of t [b, L, ...] at the places at [units, len], zeros where -1,
    padded to n positions: fp32 [units, n, ...]."""
    flat = t.reshape((-1,) + t.shape[2:]).float()
    v = flat[at.clamp(min=0)]
    v = torch.where((at >= 0).reshape(at.shape + (1,) * (v.dim() - 2)), v, torch.zeros_like(v))
    pad = torch.zeros((v.shape[0], n - v.shape[1]) + v.shape[2:], device=v.device)
    return torch.cat([v, pad], dim=1)


def _give(out, v, at):
    """Writes v [units, n, ...] to the tokens of out [b, L, ...] at their places."""
    live = at >= 0
    out.reshape((-1,) + out.shape[2:])[at[live]] = v[:, :at.shape[1]][live]


def _chunks(d, at, scale):
    """A direction's inputs by chunks [units, H, chunks, c, ...] and what the
    chunks need whatever their state."""
    H, G = d["v"].shape[2], d["k"].shape[2]
    c = min(CHUNK, at.shape[1])
    nc = -(-at.shape[1] // c)

    def part(t, rep=1):
        t = _take(t, at, nc * c)
        t = t.repeat_interleave(rep, dim=2) if rep > 1 else t
        t = t.transpose(1, 2).contiguous()
        return t.reshape(t.shape[:2] + (nc, c) + t.shape[3:])

    q, k, v = part(d["q"], H // G), part(d["k"], H // G), part(d["v"])
    beta, s = part(d["beta"]), part(d["g"]).cumsum(dim=-1)
    lower = torch.ones(c, c, device=s.device, dtype=torch.bool).tril()
    low = torch.full((), -math.inf, device=s.device)
    decay = torch.exp(torch.where(lower, s.unsqueeze(-1) - s.unsqueeze(-2), low))
    kt = k.transpose(-1, -2)
    n = (k @ kt) * decay * lower.tril(-1)
    p = (q @ kt) * decay * scale
    # (I + n beta)^-1 = (I - m)(I + m^2)(I + m^4) ..., m = n beta nilpotent
    m = n * beta.unsqueeze(-2)
    eye = torch.eye(c, device=s.device)
    t = eye - m
    power = 1
    while 2 * power < c:
        m = m @ m
        t = t + t @ m
        power *= 2
    rise, fall = torch.exp(s).unsqueeze(-1), torch.exp(s[..., -1:] - s).unsqueeze(-1)
    return dict(q=q, k=k, v=v, beta=beta.unsqueeze(-1), decay=decay, n=n, p=p, t=t, rise=rise, fall=fall,
                last=torch.exp(s[..., -1]), nc=nc, c=c, lower=lower)


def _walk(x, state):
    """The chunks' states and errors e: (states entering, errors, outputs, the last state)."""
    e0, w = x["t"] @ x["v"], x["t"] @ (x["rise"] * x["k"])
    kf = (x["fall"] * x["k"]).transpose(-1, -2).contiguous()
    states, errors = [], []
    for i in range(x["nc"]):
        e = e0[:, :, i] - w[:, :, i] @ state
        states.append(state)
        errors.append(e)
        state = x["last"][:, :, i, None, None] * state + kf[:, :, i] @ (x["beta"][:, :, i] * e)
    return torch.stack(states, dim=2), torch.stack(errors, dim=2), state


def _first(st, x):
    """The state that the first direction starts from, [units, H, N, P]."""
    if st["state"] is None:
        return torch.zeros(x["k"].shape[:2] + (x["k"].shape[-1], x["v"].shape[-1]), device=x["k"].device)
    return st["state"].transpose(-1, -2).contiguous()


def _flat(t):
    """[units, H, chunks, c, ...] as [units, positions, H, ...]."""
    return t.reshape(t.shape[:2] + (-1,) + t.shape[4:]).transpose(1, 2)


def _plain_delta(st):
    scale = st["case"]["d_state"] ** -0.5
    y, last = 0.0, None
    for i, d in enumerate(st["dirs"]):
        x = _chunks(d, st["places"][i], scale)
        first = _first(st, x) if i == 0 else torch.zeros_like(_first(st, x))
        s, e, end = _walk(x, first)
        o = scale * x["rise"] * (x["q"] @ s) + x["p"] @ (x["beta"] * e)
        part = torch.zeros(d["v"].shape, device=e.device)
        _give(part, _flat(o), st["places"][i])
        y = y + part
        if i == 0:
            last = end.transpose(-1, -2).contiguous()
    return y, last


def _plain_delta_bwd(st):
    case = st["case"]
    scale = case["d_state"] ** -0.5
    grads, dinit = [], None
    for i, d in enumerate(st["dirs"]):
        at = st["places"][i]
        x = _chunks(d, at, scale)
        first = _first(st, x) if i == 0 else torch.zeros_like(_first(st, x))
        s, e, end = _walk(x, first)
        do = _take(st["dy"], at, x["nc"] * x["c"]).transpose(1, 2).contiguous()
        do = do.reshape(do.shape[:2] + (x["nc"], x["c"]) + do.shape[3:])
        k, q, beta = x["k"], x["q"], x["beta"]
        kf, u = x["fall"] * k, beta * e
        w = x["t"] @ (x["rise"] * k)
        direct = x["p"].transpose(-1, -2) @ do
        qd = scale * (x["rise"] * q).transpose(-1, -2) @ do
        wt = w.transpose(-1, -2).contiguous()
        ds = st["dfinal"].transpose(-1, -2).contiguous() if i == 0 and st["dfinal"] is not None else torch.zeros_like(first)
        dss, dus = [], []
        for j in reversed(range(x["nc"])):
            du = direct[:, :, j] + kf[:, :, j] @ ds
            dss.append(ds)
            dus.append(du)
            ds = x["last"][:, :, j, None, None] * ds + qd[:, :, j] - wt[:, :, j] @ (beta[:, :, j] * du)
        if i == 0 and st["dfinal"] is not None:
            dinit = ds.transpose(-1, -2).contiguous()
        ds1, du = torch.stack(dss[::-1], dim=2), torch.stack(dus[::-1], dim=2)
        df = x["t"].transpose(-1, -2) @ (beta * du)
        z = du - x["n"].transpose(-1, -2) @ df
        et, st_, dst = e.transpose(-1, -2), s.transpose(-1, -2), ds1.transpose(-1, -2)
        dp = (do @ et) * beta.transpose(-1, -2) * x["decay"] * scale
        dn = -(df @ et) * beta.transpose(-1, -2) * x["decay"] * x["lower"].tril(-1)
        dq = scale * x["rise"] * (do @ st_) + dp @ k
        row = dn @ k - x["rise"] * (df @ st_)
        fall = x["fall"] * (u @ dst)
        col = dp.transpose(-1, -2) @ q + dn.transpose(-1, -2) @ k + fall
        dlog = (q * dq).sum(dim=-1) + (k * (row - col)).sum(dim=-1)
        ends = x["last"] * (s * ds1).sum(dim=(-1, -2)) + (k * fall).sum(dim=(-1, -2))
        dlog = torch.cat([dlog[..., :-1], (dlog[..., -1] + ends).unsqueeze(-1)], dim=-1)
        dg = dlog.flip(-1).cumsum(dim=-1).flip(-1)
        H, G = d["v"].shape[2], d["k"].shape[2]
        got = {}
        for name, t in (("q", dq), ("k", row + col), ("v", df), ("g", dg), ("beta", (e * z).sum(dim=-1))):
            t = _flat(t)
            if name in ("q", "k"):
                t = t.reshape(t.shape[:2] + (G, H // G, t.shape[-1])).sum(dim=3)
            got[name] = torch.zeros(d[name].shape, device=t.device)
            _give(got[name], t, at)
        grads.append(got)
    return {"grads": grads, "dinit": dinit}


# ---- one pass ---------------------------------------------------------------

def _own(st):
    import bidirectional_mamba_ssm_amd as bm
    case = st["case"]
    op = case["op"]
    if op == "rms_norm":
        r = bm.rms_norm(st["x"], st["weight"], residual=st["residual"], eps=EPS, rows8=case["rows8"],
                        dense=case["dense"])
        res = {"sum": r["sum"], "rstd": r["rstd"]}
        if case["dense"]:
            res["out"] = r["out"]
        if case["rows8"]:
            res["rows8"] = r["rows8"]
        return res
    if op == "rms_norm_bwd":
        x = bm.Act8(*st["x"]) if case["ckpt"] else st["x"]
        dx, dw = bm.rms_norm_bwd(st["dout"], x, st["rstd"], st["weight"], dsum=st["dsum"])
        return {"dx": dx, "dweight": dw}
    if op == "linear8":
        x = bm.rows8_pack(st["x"]) if case["pack"] else bm.Rows8(*st["x"])
        return bm.linear8(x, bm.Rows8(*st["weight"]), st["bias"], dtype=st["dtype"])
    fwd, bwd = st["dirs"][0], st["dirs"][1] if case["both"] else None
    if op == "delta_step":
        y = bm.delta_step(st["state"], fwd, bwd, commit=case["commit"])
        return {"y": y, "state": st["state"]}
    if op == "delta_fwd":
        last = torch.empty_like(st["state"]) if case["state"] else None
        y = bm.delta_fwd(fwd, bwd, cu_seqlens=st["cu"], init_state=st["state"], final_state=last)
        return {"y": y, "last": last}
    dinit = torch.empty_like(st["state"]) if case["state"] else None
    gf, gb = bm.delta_bwd(fwd, bwd, st["dy"], cu_seqlens=st["cu"], init_state=st["state"], dfinal=st["dfinal"],
                          dinit=dinit)
    return {"grads": [gf, gb] if gb is not None else [gf], "dinit": dinit}


def run(st):
    if own:
        res = _own(st)
        if isinstance(res, dict) and "rows8" in res:
            # as the values that the 8 bits stand for
            r = res.pop("rows8")
            res["values"], res["scale"] = (r.q.float() * r.scale.unsqueeze(1)).to(torch.bfloat16), r.scale
        return res
    case = st["case"]
    op = case["op"]
    if op == "rms_norm":
        return _plain_rms_norm(st)
    if op == "rms_norm_bwd":
        return _plain_rms_norm_bwd(st)
    if op == "linear8":
        return _plain_linear8(st)
    if op == "delta_bwd":
        return _plain_delta_bwd(st)
    y, last = _plain_delta(st)
    if op == "delta_fwd":
        return {"y": y, "last": last if case["state"] else None}
    if case["commit"]:
        st["state"].copy_(last)
    return {"y": y, "state": st["state"]}


# ---- 64 bits, from the definitions ------------------------------------------

def _exact_quantized(v):
    top = v.abs().amax(dim=1, keepdim=True)
    q = torch.round(v * 127.0 / top.clamp(min=2.0 ** -100))
    return q, top / 127.0


def _exact_rows(st):
    case = st["case"]
    if case["op"] == "linear8":
        if case["pack"]:
            xq, xs = _exact_quantized(st["x"].double())
        else:
            xq, xs = st["x"][0].double(), st["x"][1].double().unsqueeze(1)
        out = (xq * xs) @ (st["weight"][0].double() * st["weight"][1].double().unsqueeze(1)).t()
        return out + st["bias"].double() if st["bias"] is not None else out
    w = st["weight"].double() if st["weight"] is not None else 1.0
    if case["op"] == "rms_norm":
        h = st["x"]
        if st["residual"] is not None:
            h = (h.double() + st["residual"].double()).to(st["dtype"])
        h = h.double()
        rstd = 1.0 / torch.sqrt((h * h).sum(dim=1) / h.shape[1] + EPS)
        o = h * rstd[:, None] * w
        res = {"sum": h, "rstd": rstd}
        if case["dense"]:
            res["out"] = o
        if case["rows8"]:
            q, scale = _exact_quantized(o)
            res["values"], res["scale"] = q * scale, scale[:, 0]
        return res
    if case["ckpt"]:
        q, scale = st["x"]
        unit = torch.exp2(scale.double() - 133.0).repeat_interleave(32, dim=1)[:, :q.shape[1]]
        x = q.double() * unit
    else:
        x = st["x"].double()
    r = st["rstd"].double()[:, None]
    do = st["dout"].double()
    # out = w x r, r = (mean x^2 + eps)^-1/2: dr/dx = -r^3 x / C
    dr = (do * w * x).sum(dim=1, keepdim=True)
    dx = do * w * r - dr * r ** 3 * x / x.shape[1]
    if st["dsum"] is not None:
        dx = dx + st["dsum"].double()
    return {"dx": dx, "dweight": (do * x * r).sum(dim=0)}


def _steps(t, at, rep=1):
    """t [b, L, ...] in the order of at, one 64-bit tensor [units, H, ...] a
    position; zeros where there is no token."""
    flat = t.double().reshape((-1,) + t.shape[2:])
    flat = torch.cat([flat, torch.zeros_like(flat[:1])])
    v = flat[torch.where(at < 0, torch.full_like(at, flat.shape[0] - 1), at)]
    return v.repeat_interleave(rep, dim=2) if rep > 1 else v


def _exact_delta(st):
    """Token by token. A place without a token has g = beta = 0 and leaves the
    state as it is."""
    case = st["case"]
    scale = 1.0 / math.sqrt(case["d_state"])
    bwd = case["op"] == "delta_bwd"
    y, last, grads, dinit = None, None, [], None
    for i, d in enumerate(st["dirs"]):
        at = st["places"][i]
        rep = case["nheads"] // case["ngroups"]
        q, k = _steps(d["q"], at, rep), _steps(d["k"], at, rep)
        v, g, beta = (_steps(d[n], at) for n in ("v", "g", "beta"))
        n = at.shape[1]
        S = torch.zeros(v.shape[0], v.shape[2], k.shape[-1], v.shape[-1], dtype=torch.float64, device=v.device)
        if i == 0 and st["state"] is not None:
            S = st["state"].double().transpose(-1, -2).contiguous()
        out = torch.zeros_like(v)
        kept = []
        for t in range(n):
            kt = k[:, t].unsqueeze(-1)
            S = torch.exp(g[:, t])[..., None, None] * S
            if bwd:
                kept.append(S)
            e = v[:, t] - (S * kt).sum(dim=-2)
            S = S + kt * (beta[:, t].unsqueeze(-1) * e).unsqueeze(-2)
            if not bwd:
                out[:, t] = scale * (S * q[:, t].unsqueeze(-1)).sum(dim=-2)
        live = at >= 0
        if not bwd:
            part = torch.zeros(d["v"].shape, dtype=torch.float64, device=v.device)
            part.reshape((-1,) + part.shape[2:])[at[live]] = out[live]
            y = part if y is None else y + part
            if i == 0:
                last = S.transpose(-1, -2).contiguous()
            continue
        dy = _steps(st["dy"], at)
        dS = torch.zeros_like(S)
        if i == 0 and st["dfinal"] is not None:
            dS = st["dfinal"].double().transpose(-1, -2).contiguous()
        got = {m: torch.zeros_like(t) for m, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta))}
        for t in reversed(range(n)):
            S = kept.pop()   # decayed, before the token's write
            kt, qt = k[:, t].unsqueeze(-1), q[:, t].unsqueeze(-1)
            e = v[:, t] - (S * kt).sum(dim=-2)
            b = beta[:, t].unsqueeze(-1)
            do = scale * dy[:, t].unsqueeze(-2)
            after = S + kt * (b * e).unsqueeze(-2)
            got["q"][:, t] = (after * do).sum(dim=-1)
            dS = dS + qt * do
            du = (dS * kt).sum(dim=-2)
            de = b * du
            got["beta"][:, t] = (du * e).sum(dim=-1)
            got["v"][:, t] = de
            got["k"][:, t] = (dS * (b * e).unsqueeze(-2)).sum(dim=-1) - (S * de.unsqueeze(-2)).sum(dim=-1)
            dS = dS - kt * de.unsqueeze(-2)
            got["g"][:, t] = (dS * S).sum(dim=(-1, -2))
            dS = torch.exp(g[:, t])[..., None, None] * dS
        if i == 0 and st["dfinal"] is not None:
            dinit = dS.transpose(-1, -2).contiguous()
        for m in ("q", "k"):
            t = got[m]
            got[m] = t.reshape(t.shape[:2] + (case["ngroups"], rep, t.shape[-1])).sum(dim=3)
        res = {}
        for m, t in got.items():
            res[m] = torch.zeros(d[m].shape, dtype=torch.float64, device=t.device)
            res[m].reshape((-1,) + res[m].shape[2:])[at[live]] = t[live]
        grads.append(res)
    if bwd:
        return {"grads": grads, "dinit": dinit}
    if case["op"] == "delta_fwd":
        return {"y": y, "last": last if case["state"] else None}
    return {"y": y, "state": last if case["commit"] else st["state"].double()}


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_delta(st) if case["op"].startswith("delta") else _exact_rows(st)

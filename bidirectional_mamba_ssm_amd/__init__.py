"""Bidirectional Mamba-2 SSD mixer on MI355X: thin Python binding.

Every step of the computation runs in libbimamba's HIP kernels; this module
only marshals torch tensors (device memory and the current stream) into the
C ABI declared in include/bimamba.h. It has no compute path of its own and
raises if the library is not built.

Every call is enqueued on the current stream of its tensors' device, or on
``stream``, which it then makes current while it runs: the results and
workspaces that it allocates belong to that stream, and the results may be
used on the stream that was current before, too. As with any torch call on a
side stream, the caller orders that stream against the ones its inputs come
from and its results go to.
"""
import array
import ctypes
import functools
import math

import torch

from . import _abi
from ._abi import BimambaError, LibraryMissing  # noqa: F401

DTYPES = {torch.float32: _abi.F32, torch.bfloat16: _abi.BF16}


def lib():
    return _abi.load()


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# Small calls are short next to their own overhead, so they take the current
# stream's handle and device without the objects that torch.cuda makes of them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _elsewhere(dev, stream):
    """Whether a call has to go through _run_on()."""
    return stream is not None or dev.index != _current_device()


def _on(dev, stream):
    """The context of a call on another stream than the current one, or on
    tensors of another device than the current one: both are made current, so
    that what the call allocates belongs to the stream it is used on."""
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    return torch.cuda.stream(stream)


def _run_on(dev, stream, call, *args):
    """call(*args) under _on(). Its results go back to the stream that was
    current, so their memory, which is the other stream's, is not given away
    before that stream has done with them, either."""
    outer = torch.cuda.current_stream(dev) if stream is not None else None
    with _on(dev, stream):
        res = call(*args)
    if outer is not None and outer != stream:
        for t in _tensors(res):
            t.record_stream(outer)
    return res


def _tensors(res):
    if isinstance(res, torch.Tensor):
        return [res]
    if isinstance(res, (Act8, Rows8)):
        return [res.q, res.scale]
    if isinstance(res, dict):
        res = res.values()
    return [t for r in res for t in _tensors(r)] if res is not None else []


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _check(t, name, shape, dtype, device):
    """The library sees plain pointers: every tensor's device, dtype, shape and
    layout is checked here, before anything is launched."""
    if type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.is_contiguous() \
            and t.get_device() == device.index:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _within_32_bits(vals, name):
    """ctypes passes on the low 32 bits of a larger number without a word, so
    every integer that the library takes as a C int is checked first."""
    if vals and not (-2 ** 31 <= min(vals) and max(vals) < 2 ** 31):
        raise ValueError(f"{name} goes beyond 32 bits ({min(vals)} .. {max(vals)})")


def _sizes(struct, name, *vals):
    """A structure of C ints."""
    try:
        return struct.from_buffer_copy(array.array("i", vals))   # checks the range as it converts
    except OverflowError:
        _within_32_bits(vals, name)
        raise


def _int32s(vals, name):
    """A C array of integers for the library."""
    try:
        a = array.array("i", vals)   # checks the range as it converts
    except OverflowError:
        _within_32_bits(vals, name)
        raise
    return (ctypes.c_int32 * len(a)).from_buffer(a)


def _int32(v, name):
    """An integer for the library."""
    v = int(v)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name} {v} is beyond 32 bits")
    return v


def _offsets(cu_seqlens):
    """(the C array, the number of sequences) of packed-sequence offsets."""
    if cu_seqlens is None:
        return None, 0
    vals = [int(v) for v in (cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist") else cu_seqlens)]
    return _int32s(vals, "cu_seqlens"), len(vals) - 1


def _cuda_device(x):
    if x.device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, not {x.device}")
    return x.device


def _dims(d):
    x, B = d["x"], d["B"]
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [batch, L, H, P] and B [batch, L, G, N]")
    batch, L, H, P = x.shape
    return batch, L, H, P, B.shape[2], B.shape[3]


def _dir(d, dtype, dims=None, device=None, name="fwd"):
    batch, L, H, P, G, N = dims if dims is not None else _dims(d)
    device = device if device is not None else d["x"].device
    _check(d["x"], f"{name}.x", (batch, L, H, P), dtype, device)
    _check(d["dt"], f"{name}.dt", (batch, L, H), dtype, device)
    _check(d["B"], f"{name}.B", (batch, L, G, N), dtype, device)
    _check(d["C"], f"{name}.C", (batch, L, G, N), dtype, device)
    _check(d["A"], f"{name}.A", (H,), torch.float32, device)
    if d.get("D") is not None:
        _check(d["D"], f"{name}.D", (H,), torch.float32, device)
    if d.get("dt_bias") is not None:
        _check(d["dt_bias"], f"{name}.dt_bias", (H,), torch.float32, device)
    return _abi.Dir(d["x"].data_ptr(), d["dt"].data_ptr(), d["A"].data_ptr(),
                    d["B"].data_ptr(), d["C"].data_ptr(),
                    d["D"].data_ptr() if d.get("D") is not None else None,
                    d["dt_bias"].data_ptr() if d.get("dt_bias") is not None else None)


def make_shape(x, B, chunk, seqlen=None, dt_softplus=False):
    """Shape of a problem whose x is [batch, L, H, P] and B [batch, L, G, N]."""
    batch, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    if x.dtype not in DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    return _sizes(_abi.Shape, "the problem's shape", batch, L if seqlen is None else seqlen, H, P, N, G, chunk,
                  DTYPES[x.dtype], _abi.DT_SOFTPLUS if dt_softplus else 0)


def _conv_shape(*sizes):
    return _sizes(_abi.ConvShape, "the convolution's shape", *sizes)


def workspace_size(shape, nseq=0):
    n = ctypes.c_size_t(0)
    _abi.check(lib().bimamba_ssd_workspace_size(ctypes.byref(shape), nseq, ctypes.byref(n)))
    return n.value


def ssd_fwd(fwd, bwd=None, chunk=256, cu_seqlens=None, init_state=None,
            final_state=None, y=None, workspace=None, stream=None, dt_softplus=False):
    """Bidirectional SSD (see include/bimamba.h, bimamba_ssd_fwd).

    fwd/bwd: dicts of device tensors x [b,L,H,P], dt [b,L,H], A [H] f32,
    B/C [b,L,G,N], D [H] f32 or None, and (with dt_softplus, where dt is the
    pre-activation) dt_bias [H] f32 or None. cu_seqlens: host list/tensor
    of nseq+1 offsets. Returns y (float32 [b,L,H,P]).
    """
    x = fwd["x"]
    dims = _dims(fwd)
    batch, L, H, P, G, N = dims
    dtype = x.dtype
    dev = _cuda_device(x)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, ssd_fwd, fwd, bwd, chunk, cu_seqlens, init_state, final_state, y, workspace,
                       None, dt_softplus)
    shape = make_shape(x, fwd["B"], chunk, dt_softplus=dt_softplus)
    fd = _dir(fwd, dtype, dims, dev, "fwd")
    bd = _dir(bwd, dtype, dims, dev, "bwd") if bwd is not None else None
    cu_arr, nseq = _offsets(cu_seqlens)
    units = nseq if cu_seqlens is not None else batch
    for t, name in ((init_state, "init_state"), (final_state, "final_state")):
        if t is not None:
            _check(t, name, (units, H, P, N), torch.float32, dev)
    if y is None:
        y = torch.empty(x.shape, dtype=torch.float32, device=dev)
    _check(y, "y", (batch, L, H, P), torch.float32, dev)
    need = workspace_size(shape, nseq)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _abi.check(lib().bimamba_ssd_fwd(
        ctypes.byref(shape), ctypes.byref(fd), ctypes.byref(bd) if bd is not None else None,
        cu_arr, nseq, _ptr(init_state), _ptr(final_state), _ptr(y),
        _ptr(workspace), ws_bytes, _raw_stream(dev.index)))
    return y


def bwd_workspace_size(shape, has_bwd=True):
    n = ctypes.c_size_t(0)
    _abi.check(lib().bimamba_ssd_bwd_workspace_size(ctypes.byref(shape), int(bool(has_bwd)),
                                                     ctypes.byref(n)))
    return n.value


def _grads(g, dims, dev, name):
    batch, L, H, P, G, N = dims
    shapes = {"x": (batch, L, H, P), "dt": (batch, L, H), "A": (H,),
              "B": (batch, L, G, N), "C": (batch, L, G, N), "D": (H,)}
    if g is None:
        g = {k: torch.empty(v, dtype=torch.float32, device=dev) for k, v in shapes.items()}
    for k, v in shapes.items():
        if k == "D" and g.get("D") is None:
            continue
        _check(g[k], f"{name}_grad.{k}", v, torch.float32, dev)
    return g, _abi.Grad(g["x"].data_ptr(), g["dt"].data_ptr(), g["A"].data_ptr(),
                        g["B"].data_ptr(), g["C"].data_ptr(),
                        g["D"].data_ptr() if g.get("D") is not None else None)


def ssd_bwd(fwd, bwd, dy, grads=None, workspace=None, stream=None):
    """Training backward of ssd_fwd (bimamba_ssd_bwd): gradients of every
    input of both streams given dy (float32 [b,L,H,P]). Returns (gfwd, gbwd),
    dicts of float32 tensors keyed x, dt, A, B, C, D (gbwd None without bwd).
    grads: optional (gfwd, gbwd) dicts to write into."""
    x = fwd["x"]
    dims = _dims(fwd)
    batch, L, H, P, G, N = dims
    dev = _cuda_device(x)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, ssd_bwd, fwd, bwd, dy, grads, workspace)
    shape = make_shape(x, fwd["B"], 64)
    fd = _dir(fwd, x.dtype, dims, dev, "fwd")
    bd = _dir(bwd, x.dtype, dims, dev, "bwd") if bwd is not None else None
    _check(dy, "dy", (batch, L, H, P), torch.float32, dev)
    gl = list(grads) if grads is not None else [None, None]
    gf, gfs = _grads(gl[0], dims, dev, "fwd")
    gb, gbs = _grads(gl[1], dims, dev, "bwd") if bwd is not None else (None, None)
    need = bwd_workspace_size(shape, bwd is not None)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _abi.check(lib().bimamba_ssd_bwd(
        ctypes.byref(shape), ctypes.byref(fd), ctypes.byref(bd) if bd is not None else None,
        _ptr(dy), ctypes.byref(gfs), ctypes.byref(gbs) if gbs is not None else None,
        _ptr(workspace), ws_bytes, _raw_stream(dev.index)))
    return gf, gb


def ssd_fwd_noalloc(fwd, bwd, y, chunk=256, cu_seqlens=None, init_state=None,
                    final_state=None, stream=None, dt_softplus=False):
    """bimamba_ssd_fwd_noalloc: ssd_fwd with the library's static device
    buffer as its workspace (the call allocates nothing; y is the caller's
    float32 [b,L,H,P]). Returns y."""
    x = fwd["x"]
    dims = _dims(fwd)
    batch, L, H, P, G, N = dims
    dev = _cuda_device(x)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, ssd_fwd_noalloc, fwd, bwd, y, chunk, cu_seqlens, init_state, final_state, None,
                       dt_softplus)
    shape = make_shape(x, fwd["B"], chunk, dt_softplus=dt_softplus)
    fd = _dir(fwd, x.dtype, dims, dev, "fwd")
    bd = _dir(bwd, x.dtype, dims, dev, "bwd") if bwd is not None else None
    cu_arr, nseq = _offsets(cu_seqlens)
    units = nseq if cu_seqlens is not None else batch
    for t, name in ((init_state, "init_state"), (final_state, "final_state")):
        if t is not None:
            _check(t, name, (units, H, P, N), torch.float32, dev)
    _check(y, "y", (batch, L, H, P), torch.float32, dev)
    _abi.check(lib().bimamba_ssd_fwd_noalloc(
        ctypes.byref(shape), ctypes.byref(fd), ctypes.byref(bd) if bd is not None else None,
        cu_arr, nseq, _ptr(init_state), _ptr(final_state), _ptr(y), _raw_stream(dev.index)))
    return y


def ssd_fwd_streams(fwd, bwd, chunk=256, cu_seqlens=None, init_state=None,
                    final_state=None, y_fwd=None, y_bwd=None, workspace=None, stream=None):
    """bimamba_ssd_fwd_streams: the two streams' outputs kept apart.
    Returns (y_fwd, y_bwd), float32 [b,L,H,P] each."""
    x = fwd["x"]
    dims = _dims(fwd)
    batch, L, H, P, G, N = dims
    dev = _cuda_device(x)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, ssd_fwd_streams, fwd, bwd, chunk, cu_seqlens, init_state, final_state, y_fwd,
                       y_bwd, workspace)
    shape = make_shape(x, fwd["B"], chunk)
    fd = _dir(fwd, x.dtype, dims, dev, "fwd")
    bd = _dir(bwd, x.dtype, dims, dev, "bwd")
    cu_arr, nseq = _offsets(cu_seqlens)
    units = nseq if cu_seqlens is not None else batch
    for t, name in ((init_state, "init_state"), (final_state, "final_state")):
        if t is not None:
            _check(t, name, (units, H, P, N), torch.float32, dev)
    outs = []
    for t, name in ((y_fwd, "y_fwd"), (y_bwd, "y_bwd")):
        if t is None:
            t = torch.empty(x.shape, dtype=torch.float32, device=dev)
        _check(t, name, (batch, L, H, P), torch.float32, dev)
        outs.append(t)
    need = workspace_size(shape, nseq)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _abi.check(lib().bimamba_ssd_fwd_streams(
        ctypes.byref(shape), ctypes.byref(fd), ctypes.byref(bd), cu_arr, nseq,
        _ptr(init_state), _ptr(final_state), _ptr(outs[0]), _ptr(outs[1]),
        _ptr(workspace), ws_bytes, _raw_stream(dev.index)))
    return outs[0], outs[1]


def merge_linear(y_fwd, y_bwd, weight, bias=None, out=None, stream=None):
    """bimamba_merge_linear: W [y_fwd ; y_bwd] + bias per token. y_fwd,
    y_bwd float32 [..., cin]; weight bf16 [cout, 2 cin]; bias float32 [cout]
    or None. Returns float32 [..., cout]."""
    dev = _cuda_device(y_fwd)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, merge_linear, y_fwd, y_bwd, weight, bias, out)
    cin = y_fwd.shape[-1]
    rows = y_fwd.numel() // cin if cin else 0
    cout = weight.shape[0]
    _check(y_fwd, "y_fwd", tuple(y_fwd.shape), torch.float32, dev)
    _check(y_bwd, "y_bwd", tuple(y_fwd.shape), torch.float32, dev)
    _check(weight, "weight", (cout, 2 * cin), torch.bfloat16, dev)
    if bias is not None:
        _check(bias, "bias", (cout,), torch.float32, dev)
    oshape = tuple(y_fwd.shape[:-1]) + (cout,)
    if out is None:
        out = torch.empty(oshape, dtype=torch.float32, device=dev)
    _check(out, "out", oshape, torch.float32, dev)
    _within_32_bits((cin, cout), "the merge's channels")
    _abi.check(lib().bimamba_merge_linear(rows, cin, cout, _ptr(y_fwd), _ptr(y_bwd), _ptr(weight),
                                          _ptr(bias), _ptr(out), _raw_stream(dev.index)))
    return out


class State:
    """Library-owned forward-state cache: float [nslots, H, P, N] on the GPU;
    with conv=(ngroups, width, dtype) it also carries the short convolution's
    context, [nslots, width-1, channels] of that dtype (bimamba_state_alloc_conv)."""

    def __init__(self, nslots, nheads, headdim, d_state, conv=None):
        self._h = ctypes.c_void_p()
        self.conv = None
        _within_32_bits((nslots, nheads, headdim, d_state) + tuple(conv[:2] if conv is not None else ()),
                        "the state's shape")
        if conv is None:
            _abi.check(lib().bimamba_state_alloc(ctypes.byref(self._h), nslots, nheads,
                                                 headdim, d_state))
        else:
            ngroups, width, dtype = conv
            if dtype not in DTYPES:
                raise TypeError(f"unsupported dtype {dtype}")
            _abi.check(lib().bimamba_state_alloc_conv(ctypes.byref(self._h), nslots, nheads, headdim,
                                                      d_state, ngroups, width, DTYPES[dtype]))
            ch = conv_channels(nheads, headdim, ngroups, d_state)
            self.conv = (ngroups, width, dtype, ch)
        self.shape = (nslots, nheads, headdim, d_state)
        self.device = torch.device("cuda", torch.cuda.current_device())

    def ctx_tensor(self):
        """A zero-copy torch view of the convolution context (valid while
        this object lives)."""
        if self.conv is None:
            raise ValueError("this state carries no convolution context")
        ptr = lib().bimamba_state_conv_ctx(self._h)
        _, width, dtype, ch = self.conv
        shape = (self.shape[0], width - 1, ch)
        typestr = "<f4" if dtype == torch.float32 else "<u2"

        class _View:
            __cuda_array_interface__ = {
                "shape": shape, "typestr": typestr, "data": (ptr, False),
                "version": 2, "strides": None}
        t = torch.as_tensor(_View(), device="cuda")
        return t.view(torch.bfloat16) if dtype == torch.bfloat16 else t

    def data_ptr(self):
        return lib().bimamba_state_data(self._h)

    def tensor(self):
        """A zero-copy torch view of the cache (valid while this object lives)."""
        ptr = self.data_ptr()
        shape = self.shape

        class _View:
            __cuda_array_interface__ = {
                "shape": shape, "typestr": "<f4", "data": (ptr, False),
                "version": 2, "strides": None}
        return torch.as_tensor(_View(), device="cuda")

    def reset(self, slots=None, stream=None):
        arr, n = None, 0
        if slots is not None:
            slots = [int(s) for s in slots]
            n = len(slots)
            arr = _int32s(slots or [0], "slots")
        _abi.check(lib().bimamba_state_reset(self._h, arr, n, _stream(stream)))

    def free(self):
        if self._h:
            _abi.check(lib().bimamba_state_free(self._h))
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h


def block_step(state, fwd, bwd, commit=False, chunk=64, y=None, stream=None, dt_softplus=False):
    """One cached block-diffusion step (bimamba_block_step)."""
    x = fwd["x"]
    dims = _dims(fwd)
    dev = _cuda_device(x)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, block_step, state, fwd, bwd, commit, chunk, y, None, dt_softplus)
    shape = make_shape(x, fwd["B"], chunk, dt_softplus=dt_softplus)
    fd = _dir(fwd, x.dtype, dims, dev, "fwd")
    bd = _dir(bwd, x.dtype, dims, dev, "bwd")
    if y is None:
        y = torch.empty(x.shape, dtype=torch.float32, device=x.device)
    _check(y, "y", tuple(x.shape), torch.float32, x.device)
    _abi.check(lib().bimamba_block_step(state.handle, ctypes.byref(shape), ctypes.byref(fd),
                                        ctypes.byref(bd), int(bool(commit)), _ptr(y),
                                        _raw_stream(dev.index)))
    return y


def block_step_conv(state, fwd, bwd, conv_fwd, conv_bwd, commit=False, chunk=64, y=None,
                    activation="silu", conv_out=None, stream=None, dt_softplus=False):
    """One cached block step from the block's raw convolution inputs
    (bimamba_block_step_conv) for a State made with conv=...: the short
    convolution of both directions (the forward one from the state's
    context), then the block step; with commit the SSM state and the
    context both move past the block.

    conv_fwd/conv_bwd: dicts xbc [b, L, ch], weight [ch, W] f32, bias [ch] f32
    or None. fwd/bwd: dicts dt, A, D (and optionally dt_bias) of each
    direction; x, B, C are the convolution's outputs (allocated here, or
    given in conv_out as for conv1d). Returns y."""
    if state.conv is None:
        raise ValueError("the state carries no convolution context")
    ngroups, W, cdtype, ch = state.conv
    xbc = conv_fwd["xbc"]
    dev = _cuda_device(xbc)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, block_step_conv, state, fwd, bwd, conv_fwd, conv_bwd, commit, chunk, y,
                       activation, conv_out, None, dt_softplus)
    if xbc.dim() != 3:
        raise ValueError("xbc must be [batch, L, channels]")
    batch, L, chx = xbc.shape
    _, H, P, N = state.shape
    if chx != ch or conv_fwd["weight"].shape != (ch, W) or xbc.dtype != cdtype:
        raise ValueError("the convolution's inputs do not match the state's context")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation {activation!r} is not one of {sorted(map(str, ACTIVATIONS))}")
    dims = (batch, L, ch, W)
    outs = list(conv_out) if conv_out is not None else [None, None]
    fo = _conv_out(outs[0], batch, L, H, P, ngroups, N, xbc.dtype, dev, "fwd")
    bo = _conv_out(outs[1], batch, L, H, P, ngroups, N, xbc.dtype, dev, "bwd")
    cfd = _conv_dir(conv_fwd, dims, xbc.dtype, dev, fo, "fwd")
    cbd = _conv_dir(conv_bwd, dims, xbc.dtype, dev, bo, "bwd")
    sf = dict(fwd, x=fo["x"], B=fo["B"], C=fo["C"])
    sb = dict(bwd, x=bo["x"], B=bo["B"], C=bo["C"])
    sdims = _dims(sf)
    shape = make_shape(fo["x"], fo["B"], chunk, dt_softplus=dt_softplus)
    fd = _dir(sf, xbc.dtype, sdims, dev, "fwd")
    bd = _dir(sb, xbc.dtype, sdims, dev, "bwd")
    if y is None:
        y = torch.empty((batch, L, H, P), dtype=torch.float32, device=dev)
    _check(y, "y", (batch, L, H, P), torch.float32, dev)
    cshape = _conv_shape(batch, L, H, P, N, ngroups, W, DTYPES[xbc.dtype], ACTIVATIONS[activation], 0)
    _abi.check(lib().bimamba_block_step_conv(
        state.handle, ctypes.byref(cshape), ctypes.byref(cfd), ctypes.byref(cbd),
        ctypes.byref(shape), ctypes.byref(fd), ctypes.byref(bd), int(bool(commit)), _ptr(y),
        _raw_stream(dev.index)))
    return y


class BlockStepPlan:
    """A block step with its arguments checked and bound once, for decode
    loops: run() calls bimamba_block_step on the same tensors (and the
    stream current at construction) without checking them again, so a step
    costs the C call and the launch. Write each step's inputs into the
    bound tensors in place; keep them alive and unchanged in shape while the
    plan is used. Same arguments as block_step."""

    def __init__(self, state, fwd, bwd, commit=False, chunk=64, y=None, stream=None,
                 dt_softplus=False):
        x = fwd["x"]
        dims = _dims(fwd)
        self._shape = make_shape(x, fwd["B"], chunk, dt_softplus=dt_softplus)
        dev = _cuda_device(x)
        self._fd = _dir(fwd, x.dtype, dims, dev, "fwd")
        self._bd = _dir(bwd, x.dtype, dims, dev, "bwd")
        if y is None:
            y = _run_on(dev, stream, functools.partial(torch.empty, x.shape, dtype=torch.float32, device=dev))
        _check(y, "y", tuple(x.shape), torch.float32, x.device)
        self.y = y
        self._state = state
        self._keep = (fwd, bwd)
        self._fn = lib().bimamba_block_step
        with _on(dev, stream):
            self._args = (ctypes.byref(self._shape), ctypes.byref(self._fd), ctypes.byref(self._bd),
                          int(bool(commit)), _ptr(y), _raw_stream(dev.index))

    def run(self):
        # the cache's handle is read per call: a freed cache is rejected by
        # the library instead of being used through a stale pointer
        rc = self._fn(self._state.handle, *self._args)
        if rc:
            _abi.check(rc)
        return self.y


ACTIVATIONS = {None: 0, "none": 0, "silu": 1}


def conv_channels(nheads, headdim, ngroups, d_state):
    return nheads * headdim + 2 * ngroups * d_state


def _conv_dir(d, dims, dtype, device, out, name):
    batch, L, ch, W = dims
    _check(d["xbc"], f"{name}.xbc", (batch, L, ch), dtype, device)
    _check(d["weight"], f"{name}.weight", (ch, W), torch.float32, device)
    if d.get("bias") is not None:
        _check(d["bias"], f"{name}.bias", (ch,), torch.float32, device)
    return _abi.ConvDir(d["xbc"].data_ptr(), d["weight"].data_ptr(),
                        d["bias"].data_ptr() if d.get("bias") is not None else None,
                        out["x"].data_ptr(), out["B"].data_ptr(), out["C"].data_ptr())


def _conv_out(out, batch, L, nheads, headdim, ngroups, d_state, dtype, device, name):
    if out is None:
        out = dict(x=torch.empty(batch, L, nheads, headdim, dtype=dtype, device=device),
                   B=torch.empty(batch, L, ngroups, d_state, dtype=dtype, device=device),
                   C=torch.empty(batch, L, ngroups, d_state, dtype=dtype, device=device))
    _check(out["x"], f"{name}_out.x", (batch, L, nheads, headdim), dtype, device)
    _check(out["B"], f"{name}_out.B", (batch, L, ngroups, d_state), dtype, device)
    _check(out["C"], f"{name}_out.C", (batch, L, ngroups, d_state), dtype, device)
    return out


def conv1d(fwd, bwd, nheads, headdim, ngroups, d_state, activation="silu",
           cu_seqlens=None, init_ctx=None, final_ctx=None, out=None, stream=None, dtype=None):
    """Short depthwise convolution of the scan inputs (bimamba_conv1d).

    fwd/bwd: dicts of device tensors xbc [b,L,ch] (x | B | C channels, bf16 or
    fp32), weight [ch,W] f32, bias [ch] f32 or None; bwd may be None.
    init_ctx/final_ctx: [b, W-1, ch] in xbc's dtype (may be the same tensor).
    out: optional (fwd_out, bwd_out) dicts of x, B, C to write.
    xbc may be an Act8 checkpoint of it, in both directions or neither
    (bimamba_conv1d_act8; no contexts): dtype is then the outputs' (bf16 if
    not given).
    Returns (fwd_out, bwd_out), each a dict x [b,L,H,P], B, C [b,L,G,N].
    """
    xbc = fwd["xbc"]
    if isinstance(xbc, Act8):
        if init_ctx is not None or final_ctx is not None:
            raise ValueError("a convolution from a checkpoint takes no contexts")
        return _conv1d_act8(fwd, bwd, (nheads, headdim, ngroups, d_state), activation, cu_seqlens, out,
                            dtype if dtype is not None else torch.bfloat16, stream)
    if dtype is not None and dtype != xbc.dtype:
        raise TypeError(f"dtype {dtype} is not xbc's {xbc.dtype}")
    dev = _cuda_device(xbc)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, conv1d, fwd, bwd, nheads, headdim, ngroups, d_state, activation, cu_seqlens,
                       init_ctx, final_ctx, out)
    if xbc.dim() != 3 or fwd["weight"].dim() != 2:
        raise ValueError("xbc must be [batch, L, channels] and weight [channels, width]")
    batch, L, ch = xbc.shape
    W = fwd["weight"].shape[1]
    if ch != conv_channels(nheads, headdim, ngroups, d_state):
        raise ValueError(f"xbc has {ch} channels, expected nheads*headdim + 2*ngroups*d_state")
    if xbc.dtype not in DTYPES:
        raise TypeError(f"unsupported dtype {xbc.dtype}")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation {activation!r} is not one of {sorted(map(str, ACTIVATIONS))}")
    dims = (batch, L, ch, W)
    outs = list(out) if out is not None else [None, None]
    fo = _conv_out(outs[0], batch, L, nheads, headdim, ngroups, d_state, xbc.dtype, dev, "fwd")
    fd = _conv_dir(fwd, dims, xbc.dtype, dev, fo, "fwd")
    bo = bd = None
    if bwd is not None:
        bo = _conv_out(outs[1], batch, L, nheads, headdim, ngroups, d_state, xbc.dtype, dev, "bwd")
        bd = _conv_dir(bwd, dims, xbc.dtype, dev, bo, "bwd")
    cu_arr, nseq = _offsets(cu_seqlens)
    for t, name in ((init_ctx, "init_ctx"), (final_ctx, "final_ctx")):
        if t is not None:
            _check(t, name, (batch, W - 1, ch), xbc.dtype, dev)
    shape = _conv_shape(batch, L, nheads, headdim, d_state, ngroups, W,
                        DTYPES[xbc.dtype], ACTIVATIONS[activation], 0)
    n = ctypes.c_size_t(0)
    _abi.check(lib().bimamba_conv1d_workspace_size(ctypes.byref(shape), nseq, ctypes.byref(n)))
    ws = torch.empty(n.value, dtype=torch.uint8, device=dev) if n.value else None
    _abi.check(lib().bimamba_conv1d(
        ctypes.byref(shape), ctypes.byref(fd), ctypes.byref(bd) if bd is not None else None,
        cu_arr, nseq, _ptr(init_ctx), _ptr(final_ctx), _ptr(ws), n.value, _raw_stream(dev.index)))
    return fo, bo


def gated_norm(y, z, weight, group_size=None, eps=1e-5, out=None, stream=None):
    """Gated RMS norm on the scan output (bimamba_gated_norm): y float32
    [..., C], z [..., C] (bf16 or fp32, also the output dtype), weight
    float32 [C]. group_size defaults to C (one group)."""
    dev = _cuda_device(y)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, gated_norm, y, z, weight, group_size, eps, out)
    C = y.shape[-1]
    rows = y.numel() // C if C else 0
    if z.dtype not in DTYPES:
        raise TypeError(f"unsupported dtype {z.dtype}")
    _check(y, "y", tuple(y.shape), torch.float32, dev)
    _check(z, "z", tuple(y.shape), z.dtype, dev)
    _check(weight, "weight", (C,), torch.float32, dev)
    if out is None:
        out = torch.empty(y.shape, dtype=z.dtype, device=dev)
    _check(out, "out", tuple(y.shape), z.dtype, dev)
    gs = _int32(C if group_size is None else group_size, "group_size")
    _abi.check(lib().bimamba_gated_norm(rows, _int32(C, "channels"), gs, DTYPES[z.dtype], _ptr(y), _ptr(z), _ptr(weight), float(eps),
                                        _ptr(out), _raw_stream(dev.index)))
    return out


def _adr(t):
    return None if t is None else t.data_ptr()


def _out(t, name, shape, dtype, dev, like=None):
    """The caller's output, checked, or a new one; like: a tensor of just that
    kind, which is the quicker way to one."""
    if t is None:
        return torch.empty_like(like) if like is not None else torch.empty(shape, dtype=dtype, device=dev)
    _check(t, name, shape, dtype, dev)
    return t


@functools.lru_cache(maxsize=4096)
def _size(query, *sizes):
    """What a workspace query (an entry point's name) says of plain sizes."""
    n = ctypes.c_size_t(0)
    _abi.check(getattr(lib(), query)(*sizes, ctypes.byref(n)))
    return n.value


@functools.lru_cache(maxsize=4096)
def _conv_size(query, shape, *sizes):
    """(the workspace, the bimamba_conv_shape to pass, which the library only
    reads) for plain sizes."""
    n = ctypes.c_size_t(0)
    cshape = ctypes.byref(_conv_shape(*shape))
    _abi.check(getattr(lib(), query)(cshape, *sizes, ctypes.byref(n)))
    return n.value, cshape


def _workspace(nbytes, dev):
    return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None


class Act8:
    """An activation kept in 8 bits (include/bimamba.h, bimamba_act8): q int8
    [..., C] and scale uint8 [..., (C + 31) // 32], the exponent that each 32
    consecutive channels share. Made by act8_pack or layer_norm; read by
    act8_unpack and, in place of the tensor, by conv1d, conv1d_bwd,
    gated_norm_bwd and layer_norm_bwd."""

    __slots__ = ("q", "scale")

    def __init__(self, q, scale):
        self.q, self.scale = q, scale

    @property
    def shape(self):
        return self.q.shape

    @property
    def device(self):
        return self.q.device

    @staticmethod
    def empty(shape, device):
        shape = tuple(shape)
        return Act8(torch.empty(shape, dtype=torch.int8, device=device),
                    torch.empty(shape[:-1] + ((shape[-1] + 31) // 32,), dtype=torch.uint8, device=device))

    def _checked(self, name, shape, dev):
        """The addresses of q and scale."""
        _check(self.q, name + ".q", shape, torch.int8, dev)
        _check(self.scale, name + ".scale", shape[:-1] + ((shape[-1] + 31) // 32,), torch.uint8, dev)
        return self.q.data_ptr(), self.scale.data_ptr()

    def _ptrs(self, name, shape, dev):
        return _abi.Act8Ptrs(*self._checked(name, tuple(shape), dev))


def _rows(shape):
    """(rows, channels) of [..., channels]."""
    if not shape or not shape[-1]:
        raise ValueError(f"shape {tuple(shape)} has no channels")
    if shape[-1] >= 2 ** 31:
        raise ValueError(f"{shape[-1]} channels are beyond 2^31 - 1")
    return math.prod(shape[:-1]), shape[-1]


def _kept(t, name, shape, dtype, dev):
    """The addresses (data, scale) of a tensor (scale None) or of its 8-bit
    checkpoint."""
    if isinstance(t, Act8):
        return t._checked(name, shape, dev)
    _check(t, name, shape, dtype, dev)
    return t.data_ptr(), None


def _dtype_code(dtype):
    code = DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def act8_pack(x, out=None, stream=None):
    """x [..., C] (bf16 or fp32) as an 8-bit checkpoint (bimamba_act8_pack).
    out: an Act8 to write. Returns the Act8."""
    dev = _cuda_device(x)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, act8_pack, x, out)
    code, shape = _dtype_code(x.dtype), tuple(x.shape)
    _check(x, "x", shape, x.dtype, dev)
    rows, C = _rows(shape)
    if out is None:
        out = Act8.empty(shape, dev)
        p = _abi.Act8Ptrs(out.q.data_ptr(), out.scale.data_ptr())
    else:
        p = out._ptrs("out", shape, dev)
    rc = lib().bimamba_act8_pack(rows, C, code, x.data_ptr(), ctypes.byref(p), _raw_stream(dev.index))
    if rc:
        _abi.check(rc)
    return out


def act8_unpack(a, dtype=torch.bfloat16, out=None, stream=None):
    """The values an Act8 stands for, as bf16 or fp32 (bimamba_act8_unpack)."""
    dev = _cuda_device(a)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, act8_unpack, a, dtype, out)
    code, shape = _dtype_code(dtype), tuple(a.shape)
    rows, C = _rows(shape)
    p = a._ptrs("a", shape, dev)
    out = _out(out, "out", shape, dtype, dev)
    rc = lib().bimamba_act8_unpack(rows, C, code, ctypes.byref(p), out.data_ptr(), _raw_stream(dev.index))
    if rc:
        _abi.check(rc)
    return out


def layer_norm(x, weight=None, bias=None, residual=None, eps=1e-5, checkpoint=False, out=None,
               sum_out=None, stream=None):
    """Layer norm over the last dimension (bimamba_layer_norm) of h = x, or of
    h = x + residual rounded to x's dtype. x, residual [..., C] bf16 or fp32,
    C in 8..16384; weight, bias float32 [C] or None.

    checkpoint: keep h in 8 bits too (True, or an Act8 to write). sum_out:
    where to write h with a residual. sum_out may be residual or x itself,
    and so may out with a residual (without one x is what sum returns). Other
    overlaps are refused. Returns a dict: out, sum (h; x itself without a
    residual), mean and rstd (float32 [...], for layer_norm_bwd), ckpt (Act8
    or None)."""
    dev = _cuda_device(x)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, layer_norm, x, weight, bias, residual, eps, checkpoint, out, sum_out)
    dt, shape = x.dtype, tuple(x.shape)
    code = _dtype_code(dt)
    _check(x, "x", shape, dt, dev)
    rows, C = _rows(shape)
    if residual is not None:
        _check(residual, "residual", shape, dt, dev)
    elif sum_out is not None:
        raise ValueError("sum_out goes with a residual")
    if weight is not None:
        _check(weight, "weight", (C,), torch.float32, dev)
    if bias is not None:
        _check(bias, "bias", (C,), torch.float32, dev)
    if out is None:
        out = torch.empty_like(x)
    else:
        _check(out, "out", shape, dt, dev)
        if residual is None and rows and out.data_ptr() == x.data_ptr():
            raise ValueError("out overlaps x, which is returned as sum without a residual")
    if residual is not None:
        sum_out = _out(sum_out, "sum_out", shape, dt, dev, x)
    mean, rstd = torch.empty((2,) + shape[:-1], dtype=torch.float32, device=dev).unbind(0)
    ckpt = p = None
    if checkpoint:
        ckpt = checkpoint if isinstance(checkpoint, Act8) else Act8.empty(shape, dev)
        p = ctypes.byref(ckpt._ptrs("checkpoint", shape, dev))
    rc = lib().bimamba_layer_norm(
        rows, C, code, x.data_ptr(), _adr(residual), _adr(weight), _adr(bias), float(eps), out.data_ptr(), _adr(sum_out),
        mean.data_ptr(), rstd.data_ptr(), p, _raw_stream(dev.index))
    if rc:
        _abi.check(rc)
    return dict(out=out, sum=x if residual is None else sum_out, mean=mean, rstd=rstd, ckpt=ckpt)


def layer_norm_bwd(dout, x, mean, rstd, weight=None, dsum=None, wgrad=True, dx=None, stream=None):
    """Gradient of layer_norm (bimamba_layer_norm_bwd). dout [..., C]; x: what
    layer_norm returned as sum (dout's dtype) or its Act8 checkpoint; mean,
    rstd float32 [...]; dsum: the gradient reaching sum along the residual
    stream, added to dx. dx (where to write it) may be dout, dsum or the
    tensor x itself; other overlaps are refused. Returns (dx, dweight, dbias):
    dx in dout's dtype (the gradient of x and of residual), the other two
    float32 [C], None with wgrad=False."""
    dev = _cuda_device(dout)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, layer_norm_bwd, dout, x, mean, rstd, weight, dsum, wgrad, dx)
    dt, shape = dout.dtype, tuple(dout.shape)
    code = _dtype_code(dt)
    _check(dout, "dout", shape, dt, dev)
    rows, C = _rows(shape)
    xp, xs = _kept(x, "x", shape, dt, dev)
    _check(mean, "mean", shape[:-1], torch.float32, dev)
    _check(rstd, "rstd", shape[:-1], torch.float32, dev)
    if weight is not None:
        _check(weight, "weight", (C,), torch.float32, dev)
    if dsum is not None:
        _check(dsum, "dsum", shape, dt, dev)
    dx = _out(dx, "dx", shape, dt, dev, dout)
    dw = db = ws = None
    nbytes = 0
    if wgrad:
        if weight is not None:
            dw, db = torch.empty_like(weight), torch.empty_like(weight)
        else:
            dw, db = torch.empty((2, C), dtype=torch.float32, device=dev).unbind(0)
        nbytes = _size("bimamba_layer_norm_bwd_workspace_size", rows, C, code)
        ws = _workspace(nbytes, dev)
    rc = lib().bimamba_layer_norm_bwd(
        rows, C, code, xp, xs, mean.data_ptr(), rstd.data_ptr(), _adr(weight), dout.data_ptr(), _adr(dsum),
        dx.data_ptr(), _adr(dw), _adr(db), _adr(ws), nbytes, _raw_stream(dev.index))
    if rc:
        _abi.check(rc)
    return dx, dw, db


def gated_norm_bwd(dout, y, z, weight, group_size=None, eps=1e-5, wgrad=True, dy=None, dz=None, stream=None):
    """Gradient of gated_norm (bimamba_gated_norm_bwd): dout [..., C] in z's
    dtype, y float32 and z [..., C] (each the tensor or its Act8 checkpoint).
    dy and dz (where to write them) may each be one of the tensors y, z and
    dout of its dtype; other overlaps are refused. Returns (dy float32, dz in dout's dtype,
    dweight float32 [C] or None)."""
    dev = _cuda_device(dout)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, gated_norm_bwd, dout, y, z, weight, group_size, eps, wgrad, dy, dz)
    dt, shape = dout.dtype, tuple(dout.shape)
    code = _dtype_code(dt)
    _check(dout, "dout", shape, dt, dev)
    rows, C = _rows(shape)
    gs = C if group_size is None else _int32(group_size, "group_size")
    yp, ys = _kept(y, "y", shape, torch.float32, dev)
    zp, zs = _kept(z, "z", shape, dt, dev)
    _check(weight, "weight", (C,), torch.float32, dev)
    dy = _out(dy, "dy", shape, torch.float32, dev)
    dz = _out(dz, "dz", shape, dt, dev, dout)
    dw = ws = None
    nbytes = 0
    if wgrad:
        dw = torch.empty_like(weight)
        nbytes = _size("bimamba_gated_norm_bwd_workspace_size", rows, C, gs, code)
        ws = _workspace(nbytes, dev)
    rc = lib().bimamba_gated_norm_bwd(
        rows, C, gs, code, yp, ys, zp, zs, weight.data_ptr(), float(eps), dout.data_ptr(), dy.data_ptr(), dz.data_ptr(),
        _adr(dw), _adr(ws), nbytes, _raw_stream(dev.index))
    if rc:
        _abi.check(rc)
    return dy, dz, dw


def _conv_plan(xbc, weight, dims, activation, dtype):
    """The plain sizes of a bimamba_conv_shape, for an xbc that is a tensor or
    an Act8."""
    if len(xbc.shape) != 3 or weight.dim() != 2:
        raise ValueError("xbc must be [batch, L, channels] and weight [channels, width]")
    batch, L, ch = xbc.shape
    H, P, G, N = dims
    if ch != conv_channels(H, P, G, N):
        raise ValueError(f"xbc has {ch} channels, expected nheads*headdim + 2*ngroups*d_state")
    if max(batch, L, ch) >= 2 ** 31:
        raise ValueError(f"xbc's shape {tuple(xbc.shape)} is beyond 2^31 - 1")
    code = _dtype_code(dtype)
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation {activation!r} is not one of {sorted(map(str, ACTIVATIONS))}")
    return (batch, L, H, P, N, G, weight.shape[1], code, ACTIVATIONS[activation], 0), ch


def _conv1d_act8(fwd, bwd, dims, activation, cu_seqlens, out, dtype, stream):
    xbc = fwd["xbc"]
    dev = _cuda_device(xbc)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, _conv1d_act8, fwd, bwd, dims, activation, cu_seqlens, out, dtype, None)
    sizes, ch = _conv_plan(xbc, fwd["weight"], dims, activation, dtype)
    batch, L, W = sizes[0], sizes[1], sizes[6]
    H, P, G, N = dims
    outs = out if out is not None else (None, None)
    cu_arr, nseq = _offsets(cu_seqlens)
    res, args = [None, None], [None, None, None, None]
    for i, (d, name) in enumerate(((fwd, "fwd"), (bwd, "bwd"))):
        if d is None:
            continue
        if not isinstance(d["xbc"], Act8):
            raise TypeError("both directions' xbc must be Act8, or neither")
        q, scale = d["xbc"]._checked(name + ".xbc", (batch, L, ch), dev)
        _check(d["weight"], name + ".weight", (ch, W), torch.float32, dev)
        bias = d.get("bias")
        if bias is not None:
            _check(bias, name + ".bias", (ch,), torch.float32, dev)
        o = outs[i]
        if o is None:
            o = dict(x=torch.empty((batch, L, H, P), dtype=dtype, device=dev),
                     B=torch.empty((batch, L, G, N), dtype=dtype, device=dev))
            o["C"] = torch.empty_like(o["B"])
        else:
            _conv_out(o, batch, L, H, P, G, N, dtype, dev, name)
        res[i] = o
        args[2 * i] = ctypes.byref(_abi.ConvDir(None, d["weight"].data_ptr(), _adr(bias), o["x"].data_ptr(),
                                                o["B"].data_ptr(), o["C"].data_ptr()))
        args[2 * i + 1] = ctypes.byref(_abi.Act8Ptrs(q, scale))
    nbytes, cshape = _conv_size("bimamba_conv1d_act8_workspace_size", sizes, nseq)
    ws = _workspace(nbytes, dev)
    rc = lib().bimamba_conv1d_act8(cshape, *args, cu_arr, nseq, _adr(ws), nbytes,
                                   _raw_stream(dev.index))
    if rc:
        _abi.check(rc)
    return res[0], res[1]


def conv1d_bwd(fwd, bwd, gfwd, gbwd, nheads, headdim, ngroups, d_state, activation="silu",
               cu_seqlens=None, out=None, stream=None, dtype=None):
    """Gradient of conv1d (bimamba_conv1d_bwd), both directions in one call.

    fwd/bwd: the forward's dicts, xbc [b,L,ch] (or its Act8 checkpoint, in
    both directions or neither), weight [ch,W] f32, bias [ch] f32 or None;
    bwd may be None. gfwd/gbwd: float32 gradients of its outputs, dicts with
    x [b,L,H,P], B and C [b,L,G,N] (ssd_bwd's results serve as they are).
    dtype: of the returned xbc gradients; xbc's own unless xbc is a
    checkpoint (then bf16 if not given). out: optional (fwd, bwd) tensors for
    the xbc gradients; they may not overlap each other or an input (xbc
    itself least of all: a token's gradient is made from its neighbours').
    Returns (fwd, bwd) dicts: xbc [b,L,ch] in that dtype, weight [ch,W] and
    bias [ch] (None without a bias) float32; bwd None if not given."""
    xbc = fwd["xbc"]
    dev = _cuda_device(xbc)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, conv1d_bwd, fwd, bwd, gfwd, gbwd, nheads, headdim, ngroups, d_state, activation,
                       cu_seqlens, out, None, dtype)
    q8 = isinstance(xbc, Act8)
    if dtype is None:
        dtype = torch.bfloat16 if q8 else xbc.dtype
    elif not q8 and dtype != xbc.dtype:
        raise TypeError(f"dtype {dtype} is not xbc's {xbc.dtype}")
    H, P, G, N = nheads, headdim, ngroups, d_state
    sizes, ch = _conv_plan(xbc, fwd["weight"], (H, P, G, N), activation, dtype)
    batch, L, W = sizes[0], sizes[1], sizes[6]
    if (bwd is None) != (gbwd is None):
        raise ValueError("bwd and gbwd come together")
    cu_arr, nseq = _offsets(cu_seqlens)
    outs = out if out is not None else (None, None)
    f32 = torch.float32
    res, args = [None, None], [None, None]
    for i, (d, g, name) in enumerate(((fwd, gfwd, "fwd"), (bwd, gbwd, "bwd"))):
        if d is None:
            continue
        if isinstance(d["xbc"], Act8) != q8:
            raise TypeError("both directions' xbc must be Act8, or neither")
        xp, xs = _kept(d["xbc"], name + ".xbc", (batch, L, ch), dtype, dev)
        w, bias, gx, gB, gC = d["weight"], d.get("bias"), g["x"], g["B"], g["C"]
        _check(w, name + ".weight", (ch, W), f32, dev)
        _check(gx, name + "_grad.x", (batch, L, H, P), f32, dev)
        _check(gB, name + "_grad.B", (batch, L, G, N), f32, dev)
        _check(gC, name + "_grad.C", (batch, L, G, N), f32, dev)
        dxbc = _out(outs[i], name + "_out", (batch, L, ch), dtype, dev, None if q8 else d["xbc"])
        dw = torch.empty_like(w)
        db = None
        if bias is not None:
            _check(bias, name + ".bias", (ch,), f32, dev)
            db = torch.empty_like(bias)
        res[i] = dict(xbc=dxbc, weight=dw, bias=db)
        args[i] = ctypes.byref(_abi.ConvGrad(xp, xs, w.data_ptr(), _adr(bias), gx.data_ptr(), gB.data_ptr(),
                                             gC.data_ptr(), dxbc.data_ptr(), dw.data_ptr(), _adr(db)))
    nbytes, cshape = _conv_size("bimamba_conv1d_bwd_workspace_size", sizes, 0 if bwd is None else 1, nseq)
    ws = _workspace(nbytes, dev)
    rc = lib().bimamba_conv1d_bwd(cshape, args[0], args[1], cu_arr, nseq, _adr(ws),
                                  nbytes, _raw_stream(dev.index))
    if rc:
        _abi.check(rc)
    return res[0], res[1]


def seq_index(cu_seqlens, device="cuda", stream=None):
    """Per-token packed-sequence index built on the GPU (int32 [total])."""
    arr, nseq = _offsets(cu_seqlens)
    total = arr[nseq]
    if torch.device(device).type != "cuda":
        raise ValueError(f"device must be a CUDA device, not {device}")
    dev = torch.device(device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, seq_index, cu_seqlens, dev)
    out = torch.empty(max(total, 1), dtype=torch.int32, device=dev)
    _abi.check(lib().bimamba_seq_index(arr, nseq, total, _ptr(out), _raw_stream(dev.index)))
    return out[:total]


class profile:
    """Context manager: per-kernel launch counts and summed device time (ms)
    of every library kernel launched from this thread inside the block,
    measured with HIP events on each kernel's stream.

        with bm.profile() as prof:
            bm.ssd_fwd(...)
        prof.kernels  # {name: (launches, total_ms)}
    """

    def __enter__(self):
        _abi.check(lib().bimamba_profile_begin())
        self.kernels = {}
        return self

    def __exit__(self, *exc):
        cap, nl = 64, 64
        names = ctypes.create_string_buffer(cap * nl)
        counts = (ctypes.c_int * cap)()
        ms = (ctypes.c_double * cap)()
        n = lib().bimamba_profile_end(names, nl, counts, ms, cap)
        if n < 0:
            _abi.check(n)
        raw = names.raw
        for i in range(min(n, cap)):
            name = raw[i * nl:(i + 1) * nl].split(b"\0", 1)[0].decode()
            self.kernels[name] = (counts[i], ms[i])
        return False


class Rows8:
    """Rows of 8-bit integers with a scale each (include/bimamba.h,
    bimamba_rows8): q int8 [..., C] and scale float32 [...]; a row stands for
    q * scale. Made by rows8_pack (activations, or a weight [cout, cin] by output
    channel) or rms_norm; read by linear8."""

    __slots__ = ("q", "scale")

    def __init__(self, q, scale):
        self.q, self.scale = q, scale

    @property
    def shape(self):
        return self.q.shape

    @property
    def device(self):
        return self.q.device

    @staticmethod
    def empty(shape, device):
        shape = tuple(shape)
        return Rows8(torch.empty(shape, dtype=torch.int8, device=device),
                     torch.empty(shape[:-1], dtype=torch.float32, device=device))

    def _ptrs(self, name, shape, dev):
        _check(self.q, name + ".q", shape, torch.int8, dev)
        _check(self.scale, name + ".scale", shape[:-1], torch.float32, dev)
        return _abi.Rows8Ptrs(self.q.data_ptr(), self.scale.data_ptr())


def _rows8(r, name):
    if not isinstance(r, Rows8):
        raise TypeError(f"{name} must be a Rows8, not {type(r).__name__}")
    return r


def rows8_pack(x, out=None, stream=None):
    """x [..., C] (bf16 or fp32, C in 8..16384) as 8-bit rows
    (bimamba_rows8_pack). out: a Rows8 to write. Returns the Rows8."""
    dev = _cuda_device(x)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, rows8_pack, x, out)
    code, shape = _dtype_code(x.dtype), tuple(x.shape)
    _check(x, "x", shape, x.dtype, dev)
    rows, C = _rows(shape)
    out = Rows8.empty(shape, dev) if out is None else _rows8(out, "out")
    p = out._ptrs("out", shape, dev)
    rc = lib().bimamba_rows8_pack(rows, C, code, x.data_ptr(), ctypes.byref(p), _raw_stream(dev.index))
    if rc:
        _abi.check(rc)
    return out


def rms_norm(x, weight=None, residual=None, eps=1e-5, rows8=False, dense=None, out=None, sum_out=None, stream=None):
    """RMS norm over the last dimension (bimamba_rms_norm) of h = x, or of
    h = x + residual rounded to x's dtype. x, residual [..., C] bf16 or fp32,
    C in 8..16384; weight float32 [C] or None.

    rows8: write the result as 8-bit rows for linear8 (True, or a Rows8 to
    write). dense: write it in x's dtype; unless said, where rows8 is not
    asked for or out is given. sum_out: where to write h with a residual. out
    and sum_out may be residual or x itself with a residual (without one x is
    what sum returns); other overlaps are refused. Returns a dict: out (or
    None), sum (h; x itself without a residual), rstd (float32 [...], for
    rms_norm_bwd), rows8 (Rows8 or None)."""
    dev = _cuda_device(x)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, rms_norm, x, weight, residual, eps, rows8, dense, out, sum_out)
    dt, shape = x.dtype, tuple(x.shape)
    code = _dtype_code(dt)
    _check(x, "x", shape, dt, dev)
    rows, C = _rows(shape)
    if residual is not None:
        _check(residual, "residual", shape, dt, dev)
        sum_out = _out(sum_out, "sum_out", shape, dt, dev, x)
    elif sum_out is not None:
        raise ValueError("sum_out goes with a residual")
    if weight is not None:
        _check(weight, "weight", (C,), torch.float32, dev)
    if dense is None:
        dense = not rows8 or out is not None
    if not dense and (out is not None or not rows8):
        raise ValueError("dense=False goes with rows8 and without out")
    if dense:
        if out is not None and residual is None and rows and out.data_ptr() == x.data_ptr():
            raise ValueError("out overlaps x, which is returned as sum without a residual")
        out = _out(out, "out", shape, dt, dev, x)
    rstd = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
    r8 = p = None
    if rows8:
        r8 = rows8 if isinstance(rows8, Rows8) else Rows8.empty(shape, dev)
        p = ctypes.byref(r8._ptrs("rows8", shape, dev))
    rc = lib().bimamba_rms_norm(rows, C, code, x.data_ptr(), _adr(residual), _adr(weight), float(eps), _adr(out),
                                _adr(sum_out), rstd.data_ptr(), p, _raw_stream(dev.index))
    if rc:
        _abi.check(rc)
    return dict(out=out, sum=x if residual is None else sum_out, rstd=rstd, rows8=r8)


def rms_norm_bwd(dout, x, rstd, weight=None, dsum=None, wgrad=True, dx=None, stream=None):
    """Gradient of rms_norm's out (bimamba_rms_norm_bwd). dout [..., C]; x:
    what rms_norm returned as sum (dout's dtype) or its Act8 checkpoint; rstd
    float32 [...]; dsum: the gradient reaching sum along the residual stream,
    added to dx. dx (where to write it) may be dout, dsum or the tensor x
    itself; other overlaps are refused. Returns (dx, dweight): dx in dout's
    dtype (the gradient of x and of residual), dweight float32 [C], None with
    wgrad=False."""
    dev = _cuda_device(dout)
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, rms_norm_bwd, dout, x, rstd, weight, dsum, wgrad, dx)
    dt, shape = dout.dtype, tuple(dout.shape)
    code = _dtype_code(dt)
    _check(dout, "dout", shape, dt, dev)
    rows, C = _rows(shape)
    xp, xs = _kept(x, "x", shape, dt, dev)
    _check(rstd, "rstd", shape[:-1], torch.float32, dev)
    if weight is not None:
        _check(weight, "weight", (C,), torch.float32, dev)
    if dsum is not None:
        _check(dsum, "dsum", shape, dt, dev)
    dx = _out(dx, "dx", shape, dt, dev, dout)
    dw = ws = None
    nbytes = 0
    if wgrad:
        dw = torch.empty(C, dtype=torch.float32, device=dev)
        nbytes = _size("bimamba_rms_norm_bwd_workspace_size", rows, C, code)
        ws = _workspace(nbytes, dev)
    rc = lib().bimamba_rms_norm_bwd(
        rows, C, code, xp, xs, rstd.data_ptr(), _adr(weight), dout.data_ptr(), _adr(dsum), dx.data_ptr(), _adr(dw),
        _adr(ws), nbytes, _raw_stream(dev.index))
    if rc:
        _abi.check(rc)
    return dx, dw


def linear8(x, weight, bias=None, dtype=torch.bfloat16, out=None, stream=None):
    """Product of 8-bit rows (bimamba_linear8): x Rows8 [..., cin], weight
    Rows8 [cout, cin], bias float32 [cout] or None. Returns [..., cout] in
    dtype (bf16 or fp32; out's, if out is given), which may not overlap an
    input."""
    dev = _cuda_device(_rows8(x, "x"))
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, linear8, x, weight, bias, dtype, out)
    if out is not None:
        dtype = out.dtype
    code, shape = _dtype_code(dtype), tuple(x.shape)
    rows, cin = _rows(shape)
    if len(_rows8(weight, "weight").shape) != 2:
        raise ValueError(f"weight has shape {tuple(weight.shape)}, expected [cout, cin]")
    cout = _int32(weight.shape[0], "cout")
    xp = x._ptrs("x", shape, dev)
    wp = weight._ptrs("weight", (cout, cin), dev)
    if bias is not None:
        _check(bias, "bias", (cout,), torch.float32, dev)
    out = _out(out, "out", shape[:-1] + (cout,), dtype, dev)
    rc = lib().bimamba_linear8(rows, cin, cout, code, ctypes.byref(xp), ctypes.byref(wp), _adr(bias), out.data_ptr(),
                               _raw_stream(dev.index))
    if rc:
        _abi.check(rc)
    return out


DELTA = ("q", "k", "v", "g", "beta")


def _delta_dims(d):
    q, v = d["q"], d["v"]
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("v must be [batch, L, H, P] and q [batch, L, G, N]")
    return tuple(v.shape) + tuple(q.shape[2:])


def _delta_dir(d, dims, dtype, dev, name):
    batch, L, H, P, G, N = dims
    for k, shape, dt in (("q", (batch, L, G, N), dtype), ("k", (batch, L, G, N), dtype),
                         ("v", (batch, L, H, P), dtype), ("g", (batch, L, H), torch.float32),
                         ("beta", (batch, L, H), torch.float32)):
        _check(d[k], f"{name}.{k}", shape, dt, dev)
    return ctypes.byref(_abi.DeltaDir(*(d[k].data_ptr() for k in DELTA)))


@functools.lru_cache(maxsize=4096)
def _delta_size(query, dims, dtype, *rest):
    """(the workspace, the bimamba_shape to pass, which the library only reads)."""
    batch, L, H, P, G, N = dims
    n = ctypes.c_size_t(0)
    shape = ctypes.byref(_sizes(_abi.Shape, "the problem's shape", batch, L, H, P, N, G, 64, _dtype_code(dtype), 0))
    _abi.check(getattr(lib(), query)(shape, *rest, ctypes.byref(n)))
    return n.value, shape


def _delta_scale(scale, N):
    return N ** -0.5 if scale is None else float(scale)


def _delta_workspace(workspace, nbytes, dev):
    if workspace is None:
        return _workspace(nbytes, dev), nbytes
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return workspace, workspace.numel() * workspace.element_size()


def delta_workspace_size(fwd, has_bwd=True, nseq=0):
    """Bytes of workspace of delta_fwd and delta_step for such a direction, or
    for two."""
    return _delta_size("bimamba_delta_workspace_size", _delta_dims(fwd), fwd["v"].dtype, int(bool(has_bwd)),
                       _int32(nseq, "nseq"))[0]


def delta_bwd_workspace_size(fwd, nseq=0):
    """Bytes of workspace of delta_bwd for such a direction."""
    return _delta_size("bimamba_delta_bwd_workspace_size", _delta_dims(fwd), fwd["v"].dtype, _int32(nseq, "nseq"))[0]


def delta_fwd(fwd, bwd=None, scale=None, cu_seqlens=None, init_state=None, final_state=None, y=None,
              workspace=None, stream=None):
    """The gated delta rule over whole sequences (bimamba_delta_fwd).

    fwd/bwd: dicts of device tensors q, k [b,L,G,N], v [b,L,H,P] (bf16 or
    fp32), g (the decay's logarithm) and beta [b,L,H] float32; bwd, in forward
    time order, runs over the reversed sequence, and both outputs are summed.
    scale: of the output, N^-1/2 unless given. cu_seqlens: host list/tensor of
    nseq+1 offsets. init_state, final_state: float32 [sequences,H,P,N] of the
    forward direction (final_state is written and may be init_state). Returns
    y (float32 [b,L,H,P])."""
    dev = _cuda_device(fwd["v"])
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, delta_fwd, fwd, bwd, scale, cu_seqlens, init_state, final_state, y, workspace)
    dims, dtype = _delta_dims(fwd), fwd["v"].dtype
    batch, L, H, P, G, N = dims
    cu_arr, nseq = _offsets(cu_seqlens)
    nbytes, shape = _delta_size("bimamba_delta_workspace_size", dims, dtype, int(bwd is not None), max(nseq, 0))
    fd = _delta_dir(fwd, dims, dtype, dev, "fwd")
    bd = _delta_dir(bwd, dims, dtype, dev, "bwd") if bwd is not None else None
    units = nseq if cu_seqlens is not None else batch
    for t, name in ((init_state, "init_state"), (final_state, "final_state")):
        if t is not None:
            _check(t, name, (units, H, P, N), torch.float32, dev)
    y = _out(y, "y", (batch, L, H, P), torch.float32, dev)
    ws, nbytes = _delta_workspace(workspace, nbytes, dev)
    rc = lib().bimamba_delta_fwd(shape, fd, bd, _delta_scale(scale, N), cu_arr, nseq, _adr(init_state),
                                 _adr(final_state), y.data_ptr(), _adr(ws), nbytes, _raw_stream(dev.index))
    if rc:
        _abi.check(rc)
    return y


def delta_step(state, fwd, bwd=None, commit=True, scale=None, y=None, workspace=None, stream=None):
    """One cached step of the gated delta rule (bimamba_delta_step): a block
    of 1..256 tokens (one, when decoding) for each row of fwd, which continues
    the state of its number. state: a State of the shape (slots, H, P, N), or a
    float32 tensor [slots,H,P,N]; with commit the rows' last states replace
    theirs. bwd sees the block alone. Returns y (float32 [b,L,H,P])."""
    dev = _cuda_device(fwd["v"])
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, delta_step, state, fwd, bwd, commit, scale, y, workspace)
    dims, dtype = _delta_dims(fwd), fwd["v"].dtype
    batch, L, H, P, G, N = dims
    nbytes, shape = _delta_size("bimamba_delta_workspace_size", dims, dtype, int(bwd is not None), 0)
    fd = _delta_dir(fwd, dims, dtype, dev, "fwd")
    bd = _delta_dir(bwd, dims, dtype, dev, "bwd") if bwd is not None else None
    slots = state.shape[0]
    if isinstance(state, State):
        if tuple(state.shape) != (slots, H, P, N):
            raise ValueError(f"state has shape {tuple(state.shape)}, expected (slots, {H}, {P}, {N})")
        if state.device != dev:
            raise ValueError(f"state is on {state.device}, expected {dev}")
        at = state.data_ptr()
    else:
        _check(state, "state", (slots, H, P, N), torch.float32, dev)
        at = state.data_ptr()
    if batch > slots:
        raise ValueError(f"batch {batch} exceeds the state's {slots} slots")
    y = _out(y, "y", (batch, L, H, P), torch.float32, dev)
    ws, nbytes = _delta_workspace(workspace, nbytes, dev)
    rc = lib().bimamba_delta_step(shape, at, fd, bd, _delta_scale(scale, N), int(bool(commit)), y.data_ptr(),
                                  _adr(ws), nbytes, _raw_stream(dev.index))
    if rc:
        _abi.check(rc)
    return y


def _delta_grads(g, dims, dev, name):
    batch, L, H, P, G, N = dims
    shapes = dict(q=(batch, L, G, N), k=(batch, L, G, N), v=(batch, L, H, P), g=(batch, L, H), beta=(batch, L, H))
    g = {k: _out(None if g is None else g[k], f"{name}_grad.{k}", v, torch.float32, dev) for k, v in shapes.items()}
    return g, ctypes.byref(_abi.DeltaGrad(*(g[k].data_ptr() for k in DELTA)))


def delta_bwd(fwd, bwd, dy, scale=None, cu_seqlens=None, init_state=None, dfinal=None, dinit=None, grads=None,
              workspace=None, stream=None):
    """Gradient of delta_fwd (bimamba_delta_bwd) for dy (float32 [b,L,H,P],
    which both streams get) and dfinal (float32 like final_state, or None).
    init_state: the forward's. dinit: where to write init_state's gradient, or
    None. Returns (gfwd, gbwd), dicts of float32 tensors keyed q, k, v, g, beta
    (gbwd None without bwd); grads: optional such dicts to write into."""
    dev = _cuda_device(fwd["v"])
    if _elsewhere(dev, stream):
        return _run_on(dev, stream, delta_bwd, fwd, bwd, dy, scale, cu_seqlens, init_state, dfinal, dinit, grads,
                       workspace)
    dims, dtype = _delta_dims(fwd), fwd["v"].dtype
    batch, L, H, P, G, N = dims
    cu_arr, nseq = _offsets(cu_seqlens)
    nbytes, shape = _delta_size("bimamba_delta_bwd_workspace_size", dims, dtype, max(nseq, 0))
    fd = _delta_dir(fwd, dims, dtype, dev, "fwd")
    bd = _delta_dir(bwd, dims, dtype, dev, "bwd") if bwd is not None else None
    _check(dy, "dy", (batch, L, H, P), torch.float32, dev)
    units = nseq if cu_seqlens is not None else batch
    for t, name in ((init_state, "init_state"), (dfinal, "dfinal"), (dinit, "dinit")):
        if t is not None:
            _check(t, name, (units, H, P, N), torch.float32, dev)
    gl = tuple(grads) if grads is not None else (None, None)
    gf, gfp = _delta_grads(gl[0], dims, dev, "fwd")
    gb, gbp = _delta_grads(gl[1], dims, dev, "bwd") if bwd is not None else (None, None)
    ws, nbytes = _delta_workspace(workspace, nbytes, dev)
    rc = lib().bimamba_delta_bwd(shape, fd, bd, _delta_scale(scale, N), cu_arr, nseq, _adr(init_state), _adr(dfinal),
                                 dy.data_ptr(), gfp, gbp, _adr(dinit), _adr(ws), nbytes, _raw_stream(dev.index))
    if rc:
        _abi.check(rc)
    return gf, gb

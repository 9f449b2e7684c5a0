"""Training steps called from several threads at once, each on a stream of its
own: the binding's remembered sizes and the library's state serve all of them."""
import threading

import pytest
import torch

import bidirectional_mamba_ssm_amd as bm

pytestmark = pytest.mark.gpu

DEV = "cuda"
THREADS, TURNS = 4, 12


def _inputs(i):
    """Other sizes in every thread."""
    g = torch.Generator(device=DEV).manual_seed(100 + i)
    rows, C, H, P, N = 200 + 37 * i, 256 * (1 + i), 2 + i, 16, 16
    ch = H * P + 2 * N

    def r(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV).to(dtype)
    conv = [dict(xbc=bm.act8_pack(r(1, rows, ch)), weight=r(ch, 4), bias=r(ch)) for _ in range(2)]
    grads = [dict(x=r(1, rows, H, P), B=r(1, rows, 1, N), C=r(1, rows, 1, N)) for _ in range(2)]
    cu = [0, 50, 51 + i, 180, rows] if i % 2 else None
    return r(rows, C, dtype=torch.bfloat16), r(rows, C, dtype=torch.bfloat16), r(rows, C), r(C), conv, grads, cu, (H, P, 1, N)


def _step(x, res, y, w, conv, grads, cu, dims):
    o = bm.layer_norm(x, w, residual=res, checkpoint=True)
    out = list(bm.layer_norm_bwd(x, o["ckpt"], o["mean"], o["rstd"], w, dsum=res)) + [o["out"], o["ckpt"].q]
    out += list(bm.gated_norm_bwd(x, bm.act8_pack(y), res, w, group_size=256))
    for d in bm.conv1d(conv[0], conv[1], *dims, cu_seqlens=cu) + \
            bm.conv1d_bwd(conv[0], conv[1], grads[0], grads[1], *dims, cu_seqlens=cu):
        out += list(d.values())
    return out


def test_threads():
    ins = [_inputs(i) for i in range(THREADS)]
    want = [_step(*a) for a in ins]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(THREADS, timeout=60)

    def work(i):
        try:
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                start.wait()
                for turn in range(TURNS):
                    got = _step(*ins[i])
                    # refused calls between them: one by the binding, and one by the
                    # library, whose message is this thread's own
                    try:
                        bm.layer_norm_bwd(ins[i][0], ins[i][0], want[i][0], want[i][0])
                        bad.append((i, "not refused"))
                    except TypeError:
                        pass
                    try:
                        bm.layer_norm(torch.zeros(2, 4 + i, device=DEV))
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

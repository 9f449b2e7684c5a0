"""8-bit checkpoints of blocks of small magnitudes, bit for bit the oracle's."""
import numpy as np
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
from oracle import train as otrain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_small_blocks(dtype):
    r = np.random.default_rng(9)
    e = np.repeat(np.arange(-149, -110), 4)[:, None]
    x = torch.tensor(r.uniform(-1, 1, (len(e), 70)) * 2.0 ** (e + 1)).float().to(dtype)
    x[0] = 0
    x[1, :2] = torch.tensor([2.0 ** -140, 2.0 ** -135]).to(dtype)
    q, E = otrain.act8(x)
    assert (E == 0).any() and (E == 1).any() and (E > 5).any()
    a = bm.act8_pack(x.cuda())
    assert np.array_equal(a.q.cpu().numpy(), q) and np.array_equal(a.scale.cpu().numpy(), E)
    for d in (torch.bfloat16, torch.float32):
        got = bm.act8_unpack(a, dtype=d).double().cpu().numpy()
        assert np.array_equal(got, otrain.act8_values(q, E)), d
    # the same code where the norm keeps its input
    ck = bm.layer_norm(x.cuda(), checkpoint=True)["ckpt"]
    assert torch.equal(ck.q, a.q) and torch.equal(ck.scale, a.scale)

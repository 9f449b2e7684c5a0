"""8-bit checkpoints of blocks of small magnitudes: the stated error bound,
max(2^-7 of the block's largest magnitude, 2^-134), on the oracle's code."""
import numpy as np

from oracle import train as otrain


def _back(x):
    q, E = otrain.act8(x)
    return q, E, otrain.act8_values(q, E)


def test_subnormal_blocks_by_hand():
    # the unit is 2^-133 for every block without a normal number
    q, E, v = _back(np.array([[2.0 ** -140, 2.0 ** -135] + [0.0] * 30]))
    assert E[0, 0] == 0 and not q.any() and not v.any()
    q, E, v = _back(np.array([[1.9 * 2.0 ** -130]]))
    assert E[0, 0] == 0 and q[0, 0] == 15 and v[0, 0] == 15 * 2.0 ** -133
    # half a unit goes to even, the largest subnormals to the clamp
    q, E, v = _back(np.array([[2.0 ** -134, 3 * 2.0 ** -134, 2.0 ** -126 - 2.0 ** -149]]))
    assert E[0, 0] == 0 and q[0].tolist() == [0, 2, 127]
    # the smallest normal number has the same unit and E = 1 twice that
    q, E, v = _back(np.array([[2.0 ** -126]]))
    assert E[0, 0] == 1 and q[0, 0] == 64 and v[0, 0] == 2.0 ** -126


def test_bound_at_every_magnitude():
    r = np.random.default_rng(8)
    worst = 0.0
    for e in list(range(-149, -110)) + [0, 100]:
        x = (r.uniform(-1, 1, (50, 32)) * 2.0 ** (e + 1)).astype(np.float32).astype(np.float64)
        top = np.abs(x).max(axis=1, keepdims=True)
        err = np.abs(_back(x)[2] - x)
        assert np.all(err <= np.maximum(top * 2.0 ** -7, 2.0 ** -134)), e
        if e <= -130:
            worst = max(worst, float((err / np.maximum(top, 2.0 ** -149)).max()))
    assert worst == 1.0   # there is no bound relative to a small block's magnitude

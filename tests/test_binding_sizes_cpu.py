"""Numbers beyond 32 bits: the library takes C ints, and ctypes would pass on
the low 32 bits of a larger number. CPU only."""
import pytest
import torch

import bidirectional_mamba_ssm_amd as bm

FAR = 2 ** 32


@pytest.mark.parametrize("cu", [[0, FAR + 40, 2500], [0, 40, FAR + 2500], [FAR, 40, 2500], [0, 2 ** 31, 2500],
                                [0, -2 ** 31 - 1, 2500]])
@pytest.mark.parametrize("kind", [list, tuple, torch.tensor])
def test_offsets_beyond_32_bits(cu, kind):
    with pytest.raises(ValueError, match="cu_seqlens.*32 bits"):
        bm._offsets(kind(cu))


def test_offsets_within_32_bits():
    arr, n = bm._offsets([0, 5, 5, 2 ** 31 - 1])
    assert list(arr) == [0, 5, 5, 2 ** 31 - 1] and n == 3
    arr, n = bm._offsets(torch.tensor([0, 7], dtype=torch.int32))
    assert list(arr) == [0, 7] and n == 1
    # what is wrong in itself is the library's to say
    assert list(bm._offsets([0, -1, 4])[0]) == [0, -1, 4]
    assert bm._offsets([])[1] == -1
    assert bm._offsets(None) == (None, 0)


def test_seq_index_beyond_32_bits():
    with pytest.raises(ValueError, match="32 bits"):
        bm.seq_index([0, FAR + 4], device="cpu")


def test_int32():
    for v in (-2 ** 31, -1, 0, 256, 2 ** 31 - 1):
        assert bm._int32(v, "n") == v
    for v in (-2 ** 31 - 1, 2 ** 31, FAR + 256, 10 ** 30):
        with pytest.raises(ValueError, match="group_size.*32 bits"):
            bm._int32(v, "group_size")


def test_shapes_beyond_32_bits():
    x, B = torch.zeros(1, 4, 2, 16), torch.zeros(1, 4, 1, 16)
    assert bm.make_shape(x, B, 64).chunk == 64
    for kw in (dict(chunk=FAR + 64), dict(chunk=64, seqlen=FAR + 4)):
        with pytest.raises(ValueError, match="32 bits"):
            bm.make_shape(x, B, **kw)
    # a row of more tokens than fit (no memory behind it)
    far = torch.empty(1, device="meta").expand(1, FAR + 8, 1, 1)
    with pytest.raises(ValueError, match="32 bits"):
        bm.make_shape(far, far, 64)
    ok = (1, 8, 2, 16, 16, 1, 4, 0, 1, 0)
    assert bm._conv_shape(*ok).nheads == 2
    for i in range(7):
        with pytest.raises(ValueError, match="32 bits"):
            bm._conv_shape(*[v + (FAR if j == i else 0) for j, v in enumerate(ok)])


def test_state_beyond_32_bits():
    """A cache of one slot whose view would have 2^32 + 1."""
    for dims in ((FAR + 1, 2, 16, 16), (1, FAR + 2, 16, 16), (1, 2, FAR + 16, 16), (1, 2, 16, FAR + 16)):
        with pytest.raises(ValueError, match="32 bits"):
            bm.State(*dims)
    for conv in ((FAR + 1, 4, torch.float32), (1, FAR + 4, torch.float32)):
        with pytest.raises(ValueError, match="32 bits"):
            bm.State(1, 2, 16, 16, conv=conv)

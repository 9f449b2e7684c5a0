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

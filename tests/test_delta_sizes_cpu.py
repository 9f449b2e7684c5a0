"""The delta rule's workspace queries of the binding, on the CPU."""
import os

import pytest
import torch

import bidirectional_mamba_ssm_amd as bm
from bidirectional_mamba_ssm_amd import _abi
from delta_inputs import direction


@pytest.fixture(autouse=True, scope="module")
def lib():
    if not os.path.exists(_abi.LIB_PATH):
        from bidirectional_mamba_ssm_amd import build
        build.build()


def _one():
    return direction(torch.Generator().manual_seed(0), 1, 200, 2, 16, 1, 16, "bf16")


@pytest.mark.parametrize("query", [bm.delta_workspace_size, bm.delta_bwd_workspace_size])
@pytest.mark.parametrize("nseq", [2 ** 32, 2 ** 32 + 3, 2 ** 31, -2 ** 32 + 1])
def test_more_sequences_than_32_bits(query, nseq):
    """ctypes would pass on the low 32 bits: 2^32 + 3 sequences had the size of 3."""
    with pytest.raises(ValueError, match="32 bits"):
        query(_one(), nseq=nseq)


@pytest.mark.parametrize("query", [bm.delta_workspace_size, bm.delta_bwd_workspace_size])
def test_sizes(query):
    assert query(_one(), nseq=3) >= query(_one()) > 0
    with pytest.raises(bm.BimambaError, match="nseq"):
        query(_one(), nseq=-1)

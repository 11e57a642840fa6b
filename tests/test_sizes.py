"""Sizes beyond the library's 32 bits are refused by the scan's and the convolution's binding, not
taken modulo 2^32 (CPU: shapes without memory)."""
import pytest
import torch

import selective_state_space_26_amd as msel

BIG = (1 << 32) + 64


@pytest.mark.parametrize("shape", [(1, 1, BIG), (1, BIG, 1), (BIG, 1, 1)])
def test_workspace_of_a_shape_beyond_32_bits(shape):
    u = torch.empty(shape, device="meta")
    with pytest.raises(ValueError, match="32 bits"):
        msel.bwd_workspace_bytes(u, torch.empty(shape[1], 16, device="meta"))
    with pytest.raises(ValueError, match="32 bits"):
        msel.bwd_fused(u, torch.empty(shape[1], 16, device="meta"))


def test_state_beyond_32_bits():
    with pytest.raises(ValueError, match="32 bits"):
        msel.bwd_workspace_bytes(torch.empty(1, 1, 8, device="meta"),
                                 torch.empty(1, BIG, device="meta"))


def test_chunks_of_a_length_beyond_32_bits():
    for L in (BIG, 1 << 31, -BIG + 128):
        with pytest.raises(ValueError, match="32 bits"):
            msel.num_chunks(L)
    assert msel.num_chunks(msel.chunk_len()) == 1

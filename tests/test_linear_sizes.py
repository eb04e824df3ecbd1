"""Sizes and activation codes past 32 bits: the C structures hold them in 32, and
ctypes would drop the upper bits without a word.  (No GPU: meta tensors.)"""
import pytest
import torch

from dynamic_block_sparse_stats_b200 import _lib, api

WIDE = (1 << 32) + 64


def _m(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def _wide8(n=1):
    return api.alloc_ckpt8(n, WIDE, "meta")


@pytest.mark.parametrize("call", [
    lambda: api.ckpt8_pack(_m(1, WIDE)),
    lambda: api.ckpt8_unpack(_wide8()),
    lambda: api.linear_fwd(_m(1, WIDE), _m(64, WIDE)),
    lambda: api.linear_fwd(_m(1, 64), _m(WIDE, 64)),
    lambda: api.linear_fwd(_m(1, 64), _m(64, 64), act=(1 << 32) + 3),
    lambda: api.linear_bwd(_m(1, WIDE), _m(1, 64), _m(WIDE, 64)),
    lambda: api.linear_bwd(_m(1, 64), _m(1, WIDE), _m(64, WIDE)),
    lambda: api.linear_bwd(_m(1, 64), _wide8(), None, need=("dW",)),
    lambda: api.linear_bwd(_m(1, 64), _m(1, 64), _m(64, 64), _m(1, 64), act=(1 << 32) + 3),
    lambda: api.linear_workspace_size(1, WIDE, 64),
    lambda: api.linear_workspace_size(1, 64, WIDE),
    lambda: api.linear_workspace_size(1, 64, 64, (1 << 32) + 1, True),
    lambda: api.linear_workspace_size(1 << 64, 64, 64),
])
def test_past_32_bits(call):
    with pytest.raises((ValueError, _lib.PrismError), match="channels|act|tokens"):
        call()

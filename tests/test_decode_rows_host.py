"""Rows of another length than the call's would be read as other rows: the binding refuses them (stand-ins for CUDA
tensors, no GPU)."""
import pytest
import torch

import latent_moe_layer_fp32_gb300 as lm
from test_decode_devices_host import Called, calls, ints, lib, on  # noqa: F401


def bf16(*shape):
    return on(torch.zeros(*shape, dtype=torch.bfloat16))


def f32(*shape):
    return on(torch.zeros(*shape))


def test_decode_attention(lib):  # noqa: F811
    call, args = calls()["decode"]  # 3 requests, 4 heads of 64, 4 blocks
    for bad in (dict(block_table=ints(3, 5)), dict(block_table=ints(4, 3)), dict(block_table=ints(2, 3, 5)),
                dict(out=bf16(3, 5, 64)), dict(out=bf16(8, 3, 64)), dict(out=bf16(9, 96)), dict(lse=f32(3, 6)),
                dict(lse=f32(5, 3))):
        with pytest.raises(ValueError, match="rows of"):
            call(**(args | bad))
    # more rows, flat ones, pieces of rows, and rows that are two dimensions together
    for good in (dict(block_table=ints(9, 4)), dict(block_table=ints(12)), dict(block_table=ints(20)),
                 dict(block_table=ints(3, 2, 2)), dict(block_table=ints(1, 3, 4)), dict(out=bf16(3, 256)),
                 dict(out=bf16(7, 4, 64)), dict(out=bf16(768)), dict(out=bf16(12, 64)), dict(out=bf16(3, 4, 2, 32)),
                 dict(lse=f32(5, 4)), dict(lse=f32(12)), dict(lse=f32(12, 1)), dict(lse=None)):
        with pytest.raises(Called):
            call(**(args | good))
    # one request has no second row
    one = dict(dims=lm.decode_dims_of(1, 4, 4, 0.125), block_table=ints(1, 9))
    with pytest.raises(Called):
        call(**(args | one))


def test_positions(lib):  # noqa: F811
    call, args = calls()["rope"]  # 3 tokens
    two = dict(dims=lm.rope_dims_of(3, 4, 2, 64, n_axes=2))
    for bad in (ints(2, 4), ints(2, 2, 2), ints(3, 2)):
        with pytest.raises(ValueError, match="rows of"):
            call(**(args | two | dict(pos=bad)))
    for good in (ints(2, 3), ints(4, 3), ints(6)):
        with pytest.raises(Called):
            call(**(args | two | dict(pos=good)))
    with pytest.raises(Called):  # one axis: the first three of a longer buffer
        call(**(args | dict(pos=ints(1, 8))))


def test_widths_that_there_are_not(lib):  # noqa: F811
    call, args = calls()["decode"]
    for bad in (dict(max_blocks=0), dict(max_blocks=-1), dict(q_heads=0)):
        a = dict(n_requests=3, q_heads=4, max_blocks=4, scale=0.125) | bad
        more = dict(q=on(torch.zeros(3, 0, 64, dtype=torch.bfloat16))) if "q_heads" in bad else {}
        with pytest.raises(Called):  # the library's answer is its own error
            call(**(args | dict(dims=lm.decode_dims_of(**a)) | more))

"""Options of the serving operators' binding that are refused before any tensor is looked at."""
import numpy as np
import pytest
import torch

import decode_attention_int8_b200 as q8


def rope(pair_axis):
    z = torch.zeros
    pool, scale = z(4, 16, 1, 64, dtype=torch.int8), z(4, 16, 1)
    return q8.q8kv_rope_cache_write(z(2, 1, 64), pool, pool, scale, scale, z(2, 1, 64), z(2, 1, 64),
                                    z(2, 1, 64), z(2, dtype=torch.int64),
                                    z(1, 2, dtype=torch.int32), z(4, 8), pair_axis=pair_axis)


@pytest.mark.parametrize("count", [4, True, np.int64(4), np.uint8(4), torch.tensor(4)])
def test_a_count_is_no_table_of_axes(count):
    """bytes(n) of anything that counts as an integer is n zeros, which would pass as "every pair on
    axis 0"."""
    with pytest.raises(TypeError, match="pair_axis"):
        rope(count)


@pytest.mark.parametrize("axes", [[0, 0, 0, 0], (0, 0, 0, 0), bytes(4), bytearray(4),
                                  np.zeros(4, np.uint8), np.zeros(4, np.int64),
                                  torch.zeros(4, dtype=torch.int32)])
def test_sequences_of_axes_pass(axes):
    with pytest.raises(ValueError, match="CUDA"):  # (then the CPU tensors are refused)
        rope(axes)


@pytest.mark.gpu
def test_arrays_of_axes_on_a_device():
    """Arrays of any integer type give what a list of the same axes gives; one of another length,
    a single entry that could pass for a count among them, is refused."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((6, 2, 64), generator=g, device="cuda")
    pos = torch.randint(0, 9, (3, 6), generator=g, device="cuda", dtype=torch.int32)
    angles = torch.randn((9, 8), generator=g, device="cuda")
    slots = torch.arange(6, device="cuda")

    def call(axes):
        pools = [torch.zeros((1, 16, 2, 64), dtype=torch.int8, device="cuda") for _ in range(2)]
        scales = [torch.zeros((1, 16, 2), device="cuda") for _ in range(2)]
        out = torch.empty_like(x)
        q8.q8kv_rope_cache_write(out, *pools, *scales, x, x, x, slots, pos, angles, pair_axis=axes)
        return [out, *pools, *scales]

    want = call([2, 0, 1, 2])
    for axes in (np.array([2, 0, 1, 2]), np.array([2, 0, 1, 2], np.uint16), iter([2, 0, 1, 2]),
                 torch.tensor([2, 0, 1, 2]), (2, 0, 1, 2), bytes([2, 0, 1, 2])):
        for a, b in zip(call(axes), want):
            assert torch.equal(a, b)
    for axes in (torch.tensor([4]), np.array([4]), [0, 0, 0], np.zeros(1, np.uint32)):
        with pytest.raises(ValueError, match="pair_axis"):
            call(axes)
    with pytest.raises(TypeError, match="pair_axis"):
        call(np.zeros(4))

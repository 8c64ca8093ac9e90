"""How the library plans the layer operators' calls, seen through its size queries (no GPU)."""
import ctypes

import pytest
import torch

from chunked_gated_delta_09_amd import layers


def norm_bwd_bytes(R, G, C, shared=0, dtype=torch.bfloat16):
    d = layers._NormDims(R, G, C, 0, 0, shared, 1e-5, 0, 0, layers._DT[dtype])
    return layers._lib().kda_group_norm_bwd_workspace_bytes(ctypes.byref(d))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 3, 31, 32, 255, 1023, 4097, 65535])
@pytest.mark.parametrize("C", [1, 8, 16, 100, 1000])
@pytest.mark.parametrize("R", [1, 7, 1000, 100000])
def test_norm_backward_workspace(R, G, C, dtype):
    """Sums of one weight a channel: no more rows of them than rows of x, and not more bytes than x and a
    call's fixed share (1024 workgroups of at most 4096 channels, two sums, 4 bytes)."""
    if G * C > 1 << 20:
        pytest.skip("more channels than a call takes")
    got = norm_bwd_bytes(R, G, C, dtype=dtype)
    if R * G > 2 ** 31 - 65:
        assert got == 0  # refused: too many groups
        return
    row = 2 * G * C * 4
    assert 0 < got <= R * row + 256
    assert got <= row + 1024 * 4096 * 2 * 4 + 256

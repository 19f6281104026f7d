"""Refusals of the transformer-block helpers that need tensors on the GPU."""
import pytest
import torch

from tensor_compiler_tiling_amd import convtile as ct

from _gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def test_more_weights_than_32_bits_count():
    """2^32 rows of w, as a view that takes no memory."""
    x = torch.zeros(2, 1, device=DEV, dtype=BF16)
    w = torch.zeros(1, 1, device=DEV, dtype=BF16).expand(1 << 32, 1)
    q, s = torch.zeros(2, 1, device=DEV, dtype=E4M3), torch.zeros(2, device=DEV)
    wq = torch.zeros(1, 1, device=DEV, dtype=E4M3).expand(1 << 32, 1)
    with pytest.raises(ValueError, match="32 bits"):
        ct.linear(x, w)
    with pytest.raises(ValueError, match="32 bits"):
        ct.linear_q8(q, s, wq, s)

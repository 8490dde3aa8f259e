"""Ends of the paged cache's documented ranges, checked on the host (CPU only; the pointers are never
dereferenced)."""
import pytest
import torch

from fp8_quantized_gemm_amd import fp8q
from test_paged_abi import ATTEND, SHAPE, status


@pytest.mark.parametrize("scale", [2.0 ** 127 * (1 + 2.0 ** -23), -2.0 ** 127 * (1 + 2.0 ** -23), 2.4e38, 3.4e38])
def test_softmax_scales_that_overflow_in_powers_of_two(scale):
    assert status(fp8q.lib.fp8_paged_attention, ATTEND, {"scale": scale}) == SHAPE


@pytest.mark.skipif(torch.cuda.is_available(), reason="without a GPU the device check ends the call")
@pytest.mark.parametrize("scale", [2.0 ** 127, -2.0 ** 127, 0.0])
def test_largest_softmax_scale(scale):
    assert status(fp8q.lib.fp8_paged_attention, ATTEND, {"scale": scale}) != SHAPE

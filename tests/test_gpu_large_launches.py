"""Calls on sizes whose kernels have 2^32 threads and more, which HIP would cut short without an
error: many rows are quantized whole, products of that many columns or rows are refused."""
import pytest
import torch

from fp8_quantized_gemm_amd import fp8q, synth
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu


def test_quantize_rows_of_many_rows():
    rows, pattern = (1 << 24) + 37, 1 << 12
    base = synth.normal((pattern, 16), 1.0, "bf16", seed=3, device=DEV)
    base[:, 0] *= torch.arange(1, pattern + 1, device=DEV)
    want = fp8q.fp8_quantize_rows(base)
    x = base.repeat(rows // pattern + 1, 1)[:rows].contiguous()
    say("quantize_rows", rows)
    got = fp8q.fp8_quantize_rows(x)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w.repeat(rows // pattern + 1, *[1] * (w.dim() - 1))[:rows])

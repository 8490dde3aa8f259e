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


def _codes(*shape):
    return torch.zeros(shape, dtype=torch.uint8, device=DEV)


def test_products_that_cannot_be_launched_are_refused():
    """Columns (decode) or rows (tiles) for which the kernels would have 2^32 threads; one
    workgroup's fewer are computed."""
    one = torch.ones(1, device=DEV)
    K = 16
    for M, N, fits in ((3, 1 << 27, False), (3, (1 << 27) + 64, False), (3, (1 << 27) - 64, True),
                       ((1 << 30) + 512, 1, False), (1, 1 << 27, True)):
        say("fp8_gemm", M, N)
        qa, qw = _codes(M, K), _codes(N, K)
        y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
        if fits:
            fp8q.fp8_gemm(qa, one, qw, one, y)
            assert not y.any()
        else:
            with pytest.raises(fp8q.Fp8qError, match="invalid configuration"):
                fp8q.fp8_gemm(qa, one, qw, one, y)
        del qa, qw, y
    for M, N in ((3, (1 << 28) + 64), (1, (1 << 27) + 64)):
        say("nested_gemm_fp16", M, N)
        hi = _codes(N, K)
        a = torch.zeros((M, K), dtype=torch.float16, device=DEV)
        with pytest.raises(fp8q.Fp8qError, match="invalid configuration"):
            fp8q.nested_gemm_fp16(a, hi, hi)
        del hi
    say("nested_gemm_fp8")
    with pytest.raises(fp8q.Fp8qError, match="invalid configuration"):
        fp8q.nested_gemm_fp8(_codes(3, K), one, _codes((1 << 26) + 64, K))

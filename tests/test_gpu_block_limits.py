"""Block-scaled calls on more workgroups than one grid dimension holds (a launch takes fewer than
2^32 threads along x): many short rows, many small matrices, long and thin products.

The inputs repeat a pattern, so every part of the outputs has to be the pattern's own result."""
import pytest
import torch

from fp8_quantized_gemm_amd import fp8q, synth
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

PATTERN = 1 << 12                                  # rows


def _repeated(base, rows):
    return base.repeat(rows // PATTERN + 1, *[1] * (base.dim() - 1))[:rows].contiguous()


def _is_repeated(t, want, dim=0):
    """Whether t is `want` again and again along dim, its last part cut."""
    whole = t.shape[dim] // PATTERN
    step = 1 << 12
    for i in range(0, whole, step):
        n = min(step, whole - i)
        part = t.narrow(dim, i * PATTERN, n * PATTERN).unflatten(dim, (n, PATTERN))
        if not torch.equal(part, want.unsqueeze(dim).expand_as(part)):
            return False
    rest = t.shape[dim] - whole * PATTERN
    return torch.equal(t.narrow(dim, whole * PATTERN, rest), want.narrow(dim, 0, rest))


@pytest.mark.parametrize("rows,cols", [((1 << 28) + 37, 16), ((1 << 25) + 5, 272)])
def test_quantize_blocks_of_many_rows(rows, cols):
    base = synth.normal((PATTERN, cols), 1.0, "bf16", seed=3, device=DEV)
    base[:, 0] *= torch.arange(1, PATTERN + 1, device=DEV)          # a scale of its own per row
    want_q, want_s = fp8q.fp8_quantize_blocks(base)
    x = _repeated(base, rows)
    say("quantize_blocks rows", rows, cols)
    q, s = fp8q.fp8_quantize_blocks(x)
    torch.cuda.synchronize()
    assert _is_repeated(q, want_q) and _is_repeated(s, want_s, 1)


def test_quantize_weight_blocks_of_many_matrices():
    count = (1 << 24) + 37
    base = synth.normal((PATTERN, 1, 16), 1.0, "bf16", seed=4, device=DEV)
    base[:, 0, 0] *= torch.arange(1, PATTERN + 1, device=DEV)
    want_q, want_s = fp8q.fp8_quantize_weight_blocks(base)
    w = _repeated(base, count)
    say("quantize_weight_blocks matrices", count)
    q, s = fp8q.fp8_quantize_weight_blocks(w)
    torch.cuda.synchronize()
    assert _is_repeated(q, want_q) and _is_repeated(s, want_s)


@pytest.mark.parametrize("tall", [True, False])
def test_product_of_the_most_rows(tall):
    """2^30 rows of activations by one of weights, and 17 by 2^30."""
    many, few, K = 1 << 30, 1 if tall else 17, 16
    base = synth.normal((PATTERN, K), 1.0, "bf16", seed=5, device=DEV)
    other = synth.normal((few, K), 1.0, "bf16", seed=6, device=DEV)
    if tall:
        qb, sb = fp8q.fp8_quantize_blocks(base)
        qo, so = fp8q.fp8_quantize_weight_blocks(other)
        want = fp8q.fp8_gemm_blockwise(qb, sb, qo, so)
        sa = sb.repeat(1, many // PATTERN)
        say("gemm_blockwise", many, few, K)
        y = fp8q.fp8_gemm_blockwise(_repeated(qb, many), sa, qo, so)
    else:
        qb, sb = fp8q.fp8_quantize_weight_blocks(base)
        qo, so = fp8q.fp8_quantize_blocks(other)
        want = fp8q.fp8_gemm_blockwise(qo, so, qb, sb)
        sw = sb.repeat(many // PATTERN, 1)
        say("gemm_blockwise", few, many, K)
        y = fp8q.fp8_gemm_blockwise(qo, so, _repeated(qb, many), sw)
    torch.cuda.synchronize()
    assert _is_repeated(y, want, 0 if tall else 1)

"""Every tile shape of the block-scaled product over many K steps: the rings of LDS stages go
round several times, the scale pointers advance and each step's last products are folded in the
next.  Small integers with power-of-two scales: all sums are exact, so the outputs are compared
bit for bit."""
import numpy as np
import pytest
import torch

import block_ref as ref
from fp8_quantized_gemm_amd import fp8q
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

CODES = [0x00, 0x38, 0x40, 0x48, 0xB8, 0xC0, 0xC8]             # 0, +-1, +-2, +-4
VALUES = [0.0, 1.0, 2.0, 4.0, -1.0, -2.0, -4.0]

# M, N of each shape, ragged in both (64 x 64 with two workgroups per CU and one)
SIZES = {(257, 4100): "tile 128x64", (333, 6100): "tile 128x128", (64, 16400): "tile 64x64",
         (33, 8200): "tile 64x64", (500, 8200): "tile 128x192", (1100, 6100): "tile 128x256",
         (1000, 8200): "tile 256x192", (1100, 10000): "tile 256x256"}


DEPTHS = [1152, 2704, 5136]                                    # 9, 22 (the last short) and 41 steps


@pytest.mark.parametrize("K", DEPTHS)
@pytest.mark.parametrize("M,N,kernel", [(*size, kernel) for size, kernel in SIZES.items()])
def test_small_integers_over_many_steps(M, N, kernel, K):
    assert fp8q.gemm_blockwise_kernel(M, N, K) == kernel
    gen = torch.Generator(device=DEV).manual_seed(M * 7 + N * 3 + K)
    pick = lambda hi, *shape: torch.randint(0, hi, shape, generator=gen, device=DEV)
    code = torch.tensor(CODES, dtype=torch.uint8, device=DEV)
    value = torch.tensor(VALUES, dtype=torch.float64, device=DEV)
    a, w = pick(7, M, K), pick(7, N, K)
    sa = torch.exp2(pick(2, ref.blocks(K), M).float())
    sw = torch.exp2(pick(3, ref.blocks(N), ref.blocks(K)).float())
    # products up to 16, scales up to 2 * 4: every partial sum is an integer below 5136 * 128 < 2^24
    spread = lambda s, dim, n: s.double().repeat_interleave(ref.B, dim=dim).narrow(dim, 0, n)
    av = value[a] * spread(sa, 0, K).t()
    wv = value[w] * spread(spread(sw, 0, N), 1, K)
    want = (av @ wv.t().contiguous()).float().to(torch.bfloat16)
    say("blockwise tile integers", M, N, K)
    buf = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    fp8q.fp8_gemm_blockwise(code[a], sa, code[w], sw, buf[:M * N].view(M, N))
    torch.cuda.synchronize()
    assert torch.equal(buf[:M * N].view(M, N), want)
    assert torch.all(buf[M * N:] == 7.0)

"""Which kernel the block-scaled product takes for which sizes (a host function: CPU only), and
that the GPU tests reach every one of them."""
import pytest

import test_gpu_block
import test_gpu_block_tiles
from fp8_quantized_gemm_amd import fp8q

STREAMING = ["persistent", "streaming 8x16", "streaming 16x16", "streaming 32x16", "streaming 32x32"]
TILES = ["tile 256x256", "tile 256x192", "tile 128x256", "tile 128x192", "tile 128x128",
         "tile 128x64", "tile 64x64"]


@pytest.mark.parametrize("M,N,K,kernel", [
    (1, 4096, 4096, "persistent"), (16, 1, 12288, "persistent"),
    (8, 4096, 12304, "streaming 8x16"), (9, 4096, 12304, "streaming 16x16"),
    (17, 4096, 4096, "streaming 32x16"), (32, 4096, 16, "streaming 32x16"),
    (32, 4112, 4096, "streaming 32x32"), (33, 4096, 4096, "streaming 32x32"),
    (8192, 16, 144, "streaming 32x16"), (64, 4097, 272, "tile 64x64"),
    (333, 4100, 5008, "tile 128x64"), (512, 12288, 4096, "tile 128x192"),
    (2048, 12288, 4096, "tile 256x192"),
    (0, 1, 16, ""), (1, 1, 24, ""), (1, 2 ** 30 + 1, 16, ""), (2 ** 30 + 1, 1, 16, ""),
])
def test_kernel_of_sizes(M, N, K, kernel):
    assert fp8q.gemm_blockwise_kernel(M, N, K) == kernel


def test_gpu_tests_reach_every_kernel():
    lists = test_gpu_block.SHAPES + test_gpu_block.DECODE + test_gpu_block.FEW
    reached = {fp8q.gemm_blockwise_kernel(*size) for size in lists}
    assert reached >= set(STREAMING)


def test_gpu_tests_run_every_tile_over_many_steps():
    assert set(test_gpu_block_tiles.SIZES.values()) == set(TILES)
    for (M, N), kernel in test_gpu_block_tiles.SIZES.items():
        for K in test_gpu_block_tiles.DEPTHS:
            assert fp8q.gemm_blockwise_kernel(M, N, K) == kernel
    assert max(test_gpu_block_tiles.DEPTHS) >= 20 * 128

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


@pytest.mark.parametrize("heads", [1, 4])
def test_one_token_of_any_row_stride(heads):
    """The rows of one token have no distance: whatever its tensor's stride says is taken."""
    row = torch.zeros(1, 1001, dtype=torch.bfloat16)             # a stride that rows could not have
    t = row.as_strided((1, heads, 64), (1001, 64, 1))
    assert t.stride(0) == 1001
    assert fp8q._rows(t, "q", torch.bfloat16, t.shape, t.get_device()) == (t.data_ptr(), heads * 64)
    two = torch.zeros(2, 1001, dtype=torch.bfloat16).as_strided((2, heads, 64), (1001, 64, 1))
    assert fp8q._rows(two, "q", torch.bfloat16, two.shape, two.get_device()) == (two.data_ptr(), 1001)


@pytest.mark.parametrize("head_dim,whole,cut", [(64, 3200, 3264), (128, 1600, 1664), (192, 1536, 1600), (256, 1152, 1216)])
def test_one_token_is_whole_while_that_is_faster(head_dim, whole, cut):
    """Sequences whole in a workgroup need no scratch; longer ones go through it in parts."""
    for kv_heads in (1, 8):
        size = dict(tokens=1, seqs=1, max_q=1, q_heads=8 * kv_heads, kv_heads=kv_heads, page_size=64, head_dim=head_dim)
        assert fp8q.paged_attention_work_bytes(table_width=whole // 64, **size) == 16
        assert fp8q.paged_attention_work_bytes(table_width=cut // 64, **size) > 1000
    wide = dict(size, seqs=64, tokens=64)                        # 512 workgroups fill the chip without parts
    assert fp8q.paged_attention_work_bytes(table_width=2000, **wide) == 16

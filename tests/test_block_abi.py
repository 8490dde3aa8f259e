"""Refusals of the block-scaled entry points: checked on the host before any HIP call (CPU
only; the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

from fp8_quantized_gemm_amd import fp8q

OK, NULLP, SHAPE, ALIGN, DTYPE, OVERLAP = 0, 1, 2, 3, 4, 7


def at(region, offset=0):
    return ctypes.c_void_p(0x10000000 + region * 0x100000 + offset)


A, B, C, D, E, F = (at(i) for i in range(6))
A4 = at(0, 4)
A2 = at(4, 2)


@pytest.mark.parametrize("fn,args,status", [
    # fp8_quantize_blocks(x, dtype, rows, cols, q, scale)
    ("fp8_quantize_blocks", [None, 0, 1, 16, B, C, None], NULLP),
    ("fp8_quantize_blocks", [A, 0, 1, 16, B, None, None], NULLP),
    ("fp8_quantize_blocks", [A, 2, 1, 16, B, C, None], DTYPE),
    ("fp8_quantize_blocks", [A, 0, 0, 16, B, C, None], SHAPE),
    ("fp8_quantize_blocks", [A, 0, 2 ** 31, 16, B, C, None], SHAPE),
    ("fp8_quantize_blocks", [A, 0, 1, 0, B, C, None], SHAPE),
    ("fp8_quantize_blocks", [A, 0, 1, 24, B, C, None], SHAPE),
    ("fp8_quantize_blocks", [A, 0, 1, 2 ** 22 + 16, B, C, None], SHAPE),
    ("fp8_quantize_blocks", [A4, 0, 1, 16, B, C, None], ALIGN),
    ("fp8_quantize_blocks", [A, 0, 1, 16, B, A2, None], ALIGN),
    ("fp8_quantize_blocks", [A, 0, 4, 128, at(0, 512), C, None], OVERLAP),
    ("fp8_quantize_blocks", [A, 0, 4, 256, B, at(1, 1020), None], OVERLAP),
    # fp8_quantize_weight_blocks(w, dtype, batch, rows, cols, q, scale)
    ("fp8_quantize_weight_blocks", [A, 0, 1, 1, 16, None, C, None], NULLP),
    ("fp8_quantize_weight_blocks", [A, 7, 1, 1, 16, B, C, None], DTYPE),
    ("fp8_quantize_weight_blocks", [A, 0, 0, 1, 16, B, C, None], SHAPE),
    ("fp8_quantize_weight_blocks", [A, 0, 1, 0, 16, B, C, None], SHAPE),
    ("fp8_quantize_weight_blocks", [A, 0, 1, 1, 8, B, C, None], SHAPE),
    ("fp8_quantize_weight_blocks", [A, 0, 2 ** 40, 1, 16, B, C, None], SHAPE),
    ("fp8_quantize_weight_blocks", [A, 0, 2 ** 31, 1, 16, B, C, None], SHAPE),
    ("fp8_quantize_weight_blocks", [A, 0, 2 ** 30, 1, 256, B, C, None], SHAPE),
    ("fp8_quantize_weight_blocks", [A, 0, 1, 1, 16, at(1, 8), C, None], ALIGN),
    ("fp8_quantize_weight_blocks", [A, 0, 2, 130, 128, B, at(1, 2 * 130 * 128 - 4), None], OVERLAP),
    # fp8_gemm_blockwise(qa, sa, qw, sw, y, M, N, K)
    ("fp8_gemm_blockwise", [A, None, C, D, E, 1, 1, 16, None], NULLP),
    ("fp8_gemm_blockwise", [A, B, C, D, E, 0, 1, 16, None], SHAPE),
    ("fp8_gemm_blockwise", [A, B, C, D, E, 1, 1, 40, None], SHAPE),
    ("fp8_gemm_blockwise", [A, B, C, D, E, 1, 2 ** 30 + 1, 16, None], SHAPE),
    ("fp8_gemm_blockwise", [A, B, C, D, E, 2 ** 30 + 1, 1, 16, None], SHAPE),
    ("fp8_linear_blockwise", [A, 0, B, C, D, E, F, 1, 2 ** 30 + 1, 16, None], SHAPE),
    ("fp8_gemm_blockwise", [A, B, C, D, at(4, 8), 1, 1, 16, None], ALIGN),
    ("fp8_gemm_blockwise", [A, A2, C, D, E, 1, 1, 16, None], ALIGN),
    ("fp8_gemm_blockwise", [A, B, C, D, at(0, 256), 2, 16, 256, None], OVERLAP),
    # y in the last of sa's 2 x 3 scales
    ("fp8_gemm_blockwise", [A, at(4, -20 + 16), C, D, E, 3, 1, 256, None], OVERLAP),
    # y over sw's second row block
    ("fp8_gemm_blockwise", [A, B, C, at(4, -4), E, 1, 129, 16, None], OVERLAP),
    # fp8_linear_blockwise(x, dtype, qw, sw, y, q, sa, M, N, K)
    ("fp8_linear_blockwise", [A, 0, B, C, D, E, None, 1, 1, 16, None], NULLP),
    ("fp8_linear_blockwise", [A, 3, B, C, D, E, F, 1, 1, 16, None], DTYPE),
    ("fp8_linear_blockwise", [A, 0, B, C, D, E, F, 1, 1, 24, None], SHAPE),
    ("fp8_linear_blockwise", [A, 0, B, C, D, at(4, 4), F, 1, 1, 16, None], ALIGN),
    ("fp8_linear_blockwise", [A, 0, B, C, D, A, F, 1, 1, 16, None], OVERLAP),
    ("fp8_linear_blockwise", [A, 0, B, C, D, E, at(4, 32), 4, 1, 16, None], OVERLAP),
    ("fp8_linear_blockwise", [A, 0, B, C, B, E, F, 4, 1, 16, None], OVERLAP),
])
def test_refused_before_any_hip_call(fn, args, status):
    assert getattr(fp8q.lib, fn)(*args) == status


G, H, I, J, K = (at(i) for i in range(6, 11))


def moe(**change):
    """fp8_moe_blockwise(x, dtype, logits, w13, s13, w2, s2, y, ids, weights, work, T, H, I, E,
    top_k, renormalize, stream) with one argument changed."""
    args = dict(x=A, dtype=0, logits=B, w13=C, s13=D, w2=E, s2=F, y=G, ids=H, weights=I, work=J,
                T=4, H=128, I=64, E=8, top_k=2, renormalize=1, stream=None)
    assert set(change) <= set(args)
    return list({**args, **change}.values())


@pytest.mark.parametrize("change,status", [
    *[({name: None}, NULLP) for name in ("x", "logits", "w13", "s13", "w2", "s2", "y", "ids",
                                         "weights", "work")],
    ({"dtype": 2}, DTYPE),
    *[({name: v}, SHAPE) for name, v in (("T", 0), ("T", 65), ("H", 0), ("H", 24), ("H", 65552),
                                         ("I", 8), ("I", 72), ("I", 65552), ("E", 0), ("E", 513),
                                         ("top_k", 0), ("top_k", 9), ("E", 1))],
    ({"E": 32, "top_k": 17}, SHAPE),
    *[({name: at(20, 4)}, ALIGN) for name in ("x", "w13", "w2", "y", "work")],
    *[({name: at(20, 2)}, ALIGN) for name in ("logits", "s13", "s2", "ids", "weights")],
    ({"y": B}, OVERLAP),                            # y over the logits
    ({"y": at(4, 8 * 128 * 64 - 16)}, OVERLAP),     # over the last codes of w2
    ({"ids": at(6, 4 * 128 * 2 - 4)}, OVERLAP),     # ids over the end of y
    ({"weights": at(7, 28)}, OVERLAP),              # weights over the last id
    ({"work": at(0, 0)}, OVERLAP),                  # scratch over x
    ({"work": at(2, 8 * 2 * 64 * 128 - 16)}, OVERLAP),
])
def test_moe_refused_before_any_hip_call(change, status):
    assert fp8q.lib.fp8_moe_blockwise(*moe(**change)) == status


def test_moe_work_bytes():
    assert fp8q.moe_work_bytes(1, 16, 1) > 32
    assert fp8q.moe_work_bytes(64, 1024, 16) >= 64 * 1024 * 16 * 2
    for sizes in ((0, 16, 1), (65, 16, 1), (1, 8, 1), (1, 65552, 1), (1, 16, 0), (1, 16, 17)):
        assert fp8q.moe_work_bytes(*sizes) == 0


def test_binding_refuses_wrong_tensors():
    cpu = torch.zeros((2, 128), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fp8q.fp8_quantize_blocks(cpu)
    with pytest.raises(TypeError):
        fp8q.fp8_quantize_blocks(cpu.float())
    with pytest.raises(ValueError):
        fp8q.fp8_quantize_blocks(cpu[0])
    with pytest.raises(ValueError):
        fp8q.fp8_quantize_weight_blocks(cpu[0])
    with pytest.raises(ValueError):
        fp8q.fp8_gemm_blockwise(cpu, cpu, cpu[:, :64], cpu)
    with pytest.raises(TypeError):
        fp8q.fp8_linear_blockwise(cpu, cpu, cpu)
    with pytest.raises(ValueError):
        fp8q.fp8_moe_blockwise(cpu, cpu, cpu, cpu, cpu, cpu, 2)
    w13, w2 = torch.zeros((4, 2, 16, 128)), torch.zeros((4, 128, 16))
    with pytest.raises(ValueError):
        fp8q.fp8_moe_blockwise(cpu, cpu, w13, cpu, w2, cpu, 2, work=torch.zeros(8))

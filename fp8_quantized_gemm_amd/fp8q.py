"""ctypes binding of libfp8q (the C ABI in include/fp8q.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels of libfp8q.so.  torch supplies device memory (output tensors are
allocated with torch when not given) and the stream (torch's current stream
on the tensors' device).  There is no fallback: if the library is missing or
a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("FP8Q_LIB", os.path.join(_HERE, "libfp8q.so"))

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libfp8q.so not found at {LIB_PATH}; build it with "
        "`python -m fp8_quantized_gemm_amd.build` (hipcc, gfx950)")

lib = ctypes.CDLL(LIB_PATH)

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_i = ctypes.c_int
_s = ctypes.c_char_p

# fp8q_kv_cache (k, v, k_scale, v_scale, pages, kv_heads, page_size, head_dim) and fp8q_kv_batch
# (page_table, q_start, kv_lens, tokens, seqs, table_width, max_q) as bytes
_kv_cache_bytes = struct.Struct("=4Q4q").pack
_kv_batch_bytes = struct.Struct("=3Q4q").pack

_SIGS = {
    "fp8q_abi_version": (_i, []),
    "fp8q_status_str": (ctypes.c_char_p, [_i]),
    "fp8q_last_error": (ctypes.c_char_p, []),
    "fp8_quantize_act": (_i, [_p, _i, _i64, _p, _p, _p, _p]),
    "fp8_gemm": (_i, [_p, _p, _p, _p, _p, _i64, _i64, _i64, _p]),
    "fp8_linear": (_i, [_p, _i, _p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _p]),
    "nested_split": (_i, [_p, _p, _p, _i64, _p]),
    "nested_rebuild_fp16": (_i, [_p, _p, _p, _i64, _p]),
    "nested_gemm_fp16": (_i, [_p, _p, _p, _p, _i64, _i64, _i64, _p]),
    "nested_gemm_fp8": (_i, [_p, _p, _p, _p, _i64, _i64, _i64, _p]),
    "nested_linear_fp8": (_i, [_p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _p]),
    "fp8q_e4m3_encode_f32": (_i, [_p, _p, _i64, _p]),
    "fp8_quantize_rows": (_i, [_p, _i, _i64, _i64, _p, _p, _p, _p]),
    "fp8_gemm_rowwise": (_i, [_p, _p, _p, _p, _p, _i64, _i64, _i64, _p]),
    "fp8_linear_rowwise": (_i, [_p, _i, _p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _p]),
    "fp8_quantize_act_delayed": (_i, [_p, _i, _i64, _p, _p, _p, _p, _i64, _p, _p]),
    "fp8_quantize_kv": (_i, [_p, _i, _i64, _i64, _i64, _p, _p, _p, _p]),
    "nested_split_e4m3": (_i, [_p, _p, _p, _i64, _p, _p]),
    "nested_rebuild_e4m3": (_i, [_p, _p, _p, _i64, _p]),
    "nested_gemm_fp16_e4m3": (_i, [_p, _p, _p, _p, _i64, _i64, _i64, _p]),
    "nested_gemm_fp8_e4m3": (_i, [_p, _p, _p, _p, _i64, _i64, _i64, _p]),
    "nested_linear_fp8_e4m3": (_i, [_p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _p]),
    "fp8_linear_delayed": (_i, [_p, _i, _p, _p, _p, _p, _p, _p, _p, _i64, _p, _i64, _i64, _i64,
                                _p]),
    "fp8_quantize_blocks": (_i, [_p, _i, _i64, _i64, _p, _p, _p]),
    "fp8_quantize_weight_blocks": (_i, [_p, _i, _i64, _i64, _i64, _p, _p, _p]),
    "fp8_gemm_blockwise": (_i, [_p, _p, _p, _p, _p, _i64, _i64, _i64, _p]),
    "fp8_gemm_blockwise_kernel": (ctypes.c_char_p, [_i64, _i64, _i64]),
    "fp8_linear_blockwise": (_i, [_p, _i, _p, _p, _p, _p, _p, _i64, _i64, _i64, _p]),
    "fp8_moe_blockwise_work_bytes": (_i64, [_i64, _i64, _i64]),
    "fp8_moe_blockwise": (_i, [_p, _i, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _i64,
                               _i64, _i, _p]),
    "fp8_kv_append": (_i, [_s, _s, _p, _i64, _p, _i64, _i, _p, _i64, _i64, _i, _p, _i64, _p, _i64, _i64, _p]),
    "fp8_paged_attention_work_bytes": (_i64, [_s, _s, _i64]),
    "fp8_paged_attention": (_i, [_s, _s, _p, _i64, _i,
                                 _i64, ctypes.c_float, _i, _i64, _p, _p, _p, _p]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

ABI_VERSION = 3
# words of the delayed-scaling state (FP8Q_DELAYED_STATE_WORDS)
DELAYED_STATE_WORDS = 288
if lib.fp8q_abi_version() != ABI_VERSION:
    raise ImportError(f"libfp8q ABI {lib.fp8q_abi_version()} != binding ABI {ABI_VERSION}")

BF16 = 0
FP16 = 1


class Fp8qError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = lib.fp8q_status_str(status).decode()
        last = lib.fp8q_last_error().decode()
        super().__init__(f"{fn}: {msg} (status {status})" + (f": {last}" if last else ""))


def abi_version() -> int:
    return int(lib.fp8q_abi_version())


def _check(fn: str, status: int):
    if status != 0:
        raise Fp8qError(fn, status)


def _stream(t: torch.Tensor):
    return _p(torch.cuda.current_stream(t.device).cuda_stream)


def _dev(t: torch.Tensor, name: str, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.device.index != torch.cuda.current_device():
        # the library launches on the current device
        raise ValueError(f"{name} is on {t.device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return _p(t.data_ptr())


def _scalar(t: torch.Tensor, name: str):
    if t.numel() != 1:
        raise ValueError(f"{name} must hold exactly one float32")
    return _dev(t, name, torch.float32)


def fp8_quantize_act(x: torch.Tensor, q: torch.Tensor | None = None,
                     scale: torch.Tensor | None = None, amax: torch.Tensor | None = None):
    """E4M3 codes, scale = amax/448 and amax of a bf16/fp16 tensor (any shape).

    Returns (q uint8 like x, scale float32[1], amax float32[1]); all on x's device.
    """
    if x.dtype == torch.bfloat16:
        code = BF16
    elif x.dtype == torch.float16:
        code = FP16
    else:
        raise TypeError(f"x must be bfloat16 or float16, got {x.dtype}")
    if q is None:
        q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = torch.empty(1, dtype=torch.float32, device=x.device)
    if amax is None:
        amax = torch.empty(1, dtype=torch.float32, device=x.device)
    if q.numel() != x.numel():
        raise ValueError("q must have as many elements as x")
    _check("fp8_quantize_act", lib.fp8_quantize_act(
        _dev(x, "x"), code, x.numel(), _dev(q, "q", torch.uint8), _scalar(scale, "scale"),
        _scalar(amax, "amax"), _stream(x)))
    return q, scale, amax


def _mnk(a: torch.Tensor, w: torch.Tensor):
    if a.dim() != 2 or w.dim() != 2 or a.shape[1] != w.shape[1]:
        raise ValueError(f"expected a[M,K] and w[N,K], got {tuple(a.shape)} and {tuple(w.shape)}")
    return a.shape[0], w.shape[0], a.shape[1]


def fp8_gemm(qa: torch.Tensor, sa: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor,
             y: torch.Tensor | None = None) -> torch.Tensor:
    """y[M,N] bf16 = (qa[M,K] . qw[N,K]^T) * sa * sw, E4M3 operands, fp32 accumulation."""
    M, N, K = _mnk(qa, qw)
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=qa.device)
    _check("fp8_gemm", lib.fp8_gemm(
        _dev(qa, "qa", torch.uint8), _scalar(sa, "sa"), _dev(qw, "qw", torch.uint8),
        _scalar(sw, "sw"), _dev(y, "y", torch.bfloat16, (M, N)), M, N, K, _stream(qa)))
    return y


def fp8_linear(x: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor,
               y: torch.Tensor | None = None, q: torch.Tensor | None = None,
               scale: torch.Tensor | None = None, amax: torch.Tensor | None = None):
    """One FP8 linear layer: quantize x[M,K] (bf16/fp16) per tensor, then
    y[M,N] bf16 = (q . qw^T) * scale * sw.  Returns (y, q, scale, amax)."""
    if x.dtype == torch.bfloat16:
        code = BF16
    elif x.dtype == torch.float16:
        code = FP16
    else:
        raise TypeError(f"x must be bfloat16 or float16, got {x.dtype}")
    M, N, K = _mnk(x, qw)
    dev = x.device
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=dev)
    if scale is None:
        scale = torch.empty(1, dtype=torch.float32, device=dev)
    if amax is None:
        amax = torch.empty(1, dtype=torch.float32, device=dev)
    _check("fp8_linear", lib.fp8_linear(
        _dev(x, "x"), code, _dev(qw, "qw", torch.uint8), _scalar(sw, "sw"),
        _dev(y, "y", torch.bfloat16, (M, N)), _dev(q, "q", torch.uint8, (M, K)),
        _scalar(scale, "scale"), _scalar(amax, "amax"), M, N, K, _stream(x)))
    return y, q, scale, amax


def _vector(t: torch.Tensor, name: str, n: int):
    if t.numel() != n:
        raise ValueError(f"{name} must hold {n} float32 values, got {t.numel()}")
    return _dev(t, name, torch.float32)


def _dtype_code(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return BF16
    if x.dtype == torch.float16:
        return FP16
    raise TypeError(f"x must be bfloat16 or float16, got {x.dtype}")


def fp8_quantize_rows(x: torch.Tensor, q: torch.Tensor | None = None,
                      scale: torch.Tensor | None = None, amax: torch.Tensor | None = None):
    """One E4M3 scale per row of x[rows, cols] (bf16/fp16): per-token activation
    or per-channel weight scales.  Returns (q uint8 [rows, cols], scale float32
    [rows], amax float32 [rows])."""
    code = _dtype_code(x)
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D [rows, cols], got {tuple(x.shape)}")
    rows, cols = x.shape
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = torch.empty(rows, dtype=torch.float32, device=x.device)
    if amax is None:
        amax = torch.empty(rows, dtype=torch.float32, device=x.device)
    _check("fp8_quantize_rows", lib.fp8_quantize_rows(
        _dev(x, "x"), code, rows, cols, _dev(q, "q", torch.uint8, (rows, cols)),
        _vector(scale, "scale", rows), _vector(amax, "amax", rows), _stream(x)))
    return q, scale, amax


def fp8_gemm_rowwise(qa: torch.Tensor, sa: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor,
                     y: torch.Tensor | None = None) -> torch.Tensor:
    """y[M,N] bf16 = (qa . qw^T)[m,n] * fl32(sa[m] * sw[n]): per-token activation
    and per-channel weight scales, fp32 accumulation."""
    M, N, K = _mnk(qa, qw)
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=qa.device)
    _check("fp8_gemm_rowwise", lib.fp8_gemm_rowwise(
        _dev(qa, "qa", torch.uint8), _vector(sa, "sa", M), _dev(qw, "qw", torch.uint8),
        _vector(sw, "sw", N), _dev(y, "y", torch.bfloat16, (M, N)), M, N, K, _stream(qa)))
    return y


def fp8_linear_rowwise(x: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor,
                       y: torch.Tensor | None = None, q: torch.Tensor | None = None,
                       sa: torch.Tensor | None = None, amax: torch.Tensor | None = None):
    """fp8_quantize_rows on x[M,K], then fp8_gemm_rowwise with the per-channel
    weight scales sw[N].  Returns (y, q, sa, amax)."""
    code = _dtype_code(x)
    M, N, K = _mnk(x, qw)
    dev = x.device
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=dev)
    if sa is None:
        sa = torch.empty(M, dtype=torch.float32, device=dev)
    if amax is None:
        amax = torch.empty(M, dtype=torch.float32, device=dev)
    _check("fp8_linear_rowwise", lib.fp8_linear_rowwise(
        _dev(x, "x"), code, _dev(qw, "qw", torch.uint8), _vector(sw, "sw", N),
        _dev(y, "y", torch.bfloat16, (M, N)), _dev(q, "q", torch.uint8, (M, K)),
        _vector(sa, "sa", M), _vector(amax, "amax", M), M, N, K, _stream(x)))
    return y, q, sa, amax


def fp8_quantize_kv(x: torch.Tensor, q: torch.Tensor | None = None,
                    scale: torch.Tensor | None = None, amax: torch.Tensor | None = None):
    """FP8 KV cache: E4M3 codes of a K or V block x[T, H, D] (bf16/fp16) with one
    scale per head.  Returns (q uint8 [T, H, D], scale float32 [H], amax float32 [H])."""
    code = _dtype_code(x)
    if x.dim() != 3:
        raise ValueError(f"x must be [tokens, heads, head_dim], got {tuple(x.shape)}")
    T, H, D = x.shape
    if q is None:
        q = torch.empty((T, H, D), dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = torch.empty(H, dtype=torch.float32, device=x.device)
    if amax is None:
        amax = torch.empty(H, dtype=torch.float32, device=x.device)
    _check("fp8_quantize_kv", lib.fp8_quantize_kv(
        _dev(x, "x"), code, T, H, D, _dev(q, "q", torch.uint8, (T, H, D)),
        _vector(scale, "scale", H), _vector(amax, "amax", H), _stream(x)))
    return q, scale, amax


# Values per scale along K, and weight rows per scale, of the block-scaled calls.
BLOCK = 128


def _blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def _ptr(t: torch.Tensor, name: str, dtype, shape, index: int) -> int:
    """_dev without its cost where nothing is wrong (a decode call takes a few
    microseconds); index is the current device's."""
    if (type(t) is torch.Tensor and t.dtype is dtype and t.get_device() == index
            and t.shape == shape and t.is_contiguous()):
        return t.data_ptr()
    return _dev(t, name, dtype, shape).value or 0


def _where(t: torch.Tensor):
    """The current device's index and its current stream."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("the arguments must be CUDA (HIP) tensors")
    index = torch.cuda.current_device()
    # torch.cuda.current_stream(index).cuda_stream without building a Stream object
    return index, torch._C._cuda_getCurrentRawStream(index)


def fp8_quantize_blocks(x: torch.Tensor, q: torch.Tensor | None = None,
                        scale: torch.Tensor | None = None):
    """One E4M3 scale per 1 x 128 block of x[rows, cols] (bf16/fp16), along cols.
    Returns (q uint8 [rows, cols], scale float32 [ceil(cols / 128), rows])."""
    code = _dtype_code(x)
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D [rows, cols], got {tuple(x.shape)}")
    rows, cols = x.shape
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = torch.empty((_blocks(cols), rows), dtype=torch.float32, device=x.device)
    index, stream = _where(x)
    _check("fp8_quantize_blocks", lib.fp8_quantize_blocks(
        _ptr(x, "x", x.dtype, x.shape, index), code, rows, cols,
        _ptr(q, "q", torch.uint8, (rows, cols), index),
        _ptr(scale, "scale", torch.float32, (_blocks(cols), rows), index), stream))
    return q, scale


def fp8_quantize_weight_blocks(w: torch.Tensor, q: torch.Tensor | None = None,
                               scale: torch.Tensor | None = None):
    """One E4M3 scale per 128 x 128 block of each matrix of w[..., N, K] (bf16/fp16;
    leading dimensions count matrices, such as experts).  Returns (q uint8 like w,
    scale float32 [..., ceil(N / 128), ceil(K / 128)])."""
    code = _dtype_code(w)
    if w.dim() < 2:
        raise ValueError(f"w must be [..., N, K], got {tuple(w.shape)}")
    N, K = w.shape[-2:]
    lead = tuple(w.shape[:-2])
    batch = 1
    for d in lead:
        batch *= d
    sshape = lead + (_blocks(N), _blocks(K))
    if q is None:
        q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    if scale is None:
        scale = torch.empty(sshape, dtype=torch.float32, device=w.device)
    index, stream = _where(w)
    _check("fp8_quantize_weight_blocks", lib.fp8_quantize_weight_blocks(
        _ptr(w, "w", w.dtype, w.shape, index), code, batch, N, K,
        _ptr(q, "q", torch.uint8, w.shape, index),
        _ptr(scale, "scale", torch.float32, sshape, index), stream))
    return q, scale


def fp8_gemm_blockwise(qa: torch.Tensor, sa: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor,
                       y: torch.Tensor | None = None) -> torch.Tensor:
    """y[M,N] bf16 = sum over 128-blocks b of sa[b,m] * sw[n/128,b] * (qa . qw^T)_b:
    E4M3 codes with sa float32 [ceil(K/128), M] and sw float32 [ceil(N/128),
    ceil(K/128)], fp32 accumulation."""
    M, N, K = _mnk(qa, qw)
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=qa.device)
    kb = _blocks(K)
    index, stream = _where(qa)
    _check("fp8_gemm_blockwise", lib.fp8_gemm_blockwise(
        _ptr(qa, "qa", torch.uint8, (M, K), index), _ptr(sa, "sa", torch.float32, (kb, M), index),
        _ptr(qw, "qw", torch.uint8, (N, K), index),
        _ptr(sw, "sw", torch.float32, (_blocks(N), kb), index),
        _ptr(y, "y", torch.bfloat16, (M, N), index), M, N, K, stream))
    return y


def gemm_blockwise_kernel(m: int, n: int, k: int) -> str:
    """Name of the kernel that fp8_gemm_blockwise runs for these sizes, "" for sizes it refuses."""
    return lib.fp8_gemm_blockwise_kernel(m, n, k).decode()


def fp8_linear_blockwise(x: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor,
                         y: torch.Tensor | None = None, q: torch.Tensor | None = None,
                         sa: torch.Tensor | None = None):
    """fp8_quantize_blocks on x[M,K], then fp8_gemm_blockwise with the weight's codes
    and block scales.  Returns (y, q, sa)."""
    code = _dtype_code(x)
    M, N, K = _mnk(x, qw)
    kb = _blocks(K)
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if sa is None:
        sa = torch.empty((kb, M), dtype=torch.float32, device=x.device)
    index, stream = _where(x)
    _check("fp8_linear_blockwise", lib.fp8_linear_blockwise(
        _ptr(x, "x", x.dtype, (M, K), index), code, _ptr(qw, "qw", torch.uint8, (N, K), index),
        _ptr(sw, "sw", torch.float32, (_blocks(N), kb), index),
        _ptr(y, "y", torch.bfloat16, (M, N), index), _ptr(q, "q", torch.uint8, (M, K), index),
        _ptr(sa, "sa", torch.float32, (kb, M), index), M, N, K, stream))
    return y, q, sa


def fp8_moe_blockwise(x: torch.Tensor, logits: torch.Tensor, w13: torch.Tensor,
                      s13: torch.Tensor, w2: torch.Tensor, s2: torch.Tensor, top_k: int,
                      renormalize: bool = True, y: torch.Tensor | None = None,
                      ids: torch.Tensor | None = None, weights: torch.Tensor | None = None,
                      work: torch.Tensor | None = None):
    """A mixture-of-experts layer for a few tokens: y[t] = sum over the top_k experts e of
    token t's logits of softmax weight * W2[e] (silu(Wg[e] x[t]) * (Wu[e] x[t])).

    x [T, H] bf16/fp16 (T <= 64), logits float32 [T, E] (-inf: expert off), w13 uint8
    [E, 2, I, H] (gate, up) and w2 uint8 [E, H, I] E4M3 codes with the block scales s13
    and s2 that fp8_quantize_weight_blocks gives.  renormalize: weights over the chosen
    experts instead of over all.  work is scratch (uint8, allocated when not given; its
    size is moe_work_bytes).  Returns (y bf16 [T, H], ids int32 [T, top_k], weights
    float32 [T, top_k])."""
    code = _dtype_code(x)
    if x.dim() != 2 or w13.dim() != 4 or w2.dim() != 3:
        raise ValueError(f"expected x[T,H], w13[E,2,I,H] and w2[E,H,I], got {tuple(x.shape)}, "
                         f"{tuple(w13.shape)} and {tuple(w2.shape)}")
    T, H = x.shape
    E, _, I, _ = w13.shape
    dev = x.device
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    if ids is None:
        ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    need = lib.fp8_moe_blockwise_work_bytes(T, I, top_k)
    if work is None:
        # never empty: sizes that need is 0 for are refused below, as sizes
        work = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    elif work.numel() < need:
        raise ValueError(f"work must hold at least {need} bytes, got {work.numel()}")
    index, stream = _where(x)
    nb_i, nb_h = _blocks(I), _blocks(H)
    _check("fp8_moe_blockwise", lib.fp8_moe_blockwise(
        _ptr(x, "x", x.dtype, (T, H), index), code,
        _ptr(logits, "logits", torch.float32, (T, E), index),
        _ptr(w13, "w13", torch.uint8, (E, 2, I, H), index),
        _ptr(s13, "s13", torch.float32, (E, 2, nb_i, nb_h), index),
        _ptr(w2, "w2", torch.uint8, (E, H, I), index),
        _ptr(s2, "s2", torch.float32, (E, nb_h, nb_i), index),
        _ptr(y, "y", torch.bfloat16, (T, H), index),
        _ptr(ids, "ids", torch.int32, (T, top_k), index),
        _ptr(weights, "weights", torch.float32, (T, top_k), index),
        _ptr(work, "work", torch.uint8, work.shape, index),
        T, H, I, E, top_k, 1 if renormalize else 0, stream))
    return y, ids, weights


def moe_work_bytes(tokens: int, inter: int, top_k: int) -> int:
    """Bytes of scratch fp8_moe_blockwise needs (0 for sizes it refuses)."""
    return int(lib.fp8_moe_blockwise_work_bytes(tokens, inter, top_k))


def _kv_cache(k_pages, v_pages, k_scale, v_scale, index: int):
    """fp8q_kv_cache of the cache's tensors, and its number of heads and head_dim."""
    if k_pages.dim() != 4:
        raise ValueError(f"k_pages must be [pages, kv_heads, page_size, head_dim], got "
                         f"{tuple(k_pages.shape)}")
    pages, heads, size, dim = shape = k_pages.shape
    cells = (pages, heads)
    return _kv_cache_bytes(_ptr(k_pages, "k_pages", torch.uint8, shape, index),
                           _ptr(v_pages, "v_pages", torch.uint8, (pages, heads, dim, size), index),
                           _ptr(k_scale, "k_scale", torch.float32, cells, index),
                           _ptr(v_scale, "v_scale", torch.float32, cells, index),
                           pages, heads, size, dim), heads, dim


def _kv_batch(page_table, q_start, kv_lens, tokens: int, max_q: int, index: int) -> bytes:
    if page_table.dim() != 2:
        raise ValueError(f"page_table must be [seqs, width], got {tuple(page_table.shape)}")
    seqs, width = shape = page_table.shape
    return _kv_batch_bytes(_ptr(page_table, "page_table", torch.int32, shape, index),
                           _ptr(q_start, "q_start", torch.int32, (seqs + 1,), index),
                           _ptr(kv_lens, "kv_lens", torch.int32, (seqs,), index),
                           tokens, seqs, width, max_q)


def _rows(t: torch.Tensor, name: str, dtype, shape, index: int):
    """Pointer and row stride of a [tokens, heads, head_dim] tensor whose rows may lie apart."""
    if not (type(t) is torch.Tensor and t.dtype is dtype and t.get_device() == index
            and t.shape == shape):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA (HIP) tensor")
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{index}")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    tokens, heads, dim = shape
    row, head, one = t.stride()
    if ((dim > 1 and one != 1) or (heads > 1 and head != dim)) and t.numel():
        raise ValueError(f"{name}: a row's heads must be contiguous, got strides {t.stride()}")
    return t.data_ptr(), row if tokens > 1 else heads * dim


def fp8_kv_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                  k_scale: torch.Tensor, v_scale: torch.Tensor, page_table: torch.Tensor,
                  q_start: torch.Tensor, kv_lens: torch.Tensor, max_q: int,
                  rope: torch.Tensor | None = None, interleaved: bool = False,
                  q: torch.Tensor | None = None, q_out: torch.Tensor | None = None):
    """Appends a batch's new keys and values k, v [tokens, kv_heads, head_dim] (bf16/fp16) to a
    paged FP8 cache, the keys rotated by their positions, and rotates the queries
    q [tokens, q_heads, head_dim] likewise.

    The cache: k_pages uint8 [pages, kv_heads, page_size, head_dim], v_pages uint8 [pages,
    kv_heads, head_dim, page_size], k_scale and v_scale float32 [pages, kv_heads]; changed in
    place.  A page's scale is a power of two, and grows with the page.  The batch (int32):
    page_table [seqs, width] (-1: no page), q_start [seqs + 1], the first row of each sequence's
    new tokens, kv_lens [seqs], the sequences' lengths with them; max_q, the most new tokens of
    a sequence.  rope float32 [positions, R]: R/2 cosines, then R/2 sines of a position's angles
    (interleaved: pairs are neighbours).  k, v, q may be slices of one projection's output;
    q_out may be q.  Returns q_out (None without q)."""
    code = _dtype_code(k)
    index, stream = _where(k)
    cache, kv_heads, head_dim = _kv_cache(k_pages, v_pages, k_scale, v_scale, index)
    if k.dim() != 3 or (q is not None and q.dim() != 3):
        raise ValueError("k, v and q must be [tokens, heads, head_dim]")
    tokens = k.shape[0]
    batch = _kv_batch(page_table, q_start, kv_lens, tokens, max_q, index)
    shape = (tokens, kv_heads, head_dim)
    rows, dim = 0, 0
    if rope is not None:
        if rope.dim() != 2:
            raise ValueError(f"rope must be [positions, R], got {tuple(rope.shape)}")
        rows, dim = rope.shape
    heads, qp, qs, op, os_ = 0, None, 0, None, 0
    if q is not None:
        heads = q.shape[1]
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        qshape = (tokens, heads, head_dim)
        qp, qs = _rows(q, "q", k.dtype, qshape, index)
        op, os_ = _rows(q_out, "q_out", k.dtype, qshape, index)
    elif q_out is not None:
        raise ValueError("q_out without q")
    _check("fp8_kv_append", lib.fp8_kv_append(
        cache, batch, *_rows(k, "k", k.dtype, shape, index), *_rows(v, "v", k.dtype, shape, index),
        code, _ptr(rope, "rope", torch.float32, (rows, dim), index) if dim else None, rows, dim,
        1 if interleaved else 0, qp, qs, op, os_, heads, stream))
    return q_out


def paged_attention_work_bytes(tokens: int, seqs: int, table_width: int, max_q: int, q_heads: int,
                               kv_heads: int, page_size: int, head_dim: int) -> int:
    """Bytes of scratch fp8_paged_attention needs (0 for sizes it refuses)."""
    return int(lib.fp8_paged_attention_work_bytes(
        _kv_cache_bytes(0, 0, 0, 0, 1, kv_heads, page_size, head_dim),
        _kv_batch_bytes(0, 0, 0, tokens, seqs, table_width, max_q), q_heads))


def paged_attention_work(q: torch.Tensor, k_pages: torch.Tensor, page_table: torch.Tensor,
                         max_q: int) -> torch.Tensor:
    """Scratch for fp8_paged_attention calls of these sizes.  Calls that may run at the same
    time need one each, and so do captured graphs that may."""
    need = paged_attention_work_bytes(q.shape[0], page_table.shape[0], page_table.shape[1], max_q,
                                      q.shape[1], k_pages.shape[1], k_pages.shape[2], k_pages.shape[3])
    return torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)


def fp8_paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                        k_scale: torch.Tensor, v_scale: torch.Tensor, page_table: torch.Tensor,
                        q_start: torch.Tensor, kv_lens: torch.Tensor, max_q: int,
                        scale: float | None = None, causal: bool = True, window: int = 0,
                        y: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                        work: torch.Tensor | None = None):
    """softmax(scale * q k^T) v of a batch's new tokens over a paged FP8 cache (see fp8_kv_append
    for the cache and the batch; their keys and values are appended before).

    q [tokens, q_heads, head_dim] bf16/fp16; query head j reads key/value head j // (q_heads //
    kv_heads).  scale: 1/sqrt(head_dim) when not given.  causal: a token sees those at or before
    its position; window > 0: of these only the last `window`.  work is scratch (uint8,
    allocated when not given; paged_attention_work).  The kernel goes by the page table's width,
    which is known on the host: a table no wider than the longest sequence needs is the fastest.
    Returns (y like q, lse float32 [tokens, q_heads]); a row that sees no token gets zeros and -inf."""
    code = _dtype_code(q)
    index, stream = _where(q)
    cache, kv_heads, head_dim = _kv_cache(k_pages, v_pages, k_scale, v_scale, index)
    if q.dim() != 3:
        raise ValueError(f"q must be [tokens, heads, head_dim], got {tuple(q.shape)}")
    tokens, heads = q.shape[:2]
    batch = _kv_batch(page_table, q_start, kv_lens, tokens, max_q, index)
    shape = (tokens, heads, head_dim)
    if y is None:
        y = torch.empty(shape, dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((tokens, heads), dtype=torch.float32, device=q.device)
    need = lib.fp8_paged_attention_work_bytes(cache, batch, heads)
    if work is None:
        # never empty: sizes that need is 0 for are refused below, as sizes
        work = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    elif work.numel() < need:
        raise ValueError(f"work must hold at least {need} bytes, got {work.numel()}")
    _check("fp8_paged_attention", lib.fp8_paged_attention(
        cache, batch, *_rows(q, "q", q.dtype, shape, index), code, heads,
        head_dim ** -0.5 if scale is None else scale, 1 if causal else 0, window,
        _ptr(y, "y", q.dtype, shape, index), _ptr(lse, "lse", torch.float32, (tokens, heads), index),
        _ptr(work, "work", torch.uint8, work.shape, index), stream))
    return y, lse


class DelayedScaling:
    """Device state of delayed scaling for one tensor: the amax of its last
    `length` quantizations (zeros at first) and the scale the next one uses.
    Use one object per tensor and issue its calls on one stream."""

    def __init__(self, length: int = 1024, device="cuda"):
        if length < 1:
            raise ValueError("the amax history needs at least one entry")
        self.history = torch.zeros(length, dtype=torch.float32, device=device)
        self.state = torch.zeros(DELAYED_STATE_WORDS, dtype=torch.int32, device=device)

    def _args(self):
        return (_dev(self.history, "history", torch.float32), self.history.numel(),
                _dev(self.state, "state", torch.int32, (DELAYED_STATE_WORDS,)))

    @property
    def next_scale(self) -> float:
        """The scale the next call will use (1.0 before any history)."""
        s = float(self.state[:1].view(torch.float32).item())
        return s if s > 0 else 1.0

    @property
    def position(self) -> int:
        return int(self.state[2].item())


def fp8_quantize_act_delayed(x: torch.Tensor, ds: DelayedScaling, q: torch.Tensor | None = None,
                             scale: torch.Tensor | None = None,
                             amax: torch.Tensor | None = None):
    """fp8_quantize_act with delayed scaling: codes with the scale of ds's amax
    history, then x's amax recorded in it.  Returns (q, scale used, amax of x)."""
    code = _dtype_code(x)
    if q is None:
        q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = torch.empty(1, dtype=torch.float32, device=x.device)
    if amax is None:
        amax = torch.empty(1, dtype=torch.float32, device=x.device)
    if q.numel() != x.numel():
        raise ValueError("q must have as many elements as x")
    _check("fp8_quantize_act_delayed", lib.fp8_quantize_act_delayed(
        _dev(x, "x"), code, x.numel(), _dev(q, "q", torch.uint8), _scalar(scale, "scale"),
        _scalar(amax, "amax"), *ds._args(), _stream(x)))
    return q, scale, amax


def fp8_linear_delayed(x: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor, ds: DelayedScaling,
                       y: torch.Tensor | None = None, q: torch.Tensor | None = None,
                       scale: torch.Tensor | None = None, amax: torch.Tensor | None = None):
    """fp8_linear with delayed activation scaling (ds holds the amax history).
    Returns (y, q, scale used, amax of x)."""
    code = _dtype_code(x)
    M, N, K = _mnk(x, qw)
    dev = x.device
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=dev)
    if scale is None:
        scale = torch.empty(1, dtype=torch.float32, device=dev)
    if amax is None:
        amax = torch.empty(1, dtype=torch.float32, device=dev)
    hist, hlen, state = ds._args()
    _check("fp8_linear_delayed", lib.fp8_linear_delayed(
        _dev(x, "x"), code, _dev(qw, "qw", torch.uint8), _scalar(sw, "sw"),
        _dev(y, "y", torch.bfloat16, (M, N)), _dev(q, "q", torch.uint8, (M, K)),
        _scalar(scale, "scale"), _scalar(amax, "amax"), hist, hlen, state, M, N, K, _stream(x)))
    return y, q, scale, amax


def nested_split(w: torch.Tensor, hi: torch.Tensor | None = None,
                 lo: torch.Tensor | None = None):
    """NestedFP byte planes of an fp16 tensor: (hi, lo) uint8 of w's shape."""
    if hi is None:
        hi = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    if lo is None:
        lo = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    if hi.numel() != w.numel() or lo.numel() != w.numel():
        raise ValueError("hi and lo must have as many elements as w")
    _check("nested_split", lib.nested_split(
        _dev(w, "w", torch.float16), _dev(hi, "hi", torch.uint8), _dev(lo, "lo", torch.uint8),
        w.numel(), _stream(w)))
    return hi, lo


def nested_rebuild_fp16(hi: torch.Tensor, lo: torch.Tensor,
                        w: torch.Tensor | None = None) -> torch.Tensor:
    """fp16 tensor with words (hi << 8) | lo."""
    if hi.shape != lo.shape:
        raise ValueError("hi and lo must have the same shape")
    if w is None:
        w = torch.empty(hi.shape, dtype=torch.float16, device=hi.device)
    _check("nested_rebuild_fp16", lib.nested_rebuild_fp16(
        _dev(hi, "hi", torch.uint8), _dev(lo, "lo", torch.uint8),
        _dev(w, "w", torch.float16, hi.shape), hi.numel(), _stream(hi)))
    return w


def nested_gemm_fp16(a: torch.Tensor, hi: torch.Tensor, lo: torch.Tensor,
                     y: torch.Tensor | None = None) -> torch.Tensor:
    """NestedFP FP16 mode: y[M,N] fp16 = a[M,K] . fp16((hi<<8)|lo)[N,K]^T."""
    M, N, K = _mnk(a, hi)
    if lo.shape != hi.shape:
        raise ValueError("hi and lo must have the same shape")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=a.device)
    _check("nested_gemm_fp16", lib.nested_gemm_fp16(
        _dev(a, "a", torch.float16), _dev(hi, "hi", torch.uint8), _dev(lo, "lo", torch.uint8),
        _dev(y, "y", torch.float16, (M, N)), M, N, K, _stream(a)))
    return y


def nested_gemm_fp8(qa: torch.Tensor, sa: torch.Tensor, hi: torch.Tensor,
                    y: torch.Tensor | None = None) -> torch.Tensor:
    """NestedFP FP8 mode: y[M,N] fp16 = (qa . E5M2(hi)^T) * sa."""
    M, N, K = _mnk(qa, hi)
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=qa.device)
    _check("nested_gemm_fp8", lib.nested_gemm_fp8(
        _dev(qa, "qa", torch.uint8), _scalar(sa, "sa"), _dev(hi, "hi", torch.uint8),
        _dev(y, "y", torch.float16, (M, N)), M, N, K, _stream(qa)))
    return y


def nested_linear_fp8(a: torch.Tensor, hi: torch.Tensor, y: torch.Tensor | None = None,
                      q: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                      amax: torch.Tensor | None = None):
    """One NestedFP FP8-mode linear layer: quantize a[M,K] (fp16) per tensor,
    then y[M,N] fp16 = (q . E5M2(hi)^T) * scale.  Returns (y, q, scale, amax)."""
    if a.dtype != torch.float16:
        raise TypeError(f"a must be float16, got {a.dtype}")
    M, N, K = _mnk(a, hi)
    dev = a.device
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=dev)
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=dev)
    if scale is None:
        scale = torch.empty(1, dtype=torch.float32, device=dev)
    if amax is None:
        amax = torch.empty(1, dtype=torch.float32, device=dev)
    _check("nested_linear_fp8", lib.nested_linear_fp8(
        _dev(a, "a", torch.float16), _dev(hi, "hi", torch.uint8),
        _dev(y, "y", torch.float16, (M, N)), _dev(q, "q", torch.uint8, (M, K)),
        _scalar(scale, "scale"), _scalar(amax, "amax"), M, N, K, _stream(a)))
    return y, q, scale, amax


def nested_split_e4m3(w: torch.Tensor, hi: torch.Tensor | None = None,
                      lo: torch.Tensor | None = None):
    """NestedFP planes with an E4M3 upper byte: hi = sign | bits 13..7 (the E4M3
    code of w * 2^8 when |w| < 2), lo = bit 14 | bits 6..0.  Returns (hi, lo,
    out_of_range), the last an int64 device tensor counting the words outside
    the FP8 mode's range |w| < 1.875."""
    if hi is None:
        hi = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    if lo is None:
        lo = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    if hi.numel() != w.numel() or lo.numel() != w.numel():
        raise ValueError("hi and lo must have as many elements as w")
    bad = torch.zeros(1, dtype=torch.int64, device=w.device)
    _check("nested_split_e4m3", lib.nested_split_e4m3(
        _dev(w, "w", torch.float16), _dev(hi, "hi", torch.uint8), _dev(lo, "lo", torch.uint8),
        w.numel(), _dev(bad, "out_of_range", torch.int64), _stream(w)))
    return hi, lo, bad


def nested_rebuild_e4m3(hi: torch.Tensor, lo: torch.Tensor,
                        w: torch.Tensor | None = None) -> torch.Tensor:
    """fp16 words rebuilt from the E4M3-split planes."""
    if hi.shape != lo.shape:
        raise ValueError("hi and lo must have the same shape")
    if w is None:
        w = torch.empty(hi.shape, dtype=torch.float16, device=hi.device)
    _check("nested_rebuild_e4m3", lib.nested_rebuild_e4m3(
        _dev(hi, "hi", torch.uint8), _dev(lo, "lo", torch.uint8),
        _dev(w, "w", torch.float16, hi.shape), hi.numel(), _stream(hi)))
    return w


def nested_gemm_fp16_e4m3(a: torch.Tensor, hi: torch.Tensor, lo: torch.Tensor,
                          y: torch.Tensor | None = None) -> torch.Tensor:
    """NestedFP FP16 mode on E4M3-split planes: y fp16 = a . rebuilt(hi, lo)^T."""
    M, N, K = _mnk(a, hi)
    if lo.shape != hi.shape:
        raise ValueError("hi and lo must have the same shape")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=a.device)
    _check("nested_gemm_fp16_e4m3", lib.nested_gemm_fp16_e4m3(
        _dev(a, "a", torch.float16), _dev(hi, "hi", torch.uint8), _dev(lo, "lo", torch.uint8),
        _dev(y, "y", torch.float16, (M, N)), M, N, K, _stream(a)))
    return y


def nested_gemm_fp8_e4m3(qa: torch.Tensor, sa: torch.Tensor, hi: torch.Tensor,
                         y: torch.Tensor | None = None) -> torch.Tensor:
    """NestedFP FP8 mode on E4M3-split planes: y fp16 = (qa . E4M3(hi)^T) * sa * 2^-8."""
    M, N, K = _mnk(qa, hi)
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=qa.device)
    _check("nested_gemm_fp8_e4m3", lib.nested_gemm_fp8_e4m3(
        _dev(qa, "qa", torch.uint8), _scalar(sa, "sa"), _dev(hi, "hi", torch.uint8),
        _dev(y, "y", torch.float16, (M, N)), M, N, K, _stream(qa)))
    return y


def nested_linear_fp8_e4m3(a: torch.Tensor, hi: torch.Tensor, y: torch.Tensor | None = None,
                           q: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                           amax: torch.Tensor | None = None):
    """nested_linear_fp8 on E4M3-split planes.  Returns (y, q, scale, amax)."""
    if a.dtype != torch.float16:
        raise TypeError(f"a must be float16, got {a.dtype}")
    M, N, K = _mnk(a, hi)
    dev = a.device
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=dev)
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=dev)
    if scale is None:
        scale = torch.empty(1, dtype=torch.float32, device=dev)
    if amax is None:
        amax = torch.empty(1, dtype=torch.float32, device=dev)
    _check("nested_linear_fp8_e4m3", lib.nested_linear_fp8_e4m3(
        _dev(a, "a", torch.float16), _dev(hi, "hi", torch.uint8),
        _dev(y, "y", torch.float16, (M, N)), _dev(q, "q", torch.uint8, (M, K)),
        _scalar(scale, "scale"), _scalar(amax, "amax"), M, N, K, _stream(a)))
    return y, q, scale, amax


def e4m3_encode_f32(v: torch.Tensor, q: torch.Tensor | None = None) -> torch.Tensor:
    """The device E4M3 encoder on float32 values (for exhaustive checks)."""
    if q is None:
        q = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
    _check("fp8q_e4m3_encode_f32", lib.fp8q_e4m3_encode_f32(
        _dev(v, "v", torch.float32), _dev(q, "q", torch.uint8, v.shape), v.numel(), _stream(v)))
    return q

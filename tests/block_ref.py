"""Plain references of the block-scaled operators for the GPU tests: numpy in 64 bits, apart
from the codes, which come from the oracle's quantizer applied to one block at a time."""
import numpy as np

import oracle

B = 128


def blocks(n):
    return (n + B - 1) // B


def quantize_blocks(x_bits, code):
    """Codes [rows, cols] and scales [K blocks, rows] of 16-bit patterns."""
    rows, cols = x_bits.shape
    q = np.empty((rows, cols), np.uint8)
    s = np.empty((blocks(cols), rows), np.float32)
    for b in range(blocks(cols)):
        part = np.ascontiguousarray(x_bits[:, b * B:(b + 1) * B])
        q[:, b * B:(b + 1) * B], s[b], _ = oracle.quantize_rows(part, code)
    return q, s


def quantize_weight_blocks(w_bits, code):
    """Codes like w[N, K] and scales [N blocks, K blocks]."""
    n, k = w_bits.shape
    q = np.empty((n, k), np.uint8)
    s = np.empty((blocks(n), blocks(k)), np.float32)
    for i in range(blocks(n)):
        for j in range(blocks(k)):
            part = w_bits[i * B:(i + 1) * B, j * B:(j + 1) * B]
            c, s[i, j], _ = oracle.quantize(np.ascontiguousarray(part).ravel(), code)
            q[i * B:(i + 1) * B, j * B:(j + 1) * B] = c.reshape(part.shape)
    return q, s


def decode(q):
    return oracle.e4m3_decode(q)


def act_values(q, s):
    return decode(q) * np.repeat(s.astype(np.float64).T, B, axis=1)[:, :q.shape[1]]


def weight_values(q, s):
    n, k = q.shape
    return decode(q) * np.repeat(np.repeat(s.astype(np.float64), B, axis=0)[:n], B, axis=1)[:, :k]


def gemm(qa, sa, qw, sw, cols=None):
    """y in 64 bits and sum |a b|, for all columns or the given ones."""
    a = act_values(qa, sa)
    if cols is None:
        w = weight_values(qw, sw)
    else:
        w = decode(qw[cols]) * np.repeat(sw.astype(np.float64)[np.asarray(cols) // B], B, axis=1)[:, :qw.shape[1]]
    return a @ w.T, np.abs(a) @ np.abs(w).T


def gemm_tolerance(ref, ab, k):
    """How far a bf16 result may be from `ref`.

    Within a block the matrix core adds 128 products, whose order and alignment are its own:
    each of the at most 128 additions is off by at most one unit in the last place of fp32
    relative to the partial sum, which sum |a b| bounds (2^-23 a piece, so truncation is
    covered too).  The product of the scales and its FMA per block add 2^-24 each per block
    and once more for the scales' own rounding.  Then one bf16 rounding, 2^-8 relative to the
    value rounded, itself within the first part of ref."""
    acc = (B * 2.0 ** -23 + (blocks(k) + 2) * 2.0 ** -24) * ab
    return acc + 2.0 ** -8 * (np.abs(ref) + acc) + 1e-38

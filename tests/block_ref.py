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

    The matrix core adds FP8 products eight neighbours in K at a time: it aligns them to the
    largest, of exponent e, and drops what lies below 2^(e - 13) of each (measured with one
    product of 2^12 beside one of 2^(12 - r) among its eight neighbours: kept whole to r = 13,
    1.75 * 2^(12 - r) cut to 1.5 at r = 12 and to 1 at r = 13, gone from r = 14 on, alike for
    both signs; in another group of eight kept to r = 21).  The largest itself has at most eight
    significant bits and loses nothing, so a group is off by less than 7 * 2^-13 of its largest
    product, and all groups together by less than 7 * 2^-13 sum |a b|.  Adding up the groups
    of a block in fp32 costs at most 2^-23 of sum |a b| for each of its 16 additions (truncation
    is covered), the product of the scales and its FMA 2^-24 per block and 2^-24 once more.
    Then one bf16 rounding, 2^-8 relative to the value rounded, itself within the first part
    of ref."""
    acc = (7 * 2.0 ** -13 + 16 * 2.0 ** -23 + (blocks(k) + 2) * 2.0 ** -24) * ab
    return acc + 2.0 ** -8 * (np.abs(ref) + acc) + 1e-38


def route(logits, top_k, renormalize):
    """ids [T, top_k], weights in 64 bits, and how far fp32 weights may be from them.

    exp's argument l - max is rounded once, which moves the weight by |l - max| 2^-24; exp is
    good to 2 units in the last place (4 half units), a sum of up to 512 positive terms (8 in
    a lane, 6 levels of a tree; or 16 in sequence) with such errors in its terms to 16 + 8,
    the quotient to 1: less than |l - max| + 32 half units.  Weights below fp32's normal
    range are covered by the 1e-37."""
    T, E = logits.shape
    off = np.full((T, top_k), 1e-37)
    ids = np.full((T, top_k), -1, np.int32)
    weights = np.zeros((T, top_k))
    for t in range(T):
        row = np.where(np.isnan(logits[t]), -np.inf, logits[t].astype(np.float64))
        order = [e for e in np.argsort(-row, kind="stable") if row[e] > -np.inf]
        if not order:
            continue
        top = row[order[0]]
        p = {e: 1.0 if row[e] == top else float(np.exp(row[e] - top)) for e in order}
        chosen = order[:top_k]
        total = sum(p[e] for e in (chosen if renormalize else order))
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = [p[e] / total for e in chosen]
        for j, e in enumerate(chosen):
            gap = 0.0 if row[e] == top else abs(row[e] - top)
            off[t, j] += (gap + 32) * 2.0 ** -24 * weights[t, j] if weights[t, j] else 0.0
    return ids, weights, off


def moe(x, logits, w13, s13, w2, s2, top_k, renormalize):
    """y in 64 bits, how far a bf16 result may be from it, then what route() returns.

    With c = 128 * 2^-23 + (blocks + 2) * 2^-24 for a product of that many blocks (bf16 and
    fp16 operands: each of a block's 128 additions off by at most 2^-23 of sum |W x|, scale and
    FMA 2^-24 per block), g and u are off by at most c * sum |W x|.  silu's slope is below 1.1, its
    exp, sum and quotient are good to 2^-20, and h is rounded to bf16 (2^-8).  The weights are
    off as route() says, and each expert's term is added with one more FMA (2^-24 each, at
    most 16 waves' sums of 16 terms).  y gets one bf16 rounding.  A value that this leaves below bf16's normal range is covered
    by the 1e-38."""
    T, H = x.shape
    E, _, I, _ = w13.shape
    ids, weights, woff = route(logits, top_k, renormalize)
    cu = B * 2.0 ** -23 + (blocks(H) + 2) * 2.0 ** -24
    cd = B * 2.0 ** -23 + (blocks(I) + 2) * 2.0 ** -24
    y, off = np.zeros((T, H)), np.zeros((T, H))
    for e in sorted(set(ids.ravel()) - {-1}):
        t, j = np.nonzero(ids == e)
        wg, wu = (weight_values(w13[e, c], s13[e, c]) for c in (0, 1))
        wd = weight_values(w2[e], s2[e])
        g, u = x[t] @ wg.T, x[t] @ wu.T
        dg, du = (cu * (np.abs(x[t]) @ np.abs(w).T) for w in (wg, wu))
        silu = g / (1 + np.exp(-g))
        h = silu * u
        dh = (1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du)
        dh = dh + (2.0 ** -8 + 2.0 ** -20) * (np.abs(h) + dh) + 1e-38
        ab = np.abs(h) + dh
        w, dw = weights[t, j][:, None], woff[t, j][:, None]
        y[t] += w * (h @ wd.T)
        off[t] += w * (dh @ np.abs(wd).T) + (w * (cd + 32 * 2.0 ** -24) + dw) * (ab @ np.abs(wd).T)
    return y, off + 2.0 ** -8 * (np.abs(y) + off) + 1e-38, ids, weights, woff

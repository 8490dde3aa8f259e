"""What fp8_moe_blockwise keeps of h between its two kernels.

Every row of W2 takes differences of columns of h that are nearly equal, so that y consists of
the bits of h below bf16's: a form that keeps h in bf16 alone, or puts the low parts of h in
other columns, is far outside the bound.  One token to 64 (the kernels change with T), widths of
every form of the down projection, an expert width that ends inside a block, |h| from 2^-110 to
2^123.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
import oracle
from fp8_quantized_gemm_amd import fp8q
from gpu_helpers import DEV, say, to_dev_u8

ONE = 0x38                                   # E4M3 code of 1


def _case(T, E, H, I, top_k, exponent, seed):
    """x has two values per token: one that makes g and u alike in all columns, and one 2^-9 of
    it or less on which the columns differ.  W2's rows are +1 and -1 at columns 37 apart, each
    column once on either side.  u's scales are 2^exponent, which scales h alike."""
    rng = np.random.Generator(np.random.PCG64(seed))
    x = np.zeros((T, H), np.float32)
    big, small = H // 2, 3
    x[:, big] = 2.0 + np.arange(T) % 64 / 64
    x[:, small] = 2.0 ** -9
    w13 = np.zeros((E, 2, I, H), np.uint8)
    w13[..., big] = ONE
    # +-(1 + n / 8), n = 0..7
    w13[..., small] = ONE + rng.integers(0, 8, (E, 2, I)) + 0x80 * rng.integers(0, 2, (E, 2, I))
    s13 = np.ones((E, 2, ref.blocks(I), ref.blocks(H)), np.float32)
    s13[:, 1] = 2.0 ** exponent
    d = np.zeros((H, I))
    cols = np.arange(I)
    np.add.at(d, (cols % H, cols), 1.0)
    np.add.at(d, (cols % H, (cols + 37) % I), -1.0)
    w2 = np.broadcast_to(oracle.e4m3_encode(d.astype(np.float32)).reshape(1, H, I), (E, H, I)).copy()
    s2 = np.ones((E, ref.blocks(H), ref.blocks(I)), np.float32)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    return x, logits, w13, s13, w2, s2


def _bf16(v):
    return oracle.bf16_decode(oracle.bf16_encode(v.astype(np.float32))).astype(np.float64).reshape(v.shape)


def _reference(x, logits, w13, s13, w2, s2, top_k):
    """y in 64 bits, how far a bf16 result may be from it, and y with h rounded to bf16.

    As block_ref.moe, but for h: an fp16 value with a power of two per four columns is off by at
    most 2^-11 of itself where it is normal.  The largest of the four is scaled to [2^7, 2^8), so
    one that is subnormal (they are 2^-24 apart) is off by 2^-32 of the largest.  Brought to the power of
    two of their block's largest, which comes to [2^14, 2^15), subnormals are off by 2^-39 of it; four
    columns below 2^-31 of it are lost.  Together less than 2^-31 of the block's largest."""
    T, H = x.shape
    I = w2.shape[2]
    ids, weights, woff = ref.route(logits, top_k, True)
    cu = ref.B * 2.0 ** -23 + (ref.blocks(H) + 2) * 2.0 ** -24
    cd = ref.B * 2.0 ** -23 + (ref.blocks(I) + 2) * 2.0 ** -24
    y, rough, off = (np.zeros((T, H)) for _ in range(3))
    for e in sorted(set(ids.ravel())):
        t, j = np.nonzero(ids == e)
        wg, wu = (ref.weight_values(w13[e, c], s13[e, c]) for c in (0, 1))
        wd = ref.weight_values(w2[e], s2[e])
        g, u = x[t] @ wg.T, x[t] @ wu.T
        dg, du = (cu * (np.abs(x[t]) @ np.abs(w).T) for w in (wg, wu))
        silu = g / (1 + np.exp(-g))
        h = silu * u
        dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du
        dh = dh + (2.0 ** -11 + 2.0 ** -20) * (np.abs(h) + dh)
        starts = np.arange(0, I, ref.B)
        top = np.maximum.reduceat(np.abs(h) + dh, starts, axis=1)
        dh = dh + 2.0 ** -31 * np.repeat(top, ref.B, axis=1)[:, :I]
        w, dw = weights[t, j][:, None], woff[t, j][:, None]
        y[t] += w * (h @ wd.T)
        rough[t] += w * (_bf16(h) @ wd.T)
        off[t] += w * (dh @ np.abs(wd).T) + (w * (cd + 32 * 2.0 ** -24) + dw) * ((np.abs(h) + dh) @ np.abs(wd).T)
    return y, off + 2.0 ** -8 * (np.abs(y) + off) + 1e-38, rough


CASES = [
    # one row tile of the down projection, each form of the up projection
    (1, 3, 256, 272, 2, 0), (4, 3, 144, 144, 1, -24), (8, 4, 272, 400, 2, 14), (9, 4, 272, 400, 2, 0),
    (16, 4, 272, 400, 2, -60), (17, 4, 272, 400, 2, 0), (40, 5, 256, 656, 3, 60), (64, 2, 512, 272, 1, 0),
    (64, 128, 144, 528, 8, 0), (20, 128, 144, 528, 4, -24),
    # two, three and four row tiles
    (2, 2, 2064, 272, 2, -24), (8, 2, 4096, 144, 1, 0), (9, 2, 2064, 400, 1, 14), (64, 2, 4096, 256, 2, 0),
    (5, 2, 4112, 272, 1, 0), (33, 2, 6144, 144, 2, 0), (8, 2, 6160, 272, 2, 14), (64, 3, 8176, 144, 2, -24),
    # near the ends of fp32's range
    (3, 3, 272, 400, 2, 122), (12, 3, 272, 400, 2, -110), (40, 3, 2064, 144, 2, 122), (6, 3, 2064, 400, 2, -110),
]


def test_bound_tells_a_rounded_h():
    """The inputs and the bound of the GPU test: h in bf16 alone would fail it."""
    for T, E, H, I, top_k, exponent in CASES[:8]:
        args = _case(T, E, H, I, top_k, exponent, 1)
        y, off, rough = _reference(args[0].astype(np.float64), *args[1:], top_k)
        used = np.abs(y).max(axis=1) > 0
        assert used.all()
        assert ((np.abs(rough - y) > off).any(axis=1)).all(), (T, E, H, I, top_k)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,E,H,I,top_k,exponent", CASES)
def test_low_bits_of_h_are_kept(T, E, H, I, top_k, exponent, dtype):
    x, logits, *w = _case(T, E, H, I, top_k, exponent, 1)
    y, off, _ = _reference(x.astype(np.float64), logits, *w, top_k)
    xd = torch.from_numpy(x).to(torch.bfloat16 if dtype == "bf16" else torch.float16)
    assert torch.equal(xd.float(), torch.from_numpy(x))
    f32 = lambda a: torch.from_numpy(a).to(DEV)
    say("moe low bits of h", T, E, H, I, top_k, exponent, dtype)
    got, _, _ = fp8q.fp8_moe_blockwise(xd.to(DEV), f32(logits), to_dev_u8(w[0]), f32(w[1]),
                                       to_dev_u8(w[2]), f32(w[3]), top_k)
    bad = np.abs(got.double().cpu().numpy() - y) - off
    assert np.all(bad <= 0), f"{(bad > 0).sum()} outside, worst by {bad.max()}"


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I", [(3, 272, 400), (12, 272, 400), (40, 2064, 272), (64, 512, 272)])
def test_small_columns_beside_large_ones(T, H, I):
    """A quarter of the columns of h are 2^17 times the others, and no row of W2 takes them: the
    small ones keep their precision beside them."""
    x, logits, w13, s13, w2, s2 = _case(T, 3, H, I, 2, 0, 5)
    w13[:, 1, :, 3] = 0
    w13[:, 1, :, H // 2] = 0x01                                    # 2^-9
    w13[:, 1, ::4, H // 2] = 0x78                                  # 2^8
    d = np.zeros((H, I), np.float32)
    small = np.array([i for i in range(I) if i % 4])
    np.add.at(d, (small % H, small), 1.0)
    np.add.at(d, (small % H, (small + 36) // 4 * 4 % I + small % 4), -1.0)
    w2[:] = oracle.e4m3_encode(d).reshape(1, H, I)
    y, off, rough = _reference(x.astype(np.float64), logits, w13, s13, w2, s2, 2)
    assert (np.abs(rough - y) > off).any()
    f32 = lambda a: torch.from_numpy(a).to(DEV)
    say("moe small beside large", T, H, I)
    got, _, _ = fp8q.fp8_moe_blockwise(torch.from_numpy(x).to(torch.bfloat16).to(DEV), f32(logits),
                                       to_dev_u8(w13), f32(s13), to_dev_u8(w2), f32(s2), 2)
    bad = np.abs(got.double().cpu().numpy() - y) - off
    assert np.all(bad <= 0), f"{(bad > 0).sum()} outside, worst by {bad.max()}"


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 12, 40])
def test_nan_scales_and_overflow_reach_y(T):
    """A NaN scale of W2 in one block of columns and an h beyond fp32 are seen, not lost."""
    E, H, I = 2, 272, 400
    x, logits, w13, s13, w2, s2 = _case(T, E, H, I, 1, 0, 1)
    logits[:] = [0, -1]
    f32 = lambda a: torch.from_numpy(a).to(DEV)
    say("moe nan scale", T)
    xd = torch.from_numpy(x).to(torch.bfloat16).to(DEV)
    bad = s2.copy()
    bad[0, 1, 2] = np.nan
    run = lambda s13, s2: fp8q.fp8_moe_blockwise(xd, f32(logits), to_dev_u8(w13), f32(s13), to_dev_u8(w2),
                                                 f32(s2), 1)[0].float().cpu()
    clean, y = run(s13, s2), run(s13, bad)
    assert torch.isnan(y[:, 128:256]).all()
    assert torch.equal(y[:, :128], clean[:, :128]) and torch.equal(y[:, 256:], clean[:, 256:])
    large = s13.copy()
    large[0, 1] = 2.0 ** 127
    assert not torch.isfinite(run(large, s2)).any()

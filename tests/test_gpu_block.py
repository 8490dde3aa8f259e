"""GPU parity of the block-scaled operators (fp8_quantize_blocks, fp8_quantize_weight_blocks,
fp8_gemm_blockwise, fp8_linear_blockwise).

- Quantizers: codes and scales bit for bit against the oracle's quantizer run on every block
  alone, on both row orders of the activation kernel, ragged last blocks, zero blocks, large
  and tiny values.
- GEMM: bit for bit on small integers with power-of-two scales (exact sums), within a derived
  bound of the 64-bit product on random operands; one token to tile sizes, columns and K that
  end inside a block or a tile.
- Linear: equals quantizer + GEMM bit for bit, also in place, on another stream, in a replayed
  graph.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
import oracle
from fp8_quantized_gemm_amd import fp8q, synth
from gpu_helpers import DEV, host, say, to_dev_u8

pytestmark = pytest.mark.gpu

GUARD = 64


def _f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV)


def _code(dtype):
    return oracle.BF16 if dtype == "bf16" else oracle.FP16


def _same_bits(t, want):
    got = host(t)
    assert np.array_equal(got.view(np.uint8), np.ascontiguousarray(want).view(np.uint8))


# ------------------------------------------------------------------ quantizers
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 4096), (3, 272), (7, 11008), (15, 128),
                                       (16, 144), (17, 5120), (33, 112), (300, 2064), (64, 25600)])
def test_quantize_blocks_bit_exact(rows, cols, dtype):
    x = synth.activation(rows, cols, seed=synth.seed_for("qb", rows, cols, dtype), dtype=dtype,
                         outliers=True)
    x[rows // 2, :min(cols, 128)] = 0.0                      # a block of zeros: scale 1
    x[0, -16:] = -0.0
    want_q, want_s = ref.quantize_blocks(synth.bits(x), _code(dtype))
    say("quantize_blocks", dtype, rows, cols)
    q, s = fp8q.fp8_quantize_blocks(x.to(DEV))
    _same_bits(q, want_q)
    _same_bits(s, want_s)


def test_quantize_blocks_extreme_values():
    """Blocks 2^e apart, up to the types' largest and smallest values, and infinities."""
    rows = []
    base = synth.activation(1, 256, seed=5).to(torch.float32)
    for e in (-120, -60, -20, 0, 20, 60, 120):
        rows.append((base * 2.0 ** e).to(torch.bfloat16))
    x = torch.cat(rows)
    x[0, 3] = 3.3e38
    x[1, 130] = -3.3e38
    x[2, :128] = 1e-40
    x[3, 200] = float("inf")
    want_q, want_s = ref.quantize_blocks(synth.bits(x), oracle.BF16)
    say("quantize_blocks extreme")
    q, s = fp8q.fp8_quantize_blocks(x.to(DEV))
    _same_bits(s, want_s)
    finite = np.isfinite(np.repeat(want_s.T, 128, axis=1))   # inf / inf has no code
    assert np.array_equal(host(q)[finite], want_q[finite])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", [(1, 16), (127, 144), (128, 128), (129, 1040), (300, 272),
                                   (3, 130, 144), (2, 2, 64, 256)])
def test_quantize_weight_blocks_bit_exact(shape, dtype):
    w = synth.normal(shape, 0.02, dtype, seed=synth.seed_for("qw", *shape, dtype))
    w[..., :1, :16] = 0.0
    say("quantize_weight_blocks", dtype, shape)
    q, s = fp8q.fp8_quantize_weight_blocks(w.to(DEV))
    n, k = shape[-2:]
    assert tuple(s.shape) == tuple(shape[:-2]) + (ref.blocks(n), ref.blocks(k))
    hq, hs = host(q).reshape(-1, n, k), host(s).reshape(-1, ref.blocks(n), ref.blocks(k))
    for i, m in enumerate(w.reshape(-1, n, k)):
        want_q, want_s = ref.quantize_weight_blocks(synth.bits(m), _code(dtype))
        assert np.array_equal(hq[i], want_q) and np.array_equal(hs[i], want_s)


# ------------------------------------------------------------------ GEMM
def _gemm(qa, sa, qw, sw):
    M, N = qa.shape[0], qw.shape[0]
    buf = torch.full((M * N + GUARD,), 7.0, dtype=torch.bfloat16, device=DEV)
    y = buf[:M * N].view(M, N)
    fp8q.fp8_gemm_blockwise(to_dev_u8(qa), _f32(sa), to_dev_u8(qw), _f32(sw), y)
    out = host(buf)
    assert np.all(out[M * N:] == synth.bits(torch.tensor([7.0], dtype=torch.bfloat16))[0])
    return out[:M * N].reshape(M, N)


SHAPES = [(1, 1, 16), (1, 37, 160), (8, 100, 12304), (16, 40, 16400), (12, 8200, 2064), (5, 33, 8192), (1, 300, 4096), (2, 129, 272), (7, 1000, 1040), (8, 16, 128),
          (9, 257, 144), (15, 515, 11008), (16, 640, 4096), (17, 64, 272), (33, 129, 112),
          (64, 1, 16), (65, 200, 1040), (129, 257, 4096), (300, 515, 272), (513, 300, 528),
          (700, 1028, 1296)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_small_integers_bit_exact(M, N, K):
    rng = np.random.Generator(np.random.PCG64(M * 7 + N * 3 + K))
    table = np.array([0x00, 0x38, 0x40, 0x48, 0xB8, 0xC0, 0xC8], np.uint8)   # 0, +-1, +-2, +-4
    qa, qw = table[rng.integers(0, 7, (M, K))], table[rng.integers(0, 7, (N, K))]
    # scale exponents 0..3: every sum is an integer below 2^24
    sa = (2.0 ** rng.integers(0, 2, (ref.blocks(K), M))).astype(np.float32)
    sw = (2.0 ** rng.integers(0, 3, (ref.blocks(N), ref.blocks(K)))).astype(np.float32)
    say("blockwise small int", M, N, K)
    want, ab = ref.gemm(qa, sa, qw, sw)
    assert ab.max() < 2 ** 24
    y = _gemm(qa, sa, qw, sw)
    assert np.array_equal(y, oracle.bf16_encode(want.astype(np.float32)).reshape(M, N))


# tiles of 16 rows of the decode kernel (N just below 4096), each number of K blocks per wave,
# one and two groups of tokens
DECODE = [(1, 4090, 1040), (3, 4094, 2064), (2, 4090, 6000), (8, 4096, 8192), (6, 4090, 11008),
          (16, 4090, 2048), (9, 4091, 4096), (11, 4090, 8192), (13, 4090, 12288), (1, 4090, 12304)]


# more tokens than a decode step on few columns: 16 and 32 columns a workgroup, one and
# several groups of 32 tokens, long K, and one column more than they take
FEW = [(17, 4096, 1040), (32, 4090, 2320), (33, 2047, 272), (64, 1000, 16400), (250, 500, 528),
       (2100, 40, 400), (8192, 16, 144), (31, 8190, 400), (64, 4081, 1296), (200, 1170, 272),
       (4000, 64, 272), (64, 4097, 272)]


@pytest.mark.parametrize("M,N,K", SHAPES + DECODE + FEW)
def test_random_within_bound(M, N, K):
    x = synth.activation(M, K, seed=synth.seed_for("bx", M, N, K), outliers=True)
    w = synth.normal((N, K), 0.02, "fp16", seed=synth.seed_for("bw", M, N, K))
    qa, sa = ref.quantize_blocks(synth.bits(x), oracle.BF16)
    qw, sw = ref.quantize_weight_blocks(synth.bits(w), oracle.FP16)
    say("blockwise random", M, N, K)
    y = oracle.bf16_decode(_gemm(qa, sa, qw, sw)).astype(np.float64).reshape(M, N)
    want, ab = ref.gemm(qa, sa, qw, sw)
    off = np.abs(y - want) - ref.gemm_tolerance(want, ab, K)
    assert np.all(off <= 0), f"{(off > 0).sum()} outside, worst by {off.max()}"


# one size for each tile shape of the larger products (128 x 64, 128 x 128, 64 x 64 twice per
# CU, 128 x 192, 128 x 256, 256 x 192, 256 x 256), with ragged edges in M, N and K
@pytest.mark.parametrize("M,N,K", [(257, 4100, 272), (333, 6100, 272), (64, 16400, 272),
                                   (500, 8200, 400), (1100, 6100, 272), (1000, 8200, 272),
                                   (1100, 10000, 272)])
def test_each_tile_shape_within_bound(M, N, K):
    x = synth.activation(M, K, seed=synth.seed_for("tx", M, N, K), outliers=True)
    w = synth.normal((N, K), 0.02, "fp16", seed=synth.seed_for("tw", M, N, K), device=DEV)
    qa, sa = ref.quantize_blocks(synth.bits(x), oracle.BF16)
    qw, sw = (host(t) for t in fp8q.fp8_quantize_weight_blocks(w))
    say("blockwise tile", M, N, K)
    y = oracle.bf16_decode(_gemm(qa, sa, qw, sw)).astype(np.float64).reshape(M, N)
    rng = np.random.Generator(np.random.PCG64(M + N))
    cols = np.unique(np.concatenate([rng.integers(0, N, 400), np.arange(N - 300, N)]))
    want, ab = ref.gemm(qa, sa, qw, sw, cols)
    off = np.abs(y[:, cols] - want) - ref.gemm_tolerance(want, ab, K)
    assert np.all(off <= 0), f"{(off > 0).sum()} outside, worst by {off.max()}"


# ------------------------------------------------------------------ linear
LINEAR = [(1, 4096, 4096), (1, 4090, 11008), (2, 4090, 8192), (4, 4090, 6000), (1, 37, 160), (3, 515, 1040), (8, 2048, 4096), (11, 300, 5120),
          (16, 4100, 2064), (5, 2048, 4096), (9, 300, 2320), (10, 515, 2048), (8, 16400, 4096),
          (16, 32784, 2048), (17, 257, 272), (200, 640, 4096), (600, 515, 1040)]


def _linear_inputs(M, N, K, dtype):
    x = synth.activation(M, K, seed=synth.seed_for("lx", M, N, K), dtype=dtype, outliers=True,
                         device=DEV)
    w = synth.normal((N, K), 0.02, "fp16", seed=synth.seed_for("lw", M, N, K), device=DEV)
    return x, *fp8q.fp8_quantize_weight_blocks(w)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear_equals_quantize_and_gemm(M, N, K, dtype):
    x, qw, sw = _linear_inputs(M, N, K, dtype)
    want_q, want_s = ref.quantize_blocks(synth.bits(x), _code(dtype))
    q0, s0 = fp8q.fp8_quantize_blocks(x)
    y0 = fp8q.fp8_gemm_blockwise(q0, s0, qw, sw)
    say("linear_blockwise", dtype, M, N, K)
    y, q, s = fp8q.fp8_linear_blockwise(x, qw, sw)
    _same_bits(q, want_q)
    _same_bits(s, want_s)
    assert torch.equal(y.view(torch.int16), y0.view(torch.int16))


def test_linear_infinite_and_nan_activations_stay_in_their_row():
    """A row with an infinity or a NaN is outside the contract; the others are as without it."""
    M, N, K = 6, 300, 1040
    x, qw, sw = _linear_inputs(M, N, K, "bf16")
    want = fp8q.fp8_linear_blockwise(x, qw, sw)[0].clone()
    x[1, 17] = float("inf")
    x[4, 1030] = float("nan")
    say("linear_blockwise inf / nan rows")
    y = fp8q.fp8_linear_blockwise(x, qw, sw)[0]
    keep = [0, 2, 3, 5]
    assert torch.equal(y[keep], want[keep])


@pytest.mark.parametrize("M,K", [(1, 4096), (5, 1040), (40, 512)])
def test_linear_in_place(M, K):
    x, qw, sw = _linear_inputs(M, K, K, "bf16")
    want = fp8q.fp8_linear_blockwise(x, qw, sw)[0].clone()
    say("linear_blockwise in place", M, K)
    fp8q.fp8_linear_blockwise(x, qw, sw, y=x)
    assert torch.equal(x.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (16, 1000, 1040), (200, 640, 272)])
def test_linear_on_another_stream_and_in_a_graph(M, N, K):
    x, qw, sw = _linear_inputs(M, N, K, "bf16")
    want = [t.clone() for t in fp8q.fp8_linear_blockwise(x, qw, sw)]
    outs = [torch.empty_like(t) for t in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    say("linear_blockwise stream", M, N, K)
    with torch.cuda.stream(side):
        fp8q.fp8_linear_blockwise(x, qw, sw, *outs)
    side.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o.view(torch.uint8), w.view(torch.uint8))
    g = torch.cuda.CUDAGraph()
    say("linear_blockwise graph", M, N, K)
    with torch.cuda.graph(g):
        fp8q.fp8_linear_blockwise(x, qw, sw, *outs)
    for rep in range(3):
        for o in outs:
            o.view(torch.uint8).fill_(0x7f)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o.view(torch.uint8), w.view(torch.uint8)), f"replay {rep}"
    del g


@pytest.mark.parametrize("M", [1, 16, 40])
def test_weights_past_32_bits(M):
    """The last rows of a weight of more than 2^32 bytes, against the same rows alone."""
    K, tail = 4112, 512
    N = (1 << 20) + tail
    assert (N - tail) * K > 1 << 32
    say("block past 32 bits", M)
    w = synth.normal((tail, K), 0.05, "bf16", seed=77, device=DEV)
    qt, st = fp8q.fp8_quantize_weight_blocks(w)
    qw = torch.zeros((N, K), dtype=torch.uint8, device=DEV)
    sw = torch.ones((N // 128, st.shape[1]), dtype=torch.float32, device=DEV)
    qw[-tail:], sw[-(tail // 128):] = qt, st
    x = synth.activation(M, K, seed=78, outliers=True, device=DEV)
    y, q, s = fp8q.fp8_linear_blockwise(x, qw, sw)
    torch.cuda.synchronize()
    want, ab = ref.gemm(host(q), host(s), host(qt), host(st))
    got = y[:, -tail:].double().cpu().numpy()
    assert np.all(np.abs(got - want) <= ref.gemm_tolerance(want, ab, K))
    assert torch.all(y[:, :-tail] == 0)


def test_quantizers_past_32_bits():
    """Values more than 2^32 elements into the matrix, against the same rows alone."""
    K, tail = 4112, 256
    N = (1 << 20) + tail
    say("quantizers past 32 bits")
    x = torch.zeros((N, K), dtype=torch.bfloat16, device=DEV)
    x[-tail:] = synth.normal((tail, K), 1.0, "bf16", seed=79, device=DEV)
    for f, rows in ((fp8q.fp8_quantize_blocks, None), (fp8q.fp8_quantize_weight_blocks, 2)):
        q, s = f(x)
        qt, st = f(x[-tail:].contiguous())
        torch.cuda.synchronize()
        assert torch.equal(q[-tail:], qt)
        assert torch.equal(s[:, -tail:], st) if rows is None else torch.equal(s[-rows:], st)
        assert not q[:-tail].any()

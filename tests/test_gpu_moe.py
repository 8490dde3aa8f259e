"""GPU parity of fp8_moe_blockwise against the layer's definition in 64 bits.

- Selection: ids exactly, weights within a derived bound, over ties, experts switched off (-inf, NaN), fewer
  experts left than top_k, rows with none, +inf logits, both normalizations, 1 to 512 experts.
- Layer: within a derived bound (block_ref.moe) for one to 64 tokens, one expert taken by all
  tokens, widths that end inside a block, bf16 and fp16.
- Outputs are the same on every call, on another stream, in place and in a replayed graph, and
  nothing behind them is written.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
from fp8_quantized_gemm_amd import fp8q, synth
from gpu_helpers import DEV, host, say

pytestmark = pytest.mark.gpu


def _inputs(T, E, H, I, dtype="bf16", seed=0):
    x = synth.normal((T, H), 1.0, dtype, seed=synth.seed_for("mx", T, H, dtype, seed))
    w13 = synth.normal((E, 2, I, H), 0.05, "bf16", seed=synth.seed_for("m13", E, I, H), device=DEV)
    w2 = synth.normal((E, H, I), 0.05, "bf16", seed=synth.seed_for("m2", E, I, H), device=DEV)
    rng = np.random.Generator(np.random.PCG64(synth.seed_for("ml", T, E, seed)))
    logits = (rng.standard_normal((T, E)) * 1.5).astype(np.float32)
    return x, logits, *fp8q.fp8_quantize_weight_blocks(w13), *fp8q.fp8_quantize_weight_blocks(w2)


def _check(x, logits, w13, s13, w2, s2, top_k, renormalize):
    out = fp8q.fp8_moe_blockwise(x.to(DEV), torch.from_numpy(logits).to(DEV), w13, s13, w2, s2,
                                 top_k, renormalize)
    y, ids, weights = (t.float().cpu().numpy() if t.dtype != torch.int32 else host(t) for t in out)
    want, off, want_ids, want_w, off_w = ref.moe(x.double().numpy(), logits, host(w13), host(s13),
                                          host(w2), host(s2), top_k, renormalize)
    assert np.array_equal(ids, want_ids)
    assert np.all(np.abs(weights - want_w) <= off_w)
    bad = np.abs(y - want) - off
    assert np.all(bad <= 0), f"{(bad > 0).sum()} outside, worst by {bad.max()}"
    return out


@pytest.mark.parametrize("T,E,H,I,top_k,dtype,renormalize", [
    (1, 1, 16, 16, 1, "bf16", True),
    (1, 8, 256, 128, 2, "bf16", True),
    (1, 64, 2048, 256, 6, "fp16", True),
    (2, 5, 144, 272, 3, "fp16", False),
    (7, 16, 1040, 144, 4, "bf16", False),
    (8, 8, 128, 128, 8, "bf16", True),
    (9, 32, 272, 400, 2, "bf16", True),
    (17, 3, 512, 1040, 2, "bf16", False),
    (33, 130, 256, 16, 5, "fp16", True),
    (64, 16, 640, 144, 2, "bf16", True),
    (64, 512, 128, 32, 16, "bf16", False),
    (64, 1, 272, 144, 1, "fp16", True),
    (40, 300, 16, 256, 9, "bf16", True),
])
def test_layer_within_bound(T, E, H, I, top_k, dtype, renormalize):
    say("moe", T, E, H, I, top_k, dtype, renormalize)
    _check(*_inputs(T, E, H, I, dtype), top_k, renormalize)


# Enough (expert, columns) items for two row tiles each: few tokens an expert and many.
@pytest.mark.parametrize("T,E,H,I,top_k,dtype", [
    (20, 128, 144, 528, 8, "bf16"),
    (64, 128, 144, 528, 8, "fp16"),
    (64, 40, 272, 1680, 3, "bf16"),
])
def test_layer_with_many_items(T, E, H, I, top_k, dtype):
    say("moe many items", T, E, H, I, top_k, dtype)
    _check(*_inputs(T, E, H, I, dtype), top_k, True)


# Widths of the second kernel's two, three and four row tiles, with and without the rest of h,
# rows of W2 of whole and of partial lines, ends inside a tile.
@pytest.mark.parametrize("T,E,H,I,top_k,dtype", [
    (3, 4, 2064, 144, 2, "bf16"),
    (20, 6, 4096, 256, 3, "fp16"),
    (8, 4, 4112, 128, 2, "bf16"),
    (17, 5, 6128, 272, 2, "bf16"),
    (1, 300, 6160, 16, 4, "bf16"),
    (64, 3, 8176, 144, 2, "fp16"),
    (64, 260, 6160, 16, 2, "bf16"),
    (6, 2, 9232, 256, 1, "bf16"),
])
def test_layer_of_each_width(T, E, H, I, top_k, dtype):
    say("moe width", T, E, H, I, top_k, dtype)
    _check(*_inputs(T, E, H, I, dtype), top_k, True)


@pytest.mark.parametrize("renormalize", [True, False])
def test_masked_and_tied_logits(renormalize):
    T, E, H, I, top_k = 12, 70, 144, 144, 6
    x, logits, *w = _inputs(T, E, H, I)
    logits[0, :] = -np.inf                          # a token that no expert takes
    logits[1, 3:] = -np.inf                         # three experts left for six choices
    logits[2, :] = 0.25                             # all tied: the lowest indices
    logits[3, ::2] = -logits[3, ::2] * 0.0          # +0 and -0 tie too
    logits[3, 1::2] = 0.0
    logits[4, [5, 69]] = np.inf                     # two share the whole weight
    logits[5, 10] = np.nan
    logits[5, :10] = np.nan
    logits[6, :] = np.nan
    logits[7, :] = -np.inf
    logits[7, 64] = -3e38                           # one finite expert, the type's lowest range
    logits[8, :] = np.finfo(np.float32).min
    logits[9, :] = 3e38 * np.linspace(-1, 1, E).astype(np.float32)
    say("moe masked", renormalize)
    y, ids, weights = _check(x, logits, *w, top_k, renormalize)
    y, ids, weights = y.float().cpu(), ids.cpu(), weights.cpu()
    for t in (0, 6):
        assert torch.all(y[t] == 0) and torch.all(ids[t] == -1) and torch.all(weights[t] == 0)
    assert ids[2].tolist() == list(range(top_k))
    assert ids[4, :2].tolist() == [5, 69] and weights[4].tolist() == [0.5, 0.5, 0, 0, 0, 0]
    assert ids[7].tolist() == [64, -1, -1, -1, -1, -1] and weights[7, 0] == 1.0


def test_all_tokens_to_one_expert():
    """One expert's list is longer than a pass over its weights takes tokens."""
    T, E, H, I, top_k = 64, 6, 400, 272, 2
    x, logits, *w = _inputs(T, E, H, I)
    logits[:, 4] = 30.0
    say("moe one expert")
    _check(x, logits, *w, top_k, True)


def test_experts_that_no_token_chose_are_not_read():
    """NaN codes and scales of unused experts do not reach the result."""
    T, E, H, I, top_k = 5, 8, 256, 144, 2
    x, logits, w13, s13, w2, s2 = _inputs(T, E, H, I)
    logits[:, [1, 6]] = -np.inf
    for e in (1, 6):
        w13[e], w2[e] = 0x7F, 0x7F
        s13[e], s2[e] = float("nan"), float("nan")
    say("moe unused experts")
    y, _, _ = fp8q.fp8_moe_blockwise(x.to(DEV), torch.from_numpy(logits).to(DEV), w13, s13, w2, s2,
                                     top_k)
    assert torch.isfinite(y.float()).all()


@pytest.mark.parametrize("T,E,H,I,top_k", [(1, 64, 2048, 256, 6), (13, 32, 272, 400, 4),
                                           (64, 16, 640, 144, 2)])
def test_same_result_on_streams_in_graphs_and_in_place(T, E, H, I, top_k):
    x, logits, *w = _inputs(T, E, H, I)
    x, logits = x.to(DEV), torch.from_numpy(logits).to(DEV)
    want = [t.clone() for t in fp8q.fp8_moe_blockwise(x, logits, *w, top_k)]
    guard = torch.full((T * H + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    outs = [guard[:T * H].view(T, H), torch.empty_like(want[1]), torch.empty_like(want[2])]
    work = torch.full((fp8q.moe_work_bytes(T, I, top_k) + 64,), 0x5A, dtype=torch.uint8, device=DEV)

    def same():
        torch.cuda.synchronize()
        assert all(torch.equal(o, v) for o, v in zip(outs, want))
        assert torch.all(guard[T * H:] == 7.0)
        assert torch.all(work[-64:] == 0x5A)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    say("moe stream", T, E, H, I, top_k)
    with torch.cuda.stream(side):
        fp8q.fp8_moe_blockwise(x, logits, *w, top_k, True, *outs, work=work)
    same()
    g = torch.cuda.CUDAGraph()
    say("moe graph", T, E, H, I, top_k)
    with torch.cuda.graph(g):
        fp8q.fp8_moe_blockwise(x, logits, *w, top_k, True, *outs, work=work)
    for _ in range(3):
        for o in outs:
            o.view(torch.uint8).fill_(0x7f)
        work[:-64].fill_(0x7f)
        torch.cuda.synchronize()
        g.replay()
        same()
    # new logits in the graph's input: the choice is made again
    logits.copy_(logits.flip(1))
    again = [t.clone() for t in fp8q.fp8_moe_blockwise(x, logits, *w, top_k)]
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, v) for o, v in zip(outs, again))
    assert not torch.equal(again[1], want[1])
    del g
    fp8q.fp8_moe_blockwise(x, logits, *w, top_k, True, x)     # y over x
    torch.cuda.synchronize()
    assert torch.equal(x, again[0])


def test_block_path_of_a_layer():
    """The operators together, as a layer runs them: a projection with the linear, the same
    from its two parts, then the experts on its output."""
    T, E, H, I, top_k = 24, 12, 512, 272, 3
    x = synth.activation(T, H, seed=9, outliers=True, device=DEV)
    wo = synth.normal((H, H), 0.02, "bf16", seed=10, device=DEV)
    qo, so = fp8q.fp8_quantize_weight_blocks(wo)
    _, logits, *w = _inputs(T, E, H, I)
    say("block path")
    a, q, s = fp8q.fp8_linear_blockwise(x, qo, so)
    assert torch.equal(a, fp8q.fp8_gemm_blockwise(q, s, qo, so))
    want, ab = ref.gemm(host(q), host(s), host(qo), host(so))
    assert np.all(np.abs(a.double().cpu().numpy() - want) <= ref.gemm_tolerance(want, ab, H))
    _check(a.cpu(), logits, *w, top_k, True)


def test_refused_sizes():
    """Sizes outside the limits are refused as sizes, also where no buffer is passed."""
    say("moe refusals")
    for T, E, H, I, top_k in ((65, 4, 128, 128, 2), (2, 4, 128, 128, 5), (1, 20, 128, 128, 17),
                              (1, 513, 16, 16, 1), (1, 4, 24, 128, 2), (1, 4, 128, 24, 2)):
        nb = lambda n: (n + 127) // 128
        zeros = lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype, device=DEV)
        with pytest.raises(RuntimeError, match="size out of range"):
            fp8q.fp8_moe_blockwise(zeros(T, H, dtype=torch.bfloat16), zeros(T, E),
                                   zeros(E, 2, I, H, dtype=torch.uint8), zeros(E, 2, nb(I), nb(H)),
                                   zeros(E, H, I, dtype=torch.uint8), zeros(E, nb(H), nb(I)), top_k)


def test_two_calls_at_once():
    """Calls on two streams, each with a work buffer of its own."""
    T, E, H, I, top_k = 24, 32, 1024, 272, 4
    sides = [torch.cuda.Stream() for _ in range(2)]
    x, logits, *w = _inputs(T, E, H, I)
    x2, logits2, *_ = _inputs(T, E, H, I, seed=1)
    ins = [(x.to(DEV), torch.from_numpy(logits).to(DEV)), (x2.to(DEV), torch.from_numpy(logits2).to(DEV))]
    want = [[t.clone() for t in fp8q.fp8_moe_blockwise(*i, *w, top_k)] for i in ins]
    outs = [[torch.empty_like(t) for t in v] for v in want]
    works = [torch.empty(fp8q.moe_work_bytes(T, I, top_k), dtype=torch.uint8, device=DEV) for _ in ins]
    torch.cuda.synchronize()
    say("moe two streams")
    for _ in range(10):
        for side, i, o, k in zip(sides, ins, outs, works):
            with torch.cuda.stream(side):
                fp8q.fp8_moe_blockwise(*i, *w, top_k, True, *o, work=k)
    torch.cuda.synchronize()
    for o, v in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, v))


def test_weights_past_32_bits():
    """The last of 512 experts lies more than 2^32 bytes into its array."""
    E, H, I = 512, 4096, 1040
    assert (E - 1) * 2 * I * H > 1 << 32
    x, _, w13, s13, w2, s2 = _inputs(3, 1, H, I)
    say("moe past 32 bits")
    all13 = torch.zeros((E, 2, I, H), dtype=torch.uint8, device=DEV)
    all2 = torch.zeros((E, H, I), dtype=torch.uint8, device=DEV)
    sc13, sc2 = s13.repeat(E, 1, 1, 1), s2.repeat(E, 1, 1)
    all13[-1], all2[-1] = w13[0], w2[0]
    logits = torch.zeros((3, E), device=DEV)
    logits[:, -1] = 5.0
    y, ids, _ = fp8q.fp8_moe_blockwise(x.to(DEV), logits, all13, sc13, all2, sc2, 1)
    one, _, _ = fp8q.fp8_moe_blockwise(x.to(DEV), logits[:, -1:].contiguous(), w13, s13, w2, s2, 1)
    torch.cuda.synchronize()
    assert torch.all(ids == E - 1) and torch.equal(y, one) and torch.any(one != 0)


@pytest.mark.parametrize("T", [4, 8, 15, 40])
def test_infinite_and_nan_tokens_stay_in_their_row(T):
    E, H, I, top_k = 6, 272, 144, 2
    x, logits, *w = _inputs(T, E, H, I)
    x, logits = x.to(DEV), torch.from_numpy(logits).to(DEV)
    say("moe inf and nan", T)
    clean, _, _ = fp8q.fp8_moe_blockwise(x, logits, *w, top_k)
    x[1], x[2, 5] = float("nan"), float("inf")
    y, _, _ = fp8q.fp8_moe_blockwise(x, logits, *w, top_k)
    torch.cuda.synchronize()
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[1].float()).all() and not torch.isfinite(y[2].float()).any()

"""The paged cache as a model's attention layer uses it: an FP8 linear makes queries, keys and
values, their tokens are appended, the attention reads the cache and an FP8 linear takes its
output; prompts first, then single tokens, eagerly and as a replayed graph."""
import copy
import math

import pytest
import torch

import paged_ref as ref
from fp8_quantized_gemm_amd import fp8q
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

HEADS, KV_HEADS, DIM, PAGE, HIDDEN = 8, 2, 64, 32, 256


class Layer:
    """One layer's weights and cache, and a batch's arrays."""

    def __init__(self, prompts, steps, seed, room=0):
        g = torch.Generator().manual_seed(seed)
        weight = lambda n, k: fp8q.fp8_quantize_rows(                                  # noqa: E731
            (torch.randn(n, k, generator=g) / k ** 0.5).to(torch.bfloat16).to(DEV))[:2]
        self.wqkv = weight((HEADS + 2 * KV_HEADS) * DIM, HIDDEN)
        self.wo = weight(HIDDEN, HEADS * DIM)
        full = [n + steps for n in prompts]
        self.host = ref.Batch(prompts, full, KV_HEADS, DIM, PAGE, seed=seed)
        bt = self.host
        bt.table = torch.nn.functional.pad(bt.table, (0, -(-room // PAGE)), value=-1)
        bt.width = bt.table.shape[1]
        self.rope = ref.rope_table(bt.width * PAGE, DIM).to(DEV)
        self.cache = [t.to(DEV) for t in (bt.k, bt.v, bt.ks, bt.vs)]
        self.table = bt.table.to(DEV)
        self.gen = g
        self.batch(prompts, prompts)

    def batch(self, new, lens):
        bt = self.host
        bt.new, bt.lens, bt.tokens, bt.max_q = new, lens, sum(new), max(new)
        bt.q_start = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32)
        bt.kv_lens = torch.tensor(lens, dtype=torch.int32)
        self.q_start, self.kv_lens = bt.q_start.to(DEV), bt.kv_lens.to(DEV)

    def hidden(self):
        return torch.randn(self.host.tokens, HIDDEN, generator=self.gen).to(torch.bfloat16).to(DEV)

    def forward(self, x, work=None):
        qkv = fp8q.fp8_linear_rowwise(x, *self.wqkv)[0].view(x.shape[0], HEADS + 2 * KV_HEADS, DIM)
        made = qkv.clone()
        q, k, v = qkv.split([HEADS, KV_HEADS, KV_HEADS], dim=1)
        where = (*self.cache, self.table, self.q_start, self.kv_lens, self.host.max_q)
        fp8q.fp8_kv_append(k, v, *where, rope=self.rope, q=q, q_out=q)
        y, lse = fp8q.fp8_paged_attention(q, *where, work=work)
        out = fp8q.fp8_linear_rowwise(y.view(x.shape[0], HEADS * DIM), *self.wo)[0]
        return made, q, y, lse, out


def check(layer, got):
    """The codes and scales bit for bit, the queries to half a step, y and lse to their bounds."""
    bt, (made, q, y, lse, out) = layer.host, [t.cpu() for t in got]
    mq, mk, mv = made.split([HEADS, KV_HEADS, KV_HEADS], dim=1)
    qo = ref.append(bt, mk, mv, layer.rope.cpu(), False, mq)
    for want, have in zip((bt.k, bt.v, bt.ks, bt.vs), layer.cache):
        assert torch.equal(have.cpu().view(torch.uint8), want.view(torch.uint8))
    assert torch.all((q.double() - qo).abs() <= qo.abs() * ref.EPS[torch.bfloat16] + ref.TINY[torch.bfloat16])
    wy, wl, ty, tl = ref.attend(bt, q, DIM ** -0.5)
    assert torch.all((y.double() - wy).abs() <= ty) and torch.all((lse.double() - wl).abs() <= tl)
    # the products are fp32's of exact codes; the last rounding is to bf16
    codes, sa, _ = fp8q.fp8_quantize_rows(y.view(bt.tokens, -1).to(DEV))
    a = ref.TABLE[codes.cpu().long()] * sa.cpu().double()[:, None]
    w = ref.TABLE[layer.wo[0].cpu().long()] * layer.wo[1].cpu().double()[:, None]
    bound = (a.abs() @ w.abs().T) * (HEADS * DIM + 4) * 2.0 ** -24 + (a @ w.T).abs() * 2.0 ** -8
    assert torch.all((out.double() - a @ w.T).abs() <= bound)


@pytest.mark.parametrize("room", [0, 2500])
def test_prompts_then_single_tokens(room):
    prompts, steps = [37, 1, 90, 64], 4
    layer = Layer(prompts, steps, seed=40, room=room)
    say("prompts", room)
    check(layer, layer.forward(layer.hidden()))
    for i in range(1, steps + 1):
        layer.batch([1] * 4, [n + i for n in prompts])
        say("step", room, i)
        check(layer, layer.forward(layer.hidden()))


def test_prompts_in_chunks_are_prompts():
    """A prompt of 90 tokens appended at once, and in chunks whose ends lie inside pages: the cache
    holds the same up to the scales' growth, so both are checked against their own host form."""
    layer = Layer([90, 33], 0, seed=41)
    done = [0, 0]
    for take in ([50, 1], [7, 30], [33, 2]):
        done = [d + t for d, t in zip(done, take)]
        layer.batch(take, done)
        say("chunk", take)
        check(layer, layer.forward(layer.hidden()))


@pytest.mark.parametrize("room", [0, 2500])
def test_two_captured_layers(room):
    """A decode step of two layers, each with its scratch, captured as one graph and replayed as
    the sequences grow: every replay gives what eager calls on another stream give."""
    prompts, steps = [30, 5, 64, 12, 200], 5
    layers = [Layer(prompts, steps + 1, seed=s, room=room) for s in (42, 43)]
    for layer in layers:
        check(layer, layer.forward(layer.hidden()))
        layer.batch([1] * 5, [n + 1 for n in prompts])
    twins = [copy.copy(layer) for layer in layers]
    for t in twins:
        t.cache = [c.clone() for c in t.cache]
        t.kv_lens = t.kv_lens.clone()
    x = torch.zeros((5, HIDDEN), dtype=torch.bfloat16, device=DEV)
    work = [fp8q.paged_attention_work(torch.empty((5, HEADS, DIM), device=DEV), layer.cache[0], layer.table, 1)
            for layer in layers]
    side = torch.cuda.Stream()

    def step(which, scratch):
        h, out = x, []
        for layer, w in zip(which, scratch):
            out.append(layer.forward(h, w))
            h = out[-1][-1] + h
        return out

    say("warm up", room)
    kept = [[c.clone() for c in layer.cache] for layer in layers]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(layers, work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(layers, work)
    torch.cuda.synchronize()
    for layer, was in zip(layers, kept):
        for c, w in zip(layer.cache, was):
            c.copy_(w)
    for i in range(steps):
        x.copy_(torch.randn(x.shape, generator=layers[0].gen).to(torch.bfloat16))
        torch.cuda.synchronize()
        say("replay", room, i)
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            eager = step(twins, [None, None])
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert all(torch.equal(s, t) for s, t in zip(a, b))
            assert torch.isfinite(a[3]).all() and not math.isnan(float(a[4].float().sum()))
        for layer, twin in zip(layers, twins):
            assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(layer.cache, twin.cache))
            layer.kv_lens += 1
            twin.kv_lens += 1

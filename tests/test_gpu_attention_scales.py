"""fp8_paged_attention where the scales of a row's pages, or the softmax scale, lie at the ends of
their ranges, in each of its kernels: y and lse against the host form in 64 bits, within the bounds
that follow from the roundings (see paged_ref.attend)."""
import math

import pytest
import torch

import paged_ref as ref
from fp8_quantized_gemm_amd import fp8q
from gpu_helpers import DEV, say
from test_gpu_attention import call, compare, on_gpu, spoil_unused

pytestmark = pytest.mark.gpu

# New tokens, tokens and the page table's room in tokens (0: no more than needed), four query heads:
# a sequence whole in a workgroup, of one tile and of several; 20 rows on the tile kernel, uncut; the
# keys cut into parts, for few rows and for many.
KERNELS = {"one tile": (1, 60, 0), "whole": (1, 330, 0), "tiles": (5, 230, 0), "parts of few rows": (2, 700, 20000),
           "parts of many rows": (9, 900, 0)}


def attend(bt, q, room, scale, **more):
    d = on_gpu(bt)
    d["table"] = torch.nn.functional.pad(bt.table, (0, max(0, -(-room // bt.page) - bt.width)), value=-1).to(DEV)
    got = call(d, q.to(DEV), bt.max_q, scale=scale, **more)
    torch.cuda.synchronize()
    return got


def batch(kernel, page, kv_heads=1, dim=64, seed=30):
    new, length, room = KERNELS[kernel]
    bt = ref.Batch([new, 1], [length, 3], kv_heads, dim, page, seed=seed)
    spoil_unused(bt)
    return bt, room


def set_values_scales(bt, scales):
    """Page j of the first sequence gets the j-th of `scales`, in turn."""
    for j in range(-(-bt.lens[0] // bt.page)):
        bt.vs[int(bt.table[0, j])] = scales[j % len(scales)]


# The lowest page's keys count as much as the highest's in the denominator, the later half of them or
# the first; (2^-36, 2^36) and (2^-37, 2^37) are the two sides of what the kernels tell apart.
PAIRS = [(2.0 ** -100, 2.0 ** 30), (2.0 ** -100, 2.0 ** 100), (2.0 ** -36, 2.0 ** 36), (2.0 ** -37, 2.0 ** 37),
         (1.37 * 2.0 ** -36, 1.73 * 2.0 ** 34), (0.0, math.inf), (2.0 ** -100, 2.0 ** -10), (2.0 ** 10, 2.0 ** 100)]


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("kernel", list(KERNELS))
def test_every_key_counts_in_the_denominator(kernel, page):
    if kernel == "one tile":
        page = 16
    for low, high in PAIRS:
        for scales in ([low, high], [high, low], [high, low, low, low], [1.0, low, high]):
            say("scales", kernel, page, scales)
            bt, room = batch(kernel, page)
            set_values_scales(bt, scales)
            q = bt.values(4, torch.bfloat16)
            want = ref.attend(bt, q, 0.125)
            compare(bt, q, attend(bt, q, room, 0.125), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(4, 2, 128, 128), (8, 2, 192, 32), (4, 1, 256, 64), (12, 3, 96, 16)])
@pytest.mark.parametrize("kernel", list(KERNELS))
def test_scales_of_any_size(kernel, heads, kv_heads, dim, page, dtype):
    """Pages of any scales, from page to page and head to head; masks and windows on them."""
    bt, room = batch(kernel, page, kv_heads, dim, seed=31)
    bt.vs.copy_(torch.exp2(torch.randint(-100, 101, bt.vs.shape, generator=bt.gen).float()))
    bt.ks.mul_(1 + torch.rand(bt.ks.shape, generator=bt.gen))
    q = bt.values(heads, dtype)
    for causal, window in ((True, 0), (False, 0), (True, 100)):
        say("any scales", kernel, heads, kv_heads, dim, page, dtype, causal, window)
        want = ref.attend(bt, q, 0.1, causal, window)
        got = attend(bt, q, room, 0.1, causal=causal, window=window)
        # before its last rounding y lies within the bound of the 64-bit value, so where that is nearer
        # than the bound to the type's largest number y may be infinite, and is not below that value
        # less the bound
        y, largest = got[0].cpu().double(), torch.finfo(dtype).max
        least, most = want[0].abs() - want[2], want[0].abs() + want[2]
        big = most > largest
        assert torch.all(y.abs()[big] >= least[big].clamp(max=largest) * (1 - ref.EPS[dtype]))
        compare(bt, q, (torch.where(big, 0, y), got[1]), (torch.where(big, 0, want[0]), *want[1:]))


@pytest.mark.parametrize("kernel", list(KERNELS))
def test_large_logits_on_scales_far_apart(kernel):
    """Logits of some hundreds: which keys count is another set for y and for the denominator."""
    for scales in ([2.0 ** -100, 2.0 ** 100], [2.0 ** 60, 2.0 ** -60, 1.0], [2.0 ** -36, 2.0 ** 36]):
        bt, room = batch(kernel, 16, seed=32)
        set_values_scales(bt, scales)
        q = bt.values(4, torch.bfloat16, spread=20.0)
        say("large logits", kernel, scales)
        want = ref.attend(bt, q, 0.125)
        compare(bt, q, attend(bt, q, room, 0.125), want)


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("scales", [[0.0, -2.0, math.nan, 1e-38, 2.0 ** -100, 2.0 ** -99], [math.inf, 1.0, 3e38]])
def test_scales_that_are_none(kernel, scales):
    bt, room = batch(kernel, 16, seed=33)
    set_values_scales(bt, scales)
    for j in range(-(-bt.lens[0] // bt.page)):
        if j % 3 == 0:
            bt.ks[int(bt.table[0, j])] = scales[j % 2]
    q = bt.values(4, torch.bfloat16, spread=2.0 ** -120)
    say("odd scales", kernel, scales)
    want = ref.attend(bt, q, 0.125)
    compare(bt, q, attend(bt, q, room, 0.125), want)


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -36, 2.0 ** 36, 2.0 ** 100])
@pytest.mark.parametrize("seqs,new", [(520, 1), (300, 5)])
def test_many_keys_above_the_first(seqs, new, scale):
    """Thousands of keys whose logits lie a little above those that a wave begins with, on pages of the
    smallest and largest scales: sums of terms over the smallest scale stay finite."""
    length = 160 * 64
    bt = ref.Batch([new] + [0] * (seqs - 1), [length] + [0] * (seqs - 1), 1, 16, 64, seed=34)
    spoil_unused(bt)
    bt.k.zero_()
    bt.k[:, :, :, 0] = 0x38                                   # 1.0
    run = 20 if new == 1 else 160                             # tiles of a wave
    for j in range(0, 160, run):
        bt.k[int(bt.table[0, j]), :, :, 0] = 0
    bt.ks.fill_(1.0)
    bt.vs.fill_(scale)
    q = torch.zeros(bt.tokens, 4, 16, dtype=torch.bfloat16)
    q[:, :, 0] = 4.0625                                       # 5.86 in powers of two
    say("many keys", seqs, new, scale)
    want = ref.attend(bt, q, 1.0)
    compare(bt, q, attend(bt, q, 0, 1.0), want)


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("k_scale,scale", [(2.0 ** 100, 2.0 ** 30), (2.0 ** 100, -2.0 ** 127), (1.0, 2.0 ** 127),
                                           (math.inf, 2.0 ** 28)])
def test_logits_of_zero_under_large_scales(kernel, k_scale, scale):
    """A product of scales beyond fp32 counts as its largest number: a query or a key of zeros has
    logits of zero all the same."""
    bt, room = batch(kernel, 64 if kernel != "one tile" else 16, seed=35)
    bt.ks.fill_(k_scale)
    q = bt.values(4, torch.bfloat16)
    zero = torch.zeros_like(q)
    say("zero queries", kernel, k_scale, scale)
    compare(bt, zero, attend(bt, zero, room, scale), ref.attend(bt, zero, scale))
    bt.k.zero_()
    spoil_unused(bt)
    say("zero keys", kernel, k_scale, scale)
    compare(bt, q, attend(bt, q, room, scale), ref.attend(bt, q, scale))


@pytest.mark.parametrize("new,lens,room", [([1] * 3, [300, 64, 900], 0), ([1] * 3, [300, 64, 900], 20000),
                                           ([40, 1, 3], [400, 90, 64], 0)])
def test_graph_replays_as_scales_grow(new, lens, room):
    """Captured once, replayed while pages' scales move from near each other to far apart and back."""
    bt = ref.Batch(new, lens, 2, 64, 64, seed=36, width=max(-(-room // 64), -(-max(lens) // 64)))
    d = on_gpu(bt)
    q = bt.values(4, torch.bfloat16).to(DEV)
    y, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
    work = fp8q.paged_attention_work(q, d["k"], d["table"], bt.max_q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(d, q, bt.max_q, scale=0.1, y=y, lse=lse, work=work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(d, q, bt.max_q, scale=0.1, y=y, lse=lse, work=work)
    for spread in (2, 100, 30, 100, 0):
        bt.vs.copy_(torch.exp2(torch.randint(-spread, spread + 1, bt.vs.shape, generator=bt.gen).float()))
        d["vs"].copy_(bt.vs)
        want = ref.attend(bt, q.cpu(), 0.1)
        work.fill_(0xFF)
        y.fill_(3.0)
        torch.cuda.synchronize()
        say("replay", room, spread)
        graph.replay()
        torch.cuda.synchronize()
        compare(bt, q, (y, lse), want)
        again = call(d, q, bt.max_q, scale=0.1)
        torch.cuda.synchronize()
        assert torch.equal(y, again[0]) and torch.equal(lse, again[1])

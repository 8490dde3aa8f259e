"""fp8_kv_append against the host form in 64 bits: codes and scales bit for bit (every step before
the E4M3 rounding is defined in fp32), rotated queries to half a step of their type; slots, pages
and rows that gain nothing stay as they were."""
import copy
import math

import pytest
import torch

import paged_ref as ref
from fp8_quantized_gemm_amd import fp8q
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu


def on_gpu(bt):
    return {n: getattr(bt, n).to(DEV) for n in ("k", "v", "ks", "vs", "table", "q_start", "kv_lens")}


def call(d, k, v, max_q, rope=None, **more):
    return fp8q.fp8_kv_append(k, v, d["k"], d["v"], d["ks"], d["vs"], d["table"], d["q_start"],
                              d["kv_lens"], max_q, rope=rope, **more)


def same_bits(got, want):
    return torch.equal(got.cpu().contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))


def check(bt, d, want):
    torch.cuda.synchronize()
    for name in ("ks", "vs", "k", "v"):
        got = d[name].cpu()
        assert same_bits(got, getattr(want, name)), name


CASES = [
    # new, lens, kv heads, dim, page
    ([1], [1], 1, 16, 16),
    ([1, 1, 1, 1], [64, 65, 1, 130], 8, 128, 64),       # full page, fresh page, first token
    ([1, 1, 0, 1], [17, 0, 33, 128], 3, 96, 32),        # idle slots: no token, no position
    ([200], [200], 2, 128, 64),
    ([130, 1, 0, 77, 16], [300, 17, 5, 77, 32], 4, 64, 16),
    ([129, 64], [140, 128], 1, 256, 128),               # the largest tile
    ([3, 2], [3, 1], 2, 80, 16),                        # more new tokens than the sequence holds
    ([70], [500], 5, 112, 64),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new,lens,kv_heads,dim,page", CASES)
def test_codes_scales_and_queries(new, lens, kv_heads, dim, page, dtype):
    say("append", new, lens, kv_heads, dim, page, dtype)
    for rot, inter in ((dim, False), (16, True), (0, False)):
        bt = ref.Batch(new, lens, kv_heads, dim, page, seed=5, lead=2, tail=3)
        rope = ref.rope_table(bt.width * page, rot, seed=0.25)
        k = bt.values(kv_heads, dtype) * torch.where(torch.rand(dim) < 0.05, 40.0, 1.0).to(dtype)
        v, q = bt.values(kv_heads, dtype), bt.values(2 * kv_heads + 1, dtype)
        d, want = on_gpu(bt), copy.deepcopy(bt)
        qo = ref.append(want, k, v, rope, inter, q)
        out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
        got = call(d, k.to(DEV), v.to(DEV), bt.max_q, rope.to(DEV), interleaved=inter, q=q.to(DEV),
                   q_out=out)
        check(bt, d, want)
        got = got.cpu()
        inside = ~torch.isnan(qo)
        assert torch.all(got[~inside] == 7.0)            # rows outside the batch are left alone
        bound = qo.abs() * ref.EPS[dtype] + ref.TINY[dtype]
        assert torch.all((got.double() - qo).abs()[inside] <= bound[inside])


def test_page_filled_one_token_at_a_time():
    """Scales grow with the page and older codes with them; 70 calls, each checked."""
    bt = ref.Batch([1, 1], [1, 1], 2, 32, 64, seed=9, width=2)
    bt.table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    bt.pages = bt.k.shape[0]
    assert bt.pages >= 4
    d, want = on_gpu(bt), copy.deepcopy(bt)
    d["table"] = bt.table.to(DEV)
    say("append token by token")
    for step in range(1, 71):
        lens = [step, 2 * step - 1 if step < 60 else step]
        size = 2.0 ** ((step * 7) % 23 - 11)             # scales jump up and down
        k = (torch.randn(2, 2, 32, generator=bt.gen) * size).to(torch.bfloat16)
        v = (torch.randn(2, 2, 32, generator=bt.gen) / size).to(torch.bfloat16)
        want.lens = lens
        d["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        ref.append(want, k, v)
        call(d, k.to(DEV), v.to(DEV), 1)
        check(bt, d, want)


def test_scales_of_any_kind_are_kept_or_grown():
    """A page whose scale is no power of two, 0, NaN, infinite or negative."""
    scales = [3.0e-3, 0.7, 1e9, 0.0, math.nan, math.inf, -1.0, 1e-38]
    for page, older in ((16, 5), (64, 17)):
        bt = ref.Batch([2] * len(scales), [older + 2] * len(scales), 1, 48, page, seed=4)
        for b, s in enumerate(scales):
            bt.ks[bt.table[b, older // page]] = s
            bt.vs[bt.table[b, older // page]] = s
        k, v = bt.values(1, torch.float16), bt.values(1, torch.float16)
        d, want = on_gpu(bt), copy.deepcopy(bt)
        ref.append(want, k, v)
        say("append onto odd scales", page)
        call(d, k.to(DEV), v.to(DEV), 2)
        check(bt, d, want)


def test_zero_huge_infinite_and_nan_values():
    bt = ref.Batch([4, 4, 4, 2, 1], [4, 4, 4, 20, 1], 2, 32, 16, seed=6)
    k, v = bt.values(2, torch.bfloat16), bt.values(2, torch.bfloat16)
    k[0:4], v[0:4] = 0.0, -0.0                           # a page of zeros
    k[4:8] = 3.0e38                                      # beyond 448 * 2^100: saturates
    v[4, 0, 3], v[5, 1, 4] = math.inf, -math.inf         # their neighbours keep their scale
    k[8, 0, 0], v[9, 1, 5] = math.nan, math.nan
    k[14] = 1e-38                                        # below the smallest scale's steps
    d, want = on_gpu(bt), copy.deepcopy(bt)
    ref.append(want, k, v)
    say("append special values")
    call(d, k.to(DEV), v.to(DEV), 4)
    torch.cuda.synchronize()
    for name in ("ks", "vs"):
        assert same_bits(d[name], getattr(want, name))
    for name in ("k", "v"):
        got, exp = d[name].cpu(), getattr(want, name)
        nan = torch.isnan(ref.TABLE[exp.long()])
        assert torch.equal(torch.isnan(ref.TABLE[got.long()]), nan)       # of either sign
        assert torch.equal(got[~nan], exp[~nan])


def test_tokens_without_a_page_are_dropped():
    bt = ref.Batch([40, 3], [40, 3], 2, 64, 16, seed=8)
    bt.table[0, 1] = -1
    bt.table[1, 0] = bt.pages                            # ids past the pool
    k, v = bt.values(2, torch.bfloat16), bt.values(2, torch.bfloat16)
    q = bt.values(2, torch.bfloat16)
    d, want = on_gpu(bt), copy.deepcopy(bt)
    qo = ref.append(want, k, v, q=q)
    say("append without pages")
    got = call(d, k.to(DEV), v.to(DEV), 40, q=q.to(DEV))
    check(bt, d, want)
    assert torch.equal(got.cpu().double(), qo)           # the queries have positions all the same


@pytest.mark.parametrize("lens,starts", [([10 ** 9], [0, 4]), ([-5], [0, 4]), ([50], [-3, 10 ** 9]),
                                         ([50], [4, 0]), ([50], [3, 3])])
def test_arrays_out_of_bounds_stay_inside(lens, starts):
    """Values in the arrays that no batch has: nothing outside the batch's pages changes."""
    bt = ref.Batch([4], [60], 1, 32, 16, seed=2)
    k, v = bt.values(1, torch.bfloat16), bt.values(1, torch.bfloat16)
    d = on_gpu(bt)
    d["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    d["q_start"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    say("append", lens, starts)
    call(d, k.to(DEV), v.to(DEV), 4)
    torch.cuda.synchronize()
    others = [p for p in range(bt.pages) if p not in bt.table[0].tolist()]
    assert torch.equal(d["k"].cpu()[others], bt.k[others]) and torch.equal(d["v"].cpu()[others], bt.v[others])


def test_slices_of_one_projection_and_queries_in_place():
    bt = ref.Batch([33, 9], [33, 60], 2, 64, 16, seed=12)
    heads = 6
    qkv = torch.randn(bt.tokens, heads + 4, 64, generator=bt.gen).to(torch.bfloat16)
    rope = ref.rope_table(bt.width * 16, 64)
    d, want = on_gpu(bt), copy.deepcopy(bt)
    g = qkv.to(DEV)
    q, k, v = g[:, :heads], g[:, heads:heads + 2], g[:, heads + 2:]
    qo = ref.append(want, qkv[:, heads:heads + 2], qkv[:, heads + 2:], rope, False, qkv[:, :heads])
    say("append in place")
    got = call(d, k, v, 33, rope.to(DEV), q=q, q_out=q)
    assert got.data_ptr() == g.data_ptr()
    check(bt, d, want)
    assert torch.all((q.cpu().double() - qo).abs() <= qo.abs() * ref.EPS[torch.bfloat16])
    assert torch.equal(g[:, heads:].cpu(), qkv[:, heads:])


def test_pages_past_32_bits():
    """The pool is 4.3 GB for keys and as much for values; the batch's pages are its last ones."""
    pages, heads, dim, page = 66000, 8, 128, 64
    bt = ref.Batch([70], [90], heads, dim, page, seed=21)
    k, v = bt.values(heads, torch.bfloat16), bt.values(heads, torch.bfloat16)
    want = copy.deepcopy(bt)
    ref.append(want, k, v)
    d = on_gpu(bt)
    say("append past 4 GB")
    big = {n: torch.zeros((pages, *d[n].shape[1:]), dtype=d[n].dtype, device=DEV) for n in ("k", "v", "ks", "vs")}
    for n in big:
        big[n][-bt.pages:] = d[n]
    big["table"] = d["table"] + (pages - bt.pages)
    big["table"][d["table"] < 0] = -1
    big["q_start"], big["kv_lens"] = d["q_start"], d["kv_lens"]
    call(big, k.to(DEV), v.to(DEV), 70)
    check(bt, {n: big[n][-bt.pages:] for n in ("k", "v", "ks", "vs")}, want)
    for n in ("k", "v"):
        assert int(big[n][:-bt.pages].max()) == 0
        assert bool((big[n][:-bt.pages].amax(dim=(1, 2, 3)) == 0).all())


def test_graph_replays_and_another_stream():
    """A captured decode step replayed as the lengths advance, and the same steps called eagerly on
    another stream: both as the host form has them."""
    bt = ref.Batch([1] * 5, [60] * 5, 4, 128, 16, seed=31)      # pages for 60 tokens each
    bt.lens = [14 + 3 * b for b in range(5)]
    bt.kv_lens = torch.tensor(bt.lens, dtype=torch.int32)
    rope = ref.rope_table(bt.width * 16, 128).to(DEV)
    shape = (5, 4, 128)
    k, v = (torch.zeros(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = torch.zeros((5, 8, 128), dtype=torch.bfloat16, device=DEV)
    q_out = torch.zeros_like(q)
    first, second, want = on_gpu(bt), on_gpu(bt), copy.deepcopy(bt)

    def step(d):
        call(d, k, v, 1, rope, q=q, q_out=q_out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(first)                                      # lengths as they are: repeated below
    torch.cuda.synchronize()
    for n in ("k", "v", "ks", "vs"):
        first[n].copy_(second[n])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(first)
    for i in range(6):
        say("append replay", i)
        new = [torch.randn(t.shape, generator=bt.gen).to(torch.bfloat16) * 2.0 ** i for t in (k, v, q)]
        for t, x in zip((k, v, q), new):
            t.copy_(x)
        ref.append(want, new[0], new[1], rope.cpu(), False, new[2])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(bt, first, want)
        with torch.cuda.stream(side):
            step(second)
        torch.cuda.synchronize()
        check(bt, second, want)
        want.lens = [x + 1 for x in want.lens]
        first["kv_lens"] += 1
        second["kv_lens"] += 1

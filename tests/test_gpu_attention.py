"""fp8_paged_attention against the host form in 64 bits, within the bounds that follow from its
roundings (see paged_ref.attend): head layouts, page sizes, lengths from none to long ones, masks
that leave rows empty, and what unused slots and masked tokens may hold."""
import math

import pytest
import torch

import paged_ref as ref
from fp8_quantized_gemm_amd import fp8q
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu


def on_gpu(bt):
    return {n: getattr(bt, n).to(DEV) for n in ("k", "v", "ks", "vs", "table", "q_start", "kv_lens")}


def call(d, q, max_q, **more):
    return fp8q.fp8_paged_attention(q, d["k"], d["v"], d["ks"], d["vs"], d["table"], d["q_start"],
                                    d["kv_lens"], max_q, **more)


def spoil_unused(bt):
    """Codes of NaN in every slot that holds no token of a sequence."""
    used = torch.zeros(bt.pages, bt.page, dtype=torch.bool)
    for b, _, _, length in bt.seqs():
        for t in range(length):
            pid = int(bt.table[b, t // bt.page])
            if 0 <= pid < bt.pages:
                used[pid, t % bt.page] = True
    free = ~used
    bt.k.transpose(1, 2)[free] = 0x7F
    bt.v.permute(0, 3, 1, 2)[free] = 0xFF


def compare(bt, q, got, want, rows=slice(None)):
    y, lse = (t.detach().cpu().double()[rows] for t in got)
    wy, wl, ty, tl = (t[rows] for t in want)
    inside = ~torch.isnan(wl)
    empty = inside & (wl == -math.inf)
    assert torch.equal(lse[inside] == -math.inf, empty[inside])
    assert torch.all(y[empty] == 0)
    full = inside & ~empty
    err = (lse - wl).abs()[full]
    assert torch.all(err <= tl[full]), f"lse off by {float((err / tl[full]).max())} bounds"
    err = (y - wy).abs()[full]
    assert torch.all(err <= ty[full]), f"y off by {float((err / ty[full]).max())} bounds"


def run(bt, heads, dtype, causal=True, window=0, spread=1.0, spoil=True):
    if spoil:
        spoil_unused(bt)
    q = bt.values(heads, dtype, spread)
    scale = bt.dim ** -0.5
    want = ref.attend(bt, q, scale, causal, window)
    d = on_gpu(bt)
    # a narrow page table, and one that has room for more keys than a workgroup takes by itself
    for room in (0, 20000):
        d["table"] = torch.nn.functional.pad(bt.table, (0, -(-room // bt.page)), value=-1).to(DEV)
        y = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
        lse = torch.full(q.shape[:2], 7.0, device=DEV)
        got = call(d, q.to(DEV), bt.max_q, scale=scale, causal=causal, window=window, y=y, lse=lse)
        torch.cuda.synchronize()
        compare(bt, q, got, want)
        outside = torch.isnan(want[1])
        assert torch.all(y.cpu()[outside] == 7.0) and torch.all(lse.cpu()[outside] == 7.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [
    (1, 1, 16, 16), (8, 8, 64, 64), (64, 8, 128, 64), (28, 4, 64, 16), (7, 1, 80, 32), (12, 3, 96, 16),
    (20, 1, 112, 128), (6, 2, 160, 64), (5, 5, 192, 32), (16, 1, 256, 16), (34, 2, 256, 128)])
def test_single_tokens(heads, kv_heads, dim, page, dtype):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 0, 130, 257]
    say("decode", heads, kv_heads, dim, page, dtype)
    bt = ref.Batch([1] * len(lens), lens, kv_heads, dim, page, seed=3, lead=1, tail=2)
    run(bt, heads, dtype)


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 20), (True, 64), (True, 1000)])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(6, 2, 64, 16), (8, 1, 128, 64), (3, 3, 32, 32),
                                                     (4, 4, 96, 128), (9, 1, 256, 64), (4, 2, 176, 16)])
def test_several_tokens(heads, kv_heads, dim, page, causal, window):
    say("several", heads, kv_heads, dim, page, causal, window)
    # the third sequence has more new tokens than it holds: its first rows see nothing
    bt = ref.Batch([5, 1, 4, 0, 17, 9], [5, 100, 2, 40, 150, 64], kv_heads, dim, page, seed=4, lead=1, tail=1)
    run(bt, heads, torch.bfloat16, causal, window)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,kv_heads,dim,page,causal,window", [
    (4, 2, 128, 64, True, 0), (2, 2, 64, 16, True, 0), (3, 1, 128, 128, False, 0), (2, 1, 96, 32, True, 50),
    (5, 1, 256, 64, True, 0), (2, 1, 192, 16, True, 100), (8, 1, 64, 64, True, 0)])
def test_prompts(heads, kv_heads, dim, page, causal, window, dtype):
    say("prompt", heads, kv_heads, dim, page, causal, window, dtype)
    bt = ref.Batch([130, 0, 65, 200, 3], [130, 10, 300, 199, 70], kv_heads, dim, page, seed=5, lead=3, tail=2)
    run(bt, heads, dtype, causal, window)


@pytest.mark.parametrize("heads,kv_heads,new,length", [(8, 1, 1, 9001), (2, 2, 1, 4500), (4, 1, 3, 5003),
                                                        (4, 1, 33, 4700), (2, 2, 40, 9000)])
def test_long_contexts(heads, kv_heads, new, length):
    say("long", heads, kv_heads, new, length)
    bt = ref.Batch([new, 1, new], [length, 3, 70], kv_heads, 64, 64, seed=6)
    run(bt, heads, torch.bfloat16, spread=3.0)


def test_many_sequences():
    """More sequences than a workgroup has threads, most of them short or idle."""
    lens = [(b * 37) % 91 for b in range(700)]
    say("many sequences")
    bt = ref.Batch([1] * 700, lens, 1, 32, 16, seed=7)
    run(bt, 2, torch.float16)


@pytest.mark.parametrize("kv_heads,dim,page", [(1, 32, 16), (2, 128, 64), (1, 256, 32)])
def test_many_short_sequences(kv_heads, dim, page):
    """So many that a workgroup of one wave has a sequence and head whole."""
    lens = [(b * 29) % 62 for b in range(520)]
    say("many short sequences", kv_heads, dim, page)
    bt = ref.Batch([1] * 520, lens, kv_heads, dim, page, seed=26)
    run(bt, kv_heads * 2, torch.bfloat16)


@pytest.mark.parametrize("heads,kv_heads,page", [(8, 1, 16), (4, 4, 64), (6, 2, 128)])
def test_many_sequences_of_several_tokens(heads, kv_heads, page):
    """More sequences than a wave has lanes, of which some bring many rows and some are long."""
    new = [1 + (b * 5) % 7 if b % 9 else 0 for b in range(90)]
    lens = [n + (b * 53) % 80 for b, n in enumerate(new)]
    new[30], lens[30], lens[60] = 40, 700, 1300
    say("many sequences of several tokens", heads, kv_heads, page)
    bt = ref.Batch(new, lens, kv_heads, 32, page, seed=22, lead=2, tail=1)
    run(bt, heads, torch.bfloat16)


@pytest.mark.parametrize("seqs,kv_heads,page,length,group", [
    (70, 4, 16, 2500, 1), (33, 8, 64, 5000, 1), (70, 4, 128, 4500, 1), (1, 512, 16, 10000, 1),
    (260, 2, 64, 40000, 1), (70, 4, 16, 2500, 17), (33, 8, 64, 5000, 17)])
def test_long_among_many_units(seqs, kv_heads, page, length, group):
    """A wave goes through more key tiles than it looks pages up for at once."""
    lens = [length] + [1 + b % 40 for b in range(1, seqs)]
    say("long among many", seqs, kv_heads, page, length, group)
    bt = ref.Batch([1] * seqs, lens, kv_heads, 16, page, seed=23)
    run(bt, kv_heads * group, torch.float16)


@pytest.mark.parametrize("page,window", [(16, 1000), (64, 1), (128, 2100)])
def test_windows_in_long_contexts(page, window):
    say("window", page, window)
    bt = ref.Batch([1, 3, 0, 20], [5000, 3001, 900, 2203], 2, 64, page, seed=24)
    run(bt, 4, torch.bfloat16, window=window)


@pytest.mark.parametrize("seed", range(6))
def test_mixtures(seed):
    """Batches of any mixture of new tokens, lengths, layouts and masks."""
    g = torch.Generator().manual_seed(100 + seed)
    pick = lambda *xs: xs[int(torch.randint(len(xs), (1,), generator=g))]              # noqa: E731
    most, longest = pick(1, 3, 90), pick(60, 900, 3500)
    new = torch.randint(0, most + 1, (pick(3, 20),), generator=g).tolist()
    lens = [n + int(torch.randint(longest, (1,), generator=g)) for n in new]
    kv_heads, group = pick(1, 2, 3), pick(1, 3, 8)
    dim, page, dtype = pick(48, 64, 128, 224), pick(16, 32, 64, 128), pick(torch.bfloat16, torch.float16)
    causal, window = pick((True, 0), (True, 300), (False, 0))
    say("mixture", seed, most, longest, len(new), kv_heads, group, dim, page, dtype, causal, window)
    if sum(new) * group * kv_heads > 600:
        new, lens = new[:3], lens[:3]
    bt = ref.Batch(new or [1], lens or [1], kv_heads, dim, page, seed=seed, lead=1, tail=3)
    run(bt, group * kv_heads, dtype, causal, window)


def test_scales_far_apart():
    """Pages whose values' scales differ by 2^80, and scales that are no powers of two: every page
    keeps its bits where it is the one that counts."""
    bt = ref.Batch([1] * 6, [200] * 6, 1, 64, 16, seed=8)
    spoil_unused(bt)
    for b in range(6):
        for j in range(13):
            p = int(bt.table[b, j])
            bt.vs[p] = [2.0 ** -30 * 1.37, 2.0 ** (-80 + 6 * j), 2.0 ** (7 * (j % 3) - 40), 3.0 + j, 0.0,
                        2.0 ** -10 if j else 2.0 ** 40][b]
            bt.ks[p] = 0.011 * (1 + j % 4)
    q = bt.values(8, torch.bfloat16)
    say("scales far apart")
    want = ref.attend(bt, q, 0.125)
    got = call(on_gpu(bt), q.to(DEV), 1, scale=0.125)
    torch.cuda.synchronize()
    compare(bt, q, got, want)


def test_scales_that_are_none():
    """Zero, negative, infinite and NaN scales count as the ends of the range."""
    bt = ref.Batch([1], [96], 1, 64, 16, seed=8)
    for j, s in enumerate([0.0, -2.0, math.nan, 1e-38, 2.0 ** -100, 2.0 ** -99]):
        bt.vs[int(bt.table[0, j])] = s
        bt.ks[int(bt.table[0, j])] = s
    q = bt.values(4, torch.bfloat16)
    say("odd scales")
    want = ref.attend(bt, q, 0.125)
    got = call(on_gpu(bt), q.to(DEV), 1, scale=0.125)
    torch.cuda.synchronize()
    compare(bt, q, got, want)


def test_large_logits():
    """Logits of some thousands: one key takes all, and nothing overflows."""
    bt = ref.Batch([1, 4], [100, 200], 1, 64, 64, seed=9)
    bt.ks *= 64
    say("large logits")
    run(bt, 8, torch.bfloat16, spread=30.0)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-30])
def test_any_softmax_scale(scale):
    """Negative (the sign goes to the queries), zero and tiny: masked keys stay masked."""
    say("softmax scale", scale)
    for new, lens in (([1, 1], [70, 130]), ([70, 3], [100, 90])):
        bt = ref.Batch(new, lens, 2, 64, 32, seed=20)
        q = bt.values(4, torch.float16)
        want = ref.attend(bt, q, scale)
        got = call(on_gpu(bt), q.to(DEV), bt.max_q, scale=scale)
        torch.cuda.synchronize()
        compare(bt, q, got, want)


def test_pages_that_are_none():
    """Tokens on ids outside the pool are not seen; a sequence of nothing else gets zeros."""
    bt = ref.Batch([1, 3, 1, 20], [150, 70, 40, 60], 2, 64, 16, seed=10)
    bt.table[0, 2] = -1
    bt.table[1, 4] = bt.pages
    bt.table[1, 0] = 2 ** 31 - 1
    bt.table[2, :] = -7
    bt.table[3, 0] = -1
    say("no pages")
    run(bt, 4, torch.bfloat16)
    run(bt, 4, torch.bfloat16, window=17)


def test_nan_reaches_only_the_rows_that_see_it():
    """NaN among the keys and values of a late token: earlier rows are as without it, later rows
    are NaN where the plain sum is."""
    say("nan")
    for new, length, heads in ((12, 80, 2), (150, 170, 2), (1, 64, 8)):
        bt = ref.Batch([new], [length], 1, 64, 64, seed=11)
        q = bt.values(heads, torch.bfloat16)
        late = length - max(1, new // 2)
        pid, slot = int(bt.table[0, late // 64]), late % 64
        clean = ref.attend(bt, q, 0.125)
        bt.v[pid, 0, 5, slot] = 0x7F
        got = call(on_gpu(bt), q.to(DEV), bt.max_q, scale=0.125)
        torch.cuda.synchronize()
        y = got[0].cpu().double()
        sees = torch.arange(length - new, length) >= late
        assert torch.all(torch.isnan(y[sees][:, :, 5]))
        others = torch.ones(64, dtype=torch.bool)
        others[5] = False
        assert not torch.isnan(y[:, :, others]).any()
        compare(bt, q, got, clean, rows=~sees)
        bt.v[pid, 0, 5, slot] = 0x30
        bt.k[pid, 0, slot, 7] = 0xFF
        clean = ref.attend(bt, q, 0.125)
        got = call(on_gpu(bt), q.to(DEV), bt.max_q, scale=0.125)
        torch.cuda.synchronize()
        assert torch.all(torch.isnan(got[0].cpu()[sees]))
        compare(bt, q, got, clean, rows=~sees)


def test_nan_and_infinite_queries_stay_in_their_rows():
    bt = ref.Batch([5, 40], [70, 40], 1, 64, 64, seed=12)
    q = bt.values(2, torch.float16)
    bad = q.clone()
    bad[2, 1, 3], bad[20, 0, 0] = math.nan, math.inf
    want = ref.attend(bt, q, 0.125)
    say("nan queries")
    got = call(on_gpu(bt), bad.to(DEV), 40, scale=0.125)
    torch.cuda.synchronize()
    assert torch.isnan(got[0][2, 1]).all()
    for t in (*got,):
        t[2, 1] = 0
        t[20, 0] = 0
    for t in want:
        t[2, 1] = 0
        t[20, 0] = 0
    compare(bt, q, got, want)


@pytest.mark.parametrize("lens,starts", [([10 ** 9], [0, 4]), ([-5], [0, 4]), ([50], [-3, 10 ** 9]),
                                         ([50], [4, 0]), ([50], [3, 3])])
def test_arrays_out_of_bounds_stay_inside(lens, starts):
    bt = ref.Batch([4], [60], 1, 32, 16, seed=2)
    q = bt.values(2, torch.bfloat16)
    d = on_gpu(bt)
    d["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    d["q_start"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    say("attend", lens, starts)
    y = torch.full((8, 2, 32), 7.0, dtype=torch.bfloat16, device=DEV)
    call(d, q.to(DEV), 4, y=y[2:6])
    torch.cuda.synchronize()
    assert torch.all(y[:2] == 7.0) and torch.all(y[6:] == 7.0)


def test_fewer_rows_than_announced():
    """max_q may be larger than any sequence's new tokens, up to the batch's tokens."""
    bt = ref.Batch([3, 1, 60], [40, 9, 80], 2, 64, 32, seed=13)
    q = bt.values(4, torch.bfloat16)
    want = ref.attend(bt, q, 0.1)
    say("max_q")
    for max_q in (60, 64):
        got = call(on_gpu(bt), q.to(DEV), max_q, scale=0.1)
        torch.cuda.synchronize()
        compare(bt, q, got, want)


def test_strided_queries_are_the_dense_ones():
    bt = ref.Batch([9, 1, 80], [70, 64, 90], 2, 64, 64, seed=14)
    wide = torch.randn(bt.tokens, 11, 64, generator=bt.gen).to(torch.bfloat16).to(DEV)
    d = on_gpu(bt)
    say("strides")
    a = call(d, wide[:, 3:7], 80)
    b = call(d, wide[:, 3:7].contiguous(), 80)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_scratch_of_the_callers():
    bt = ref.Batch([2, 1], [3000, 70], 2, 64, 64, seed=25)
    q, d = bt.values(8, torch.bfloat16).to(DEV), on_gpu(bt)
    work = fp8q.paged_attention_work(q, d["k"], d["table"], 2)
    say("scratch")
    want = call(d, q, 2)
    got = call(d, q, 2, work=torch.full((work.numel() + 64,), 0xFF, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(ValueError, match="work must hold"):
        call(d, q, 2, work=work[:-1])
    with pytest.raises(ValueError, match="y must have shape"):
        call(d, q, 2, y=torch.empty((3, 8, 32), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError, match="lse must be"):
        call(d, q, 2, lse=torch.empty((3, 8), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError, match="heads must be contiguous"):
        call(d, q.transpose(0, 1).contiguous().transpose(0, 1), 2)


def test_results_repeat_bit_for_bit():
    bt = ref.Batch([1] * 20, [50 + 97 * b for b in range(20)], 2, 128, 64, seed=15)
    q = bt.values(16, torch.bfloat16).to(DEV)
    d = on_gpu(bt)
    say("repeat")
    a = call(d, q, 1)
    for _ in range(3):
        b = call(d, q, 1)
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_pages_past_32_bits():
    pages, heads, dim, page = 66000, 8, 128, 64
    for new, length in ((1, 200), (70, 130)):
        bt = ref.Batch([new], [length], heads, dim, page, seed=16)
        spoil_unused(bt)
        q = bt.values(heads, torch.bfloat16)
        want = ref.attend(bt, q, 0.09)
        d = on_gpu(bt)
        say("attend past 4 GB", new, length)
        big = {n: torch.zeros((pages, *d[n].shape[1:]), dtype=d[n].dtype, device=DEV) for n in ("k", "v", "ks", "vs")}
        for n in big:
            big[n][-bt.pages:] = d[n]
        big["table"] = torch.where(d["table"] < 0, d["table"], d["table"] + (pages - bt.pages))
        big["q_start"], big["kv_lens"] = d["q_start"], d["kv_lens"]
        got = call(big, q.to(DEV), new, scale=0.09)
        torch.cuda.synchronize()
        compare(bt, q, got, want)


@pytest.mark.parametrize("new,lens", [([1] * 6, [3, 700, 64, 0, 1500, 65]), ([70, 1, 33], [70, 500, 90])])
def test_graph_replays(new, lens):
    """Captured once, replayed with other queries, lengths and cache contents."""
    bt = ref.Batch(new, lens, 2, 64, 64, seed=17)
    d = on_gpu(bt)
    q = torch.zeros((bt.tokens, 8, 64), dtype=torch.bfloat16, device=DEV)
    y, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
    work = fp8q.paged_attention_work(q, d["k"], d["table"], bt.max_q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(d, q, bt.max_q, y=y, lse=lse, work=work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(d, q, bt.max_q, y=y, lse=lse, work=work)
    for i in range(4):
        q.copy_(torch.randn(q.shape, generator=bt.gen).to(torch.bfloat16))
        d["k"].copy_(bt._codes(bt.k.shape))
        d["kv_lens"].copy_(torch.tensor([max(n, x - 7 * i) if x else 0 for n, x in zip(new, lens)]))
        work.fill_(0xFF)
        say("attend replay", i)
        a = call(d, q, bt.max_q)
        torch.cuda.synchronize()
        y.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, a[0]) and torch.equal(lse, a[1])


def test_two_streams_at_once():
    """Calls on two streams, each with its scratch, give what they give alone."""
    parts = []
    for seed in (18, 19):
        bt = ref.Batch([1] * 8, [2000 + 100 * b for b in range(8)], 2, 128, 64, seed=seed)
        d, q = on_gpu(bt), bt.values(8, torch.bfloat16).to(DEV)
        parts.append((d, q, call(d, q, 1), fp8q.paged_attention_work(q, d["k"], d["table"], 1)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in parts]
    got = [[], []]
    say("two streams")
    for _ in range(10):
        for i, (s, (d, q, _, work)) in enumerate(zip(streams, parts)):
            with torch.cuda.stream(s):
                got[i].append(call(d, q, 1, work=work))
    torch.cuda.synchronize()
    for i, (_, _, want, _) in enumerate(parts):
        for g in got[i]:
            assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])

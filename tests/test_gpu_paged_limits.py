"""The paged cache's entry points at calls that their documentation allows and a serving loop seldom
makes, against the host form in 64 bits."""
import copy

import pytest
import torch

import paged_ref as ref
from fp8_quantized_gemm_amd import fp8q
from gpu_helpers import DEV, say
from test_gpu_attention import call, compare, on_gpu, spoil_unused

pytestmark = pytest.mark.gpu


def append(d, k, v, max_q, **more):
    return fp8q.fp8_kv_append(k, v, d["k"], d["v"], d["ks"], d["vs"], d["table"], d["q_start"], d["kv_lens"], max_q,
                              **more)


def same_cache(d, want):
    for n in ("k", "v", "ks", "vs"):
        assert torch.equal(d[n].cpu().view(torch.uint8), getattr(want, n).view(torch.uint8)), n


def test_one_token_in_a_row_of_any_length():
    """Queries, keys and values of one token inside a buffer whose length no row stride could have."""
    bt = ref.Batch([1], [70], 2, 64, 16, seed=50)
    row = torch.randn(1, 1001, generator=bt.gen).to(torch.bfloat16)
    parts = lambda t: (t.as_strided((1, n, 64), (1001, 64, 1), at * 64) for at, n in ((0, 8), (8, 2), (10, 2)))  # noqa: E731
    q, k, v = parts(row)
    rope = ref.rope_table(bt.width * 16, 64)
    d, want = on_gpu(bt), copy.deepcopy(bt)
    qo = ref.append(want, k, v, rope, False, q)
    g = row.to(DEV)
    gq, gk, gv = parts(g)
    say("one token of a row of 1001")
    append(d, gk, gv, 1, rope=rope.to(DEV), q=gq, q_out=gq)
    torch.cuda.synchronize()
    same_cache(d, want)
    assert torch.all((gq.cpu().double() - qo).abs() <= qo.abs() * ref.EPS[torch.bfloat16])
    assert torch.equal(g[:, 12 * 64:].cpu(), row[:, 12 * 64:])
    got = call(d, gq, 1, scale=0.1)
    torch.cuda.synchronize()
    compare(want, gq.cpu(), got, ref.attend(want, gq.cpu(), 0.1))


@pytest.mark.parametrize("heads,room", [(4, 0), (4, 20000), (24, 0), (24, 1500)])
def test_rows_beyond_max_q_are_left_out(heads, room):
    """Sequences with more new tokens than max_q: the first max_q are appended and answered, the others
    are left as they are."""
    for max_q in (1, 3):
        new, lens = [5, 1, 9, 2], [40, 6, 70, 2]
        bt = ref.Batch(new, lens, 2, 64, 16, seed=51, lead=1, tail=1, width=max(5, -(-room // 16)))
        spoil_unused(bt)
        k, v, q = bt.values(2, torch.bfloat16), bt.values(2, torch.bfloat16), bt.values(heads, torch.bfloat16)
        d, want = on_gpu(bt), copy.deepcopy(bt)
        say("beyond max_q", heads, room, max_q)
        # as sequences of the first tokens only, whose positions are the same; the rows lie elsewhere
        cut = [min(n, max_q) for n in new]
        want.new, want.lens = cut, [x - n + c for x, n, c in zip(lens, new, cut)]
        ref.append(want, k, v)
        append(d, k.to(DEV), v.to(DEV), max_q)
        torch.cuda.synchronize()
        same_cache(d, want)
        # attention: the same rows see the keys that are there for them
        spoil = copy.deepcopy(want)
        y = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
        lse = torch.full(q.shape[:2], 7.0, device=DEV)
        got = call(d, q.to(DEV), max_q, scale=0.1, y=y, lse=lse)
        torch.cuda.synchronize()
        result = ref.attend(spoil, q, 0.1)
        compare(want, q, got, result)
        left = torch.isnan(result[1])
        assert torch.all(y.cpu()[left] == 7.0) and torch.all(lse.cpu()[left] == 7.0)


@pytest.mark.parametrize("heads,kv_heads,new,room", [(160, 1, 2, 0), (160, 1, 2, 3000), (1024, 4, 1, 0), (300, 2, 3, 0)])
def test_more_query_heads_than_a_workgroup_has_rows(heads, kv_heads, new, room):
    bt = ref.Batch([new, 1], [90, 33], kv_heads, 32, 16, seed=52, width=max(6, -(-room // 16)))
    spoil_unused(bt)
    q = bt.values(heads, torch.float16)
    say("heads", heads, kv_heads, new, room)
    got = call(on_gpu(bt), q.to(DEV), new, scale=0.2)
    torch.cuda.synchronize()
    compare(bt, q, got, ref.attend(bt, q, 0.2))


@pytest.mark.parametrize("new,heads", [(1, 1), (5, 4)])
def test_the_longest_table(new, heads):
    """2^24 tokens, all on one page: logits of zero, so that every one counts the same.  A sum of 2^24
    equal terms is one of at most 2^13 additions a lane (parts of 2^15 keys and more, 16 keys of a tile
    a lane), 2^13 * 2^-24 of it at most, after those of at most 512 parts."""
    page, dim = 128, 16
    width = 2 ** 24 // page
    d = {"k": torch.zeros((1, 1, page, dim), dtype=torch.uint8), "ks": torch.ones(1, 1), "vs": torch.ones(1, 1),
         "v": ref.e4m3_codes(torch.arange(page * dim).double().view(1, 1, dim, page) % 61 / 8 + 1),
         "table": torch.zeros((1, width), dtype=torch.int32), "q_start": torch.tensor([0, new], dtype=torch.int32),
         "kv_lens": torch.tensor([2 ** 24], dtype=torch.int32)}
    mean = ref.TABLE[d["v"].long()].mean(dim=3)[0, 0]
    d = {n: t.to(DEV) for n, t in d.items()}
    q = torch.randn(new, heads, dim).to(torch.float16).to(DEV)
    say("longest table", new, heads)
    y, lse = call(d, q, new, causal=False)
    torch.cuda.synchronize()
    off = 2.0 ** -11 + 2.0 ** -13
    assert torch.all((lse.cpu().double() - 24 * 0.6931471805599453).abs() <= off)
    assert torch.all((y.cpu().double() - mean).abs() <= mean * (2 * off + 2.0 ** -11))

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

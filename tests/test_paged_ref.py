"""The host forms that the paged cache's GPU tests compare with, against torch's own conversions
and a softmax in other words (CPU)."""
import math

import pytest
import torch

import paged_ref as ref


def test_codes_round_trip_and_match_torch():
    fin = ~torch.isnan(ref.TABLE)
    assert int(fin.sum()) == 254
    assert torch.equal(ref.e4m3_codes(ref.TABLE[fin]), torch.arange(256)[fin].to(torch.uint8))
    x = torch.cat([torch.randn(20000) * 100, torch.randn(20000) * 0.01, torch.tensor([0.0, -0.0, 500.0, -1e9])])
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(ref.e4m3_codes(x.double()), want)


@pytest.mark.parametrize("page,new,lens", [(16, [3, 0, 20], [3, 0, 37]), (64, [1], [64])])
def test_append_then_attend_is_plain_attention(page, new, lens):
    """A value written by append and read by attend is within E4M3's half step of itself."""
    bt = ref.Batch(new, lens, 2, 32, page, seed=3)
    k, v = bt.values(2, torch.bfloat16), bt.values(2, torch.bfloat16)
    ref.append(bt, k, v)
    for b, row0, n, length in bt.seqs():
        for i in range(n):
            p = length - n + i
            pid, slot = int(bt.table[b, p // page]), p % page
            got = ref.TABLE[bt.k[pid, :, slot].long()] * bt.ks[pid].double()[:, None]
            x = k[row0 + i].double()
            assert torch.all((got - x).abs() <= x.abs() * 2.0 ** -4 + bt.ks[pid].double()[:, None] * 2.0 ** -10)
            got = ref.TABLE[bt.v[pid, :, :, slot].long()] * bt.vs[pid].double()[:, None]
            x = v[row0 + i].double()
            assert torch.all((got - x).abs() <= x.abs() * 2.0 ** -4 + bt.vs[pid].double()[:, None] * 2.0 ** -10)
    q = bt.values(4, torch.bfloat16)
    y, lse, _, _ = ref.attend(bt, q, 0.2)
    b, row0, n, length = 0, int(bt.q_start[0]), new[0], lens[0]
    pid = bt.table[b, torch.arange(length) // page].long()
    kk = ref.TABLE[bt.k[pid, :, torch.arange(length) % page].long()] * bt.ks[pid].double()[:, :, None]
    vv = ref.TABLE[bt.v[pid, :, :, torch.arange(length) % page].long()] * bt.vs[pid].double()[:, :, None]
    for j in range(4):
        z = q[row0 + n - 1, j].double() @ kk[:, j // 2].t() * 0.2
        assert torch.allclose(y[row0 + n - 1, j], torch.softmax(z, 0) @ vv[:, j // 2])
        assert math.isclose(float(lse[row0 + n - 1, j]), float(torch.logsumexp(z, 0)))


def test_rotation_keeps_lengths():
    x = torch.randn(3, 32, dtype=torch.float64).float().double()
    row = ref.rope_table(10, 32)[7]
    for inter in (False, True):
        y = ref.rotate(x, row, inter)
        assert torch.allclose(y.norm(dim=1), x.norm(dim=1), rtol=1e-6)
        assert not torch.allclose(y, x)

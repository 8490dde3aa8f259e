"""Refusals of the paged cache's entry points: checked on the host before any HIP call (CPU only;
the pointers are never dereferenced)."""
import ctypes
import math

import pytest
import torch

from fp8_quantized_gemm_amd import fp8q

OK, NULLP, SHAPE, ALIGN, DTYPE, OVERLAP = 0, 1, 2, 3, 4, 7


def at(region, offset=0):
    return 0x100000000 + region * 0x10000000 + offset


CACHE = dict(k=at(0), v=at(1), k_scale=at(2), v_scale=at(3), pages=100, kv_heads=2, page_size=64,
             head_dim=128)
BATCH = dict(page_table=at(4), q_start=at(5), kv_lens=at(6), tokens=32, seqs=4, table_width=10, max_q=8)
APPEND = dict(kp=at(7), k_stride=256, vp=at(8), v_stride=256, dtype=0, rope=at(9), rope_rows=640,
              rope_dim=128, interleaved=0, q=at(10), q_stride=1024, q_out=at(11), q_out_stride=1024,
              q_heads=8, stream=None)
ATTEND = dict(q=at(10), q_stride=1024, dtype=0, q_heads=8, scale=0.1, causal=1, window=0, y=at(11),
              lse=at(12), work=at(13), stream=None)


class Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p if n in ("k", "v", "k_scale", "v_scale") else ctypes.c_int64) for n in CACHE]


class Batch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p if n in ("page_table", "q_start", "kv_lens") else ctypes.c_int64)
                for n in BATCH]


def cache_of(c=CACHE):
    return bytes(Cache(*c.values()))


def batch_of(b=BATCH):
    return bytes(Batch(*b.values()))


def status(fn, own, change):
    c, b, a = ({k: change.get(k, v) for k, v in d.items()} for d in (CACHE, BATCH, own))
    assert set(change) <= set(c) | set(b) | set(a)
    return fn(cache_of(c), batch_of(b), *a.values())


def test_structs_of_the_binding():
    assert fp8q._kv_cache_bytes(*CACHE.values()) == cache_of()
    assert fp8q._kv_batch_bytes(*BATCH.values()) == batch_of()


COMMON = [
    *[({n: None}, NULLP) for n in ("k", "v", "k_scale", "v_scale", "page_table", "q_start", "kv_lens")],
    *[({n: x}, SHAPE) for n, xs in (
        ("page_size", (0, 8, 48, 256)), ("head_dim", (0, 8, 24, 272)), ("kv_heads", (0, 1025)),
        ("pages", (0, 2 ** 31, 2 ** 29)), ("tokens", (0, 2 ** 26 + 1)), ("seqs", (0, 65537)),
        ("max_q", (0, 33)), ("table_width", (0, 2 ** 18 + 1)), ("q_stride", (1016, 1028, 2 ** 32 + 8)),
        ("q_heads", (0, 1025))) for x in xs],
    *[({n: at(20, 8)}, ALIGN) for n in ("k", "v", "q")],
    *[({n: at(20, 2)}, ALIGN) for n in ("k_scale", "v_scale", "page_table", "q_start", "kv_lens")],
    ({"dtype": 2}, DTYPE),
]


@pytest.mark.parametrize("change,want", COMMON + [
    *[({n: None}, NULLP) for n in ("kp", "vp", "rope", "q", "q_out")],
    *[({n: x}, SHAPE) for n, xs in (
        ("k_stride", (248, 260)), ("v_stride", (248, 260)), ("q_out_stride", (1016, 1028)),
        ("rope_dim", (-16, 8, 144)), ("rope_rows", (639, 2 ** 31))) for x in xs],
    *[({n: at(20, 8)}, ALIGN) for n in ("kp", "vp", "q_out", "rope")],
    ({"v": at(0, 100 * 2 * 64 * 128 - 16)}, OVERLAP),        # values over the last keys
    ({"k_scale": at(3, 100 * 2 * 4 - 4)}, OVERLAP),
    ({"kp": at(0, 64)}, OVERLAP),                            # new keys inside the pool
    ({"v_scale": at(4, 4 * 10 * 4 - 4)}, OVERLAP),           # over the page table's last id
    ({"k_scale": at(5, 16)}, OVERLAP),                       # over q_start's last entry
    ({"v_scale": at(6, 12)}, OVERLAP),
    ({"q_out": at(7, 16)}, OVERLAP),                         # queries over the new keys
    ({"q_out": at(9, 640 * 128 * 4 - 16)}, OVERLAP),         # over the last sines
    ({"q_out": at(10, 2048)}, OVERLAP),                      # shifted over their input
    ({"q_out": at(10), "q_out_stride": 2048}, OVERLAP),      # in place with another stride
    ({"q_out": at(1, 1024)}, OVERLAP),
    ({"q": at(1, 1024)}, OVERLAP),
])
def test_append_refused(change, want):
    assert status(fp8q.lib.fp8_kv_append, APPEND, change) == want


@pytest.mark.parametrize("change,want", COMMON + [
    *[({n: None}, NULLP) for n in ("q", "y", "work")],
    ({"q_heads": 7}, SHAPE), ({"q_heads": 1}, SHAPE),
    ({"q_heads": 64, "q_stride": 64 * 128, "tokens": 2 ** 25 + 1}, SHAPE),
    *[({"scale": x}, SHAPE) for x in (math.inf, -math.inf, math.nan)],
    ({"window": -1}, SHAPE), ({"window": 2 ** 24 + 1}, SHAPE), ({"window": 5, "causal": 0}, SHAPE),
    *[({n: at(20, 8)}, ALIGN) for n in ("y", "work")],
    ({"lse": at(20, 2)}, ALIGN),
    ({"y": at(10, 31 * 2048 + 2000)}, OVERLAP),
    ({"y": at(0, 16)}, OVERLAP), ({"y": at(1, 16)}, OVERLAP), ({"y": at(6)}, OVERLAP),
    ({"lse": at(11, 32 * 8 * 256 - 4)}, OVERLAP),
    ({"lse": at(2)}, OVERLAP), ({"lse": at(3, 796)}, OVERLAP),
    ({"work": at(4, 0)}, OVERLAP), ({"work": at(5)}, OVERLAP), ({"work": at(12, 32 * 8 * 4 - 16)}, OVERLAP),
])
def test_attention_refused(change, want):
    assert status(fp8q.lib.fp8_paged_attention, ATTEND, change) == want


def test_refused_without_structs():
    a, b = list(APPEND.values()), list(ATTEND.values())
    assert fp8q.lib.fp8_kv_append(None, batch_of(), *a) == NULLP
    assert fp8q.lib.fp8_kv_append(cache_of(), None, *a) == NULLP
    assert fp8q.lib.fp8_paged_attention(None, batch_of(), *b) == NULLP
    assert fp8q.lib.fp8_paged_attention(cache_of(), None, *b) == NULLP


@pytest.mark.skipif(torch.cuda.is_available(), reason="without a GPU the device check ends the call")
def test_overlap_of_interleaved_rows():
    """Rows of one stride between each other are no overlap (q, k, v and q_out of one buffer); the
    next check to fail is then the device's."""
    row = (8 + 2 + 2) * 128
    base = at(30)
    change = dict(q=base, q_stride=row, q_out=base, q_out_stride=row, kp=base + 8 * 256, k_stride=row,
                  vp=base + 10 * 256, v_stride=row)
    assert status(fp8q.lib.fp8_kv_append, APPEND, change) not in (NULLP, SHAPE, ALIGN, DTYPE, OVERLAP)
    for off in (16, 8 * 256 - 16, -16):                     # one vector into q, the keys, or both ends
        assert status(fp8q.lib.fp8_kv_append, APPEND, {**change, "q_out": base + off}) == OVERLAP
    assert status(fp8q.lib.fp8_kv_append, APPEND, {**change, "kp": base + 8 * 256 - 16}) == OVERLAP
    wide = 20 * 128                                         # q_out beside v in wider rows
    beside = {**change, "q_stride": wide, "k_stride": wide, "v_stride": wide, "q_out_stride": wide,
              "q_out": base + 12 * 256}
    assert status(fp8q.lib.fp8_kv_append, APPEND, beside) not in (NULLP, SHAPE, ALIGN, DTYPE, OVERLAP)
    assert status(fp8q.lib.fp8_kv_append, APPEND, {**beside, "q_out": base + 12 * 256 + 16}) == OVERLAP


def test_work_bytes():
    good = dict(tokens=4, seqs=2, table_width=20, max_q=2, q_heads=8, kv_heads=2, page_size=64, head_dim=128)
    assert fp8q.paged_attention_work_bytes(**good) > 0
    assert fp8q.paged_attention_work_bytes(**{**good, "max_q": 4, "q_heads": 64}) > 0
    for change in (dict(q_heads=0), dict(q_heads=3), dict(q_heads=2048), dict(kv_heads=0), dict(head_dim=24),
                   dict(head_dim=272), dict(max_q=0), dict(max_q=5), dict(page_size=48), dict(seqs=0),
                   dict(tokens=0), dict(tokens=2 ** 26, q_heads=64), dict(table_width=0), dict(table_width=2 ** 18 + 1)):
        assert fp8q.paged_attention_work_bytes(**{**good, **change}) == 0


def test_binding_refuses_wrong_tensors():
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    p, s, t = torch.zeros((3, 2, 16, 64), dtype=torch.uint8), torch.zeros((3, 2)), torch.zeros((1, 2), dtype=torch.int32)
    for call in (lambda **m: fp8q.fp8_kv_append(x, x, p, p, s, s, t, t, t, 4, **m),
                 lambda **m: fp8q.fp8_paged_attention(x, p, p, s, s, t, t, t, 4, **m)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(TypeError):
        fp8q.fp8_kv_append(x.float(), x, p, p, s, s, t, t, t, 4)
    with pytest.raises(TypeError):
        fp8q.fp8_paged_attention(x.float(), p, p, s, s, t, t, t, 4)

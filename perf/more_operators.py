"""Cases of the paged FP8 key/value cache: what each operator computes in elementary torch
operations, the framework's call that computes the same, and what a pass has to move.

The cache is a pool of pages of P tokens.  A page holds, for each key/value head, the E4M3
codes of its keys [P, D] and of its values, channel by channel, [D, P], with one fp32 scale
for each of the two.  A batch is described by page_table [B, W], q_start [B + 1] (rows of the
batch's tokens) and kv_lens [B] (tokens in the cache, the new ones included): token i of the n
new ones of sequence b sits at position kv_lens[b] - n + i.

- append: the new tokens' queries and keys rotated by their positions, keys and values
  quantized into their pages.  A page's scale is a power of two that holds its largest value;
  where a page that has tokens already needs a larger one, its codes are scaled down.
- attend: softmax(scale * q k^T) v over the cached tokens, causal or not, with an optional
  sliding window, and the logarithm of the softmax's denominator.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
LOG2_MIN, LOG2_MAX = -100, 100             # exponents of the scales
MAX_BYTES = 64 * 8192 * 8 * 2 * 128        # of the largest listed cases
MAX_PAIRS = 64 * 4096 * 4096               # (query row, key) pairs of one head size, padded
MAX_FLOPS = 4 * 128 * MAX_PAIRS


# ------------------------------------------------------------------ cases
def _case(name, op, batch, new, length, heads, kv_heads, dim, page=64, dtype="bf16", ragged=False,
          **more):
    """`new` and `length` are the longest sequence's new tokens and tokens in the cache."""
    return {"name": name, "op": op, "batch": batch, "new": new, "length": length, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "ragged": ragged,
            **more}


def _append(name, *sizes, rotary=None, interleaved=False, **more):
    case = _case(name, "append", *sizes, **more)
    return {**case, "rotary": case["dim"] if rotary is None else rotary, "interleaved": interleaved}


def _attend(name, *sizes, causal=True, window=0, **more):
    return {**_case(name, "attend", *sizes, **more), "causal": causal, "window": window}


def listed():
    return [
        # one user's next token: the smallest call, all latency (64 query, 8 key/value heads)
        _append("append 1x1 64/8x128", 1, 1, 1000, 64, 8, 128),
        # a decode batch with idle slots, every sequence at another place of its page
        _append("append 48x1 32/32x128", 48, 1, 1024, 32, 32, 128, ragged=True),
        # a long prompt into empty pages
        _append("append 2048 32/32x128", 1, 2048, 2048, 32, 32, 128),
        # a ragged batch of prompt chunks that begin inside a page; small pages, an odd head
        # count, part of each head rotated, in interleaved pairs
        _append("append 7x700 12/3x96", 7, 701, 1500, 12, 3, 96, rotary=64, interleaved=True,
                page=16, dtype="fp16", ragged=True),
        # one user's next token after a short prompt: the smallest call of the attention
        _attend("decode 1x500 64/8x128", 1, 1, 500, 64, 8, 128),
        # a ragged decode batch, a key/value head for every query head
        _attend("decode 24x2048 32/32x128", 24, 1, 2048, 32, 32, 128, ragged=True),
        # a large decode batch of long contexts
        _attend("decode 64x8192 64/8x128", 64, 1, 8192, 64, 8, 128),
        # one very long context: few rows, so that the keys have to be shared out
        _attend("decode 1x131072 64/8x128", 1, 1, 131072, 64, 8, 128),
        # drafted tokens checked together, with a sliding window over small pages
        _attend("draft 13x5 of 4099 28/4x64", 13, 5, 4099, 28, 4, 64, page=16, dtype="fp16",
                window=1000, ragged=True),
        # a long prompt
        _attend("prompt 2048 32/32x128", 1, 2048, 2048, 32, 32, 128),
        # chunks of prompts behind longer cached contexts, lengths that end inside a page
        _attend("chunks 4x777 of 2900 40/8x128", 4, 777, 2900, 40, 8, 128, ragged=True),
        # the largest prompt
        _attend("prompt 4096 64/8x128", 1, 4096, 4096, 64, 8, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend"])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 12, 16) if g * kv_heads <= 64])
    dim = rng.choice([64, 80, 96, 112, 128, 128, 160, 192, 256])
    page = rng.choice([16, 32, 64, 64, 128])
    heads = group * kv_heads
    more = {"page": page, "dtype": rng.choice(["bf16", "fp16"]), "ragged": rng.random() < 0.6}
    if op == "append":
        batch = _log(rng, 1, 64)
        new = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, 4096 // batch))
        new = max(1, min(new, 2048 * 96 * 128 // (batch * (heads + 2 * kv_heads) * dim)))
        length = min(new + _log(rng, 1, 2048), 1 + 2 ** 28 // (2 * batch * kv_heads * dim))
        case = _append("", batch, new, max(new, length), heads, kv_heads, dim,
                       rotary=rng.choice([dim, dim, 32, 0]), interleaved=rng.random() < 0.4, **more)
    else:
        kind = rng.choice(["decode", "decode", "draft", "prompt"])
        batch = _log(rng, 1, 64) if kind != "prompt" else _log(rng, 1, 8)
        longest = min(131072, MAX_BYTES // (batch * kv_heads * 2 * dim))
        if kind == "prompt":
            new = _log(rng, 16, min(4096, math.isqrt(min(MAX_PAIRS, MAX_FLOPS // (4 * dim))
                                                     // (batch * heads))))
            longest = min(longest, MAX_PAIRS // (batch * heads * new),
                          MAX_FLOPS // (4 * dim * batch * heads * new))
            length = new if rng.random() < 0.4 else _log(rng, new, longest)
        else:
            new = 1 if kind == "decode" else rng.randint(2, 9)
            longest = min(longest, MAX_PAIRS // (batch * heads * new))
            length = _log(rng, new, max(new, longest))
        causal = rng.random() < 0.8
        window = _log(rng, 1, 2 * length) if causal and rng.random() < 0.25 else 0
        case = _attend("", batch, new, length, heads, kv_heads, dim, causal=causal, window=window,
                       **more)
    del case["name"]
    return case


def _sequences(case):
    """New tokens and cached tokens of each sequence: equal, or ragged with an idle slot."""
    batch, new, length = case["batch"], case["new"], case["length"]
    if not case["ragged"]:
        return [new] * batch, [length] * batch
    spread = [(b * 0x9E3779B1 + 7) % 65536 / 65536 for b in range(batch)]
    n = [new if b == 0 else max(1, math.ceil(new * (1 - spread[b]))) for b in range(batch)]
    lens = [length if b == 0 else max(n[b], math.ceil(length * spread[b])) for b in range(batch)]
    if batch > 2:                          # a slot of the batch that holds no sequence: no cached
        lens[batch // 2] = 0               # token; in a decode batch its row is there, and empty
        n[batch // 2] = 1 if new == 1 and case["op"] == "attend" else 0
    return n, lens


# ------------------------------------------------------------------ plain forms
def _rotate(x, rope, pos, interleaved):
    """x [T, H, D] in fp32; rope [positions, R]: R / 2 cosines, then R / 2 sines."""
    half = rope.shape[1] // 2
    if half == 0:
        return x
    row = rope[pos][:, None]
    c, s = row[..., :half], row[..., half:]
    y = x.clone()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else \
        (slice(0, half), slice(half, 2 * half))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _scale_for(amax):
    """The smallest power of two s with amax <= 448 s."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.exp2(torch.where(amax > 0, e, LOG2_MIN).clamp(LOG2_MIN, LOG2_MAX).float())


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _codes(v):
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _place(st):
    """Sequence, place in the sequence's new tokens and position of every token of the batch."""
    t = torch.arange(st["tokens"], device=st["q_start"].device, dtype=torch.int32)
    seq = torch.searchsorted(st["q_start"], t, right=True) - 1
    i = t - st["q_start"][seq]
    new = st["q_start"].diff()
    return seq, i, st["kv_lens"][seq] - new[seq] + i


def _first_pages(st):
    """The page of each sequence's first new token, and how many older tokens it holds (none for
    a sequence without new tokens)."""
    new = st["q_start"].diff()
    start = st["kv_lens"] - new
    p = st["page"]
    at = (start // p).clamp(0, st["page_table"].shape[1] - 1)
    page = st["page_table"].gather(1, at[:, None].long())[:, 0].clamp(min=0)
    return page.long(), torch.where(new > 0, start % p, 0)


def _quantize_into(pages, scale, x, page, slot, first, older, channel_major):
    """Quantizes x [T, H, D] into (page, slot) and grows the scales of the pages it touches."""
    p = pages.shape[3 if channel_major else 2]
    amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(dim=2), "amax")
    need = _scale_for(amax)
    held = (older > 0)[:, None]
    old = scale[first]
    grown = torch.where(held, torch.maximum(old, need[first]), old)
    codes = pages[first]
    less = _codes(_values(codes) * (old / grown)[:, :, None, None])
    kept = torch.arange(p, device=x.device) < older[:, None]
    kept = kept[:, None, None, :] if channel_major else kept[:, None, :, None]
    pages[first] = torch.where(kept, less, codes)
    new_scale = scale.clone()
    new_scale[page] = need[page]
    new_scale[first] = torch.where(held, grown, new_scale[first])
    scale.copy_(new_scale)
    q = _codes(x / scale[page][:, :, None])
    if channel_major:
        pages[page, :, :, slot] = q
    else:
        pages[page, :, slot] = q


def plain_append(st):
    seq, _, pos = _place(st)
    page = st["page_table"][seq, pos // st["page"]].long()
    slot = (pos % st["page"]).long()
    first, older = _first_pages(st)
    k = _rotate(st["k"].float(), st["rope"], pos, st["interleaved"])
    _quantize_into(st["k_pages"], st["k_scale"], k, page, slot, first, older, False)
    _quantize_into(st["v_pages"], st["v_scale"], st["v"].float(), page, slot, first, older, True)
    return _rotate(st["q"].float(), st["rope"], pos, st["interleaved"]).to(st["q"].dtype)


def plain_attend(st):
    """All sequences at once, padded to the longest."""
    table, new = st["page_table"].clamp(min=0).long(), st["q_start"].diff()
    batch, width = table.shape
    q, p, most = st["q"], st["page"], st["max_q"]
    heads, dim = q.shape[1:]
    kv_heads = st["k_scale"].shape[1]
    group, length = heads // kv_heads, width * p
    k = _values(st["k_pages"][table]).mul_(st["k_scale"][table][..., None, None])
    k = k.transpose(1, 2).reshape(batch, kv_heads, length, dim)
    i = torch.arange(most, device=q.device)
    rows = (st["q_start"][:-1, None] + i).clamp(max=st["tokens"] - 1)
    qs = q[rows].float().view(batch, most, kv_heads, group, dim).transpose(1, 2)
    qs = qs.reshape(batch, kv_heads, most * group, dim)
    x = (qs @ k.transpose(2, 3)).mul_(st["scale"]).view(batch, kv_heads, most, group, length)
    del k
    key = torch.arange(length, device=q.device)
    pos = (st["kv_lens"] - new)[:, None] + i
    seen = (key < st["kv_lens"][:, None])[:, None].expand(batch, most, length)
    if st["causal"]:
        seen = seen & (key <= pos[..., None])
        if st["window"]:
            seen = seen & (pos[..., None] - key < st["window"])
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(dim=4, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    x = x.sub_(top).exp_()
    total = x.sum(dim=4, keepdim=True)
    lse = (torch.log(total) + top)[..., 0]
    x = x.div_(torch.where(total > 0, total, torch.ones_like(total)))
    # unused slots hold anything: their weight is zero, their values must not count
    v = _values(st["v_pages"][table]).mul_(st["v_scale"][table][..., None, None])
    v = v.permute(0, 2, 1, 4, 3).reshape(batch, kv_heads, length, dim)
    v.masked_fill_((key >= st["kv_lens"][:, None])[:, None, :, None], 0.0)
    y = x.view(batch, kv_heads, most * group, length) @ v
    y = y.view(batch, kv_heads, most, group, dim).transpose(1, 2).reshape(batch, most, heads, dim)
    lse = lse.permute(0, 2, 1, 3).reshape(batch, most, heads)
    seq, at, _ = _place(st)
    return y[seq, at].to(q.dtype), lse[seq, at]


# ------------------------------------------------------------------ one pass
def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    n, lens = _sequences(case)
    heads, kv_heads, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    tokens, width = sum(n), max(1, -(-max(lens) // page))
    each = [-(-x // page) for x in lens]
    pages = 1 + sum(each)                  # page 0 is nobody's
    st = {"op": case["op"], "tokens": tokens, "max_q": max(n), "page": page}

    def whole(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    st["q_start"] = whole([sum(n[:b]) for b in range(len(n) + 1)])
    st["kv_lens"] = whole(lens)
    used = torch.arange(width, device=dev) < whole(each)[:, None]
    table = torch.full((len(n), width), -1, dtype=torch.int32, device=dev)
    # pages are handed out as they get free: in no order
    table[used] = (1 + torch.randperm(pages - 1, generator=gen, device=dev)).to(torch.int32)
    st["page_table"] = table
    # codes of values with a typical spread; scales as the pages' largest values give them
    for name, shape in (("k", (pages, kv_heads, page, dim)), ("v", (pages, kv_heads, dim, page))):
        x = torch.empty(shape, dtype=torch.float16, device=dev).normal_(0.0, 60.0, generator=gen)
        st[name + "_pages"] = x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        del x
        st[name + "_scale"] = torch.exp2(torch.randint(-8, -5, (pages, kv_heads), generator=gen,
                                                       device=dev).float())
    # the fused projection's output, of which q, k and v are views
    qkv = torch.randn(tokens, heads + 2 * kv_heads, dim, generator=gen, device=dev)
    if case["op"] == "append":             # a few channels of the keys are larger, as in trained models
        hot = torch.randint(0, dim, (max(1, dim // 64),), generator=gen, device=dev)
        qkv[:, heads:heads + kv_heads, hot] *= 12.0
    qkv = qkv.to(DTYPES[case["dtype"]])
    st["q"] = qkv[:, :heads]
    if case["op"] == "append":
        st["k"], st["v"] = qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
        half = case["rotary"] // 2
        turn = torch.arange(width * page, device=dev, dtype=torch.float64)[:, None] * \
            torch.exp2(torch.arange(half, device=dev, dtype=torch.float64) * (-13.2877 / max(1, half)))
        st["rope"] = torch.cat([turn.cos(), turn.sin()], dim=1).float()
        st["interleaved"] = case["interleaved"]
        st["q_out"] = torch.empty(tokens, heads, dim, dtype=qkv.dtype, device=dev)
    else:
        st["scale"], st["causal"], st["window"] = dim ** -0.5, case["causal"], case["window"]
        st["y"] = torch.empty(tokens, heads, dim, dtype=qkv.dtype, device=dev)
        st["lse"] = torch.empty(tokens, heads, device=dev)
        st["work"] = None                  # the attention's scratch, kept from the first pass on
    return st


def run(st):
    if st["op"] == "append":
        if own:
            from fp8_quantized_gemm_amd import fp8q
            q = fp8q.fp8_kv_append(
                st["k"], st["v"], st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"],
                st["page_table"], st["q_start"], st["kv_lens"], st["max_q"], rope=st["rope"],
                interleaved=st["interleaved"], q=st["q"], q_out=st["q_out"])
        else:
            q = plain_append(st)
        return {"k": st["k_pages"].view(torch.float8_e4m3fn), "k_scale": st["k_scale"],
                "v": st["v_pages"].view(torch.float8_e4m3fn), "v_scale": st["v_scale"], "q": q}
    if own:
        from fp8_quantized_gemm_amd import fp8q
        if st["work"] is None:
            st["work"] = fp8q.paged_attention_work(st["q"], st["k_pages"], st["page_table"],
                                                   st["max_q"])
        y, lse = fp8q.fp8_paged_attention(
            st["q"], st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"], st["page_table"],
            st["q_start"], st["kv_lens"], st["max_q"], scale=st["scale"], causal=st["causal"],
            window=st["window"], y=st["y"], lse=st["lse"], work=st["work"])
    else:
        y, lse = plain_attend(st)
    return {"y": y, "lse": lse}


# ------------------------------------------------------------------ what a pass cannot do without
def _seen(first, length, case):
    """The keys that the query at position `first` sees: from, to."""
    if not case["causal"]:
        return 0, length
    low = max(0, first - case["window"] + 1) if case["window"] else 0
    return min(low, length), max(0, min(length, first + 1))


def work(case):
    n, lens = _sequences(case)
    heads, kv_heads, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    tokens = sum(n)
    if case["op"] == "append":
        touched = sum(-(-x // page) - (x - m) // page for m, x in zip(n, lens) if m)
        half = case["rotary"] // 2
        return {"bytes": tokens * dim * (4 * heads + 6 * kv_heads) + 8 * touched * kv_heads
                + 8 * tokens * half + 4 * touched + 8 * len(n),
                "flops": tokens * (6 * half * (heads + kv_heads) + 6 * kv_heads * dim)}
    pairs = keys = 0
    for m, x in zip(n, lens):
        ends = [_seen(x - m + i, x, case) for i in range(m)]
        pairs += sum(hi - lo for lo, hi in ends)
        some = [e for e in ends if e[1] > e[0]]
        keys += max(e[1] for e in some) - min(e[0] for e in some) if some else 0
    return {"bytes": keys * kv_heads * 2 * dim + 4 * (2 * kv_heads + 1) * keys // page
            + tokens * heads * (4 * dim + 4) + 8 * len(n),
            "flops": 4 * dim * heads * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits
def _table(dev):
    """Values of the 256 E4M3 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    c = torch.arange(256, device=dev)
    e, m = ((c >> 3) & 15).double(), (c & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6)
    v = torch.where((c & 127) == 127, torch.full_like(v, math.nan), v)
    return torch.where(c >= 128, -v, v)


def _e4m3(v):
    """The E4M3 value next to v, ties to even, no further than 448."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _f32(v):
    return v.float().double()


def _exact_turn(x, cos, sin, interleaved):
    """The pairs of x [n, H, D] turned by angles given as cosines and sines [n, R / 2]."""
    half = cos.shape[1]
    x = x.clone()
    for j in range(half):
        ia, ib = (2 * j, 2 * j + 1) if interleaved else (j, half + j)
        a, b = x[:, :, ia].clone(), x[:, :, ib].clone()
        c, s = cos[:, None, j].double(), sin[:, None, j].double()
        x[:, :, ia] = _f32(_f32(a * c) - _f32(b * s))
        x[:, :, ib] = _f32(_f32(b * c) + _f32(a * s))
    return x


def _exact_append(case, st):
    n, lens = _sequences(case)
    page, half = case["page"], case["rotary"] // 2
    dev = st["k_pages"].device
    table, ids = _table(dev), st["page_table"].tolist()
    out = {"k": table[st["k_pages"].long()], "v": table[st["v_pages"].long()].transpose(2, 3),
           "k_scale": st["k_scale"].double(), "v_scale": st["v_scale"].double(),
           "q": st["q"].double()}
    at = 0
    for b, (m, length) in enumerate(zip(n, lens)):
        start = length - m
        turn = st["rope"][start:length]
        cos, sin = turn[:, :half], turn[:, half:]
        out["q"][at:at + m] = _exact_turn(out["q"][at:at + m], cos, sin, case["interleaved"])
        both = {"k": _exact_turn(st["k"][at:at + m].double(), cos, sin, case["interleaved"]),
                "v": st["v"][at:at + m].double()}
        for slot in range(start // page, -(-length // page) if m else 0):
            lo, hi = max(start, slot * page), min(length, (slot + 1) * page)
            older, pid = lo - slot * page, ids[b][slot]
            for name, x in both.items():
                x = x[lo - start:hi - start].transpose(0, 1)                     # [H, new, D]
                amax = x.abs().amax(dim=(1, 2))
                e = torch.ceil(torch.log2(torch.where(amax > 0, amax, 1) / 448.0))
                e = torch.where(448.0 * torch.exp2(e - 1) >= amax, e - 1, e)
                e = torch.where(448.0 * torch.exp2(e) < amax, e + 1, e)
                s = torch.exp2(torch.where(amax > 0, e, LOG2_MIN).clamp(LOG2_MIN, LOG2_MAX))
                if older:
                    was = out[name + "_scale"][pid]
                    s = torch.maximum(s, was)
                    old = out[name][pid, :, :older] * (was / s)[:, None, None]
                    out[name][pid, :, :older] = _e4m3(old)
                out[name][pid, :, older:hi - slot * page] = _e4m3(x / s[:, None, None])
                out[name + "_scale"][pid] = s
        at += m
    out["v"] = out["v"].transpose(2, 3).contiguous()
    return out


def _exact_attend(case, st):
    n, lens = _sequences(case)
    page, kv_heads = case["page"], case["kv_heads"]
    group = case["heads"] // kv_heads
    dev = st["q"].device
    table = _table(dev)
    y = torch.zeros(st["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device=dev)
    at = 0
    for b, (m, length) in enumerate(zip(n, lens)):
        ids = st["page_table"][b, :-(-length // page)].long()
        key = torch.arange(length, device=dev)
        see = torch.ones(m, length, dtype=torch.bool, device=dev)
        if case["causal"]:
            back = torch.arange(length - m, length, device=dev)[:, None] - key
            see = (back >= 0) & (back < (case["window"] or length + 1))
        for h in range(kv_heads if length and m else 0):
            k = table[st["k_pages"][ids, h].long()] * st["k_scale"][ids, h].double()[:, None, None]
            v = table[st["v_pages"][ids, h].long()] * st["v_scale"][ids, h].double()[:, None, None]
            k, v = k.reshape(-1, case["dim"])[:length], v.transpose(1, 2).reshape(-1, case["dim"])[:length]
            for g in range(h * group, (h + 1) * group):
                x = st["q"][at:at + m, g].double() @ k.t() * st["scale"]
                x = torch.where(see, x, -math.inf)
                total = torch.logsumexp(x, dim=1)
                lse[at:at + m, g] = total
                y[at:at + m, g] = torch.nan_to_num(torch.exp(x - total[:, None]), nan=0.0) @ v
        at += m
    return {"y": y, "lse": lse}


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_append(case, st) if case["op"] == "append" else _exact_attend(case, st)

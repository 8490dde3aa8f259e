"""Cases of the block-scaled FP8 operators: what each one computes in elementary torch
operations, the framework's call that computes the same, and what a pass has to move.

The operators share one number format: E4M3 codes with an fp32 scale for every block of 128
values along K (activations, 1 x 128, scales stored [K blocks, rows]) or for every 128 x 128
block of a weight matrix.

- quantize / quantize_weight: codes and block scales of a bf16 or fp16 matrix.
- gemm: the product of codes with block scales on both operands.
- linear: quantize, then gemm.
- moe: a mixture-of-experts layer for a few tokens on block-scaled weights: top-k of the
  router's logits, gated experts, weighted sum.
"""
import math

import torch

own = False

BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases
def _quantize(name, rows, cols, dtype):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "dtype": dtype}


def _product(name, op, m, n, k, dtype="bf16"):
    return {"name": name, "op": op, "m": m, "n": n, "k": k, "dtype": dtype}


def _moe(name, tokens, experts, top_k, hidden, inter, dtype, renormalize, masked):
    return {"name": name, "op": "moe", "tokens": tokens, "experts": experts, "top_k": top_k,
            "hidden": hidden, "inter": inter, "dtype": dtype, "renormalize": renormalize,
            "masked": masked}


def listed():
    return [
        # a decode batch's activation before one linear: the smallest call, all latency
        _quantize("quantize 16x4096", 16, 4096, "bf16"),
        # a long prompt's activation before the down projection
        _quantize("quantize 2048x11008", 2048, 11008, "bf16"),
        # laying out a checkpoint's weight matrix (done once per matrix while loading)
        {"name": "quantize_weight 4096x11008", "op": "quantize_weight", "n": 4096, "k": 11008,
         "dtype": "fp16"},
        # QKV projection of a prompt whose codes the previous kernel has already made
        _product("gemm 512x12288x4096", "gemm", 512, 12288, 4096),
        # a ragged batch of prompts, vocabulary-like odd N, K that ends inside a block
        _product("gemm 333x4100x5008", "gemm", 333, 4100, 5008),
        # one token, one output projection: the latency of a decode step's smallest linear
        _product("linear 1x4096x4096", "linear", 1, 4096, 4096),
        # a small decode batch on the fused gate and up projection
        _product("linear 8x22016x4096", "linear", 8, 22016, 4096),
        # a larger decode batch, fp16 activations
        _product("linear 16x10240x5120", "linear", 16, 10240, 5120, "fp16"),
        # a long prompt through the QKV projection
        _product("linear 2048x12288x4096", "linear", 2048, 12288, 4096),
        # single-token decoding: six small experts of 64
        _moe("moe 1 token 6 of 64", 1, 64, 6, 2048, 1408, "bf16", True, "none"),
        # a ragged decode batch with some experts switched off, plain softmax weights, an
        # expert width that ends inside a block
        _moe("moe 13 tokens 4 of 32", 13, 32, 4, 4096, 1392, "fp16", False, "some"),
        # the largest decode batch: nearly every expert is read
        _moe("moe 64 tokens 8 of 128", 64, 128, 8, 2048, 768, "bf16", True, "none"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, step=16):
    return min(hi, max(lo, step * (_log(rng, lo, hi) // step)))


def draw(rng):
    op = rng.choice(["quantize", "quantize_weight", "gemm", "linear", "linear", "moe", "moe"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "quantize":
        cols = _mult(rng, 16, 25600)
        rows = _log(rng, 1, max(1, min(4096, 2048 * 11008 // cols)))
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype}
    if op == "quantize_weight":
        k = _mult(rng, 256, 25600)
        return {"op": op, "n": _log(rng, 16, min(16384, 4096 * 11008 // k)), "k": k, "dtype": dtype}
    if op in ("gemm", "linear"):
        m = _log(rng, 1, 2048)
        k = _mult(rng, 256, 11008)
        n = _log(rng, 64, min(22016, 4096 * 22016 // k, 2048 * 12288 * 4096 // (m * k)))
        return {"op": op, "m": m, "n": n, "k": k, "dtype": dtype}
    top_k = rng.randint(1, 8)
    experts = _log(rng, max(4, top_k), 128)
    hidden = _mult(rng, 512, 4096)
    inter = _mult(rng, 256, min(4096, 128 * 2048 * 768 // (experts * hidden)))
    return {"op": "moe", "tokens": _log(rng, 1, 64), "experts": experts, "top_k": top_k,
            "hidden": hidden, "inter": inter, "dtype": dtype,
            "renormalize": rng.random() < 0.5, "masked": rng.choice(["none", "some", "row"])}


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


# ------------------------------------------------------------------ plain forms
def _divide(a, b):
    # the correctly rounded fp32 quotient: the division in 64 bits, rounded once
    return (a.double() / b.double()).float()


def _pad(t, rows, cols):
    return torch.nn.functional.pad(t, (0, cols - t.shape[-1], 0, rows - t.shape[-2]))


def _scale(amax):
    return torch.where(amax > 0, _divide(amax, torch.full_like(amax, 448.0)), torch.ones_like(amax))


def _encode(v):
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def plain_quantize(x):
    """Codes [rows, cols] and scales [K blocks, rows], one per 1 x 128 block."""
    rows, cols = x.shape
    kb = _blocks(cols)
    v = _pad(x.float(), rows, kb * BLOCK).view(rows, kb, BLOCK)
    s = _scale(v.abs().amax(dim=2))
    q = _encode(_divide(v, s[:, :, None])).view(rows, kb * BLOCK)[:, :cols].contiguous()
    return q, s.t().contiguous()


def plain_quantize_weight(w):
    """Codes like w[..., N, K] and scales [..., N blocks, K blocks]."""
    n, k = w.shape[-2:]
    nb, kb = _blocks(n), _blocks(k)
    v = _pad(w.float(), nb * BLOCK, kb * BLOCK).view(*w.shape[:-2], nb, BLOCK, kb, BLOCK)
    s = _scale(v.abs().amax(dim=(-3, -1)))
    q = _encode(_divide(v, s[..., :, None, :, None])).view(*w.shape[:-2], nb * BLOCK, kb * BLOCK)
    return q[..., :n, :k].contiguous(), s


def _values(q, s):
    """fp32 values of activation codes with scales [K blocks, rows]."""
    return q.float() * s.t().repeat_interleave(BLOCK, dim=1)[:, :q.shape[1]]


def _weight_values(q, s):
    """fp32 values of weight codes [..., N, K] with scales [..., N blocks, K blocks]."""
    n, k = q.shape[-2:]
    nb, kb = s.shape[-2:]
    v = _pad(q.float(), nb * BLOCK, kb * BLOCK).view(*q.shape[:-2], nb, BLOCK, kb, BLOCK)
    v = (v * s[..., :, None, :, None]).view(*q.shape[:-2], nb * BLOCK, kb * BLOCK)
    return v[..., :n, :k]


def plain_gemm(qa, sa, qw, sw):
    return (_values(qa, sa) @ _weight_values(qw, sw).t()).to(torch.bfloat16)


def plain_route(logits, top_k, renormalize):
    """Ids (descending logit, ties to the lower index; -1 where no finite logit is left) and
    softmax weights, over the chosen experts or over all."""
    best, order = torch.sort(logits, dim=1, descending=True, stable=True)
    best, ids = best[:, :top_k], order[:, :top_k]
    chosen = best > -math.inf
    top = torch.where(chosen[:, :1], best[:, :1], torch.zeros_like(best[:, :1]))
    p = torch.exp(best - top)
    total = (p if renormalize else torch.exp(logits - top)).sum(dim=1, keepdim=True)
    weights = torch.where(chosen, p / total, torch.zeros_like(p))
    return torch.where(chosen, ids, torch.full_like(ids, -1)).to(torch.int32), weights


def plain_moe(x, logits, w13, s13, w2, s2, top_k, renormalize):
    """Where the tokens choose fewer (token, expert) pairs than there are experts, each pair
    with its expert's weights; else all experts on all tokens, in two products, the chosen
    ones carrying their weight."""
    experts, _, inter, hidden = w13.shape
    ids, weights = plain_route(logits, top_k, renormalize)
    if ids.numel() < experts:
        pick = ids.clamp(min=0).long().view(-1)
        rows = x.float().repeat_interleave(top_k, dim=0)
        up = (_weight_values(w13[pick], s13[pick]) @ rows[:, None, :, None]).squeeze(-1)
        act = up[:, 0] * torch.sigmoid(up[:, 0]) * up[:, 1]
        out = (_weight_values(w2[pick], s2[pick]) @ act[:, :, None]).view(-1, top_k, hidden)
        return (out * weights[:, :, None]).sum(dim=1).to(torch.bfloat16), ids, weights
    gate = torch.zeros_like(logits).scatter_add_(1, ids.clamp(min=0).long(), weights)
    up = x.float() @ _weight_values(w13, s13).reshape(experts * 2 * inter, hidden).t()
    up = up.view(-1, experts, 2, inter)
    act = up[:, :, 0] * torch.sigmoid(up[:, :, 0]) * up[:, :, 1] * gate[:, :, None]
    down = _weight_values(w2, s2).transpose(1, 2).reshape(experts * inter, hidden)
    y = act.reshape(-1, experts * inter) @ down
    return y.to(torch.bfloat16), ids, weights


# ------------------------------------------------------------------ one pass
def _activation(rows, cols, dtype, gen, dev):
    # 0.1% of the channels are outliers, as in trained models
    x = torch.randn(rows, cols, generator=gen, device=dev)
    hot = torch.randint(0, cols, (max(1, round(cols / 1000)),), generator=gen, device=dev)
    x[:, hot] *= 50.0
    return x.to(DTYPES[dtype])


def _weight(shape, gen, dev):
    return plain_quantize_weight(torch.randn(*shape, generator=gen, device=dev) * 0.02)


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op = case["op"]
    st = {"op": op}

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device=dev)

    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        st["x"] = _activation(rows, cols, case["dtype"], gen, dev)
        st["q"] = empty(rows, cols, dtype=torch.uint8)
        st["scale"] = empty(_blocks(cols), rows)
    elif op == "quantize_weight":
        n, k = case["n"], case["k"]
        st["w"] = (torch.randn(n, k, generator=gen, device=dev) * 0.02).to(DTYPES[case["dtype"]])
        st["q"] = empty(n, k, dtype=torch.uint8)
        st["scale"] = empty(_blocks(n), _blocks(k))
    elif op in ("gemm", "linear"):
        m, n, k = case["m"], case["n"], case["k"]
        x = _activation(m, k, case["dtype"], gen, dev)
        qw, st["sw"] = _weight((n, k), gen, dev)
        st["qw"] = qw.view(torch.uint8)
        st["y"] = empty(m, n, dtype=torch.bfloat16)
        if op == "gemm":
            qa, st["sa"] = plain_quantize(x)
            st["qa"] = qa.view(torch.uint8)
        else:
            st["x"] = x
            st["q"] = empty(m, k, dtype=torch.uint8)
            st["sa"] = empty(_blocks(k), m)
    else:
        t, e, i, h = case["tokens"], case["experts"], case["inter"], case["hidden"]
        st["x"] = torch.randn(t, h, generator=gen, device=dev).to(DTYPES[case["dtype"]])
        logits = torch.randn(t, e, generator=gen, device=dev) * 1.5
        if case["masked"] != "none":       # a quarter of the experts are switched off
            logits[:, torch.randperm(e, generator=gen, device=dev)[:e // 4]] = -math.inf
        if case["masked"] == "row":        # a padding token that no expert takes
            logits[t // 2] = -math.inf
        st["logits"] = logits
        w13, st["s13"] = _weight((e, 2, i, h), gen, dev)
        w2, st["s2"] = _weight((e, h, i), gen, dev)
        st["w13"], st["w2"] = w13.view(torch.uint8), w2.view(torch.uint8)
        st["top_k"], st["renormalize"] = case["top_k"], case["renormalize"]
        st["y"] = empty(t, h, dtype=torch.bfloat16)
        st["ids"] = empty(t, case["top_k"], dtype=torch.int32)
        st["weights"] = empty(t, case["top_k"])
    return st


def _codes(q):
    return q.view(torch.float8_e4m3fn)


def run(st):
    op = st["op"]
    if own:
        from fp8_quantized_gemm_amd import fp8q
        if op == "quantize":
            q, s = fp8q.fp8_quantize_blocks(st["x"], st["q"], st["scale"])
            return {"codes": _codes(q), "scale": s}
        if op == "quantize_weight":
            q, s = fp8q.fp8_quantize_weight_blocks(st["w"], st["q"], st["scale"])
            return {"codes": _codes(q), "scale": s}
        if op == "gemm":
            return {"y": fp8q.fp8_gemm_blockwise(st["qa"], st["sa"], st["qw"], st["sw"], st["y"])}
        if op == "linear":
            y, q, s = fp8q.fp8_linear_blockwise(st["x"], st["qw"], st["sw"], st["y"], st["q"],
                                                st["sa"])
            return {"y": y, "codes": _codes(q), "scale": s}
        y, ids, weights = fp8q.fp8_moe_blockwise(
            st["x"], st["logits"], st["w13"], st["s13"], st["w2"], st["s2"], st["top_k"],
            st["renormalize"], st["y"], st["ids"], st["weights"])
        return {"y": y, "ids": ids, "weights": weights}
    if op == "quantize":
        q, s = plain_quantize(st["x"])
        return {"codes": q, "scale": s}
    if op == "quantize_weight":
        q, s = plain_quantize_weight(st["w"])
        return {"codes": q, "scale": s}
    if op == "gemm":
        return {"y": plain_gemm(_codes(st["qa"]), st["sa"], _codes(st["qw"]), st["sw"])}
    if op == "linear":
        q, s = plain_quantize(st["x"])
        return {"y": plain_gemm(q, s, _codes(st["qw"]), st["sw"]), "codes": q, "scale": s}
    y, ids, weights = plain_moe(st["x"], st["logits"], _codes(st["w13"]), st["s13"],
                                _codes(st["w2"]), st["s2"], st["top_k"], st["renormalize"])
    return {"y": y, "ids": ids, "weights": weights}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        return {"bytes": 3 * r * c + 4 * r * _blocks(c), "flops": 3 * r * c}
    if op == "quantize_weight":
        n, k = case["n"], case["k"]
        return {"bytes": 3 * n * k + 4 * _blocks(n) * _blocks(k), "flops": 3 * n * k}
    if op in ("gemm", "linear"):
        m, n, k = case["m"], case["n"], case["k"]
        scales = 4 * _blocks(k) * (m + _blocks(n))
        a = m * k if op == "gemm" else 3 * m * k      # codes; or 16-bit values in, codes out
        return {"bytes": a + n * k + scales + 2 * m * n, "flops": 2 * m * n * k}
    t, e, k, h, i = (case[c] for c in ("tokens", "experts", "top_k", "hidden", "inter"))
    alive = e if case["masked"] == "none" else e - e // 4
    rows = t - 1 if case["masked"] == "row" else t
    k = min(k, alive)
    active = alive * (1.0 - (1.0 - k / alive) ** rows)     # distinct experts of `rows` tokens
    per = 3 * i * h + 4 * (2 * _blocks(i) * _blocks(h) + _blocks(h) * _blocks(i))
    return {"bytes": active * per + 4 * t * h + 4 * t * e + 8 * t * case["top_k"],
            "flops": 6 * rows * k * h * i}


# ------------------------------------------------------------------ the definitions in 64 bits
def _table(dev):
    """Values of the 256 E4M3 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    c = torch.arange(256, device=dev)
    e, m = ((c >> 3) & 15).double(), (c & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6)
    v = torch.where((c & 127) == 127, torch.full_like(v, math.nan), v)
    return torch.where(c >= 128, -v, v)


def _spread(s, dim, n):
    """A scale for every element along `dim`, from one for every 128."""
    return s.double().index_select(dim, torch.arange(n, device=s.device) // BLOCK)


def _exact_quantize(x, rows_per_block):
    """Codes' values and scales [row blocks, K blocks] of a 2-D matrix."""
    n, k = x.shape
    v = x.double()
    at_n = torch.arange(n, device=x.device) // rows_per_block
    at_k = torch.arange(k, device=x.device) // BLOCK
    cell = at_n[:, None] * _blocks(k) + at_k[None, :]
    amax = torch.zeros(-(-n // rows_per_block) * _blocks(k), dtype=torch.float64, device=x.device)
    amax.scatter_reduce_(0, cell.reshape(-1), v.abs().reshape(-1), "amax")
    s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax)).float().double()
    r = (v / s[cell]).float().double()                       # the fp32 quotient
    _, e = torch.frexp(r)                                    # |r| in [2^(e-1), 2^e)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)    # spacing of E4M3 there
    r = (torch.round(r / step) * step).clamp(-448.0, 448.0)  # torch.round: half to even
    return r, s.view(-1, _blocks(k)).float()


def _exact_product(a, sa, qw, sw, table):
    """a[M, K] code values with scales [K blocks, M], weight codes [N, K]."""
    n, k = qw.shape
    w = table[qw.long()] * _spread(_spread(sw, 0, n), 1, k)
    return (a * _spread(sa, 0, k).t()) @ w.t()


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op in ("quantize", "quantize_weight"):
        q, s = _exact_quantize(st["x" if op == "quantize" else "w"], 1 if op == "quantize" else BLOCK)
        return {"codes": q, "scale": s.t().contiguous() if op == "quantize" else s}
    dev = st["y"].device
    table = _table(dev)
    if op == "gemm":
        return {"y": _exact_product(table[st["qa"].long()], st["sa"], st["qw"], st["sw"], table)}
    if op == "linear":
        q, s = _exact_quantize(st["x"], 1)
        s = s.t().contiguous()
        return {"y": _exact_product(q, s, st["qw"], st["sw"], table), "codes": q, "scale": s}
    x, logits, top_k = st["x"].double(), st["logits"].double().cpu(), st["top_k"]
    experts, _, inter, hidden = st["w13"].shape
    tokens = x.shape[0]
    ids = torch.full((tokens, top_k), -1, dtype=torch.int32)
    weights = torch.zeros(tokens, top_k, dtype=torch.float64)
    for t in range(tokens):
        row = logits[t].tolist()
        best = sorted((e for e in range(experts) if row[e] > -math.inf), key=lambda e: (-row[e], e))
        over = best[:top_k] if st["renormalize"] else best
        total = sum(math.exp(row[e] - row[best[0]]) for e in over)
        for j, e in enumerate(best[:top_k]):
            ids[t, j] = e
            weights[t, j] = math.exp(row[e] - row[best[0]]) / total
    y = torch.zeros(tokens, hidden, dtype=torch.float64, device=dev)
    for e in range(experts):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not len(t):
            continue
        pair = [table[st["w13"][e, c].long()] * _spread(_spread(st["s13"][e, c], 0, inter), 1, hidden)
                for c in (0, 1)]
        g, u = (x[t.to(dev)] @ w.t() for w in pair)
        down = table[st["w2"][e].long()] * _spread(_spread(st["s2"][e], 0, hidden), 1, inter)
        y.index_add_(0, t.to(dev), weights[t, j].to(dev)[:, None] * ((g / (1 + torch.exp(-g)) * u) @ down.t()))
    return {"y": y, "ids": ids.to(dev), "weights": weights.to(dev)}

"""Plain 64-bit forms of the paged FP8 cache's operators on the host, and how far a result may
lie from them.  Loops over sequences, heads and pages; shares no code with the kernels."""
import math

import torch

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}     # half a step
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half a step of subnormals
LOW, HIGH = 2.0 ** -100, 2.0 ** 100


def e4m3_table():
    c = torch.arange(256)
    e, m = ((c >> 3) & 15).double(), (c & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6)
    v = torch.where((c & 127) == 127, torch.full_like(v, math.nan), v)
    return torch.where(c >= 128, -v, v)


TABLE = e4m3_table()


def e4m3_codes(v):
    """float64 values -> codes: one rounding, ties to even, saturation; NaN -> 0x7F."""
    code = torch.zeros(v.shape, dtype=torch.int64)
    a = v.abs().clamp(max=448.0)
    _, e = torch.frexp(a)
    e = (e - 1).clamp(min=-6)
    n = torch.round(a / torch.exp2(e.double() - 3)).long()        # eighths of 2^e
    up = n >= 16
    e, n = torch.where(up, e + 1, e), torch.where(up, n // 2, n)
    code = torch.where(n >= 8, (e.long() + 7) * 8 + n - 8, n)     # normal, or subnormal (e = -6)
    code = torch.where(torch.signbit(v), code + 128, code)
    return torch.where(torch.isnan(v), torch.full_like(code, 127), code).to(torch.uint8)


def clamp_scale(s):
    s = torch.nan_to_num(s.double(), nan=LOW, posinf=HIGH, neginf=LOW)
    return s.clamp(LOW, HIGH)


class Batch:
    """A cache and a batch on the host; `new` and `lens` per sequence.  Pages are handed out in a
    shuffled order; page_table has -1 behind a sequence's last page."""

    def __init__(self, new, lens, kv_heads, dim, page, seed, spare=2, lead=0, tail=0, width=None):
        g = torch.Generator().manual_seed(seed)
        self.new, self.lens, self.page, self.kv_heads, self.dim = new, lens, page, kv_heads, dim
        need = [-(-x // page) for x in lens]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        self.width = width or max(1, max(need))
        table = torch.full((len(new), self.width), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            for j in range(n):
                table[b, j] = order.pop()
        self.table = table
        self.q_start = torch.tensor([lead + sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32)
        self.kv_lens = torch.tensor(lens, dtype=torch.int32)
        self.tokens = lead + sum(new) + tail
        self.max_q = max(1, max(new))
        self.gen = g
        # any bytes but the codes of NaN; scales of pages nobody has are NaN
        shape = (self.pages, kv_heads)
        self.k = self._codes((*shape, page, dim))
        self.v = self._codes((*shape, dim, page))
        self.ks = torch.exp2(torch.randint(-9, -5, shape, generator=g).float())
        self.vs = torch.exp2(torch.randint(-9, -5, shape, generator=g).float())
        for p in order:
            self.ks[p] = math.nan
            self.vs[p] = math.inf

    def _codes(self, shape):
        x = torch.randn(shape, generator=self.gen) * 60
        return e4m3_codes(x.double())

    def values(self, heads, dtype, spread=1.0):
        x = torch.randn(self.tokens, heads, self.dim, generator=self.gen) * spread
        return x.to(dtype)

    def seqs(self):
        for b, (n, length) in enumerate(zip(self.new, self.lens)):
            yield b, int(self.q_start[b]), n, length


def rope_table(rows, dim, seed=0):
    half = dim // 2
    turn = torch.arange(rows, dtype=torch.float64)[:, None] * \
        torch.exp2(-13.2877 * torch.arange(half, dtype=torch.float64) / max(1, half)) + seed
    return torch.cat([turn.cos(), turn.sin()], dim=1).float()


def rotate(x, row, interleaved):
    """x [H, D] float64, row: one position's cosines and sines; fp32 roundings as documented."""
    half = row.numel() // 2
    y = x.clone()
    f = lambda v: v.float().double()                                               # noqa: E731
    for i in range(half):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        a, b, c, s = x[:, ia], x[:, ib], row[i].double(), row[half + i].double()
        y[:, ia], y[:, ib] = f(f(a * c) - f(b * s)), f(f(b * c) + f(a * s))
    return y


def append(bt, k, v, rope=None, interleaved=False, q=None):
    """Changes bt's cache; returns the rotated queries in 64 bits (rows outside the batch: NaN)."""
    qo = torch.full(q.shape, math.nan, dtype=torch.float64) if q is not None else None
    for b, row0, n, length in bt.seqs():
        turned = {}
        for i in range(n):
            p = length - n + i
            if p < 0:
                continue
            row = rope[p] if rope is not None else torch.zeros(0)
            turned[p] = {"k": rotate(k[row0 + i].double(), row, interleaved), "v": v[row0 + i].double()}
            if q is not None:
                qo[row0 + i] = rotate(q[row0 + i].double(), row, interleaved)
        for slot in sorted({p // bt.page for p in turned}):
            pid = int(bt.table[b, slot])
            if not 0 <= pid < bt.pages:
                continue
            mine = [p for p in turned if p // bt.page == slot]
            older = mine[0] - slot * bt.page
            for name, codes, scale in (("k", bt.k, bt.ks), ("v", bt.v.transpose(2, 3), bt.vs)):
                for h in range(bt.kv_heads):
                    x = torch.stack([turned[p][name][h] for p in mine])
                    fin = x[torch.isfinite(x)].abs()
                    amax = float(fin.max()) if fin.numel() else 0.0
                    e = -100
                    while e < 100 and 448.0 * 2.0 ** e < amax:
                        e += 1
                    s = 2.0 ** e
                    if older:
                        was = float(clamp_scale(scale[pid, h]))
                        if was >= s:
                            s = was
                        else:
                            # .float(): the quotient of the scales, as documented
                            ratio = (torch.tensor(was).float() / torch.tensor(s).float()).double()
                            old = TABLE[codes[pid, h, :older].long()] * ratio
                            codes[pid, h, :older] = e4m3_codes(old.float().double())
                    q8 = e4m3_codes((x / s).float().double())
                    codes[pid, h, older:older + len(mine)] = q8
                    scale[pid, h] = s
    return qo


def attend(bt, q, scale, causal=True, window=0):
    """y, lse in 64 bits and their bounds; rows outside the batch: NaN."""
    tokens, heads, dim = q.shape
    group = heads // bt.kv_heads
    y = torch.full(q.shape, math.nan, dtype=torch.float64)
    lse = torch.full((tokens, heads), math.nan, dtype=torch.float64)
    ytol, ltol = torch.zeros_like(y), torch.zeros_like(lse)
    for b, row0, n, length in bt.seqs():
        ids = [int(p) for p in bt.table[b]]
        keys = [t for t in range(length) if 0 <= ids[t // bt.page] < bt.pages]
        at = [(ids[t // bt.page], t % bt.page) for t in keys]
        pg = torch.tensor([p for p, _ in at], dtype=torch.long)
        sl = torch.tensor([s for _, s in at], dtype=torch.long)
        tt = torch.tensor(keys, dtype=torch.long)
        for h in range(bt.kv_heads):
            k = TABLE[bt.k[pg, h, sl].long()] * clamp_scale(bt.ks[pg, h])[:, None]
            v = TABLE[bt.v[pg, h, :, sl].long()] * clamp_scale(bt.vs[pg, h])[:, None]
            for i in range(n):
                p = length - n + i
                see = torch.ones(len(keys), dtype=torch.bool)
                if causal:
                    see = (tt <= p) & ((p - tt < window) if window else True)
                for j in range(h * group, (h + 1) * group):
                    r = row0 + i
                    if not see.any():
                        y[r, j], lse[r, j] = 0.0, -math.inf
                        continue
                    qd = q[r, j].double()
                    z = (k[see] @ qd) * scale
                    # fp32 products are exact; their sum of D terms and a few fp32 operations on it
                    dz = ((k[see].abs() @ qd.abs()) * abs(scale) * (dim + 8) * 2.0 ** -24
                          + z.abs() * 2.0 ** -22).max()
                    lse[r, j] = torch.logsumexp(z, 0)
                    w = torch.exp(z - lse[r, j])
                    y[r, j] = w @ v[see]
                    mass = w @ v[see].abs()
                    # a term is off by its logit's error, its rounding to 11 bits (or, fp16's smallest
                    # half step 2^-25 over 2^9, to 2^-34 of the largest term times scale) and the exponential's; the denominator by the same
                    # without the rounding; sums of fp32
                    rel = 2 * dz + 2.0 ** -11 + 2.0 ** -20 + len(w) * 2.0 ** -24
                    least = (torch.exp(z - z.max()) * clamp_scale(bt.vs[pg[see], h])).max() * \
                        torch.exp(z.max() - lse[r, j]) * 448 * len(w) * 2.0 ** -34
                    ytol[r, j] = mass * rel + least + y[r, j].abs() * EPS[q.dtype] + TINY[q.dtype]
                    ltol[r, j] = dz + 2.0 ** -20 * (1 + lse[r, j].abs()) + len(w) * 2.0 ** -24
    return y, lse, ytol, ltol

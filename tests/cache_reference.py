"""The 8-bit key / value cache on the host: storing by the same roundings in
numpy / torch CPU, attention from the definition in fp64, and the error bound
that the attention kernels are held to."""
import math

import numpy as np
import torch

E4 = torch.float8_e4m3fn


def scale_byte(a):
    """The byte of the smallest e with a <= 448 * 2^e, 255 for NaN and infinity."""
    if not math.isfinite(a):
        return 255
    if a == 0:
        return 0
    m, e = math.frexp(a)
    return min(max(e - 9 + (1 if m > 0.875 else 0) + 127, 0), 254)


def to_codes(x):
    """fp64 tensor within +-448 -> e4m3 codes, nearest even (fp32 holds every
    value used here exactly)."""
    return x.float().to(E4).view(torch.uint8)


class Cache:
    """CPU copies of the four tensors."""

    def __init__(self, pages, heads, page, dim, seed=0):
        g = torch.Generator().manual_seed(seed)
        # whatever the slots held before: every byte, NaN codes and scale bytes included
        self.k = torch.randint(0, 256, (pages, heads, page, dim), dtype=torch.uint8, generator=g)
        self.v = torch.randint(0, 256, (pages, heads, dim, page), dtype=torch.uint8, generator=g)
        self.ks = torch.randint(0, 256, (pages, heads), dtype=torch.uint8, generator=g)
        self.vs = torch.randint(0, 256, (pages, heads), dtype=torch.uint8, generator=g)
        self.page, self.heads, self.dim, self.pages = page, heads, dim, pages

    def tensors(self):
        return self.k, self.ks, self.v, self.vs

    def append(self, table, q_start, ctx_len, K, V, max_q=1 << 30):
        P, reach = self.page, table.shape[1] * self.page
        for s in range(table.shape[0]):
            q0, n = int(q_start[s]), int(q_start[s + 1] - q_start[s])
            first = int(ctx_len[s]) - n
            last = min(int(ctx_len[s]), reach, first + min(n, max_q, K.shape[0] - q0))
            for pg in range(max(first, 0) // P, -(-max(last, 0) // P)):
                a, b = max(first, 0, pg * P) - pg * P, min(last, pg * P + P) - pg * P
                at = int(table[s, pg])
                if a >= b or not 0 <= at < self.pages:
                    continue
                row = q0 + pg * P + a - first
                for X, codes, scales, turned in ((K, self.k, self.ks, False), (V, self.v, self.vs, True)):
                    for h in range(self.heads):
                        x = X[row:row + b - a, h].double()
                        page = codes[at, h].t() if turned else codes[at, h]
                        bits = scale_byte(float(x.abs().max()) if not x.isnan().any() else math.nan)
                        was = int(scales[at, h])
                        if a > 0:
                            bits = max(bits, was)
                            if bits > was and bits < 255:
                                old = page[:a].contiguous().view(E4).double() * 2.0 ** (was - bits)
                                page[:a] = to_codes(old)
                        page[a:b] = 0 if bits == 255 else to_codes(x * 2.0 ** (127 - bits))
                        scales[at, h] = bits


def attend(c, table, q_start, ctx_len, Q, scale, window, sinks):
    """(O, lse, bound of |O - exact|, bound of |lse - exact|) in fp64, NaN in
    rows of no sequence.  The bound: probabilities are rounded to bf16 (2^-8
    of each at most) and the output too; a score is a sum of D exact products
    in fp32 (D / 32 MFMA roundings, its scales, the subtraction and the
    exponential: 12 half steps of fp32 relative to sum |q k|), which moves p
    by as much, relatively."""
    T, Hq, D = Q.shape
    G = Hq // c.heads
    O = torch.full((T, Hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    to, tl = torch.zeros_like(O), torch.zeros_like(lse)
    P = c.page
    for s in range(table.shape[0]):
        q0, n = int(q_start[s]), int(q_start[s + 1] - q_start[s])
        ctx = min(int(ctx_len[s]), table.shape[1] * P)
        ctx = max(ctx, 0)
        first = int(ctx_len[s]) - n
        ids = table[s, :-(-ctx // P)].long()
        bad = (ids < 0) | (ids >= c.pages)
        ids = ids.clamp(0, c.pages - 1)
        pos = torch.arange(first, first + n)[:, None]
        key = torch.arange(ctx)
        see = (key <= pos) & ~bad.repeat_interleave(P)[:ctx]
        if window:
            see &= (key > pos - window) | (key < sinks)
        for h in range(c.heads):
            k = c.k[ids, h].view(E4).double() * pow2(c.ks[ids, h])[:, None, None]
            v = c.v[ids, h].view(E4).double() * pow2(c.vs[ids, h])[:, None, None]
            k, v = k.reshape(-1, D)[:ctx], v.transpose(1, 2).reshape(-1, D)[:ctx]
            none = ~see.any(0)                        # keys no row sees may hold anything
            k, v = k.masked_fill(none[:, None], 0.0), v.masked_fill(none[:, None], 0.0)
            for j in range(G):
                q = Q[q0:q0 + n, h * G + j].double()
                x = (q @ k.t() * scale).masked_fill(~see, -math.inf)
                es = (12 * 2.0 ** -24 * abs(scale) * (q.abs() @ k.abs().t())).masked_fill(~see, 0)
                es = es.amax(1, keepdim=True) if ctx else torch.zeros((n, 1), dtype=torch.float64)
                l = torch.logsumexp(x, 1) if ctx else torch.full((n,), -math.inf, dtype=torch.float64)
                es = es.nan_to_num(0.0)
                p = torch.exp(x - l[:, None]).masked_fill(~see, 0.0)      # a row of NaN where a visible score is
                p = p.masked_fill(l[:, None] == -math.inf, 0.0)
                o = p @ v.nan_to_num(0.0)
                # a visible value of a NaN page makes its row NaN, an invisible one nothing
                o = o.masked_fill((see & v.isnan().any(1)).any(1)[:, None], math.nan)
                r = slice(q0, q0 + n)
                O[r, h * G + j], lse[r, h * G + j] = o, l
                a = p @ v.nan_to_num(0.0).abs()
                t = (2.0 ** -8 + 2 * es + (ctx / 16 + 64) * 2.0 ** -24) * a
                to[r, h * G + j] = t + 2.0 ** -8 * (o.abs() + t) + 1e-37
                tl[r, h * G + j] = es[:, 0] + 8 * 2.0 ** -23 * (1 + l.abs().nan_to_num(posinf=0, neginf=0)) + \
                    (ctx / 16) * 2.0 ** -24
    return O, lse, to, tl


def pow2(b):
    x = torch.exp2(b.double() - 127)
    return torch.where(b == 255, torch.full_like(x, math.nan), x)


def batch(S, n, ctx, page, seed, extra=3, spread=True):
    """(table, q_start, ctx_len, pages) of S sequences with n[s] new tokens and ctx[s] in all."""
    need = [max(1, -(-c // page)) for c in ctx]
    pages = sum(need) + extra
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((S, max(need)), -1, dtype=torch.int32)
    at = 0
    for s in range(S):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
    q = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32)
    return table, q, torch.tensor(ctx, dtype=torch.int32), pages

"""Timed cases of the block-128 product, its quantization, and the 8-bit
key/value cache (append, attention, attention with a window and sinks).

``run`` computes each operator in plain torch (fp32 arithmetic, one rounding
at the end) while ``own`` is false, and through this repository's library
when it is true.  ``exact`` evaluates the definitions in fp64.

Operators:
  product   C = (A * sa) @ (B * sb)^T, fp8 codes, fp32 scales: A one scale per
            row and 128 K, B one per 128 x 128 block (a weight) or per row and
            128 K (the weight gradient's second factor)
  quantize  fp32 / bf16 matrix -> fp8 codes and fp32 scales, and the codes of
            its transpose (operands of the two products of a backward pass)
  append    new keys and values -> e4m3 codes in cache pages, one e8m0 scale
            byte per page and head
  attend    softmax attention of new queries over such pages, causal, and with
            a window and a few first tokens that stay visible
"""
import math

import torch

own = False

DEV = "cuda:0"
FMT = {"e4m3": 0, "e5m2": 1}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}


def listed():
    return [
        # a linear layer's forward over a long batch of prompts, on the fp8 matrix instructions
        dict(name="product 8192 cube", op="product", M=8192, N=8192, K=8192, fa="e4m3", fb="e4m3",
             rows_b=128, out="bf16", native=True),
        # a decode step's projection: 64 tokens against one large weight
        dict(name="product decode", op="product", M=64, N=28672, K=8192, fa="e4m3", fb="e4m3",
             rows_b=128, out="f32", native=False),
        # a short mixed batch; K ends inside a block of 128
        dict(name="product ragged", op="product", M=333, N=3584, K=4112, fa="e5m2", fb="e4m3",
             rows_b=128, out="bf16", native=False),
        # a weight gradient: the reduction runs over 4096 tokens, fp32 result
        dict(name="product weight gradient", op="product", M=4096, N=4096, K=4096, fa="e5m2",
             fb="e4m3", rows_b=1, out="f32", native=False),
        # an fp32 master weight, quantized for the forward and (transposed) the input gradient
        dict(name="quantize weight", op="quantize", R=28672, K=8192, x="f32", rows=128, fmt="e4m3",
             both=True),
        # a layer's bf16 activations, an odd number of tokens, for the forward and the weight gradient
        dict(name="quantize activations", op="quantize", R=4095, K=8192, x="bf16", rows=1,
             fmt="e4m3", both=True),
        # one new token in each of 128 sequences
        dict(name="append decode", op="append", S=128, n=1, ctx=2048, page=64, kv=8, D=128, x="bf16"),
        # four prompts of up to 2048 tokens entering the cache
        dict(name="append prompts", op="append", S=4, n=2048, ctx=2048, page=64, kv=8, D=128, x="bf16"),
        # a decode step over long contexts of different lengths, 8 query heads a kv head
        dict(name="attend decode", op="attend", S=64, n=1, ctx=8192, page=64, q=64, kv=8, D=128,
             window=0, sinks=0),
        # the last pieces of two prompts entered in pieces
        dict(name="attend prompts", op="attend", S=2, n=2048, ctx=8192, page=64, q=32, kv=8, D=128,
             window=0, sinks=0),
        # a decode step with a window and sinks over contexts far longer than the window
        dict(name="attend window decode", op="attend", S=32, n=1, ctx=32768, page=64, q=32, kv=8,
             D=128, window=4096, sinks=4),
        # the smallest call: three tokens of one short sequence, where latency counts
        dict(name="attend window small", op="attend", S=1, n=3, ctx=77, page=16, q=9, kv=3, D=64,
             window=32, sinks=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "quantize", "append", "attend", "attend"])
    if op == "product":
        rows_b = rng.choice([128, 128, 1])
        c = dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 16, 28672), K=16 * _log(rng, 8, 512),
                 fa=rng.choice(["e4m3", "e5m2"]), fb=rng.choice(["e4m3", "e4m3", "e5m2"]),
                 rows_b=rows_b, out="f32" if rows_b == 1 else rng.choice(["bf16", "bf16", "f32"]))
        c["M"] = max(1, min(c["M"], 8192 ** 3 // (2 * c["N"] * c["K"])))
        c["native"] = c["out"] == "bf16" and rng.random() < 0.5
        return c
    if op == "quantize":
        return dict(op=op, R=_log(rng, 1, 28672), K=16 * _log(rng, 4, 512),
                    x=rng.choice(["f32", "bf16"]), rows=rng.choice([1, 128]),
                    fmt=rng.choice(["e4m3", "e5m2"]), both=rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    kv, D = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128])
    if op == "append":
        ctx = _log(rng, 16, 4096)
        n = rng.choice([1, 1, rng.randint(2, 7), _log(rng, 8, 2048)])
        return dict(op=op, S=_log(rng, 1, 128 if n < 8 else 4), n=min(n, ctx), ctx=ctx, page=page, kv=kv, D=D,
                    x=rng.choice(["bf16", "f32"]))
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    ctx = _log(rng, 16, 32768)
    n = min(ctx, rng.choice([1, 1, rng.randint(2, 9), _log(rng, 16, 2048)]))
    top = 1 << 29  # scores of one pass
    S = max(1, min(_log(rng, 1, 64), top // (n * kv * group * ctx), (1 << 28) // (ctx * kv * D)))
    n = max(1, min(n, top // (S * kv * group * ctx)))
    window = rng.choice([0, 0, _log(rng, 8, 8192)])
    return dict(op=op, S=S, n=n, ctx=ctx, page=page, q=kv * group, kv=kv, D=D, window=window,
                sinks=rng.choice([0, 1, 4, 5]) if window else 0)


# ---- the batch of a cache case: lengths from the case alone --------------------------------


def _lengths(case):
    """(new tokens, context with them) of each sequence: ragged, the first one the longest."""
    n, ctx = [], []
    for s in range(case["S"]):
        c = case["ctx"] - (s * 977) % (case["ctx"] // 2 + 1)
        ctx.append(c)
        n.append(max(1, min(c, case["n"] - (s * 131) % (case["n"] // 4 + 1))))
    return n, ctx


def _visible(case):
    """Pairs (query position, key) that the mask leaves, and keys that some query sees, over all sequences."""
    pairs = keys = 0
    w, k = case["window"], case["sinks"]
    for n, c in zip(*_lengths(case)):
        for p in range(c - n, c):
            lo = max(0, p - w + 1) if w else 0
            pairs += p + 1 - lo + min(k, lo)
        lo = max(0, c - n - w + 1) if w else 0
        keys += c - lo + min(k, lo)
    return pairs, keys


def work(case):
    op = case["op"]
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // 128)
        nb = N if case["rows_b"] == 1 else -(-N // 128)
        return {"bytes": M * K + N * K + 4 * kb * (M + nb) + M * N * (4 if case["out"] == "f32" else 2),
                "flops": 2 * M * N * K}
    if op == "quantize":
        R, K = case["R"], case["K"]
        rb, kb, two = -(-R // 128), -(-K // 128), 2 if case["both"] else 1
        s = rb * kb * two if case["rows"] == 128 else R * kb + (K * rb if case["both"] else 0)
        return {"bytes": R * K * (4 if case["x"] == "f32" else 2) + two * R * K + 4 * s,
                "flops": 2 * two * R * K}
    n, ctx = _lengths(case)
    if op == "append":
        x = 4 if case["x"] == "f32" else 2
        e = 2 * sum(n) * case["kv"] * case["D"]
        return {"bytes": e * (x + 1), "flops": 2 * e}
    pairs, keys = _visible(case)
    rows = sum(n) * case["q"] * case["D"]
    return {"bytes": 2 * keys * case["kv"] * case["D"] + 4 * rows + 4 * sum(n) * case["q"],
            "flops": 4 * pairs * case["q"] * case["D"]}


# ---- inputs ---------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _blocks(x, rows):
    """x (R, K) padded to whole blocks of `rows` x 128 and their largest magnitudes."""
    R, K = x.shape
    rb, kb = -(-R // rows), -(-K // 128)
    y = torch.zeros((rb * rows, kb * 128), dtype=torch.float32, device=x.device)
    y[:R, :K] = x
    return y, y.view(rb, rows, kb, 128).abs().amax(dim=(1, 3))


def _quantized(x, rows, fmt):
    """Codes and fp32 scales of x for blocks of `rows` x 128, as quantize gives them."""
    y, a = _blocks(x, rows)
    a = a.clamp_min(2.0 ** -100)
    inv = FMAX[fmt] / a
    q = (y.view(a.shape[0], rows, a.shape[1], 128) * inv[:, None, :, None]).clamp(-FMAX[fmt], FMAX[fmt])
    q = q.view(y.shape)[:x.shape[0], :x.shape[1]].to(F8[fmt]).contiguous()
    return q, a / FMAX[fmt]


def _scale_byte(a):
    """The e8m0 byte of the smallest e with a <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(a)
    return torch.where(a > 0, e - 9 + (m > 0.875) + 127, torch.zeros_like(e)).clamp(0, 254)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = dict(case)
    if own:
        st["gemm"] = _handle(case.get("native", False))
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        A = torch.randn((M, K), generator=g, device=DEV)
        A *= 1 + 15 * (torch.rand((1, K), generator=g, device=DEV) < 0.002)  # a few channels stand out
        B = torch.randn((N, K), generator=g, device=DEV) * 0.02
        st["A"], st["sa"] = _quantized(A, 1, case["fa"])
        st["B"], st["sb"] = _quantized(B, case["rows_b"], case["fb"])
        st["A"], st["B"] = st["A"].view(torch.uint8), st["B"].view(torch.uint8)
        return st
    if op == "quantize":
        x = torch.randn((case["R"], case["K"]), generator=g, device=DEV) * (0.02 if case["rows"] == 128 else 1.0)
        st["X"] = x if case["x"] == "f32" else x.bfloat16()
        return st
    P, H, D = case["page"], case["kv"], case["D"]
    n, ctx = _lengths(case)
    need = [-(-c // P) for c in ctx]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table, at = torch.zeros((case["S"], max(need)), dtype=torch.int32, device=DEV), 0
    for s, k in enumerate(need):
        table[s, :k] = order[at:at + k]
        at += k
    k = torch.randn((pages, H, P, D), generator=g, device=DEV)
    k *= torch.exp(0.5 * torch.randn((1, H, 1, D), generator=g, device=DEV))  # keys differ by channel
    kb = _scale_byte(k.abs().amax(dim=(2, 3)))
    k *= torch.exp2((127 - kb).float())[:, :, None, None]
    st["k_codes"] = k.to(torch.float8_e4m3fn).view(torch.uint8)
    del k
    v = torch.randn((pages, H, D, P), generator=g, device=DEV)
    vb = _scale_byte(v.abs().amax(dim=(2, 3)))
    v *= torch.exp2((127 - vb).float())[:, :, None, None]
    st["v_codes"] = v.to(torch.float8_e4m3fn).view(torch.uint8)
    del v
    st["k_scales"], st["v_scales"] = kb.to(torch.uint8), vb.to(torch.uint8)
    start = [0]
    for c in n:
        start.append(start[-1] + c)
    st.update(table=table, q_start=torch.tensor(start, dtype=torch.int32, device=DEV),
              ctx_len=torch.tensor(ctx, dtype=torch.int32, device=DEV), max_q=max(n), max_ctx=max(ctx))
    T = start[-1]
    if op == "append":
        dt = torch.float32 if case["x"] == "f32" else torch.bfloat16
        st["K"] = (torch.randn((T, H, D), generator=g, device=DEV) * 1.3).to(dt)
        st["V"] = (torch.randn((T, H, D), generator=g, device=DEV) * 1.3).to(dt)
    else:
        st["Q"] = torch.randn((T, case["q"], D), generator=g, device=DEV).bfloat16()
    if own:
        import level_dsl_amd as L
        st["cache"] = L.KVCache(st["gemm"], st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"])
        st["batch"] = L.Batch(table, st["q_start"], st["ctx_len"], max_q=st["max_q"], max_ctx=st["max_ctx"])
    return st


_handles = {}


def _handle(native):
    """One handle a process and arithmetic, as a program keeps it."""
    if native not in _handles:
        import level_dsl_amd as L
        h = L.Gemm()
        if native:
            h.set_variant(L.MXGEMM_VARIANT_LARGE_NATIVE)
        _handles[native] = h
    return _handles[native]


# ---- the operators ----------------------------------------------------------------------------


def run(st):
    return (_own if own else _plain)[st["op"]](st)


def _own_product(st):
    f32 = st["out"] == "f32"
    C = torch.empty((st["M"], st["N"]), dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
    return st["gemm"].block128(st["A"], st["sa"], FMT[st["fa"]], st["B"], st["sb"], FMT[st["fb"]], C)


def _own_quantize(st):
    out = st["gemm"].quantize_block128(st["X"], FMT[st["fmt"]], rows=st["rows"], transposed=st["both"])
    return [t.view(F8[st["fmt"]]) if t.dtype == torch.uint8 else t for t in out]


def _own_append(st):
    st["cache"].append(st["batch"], st["K"], st["V"])
    return _pages(st)


def _own_attend(st):
    return st["cache"].attend(st["batch"], st["Q"], window=st["window"], sinks=st["sinks"])


def _pages(st):
    return {"k": st["k_codes"].view(torch.float8_e4m3fn), "v": st["v_codes"].view(torch.float8_e4m3fn),
            "k_scales": st["k_scales"], "v_scales": st["v_scales"]}


def _plain_product(st):
    K = st["K"]

    def values(codes, fmt, s, rows):
        s = s.repeat_interleave(128, dim=1)[:, :K]
        if rows == 128:
            s = s.repeat_interleave(128, dim=0)[:codes.shape[0]]
        return codes.view(F8[fmt]).float() * s

    C = values(st["A"], st["fa"], st["sa"], 1) @ values(st["B"], st["fb"], st["sb"], st["rows_b"]).t()
    return C if st["out"] == "f32" else C.bfloat16()


def _plain_quantize(st):
    x, rows, fmt = st["X"].float(), st["rows"], st["fmt"]
    out = list(_quantized(x, rows, fmt))
    if st["both"]:
        pad = -x.shape[0] % 16  # rows of the transpose are padded to 16 codes with zeros
        xt = torch.cat([x, torch.zeros((pad, x.shape[1]), device=DEV)]).t()
        if rows == 128:
            q, s = _quantized(x, rows, fmt)
            q = torch.cat([q.view(torch.uint8), torch.zeros((pad, x.shape[1]), dtype=torch.uint8, device=DEV)])
            out += [q.t().contiguous().view(F8[fmt]), s.t().contiguous()]
        else:
            out += list(_quantized(xt, 1, fmt))
    return out


def _plain_append(st):
    P, S = st["page"], st["S"]
    n, ctx = (st["q_start"][1:] - st["q_start"][:-1]).long(), st["ctx_len"].long()
    first = ctx - n
    k = (st["max_q"] + P - 2) // P + 1
    pg = (first // P)[:, None] + torch.arange(k, device=DEV)
    live = pg * P < ctx[:, None]
    ids = st["table"].gather(1, pg.clamp_max(st["table"].shape[1] - 1)).long()[live]
    pos = (pg[..., None] * P + torch.arange(P, device=DEV))[live]
    seq = torch.arange(S, device=DEV)[:, None].expand(S, k)[live]
    new = (pos >= first[seq, None]) & (pos < ctx[seq, None])
    old = (pos < first[seq, None])
    row = (st["q_start"].long()[seq, None] + pos - first[seq, None]).clamp(0, st["K"].shape[0] - 1)
    for X, codes, scales, turned in ((st["K"], st["k_codes"], st["k_scales"], False),
                                     (st["V"], st["v_codes"], st["v_scales"], True)):
        x = torch.where(new[:, :, None, None], X[row].float(), torch.zeros((), device=DEV)).transpose(1, 2)
        b = _scale_byte(x.abs().amax(dim=(2, 3)))
        was = scales[ids].int()
        b = torch.where(old.any(1)[:, None], torch.maximum(was, b), b)
        have = codes[ids].transpose(2, 3) if turned else codes[ids]
        kept = (have.view(torch.float8_e4m3fn).float() * torch.exp2((was - b).float())[:, :, None, None])
        now = x * torch.exp2((127 - b).float())[:, :, None, None]
        q = torch.where(old[:, None, :, None], kept, now).clamp(-448, 448).to(torch.float8_e4m3fn)
        q = torch.where((old | new)[:, None, :, None], q.view(torch.uint8), have)
        codes[ids] = q.transpose(2, 3) if turned else q
        scales[ids] = b.to(torch.uint8)
    return _pages(st)


def _plain_attend(st):
    S, P, H, D, Hq = st["S"], st["page"], st["kv"], st["D"], st["q"]
    G, nm = Hq // H, st["max_q"]
    q0, ctx = st["q_start"].long(), st["ctx_len"].long()
    n = q0[1:] - q0[:-1]
    ids = st["table"].long()
    L = ids.shape[1] * P
    key = torch.arange(L, device=DEV)
    here = key < ctx[:, None]
    K = st["k_codes"][ids].view(torch.float8_e4m3fn).float()
    K *= torch.exp2(st["k_scales"][ids].float() - 127)[..., None, None]
    K = K.permute(0, 2, 1, 3, 4).reshape(S * H, L, D)
    i = torch.arange(nm, device=DEV)
    row = (q0[:-1, None] + i).clamp_max(st["Q"].shape[0] - 1)
    Q = st["Q"].float()[row].view(S, nm, H, G, D).permute(0, 2, 1, 3, 4).reshape(S * H, nm * G, D)
    s = torch.bmm(Q, K.transpose(1, 2).contiguous()).view(S, H, nm, G, L)
    del K
    s *= D ** -0.5
    pos = (ctx - n)[:, None] + i
    see = (key <= pos[..., None]) & here[:, None]
    if st["window"]:
        see &= (key > pos[..., None] - st["window"]) | (key < st["sinks"])
    s.masked_fill_(~see[:, None, :, None], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    s.sub_(m).exp_()
    l = s.sum(dim=-1, keepdim=True)
    V = st["v_codes"][ids].view(torch.float8_e4m3fn).float()
    V *= torch.exp2(st["v_scales"][ids].float() - 127)[..., None, None]
    V = V.permute(0, 2, 1, 4, 3).reshape(S, H, L, D)
    V = torch.where(here[:, None, :, None], V, torch.zeros((), device=DEV)).view(S * H, L, D)
    o = torch.bmm(s.view(S * H, nm * G, L), V).view(S, H, nm, G, D)
    o = torch.where(l > 0, o / l, torch.zeros_like(o)).permute(0, 2, 1, 3, 4).reshape(S * nm, Hq, D)
    lse = (m + torch.log(l)).squeeze(-1).permute(0, 2, 1, 3).reshape(S * nm, Hq)
    T = st["Q"].shape[0]
    put = torch.where(i < n[:, None], q0[:-1, None] + i, torch.full_like(row, T)).view(-1)
    out = torch.zeros((T + 1, Hq, D), dtype=torch.bfloat16, device=DEV)
    out[put] = o.bfloat16()
    all_lse = torch.zeros((T + 1, Hq), device=DEV)
    all_lse[put] = lse
    return out[:T], all_lse[:T]


_plain = {"product": _plain_product, "quantize": _plain_quantize, "append": _plain_append, "attend": _plain_attend}
_own = {"product": _own_product, "quantize": _own_quantize, "append": _own_append, "attend": _own_attend}


# ---- the definitions in fp64 -----------------------------------------------------------------


def _table64(fmt):
    """The 256 values of a format, from its bit fields."""
    eb, mb, bias = (4, 3, 7) if fmt == "e4m3" else (5, 2, 15)
    t = []
    for c in range(256):
        e, m = (c >> mb) & ((1 << eb) - 1), c & ((1 << mb) - 1)
        if fmt == "e4m3" and (c & 127) == 127:
            v = math.nan
        elif fmt == "e5m2" and e == 31:
            v = math.nan if m else math.inf
        else:
            v = math.ldexp(m, 1 - bias - mb) if e == 0 else math.ldexp((1 << mb) + m, e - bias - mb)
        t.append(-v if c & 128 else v)
    return torch.tensor(t, dtype=torch.float64, device=DEV)


def _grid64(x, fmt):
    """x (fp64) rounded to the nearest value of the format, ties to even, large ones to the largest."""
    mb, low = (3, -6) if fmt == "e4m3" else (2, -14)
    _, e = torch.frexp(x)
    step = torch.exp2((torch.clamp(e - 1, min=low) - mb).double())
    return (torch.round(x / step) * step).clamp(-FMAX[fmt], FMAX[fmt])


def _exact_product(st):
    M, N, K = st["M"], st["N"], st["K"]
    C = torch.zeros((M, N), dtype=torch.float64, device=DEV)
    ta, tb = _table64(st["fa"]), _table64(st["fb"])
    rows = torch.arange(N, device=DEV) // st["rows_b"]
    for b in range(0, K, 128):
        a = ta[st["A"][:, b:b + 128].long()] * st["sa"][:, b // 128, None].double()
        w = tb[st["B"][:, b:b + 128].long()] * st["sb"][rows, b // 128, None].double()
        C.addmm_(a, w.t())
    return C


def _exact_codes(x, rows, fmt):
    """Codes and scales of blocks of `rows` x 128 of the fp64 matrix x."""
    R, K = x.shape
    q = torch.empty_like(x)
    s = torch.empty((-(-R // rows), -(-K // 128)), dtype=torch.float64, device=DEV)
    for b in range(0, K, 128):
        cols = x[:, b:b + 128].abs().amax(dim=1)
        top = torch.zeros(s.shape[0] * rows, dtype=torch.float64, device=DEV)
        top[:R] = cols
        top = top.view(-1, rows).amax(dim=1).clamp_min(2.0 ** -100) / FMAX[fmt]
        s[:, b // 128] = top
        q[:, b:b + 128] = _grid64(x[:, b:b + 128] / top.repeat_interleave(rows)[:R, None], fmt)
    return q, s


def _exact_quantize(st):
    x, rows, fmt = st["X"].double(), st["rows"], st["fmt"]
    q, s = _exact_codes(x, rows, fmt)
    if not st["both"]:
        return [q, s]
    pad = torch.zeros((-x.shape[0] % 16, x.shape[1]), dtype=torch.float64, device=DEV)
    if rows == 128:
        return [q, s, torch.cat([q, pad]).t().contiguous(), s.t().contiguous()]
    return [q, s, *_exact_codes(torch.cat([x, pad]).t().contiguous(), 1, fmt)]


def _exact_append(st):
    t, P = _table64("e4m3"), st["page"]
    out = {"k": t[st["k_codes"].long()], "v": t[st["v_codes"].long()], "k_scales": None, "v_scales": None}
    q0, ctx, table = st["q_start"].tolist(), st["ctx_len"].tolist(), st["table"].tolist()
    for s in range(st["S"]):
        n = q0[s + 1] - q0[s]
        first = ctx[s] - n
        for pg in range(first // P, (ctx[s] - 1) // P + 1):
            a, b, at = max(first, pg * P), min(ctx[s], pg * P + P), table[s][pg]
            for name, X in (("k", st["K"]), ("v", st["V"])):
                x = X[q0[s] + a - first:q0[s] + b - first].double().transpose(0, 1)
                e = torch.ceil(torch.log2(x.abs().amax(dim=(1, 2)) / 448))
                page = out[name][at] if name == "k" else out[name][at].transpose(1, 2)
                if a > pg * P:
                    was = st[name + "_scales"][at].double() - 127
                    e = torch.maximum(e, was)
                    old = page[:, :a - pg * P]
                    old.copy_(_grid64(old * torch.exp2(was - e)[:, None, None], "e4m3"))
                page[:, a - pg * P:b - pg * P] = _grid64(x * torch.exp2(-e)[:, None, None], "e4m3")
    return out


def _exact_attend(st):
    t, P, D, G = _table64("e4m3"), st["page"], st["D"], st["q"] // st["kv"]
    out = torch.zeros(st["Q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(st["Q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    q0, ctx = st["q_start"].tolist(), st["ctx_len"].tolist()
    for s in range(st["S"]):
        n, c = q0[s + 1] - q0[s], ctx[s]
        ids = st["table"][s, :-(-c // P)].long()
        pos = torch.arange(c - n, c, device=DEV)[:, None]
        key = torch.arange(c, device=DEV)
        see = key <= pos
        if st["window"]:
            see &= (pos - key < st["window"]) | (key < st["sinks"])
        for h in range(st["kv"]):
            k = t[st["k_codes"][ids, h].long()] * torch.exp2(st["k_scales"][ids, h].double() - 127)[:, None, None]
            v = t[st["v_codes"][ids, h].long()] * torch.exp2(st["v_scales"][ids, h].double() - 127)[:, None, None]
            k, v = k.reshape(-1, D)[:c], v.transpose(1, 2).reshape(-1, D)[:c]
            for j in range(G):
                x = (st["Q"][q0[s]:q0[s + 1], h * G + j].double() @ k.t()) / math.sqrt(D)
                x = x.masked_fill(~see, -math.inf)
                lse[q0[s]:q0[s + 1], h * G + j] = torch.logsumexp(x, dim=1)
                out[q0[s]:q0[s + 1], h * G + j] = torch.softmax(x, dim=1) @ v
    return out, lse


_exact = {"product": _exact_product, "quantize": _exact_quantize, "append": _exact_append, "attend": _exact_attend}


def exact(case, seed):
    return _exact[case["op"]](prepare(case, seed))

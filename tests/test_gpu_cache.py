"""The 8-bit key / value cache on the GPU: storing tokens bit for bit against
the host's roundings, attention against the definition in fp64 (bounds in
cache_reference.attend)."""
import math

import pytest
import torch

import cache_reference as ref
import level_dsl_amd as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def gemm():
    g = L.Gemm()
    yield g
    g.close()


def upload(gemm, c):
    return L.KVCache(gemm, *(t.to(DEV) for t in c.tensors()))


def same(kv, c):
    for got, want in zip(kv.tensors, c.tensors()):
        assert torch.equal(got.cpu(), want)


def rand(shape, seed, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if spread:
        x *= torch.exp2(spread * torch.randn(shape[:-1] + (1,), generator=g))
    return x


def fill(c, table, q_start, ctx_len, seed, spread=1.0):
    """All ctx_len tokens into the host cache, in three pieces, so that pages
    have been opened and rescaled as they are in use."""
    for cut, done in ((0.3, 0.0), (0.6, 0.3), (1.0, 0.6)):
        a = [int(int(x) * done) for x in ctx_len]
        b = [int(int(x) * cut) for x in ctx_len]
        n = [y - x for x, y in zip(a, b)]
        if not sum(n):
            continue
        q = torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=torch.int32)
        kv = [rand((sum(n), c.heads, c.dim), seed + i + int(10 * cut), spread).bfloat16() for i in (0, 100)]
        c.append(table, q, torch.tensor(b), *kv)


CASES = [  # heads, dim, page, new tokens, contexts
    (1, 64, 16, [1], [1]),
    (2, 64, 16, [1, 5, 17, 0], [33, 5, 40, 9]),
    (3, 128, 32, [70, 1, 33], [70, 32, 97]),
    (2, 128, 64, [1, 64, 130], [65, 128, 200]),
    (1, 64, 128, [129, 2], [300, 128]),
    (8, 128, 64, [1] * 6, [64, 63, 65, 1, 128, 100]),
]


@pytest.mark.parametrize("heads,dim,page,n,ctx", CASES)
@pytest.mark.parametrize("bf16", [False, True])
def test_append(gemm, heads, dim, page, n, ctx, bf16):
    table, q, cl, pages = ref.batch(len(n), n, ctx, page, 7)
    c = ref.Cache(pages, heads, page, dim, 1)
    fill(c, table, q, cl - torch.tensor(n), 3)
    kv = upload(gemm, c)
    K, V = (rand((sum(n) + 2, heads, dim), s, 2.0) for s in (11, 12))
    if bf16:
        K, V = K.bfloat16(), V.bfloat16()
    b = L.Batch(table.to(DEV), q.to(DEV), cl.to(DEV), max_q=max(n))
    c.append(table, q, cl, K, V)
    kv.append(b, K.to(DEV), V.to(DEV))
    same(kv, c)
    kv.append(b, K.to(DEV), V.to(DEV))      # the same tokens again: the same pages
    same(kv, c)


def test_append_strided_and_edges(gemm):
    """Views of a fused projection; an empty sequence; tokens before position
    zero; a table entry that is none; tokens past the table; a bound on the new
    tokens; token matrices that end early; NaN and infinity."""
    heads, dim, page = 2, 64, 16
    table, q, cl, pages = ref.batch(6, [4, 0, 20, 33, 5, 3], [2, 0, 40, 50, 21, 60], page, 3)
    table[2, 1] = -1
    table[3, 3] = 10 ** 6
    cl[5] = 70                                # the table reaches 64
    for max_q, rows in ((33, 70), (7, 70), (33, 50)):
        c = ref.Cache(pages, heads, page, dim, 2)
        for t in c.tensors()[1::2]:
            t[:] = 120                        # bytes whose pages can be rescaled
        for t in c.tensors()[::2]:
            t[:] = t % 127                    # codes that are none of NaN
        kv = upload(gemm, c)
        W = rand((rows, 5 * heads * dim), 4, 1.0)
        W[6, 3] = math.nan
        W[9, heads * dim + 130] = math.inf
        K, V = (W[:, i * heads * dim:(i + 1) * heads * dim].view(rows, heads, dim) for i in (0, 1))
        Wd = W.to(DEV)
        Kd, Vd = (Wd[:, i * heads * dim:(i + 1) * heads * dim].view(rows, heads, dim) for i in (0, 1))
        assert not Kd.is_contiguous()
        c.append(table, q, cl, K, V, max_q)
        kv.append(L.Batch(table.to(DEV), q.to(DEV), cl.to(DEV), max_q=max_q), Kd, Vd)
        same(kv, c)


def run_case(gemm, heads, group, dim, page, n, ctx, window=0, sinks=0, seed=5, scale=None, max_ctx=None,
             spread=1.0, mutate=None, rows_after=2, max_q=None, reach=0):
    table, q, cl, pages = ref.batch(len(n), n, ctx, page, seed)
    c = ref.Cache(pages, heads, page, dim, seed)
    fill(c, table, q, cl, seed, spread)
    if reach > table.shape[1] * page:
        table = torch.nn.functional.pad(table, (0, reach // page - table.shape[1]), value=-1)
    if mutate:
        mutate(c, table)
    T = sum(n) + rows_after
    Q = rand((T, heads * group, dim), seed + 9).bfloat16()
    sc = dim ** -0.5 if scale is None else scale
    O, lse, to, tl = ref.attend(c, table, q, cl, Q, sc, window, sinks)
    kv = upload(gemm, c)
    b = L.Batch(table.to(DEV), q.to(DEV), cl.to(DEV), max_q=max_q or max(max(n), 1), max_ctx=max_ctx or max(max(ctx), 1))
    out = torch.full((T, heads * group, dim), 3.0, dtype=torch.bfloat16, device=DEV)
    ls = torch.full((T, heads * group), 3.0, device=DEV)
    kv.attend(b, Q.to(DEV), scale=scale, window=window, sinks=sinks, out=out, lse=ls)
    torch.cuda.synchronize()
    compare(out, ls, O, lse, to, tl, sum(n))
    return kv, b, Q, out, ls


def compare(out, ls, O, lse, to, tl, T):
    out, ls = out.double().cpu(), ls.double().cpu()
    assert (out[T:] == 3.0).all() and (ls[T:] == 3.0).all(), "rows of no sequence were written"
    out, ls, O, lse, to, tl = (x[:T] for x in (out, ls, O, lse, to, tl))
    assert torch.equal(out.isnan(), O.isnan()) and torch.equal(ls.isnan(), lse.isnan())
    assert torch.equal(ls.isinf(), lse.isinf())
    ok = ~O.isnan()
    bad = ok & ~((out - O).abs() <= to)
    assert not bad.any(), f"{int(bad.sum())} outputs outside, worst {float(((out - O).abs() / to)[ok].max())}"
    ok = lse.isfinite()
    bad = ok & ~((ls - lse).abs() <= tl)
    assert not bad.any(), f"{int(bad.sum())} lse outside, worst {float(((ls - lse).abs() / tl)[ok].max())}"


@pytest.mark.parametrize("heads,group,dim,page,n,ctx", [
    (1, 1, 64, 16, [1], [1]),
    (1, 1, 128, 64, [1], [64]),
    (2, 3, 64, 16, [1, 1, 1], [17, 63, 65]),
    (2, 8, 128, 64, [1, 1, 0, 1], [200, 1, 5, 130]),
    (3, 4, 128, 32, [5, 1, 9], [5, 77, 100]),
    (1, 16, 64, 128, [3, 2], [257, 128]),
    (2, 7, 128, 16, [2, 3], [40, 3]),
    (1, 5, 128, 64, [1, 1], [1500, 700]),
    (1, 20, 64, 32, [2], [1025]),
])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 0), (64, 3), (7, 70), (1, 0)])
def test_attend_few_rows(gemm, heads, group, dim, page, n, ctx, window, sinks):
    run_case(gemm, heads, group, dim, page, n, ctx, window, sinks)


@pytest.mark.parametrize("heads,group,dim,page,n,ctx", [
    (1, 1, 64, 16, [100], [100]),
    (2, 4, 128, 64, [65, 130], [65, 300]),
    (2, 3, 64, 32, [33, 1, 200], [90, 10, 200]),
    (1, 8, 128, 128, [40, 129], [700, 129]),
    (3, 2, 128, 16, [256], [256]),
    (1, 7, 64, 64, [150], [333]),
])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 4), (130, 0)])
def test_attend_prompts(gemm, heads, group, dim, page, n, ctx, window, sinks):
    run_case(gemm, heads, group, dim, page, n, ctx, window, sinks)


def prompt_launch(heads, group, n, ctx, split):
    """Arguments of a batch whose stated bounds (rows, new tokens, context) are
    those of long prompts, so that the kernel for them runs, whole or with its
    keys split, whatever the real lengths."""
    wide = len(n) * heads * group              # rows per new token
    if split:
        rows = min(max(16000 // wide, 2000), 32000 // wide)     # at most 256 tiles of 128 rows
        return {"rows_after": rows, "max_q": rows, "max_ctx": 16384, "reach": 16384}
    blocks = -(-max(ctx) // 64)
    rows = 4 * (16 * 16384 // (blocks * wide) + 16)
    return {"rows_after": rows, "max_q": rows}


@pytest.mark.parametrize("heads,group,dim,page,n,ctx", [
    (1, 1, 64, 16, [100], [100]),
    (2, 4, 128, 64, [65, 130], [65, 300]),
    (2, 3, 64, 32, [33, 1, 200], [90, 10, 200]),
    (1, 8, 128, 128, [40, 129], [700, 129]),
    (3, 2, 128, 16, [256], [256]),
    (1, 7, 64, 64, [150], [333]),
    (1, 3, 128, 64, [5, 3, 0, 70], [2, 0, 40, 40]),
])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 4), (130, 0), (7, 90), (1, 0)])
@pytest.mark.parametrize("split", [False, True])
def test_attend_prompt_kernel(gemm, heads, group, dim, page, n, ctx, window, sinks, split):
    run_case(gemm, heads, group, dim, page, n, ctx, window, sinks, **prompt_launch(heads, group, n, ctx, split))


@pytest.mark.parametrize("dim,page", [(128, 64), (64, 16)])
@pytest.mark.parametrize("sinks", [0, 70])
def test_attend_prompt_kernel_window_split(gemm, dim, page, sinks):
    """A window long enough for its keys to be split."""
    run_case(gemm, 1, 4, dim, page, [150], [1500], 700, sinks, rows_after=8150, max_q=8150)


@pytest.mark.parametrize("split", [False, True])
def test_attend_prompt_kernel_special(gemm, split):
    """Pages of NaN, scale bytes far apart, softmax scales that are large, zero
    and negative, hidden pages."""
    def nan(c, table):
        c.ks[int(table[0, 3]), 0] = 255
        c.vs[int(table[0, 4]), 1] = 255

    def scales(c, table):
        c.vs[int(table[0, 1]), 0] = 167
        c.vs[int(table[0, 2]), 0] = 20
        c.ks[int(table[0, 2]), 0] = 100

    def hide(c, table):
        table[0, 2] = -1
        table[0, 5] = 1 << 20
    for window, sinks in ((0, 0), (20, 17)):
        run_case(gemm, 2, 2, 64, 16, [100], [120], window, sinks, mutate=nan, **prompt_launch(2, 2, [100], [120], split))
        run_case(gemm, 2, 2, 64, 16, [100], [120], window, sinks, mutate=hide, **prompt_launch(2, 2, [100], [120], split))
    one = prompt_launch(1, 2, [50], [100], split)
    run_case(gemm, 1, 2, 64, 32, [40], [100], mutate=scales, **one)
    run_case(gemm, 1, 2, 128, 16, [50], [100], scale=40.0, **one)
    run_case(gemm, 1, 2, 128, 16, [50], [100], scale=0.0, **one)
    run_case(gemm, 1, 2, 128, 16, [50], [100], scale=-0.3, **one)


def test_prompt_kernel_repeats_and_replays(gemm):
    """The same bits again, also from a captured call between eager ones."""
    kv, b, Q, out, ls = run_case(gemm, 1, 4, 128, 64, [70, 200], [90, 500], **prompt_launch(1, 4, [70, 200], [90, 500], True))
    q, dst = Q.to(DEV), torch.zeros_like(out)
    lse = torch.zeros_like(ls)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.attend(b, q, out=dst, lse=lse)
    for _ in range(3):
        dst.zero_()
        graph.replay()
        o2, l2 = kv.attend(b, q)
        torch.cuda.synchronize()
        assert torch.equal(dst[:270], out[:270]) and torch.equal(lse[:270], ls[:270])
        assert torch.equal(o2[:270], out[:270]) and torch.equal(l2[:270], ls[:270])


def test_attend_long_context_splits(gemm):
    """One sequence over a context long enough to be split, its lengths not
    those that shaped the launch."""
    for max_ctx in (6000, 200, 100000):
        run_case(gemm, 1, 4, 128, 64, [1], [6000], max_ctx=max_ctx)
    run_case(gemm, 1, 4, 64, 16, [3, 1], [4097, 2], window=1000, sinks=5)


@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 3)])
def test_attend_few_rows_over_many_keys(gemm, window, sinks):
    """More rows than the decode kernel takes, few enough that the keys are split."""
    run_case(gemm, 1, 8, 128, 64, [20], [3000], window, sinks)
    run_case(gemm, 2, 7, 64, 16, [9, 30], [1500, 40], window, sinks)
    run_case(gemm, 1, 4, 128, 32, [33, 1], [1025, 2000], window, sinks, max_ctx=5000)


def test_attend_rows_that_see_nothing(gemm):
    """More new tokens than the context holds: the first rows lie before
    position zero and get zeros; an empty context; pages that are hidden."""
    heads, dim, page = 2, 64, 16
    table, q, cl, pages = ref.batch(3, [5, 3, 4], [2, 0, 40], page, 3)
    table[2, :2] = -7
    c = ref.Cache(pages, heads, page, dim, 4)
    fill(c, table, q, torch.tensor([2, 0, 40]), 8)
    Q = rand((12, 4, dim), 1).bfloat16()
    for window, sinks in ((0, 0), (4, 2), (30, 3)):
        O, lse, to, tl = ref.attend(c, table, q, cl, Q, 0.125, window, sinks)
        assert (O[:3] == 0).all() and lse[:3].isinf().all() and (O[5:8] == 0).all()
        kv = upload(gemm, c)
        out, ls = kv.attend(L.Batch(table.to(DEV), q.to(DEV), cl.to(DEV), max_q=5, max_ctx=40), Q.to(DEV),
                            window=window, sinks=sinks)
        compare(out, ls, O, lse, to, tl, 12)


@pytest.mark.parametrize("n", [[1], [100]])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 17)])
def test_attend_nan_pages(gemm, n, window, sinks):
    """A page whose scale byte is 255: the rows that see it are NaN, the
    others are not touched by it.  Unwritten slots hold every byte."""
    def mutate(c, table):
        c.ks[int(table[0, 3]), 0] = 255
        c.vs[int(table[0, 4]), 1] = 255
    run_case(gemm, 2, 2, 64, 16, n, [120], window, sinks, mutate=mutate)


def test_attend_scales_of_all_sizes(gemm):
    """Pages whose values differ by 2^40, and a softmax scale that makes a row
    one-hot."""
    def mutate(c, table):
        c.vs[int(table[0, 1]), 0] = 167
        c.vs[int(table[0, 2]), 0] = 20
        c.ks[int(table[0, 2]), 0] = 100
    run_case(gemm, 1, 2, 64, 32, [1], [100], mutate=mutate)
    run_case(gemm, 1, 2, 64, 32, [40], [100], mutate=mutate)
    run_case(gemm, 1, 2, 128, 16, [2], [100], scale=40.0)
    run_case(gemm, 1, 2, 128, 16, [50], [100], scale=0.0)
    run_case(gemm, 1, 2, 128, 16, [50], [100], scale=-0.3)


def test_attend_row_bound(gemm):
    """New tokens past max_q keep their output rows."""
    heads, dim, page = 1, 64, 16
    table, q, cl, pages = ref.batch(2, [9, 4], [30, 20], page, 3)
    c = ref.Cache(pages, heads, page, dim, 4)
    fill(c, table, q, cl, 8)
    Q = rand((13, 16, dim), 1).bfloat16()
    O, lse, to, tl = ref.attend(c, table, q, cl, Q, 0.125, 0, 0)
    out = torch.full((13, 16, dim), 3.0, dtype=torch.bfloat16, device=DEV)
    ls = torch.full((13, 16), 3.0, device=DEV)
    kv = upload(gemm, c)
    kv.attend(L.Batch(table.to(DEV), q.to(DEV), cl.to(DEV), max_q=5), Q.to(DEV), out=out, lse=ls)
    keep = [0, 1, 2, 3, 4, 9, 10, 11, 12]
    assert (out[5:9] == 3.0).all() and (ls[5:9] == 3.0).all()
    compare(out[keep], ls[keep], *(x[keep] for x in (O, lse, to, tl)), 9)


@pytest.mark.parametrize("n", [[1, 2], [70, 1]])
def test_attend_shared_pages(gemm, n):
    """Two sequences that read the same first pages, one of them twice."""
    heads, dim, page = 2, 64, 16
    table, q, cl, pages = ref.batch(2, n, [150, 100], page, 3)
    c = ref.Cache(pages, heads, page, dim, 4)
    fill(c, table, q, cl, 8)
    table[1, :4] = table[0, :4]
    table[1, 4] = table[0, 0]
    Q = rand((sum(n), 8, dim), 1).bfloat16()
    O, lse, to, tl = ref.attend(c, table, q, cl, Q, 0.125, 0, 0)
    out, ls = upload(gemm, c).attend(L.Batch(table.to(DEV), q.to(DEV), cl.to(DEV), max_q=max(n)), Q.to(DEV))
    compare(out, ls, O, lse, to, tl, sum(n))


@pytest.mark.parametrize("n", [[1, 3], [60, 9]])
@pytest.mark.parametrize("page,dim", [(64, 128), (16, 64)])
def test_pages_past_32_bits(gemm, n, page, dim):
    """Pages whose bytes lie past 2^32 of the codes: stored and read as the same
    pages of a small cache."""
    heads = 4
    table, q, cl, pages = ref.batch(2, n, [150, 100], page, 3)
    c = ref.Cache(pages, heads, page, dim, 4)
    fill(c, table, q, cl - torch.tensor(n), 8)
    K, V, Q = (rand((sum(n), h, dim), s).bfloat16().to(DEV) for h, s in ((heads, 1), (heads, 2), (8, 3)))
    base = 2 ** 32 // (heads * page * dim) + 1
    small, big = upload(gemm, c), L.KVCache.empty(gemm, base + pages, page, heads, dim)
    for t, x in zip(big.tensors, small.tensors):
        t[base:] = x
    assert big.tensors[0][base:].data_ptr() - big.tensors[0].data_ptr() > 2 ** 32
    got = []
    for kv, at in ((small, 0), (big, base)):
        b = L.Batch((table + at).to(DEV), q.to(DEV), cl.to(DEV), max_q=max(n))
        kv.append(b, K, V)
        got.append(kv.attend(b, Q))
    assert all(torch.equal(t[base:], x) for t, x in zip(big.tensors, small.tensors))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert not big.tensors[0][:base].any() and not big.tensors[2][:base].any()


def test_attend_strided_heads(gemm):
    """Q as a view of a fused projection, out as a view of a wider buffer."""
    kv, b, Q, out, ls = run_case(gemm, 2, 2, 64, 16, [3, 20], [30, 25], rows_after=0)
    wide = torch.zeros((23, 10, 64), dtype=torch.bfloat16, device=DEV)
    wide[:, 3:7] = Q.to(DEV)
    dst = torch.full((23, 6, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    got, ls2 = kv.attend(b, wide[:, 3:7], out=dst[:, 1:5])
    assert torch.equal(got, out) and torch.equal(ls2, ls)
    assert (dst[:, 0] == 5.0).all() and (dst[:, 5] == 5.0).all()


def test_refusals(gemm):
    kv = L.KVCache.empty(gemm, 4, 16, 2, 64)
    t = torch.zeros((1, 4), dtype=torch.int32, device=DEV)
    q, c = torch.tensor([0, 2], dtype=torch.int32, device=DEV), torch.tensor([2], dtype=torch.int32, device=DEV)
    b = L.Batch(t, q, c, max_q=2)
    K = torch.zeros((2, 2, 64), device=DEV)
    Q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device=DEV)
    for args in ((t[0], q, c), (t, c, c), (t, q, q), (t.long(), q, c), (t.cpu(), q, c), (t, q.float(), c)):
        with pytest.raises(ValueError):
            L.Batch(*args, max_q=2)
    for k, v in ((K.half(), K.half()), (K, K.bfloat16()), (K[:, :1], K[:, :1]), (K.cpu(), K.cpu()),
                 (K.transpose(0, 1), K.transpose(0, 1)), (K[..., ::2], K[..., ::2]), (K, K[:1])):
        with pytest.raises(ValueError):
            kv.append(b, k, v)
    for x, kw in ((Q.float(), {}), (Q[0], {}), (Q.cpu(), {}), (Q[..., :32], {}), (Q, {"out": Q.float()}),
                  (Q, {"out": Q[:1]}), (Q, {"lse": torch.zeros((2, 3), device=DEV)}),
                  (Q, {"lse": torch.zeros((2, 4), device=DEV).double()})):
        with pytest.raises(ValueError):
            kv.attend(b, x, **kw)
    for x, kw in ((Q[:, :3].contiguous(), {}), (Q, {"window": -1}), (Q, {"sinks": 2}), (Q, {"out": Q}),
                  (Q, {"scale": math.inf})):
        with pytest.raises(L.MxgemmError):
            kv.attend(b, x, **kw)
    ks = kv.tensors
    for bad in ((ks[0].float(), *ks[1:]), (ks[0], ks[1][:3], *ks[2:]), (ks[0], ks[1], ks[0], ks[3]),
                (ks[0].cpu(), *ks[1:])):
        with pytest.raises(ValueError):
            L.KVCache(gemm, *bad)
    assert kv.append(b, K[:0], K[:0]) is None
    assert kv.attend(b, Q[:0])[0].shape == (0, 4, 64)


def test_serving_run(gemm):
    """Prompts entered in two pieces, then decode steps, as a server runs them:
    projection by the block-128 product, append, attend, output projection;
    the decode step captured once and replayed, its lengths and tokens changing
    in the device arrays, with eager work between the replays."""
    S, Hq, H, D, page, hidden = 3, 8, 2, 64, 16, 256
    g = torch.Generator().manual_seed(1)
    wq = torch.randn(((Hq + 2 * H) * D, hidden), generator=g).to(DEV) * 0.1
    wo = torch.randn((hidden, Hq * D), generator=g).to(DEV) * 0.1
    qkv_w, out_w = gemm.quantize_block128(wq, 0, rows=128), gemm.quantize_block128(wo, 0, rows=128)

    def layer(kv, batch, x):
        T = x.shape[0]
        xq, xs = gemm.quantize_block128(x, 0)
        p = gemm.block128(xq, xs, 0, qkv_w[0], qkv_w[1], 0,
                          torch.empty((T, (Hq + 2 * H) * D), dtype=torch.bfloat16, device=DEV))
        p = p.view(T, Hq + 2 * H, D)
        kv.append(batch, p[:, Hq:Hq + H], p[:, Hq + H:])
        o, _ = kv.attend(batch, p[:, :Hq], window=24, sinks=2)
        oq, os_ = gemm.quantize_block128(o.view(T, Hq * D), 0)
        return p, gemm.block128(oq, os_, 0, out_w[0], out_w[1], 0,
                                torch.empty((T, hidden), dtype=torch.bfloat16, device=DEV)), o

    table = torch.randperm(S * 5, generator=g).to(torch.int32).view(S, 5)
    host = ref.Cache(S * 5, H, page, D, 5)
    kv = upload(gemm, host)
    ctx = torch.zeros(S, dtype=torch.int32)
    for n in ([10, 3, 21], [7, 16, 1]):
        ctx += torch.tensor(n, dtype=torch.int32)
        q = torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=torch.int32)
        b = L.Batch(table.to(DEV), q.to(DEV), ctx.to(DEV), max_q=max(n), max_ctx=80)
        p, y, o = layer(kv, b, torch.randn((sum(n), hidden), generator=g).bfloat16().to(DEV))
        p = p.cpu()
        host.append(table, q, ctx, p[:, Hq:Hq + H], p[:, Hq + H:])
        same(kv, host)
        want = ref.attend(host, table, q, ctx, p[:, :Hq], D ** -0.5, 24, 2)
        assert ((o.double().cpu() - want[0]).abs() <= want[2]).all()

    q = torch.arange(S + 1, dtype=torch.int32)
    x, dctx = torch.zeros((S, hidden), dtype=torch.bfloat16, device=DEV), ctx.to(DEV)
    b = L.Batch(table.to(DEV), q.to(DEV), dctx, max_q=1, max_ctx=80)
    saved = [t.clone() for t in kv.tensors]
    dctx += 1
    layer(kv, b, x)                          # warm up, then undo
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gp, gy, go = layer(kv, b, x)
    for t, s in zip(kv.tensors, saved):
        t.copy_(s)
    dctx -= 1
    for step in range(4):
        x.copy_(torch.randn((S, hidden), generator=g))
        dctx += 1
        ctx += 1
        graph.replay()
        torch.cuda.synchronize()
        p = gp.cpu()
        host.append(table, q, ctx, p[:, Hq:Hq + H], p[:, Hq + H:])
        same(kv, host)
        want = ref.attend(host, table, q, ctx, p[:, :Hq], D ** -0.5, 24, 2)
        assert ((go.double().cpu() - want[0]).abs() <= want[2]).all()
        replayed = gy.clone()
        _, y, o = layer(kv, b, x)            # eager: the same tokens again
        assert torch.equal(y, replayed) and torch.equal(o, go)
        same(kv, host)


def test_two_streams(gemm):
    """Two caches on two streams at once give what they give alone."""
    a = run_case(gemm, 2, 8, 128, 64, [1, 1], [3000, 2500], seed=5)
    c = run_case(gemm, 2, 8, 128, 64, [1, 1], [2000, 2900], seed=6)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    qa, qc = a[2].to(DEV), c[2].to(DEV)
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        got.append((a[0].attend(a[1], qa, stream=s1), c[0].attend(c[1], qc, stream=s2)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x[0][:2], a[3][:2]) and torch.equal(y[0][:2], c[3][:2])
        assert torch.equal(x[1][:2], a[4][:2]) and torch.equal(y[1][:2], c[4][:2])


def run_prompt_both(gemm, heads, group, dim, page, n, ctx, window=0, sinks=0, seed=5, scale=None, mutate=None):
    """The prompt kernel with its keys split, then whole, against the definition.
    The stated bounds (new tokens, context) are those of long prompts; that
    the prompt kernel is the one they choose is read off the workspace, whose
    parts are tiles of 128 rows (of 16 in the other kernel).  The unsplit run
    is the same call without a workspace."""
    table, q, cl, pages = ref.batch(len(n), n, ctx, page, seed)
    c = ref.Cache(pages, heads, page, dim, seed)
    fill(c, table, q, cl, seed)
    reach = 16384
    table = torch.nn.functional.pad(table, (0, reach // page - table.shape[1]), value=-1)
    if mutate:
        mutate(c, table)
    Hq, wide = heads * group, len(n) * heads
    rows = 250 // wide * 128 // group - 11
    T = max(rows, sum(n) + 2)
    Q = rand((T, Hq, dim), seed + 9).bfloat16()
    used = sum(n) + 2                        # the rows past the last sequence's need no reference
    sc = dim ** -0.5 if scale is None else scale
    O, lse, to, tl = ref.attend(c, table, q, cl, Q[:used], sc, window, sinks)
    to += lost(c, table, q, cl, used, group)
    kv = upload(gemm, c)
    b = L.Batch(table.to(DEV), q.to(DEV), cl.to(DEV), max_q=rows, max_ctx=reach)
    st = b.struct(kv, T)
    part = wide * -(-rows * group // 128) * 128 * (dim + 2) * 4
    nbytes = L.mxgemm_cache_attention_workspace(kv.struct, st, Hq, window)
    assert 0 < rows * group % 128 <= 112
    assert nbytes >= 2 * part and nbytes % part == 0, "not the prompt kernel's workspace for two splits or more"
    Qd = Q.to(DEV)
    for split in (True, False):
        out = torch.full((T, Hq, dim), 3.0, dtype=torch.bfloat16, device=DEV)
        ls = torch.full((T, Hq), 3.0, device=DEV)
        if split:
            kv.attend(b, Qd, scale=scale, window=window, sinks=sinks, out=out, lse=ls)
        else:
            L.mxgemm_cache_attention(gemm.h, kv.struct, st, Qd, Hq, Hq * dim, sc, window, sinks, out, Hq * dim, ls,
                                     None, 0)
        torch.cuda.synchronize()
        assert (out[used:] == 3.0).all() and (ls[used:] == 3.0).all()
        compare(out[:used], ls[:used], O, lse, to, tl, sum(n))


def lost(c, table, q_start, ctx_len, T, group):
    """What a row's output may lose where probabilities leave the fp32 range,
    which counts beside values that differ by 2^100 or more.  A probability is
    2^(x - m) with m at most the row's largest score, and is lost below 2^-126.  It
    may be 2^8, and is scaled down when m grows and when the splits' sums meet, by
    factors that are lost below 2^-126 too: at most 2^8 2^-126 of a value, three
    times.  The sum that it is divided by is at least 1, the largest score's own
    term.  Together under 2^-116 of the sum of the values' magnitudes (those in
    slots behind the context are counted along: a bound still)."""
    t = torch.zeros((T, c.heads * group, c.dim), dtype=torch.float64)
    for s in range(table.shape[0]):
        ids = table[s, :-(-int(ctx_len[s]) // c.page)].long()
        ids = ids[(ids >= 0) & (ids < c.pages)]
        for h in range(c.heads):
            v = c.v[ids, h].view(ref.E4).double() * ref.pow2(c.vs[ids, h])[:, None, None]
            t[int(q_start[s]):int(q_start[s + 1]), h * group:(h + 1) * group] = \
                2.0 ** -116 * v.nan_to_num(0.0).abs().sum((0, 2))
    return t


def at_tokens(table, seq, *tokens, page):
    return [int(table[seq, t // page]) for t in tokens]


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (128, 16), (64, 128)])
@pytest.mark.parametrize("n,ctx", [([100, 33], [420, 1000]), ([129], [519])])
def test_attend_prompt_whole_blocks(gemm, dim, page, n, ctx):
    run_prompt_both(gemm, 2, 3, dim, page, n, ctx)


# a window that leaves whole blocks between its edges, alone and with sinks
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("sinks", [0, 3, 200])
def test_attend_prompt_window_blocks(gemm, dim, page, sinks):
    run_prompt_both(gemm, 2, 3, dim, page, [150, 1], [2300, 1700], 1600, sinks)


# tokens of interior blocks, which every row of the prompt sees whole (first
# row at 320 without a window; 880 to 2200 and the sinks with it), and of a
# block that the window's lower edge cuts
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("window,sinks,n,ctx,token", [(0, 0, 100, 420, 70), (0, 0, 100, 420, 200),
                                                     (1500, 130, 100, 2300, 1100), (1500, 130, 100, 2300, 10),
                                                     (1500, 0, 100, 2300, 740)])
def test_attend_prompt_interior_special(gemm, dim, page, window, sinks, n, ctx, token):
    """Pages inside the unmasked blocks of long prompts: a byte of NaN for keys
    (head 0) or values (head 1) makes NaN of exactly the rows and head that see
    it; hidden pages; bytes below 10 and far above 127; and all of them at
    once in neighbouring pages."""
    def at(table, *more):
        return at_tokens(table, 0, token, *(token + page * m for m in more), page=page)

    def nan_key(c, table):
        c.ks[at(table)[0], 0] = 255

    def nan_value(c, table):
        c.vs[at(table)[0], 1] = 255

    def hide(c, table):
        table[0, token // page] = -1

    def far(c, table):
        p = at(table, 1, 2)
        c.vs[p[0], 0], c.vs[p[1], 0], c.vs[p[2], 0] = 3, 190, 9
        c.ks[p[0], 1], c.ks[p[1], 1], c.ks[p[2], 0] = 0, 9, 135

    def tiny(c, table):
        c.vs[:, 0] = 6

    def mixed(c, table):
        hide(c, table)
        c.ks[at_tokens(table, 0, token + page, page=page)[0], 0] = 255
        far_page = at_tokens(table, 0, token + 2 * page, page=page)[0]
        c.vs[far_page, 1] = 200
    for mutate in (nan_key, nan_value, hide, far, tiny, mixed):
        run_prompt_both(gemm, 2, 2, dim, page, [n], [ctx], window, sinks, mutate=mutate)


@pytest.mark.parametrize("scale", [3.0, 0.0, -0.3])
def test_attend_prompt_whole_blocks_scales(gemm, scale):
    run_prompt_both(gemm, 1, 3, 128, 64, [100], [700], scale=scale)
    run_prompt_both(gemm, 1, 3, 64, 16, [100], [700], scale=scale)


@pytest.mark.parametrize("n,ctx", [([2, 1], [40, 9]), ([90, 5], [300, 5])])
def test_rows_before_the_first_sequence(gemm, n, ctx):
    """q_start may begin past zero: the rows before it belong to no sequence."""
    off, heads, dim, page = 3, 2, 64, 16
    table, q, cl, pages = ref.batch(len(n), n, ctx, page, 3)
    c = ref.Cache(pages, heads, page, dim, 4)
    fill(c, table, q, cl - torch.tensor(n), 8)
    T = off + sum(n)
    K, V, Q = (rand((T, h, dim), s).bfloat16() for h, s in ((heads, 1), (heads, 2), (4 * heads, 3)))
    kv = upload(gemm, c)
    c.append(table, q + off, cl, K, V)
    b = L.Batch(table.to(DEV), (q + off).to(DEV), cl.to(DEV), max_q=max(n))
    kv.append(b, K.to(DEV), V.to(DEV))
    same(kv, c)
    out = torch.full((T, 4 * heads, dim), 3.0, dtype=torch.bfloat16, device=DEV)
    ls = torch.full((T, 4 * heads), 3.0, device=DEV)
    kv.attend(b, Q.to(DEV), out=out, lse=ls)
    assert (out[:off] == 3.0).all() and (ls[:off] == 3.0).all()
    compare(out[off:], ls[off:], *(x[off:] for x in ref.attend(c, table, q + off, cl, Q, dim ** -0.5, 0, 0)), sum(n))

"""The block-128 product and its quantization on the GPU.

Product: against the definition in fp64 (codes decoded by torch, scales as
they are).  With S = sum |a b| over the scaled factors, KB = ceil(K / 128):
  fp32 out  |err| <= (KB + 16) 2^-24 S   (4 roundings inside a block's sum, 3
            of its scales, one per block in the running sum, 8 where partial
            sums over parts of K meet, 1 with the previous C)
  bf16 out  + 2^-8 |C|  (half a step of bf16, relative)
  native    + 8 * 2^-13 * (largest |a b| of each 8 products), summed: the fp8
            MFMA keeps 13 bits below a group's largest product
Quantization: bit for bit against the same fp32 operations in numpy, and
against fp64: a code's value is within half a step (relative 2^-4 for e4m3,
2^-3 for e5m2, or half the subnormal step) of x / scale, plus three fp32
roundings.
"""
import numpy as np
import pytest
import torch

import level_dsl_amd as L

pytestmark = pytest.mark.gpu
F8 = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}
FMAX = {0: 448.0, 1: 57344.0}
DEV = "cuda:0"


@pytest.fixture(scope="module")
def gemm():
    g = L.Gemm()
    yield g
    g.close()


def cdiv(a, b):
    return -(-a // b)


def problem(M, N, K, fa, fb, rows_b, seed, finite=True):
    g = torch.Generator().manual_seed(seed)
    def codes(r, k, f):
        c = (torch.randn((r, k), generator=g) * (4.0 if f == 0 else 64.0)).to(F8[f])
        return c.view(torch.uint8)
    A, B = codes(M, K, fa), codes(N, K, fb)
    kb = cdiv(K, 128)
    sa = torch.exp2(torch.randn((M, kb), generator=g) * 2)
    sb = torch.exp2(torch.randn((N if rows_b == 1 else cdiv(N, 128), kb), generator=g) * 2)
    return A, sa, B, sb


def scaled(codes, f, s, rows):
    K = codes.shape[1]
    x = codes.view(F8[f]).double()
    s = s.double().repeat_interleave(128, 1)[:, :K]
    if rows == 128:
        s = s.repeat_interleave(128, 0)[:codes.shape[0]]
    return x * s


def check(gemm, M, N, K, fa=0, fb=0, rows_b=128, bf16=False, acc=False, seed=1, native=False, stream=None,
          where="cpu"):
    """where: the device of the fp64 reference"""
    A, sa, B, sb = problem(M, N, K, fa, fb, rows_b, seed)
    a, b = scaled(A, fa, sa, 1).to(where), scaled(B, fb, sb, rows_b).to(where)
    ref, mag = a @ b.t(), a.abs() @ b.abs().t()
    dt = torch.bfloat16 if bf16 else torch.float32
    pad = 64
    buf = torch.full((M * N + 2 * pad,), 7.0, dtype=dt, device=DEV)
    C = buf[pad:pad + M * N].view(M, N)
    C.fill_(float("nan"))
    if acc:
        C0 = torch.randn((M, N), generator=torch.Generator().manual_seed(seed + 1)).to(dt)
        C.copy_(C0)
        ref, mag = ref + C0.to(where).double(), mag + C0.to(where).double().abs()
    tol = (cdiv(K, 128) + 17) * 2.0 ** -24 * mag
    if native:
        p = torch.zeros_like(mag)
        for k in range(0, K, 8):
            p += (a[:, None, k:k + 8] * b[None, :, k:k + 8]).abs().amax(-1)
        tol += 8 * 2.0 ** -13 * p
    if bf16:
        tol += 2.0 ** -8 * (ref.abs() + tol)
    to = [t.to(DEV) for t in (A, sa, B, sb)]
    gemm.block128(to[0], to[1], fa, to[2], to[3], fb, C, use_acc=acc, stream=stream)
    torch.cuda.synchronize()
    got = C.double().to(where)
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, worst {float(((got - ref).abs() / tol).max())}"
    assert (buf[:pad] == 7.0).all() and (buf[-pad:] == 7.0).all(), "store outside C"
    return got


SMALL = [(1, 1, 16), (1, 130, 128), (3, 16, 144), (16, 32, 112), (17, 33, 256), (64, 96, 1024), (65, 129, 1040),
         (130, 257, 400), (1, 512, 4096), (40, 7, 2064)]


@pytest.mark.parametrize("M,N,K", SMALL)
@pytest.mark.parametrize("rows_b", [1, 128])
@pytest.mark.parametrize("bf16", [False, True])
def test_product_shapes(gemm, M, N, K, rows_b, bf16):
    gemm.set_variant(L.MXGEMM_VARIANT_AUTO)
    check(gemm, M, N, K, rows_b=rows_b, bf16=bf16, seed=M + N)


@pytest.mark.parametrize("variant", [L.MXGEMM_VARIANT_SKINNY, L.MXGEMM_VARIANT_LARGE, L.MXGEMM_VARIANT_LARGE_NATIVE])
@pytest.mark.parametrize("M,N,K", [(300, 520, 1168), (513, 264, 256), (66, 4, 16), (257, 130, 640)])
@pytest.mark.parametrize("fa,fb,rows_b,bf16,acc", [(0, 0, 128, True, False), (1, 0, 1, False, True),
                                                  (0, 1, 128, False, False), (1, 1, 1, True, True)])
def test_product_variants(gemm, variant, M, N, K, fa, fb, rows_b, bf16, acc):
    gemm.set_variant(variant)
    try:
        check(gemm, M, N, K, fa, fb, rows_b, bf16, acc, seed=M + K, native=variant == L.MXGEMM_VARIANT_LARGE_NATIVE)
    finally:
        gemm.set_variant(L.MXGEMM_VARIANT_AUTO)


# the wider small tiles, taken where they still give a workgroup to every CU
@pytest.mark.parametrize("M,N,K", [(20, 16391, 272), (32, 8200, 400), (33, 16390, 144), (64, 8198, 272),
                                   (300, 4104, 1040), (1, 28680, 16)])
@pytest.mark.parametrize("fa,rows_b,bf16,acc", [(0, 128, True, False), (1, 1, False, True)])
def test_product_many_columns(gemm, M, N, K, fa, rows_b, bf16, acc):
    check(gemm, M, N, K, fa, 0, rows_b, bf16, acc, seed=M, where=DEV)


# the fp8 MFMA, taken where 256 x 256 tiles fill the GPU well enough
@pytest.mark.parametrize("M,N,K", [(2600, 2080, 400), (2561, 2310, 144), (2817, 2050, 16), (257, 21000, 1168)])
@pytest.mark.parametrize("fa,fb,rows_b,bf16,acc", [(0, 0, 128, True, False), (1, 0, 1, False, True),
                                                  (0, 1, 128, False, False), (1, 1, 1, True, True)])
def test_product_native(gemm, M, N, K, fa, fb, rows_b, bf16, acc):
    gemm.set_variant(L.MXGEMM_VARIANT_LARGE_NATIVE)
    try:
        got = check(gemm, M, N, K, fa, fb, rows_b, bf16, acc, seed=M + K, native=True, where=DEV)
    finally:
        gemm.set_variant(L.MXGEMM_VARIANT_AUTO)
    assert got.isfinite().all()


# every number of blocks behind the last whole group of four
@pytest.mark.parametrize("variant,M,N", [(L.MXGEMM_VARIANT_LARGE, 257, 130), (L.MXGEMM_VARIANT_LARGE_NATIVE, 2561, 2310)])
@pytest.mark.parametrize("K", [128, 256, 384, 512, 640, 880, 1024, 1920])
@pytest.mark.parametrize("rows_b,bf16,acc", [(128, True, False), (1, False, True)])
def test_product_large_stages(gemm, variant, M, N, K, rows_b, bf16, acc):
    gemm.set_variant(variant)
    try:
        check(gemm, M, N, K, 0, 0, rows_b, bf16, acc, seed=K, native=variant == L.MXGEMM_VARIANT_LARGE_NATIVE, where=DEV)
    finally:
        gemm.set_variant(L.MXGEMM_VARIANT_AUTO)


@pytest.mark.parametrize("variant", [L.MXGEMM_VARIANT_AUTO, L.MXGEMM_VARIANT_SKINNY])
@pytest.mark.parametrize("M", [2 ** 26 - 70, 2 ** 26 + 37])
def test_product_many_rows(gemm, variant, M):
    """As many rows as the small tiles take, and more."""
    A, sa, B, sb = (t.to(DEV) for t in problem(4099, 24, 16, 0, 0, 1, 9))
    n = cdiv(M, 4099)
    gemm.set_variant(variant)
    try:
        got = gemm.block128(A.repeat(n, 1)[:M], sa.repeat(n, 1)[:M], 0, B, sb, 0,
                            torch.empty((M, 24), dtype=torch.bfloat16, device=DEV))
    finally:
        gemm.set_variant(L.MXGEMM_VARIANT_AUTO)
    a, b = scaled(A.cpu(), 0, sa.cpu(), 1), scaled(B.cpu(), 0, sb.cpu(), 1)
    ref, mag = (a @ b.t()).to(DEV), (a.abs() @ b.abs().t()).to(DEV)
    tol = 18 * 2.0 ** -24 * mag
    tol += 2.0 ** -8 * (ref.abs() + tol)
    for at in (0, M // 4099 // 2 * 4099, M // 4099 * 4099 - 4099, M - M % 4099):
        x = got[at:at + 4099].double()
        assert ((x - ref[:len(x)]).abs() <= tol[:len(x)]).all()


def test_product_past_32_bits(gemm):
    """Operand and output bytes past 2^32: the last rows and columns agree with
    the same rows and columns multiplied alone."""
    g = torch.Generator(DEV).manual_seed(3)
    N, K = 140001, 32768
    B = torch.randint(0, 120, (N, K), generator=g, dtype=torch.uint8, device=DEV)
    sb = torch.rand((cdiv(N, 128), K // 128), generator=g, device=DEV)
    A = torch.randint(0, 120, (5, K), generator=g, dtype=torch.uint8, device=DEV)
    sa = torch.rand((5, K // 128), generator=g, device=DEV)
    got = gemm.block128(A, sa, 0, B, sb, 0, torch.empty((5, N), device=DEV))
    n0 = (N - 200) // 128 * 128
    assert n0 * K > 2 ** 32
    a = A.view(F8[0]).double() * sa.double().repeat_interleave(128, 1)
    b = B[n0:].view(F8[0]).double() * sb[n0 // 128:].double().repeat_interleave(128, 1) \
        .repeat_interleave(128, 0)[:N - n0]
    ref = a @ b.t().contiguous()              # codes and scales are positive: the sum of magnitudes too
    assert ((got[:, n0:].double() - ref).abs() <= (K // 128 + 16) * 2.0 ** -24 * ref).all()
    del B, b
    M, N, K = 66000, 33000, 16
    A = torch.randint(0, 120, (M, K), generator=g, dtype=torch.uint8, device=DEV)
    B = torch.randint(0, 120, (N, K), generator=g, dtype=torch.uint8, device=DEV)
    sa, sb = torch.rand((M, 1), generator=g, device=DEV), torch.rand((N, 1), generator=g, device=DEV)
    got = gemm.block128(A, sa, 0, B, sb, 0, torch.empty((M, N), dtype=torch.bfloat16, device=DEV))
    ref = (A[-300:].view(F8[0]).double() * sa[-300:]) @ (B.view(F8[0]).double() * sb).t().contiguous()
    assert ((got[-300:].double() - ref).abs() <= 2.0 ** -8 * ref * 1.01).all()


def test_product_special_values(gemm):
    """A NaN code or scale stays in its row (column), zero scales give zeros
    even beside the largest codes, and infinities meet their sign."""
    A, sa, B, sb = problem(70, 40, 256, 1, 0, 1, 3)
    A[5, 17] = 0x7c    # e5m2 infinity
    A[6, 200] = 0x7e   # NaN
    B[9, 30] = 0x7f    # NaN
    sa[8] = 0.0
    sa[11, 1] = float("nan")
    sb[20] = 0.0
    ref = scaled(A, 1, sa, 1) @ scaled(B, 0, sb, 1).t()
    C = torch.empty((70, 40), device=DEV)
    gemm.block128(A.to(DEV), sa.to(DEV), 1, B.to(DEV), sb.to(DEV), 0, C)
    got = C.double().cpu()
    assert torch.equal(got.isnan(), ref.isnan())
    inf = ref.isinf()
    assert torch.equal(got[inf], ref[inf])
    ok = ~(ref.isnan() | inf)
    assert (got[8][ok[8]] == 0).all() and (got[:, 20][ok[:, 20]] == 0).all()
    mag = scaled(A.clamp(max=0x77), 1, sa.nan_to_num(), 1).abs().nan_to_num(posinf=0) @ \
        scaled(B, 0, sb, 1).abs().nan_to_num().t()
    assert ((got - ref).abs()[ok] <= (18 * 2.0 ** -24 * mag + 1e-30)[ok]).all()


def far_scales(M, N, K, t, size, seed):
    """Codes of magnitude about `size`, and a scale per row of both factors near
    2^t[b] (A) and 2^-t[b] (B) in block b, so that their product is about 1."""
    g = torch.Generator().manual_seed(seed)
    kb = cdiv(K, 128)
    e = torch.tensor([float(t[b % len(t)]) for b in range(kb)])
    A, B = ((torch.randn((r, K), generator=g) * size).to(F8[0]).view(torch.uint8) for r in (M, N))
    sa, sb = (torch.exp2(x) * (1 + 0.9 * torch.rand((r, kb), generator=g)) for r, x in ((M, e), (N, -e)))
    return A, sa, B, sb


# block sums that pass the fp32 range, on either side, if one scale is applied before the other
@pytest.mark.parametrize("variant,M,N", [(L.MXGEMM_VARIANT_SKINNY, 130, 140), (L.MXGEMM_VARIANT_LARGE, 130, 140),
                                         (L.MXGEMM_VARIANT_LARGE, 257, 130),
                                         (L.MXGEMM_VARIANT_LARGE_NATIVE, 2561, 2310)])
@pytest.mark.parametrize("t,size", [((124, -124), 40.0), ((-125,), 2.0 ** -6), ((125,), 2.0 ** -6), ((-125, 90, 0), 4.0)])
def test_product_far_scales(gemm, variant, M, N, t, size):
    """The two scales of an output and block are multiplied first: scales far
    from 1 whose products are not, against the bound of every other call.  (An
    fp8 MFMA's window adds 2^-13 of the largest of each 8 products, at most
    max |a| max |b| of the block's codes times the scales.)"""
    K = 400
    A, sa, B, sb = far_scales(M, N, K, t, size, M + len(t))
    a, b = scaled(A, 0, sa, 1).to(DEV), scaled(B, 0, sb, 1).to(DEV)
    ref, tol = a @ b.t().contiguous(), (cdiv(K, 128) + 16) * 2.0 ** -24 * (a.abs() @ b.abs().t().contiguous())
    if variant == L.MXGEMM_VARIANT_LARGE_NATIVE:
        for k in range(0, K, 8):
            tol += 8 * 2.0 ** -13 * a[:, k:k + 8].abs().amax(1)[:, None] * b[:, k:k + 8].abs().amax(1)
    gemm.set_variant(variant)
    try:
        C = gemm.block128(A.to(DEV), sa.to(DEV), 0, B.to(DEV), sb.to(DEV), 0, torch.empty((M, N), device=DEV))
    finally:
        gemm.set_variant(L.MXGEMM_VARIANT_AUTO)
    bad = ~((C.double() - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, {int((~C.isfinite()).sum())} not finite"


@pytest.mark.parametrize("rows_b", [1, 128])
@pytest.mark.parametrize("variant,M,N", [(L.MXGEMM_VARIANT_SKINNY, 130, 140), (L.MXGEMM_VARIANT_LARGE, 130, 140),
                                         (L.MXGEMM_VARIANT_LARGE_NATIVE, 2561, 2310)])
def test_product_scales_that_overflow(gemm, variant, M, N, rows_b):
    """Where the product of the two scales overflows, a sum of zero gives NaN
    and any other an infinity of its sign, whatever tile the shape takes."""
    K = 256
    A, sa, B, sb = problem(M, N, K, 0, 0, rows_b, 5)
    A[:, 128:] = 0x38                     # 1: the second block's sums are sums of B's row
    B[:, 128:] = 0x38
    B[3, 128:] = 0xb8                     # -1
    B[7, 128:] = 0
    sa[:, 1], sb[:, 1] = 2.0 ** 100, 2.0 ** 100
    sa[0, 1] = 2.0 ** -100                # this row's product is 1
    gemm.set_variant(variant)
    try:
        C = gemm.block128(A.to(DEV), sa.to(DEV), 0, B.to(DEV), sb.to(DEV), 0, torch.empty((M, N), device=DEV)).cpu()
    finally:
        gemm.set_variant(L.MXGEMM_VARIANT_AUTO)
    assert C[0].isfinite().all()
    want = torch.full((N,), float("inf"))
    want[3], want[7] = -float("inf"), float("nan")
    assert torch.equal(C[1:].nan_to_num(nan=5.0), want.nan_to_num(nan=5.0).expand(M - 1, N))


def test_product_refusals(gemm):
    A = torch.zeros((4, 128), dtype=torch.uint8, device=DEV)
    s1, C = torch.ones((4, 1), device=DEV), torch.zeros((4, 4), device=DEV)
    ok = (A, s1, 0, A.clone(), s1, 0, C)
    for i, bad in ((0, A[:, :64]), (1, s1.double()), (1, torch.ones((4, 2), device=DEV)), (3, A.cpu()),
                   (4, torch.ones((3, 1), device=DEV)), (6, C.half()), (6, C[:3]), (0, A.float()),
                   (6, torch.zeros((4, 8), device=DEV)[:, ::2])):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            gemm.block128(*args)
    with pytest.raises(L.MxgemmError):
        gemm.block128(A, s1, 2, A, s1, 0, C)
    gemm.set_variant(L.MXGEMM_VARIANT_SKINNY_NATIVE)
    try:
        with pytest.raises(L.MxgemmError) as e:
            gemm.block128(*ok)
        assert e.value.code == L.STATUS_CODE["MXGEMM_ERR_VARIANT"]
    finally:
        gemm.set_variant(L.MXGEMM_VARIANT_AUTO)


# ---- quantization -----------------------------------------------------------------------------


def np_quantize(x, rows, fmt):
    """Codes and scales of x (fp32 numpy) by the same fp32 operations."""
    R, K = x.shape
    rb, kb = cdiv(R, rows), cdiv(K, 128)
    y = np.zeros((rb * rows, kb * 128), np.float32)
    y[:R, :K] = np.abs(x)
    t = y.reshape(rb, rows, kb, 128)
    a = np.maximum(t.max(axis=(1, 3)), np.float32(2.0 ** -100))
    a = np.where(np.isnan(t).any(axis=(1, 3)), np.float32(np.nan), a)
    scale = (a / np.float32(FMAX[fmt])).astype(np.float32)
    inv = (np.float32(FMAX[fmt]) / a).astype(np.float32)
    with np.errstate(invalid="ignore"):
        q = (x * np.repeat(np.repeat(inv, rows, 0)[:R], 128, 1)[:, :K]).astype(np.float32)
    codes = torch.from_numpy(q).clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt]).view(torch.uint8).numpy()
    return codes, scale


def values(seed, R, K, bf16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((R, K), generator=g) * torch.exp2(torch.randint(-20, 20, (R, 1), generator=g).float())
    x *= torch.exp2(torch.randint(-3, 3, (1, K), generator=g).float())
    if R > 2:
        x[1] = 0.0                       # an empty row
        x[2] *= 2.0 ** -110              # below the smallest scale
        x[R // 2] = torch.where(x[R // 2] > 0, 2.0 ** 120, -2.0 ** 120)
    return x.bfloat16() if bf16 else x


@pytest.mark.parametrize("R,K", [(1, 16), (1, 8192), (5, 144), (128, 128), (129, 272), (300, 1040), (16, 112)])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("bf16", [False, True])
def test_quantize(gemm, R, K, rows, fmt, bf16):
    x = values(R + K, R, K, bf16)
    codes, scales, codes_t, scales_t = (t.cpu().numpy() for t in gemm.quantize_block128(
        x.to(DEV), fmt, rows=rows, transposed=True))
    xf = x.float().numpy()
    want_c, want_s = np_quantize(xf, rows, fmt)
    assert np.array_equal(scales, want_s) and np.array_equal(codes, want_c)
    Rp = cdiv(R, 16) * 16
    pad = np.zeros((Rp, K), np.float32)
    pad[:R] = xf
    if rows == 128:
        want_t = np.zeros((K, Rp), np.uint8)
        want_t[:, :R] = want_c.T
        assert np.array_equal(codes_t, want_t) and np.array_equal(scales_t, want_s.T)
    else:
        want_t, want_st = np_quantize(np.ascontiguousarray(pad.T), 1, fmt)
        assert np.array_equal(codes_t, want_t) and np.array_equal(scales_t, want_st)
    # in 64 bits: within half a step of x / scale
    s = np.repeat(np.repeat(scales.astype(np.float64), rows, 0)[:R], 128, 1)[:, :K]
    got = torch.from_numpy(codes).view(F8[fmt]).double().numpy()
    y = xf.astype(np.float64) / s
    half, sub = (2.0 ** -4, 2.0 ** -10) if fmt == 0 else (2.0 ** -3, 2.0 ** -17)
    assert (np.abs(got - y) <= np.maximum(half * np.abs(y), sub) + 3 * 2.0 ** -23 * np.abs(y)).all()
    # one output pair at a time gives the same bytes
    only = gemm.quantize_block128(x.to(DEV), fmt, rows=rows)
    turn = gemm.quantize_block128(x.to(DEV), fmt, rows=rows, normal=False, transposed=True)
    assert np.array_equal(only[0].cpu().numpy(), codes) and np.array_equal(only[1].cpu().numpy(), scales)
    assert np.array_equal(turn[0].cpu().numpy(), codes_t) and np.array_equal(turn[1].cpu().numpy(), scales_t)


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_past_32_bits(gemm, rows):
    """More than 2^32 elements: the last rows' codes are those that the rows get
    alone, and so are the transpose's."""
    R, K = 2 ** 17 + 200, 2 ** 15 + 16
    x = torch.randn((R, K), dtype=torch.bfloat16, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    c, s, ct, st = gemm.quantize_block128(x, 1, rows=rows, transposed=True)
    r0 = 2 ** 17
    assert c[r0:].data_ptr() - c.data_ptr() > 2 ** 32
    tail = gemm.quantize_block128(x[r0:], 1, rows=rows, transposed=True)
    assert torch.equal(c[r0:], tail[0]) and torch.equal(s[r0 // rows:], tail[1])
    assert torch.equal(ct[:, r0:], tail[2]) and torch.equal(st[:, r0 // 128:], tail[3])


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_quantize_nonfinite(gemm, rows, value):
    """The block that holds a NaN or an infinity decodes to NaN, no other."""
    x = torch.randn((200, 400), generator=torch.Generator().manual_seed(5))
    x[130, 129] = value
    c, s, ct, st = (t.cpu() for t in gemm.quantize_block128(x.to(DEV), 0, rows=rows, transposed=True))
    got = scaled(c, 0, s, rows).isnan()
    want = torch.zeros((200, 400), dtype=torch.bool)
    want[130 if rows == 1 else slice(128, 200), 128:256] = True
    assert torch.equal(got, want)
    got_t = scaled(ct, 0, st, rows).isnan()[:, :200]
    want_t = torch.zeros((400, 200), dtype=torch.bool)
    want_t[129 if rows == 1 else slice(128, 256), 128:200] = True
    assert torch.equal(got_t, want_t)


def test_quantize_refusals(gemm):
    x = torch.zeros((4, 128), device=DEV)
    for bad, kw in ((x.half(), {}), (x.cpu(), {}), (x.t(), {}), (x[0], {}), (x, {"rows": 64}), (x, {"normal": False})):
        with pytest.raises(ValueError):
            gemm.quantize_block128(bad, 0, **kw)
    with pytest.raises(L.MxgemmError):
        gemm.quantize_block128(x, 4)
    with pytest.raises(L.MxgemmError):
        gemm.quantize_block128(torch.zeros((4, 24), device=DEV), 0)


# ---- together -------------------------------------------------------------------------------------


def linear_step(gemm, x, w, dy):
    """Forward and both gradients of y = x w^T on quantized factors: x (T, I),
    w (O, I), dy (T, O)."""
    T, I, O = x.shape[0], x.shape[1], w.shape[0]
    xq, xs, xqt, xst = gemm.quantize_block128(x, 0, rows=1, transposed=True)
    wq, ws, wqt, wst = gemm.quantize_block128(w, 0, rows=128, transposed=True)
    gq, gs, gqt, gst = gemm.quantize_block128(dy, 1, rows=1, transposed=True)
    y = gemm.block128(xq, xs, 0, wq, ws, 0, torch.empty((T, O), dtype=torch.bfloat16, device=DEV))
    dx = gemm.block128(gq, gs, 1, wqt, wst, 0, torch.empty((T, I), dtype=torch.bfloat16, device=DEV))
    dw = gemm.block128(gqt, gst, 1, xqt, xst, 0, torch.empty((O, I), device=DEV))
    return y, dx, dw, (xq, xs, xqt, xst, wq, ws, wqt, wst, gq, gs, gqt, gst)


@pytest.mark.parametrize("T,I,O", [(37, 256, 144), (300, 400, 272)])
def test_linear_layer_step(gemm, T, I, O):
    """A linear layer's forward, input gradient and weight gradient, against the
    formulas in fp64: on the quantized factors within the products' own
    bounds, and dw against differences of the loss <y, dy> in those factors."""
    g = torch.Generator().manual_seed(T)
    x, w, dy = (torch.randn(s, generator=g) for s in ((T, I), (O, I), (T, O)))
    y, dx, dw, q = linear_step(gemm, x.bfloat16().to(DEV), w.to(DEV), dy.bfloat16().to(DEV))
    q = [t.cpu() for t in q]
    xv, wv, gv = scaled(q[0], 0, q[1], 1), scaled(q[4], 0, q[5], 128), scaled(q[8], 1, q[9], 1)
    xt, wt, gt = scaled(q[2], 0, q[3], 1), scaled(q[6], 0, q[7], 128), scaled(q[10], 1, q[11], 1)
    assert torch.equal(wt[:, :O], wv.t())
    for got, a, b in ((y, xv, wv), (dx, gv, wt), (dw, gt, xt)):
        ref, mag = a @ b.t(), a.abs() @ b.abs().t()
        tol = (cdiv(a.shape[1], 128) + 16) * 2.0 ** -24 * mag
        if got.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (ref.abs() + tol)
        assert ((got.double().cpu() - ref).abs() <= tol).all()
    # difference of the loss sum(y * dy) in one weight, with the factors that dw saw: the loss is linear in it
    for o, i in ((0, 0), (O - 1, I - 1), (O // 2, 3)):
        loss = lambda v: float((xt[i, :T] * gt[o, :T] * v).sum())
        d = (loss(1.5) - loss(0.5)) / 1.0
        bound = (cdiv(T, 128) + 16) * 2.0 ** -24 * float((xt[i].abs() * gt[o].abs()).sum())
        assert abs(float(dw[o, i]) - d) <= bound + 1e-12 * abs(d)


def quant_error(x, rows, fmt):
    """Bound of |code * scale - x| for the quantization of x (R, K) in blocks of
    `rows` x 128: half a step of the format (relative, or of its subnormals in
    units of the scale) and three fp32 roundings."""
    R, K = x.shape
    a = torch.zeros((cdiv(R, rows) * rows, cdiv(K, 128) * 128), dtype=torch.float64)
    a[:R, :K] = x.abs()
    top = a.view(-1, rows, cdiv(K, 128), 128).amax(dim=(1, 3))
    s = (top / FMAX[fmt]).repeat_interleave(rows, 0)[:R].repeat_interleave(128, 1)[:, :K]
    half, sub = (2.0 ** -4, 2.0 ** -10) if fmt == 0 else (2.0 ** -3, 2.0 ** -17)
    return torch.maximum(half * x.abs(), sub * s) + 3 * 2.0 ** -23 * x.abs()


@pytest.mark.parametrize("T,I,O", [(256, 256, 256), (37, 272, 144)])
def test_linear_layer_gradients(gemm, T, I, O):
    """y, dx and dw against x w^T, dy w and dy^T x of the factors before their
    quantization, in fp64, and dx and dw against differences of the loss <x w^T,
    dy> taken through the forward.  All entries are positive and their size
    goes up and down along every axis at a pace of its own, so that the bound
    (every factor off by its quantization's half step, the product's own, the
    output's rounding) is a fraction of each result, and a factor that is
    swapped, turned or left out is far outside it."""
    g = torch.Generator().manual_seed(T)
    wave = lambda n, p: torch.exp2((torch.arange(n) % p).double())
    fac = lambda r, c, p, q: (0.5 + torch.rand((r, c), generator=g).double()) * wave(r, p)[:, None] * wave(c, q)
    x, w, dy = fac(T, I, 3, 5).bfloat16(), fac(O, I, 4, 3).float(), fac(T, O, 5, 3).bfloat16()
    y, dx, dw, _ = linear_step(gemm, x.to(DEV), w.to(DEV), dy.to(DEV))
    y, dx, dw = (t.double().cpu() for t in (y, dx, dw))
    x, w, dy = x.double(), w.double(), dy.double()

    def bound(a, ea, b, eb, bf16):
        """of a b^T, a and b off by ea and eb"""
        t = ea @ b.t() + a @ eb.t() + ea @ eb.t()
        ref = a @ b.t()
        t = t + (cdiv(a.shape[1], 128) + 16) * 2.0 ** -24 * (ref + t)
        return ref, t + 2.0 ** -8 * (ref + t) if bf16 else t
    got = {"y": y, "dx": dx, "dw": dw}
    ew = quant_error(w, 128, 0)
    want = {"y": bound(x, quant_error(x, 1, 0), w, ew, True),
            "dx": bound(dy, quant_error(dy, 1, 1), w.t(), ew.t(), True),
            "dw": bound(dy.t(), quant_error(dy.t(), 1, 1), x.t(), quant_error(x.t(), 1, 0), False)}
    for name, (ref, tol) in want.items():
        assert (tol < 0.25 * ref).all()
        assert ((got[name] - ref).abs() <= tol).all(), name
        if T == I == O:         # the bound tells every result from its transpose and from the others
            for other in ("y", "dx", "dw"):
                for r in (want[other][0], want[other][0].t()):
                    assert r is ref or int(((r - ref).abs() > tol).sum()) > T * T // 2
    loss = lambda x, w: float(((x @ w.t()) * dy).sum())
    for o, i in ((0, 0), (O - 1, I - 1), (O // 2, 3)):
        e = torch.zeros_like(w)
        e[o, i] = 0.25
        d = (loss(x, w + e) - loss(x, w - e)) / 0.5
        assert abs(float(dw[o, i]) - d) <= float(want["dw"][1][o, i]) + 1e-6 * abs(d)
    for t, i in ((0, 0), (T - 1, I - 1), (T // 2, 3)):
        e = torch.zeros_like(x)
        e[t, i] = 0.25
        d = (loss(x + e, w) - loss(x - e, w)) / 0.5
        assert abs(float(dx[t, i]) - d) <= float(want["dx"][1][t, i]) + 1e-6 * abs(d)


def test_captured_step(gemm):
    """quantize and the three products in one captured graph, replayed over new
    inputs in the same buffers, with eager work between the replays."""
    T, I, O = 130, 384, 256
    x = torch.zeros((T, I), dtype=torch.bfloat16, device=DEV)
    w, dy = torch.zeros((O, I), device=DEV), torch.zeros((T, O), dtype=torch.bfloat16, device=DEV)
    linear_step(gemm, x, w, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dx, dw, _ = linear_step(gemm, x, w, dy)
    for r in range(3):
        g = torch.Generator().manual_seed(50 + r)
        for t in (x, w, dy):
            t.copy_(torch.randn(t.shape, generator=g))
        want = [t.clone() for t in linear_step(gemm, x, w, dy)[:3]]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, dx, dw), want))


def test_two_streams_and_handles(gemm):
    """Calls that overlap, on two streams of one handle: same results as alone."""
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ins = []
    for seed in (1, 2):
        A, sa, B, sb = (t.to(DEV) for t in problem(200, 300, 1024, 0, 0, 128, seed))
        ins.append((A, sa, 0, B, sb, 0, torch.empty((200, 300), device=DEV)))
    want = [gemm.block128(*a[:6], torch.empty((200, 300), device=DEV)) for a in ins]
    torch.cuda.synchronize()
    for _ in range(4):
        gemm.block128(*ins[0], stream=s1)
        gemm.block128(*ins[1], stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(ins[0][6], want[0]) and torch.equal(ins[1][6], want[1])

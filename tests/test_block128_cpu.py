"""Host-side argument checks of the block-128 product and its quantization
(no GPU call)."""
import pytest

import level_dsl_amd as L

OK, NULL, FMT, DTYPE, SHAPE, ALIGN, ALIAS = (L.STATUS_CODE["MXGEMM_" + n] for n in (
    "OK", "ERR_NULL", "ERR_FMT", "ERR_DTYPE", "ERR_SHAPE", "ERR_ALIGN", "ERR_ALIAS"))
A, AS, B, BS, C = 0x100000, 0x200004, 0x300000, 0x400008, 0x1000000


def v(**kw):
    a = dict(A=A, A_scale=AS, fmtA=0, B=B, B_scale=BS, fmtB=0, b_rows=128, C=C, M=64, N=64, K=128,
             use_acc=0, out_dtype=0)
    a.update(kw)
    return L.mxgemm_validate_block128(**a)


@pytest.mark.parametrize("kw,code", [
    ({}, OK), ({"b_rows": 1}, OK), ({"M": 1, "N": 1, "K": 16}, OK), ({"fmtA": 1, "fmtB": 1}, OK),
    ({"K": 144, "out_dtype": 1, "use_acc": 1}, OK),
    ({"A": 0}, NULL), ({"A_scale": 0}, NULL), ({"B": 0}, NULL), ({"B_scale": 0}, NULL), ({"C": 0}, NULL),
    ({"fmtA": 2}, FMT), ({"fmtB": 4}, FMT), ({"fmtB": -1}, FMT),
    ({"out_dtype": 2}, DTYPE), ({"use_acc": -1}, DTYPE),
    ({"b_rows": 64}, SHAPE), ({"b_rows": 0}, SHAPE), ({"M": 0}, SHAPE), ({"N": 0}, SHAPE), ({"K": 0}, SHAPE),
    ({"K": 8}, SHAPE), ({"K": 136}, SHAPE), ({"K": (1 << 21) + 16}, SHAPE), ({"N": (1 << 20) + 1}, SHAPE),
    ({"M": (1 << 30) + 1}, SHAPE), ({"M": 1 << 20, "N": 1 << 17}, SHAPE), ({"M": -5}, SHAPE),
    ({"A": A + 8}, ALIGN), ({"B": B + 4}, ALIGN), ({"C": C + 2}, ALIGN), ({"A_scale": AS + 2}, ALIGN),
    ({"B_scale": BS + 1}, ALIGN),
    ({"C": A + 64 * 128 - 16}, ALIAS), ({"C": A + 64 * 128}, OK), ({"C": B}, ALIAS),
    # scales: 64 x 1 fp32 of A; 1 x 1 (or 64 x 1) of B
    ({"C": 0x200100}, ALIAS), ({"C": 0x200110}, OK),
    ({"C": 0x400010}, OK), ({"C": 0x400010, "b_rows": 1}, ALIAS),
])
def test_validate_product(kw, code):
    assert v(**kw) == code


X, Q, S, QT, ST = 0x100000, 0x400000, 0x500000, 0x600000, 0x700000


def vq(**kw):
    a = dict(X=X, x_dtype=0, R=100, K=144, rows=1, fmt=0, codes=Q, scales=S, codes_t=QT, scales_t=ST)
    a.update(kw)
    return L.mxgemm_validate_quantize_block128(**a)


@pytest.mark.parametrize("kw,code", [
    ({}, OK), ({"rows": 128, "fmt": 1, "x_dtype": 1}, OK), ({"codes": 0, "scales": 0}, OK),
    ({"codes_t": 0, "scales_t": 0}, OK), ({"R": 1, "K": 16}, OK),
    ({"X": 0}, NULL), ({"codes": 0}, NULL), ({"scales": 0}, NULL), ({"codes_t": 0}, NULL), ({"scales_t": 0}, NULL),
    ({"codes": 0, "scales": 0, "codes_t": 0, "scales_t": 0}, NULL),
    ({"fmt": 2}, FMT), ({"x_dtype": 2}, DTYPE), ({"rows": 32}, SHAPE), ({"R": 0}, SHAPE), ({"K": 24}, SHAPE),
    ({"K": 0}, SHAPE), ({"K": (1 << 21) + 16}, SHAPE), ({"R": (1 << 21) + 1}, SHAPE),
    ({"R": (1 << 21) + 1, "K": 16, "codes_t": 0, "scales_t": 0, "X": 1 << 40, "codes": 1 << 41,
      "scales": 1 << 42}, OK),
    # 2^24 workgroups of 256 threads are one too many
    ({"R": 1 << 30, "K": 144, "codes_t": 0, "scales_t": 0, "X": 1 << 44, "codes": 1 << 45,
      "scales": 1 << 46}, SHAPE),
    ({"R": (1 << 30) - 128, "K": 144, "codes_t": 0, "scales_t": 0, "X": 1 << 44, "codes": 1 << 45,
      "scales": 1 << 46}, OK),
    ({"X": X + 4}, ALIGN), ({"codes": Q + 8}, ALIGN), ({"codes_t": QT + 4}, ALIGN), ({"scales": S + 2}, ALIGN),
    ({"scales_t": ST + 3}, ALIGN),
    ({"codes": X + 100 * 144 * 4 - 16}, ALIAS), ({"codes": X + 100 * 144 * 4}, OK), ({"scales": Q + 4}, ALIAS),
    # the transpose has 144 rows of 112 codes
    ({"scales_t": QT + 144 * 112 - 4}, ALIAS), ({"scales_t": QT + 144 * 112}, OK), ({"codes_t": Q}, ALIAS),
])
def test_validate_quantize(kw, code):
    assert vq(**kw) == code


def test_bad_handle_launches_nothing():
    lib = L.load_library()
    bad = L.STATUS_CODE["MXGEMM_ERR_HANDLE"]
    assert lib.mxgemm_run_block128(None, A, AS, 0, B, BS, 0, 128, C, 64, 64, 128, 0, 0, None) == bad
    assert lib.mxgemm_quantize_block128(None, X, 0, 100, 144, 1, 0, Q, S, QT, ST, None) == bad

"""Host-side argument checks of the 8-bit key / value cache (no GPU call)."""
import ctypes

import pytest
import torch

import level_dsl_amd as L

OK, NULL, DTYPE, SHAPE, ALIGN, ALIAS, WS = (L.STATUS_CODE["MXGEMM_" + n] for n in (
    "OK", "ERR_NULL", "ERR_DTYPE", "ERR_SHAPE", "ERR_ALIGN", "ERR_ALIAS", "ERR_WORKSPACE"))
MB = 1 << 20
# 100 pages x 2 heads x 64 tokens x 128 dims: 1638400 bytes of codes each
CACHE = dict(k_codes=16 * MB, k_scales=32 * MB + 3, v_codes=48 * MB, v_scales=64 * MB + 1, pages=100,
             page_size=64, kv_heads=2, head_dim=128)
BATCH = dict(page_table=80 * MB, q_start=81 * MB, ctx_len=82 * MB, seqs=4, max_pages=20, rows=10, max_q=5,
             max_ctx=1000)
K, V, Q, O, LSE, WSP = 90 * MB, 91 * MB, 92 * MB, 93 * MB, 94 * MB, 128 * MB


def structs(kw):
    kw = dict(kw)
    c = L.CacheStruct(**{k: kw.pop(k, v) for k, v in CACHE.items()})
    b = L.BatchStruct(**{k: kw.pop(k, v) for k, v in BATCH.items()})
    return c, b, kw


COMMON = [
    ({}, OK), ({"page_size": 16, "head_dim": 64}, OK), ({"page_size": 128}, OK), ({"page_size": 32}, OK),
    ({"max_ctx": 1}, OK), ({"max_q": 1000}, OK),
    ({"k_codes": 0}, NULL), ({"k_scales": 0}, NULL), ({"v_codes": 0}, NULL), ({"v_scales": 0}, NULL),
    ({"page_table": 0}, NULL), ({"q_start": 0}, NULL), ({"ctx_len": 0}, NULL),
    ({"page_size": 48}, SHAPE), ({"page_size": 0}, SHAPE), ({"page_size": 256}, SHAPE), ({"head_dim": 96}, SHAPE),
    ({"kv_heads": 0}, SHAPE), ({"kv_heads": 1025}, SHAPE), ({"pages": 0}, SHAPE), ({"pages": 1 << 31}, SHAPE),
    ({"seqs": 0}, SHAPE), ({"max_pages": 0}, SHAPE), ({"rows": 0}, SHAPE), ({"max_q": 0}, SHAPE),
    ({"max_ctx": 0}, SHAPE), ({"rows": 1 << 31}, SHAPE), ({"max_q": 1 << 31}, SHAPE), ({"seqs": -1}, SHAPE),
    ({"k_codes": 16 * MB + 8}, ALIGN), ({"v_codes": 48 * MB + 4}, ALIGN), ({"page_table": 80 * MB + 2}, ALIGN),
    ({"q_start": 81 * MB + 1}, ALIGN), ({"ctx_len": 82 * MB + 2}, ALIGN),
]


def va(kw):
    c, b, kw = structs(kw)
    a = dict(K=K, V=V, x_dtype=1, kv_stride=256)
    a.update(kw)
    return L.mxgemm_validate_cache_append(c, b, **a)


@pytest.mark.parametrize("kw,code", COMMON + [
    ({"K": 0}, NULL), ({"V": 0}, NULL), ({"x_dtype": 2}, DTYPE), ({"kv_stride": 248}, SHAPE),
    ({"kv_stride": 260}, SHAPE), ({"kv_stride": 264}, OK), ({"K": K + 8}, ALIGN), ({"V": V + 4}, ALIGN),
    # more workgroups than a grid holds
    ({"seqs": 1 << 30, "max_pages": 1, "page_table": 1 << 44, "q_start": 1 << 45, "ctx_len": 1 << 46}, SHAPE),
    ({"seqs": (1 << 24) - 1, "max_pages": 1, "page_table": 1 << 44, "q_start": 1 << 45, "ctx_len": 1 << 46}, OK),
    ({"seqs": 1 << 24, "max_pages": 1, "page_table": 1 << 44, "q_start": 1 << 45, "ctx_len": 1 << 46}, SHAPE),
    ({"v_codes": 16 * MB + 1638400}, OK), ({"v_codes": 16 * MB + 1638400 - 16}, ALIAS),
    ({"k_scales": 16 * MB}, ALIAS), ({"v_scales": 32 * MB + 4}, ALIAS), ({"K": 16 * MB}, ALIAS),
    ({"V": 48 * MB + 16}, ALIAS), ({"k_scales": 80 * MB + 4 * 20 * 4 - 1}, ALIAS), ({"k_scales": 81 * MB}, ALIAS),
    ({"v_scales": 82 * MB + 15}, ALIAS), ({"v_scales": 82 * MB + 16}, OK),
    # K and V may be views of one matrix
    ({"V": K + 512, "kv_stride": 512}, OK),
])
def test_validate_append(kw, code):
    assert va(kw) == code


def vt(kw):
    c, b, kw = structs(kw)
    a = dict(Q=Q, q_heads=8, q_stride=8 * c.head_dim, softmax_scale=0.1, window=0, sinks=0, O=O,
             o_stride=8 * c.head_dim, lse=LSE, ws=0, ws_bytes=0)
    a.update(kw)
    return L.mxgemm_validate_cache_attention(c, b, **a)


@pytest.mark.parametrize("kw,code", [x for x in COMMON if x[0].get("kv_heads") != 1025] + [
    ({"Q": 0}, NULL), ({"O": 0}, NULL), ({"lse": 0}, OK), ({"q_heads": 7}, SHAPE), ({"q_heads": 0}, SHAPE),
    ({"q_heads": 6, "q_stride": 768, "o_stride": 768}, OK), ({"q_heads": 4098, "q_stride": 1 << 20}, SHAPE),
    ({"q_stride": 1016}, SHAPE), ({"o_stride": 1016}, SHAPE), ({"q_stride": 1028}, SHAPE), ({"q_stride": 2048}, OK),
    ({"window": (1 << 63) - 1, "ws": WSP, "ws_bytes": 64 * MB}, OK),
    ({"window": -1}, SHAPE), ({"sinks": 4}, SHAPE), ({"sinks": 4, "window": 16}, OK),
    ({"sinks": -1, "window": 16}, SHAPE), ({"window": 1 << 40}, OK),
    ({"softmax_scale": float("nan")}, SHAPE), ({"softmax_scale": float("inf")}, SHAPE), ({"softmax_scale": 0.0}, OK),
    ({"Q": Q + 8}, ALIGN), ({"O": O + 2}, ALIGN), ({"lse": LSE + 2}, ALIGN),
    ({"O": Q}, ALIAS), ({"O": Q + 10 * 1024 * 2}, OK), ({"O": Q + 10 * 1024 * 2 - 16}, ALIAS),
    ({"lse": O + 16}, ALIAS), ({"O": 16 * MB}, ALIAS), ({"lse": 32 * MB}, ALIAS), ({"lse": 64 * MB}, ALIAS),
    ({"lse": 81 * MB}, ALIAS),
    ({"ws": WSP, "ws_bytes": 0}, WS), ({"ws": WSP + 128, "ws_bytes": MB}, WS), ({"ws": WSP, "ws_bytes": 64 * MB}, OK),
    ({"ws": 48 * MB, "ws_bytes": 64 * MB}, ALIAS),
    ({"seqs": 1 << 30, "max_pages": 1, "page_table": 1 << 44, "q_start": 1 << 45, "ctx_len": 1 << 46}, SHAPE),
])
def test_validate_attention(kw, code):
    assert vt(kw) == code


def test_workspace_is_what_the_check_asks_for():
    for kw in ({}, {"max_ctx": 100000, "max_pages": 4000}, {"head_dim": 64, "max_q": 100, "rows": 400},
               {"seqs": 500, "max_ctx": 4096, "max_pages": 64}):
        c, b, _ = structs(kw)
        for heads in (2, 8, 34):
            n = L.mxgemm_cache_attention_workspace(c, b, heads)
            assert n >= 0
            if n == 0:
                continue
            args = dict(kw, q_heads=heads, q_stride=8192, o_stride=8192, ws=1 << 40, Q=1 << 41, O=1 << 42,
                        lse=1 << 43)
            assert vt(dict(args, ws_bytes=n)) == OK and vt(dict(args, ws_bytes=n - 1)) == WS


def test_few_rows_want_no_prompt_workspace():
    """A part of a split holds its row tile's rows: 16 (little work, or at most
    48 rows) or 128, each of head_dim + 2 floats."""
    for max_q, max_ctx, rows in ((1, 65536, 16), (24, 65536, 16), (25, 65536, 128), (100, 2048, 16), (2048, 65536, 128)):
        c, b, _ = structs({"seqs": 1, "rows": 4096, "max_q": max_q, "max_ctx": max_ctx, "max_pages": 4096})
        n = L.mxgemm_cache_attention_workspace(c, b, 2 * c.kv_heads)
        tiles = c.kv_heads * -(-2 * max_q // rows)
        parts = n // (rows * (c.head_dim + 2) * 4)
        assert n and n % (tiles * rows * (c.head_dim + 2) * 4) == 0 and 2 <= parts // tiles <= 64


def test_workspace_of_invalid_arguments():
    c, b, _ = structs({})
    assert L.mxgemm_cache_attention_workspace(c, b, 3) == -1
    assert L.mxgemm_cache_attention_workspace(c, b, 4, -1) == -1
    assert L.mxgemm_cache_attention_workspace(None, b, 4) == -1
    c.page_size = 5
    assert L.mxgemm_cache_attention_workspace(c, b, 4) == -1


def test_bad_handle_launches_nothing():
    lib = L.load_library()
    c, b, _ = structs({})
    bad = L.STATUS_CODE["MXGEMM_ERR_HANDLE"]
    pc, pb = ctypes.addressof(c), ctypes.addressof(b)
    assert lib.mxgemm_cache_append(None, pc, pb, K, V, 1, 256, None) == bad
    assert lib.mxgemm_cache_attention(None, pc, pb, Q, 8, 1024, 0.1, 0, 0, O, 1024, LSE, None, 0, None) == bad


class OtherGpu:
    """A handle of a GPU that none of the tensors is on; a call that got past
    the checks would have no library to go to."""
    h, lib, device = None, None, 1


def test_tensors_elsewhere_are_refused():
    u8 = torch.zeros((4, 128), dtype=torch.uint8)
    f = torch.ones((4, 1))
    with pytest.raises(ValueError, match="GPU"):
        L.Gemm.block128(OtherGpu, u8, f, 0, u8.clone(), f, 0, torch.zeros((4, 4)))
    with pytest.raises(ValueError, match="GPU"):
        L.Gemm.quantize_block128(OtherGpu, torch.zeros((4, 128)), 0)
    codes = torch.zeros((2, 1, 16, 64), dtype=torch.uint8)
    scales = torch.zeros((2, 1), dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        L.KVCache(OtherGpu, codes, scales, codes.transpose(2, 3).contiguous(), scales.clone())

// mxcache.hip -- host side of the 8-bit key / value cache: argument checks,
// the choice of kernel and splits, and the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "mxcache.h"
#include "mxgemm.h"
#include "mxgemm_ctx.h"

using mxg::overlaps;

namespace {

constexpr int64_t kMaxInt = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxGrid = ((int64_t)1 << 24) - 1;  // workgroups of 256 threads: 2^32 work-items are too many

int page_shift(int page_size)
{
    switch (page_size) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    default: return -1;
    }
}

bool count_ok(int64_t x) { return x >= 1 && x <= kMaxInt; }

uint64_t code_bytes(const mxgemm_cache *c)
{
    return (uint64_t)c->pages * c->kv_heads * c->page_size * c->head_dim;
}

// what both entry points ask of the cache and the batch
int check_common(const mxgemm_cache *c, const mxgemm_batch *b)
{
    if (!c || !b || !c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales || !b->page_table || !b->q_start ||
        !b->ctx_len)
        return MXGEMM_ERR_NULL;
    if (page_shift(c->page_size) < 0 || (c->head_dim != 64 && c->head_dim != 128) || c->kv_heads < 1 ||
        c->kv_heads > 1024 || !count_ok(c->pages) || !count_ok(b->seqs) || !count_ok(b->max_pages) ||
        !count_ok(b->rows) || !count_ok(b->max_q) || !count_ok(b->max_ctx))
        return MXGEMM_ERR_SHAPE;
    if (((uintptr_t)c->k_codes | (uintptr_t)c->v_codes) & 15u) return MXGEMM_ERR_ALIGN;
    if (((uintptr_t)b->page_table | (uintptr_t)b->q_start | (uintptr_t)b->ctx_len) & 3u) return MXGEMM_ERR_ALIGN;
    return MXGEMM_OK;
}

// whether [w, w + n) overlaps an array of the batch
bool hits_batch(const void *w, uint64_t n, const mxgemm_batch *b)
{
    return overlaps(w, n, b->page_table, (uint64_t)b->seqs * b->max_pages * 4) ||
           overlaps(w, n, b->q_start, ((uint64_t)b->seqs + 1) * 4) || overlaps(w, n, b->ctx_len, (uint64_t)b->seqs * 4);
}

mxg::cache::Pages pages_of(const mxgemm_cache *c, const mxgemm_batch *b)
{
    mxg::cache::Pages p;
    p.k = c->k_codes;
    p.ks = c->k_scales;
    p.v = c->v_codes;
    p.vs = c->v_scales;
    p.table = b->page_table;
    p.q_start = b->q_start;
    p.ctx_len = b->ctx_len;
    p.rows = b->rows;
    p.pages = (int)c->pages;
    p.max_pages = (int)b->max_pages;
    p.seqs = (int)b->seqs;
    p.max_q = (int)std::min(b->max_q, b->rows);
    p.kv_heads = c->kv_heads;
    p.shift = page_shift(c->page_size);
    return p;
}

// pages that max_q new tokens of one sequence can reach
int64_t append_steps(const mxgemm_cache *c, const mxgemm_batch *b)
{
    const int64_t q = std::min(b->max_q, b->rows);
    return std::min((q + c->page_size - 2) / c->page_size + 1, b->max_pages);
}

int64_t rows_of(const mxgemm_cache *c, const mxgemm_batch *b, int q_heads)
{
    return std::min(b->max_q, b->rows) * (q_heads / c->kv_heads);
}

int64_t tiles_of(const mxgemm_cache *c, const mxgemm_batch *b, int q_heads, int rows)
{
    return (rows_of(c, b, q_heads) + rows - 1) / rows;
}

bool heads_ok(const mxgemm_cache *c, int q_heads)
{
    return q_heads >= 1 && q_heads <= 4096 && q_heads % c->kv_heads == 0;
}

bool grid_ok(const mxgemm_cache *c, const mxgemm_batch *b, int q_heads)
{
    const int64_t t = tiles_of(c, b, q_heads, mxg::kDecodeRows);
    return t <= kMaxGrid && b->seqs * c->kv_heads <= kMaxGrid / t;
}

// How a call that passed grid_ok runs.
struct Plan {
    bool prompt;
    int64_t row_tiles, splits, bytes;  // bytes of workspace
};
Plan plan_of(const mxgemm_cache *c, const mxgemm_batch *b, int q_heads, int64_t window)
{
    const int64_t reach = std::min(b->max_ctx, b->max_pages * c->page_size);
    const int64_t heads = b->seqs * c->kv_heads, tokens = std::min(b->max_q, b->rows);
    const bool windowed = window > 0 && window < reach;
    // blocks that a tile of so many rows sees at most (but for sinks)
    auto blocks_of = [&](int rows) {
        const int64_t own = std::min(tokens, (int64_t)rows * c->kv_heads / q_heads + 1);
        return ((windowed ? std::min(reach, window + own) : reach) + 63) / 64;
    };
    Plan p;
    // The prompt kernel, or the decode kernel, which reads the keys once for
    // every 16 rows, but splits the work more finely: by the 16-row tiles times
    // the blocks that a row sees on average, and for many tiles of few blocks,
    // where the decode kernel's fixed work counts, by the tiles alone.  Measured
    // (us, dim 128, decode / prompt kernel, tiles x blocks in brackets):
    //   64 x 8 rows, 512 keys, 4 heads  13 / 18 [128 x 8]          4096 rows, 1024 keys, 2 heads  13 / 29 [512 x 8]
    //   6000 rows, 1500 keys, 2 heads  25 / 31 [750 x 12]          4 x 64 rows, 8192 keys, 8 heads  28 / 30 [128 x 128]
    //   2 x 2048 rows, 4096 keys, 2 heads  36 / 39 [512 x 60]      4 x 512 rows, 2048 keys, 8 heads  32 / 35 [1024 x 28]
    //   4 x 96 rows, 8192 keys, 8 heads  43 / 32 [192 x 128]       16 x 64 rows, 8192 keys, 8 heads  122 / 80 [512 x 128]
    //   8 x 128 rows, 128 keys, 8 heads  8.8 / 9.7 [512 x 1]       64 x 80 rows, 40 keys, 8 heads  29 / 12 [2560 x 1]
    //   49 x 72 rows, 72 keys, 4 heads  14 / 9.2 [980 x 1]         5 x 916 rows, 229 keys, 8 heads  24 / 16 [2320 x 2]
    //   16 x 32 rows, 8192 keys, 8 heads  77 / 98, 48 rows: 109 / 114
    // The limit of 24000 lies between [128 x 128] and [192 x 128]; two pairs of
    // fewer blocks, [512 x 60] and [1024 x 28], take the prompt kernel by it
    // although the other is 8 to 9 % faster there.
    const int64_t small = tiles_of(c, b, q_heads, mxg::kDecodeRows);
    const int64_t seen = windowed ? blocks_of(mxg::kDecodeRows) : (reach - std::min(tokens, reach) / 2 + 63) / 64;
    p.prompt = rows_of(c, b, q_heads) > 48 && (heads * small > 24000 / seen || (heads * small > 900 && seen <= 8));
    const int rows = p.prompt ? mxg::kPromptRows : mxg::kDecodeRows;
    p.row_tiles = tiles_of(c, b, q_heads, rows);
    // Splits of the visible keys: as many as make at most two workgroups for
    // each of the 256 CUs, which is what they hold at dim 128 (4 x 96 rows, 8192
    // keys, 8 heads, decode kernel: 384 workgroups 45 us, 576: 65 us), with at
    // least four 64-key blocks a split, one per wave of the decode kernel.  More
    // than one round of them costs more than its balance gains (decode, 64
    // sequences of 4097 to 8192 tokens, 8 kv heads: 1 split 160 us, 2: 176, 4:
    // 173).
    const int64_t tiles = heads * p.row_tiles;
    p.splits = std::max<int64_t>(1, std::min({512 / tiles, blocks_of(rows) / 4, (int64_t)mxg::kMaxSplits}));
    p.bytes = p.splits == 1 ? 0 : tiles * p.splits * rows * (c->head_dim + 2) * 4;
    return p;
}

} // namespace

extern "C" {

int mxgemm_validate_cache_append(const mxgemm_cache *cache, const mxgemm_batch *batch, const void *K,
                                 const void *V, int x_dtype, int64_t kv_stride)
{
    if (!K || !V) return MXGEMM_ERR_NULL;
    const int rc = check_common(cache, batch);
    if (rc != MXGEMM_OK) return rc;
    if (x_dtype != MXGEMM_X_F32 && x_dtype != MXGEMM_X_BF16) return MXGEMM_ERR_DTYPE;
    const int64_t width = (int64_t)cache->kv_heads * cache->head_dim;
    if (kv_stride < width || kv_stride > kMaxInt || kv_stride % 8 != 0) return MXGEMM_ERR_SHAPE;
    if (batch->seqs > kMaxGrid / append_steps(cache, batch)) return MXGEMM_ERR_SHAPE;
    if (((uintptr_t)K | (uintptr_t)V) & 15u) return MXGEMM_ERR_ALIGN;
    const uint64_t x = ((uint64_t)(batch->rows - 1) * kv_stride + width) * (x_dtype == MXGEMM_X_F32 ? 4u : 2u);
    const uint64_t n = code_bytes(cache), ns = (uint64_t)cache->pages * cache->kv_heads;
    const void *w[4] = {cache->k_codes, cache->v_codes, cache->k_scales, cache->v_scales};
    const uint64_t wn[4] = {n, n, ns, ns};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlaps(w[i], wn[i], w[j], wn[j])) return MXGEMM_ERR_ALIAS;
        if (overlaps(w[i], wn[i], K, x) || overlaps(w[i], wn[i], V, x) || hits_batch(w[i], wn[i], batch))
            return MXGEMM_ERR_ALIAS;
    }
    return MXGEMM_OK;
}

int mxgemm_cache_append(mxgemm_t h, const mxgemm_cache *cache, const mxgemm_batch *batch, const void *K,
                        const void *V, int x_dtype, int64_t kv_stride, hipStream_t stream)
{
    if (!h || h->magic != mxg::kMagic) return MXGEMM_ERR_HANDLE;
    int rc = mxgemm_validate_cache_append(cache, batch, K, V, x_dtype, kv_stride);
    if (rc != MXGEMM_OK) return rc;
    rc = mxg::check_device(h);
    if (rc != MXGEMM_OK) return rc;
    mxg::cache::AppendArgs a;
    a.c = pages_of(cache, batch);
    a.K = (const uint8_t *)K;
    a.V = (const uint8_t *)V;
    a.stride = kv_stride;
    a.steps = (int)append_steps(cache, batch);
    return mxg::launch_cache_append(x_dtype == MXGEMM_X_BF16, cache->head_dim, a, stream) == hipSuccess
               ? MXGEMM_OK
               : MXGEMM_ERR_HIP;
}

int64_t mxgemm_cache_attention_workspace(const mxgemm_cache *cache, const mxgemm_batch *batch, int q_heads,
                                         int64_t window)
{
    if (check_common(cache, batch) != MXGEMM_OK || !heads_ok(cache, q_heads) || !grid_ok(cache, batch, q_heads) ||
        window < 0)
        return -1;
    return plan_of(cache, batch, q_heads, window).bytes;
}

int mxgemm_validate_cache_attention(const mxgemm_cache *cache, const mxgemm_batch *batch, const void *Q,
                                    int q_heads, int64_t q_stride, float softmax_scale, int64_t window,
                                    int64_t sinks, const void *O, int64_t o_stride, const float *lse,
                                    const void *ws, size_t ws_bytes)
{
    if (!Q || !O) return MXGEMM_ERR_NULL;
    const int rc = check_common(cache, batch);
    if (rc != MXGEMM_OK) return rc;
    if (!heads_ok(cache, q_heads) || !grid_ok(cache, batch, q_heads)) return MXGEMM_ERR_SHAPE;
    const int64_t width = (int64_t)q_heads * cache->head_dim;
    if (q_stride < width || o_stride < width || q_stride > kMaxInt || o_stride > kMaxInt || q_stride % 8 != 0 ||
        o_stride % 8 != 0 || window < 0 || sinks < 0 || (sinks > 0 && window == 0) || !std::isfinite(softmax_scale))
        return MXGEMM_ERR_SHAPE;
    if (((uintptr_t)Q | (uintptr_t)O) & 15u || (uintptr_t)lse & 3u) return MXGEMM_ERR_ALIGN;
    const int64_t need = ws ? plan_of(cache, batch, q_heads, window).bytes : 0;
    if (ws && (((uintptr_t)ws & 255u) || (uint64_t)need > ws_bytes)) return MXGEMM_ERR_WORKSPACE;
    const uint64_t n = code_bytes(cache), ns = (uint64_t)cache->pages * cache->kv_heads;
    const uint64_t qn = ((uint64_t)(batch->rows - 1) * q_stride + width) * 2;
    const void *w[3] = {O, lse, need ? ws : nullptr};
    const uint64_t wn[3] = {((uint64_t)(batch->rows - 1) * o_stride + width) * 2, (uint64_t)batch->rows * q_heads * 4,
                            (uint64_t)need};
    for (int i = 0; i < 3; ++i) {
        if (!w[i]) continue;
        for (int j = 0; j < i; ++j)
            if (w[j] && overlaps(w[i], wn[i], w[j], wn[j])) return MXGEMM_ERR_ALIAS;
        if (overlaps(w[i], wn[i], Q, qn) || overlaps(w[i], wn[i], cache->k_codes, n) ||
            overlaps(w[i], wn[i], cache->v_codes, n) || overlaps(w[i], wn[i], cache->k_scales, ns) ||
            overlaps(w[i], wn[i], cache->v_scales, ns) || hits_batch(w[i], wn[i], batch))
            return MXGEMM_ERR_ALIAS;
    }
    return MXGEMM_OK;
}

int mxgemm_cache_attention(mxgemm_t h, const mxgemm_cache *cache, const mxgemm_batch *batch, const void *Q,
                           int q_heads, int64_t q_stride, float softmax_scale, int64_t window, int64_t sinks,
                           void *O, int64_t o_stride, float *lse, void *ws, size_t ws_bytes, hipStream_t stream)
{
    if (!h || h->magic != mxg::kMagic) return MXGEMM_ERR_HANDLE;
    int rc = mxgemm_validate_cache_attention(cache, batch, Q, q_heads, q_stride, softmax_scale, window, sinks, O,
                                             o_stride, lse, ws, ws_bytes);
    if (rc != MXGEMM_OK) return rc;
    rc = mxg::check_device(h);
    if (rc != MXGEMM_OK) return rc;
    mxg::cache::AttnArgs a;
    a.c = pages_of(cache, batch);
    a.Q = (const uint16_t *)Q;
    a.O = (uint16_t *)O;
    a.lse = lse;
    a.q_stride = q_stride;
    a.o_stride = o_stride;
    a.q_heads = q_heads;
    a.group = q_heads / cache->kv_heads;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.window = (int)std::min(window, kMaxInt);
    a.sinks = (int)std::min(sinks, kMaxInt);
    const Plan plan = plan_of(cache, batch, q_heads, window);
    a.row_tiles = (int)plan.row_tiles;
    a.splits = ws ? (int)plan.splits : 1;
    a.ws = (float *)ws;
    const hipError_t e = plan.prompt ? mxg::launch_attn_prompt(cache->head_dim, a, stream)
                                     : mxg::launch_attn_decode(cache->head_dim, a, stream);
    return e == hipSuccess ? MXGEMM_OK : MXGEMM_ERR_HIP;
}

} // extern "C"

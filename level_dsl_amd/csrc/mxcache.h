// mxcache.h -- arguments and launchers of the 8-bit key / value cache: storing
// new tokens (mxgemm_cache_append) and attention over it
// (mxgemm_cache_attention), and the addressing both share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxg {
namespace cache {

struct Pages {
    uint8_t *k, *ks, *v, *vs;
    const int32_t *table, *q_start, *ctx_len;
    int64_t rows;
    int pages, max_pages, seqs, max_q;
    int kv_heads, shift;  // page_size = 1 << shift
};

struct AppendArgs {
    Pages c;
    const uint8_t *K, *V;
    int64_t stride;       // elements between tokens
    int steps;            // pages one sequence's max_q tokens can reach
};

struct AttnArgs {
    Pages c;
    const uint16_t *Q;
    uint16_t *O;
    float *lse;           // or NULL
    int64_t q_stride, o_stride;
    int q_heads, group;   // group = q_heads / kv_heads
    float scale_log2;     // softmax_scale * log2(e)
    int window, sinks;
    int row_tiles, splits;
    float *ws;            // split partials (splits > 1)
};

// One sequence of the batch, its device values brought into range: new rows
// q0 .. q0 + n - 1 (n at most max_q, inside the token matrices), context
// ctx, position of the first new token (may be below zero).
struct Seq {
    int64_t q0;
    int n, ctx, first;
};
__device__ __forceinline__ Seq sequence(const Pages &c, int s)
{
    Seq r;
    const int64_t a = c.q_start[s], b = c.q_start[s + 1];
    // the table's reach; at most 2^31 - 128, so that a rounded-up length still fits an int
    const int64_t reach = min((int64_t)c.max_pages << c.shift, (int64_t)0x7fffff80);
    const int64_t ctx = max((int64_t)0, min((int64_t)c.ctx_len[s], reach));
    const int64_t n = a < 0 ? 0 : max((int64_t)0, b - a);
    r.q0 = a;
    r.ctx = (int)ctx;
    // positions count back from the stated length, before any cut
    const int64_t first = (int64_t)c.ctx_len[s] - n;
    r.first = (int)max(first, -(int64_t)0x7fffffff);
    r.n = (int)min(min(n, (int64_t)c.max_q), max((int64_t)0, c.rows - a));
    return r;
}

// Page of a sequence's block of tokens, or -1 where the table gives none.
__device__ __forceinline__ int page_of(const Pages &c, int s, int index)
{
    if (index < 0 || index >= c.max_pages) return -1;
    const int id = c.table[(int64_t)s * c.max_pages + index];
    return id >= 0 && id < c.pages ? id : -1;
}

} // namespace cache

hipError_t launch_cache_append(int x_bf16, int head_dim, const cache::AppendArgs &a, hipStream_t s);  // k_cache.hip
hipError_t launch_attn_decode(int head_dim, const cache::AttnArgs &a, hipStream_t s);                  // k_attn_decode.hip

hipError_t launch_attn_prompt(int head_dim, const cache::AttnArgs &a, hipStream_t s);                  // k_attn_prompt.hip

// rows of one row tile of the prompt kernel
constexpr int kPromptRows = 128;
// rows of one row tile of the decode kernel (queries times heads of a group)
constexpr int kDecodeRows = 16;
constexpr int kMaxSplits = 64;

} // namespace mxg

// mxattn.h -- what the attention kernels over the 8-bit cache share: which
// keys a tile of rows sees, and a block of 64 tokens' keys and values on its
// way into LDS.
#pragma once

#include "mxcache.h"
#include "mxgemm_common.h"

namespace mxg {
namespace attn {

using cache::AttnArgs;
using cache::Pages;
using cache::Seq;

constexpr int BLOCK = 64;                  // tokens of a block: four chunks of 16
constexpr float kNone = -__builtin_inff();  // a masked score
constexpr float kLn2 = 0.6931471805599453f;

// The keys that rows with positions pmin .. pmax (-1 or more) see together, as
// blocks: list entry i is block i for i < sink_blocks, else first + (i -
// sink_blocks).  Positions fit 32 bits: cache::sequence cuts a context to
// 2^31 - 128, the host the window and the sinks to 2^31 - 1.
struct Range {
    int lo, hi, sinks;  // visible to some row: [lo, hi) and [0, sinks), sinks <= lo
    int sink_blocks, first, count;
    __device__ __forceinline__ int start(int i) const
    {
        return (i < sink_blocks ? i : first + (i - sink_blocks)) * BLOCK;
    }
};
__device__ __forceinline__ Range range_of(const AttnArgs &p, int ctx, int pmin, int pmax)
{
    Range r;
    r.hi = max(0, min(ctx, pmax + 1));
    r.lo = p.window ? max(0, pmin - p.window + 1) : 0;
    r.lo = min(r.lo, r.hi);
    r.sinks = min(p.sinks, r.lo);
    r.first = r.lo / BLOCK;
    const int end = (r.hi + BLOCK - 1) / BLOCK;
    r.sink_blocks = min((r.sinks + BLOCK - 1) / BLOCK, r.first);
    r.count = r.hi > 0 ? r.sink_blocks + (end - r.first) : 0;
    return r;
}
// position of a sequence's new token i; all before zero count as -1
__device__ __forceinline__ int position(const Seq &q, int64_t i) { return (int)max((int64_t)q.first + i, (int64_t)-1); }

// The pages of a block's four chunks (page sizes are multiples of 16; SMALL:
// below 64, otherwise all four lie in one), -1 where the table gives none.
// Wave-uniform, through the scalar cache; an entry is looked at only where it
// is used, so that a load can be in flight until then.  A chunk past the
// visible keys repeats the last one's (its tokens are masked by position).
template <bool SMALL>
struct Ids {
    int entry[SMALL ? 4 : 1], pages;
    __device__ __forceinline__ int id(int j) const { return (unsigned)entry[j] < (unsigned)pages ? entry[j] : -1; }
    __device__ __forceinline__ int of(int chunk) const
    {
        if constexpr (!SMALL) return id(0);
        else return chunk == 0 ? id(0) : chunk == 1 ? id(1) : chunk == 2 ? id(2) : id(3);
    }
    __device__ __forceinline__ bool all() const
    {
        if constexpr (!SMALL) return id(0) >= 0;
        else return (id(0) | id(1) | id(2) | id(3)) >= 0;
    }
};
// row: the sequence's row of the page table; t0 < hi, and hi is inside the table's reach
template <bool SMALL>
__device__ __forceinline__ Ids<SMALL> ids_of(const Pages &c, const int32_t *row, int t0, int hi)
{
    Ids<SMALL> r;
    r.pages = c.pages;
#pragma unroll
    for (int j = 0; j < (SMALL ? 4 : 1); ++j) {
        const int at = min(t0 + 16 * j, hi - 1) >> c.shift;
        r.entry[j] = *(const __attribute__((address_space(4))) int32_t *)(uintptr_t)(row + at);
    }
    return r;
}

__device__ __forceinline__ void lds_from(const uint8_t *src, uint8_t *dst)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src, (lds_ptr_t)dst, 16, 0, 0);
}

// Wait until every LDS read of this wave has returned.
__device__ __forceinline__ void wait_lds()
{
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// A block in LDS: keys [token][D] then values [dim][64 tokens], in chunks of 16
// bytes whose place in a row is turned by the row, so that the eight lanes of
// one ds_read_b128 pass hit different banks:
//   keys   chunk x of token t at x ^ ((t & 3) | (t >> 4 & 1) << 2), D = 64: x ^ (t >> 4)
//          (a pass reads tokens t .. t+3 and t+16 .. t+19)
//   values chunk x of dim d at x ^ (d >> 2 & 3)
template <int D>
struct Tile {
    static constexpr int K_BYTES = BLOCK * D, BYTES = 2 * K_BYTES;
    static constexpr int LOADS = BYTES / 1024;  // direct-to-LDS loads of a wave's 64 lanes
    __device__ static __forceinline__ uint32_t key(int token, int chunk)
    {
        const int turn = D == 128 ? ((token & 3) | ((token >> 4 & 1) << 2)) : (token >> 4 & 3);
        return (uint32_t)(token * D + ((chunk ^ turn) << 4));
    }
    __device__ static __forceinline__ uint32_t value(int dim, int chunk)   // from the values' start
    {
        return (uint32_t)(dim * 64 + ((chunk ^ (dim >> 2 & 3)) << 4));
    }
    static constexpr int HALF = LOADS / 2;       // of the keys, and of the values
    // Loads part, part + PARTS, ... of a block's keys into dst, values into
    // dst + K_BYTES: all of them for a wave of its own tile, every fourth for
    // four waves that share one.  Chunks without a page read page 0 (and are
    // masked by their reader).  head_at: bytes from a page's start to the
    // head's part, page: bytes of a page.
    template <int PARTS, bool SMALL>
    __device__ static __forceinline__ void load_keys(const Pages &c, const Ids<SMALL> &ids, uint32_t head_at, uint32_t page,
                                                     int t0, int part, uint8_t *dst)
    {
        const int lane = threadIdx.x & 63;
        const int pmask = (1 << c.shift) - 1;
        constexpr int LPR = D / 16, RPL = 64 / LPR;   // lanes per key row, rows per load
#pragma unroll
        for (int i = 0; i < HALF / PARTS; ++i) {
            const int j = part + PARTS * i;
            const int t = RPL * j + lane / LPR;        // the load's rows lie in one chunk of tokens
            const uint8_t *base = c.k + (size_t)(uint32_t)max(ids.of(RPL * j / 16), 0) * page + head_at;
            const int x = (lane % LPR) ^ (D == 128 ? ((t & 3) | ((t >> 4 & 1) << 2)) : (t >> 4 & 3));
            lds_from(base + (uint32_t)(((t0 + t) & pmask) * D + 16 * x), dst + j * 1024);
        }
    }
    template <int PARTS, bool SMALL>
    __device__ static __forceinline__ void load_values(const Pages &c, const Ids<SMALL> &ids, uint32_t head_at, uint32_t page,
                                                       int t0, int part, uint8_t *dst)
    {
        const int lane = threadIdx.x & 63;
        const int pmask = (1 << c.shift) - 1;
        // dim 16 j + lane / 4, chunk (lane % 4) ^ (dim >> 2 & 3): the same chunk for every j
        const int x = (lane & 3) ^ (lane >> 4);
        const uint8_t *base = c.v + (size_t)(uint32_t)max(ids.of(x), 0) * page + head_at;
        const uint32_t at = (uint32_t)((t0 + 16 * x) & pmask) + ((uint32_t)(lane >> 2) << c.shift);
#pragma unroll
        for (int i = 0; i < HALF / PARTS; ++i) {
            const int j = part + PARTS * i;
            lds_from(base + (at + ((uint32_t)(16 * j) << c.shift)), dst + j * 1024);
        }
    }
};

// Maximum over the four lane groups of 16 (lanes l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float max_groups(float x)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    const auto u = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const uint32_t u0 = u[0], u1 = u[1];
    x = fmaxf(__builtin_bit_cast(float, u0), __builtin_bit_cast(float, u1));
    const uint32_t d = __builtin_bit_cast(uint32_t, x);
    const auto v = __builtin_amdgcn_permlane16_swap(d, d, false, false);
    const uint32_t v0 = v[0], v1 = v[1];
    return fmaxf(__builtin_bit_cast(float, v0), __builtin_bit_cast(float, v1));
}

// Scale bytes with which the widening to bf16 stays exact for every code
// (normal bf16 numbers).
__device__ __forceinline__ bool plain_scale(uint32_t b) { return b - (uint32_t)scale_lo<0>() <= (uint32_t)window_width<0>(); }

// The lowest n bits of 16 (none for n below zero).
__device__ __forceinline__ uint32_t below16(int n) { return (1u << min(max(n, 0), 16)) - 1; }
// Bit e: whether key t + e, e = 0 .. 15, lies in [lo, hi) or, below hi, in [0, sinks).
__device__ __forceinline__ uint32_t seen16(int lo, int hi, int sinks, int t)
{
    return below16(hi - t) & (~below16(lo - t) | below16(sinks - t));
}
// all bits set where bit e of keep is
__device__ __forceinline__ uint32_t spread(uint32_t keep, int e) { return (uint32_t)((int)(keep << (31 - e)) >> 31); }
// x where m's bits are set, a masked score elsewhere, whatever x is
__device__ __forceinline__ float score_or_none(uint32_t m, float x)
{
    return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, x) & m) | (~m & 0xff800000u));
}
__device__ __forceinline__ float value_or_zero(uint32_t m, float x)
{
    return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x) & m);
}
// 16 codes with those of the cleared bits zeroed
__device__ __forceinline__ v4i keep16(v4i x, uint32_t keep)
{
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const uint32_t n = (keep >> (4 * w) & 15u) * 0x204081u & 0x01010101u;   // bit i to byte i
        x[w] &= (int)((n << 8) - n);
    }
    return x;
}

} // namespace attn
} // namespace mxg

// mxattn_decode.h -- attention over the 8-bit cache for few query rows
// (decode steps): the cache is streamed once, straight into MFMA operands.
//
// A row is one (new token, query head of the group) pair of a sequence and kv
// head, rows in token order; a workgroup of four waves takes 16 of them and a
// part of the visible keys (a split).  Keys come in blocks of 64, dealt to the
// waves in turn.  Per block a wave computes
//   S^T = K Q^T   16x16x32 bf16 MFMA, K's rows (tokens) by Q's columns (rows)
//   O^T += V^T P^T
// with the running maximum and sum of the softmax per column.  A lane holds
// column q = l % 16 of S^T; what it holds of the 64 tokens is what it must
// supply to the second product, without any exchange, because the token that
// MFMA row r of tile t stands for is chosen as
//   token = 16 (r / 4) + 4 t + r % 4:
// a lane's 4 tiles x 4 registers are then tokens 16 g .. 16 g + 15 (g = l /
// 16) in order, which are also 16 contiguous bytes of each row of the
// token-contiguous values.  Page sizes are multiples of 16, so such a chunk
// has one page and one scale byte of keys and of values: the key's scale
// multiplies the scores, the value's the probabilities, both in fp32.
//
// Masked scores are selected away after the product, and value codes no row of
// the tile may see are zeroed before it, so what unwritten or foreign slots
// hold never reaches a result.
//
// The waves' partial sums meet in LDS; with splits they go to the workspace
// and a second kernel joins them (fixed order, so results repeat bit for
// bit).  Bound by HBM: one read of every visible key and value.
#pragma once

#include "mxcache.h"
#include "mxgemm_common.h"

namespace mxg {
namespace attn {

using cache::AttnArgs;
using cache::Pages;
using cache::Seq;

constexpr int WAVES = 4, THREADS = 64 * WAVES, ROWS = 16, BLOCK = 64;
constexpr float kNone = -__builtin_inff();

// e8m0 byte -> 2^(s - 127) as used here: byte 255 is NaN
__device__ __forceinline__ float scale_of(uint32_t s) { return e8m0_to_f32(s); }

// 0xff in byte j of dword i where bit 4 i + j of m is set
__device__ __forceinline__ uint32_t byte_mask(uint32_t m, int i)
{
    const uint32_t n = (m >> (4 * i)) & 15u;
    return ((n & 1u) ? 0xffu : 0u) | ((n & 2u) ? 0xff00u : 0u) | ((n & 4u) ? 0xff0000u : 0u) |
           ((n & 8u) ? 0xff000000u : 0u);
}

// The keys the rows with positions pmin .. pmax see together, as blocks: list
// entry i is block i for i < sink_blocks, else first + (i - sink_blocks).
struct Range {
    int64_t lo, hi, sinks;       // visible: [lo, hi) and [0, sinks), sinks <= lo
    int sink_blocks, first, count;
    __device__ __forceinline__ int block(int i) const { return i < sink_blocks ? i : first + (i - sink_blocks); }
};
template <int BLK>
__device__ __forceinline__ Range range_of(const AttnArgs &p, int ctx, int64_t pmin, int64_t pmax)
{
    Range r;
    r.hi = max((int64_t)0, min((int64_t)ctx, pmax + 1));
    r.lo = p.window ? max((int64_t)0, pmin - p.window + 1) : 0;
    r.lo = min(r.lo, r.hi);
    r.sinks = min(p.sinks, r.lo);
    r.first = (int)(r.lo / BLK);
    const int end = (int)((r.hi + BLK - 1) / BLK);
    r.sink_blocks = min((int)((r.sinks + BLK - 1) / BLK), r.first);
    r.count = r.hi > 0 ? r.sink_blocks + (end - r.first) : 0;
    return r;
}

template <int D>
__global__ __launch_bounds__(THREADS, 2) void decode_kernel(AttnArgs p)
{
    constexpr int CH = D / 64;      // 16-byte key chunks per lane and token
    constexpr int DT = D / 16;      // 16-row tiles of O^T
    const Pages &c = p.c;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    int bid = blockIdx.x;
    const int sp = bid % p.splits;
    bid /= p.splits;
    const int rt = bid % p.row_tiles;
    bid /= p.row_tiles;
    const int head = bid % c.kv_heads, s = bid / c.kv_heads;

    const Seq q = cache::sequence(c, s);
    const int G = p.group;
    const int64_t rows = (int64_t)q.n * G;
    const int64_t row0 = (int64_t)rt * ROWS;
    if (row0 >= rows) return;
    const int64_t row_end = min(row0 + ROWS, rows);
    const Range rg = range_of<BLOCK>(p, q.ctx, q.first + row0 / G, q.first + (row_end - 1) / G);

    // this lane's column: a row of the tile
    const int64_t row = row0 + r16;
    const bool live = row < rows;
    const int qi = (int)((live ? row : row0) / G), qh = (int)((live ? row : row0) % G);
    const int64_t pos = (int64_t)q.first + qi;
    const int64_t wlo = p.window ? pos - p.window : -1;   // key > wlo is inside the window
    v8bf qf[2 * CH];
    {
        const uint16_t *src = p.Q + (q.q0 + qi) * p.q_stride + (int64_t)(head * G + qh) * D;
#pragma unroll
        for (int h = 0; h < CH; ++h)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                qf[2 * h + u] = *reinterpret_cast<const v8bf *>(src + 64 * h + 16 * g + 8 * u);
    }

    const int per = (rg.count + p.splits - 1) / p.splits;
    const int b0 = sp * per, b1 = min(rg.count, b0 + per);

    v4f o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = v4f{0.f, 0.f, 0.f, 0.f};
    float m = kNone, l = 0.0f;

    const size_t page_bytes = (size_t)D << c.shift;
    const int pmask = (1 << c.shift) - 1;
    for (int i = b0 + wave; i < b1; i += WAVES) {
        const int64_t t0 = (int64_t)rg.block(i) * BLOCK;
        // chunk of this lane's key rows (r16 / 4) and of its values and scores (g)
        const int64_t tk = t0 + 16 * (r16 >> 2), tv = t0 + 16 * g;
        const int pk = tk < rg.hi ? cache::page_of(c, s, (int)(tk >> c.shift)) : -1;
        const int pv = tv < rg.hi ? cache::page_of(c, s, (int)(tv >> c.shift)) : -1;
        const size_t ak = (size_t)max(pk, 0) * c.kv_heads + head, av = (size_t)max(pv, 0) * c.kv_heads + head;
        const float ks = scale_of(c.ks[av]) * p.scale_log2, vs = scale_of(c.vs[av]);

        v4f st[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint8_t *src = c.k + ak * page_bytes + (size_t)(((int)tk & pmask) + 4 * t + (r16 & 3)) * D + 16 * g;
            st[t] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < CH; ++h) {
                v8bf lo, hi;
                decode16<0>(*reinterpret_cast<const v4i *>(src + 64 * h), 1.0f, lo, hi);
                st[t] = mfma_bf16_16(lo, qf[2 * h], st[t]);
                st[t] = mfma_bf16_16(hi, qf[2 * h + 1], st[t]);
            }
        }
        float mx = kNone;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t key = tv + 4 * t + e;
                const bool see = pv >= 0 && key <= pos && key < rg.hi && (key > wlo || key < p.sinks);
                st[t][e] = see ? st[t][e] * ks : kNone;
                mx = fmaxf(mx, st[t][e]);   // a NaN score passes by: it makes the row's sum NaN
            }
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        const float mn = fmaxf(m, mx);
        const float mu = mn == kNone ? 0.0f : mn;
        const float alpha = __builtin_amdgcn_exp2f(m - mu);
        m = mn;
        v8bf pf[2];
        float sum = 0.0f;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = __builtin_amdgcn_exp2f(st[t][e] - mu);
                sum += x;
                pf[t >> 1][4 * (t & 1) + e] = (__bf16)(st[t][e] == kNone ? 0.0f : x * vs);
            }
        l = l * alpha + sum;

        // which of this lane's 16 value tokens some row of the tile sees
        uint32_t keep = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int64_t key = tv + e;
            keep |= (pv >= 0 && key < rg.hi && (key >= rg.lo || key < rg.sinks) ? 1u : 0u) << e;
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            v4i x = *reinterpret_cast<const v4i *>(c.v + av * page_bytes +
                                                   ((size_t)(16 * d + r16) << c.shift) + ((int)tv & pmask));
#pragma unroll
            for (int w = 0; w < 4; ++w) x[w] &= (int)byte_mask(keep, w);
            v8bf lo, hi;
            decode16<0>(x, 1.0f, lo, hi);
            o[d] *= alpha;
            o[d] = mfma_bf16_16(lo, pf[0], o[d]);
            o[d] = mfma_bf16_16(hi, pf[1], o[d]);
        }
    }
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);

    // the four waves' sums, joined in wave order
    __shared__ float wm[WAVES][ROWS], wl[WAVES][ROWS];
    __shared__ v4f wo[WAVES][DT][64];
    if (g == 0) {
        wm[wave][r16] = m;
        wl[wave][r16] = l;
    }
    __syncthreads();
    float mt = kNone;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) mt = fmaxf(mt, wm[w][r16]);
    const float mu = mt == kNone ? 0.0f : mt;
    float lt = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) lt += wl[w][r16] * __builtin_amdgcn_exp2f(wm[w][r16] - mu);
    const float mine = __builtin_amdgcn_exp2f(m - mu);
#pragma unroll
    for (int d = 0; d < DT; ++d) wo[wave][d][lane] = o[d] * mine;
    __syncthreads();
    const int64_t tile = (((int64_t)s * c.kv_heads + head) * p.row_tiles + rt) * p.splits + sp;
    float *const part = p.ws + tile * (ROWS * (D + 2));
#pragma unroll
    for (int d = wave; d < DT; d += WAVES) {
        v4f v = wo[0][d][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v += wo[w][d][lane];
        // column r16, rows (dims) 16 d + 4 g .. + 3
        if (p.splits > 1) {
            *reinterpret_cast<v4f *>(part + r16 * D + 16 * d + 4 * g) = v;
        } else if (live) {
            const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
            v *= inv;
            *reinterpret_cast<v2i *>(p.O + (q.q0 + qi) * p.o_stride + (int64_t)(head * G + qh) * D + 16 * d + 4 * g) =
                v2i{(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3])};
        }
    }
    if (wave == 0 && g == 0) {
        if (p.splits > 1) {
            part[ROWS * D + r16] = mt;
            part[ROWS * D + ROWS + r16] = lt;
        } else if (live && p.lse) {
            p.lse[(q.q0 + qi) * p.q_heads + head * G + qh] = (mu + __builtin_log2f(lt)) * 0.6931471805599453f;
        }
    }
}

// The splits' partial sums of one row tile, joined in split order.
template <int D>
__global__ __launch_bounds__(THREADS) void join_kernel(AttnArgs p)
{
    const Pages &c = p.c;
    int bid = blockIdx.x;
    const int rt = bid % p.row_tiles;
    bid /= p.row_tiles;
    const int head = bid % c.kv_heads, s = bid / c.kv_heads;
    const Seq q = cache::sequence(c, s);
    const int G = p.group;
    const int64_t rows = (int64_t)q.n * G, row0 = (int64_t)rt * ROWS;
    if (row0 >= rows) return;
    const float *const part = p.ws + (int64_t)blockIdx.x * p.splits * (ROWS * (D + 2));
    constexpr int64_t PITCH = ROWS * (D + 2);
    for (int i = threadIdx.x; i < ROWS * D / 4; i += THREADS) {
        const int r = i / (D / 4), d = 4 * (i % (D / 4));
        const int64_t row = row0 + r;
        if (row >= rows) continue;
        float mt = kNone;
        for (int k = 0; k < p.splits; ++k) mt = fmaxf(mt, part[k * PITCH + ROWS * D + r]);
        const float mu = mt == kNone ? 0.0f : mt;
        float lt = 0.0f;
        v4f v = {0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < p.splits; ++k) {
            const float f = __builtin_amdgcn_exp2f(part[k * PITCH + ROWS * D + r] - mu);
            lt += part[k * PITCH + ROWS * D + ROWS + r] * f;
            v += *reinterpret_cast<const v4f *>(part + k * PITCH + r * D + d) * f;
        }
        v *= lt == 0.0f ? 0.0f : 1.0f / lt;
        const int64_t token = q.q0 + row / G;
        const int h = head * G + (int)(row % G);
        *reinterpret_cast<v2i *>(p.O + token * p.o_stride + (int64_t)h * D + d) =
            v2i{(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3])};
        if (d == 0 && p.lse) p.lse[token * p.q_heads + h] = (mu + __builtin_log2f(lt)) * 0.6931471805599453f;
    }
}

} // namespace attn
} // namespace mxg

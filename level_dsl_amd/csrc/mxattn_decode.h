// mxattn_decode.h -- attention over the 8-bit cache for few query rows
// (decode steps): the cache is streamed once, each block by one wave.
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
// has one page and one scale byte of keys and of values, which the widening
// to bf16 applies: exact for bytes 10 .. 246.
//
// The waves share nothing until the end: each streams its blocks through LDS
// buffers of its own (keys, values) by direct-to-LDS loads: whole lines, no
// registers, no barrier.  A block's keys are loaded while the block before is
// in its softmax and second product, its values behind that product.  As
// compiled, the loop ends with a wait for all of them (the values' scale byte
// changes registers there, which waits for every load before it), so the values,
// and what is left of the keys, are hidden by the other of the SIMD's two waves
// only.  The waits that the kernel itself asks for count on the order: keys
// first, values behind them.  (Two buffers of both,
// one wave per SIMD: 210 us where this takes 153 us, 64 sequences of 4097 to
// 8192 tokens, 64 / 8 heads, dim 128: 5.35 TB/s.)  The running maximum lags: it moves, and
// what was summed is scaled, only where a score passes it by more than 8
// (log2), so that probabilities stay below 2^8; the result does not depend on
// it.
//
// Masked scores are selected away after the product, and value codes no row of
// the tile may see are zeroed before it, so what unwritten or foreign slots
// hold never reaches a result.  Blocks that every row sees whole, with scale
// bytes as above, skip both; the others apply the scales in fp32, to the
// scores and the probabilities (byte 255 there makes NaN of what sees it).
//
// The waves' partial sums meet in LDS; with splits they go to the workspace
// and a second kernel joins them (fixed order, so results repeat bit for
// bit).  Bound by HBM: one read of every visible key and value.
#pragma once

#include "mxattn.h"

#include <type_traits>

namespace mxg {
namespace attn {

constexpr int WAVES = 4, THREADS = 64 * WAVES, ROWS = 16;

template <int D, bool SMALL>
__global__ __launch_bounds__(THREADS, 2) void decode_kernel(AttnArgs p)
{
    constexpr int CH = D / 64;      // 16-byte key chunks per lane and token
    constexpr int DT = D / 16;      // 16-row tiles of O^T
    using T = Tile<D>;
    constexpr int HALF = T::HALF + 1;  // vector-memory operations of a block's keys, or values: loads, a scale byte
    // separate objects: a read of one then does not wait for loads into the other
    __shared__ __attribute__((aligned(1024))) uint8_t keys[WAVES * T::K_BYTES], values[WAVES * T::K_BYTES];
    const Pages &c = p.c;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    uint32_t bid = blockIdx.x;
    const int sp = (int)(bid % (uint32_t)p.splits);
    bid /= (uint32_t)p.splits;
    const int rt = (int)(bid % (uint32_t)p.row_tiles);
    bid /= (uint32_t)p.row_tiles;
    const int head = (int)(bid % (uint32_t)c.kv_heads), s = (int)(bid / (uint32_t)c.kv_heads);

    const Seq q = cache::sequence(c, s);
    const uint32_t G = p.group;       // the launch has fewer than 2^24 tiles, so rows fit 32 bits
    const uint32_t rows = (uint32_t)q.n * G, row0 = (uint32_t)rt * ROWS;
    if (row0 >= rows) return;
    const int pmin = position(q, row0 / G), pmax = position(q, (min(row0 + ROWS, rows) - 1) / G);
    const Range rg = range_of(p, q.ctx, pmin, pmax);

    const int per = (rg.count + p.splits - 1) / p.splits;
    const int b0 = sp * per + wave, b1 = min(rg.count, sp * per + per);

    const uint32_t page1 = (uint32_t)D << c.shift, head_at = head * page1, page = page1 * c.kv_heads;
    const int32_t *const table = c.table + (int64_t)s * c.max_pages;
    uint8_t *const my_keys = keys + wave * T::K_BYTES, *const my_values = values + wave * T::K_BYTES;
    uint32_t kb = 0, vb = 0;        // scale bytes: keys of chunk r16 / 4, values of chunk g
    auto fetch_keys = [&](const Ids<SMALL> &ids, int t0) MXG_INLINE {
        T::template load_keys<1>(c, ids, head_at, page, t0, 0, my_keys);
        kb = c.ks[(size_t)max(ids.of(r16 >> 2), 0) * c.kv_heads + head];
    };
    auto fetch_values = [&](const Ids<SMALL> &ids, int t0) MXG_INLINE {
        T::template load_values<1>(c, ids, head_at, page, t0, 0, my_values);
        vb = c.vs[(size_t)max(ids.of(g), 0) * c.kv_heads + head];
    };
    Ids<SMALL> here = {}, next = {};
    if (b0 < b1) {
        here = ids_of<SMALL>(c, table, rg.start(b0), rg.hi);
        fetch_keys(here, rg.start(b0));
        __atomic_signal_fence(__ATOMIC_SEQ_CST);   // the waits count on this order
        fetch_values(here, rg.start(b0));
        if (b0 + WAVES < b1) next = ids_of<SMALL>(c, table, rg.start(b0 + WAVES), rg.hi);
    }

    // this lane's column: a row of the tile.  A negative softmax scale goes
    // into the sign of Q, so that the largest product is the largest score.
    const uint32_t row = row0 + r16;
    const bool live = row < rows;
    const int qi = (int)((live ? row : row0) / G), qh = (int)((live ? row : row0) % G);
    const int pos = position(q, qi);
    const int from = p.window ? max(pos - p.window + 1, 0) : 0;    // the window's first key
    const float scale = fabsf(p.scale_log2);
    v8bf qf[2 * CH];
    {
        const uint16_t *src = p.Q + (q.q0 + qi) * p.q_stride + (int64_t)(head * G + qh) * D;
        const int flip = p.scale_log2 < 0.0f ? (int)0x80008000u : 0;
#pragma unroll
        for (int h = 0; h < CH; ++h)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                v4i x = *reinterpret_cast<const v4i *>(src + 64 * h + 16 * g + 8 * u);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] ^= flip;
                qf[2 * h + u] = __builtin_bit_cast(v8bf, x);
            }
    }

    v4f o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = v4f{0.f, 0.f, 0.f, 0.f};
    float m = kNone, l = 0.0f;

    // scores of the block in my_keys, each key scaled by ks (chunk r16 / 4)
    auto scores = [&](v4f (&st)[4], float ks) MXG_INLINE {
        v8bf kf[4][2 * CH];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int token = 16 * (r16 >> 2) + 4 * t + (r16 & 3);
#pragma unroll
            for (int h = 0; h < CH; ++h)
                decode16<0>(*reinterpret_cast<const v4i *>(my_keys + T::key(token, 4 * h + g)), ks, kf[t][2 * h],
                            kf[t][2 * h + 1]);
            st[t] = v4f{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int h = 0; h < 2 * CH; ++h)
#pragma unroll
            for (int t = 0; t < 4; ++t) st[t] = mfma_bf16_16(kf[t][h], qf[h], st[t]);
    };
    // the running maximum follows a block's largest score
    auto follow = [&](float mx) MXG_INLINE {
        mx = max_groups(mx);
        if (__builtin_amdgcn_ballot_w64(mx > m + 8.0f)) {
            const float mn = fmaxf(m, mx), alpha = mn == kNone ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= alpha;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= alpha;
        }
        return m == kNone ? 0.0f : m;
    };
    // O^T += V^T P^T from my_values; keep: which of the lane's chunk counts
    auto add = [&](auto EDGE, const v8bf (&pf)[2], float vs, uint32_t keep) MXG_INLINE {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            v4i x = *reinterpret_cast<const v4i *>(my_values + T::value(16 * d + r16, g));
            if constexpr (decltype(EDGE)::value) x = keep16(x, keep);
            v8bf lo, hi;
            decode16<0>(x, vs, lo, hi);
            o[d] = mfma_bf16_16(lo, pf[0], o[d]);
            o[d] = mfma_bf16_16(hi, pf[1], o[d]);
        }
    };

    for (int i = b0; i < b1; i += WAVES) {
        const int t0 = rg.start(i);
        const bool more = i + WAVES < b1;
        wait_vmcnt<HALF>();   // the keys; the values were loaded behind them
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        const uint32_t kb_now = kb;
        auto next_keys = [&]() MXG_INLINE {   // the keys' reads have returned
            wait_lds();
            if (more) fetch_keys(next, rg.start(i + WAVES));
        };
        auto wait_values = [&]() MXG_INLINE {
            if (more) wait_vmcnt<HALF>();
            else wait_vmem();
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
        };
        v4f st[4];
        v8bf pf[2];
        uint32_t see = 0xffff;      // which of the lane's keys its row sees
        // the values' byte came behind the keys: it is waited for with the values
        const bool whole = here.all() && t0 + BLOCK <= rg.hi && t0 + BLOCK - 1 <= pmin &&
                           (!p.window || t0 > pmax - p.window) &&
                           __builtin_amdgcn_ballot_w64(!plain_scale(kb_now)) == 0;
        if (whole) {
            scores(st, e8m0_to_f32(kb_now));
            next_keys();
            float mx = kNone;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) mx = fmaxf(mx, st[t][e]);   // a NaN score passes by: it makes the sum NaN
            const float mu = follow(mx * scale);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    st[t][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(st[t][e], scale, -mu));
                    l += st[t][e];
                }
        } else {
            scores(st, 1.0f);
            next_keys();
            // chunk g's byte is held by the lanes with r16 / 4 = g
            const float ks = e8m0_to_f32((uint32_t)__shfl((int)kb_now, 4 * g, 64)) * scale;
            see = here.of(g) >= 0 ? seen16(from, min(pos + 1, rg.hi), p.sinks, t0 + 16 * g) : 0;
            float mx = kNone;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    st[t][e] = score_or_none(spread(see, 4 * t + e), st[t][e] * ks);
                    mx = fmaxf(mx, st[t][e]);
                }
            const float mu = follow(mx);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    st[t][e] = __builtin_amdgcn_exp2f(st[t][e] - mu);   // 0 where masked
                    l += st[t][e];
                }
        }
        wait_values();
        const float vs = e8m0_to_f32(vb);
        if (whole && __builtin_amdgcn_ballot_w64(!plain_scale(vb)) == 0) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) pf[t >> 1][4 * (t & 1) + e] = (__bf16)st[t][e];
            add(std::false_type{}, pf, vs, 0);
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    pf[t >> 1][4 * (t & 1) + e] = (__bf16)value_or_zero(spread(see, 4 * t + e), st[t][e] * vs);
            add(std::true_type{}, pf, 1.0f, here.of(g) >= 0 ? seen16(rg.lo, rg.hi, rg.sinks, t0 + 16 * g) : 0);
        }
        wait_lds();           // the values' reads have returned
        if (more) {
            fetch_values(next, rg.start(i + WAVES));
            here = next;
            if (i + 2 * WAVES < b1) next = ids_of<SMALL>(c, table, rg.start(i + 2 * WAVES), rg.hi);
        }
    }
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);

    // the waves' sums, joined in wave order, in the keys' buffer
    __shared__ float wm[WAVES][ROWS], wl[WAVES][ROWS];
    v4f *const wo = reinterpret_cast<v4f *>(keys);
    static_assert(WAVES * DT * 64 * 16 <= WAVES * T::K_BYTES, "the sums fit");
    wait_lds();
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
    for (int d = 0; d < DT; ++d) wo[(wave * DT + d) * 64 + lane] = o[d] * mine;
    __syncthreads();
    const int64_t tile = (((int64_t)s * c.kv_heads + head) * p.row_tiles + rt) * p.splits + sp;
    float *const part = p.ws + tile * (ROWS * (D + 2));
#pragma unroll
    for (int d = wave; d < DT; d += WAVES) {
        v4f v = wo[d * 64 + lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v += wo[(w * DT + d) * 64 + lane];
        // column r16, rows (dims) 16 d + 4 g .. + 3
        if (p.splits > 1) {
            if (live) *reinterpret_cast<v4f *>(part + r16 * D + 16 * d + 4 * g) = v;
        } else if (live) {
            v *= lt == 0.0f ? 0.0f : 1.0f / lt;
            *reinterpret_cast<v2i *>(p.O + (q.q0 + qi) * p.o_stride + (int64_t)(head * G + qh) * D + 16 * d + 4 * g) =
                v2i{(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3])};
        }
    }
    if (wave == 0 && g == 0) {
        if (p.splits > 1) {   // rows past the sequence's are never joined
            part[ROWS * D + r16] = mt;
            part[ROWS * D + ROWS + r16] = lt;
        } else if (live && p.lse) {
            p.lse[(q.q0 + qi) * p.q_heads + head * G + qh] = (mu + __builtin_log2f(lt)) * kLn2;
        }
    }
}

} // namespace attn
} // namespace mxg

// mxattn_prompt.h -- attention over the 8-bit cache for many query rows
// (prompts, entered whole or in pieces): MFMA- and VALU-bound.
//
// A workgroup of four waves takes 128 rows ((new token, query head of the
// group) pairs, in token order), 32 a wave, and walks the visible keys in
// blocks of 64, whose keys and values the waves load into one of two LDS
// buffers together while the other is used: as codes, so that a read moves
// half the bytes; each wave widens what it reads.  As compiled, a wave's own
// work hides little of these loads: with pages of 64 and more a block's scale
// bytes are wave-uniform, so the compiler moves them to scalar registers as
// soon as they are asked for, and waits for the whole block with them (loads
// return in order) before it starts on the one at hand; with smaller pages the
// bytes stay per lane and that wait stands behind the first product.  The
// SIMD's other wave computes meanwhile.  Per block a wave computes
//   S^T = K Q^T, O^T += V^T P^T     32x32x16 bf16 MFMA
// with a row in each MFMA column (lane l: row l % 32, lane half h = l / 32).
// As in the decode kernel the softmax needs no exchange of data: the token
// that MFMA row r of tile t (32 tokens) stands for is
//   32 t + 16 (r / 4 % 2) + 8 (r / 16) + 4 (r / 8 % 2) + r % 4,
// so that a lane's registers are the 16 tokens of chunk 2 t + h in order,
// which is what it supplies to the second product, and 16 contiguous bytes of
// each row of the values.  The chunk's scale bytes go into the widening.
//
// Blocks beyond a wave's own rows (causality, the window) are skipped by the
// wave; pairs of whole blocks run in a loop without masks.  The running maximum
// lags as in the decode kernel (rescaling 64 registers at every block
// otherwise).  The longest rows' workgroups start first.  Few rows over many
// keys are split along the keys.
//
// 2 x 2048 rows over 8192 keys, 32 / 8 heads, dim 128: 443 us, 985 TFLOP/s.
// The SIMDs are busy issuing: per wave and block 32 MFMAs (1024 cycles) and
// about 280 other vector instructions (1300 cycles), 128 of them the widening.
// Widening once for all four waves through LDS (540 us) and running the first
// product a block ahead (540 us) spent as many instructions elsewhere.  Of a
// SIMD's two waves the one in its products goes first (470 us without; at dim
// 64, where the softmax is half the work, 305 us without and 323 us with).
#pragma once

#include "mxattn.h"

#include <type_traits>

namespace mxg {
namespace attn_prompt {

using namespace attn;

constexpr int WAVES = 4, THREADS = 64 * WAVES, WAVE_ROWS = 32, ROWS = WAVES * WAVE_ROWS;

// SPLIT: an instantiation of its own, whose epilogue costs the other no registers
template <int D, bool SMALL, bool SPLIT>
__global__ __launch_bounds__(THREADS, 2) void kernel(AttnArgs p)
{
    constexpr int CH = D / 32;      // 16-byte key chunks per lane and token
    constexpr int DT = D / 32;      // 32-row tiles of O^T
    constexpr bool PRIO = D == 128; // the products before the other wave's softmax
    using T = Tile<D>;
    __shared__ __attribute__((aligned(1024))) uint8_t buf0[T::BYTES], buf1[T::BYTES];
    const Pages &c = p.c;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r32 = lane & 31, h = lane >> 5;
    uint32_t bid = blockIdx.x;
    const int sp = SPLIT ? (int)(bid % (uint32_t)p.splits) : 0;
    if constexpr (SPLIT) bid /= (uint32_t)p.splits;
    const int head = (int)(bid % (uint32_t)c.kv_heads);
    bid /= (uint32_t)c.kv_heads;
    const int s = (int)(bid % (uint32_t)c.seqs);
    const int rt = p.row_tiles - 1 - (int)(bid / (uint32_t)c.seqs);

    const Seq q = cache::sequence(c, s);
    const uint32_t G = p.group;       // the launch has fewer than 2^24 tiles, so rows fit 32 bits
    const uint32_t rows = (uint32_t)q.n * G, row0 = (uint32_t)rt * ROWS;
    if (row0 >= rows) return;
    const Range rg = range_of(p, q.ctx, position(q, row0 / G), position(q, (min(row0 + ROWS, rows) - 1) / G));
    // this wave's rows
    const uint32_t w0 = row0 + wave * WAVE_ROWS;
    const bool any = w0 < rows;
    const int pmin = position(q, (any ? w0 : row0) / G);
    const int pmax = position(q, (any ? min(w0 + WAVE_ROWS, rows) - 1 : row0) / G);
    const uint32_t row = w0 + r32;
    const bool live = row < rows;
    const int qi = (int)((live ? row : row0) / G), qh = (int)((live ? row : row0) % G);
    const int pos = position(q, qi);
    const int from = p.window ? max(pos - p.window + 1, 0) : 0;    // the window's first key
    const float scale = fabsf(p.scale_log2);

    const uint32_t page1 = (uint32_t)D << c.shift, head_at = head * page1, page = page1 * c.kv_heads;
    const int32_t *const table = c.table + (int64_t)s * c.max_pages;
    // a block's tile into LDS, and the scale bytes of this lane's chunks 2t + h
    uint32_t kb[2] = {}, vb[2] = {};
    auto fetch = [&](uint8_t *dst, const Ids<SMALL> &ids, int t0) MXG_INLINE {
        T::template load_keys<WAVES>(c, ids, head_at, page, t0, wave, dst);
        T::template load_values<WAVES>(c, ids, head_at, page, t0, wave, dst + T::K_BYTES);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const size_t at = (size_t)(uint32_t)max(ids.of(2 * t + h), 0) * c.kv_heads + head;
            kb[t] = c.ks[at];
            vb[t] = c.vs[at];
        }
    };
    // this split's blocks
    const int per = SPLIT ? (rg.count + p.splits - 1) / p.splits : rg.count;
    const int b0 = sp * per, b1 = min(rg.count, b0 + per);
    Ids<SMALL> here = {}, next = {};        // of the block at hand and the one behind it
    if (b0 < b1) {
        here = ids_of<SMALL>(c, table, rg.start(b0), rg.hi);
        fetch(buf0, here, rg.start(b0));
        if (b0 + 1 < b1) next = ids_of<SMALL>(c, table, rg.start(b0 + 1), rg.hi);
    }

    v8bf qf[2 * CH];
    {
        const uint16_t *src = p.Q + (q.q0 + qi) * p.q_stride + (int64_t)(head * G + qh) * D;
        const int flip = p.scale_log2 < 0.0f ? (int)0x80008000u : 0;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                v4i x = *reinterpret_cast<const v4i *>(src + 16 * (2 * i + h) + 8 * u);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] ^= flip;
                qf[2 * i + u] = __builtin_bit_cast(v8bf, x);
            }
    }
    v16f o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = v16f{};
    float m = kNone, l = 0.0f;
    // token of MFMA row r32 in its tile, and that row's chunk
    const int token = 16 * (r32 >> 2 & 1) + 8 * (r32 >> 4) + 4 * (r32 >> 3 & 1) + (r32 & 3);

    auto block = [&](auto EDGE, const uint8_t *src, const Ids<SMALL> &ids, int t0, const uint32_t (&kb)[2],
                     const uint32_t (&vb)[2]) MXG_INLINE {
        constexpr bool edge = decltype(EDGE)::value;
        v16f st[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            // kb, vb are of the lane's own chunk 2t + h; the key row r32 lies in
            // chunk 2t + (r32 / 4 % 2)
            float ks = 1.0f;
            if constexpr (!edge)
                ks = e8m0_to_f32(SMALL ? (uint32_t)__shfl((int)kb[t], 32 * (r32 >> 2 & 1), 64) : kb[t]);
            st[t] = v16f{};
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                v8bf lo, hi;
                decode16<0>(*reinterpret_cast<const v4i *>(src + T::key(32 * t + token, 2 * i + h)), ks, lo, hi);
                st[t] = mfma_bf16_32(lo, qf[2 * i], st[t]);
                st[t] = mfma_bf16_32(hi, qf[2 * i + 1], st[t]);
            }
        }
        if constexpr (PRIO) __builtin_amdgcn_s_setprio(0);
        float mx = kNone;
        uint32_t see[2] = {};       // which of the lane's keys its row sees
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const float ks = edge ? e8m0_to_f32(kb[t]) * scale : 1.0f;
            if constexpr (edge)
                see[t] = ids.of(2 * t + h) >= 0 ? seen16(from, min(pos + 1, rg.hi), p.sinks, t0 + 32 * t + 16 * h) : 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                if constexpr (edge) st[t][e] = score_or_none(spread(see[t], e), st[t][e] * ks);
                mx = fmaxf(mx, st[t][e]);   // a NaN score passes by: it makes the row's sum NaN
            }
        }
        if constexpr (!edge) mx *= scale;
        {
            const uint32_t b = __builtin_bit_cast(uint32_t, mx);
            const auto u = __builtin_amdgcn_permlane32_swap(b, b, false, false);
            const uint32_t u0 = u[0], u1 = u[1];
            mx = fmaxf(__builtin_bit_cast(float, u0), __builtin_bit_cast(float, u1));
        }
        if (__builtin_amdgcn_ballot_w64(mx > m + 8.0f)) {
            const float mn = fmaxf(m, mx), alpha = mn == kNone ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= alpha;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= alpha;
        }
        const float mu = m == kNone ? 0.0f : m;
        v8bf pf[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const float vs = edge ? e8m0_to_f32(vb[t]) : 1.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                float x;
                if constexpr (edge) {
                    x = __builtin_amdgcn_exp2f(st[t][e] - mu);     // 0 where masked
                    l += x;
                    x = value_or_zero(spread(see[t], e), x * vs);
                } else {
                    x = __builtin_amdgcn_exp2f(__builtin_fmaf(st[t][e], scale, -mu));
                    l += x;
                }
                pf[t][e >> 3][e & 7] = (__bf16)x;
            }
        }
        if constexpr (PRIO) __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const float vs = edge ? 1.0f : e8m0_to_f32(vb[t]);
            // what no row sees is no number that may meet a zero
            const uint32_t keep =
                edge && ids.of(2 * t + h) >= 0 ? seen16(rg.lo, rg.hi, rg.sinks, t0 + 32 * t + 16 * h) : 0;
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                v4i x = *reinterpret_cast<const v4i *>(src + T::K_BYTES + T::value(32 * d + r32, 2 * t + h));
                if constexpr (edge) x = keep16(x, keep);
                v8bf lo, hi;
                decode16<0>(x, vs, lo, hi);
                o[d] = mfma_bf16_32(lo, pf[t][0], o[d]);
                o[d] = mfma_bf16_32(hi, pf[t][1], o[d]);
            }
        }
    };

    // Block i has landed for every wave and the other buffer is read out: load
    // block i + 1 there.
    auto advance = [&](int i, uint8_t *other, uint32_t (&kb_now)[2], uint32_t (&vb_now)[2]) MXG_INLINE {
        wait_vmem();
        wait_lds();
        barrier_nofence();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            kb_now[t] = kb[t];
            vb_now[t] = vb[t];
        }
        if (i + 1 < b1) {
            fetch(other, next, rg.start(i + 1));
            here = next;
            if (i + 2 < b1) next = ids_of<SMALL>(c, table, rg.start(i + 2), rg.hi);
        }
    };
    auto step = [&](auto EDGE, int i, const uint8_t *src, uint8_t *other) MXG_INLINE {
        const int t0 = rg.start(i);
        const Ids<SMALL> ids = here;
        uint32_t kb_now[2], vb_now[2];
        advance(i, other, kb_now, vb_now);
        if constexpr (decltype(EDGE)::value) {
            // a wave that sees nothing of the block has no part in it
            if (!any || t0 > pmax || (p.window && t0 + BLOCK - 1 <= pmin - p.window && t0 >= p.sinks)) return;
        }
        block(EDGE, src, ids, t0, kb_now, vb_now);
    };
    // every row of this wave sees the whole block, whose pages are all there
    // (then a byte 255 may spread: every row is due its NaN)
    auto whole = [&](int i, const Ids<SMALL> &ids) MXG_INLINE {
        const int t0 = rg.start(i);
        return any && ids.all() && t0 + BLOCK <= rg.hi && t0 + BLOCK - 1 <= pmin && (!p.window || t0 > pmax - p.window);
    };
    // Pairs of whole blocks run in a loop of their own: with both kinds of block
    // in one loop the sums changed registers at every block.
    for (int i = b0; i < b1; i += 2) {
        for (; i + 1 < b1 && whole(i, here) && whole(i + 1, next); i += 2) {
            step(std::false_type{}, i, buf0, buf1);
            step(std::false_type{}, i + 1, buf1, buf0);
        }
        if (i >= b1) break;
        step(std::true_type{}, i, buf0, buf1);
        if (i + 1 < b1) step(std::true_type{}, i + 1, buf1, buf0);
    }

    l += __shfl_xor(l, 32, 64);
    if (!live) return;
    if constexpr (SPLIT) {
        // a part of its own for every split of the tile, joined by a second kernel
        const int64_t tile = (((int64_t)s * c.kv_heads + head) * p.row_tiles + rt) * p.splits + sp;
        float *const part = p.ws + tile * (ROWS * (D + 2));
        const int r = wave * WAVE_ROWS + r32;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<v4f *>(part + r * D + 32 * d + 8 * e + 4 * h) =
                    v4f{o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
        if (h == 0) {
            part[ROWS * D + r] = m;
            part[ROWS * D + ROWS + r] = l;
        }
        return;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    // column r32, rows (dims) 32 d + 8 e + 4 h .. + 3
    uint16_t *const dst = p.O + (q.q0 + qi) * p.o_stride + (int64_t)(head * G + qh) * D;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x0 = o[d][4 * e] * inv, x1 = o[d][4 * e + 1] * inv, x2 = o[d][4 * e + 2] * inv,
                        x3 = o[d][4 * e + 3] * inv;
            *reinterpret_cast<v2i *>(dst + 32 * d + 8 * e + 4 * h) = v2i{(int)pack_bf16x2(x0, x1), (int)pack_bf16x2(x2, x3)};
        }
    if (h == 0 && p.lse)
        p.lse[(q.q0 + qi) * p.q_heads + head * G + qh] = ((m == kNone ? 0.0f : m) + __builtin_log2f(l)) * kLn2;
}

} // namespace attn_prompt
} // namespace mxg

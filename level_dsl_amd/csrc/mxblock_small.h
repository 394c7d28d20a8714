// mxblock_small.h -- product of codes with one fp32 scale per 128 K, small
// tiles: every shape, meant for those that leave the 256 x 256 tiles' grid
// short (few rows, or few columns).
//
// One workgroup of 8 waves computes 16 MT rows by 16 CT columns of C.  The
// waves split K: wave w takes blocks w, w + 8, ... of 128, so together they
// read 1 KiB of a row at a time, each wave straight from global memory into
// the MFMA operand registers (no operand byte is used by two waves, so LDS
// would add a trip and nothing else).  Block sums meet in LDS at the end, in
// wave order.
//
// One block b of 16 x 16 outputs: the codes are widened to bf16 (exact) and
// summed by four 16x16x32 bf16 MFMAs into a fresh register tile, which joins
// the fp32 accumulator times the block's scales (one FMA per output).
// Roles as in the other kernels: B supplies the MFMA's rows and A its columns,
// so a lane holds four consecutive columns of one row of C.
// An MFMA sums over its K positions in any order, so lane group g = l / 16
// takes bytes 16g .. +15 and 64 + 16g .. +15 of the block for both operands:
// each load instruction reads 64 contiguous bytes per row.
#pragma once

#include "mxblock.h"
#include "mxgemm_common.h"

namespace mxg {
namespace block_small {

constexpr int WAVES = 8, THREADS = 64 * WAVES;

template <int FA, int FB, int ROWS_B, int MT, int CT>
__global__ __launch_bounds__(THREADS, 2) void kernel(block::Args p)
{
    static_assert(128 % (16 * CT) == 0, "a tile's columns share one 128-column block of scales");
    constexpr int BM = 16 * MT, BN = 16 * CT;
    __shared__ v4f red[WAVES][MT * CT][64];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    // rows fastest: the workgroups that share columns of B run together
    const int tm = blockIdx.x % p.tiles_m, tn = blockIdx.x / p.tiles_m;
    const int m0 = tm * BM, n0 = tn * BN;
    const int rows_a = min(BM, p.M - m0), rows_b = min(BN, p.N - n0);
    const int K = p.K, KB = p.KB;
    const rsrc_t rA = make_rsrc(p.A + (size_t)m0 * K, (uint32_t)rows_a * K);
    const rsrc_t rB = make_rsrc(p.B + (size_t)n0 * K, (uint32_t)rows_b * K);
    const rsrc_t rAs = make_rsrc(p.As + (size_t)m0 * KB, (uint32_t)rows_a * KB * 4);
    const float *const bs = p.Bs + (size_t)(ROWS_B == 1 ? n0 : n0 / 128) * KB;
    const rsrc_t rBs = make_rsrc(bs, ROWS_B == 1 ? (uint32_t)rows_b * KB * 4 : (uint32_t)KB * 4);

    struct Raw {
        v4i a[MT][2], b[CT][2];
        float sa[MT];
        float sb[ROWS_B == 1 ? CT : 1][ROWS_B == 1 ? 4 : 1];
    };
    auto load = [&](int kb, Raw &r) MXG_INLINE {
        // blocks past the end, and chunks past K in the last one, read as zero
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t k = (uint32_t)kb * 128 + 64 * h + 16 * g;
            const bool in = (int)k < K;
#pragma unroll
            for (int i = 0; i < MT; ++i) r.a[i][h] = load16(rA, in ? (uint32_t)(16 * i + r16) * K + k : kOob);
#pragma unroll
            for (int c = 0; c < CT; ++c) r.b[c][h] = load16(rB, in ? (uint32_t)(16 * c + r16) * K + k : kOob);
        }
        const bool in = kb < KB;
#pragma unroll
        for (int i = 0; i < MT; ++i)
            r.sa[i] = __builtin_bit_cast(float, load4(rAs, in ? (uint32_t)((16 * i + r16) * KB + kb) * 4 : kOob));
        if constexpr (ROWS_B == 1) {
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    r.sb[c][e] = __builtin_bit_cast(
                        float, load4(rBs, in ? (uint32_t)((16 * c + 4 * g + e) * KB + kb) * 4 : kOob));
        } else {
            r.sb[0][0] = __builtin_bit_cast(float, load4(rBs, in ? (uint32_t)kb * 4 : kOob));
        }
    };

    v4f acc[MT][CT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[i][c] = v4f{0.f, 0.f, 0.f, 0.f};

    Raw cur, nxt;
    load(wave, cur);
    for (int kb = wave; kb < KB; kb += WAVES) {
        load(kb + WAVES, nxt);
        v8bf fa[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) decode16<FA>(cur.a[i][h], 1.0f, fa[i][2 * h], fa[i][2 * h + 1]);
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            v8bf fb[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) decode16<FB>(cur.b[c][h], 1.0f, fb[2 * h], fb[2 * h + 1]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                v4f t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < 4; ++q) t = mfma_bf16_16(fb[q], fa[i][q], t);
                if constexpr (ROWS_B == 1) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][c][e] += t[e] * (cur.sa[i] * cur.sb[c][e]);
                } else {
                    const float s = cur.sa[i] * cur.sb[0][0];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][c][e] += t[e] * s;
                }
            }
        }
        cur = nxt;
    }

#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < CT; ++c) red[wave][i * CT + c][lane] = acc[i][c];
    __syncthreads();
    const int esz = p.out_bf16 ? 2 : 4;
    const rsrc_t rC = make_rsrc((uint8_t *)p.C + (size_t)m0 * p.N * esz, (uint32_t)rows_a * p.N * esz);
    for (int t = wave; t < MT * CT; t += WAVES) {
        v4f v = red[0][t][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v += red[w][t][lane];
        const int n = n0 + 16 * (t % CT) + 4 * g;
        store_c4(rC, (uint32_t)(16 * (t / CT) + r16) * p.N + n, n, p.N, v, p.out_bf16, p.use_acc, p.c_vec);
    }
}

} // namespace block_small
} // namespace mxg

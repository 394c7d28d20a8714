// mxblock_small.h -- product of codes with one fp32 scale per 128 K, small
// tiles: every shape, meant for those that leave the 256-row tiles' grid short
// (few rows, or few columns).
//
// One workgroup of W waves computes 16 MT rows by 16 CT columns of C.  The
// waves split K: wave w takes blocks w, w + W, ... of 128.  No operand byte is
// used by two waves, so each runs on its own, without barriers until the waves'
// sums meet at the end, in wave order.  A block's codes come by direct-to-LDS
// loads into the wave's only buffer and from there into registers as they are;
// then the next block's loads go out, and the block is multiplied meanwhile.
// (A ring of buffers read during the product holds fewer waves: 1024 x 1024 x
// 4096: 14 us, with two buffers of twice the size 21 us.)  The loads go through
// LDS although nothing is shared because of the address path: loading MFMA
// operands straight into registers, neighbouring lanes read different rows,
// every 16 bytes a cache-line lookup of its own (M = 64, N = 28672, K = 8192:
// 140 us, against 63); a direct-to-LDS load reads whole 128-byte lines of 8 rows.
//
// One block b of 16 x 16 outputs: the codes are widened to bf16 (exact) and
// summed by four 16x16x32 bf16 MFMAs into a fresh register tile, which joins
// the fp32 accumulator times the block's scales (one FMA per output).
// Roles as in the other kernels: B supplies the MFMA's rows and A its columns,
// so a lane holds four consecutive columns of one row of C.
// An MFMA sums over its K positions in any order, so lane group g = l / 16
// takes chunks g and 4 + g (of 16 bytes) of a row for both operands.  Chunk c
// of row r sits at position c ^ (r & 7) of its 128 bytes.  A's scales of a
// block are one dword load (lane l: row l), handed out by lane exchanges.
//
// Bound by the bytes that move from the L2s into LDS, about 50 GB/s a CU: a
// 64 x 64 tile reads 16 KB for 2^19 products.  The workgroups of one XCD take
// neighbouring tiles, so that its L2 reads few columns of B (333 x 3584 x 4112:
// 24 us, 30 with tiles dealt in order).
#pragma once

#include "mxblock.h"
#include "mxgemm_common.h"
#include "mxgemm_large.h"

namespace mxg {
namespace block_small {

// Wait until every LDS read of this wave has returned.
__device__ __forceinline__ void wait_lds()
{
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

template <int FA, int FB, int ROWS_B, int MT, int CT, int W>
__global__ __launch_bounds__(64 * W, 2) void kernel(block::Args p)
{
    static_assert(128 % (16 * CT) == 0, "a tile's columns share one 128-column block of scales");
    static_assert(MT <= 4 && CT <= 4, "one lane per row of scales");
    constexpr int BM = 16 * MT, BN = 16 * CT;
    constexpr int A_BYTES = BM * 128, STEP = (BM + BN) * 128;
    static_assert(MT * CT * 64 * 16 <= STEP, "the waves' sums fit their buffers");
    __shared__ __attribute__((aligned(1024))) uint8_t bufs[W * STEP];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    uint8_t *const buf = bufs + wave * STEP;
    int tm, tn;
    large::tile_of(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int rows_a = min(BM, p.M - m0), rows_b = min(BN, p.N - n0);
    const int K = p.K, KB = p.KB;
    const rsrc_t rA = make_rsrc(p.A + (size_t)m0 * K, (uint32_t)rows_a * K);
    const rsrc_t rB = make_rsrc(p.B + (size_t)n0 * K, (uint32_t)rows_b * K);
    const rsrc_t rAs = make_rsrc(p.As + (size_t)m0 * KB, (uint32_t)rows_a * KB * 4);
    const float *const bs = p.Bs + (size_t)(ROWS_B == 1 ? n0 : n0 / 128) * KB;
    const rsrc_t rBs = make_rsrc(bs, ROWS_B == 1 ? (uint32_t)rows_b * KB * 4 : (uint32_t)KB * 4);

    struct Scales {
        float a, b;  // lane l: row l's; b: column l's, or the tile's
    };
    const uint32_t chunk = (uint32_t)((lane & 7) ^ (lane >> 3)) * 16, row8 = (uint32_t)(lane >> 3) * K;
    // block kb into the buffer; past the end of K everything reads as zero
    auto load = [&](int kb, Scales &sc) MXG_INLINE {
        const uint32_t k = (uint32_t)kb * 128 + chunk;
        const bool in = (int)k < K;
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) load16_lds(rA, buf + i * 1024, in ? row8 + (uint32_t)(8 * i) * K + k : kOob);
#pragma unroll
        for (int i = 0; i < 2 * CT; ++i)
            load16_lds(rB, buf + A_BYTES + i * 1024, in ? row8 + (uint32_t)(8 * i) * K + k : kOob);
        sc.a = __builtin_bit_cast(float, load4(rAs, kb < KB && lane < BM ? (uint32_t)(lane * KB + kb) * 4 : kOob));
        if constexpr (ROWS_B == 1)
            sc.b = __builtin_bit_cast(float, load4(rBs, kb < KB && lane < BN ? (uint32_t)(lane * KB + kb) * 4 : kOob));
        else
            sc.b = scalar_load(bs + min(kb, KB - 1));
    };

    v4f acc[MT][CT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[i][c] = v4f{0.f, 0.f, 0.f, 0.f};

    const int sw = r16 & 7;
    const uint32_t o0 = (uint32_t)(r16 * 128 + ((g ^ sw) << 4)), o1 = (uint32_t)(r16 * 128 + (((4 + g) ^ sw) << 4));
    Scales now, next;
    load(wave, next);
    // every wave takes the same number of steps; blocks past K add zeros
    const int steps = (KB + W - 1) / W;
    for (int t = 0; t < steps; ++t) {
        wait_vmem();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        now = next;
        v4i xa[MT][2], xb[CT][2];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            xb[c][0] = *reinterpret_cast<const v4i *>(buf + A_BYTES + c * 2048 + o0);
            xb[c][1] = *reinterpret_cast<const v4i *>(buf + A_BYTES + c * 2048 + o1);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            xa[i][0] = *reinterpret_cast<const v4i *>(buf + i * 2048 + o0);
            xa[i][1] = *reinterpret_cast<const v4i *>(buf + i * 2048 + o1);
        }
        wait_lds();   // the buffer is free
        if (t + 1 < steps) load(wave + W * (t + 1), next);
        v8bf fb[CT][4];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            decode16<FB>(xb[c][0], 1.0f, fb[c][0], fb[c][1]);
            decode16<FB>(xb[c][1], 1.0f, fb[c][2], fb[c][3]);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            v8bf fa[4];
            decode16<FA>(xa[i][0], 1.0f, fa[0], fa[1]);
            decode16<FA>(xa[i][1], 1.0f, fa[2], fa[3]);
            float s = __shfl(now.a, 16 * i + r16, 64);
            if constexpr (ROWS_B != 1) s *= now.b;
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                v4f u = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 4; ++h) u = mfma_bf16_16(fb[c][h], fa[h], u);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (ROWS_B == 1)
                        acc[i][c][e] += u[e] * (s * __shfl(now.b, 16 * c + 4 * g + e, 64));
                    else
                        acc[i][c][e] += u[e] * s;
                }
            }
        }
    }

    __syncthreads();   // every load has landed and been read
    v4f *const red = reinterpret_cast<v4f *>(bufs);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < CT; ++c) red[(wave * MT * CT + i * CT + c) * 64 + lane] = acc[i][c];
    __syncthreads();
    const int esz = p.out_bf16 ? 2 : 4;
    const rsrc_t rC = make_rsrc((uint8_t *)p.C + (size_t)m0 * p.N * esz, (uint32_t)rows_a * p.N * esz);
    for (int t = wave; t < MT * CT; t += W) {
        v4f v = red[t * 64 + lane];
#pragma unroll
        for (int w = 1; w < W; ++w) v += red[(w * MT * CT + t) * 64 + lane];
        const int n = n0 + 16 * (t % CT) + 4 * g;
        store_c4(rC, (uint32_t)(16 * (t / CT) + r16) * p.N + n, n, p.N, v, p.out_bf16, p.use_acc, p.c_vec);
    }
}

} // namespace block_small
} // namespace mxg

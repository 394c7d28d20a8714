// mxblock_large.h -- product of codes with one fp32 scale per 128 K, large
// tiles (MFMA-bound shapes).
//
// One workgroup of eight waves, two per SIMD, computes 256 rows by BN columns
// of C; a wave owns 64 x (16 NT).  A stage is one block of 128 K: its A and B
// tiles come by direct-to-LDS loads into one of two LDS buffers while the
// other is multiplied, swizzled like the other kernels' (16-byte chunk c of
// row r at position c ^ (r & 7): eight consecutive rows' same chunk, one LDS
// pass, hits all banks once).
//
// The scales are fp32, so they cannot ride in the MFMA's e8m0 operands: a
// block's sum starts at zero in a register tile of its own and joins the
// accumulator by one FMA per output.  VALU instructions cannot read
// accumulator registers (AGPRs), which is why a wave's tile is 64 x 128
// (128 accumulators in ordinary registers) and not the 128 x 128 of the kernels
// that scale inside the MFMA.  The 16x16 MFMA shapes keep the block sums
// short-lived (4 registers each): the sums of column tile j are scaled while
// the MFMAs of tile j + 1 run.
//   native: one 16x16x128 fp8 MFMA is a whole block
//   exact:  codes widened to bf16, four 16x16x32 bf16 MFMAs; NT is 4, so that the
//           wave's A rows fit as bf16 (64 registers, widened once a stage)
// An MFMA sums over its K positions in any order, so lane group g = l / 16
// takes chunks g and 4 + g of a row for both operands.
//
// Scales come four stages at a time (16 bytes of a row of As, or of Bs when B
// has a scale per row), loaded a window ahead into registers and turned into
// [stage][row] order in LDS, so that a lane's rows are one conflict-free
// read.  With 128 x 128 blocks, B's scale is one scalar per wave and stage.
#pragma once

#include "mxblock.h"
#include "mxgemm_common.h"
#include "mxgemm_large.h"

namespace mxg {
namespace block_large {

constexpr int WAVES = 8, THREADS = 64 * WAVES;
constexpr int BM = 256, BK = 128, MT = 4;

template <bool NATIVE>
constexpr int columns() { return NATIVE ? 256 : 128; }

// One 16x16x128 fp8 MFMA without block scales.
template <int FX, int FY>
__device__ __forceinline__ v4f mfma_f8_16(v8i x, v8i y, v4f c)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, FX, FY, 0, 0, 0, 0);
}

template <int FA, int FB, int ROWS_B, bool NATIVE>
__global__ __launch_bounds__(THREADS, 2) void kernel(block::Args p)
{
    constexpr int BN = columns<NATIVE>(), NT = BN / 32;   // column tiles of a wave
    constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK;
    constexpr int A_SEGS = A_BYTES / 1024 / WAVES, B_SEGS = B_BYTES / 1024 / WAVES;
    // separate objects, so that a read of one does not wait for loads into the other
    __shared__ __attribute__((aligned(1024))) uint8_t lds0[A_BYTES + B_BYTES];
    __shared__ __attribute__((aligned(1024))) uint8_t lds1[A_BYTES + B_BYTES];
    __shared__ float scale_a[2][4][BM];
    __shared__ float scale_b[ROWS_B == 1 ? 2 : 1][ROWS_B == 1 ? 4 : 1][ROWS_B == 1 ? BN : 1];

    int tm, tn;
    large::tile_of(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int rows_a = min(BM, p.M - m0), rows_b = min(BN, p.N - n0);
    const int K = p.K, KB = p.KB;
    const rsrc_t rA = make_rsrc(p.A + (size_t)m0 * K, (uint32_t)rows_a * K);
    const rsrc_t rB = make_rsrc(p.B + (size_t)n0 * K, (uint32_t)rows_b * K);
    const rsrc_t rAs = make_rsrc(p.As + (size_t)m0 * KB, (uint32_t)rows_a * KB * 4);

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 3, wn = wave >> 2;
    const int r16 = lane & 15, g = lane >> 4;

    // B's scales: one row of Bs per 128 columns, or one per column
    const int nb = min(n0 + wn * 16 * NT, p.N - 1) / 128;
    const float *const bs = p.Bs + (size_t)(ROWS_B == 1 ? n0 : nb) * KB;
    const rsrc_t rBs = make_rsrc(bs, ROWS_B == 1 ? (uint32_t)rows_b * KB * 4 : (uint32_t)KB * 4);

    // segment s holds tile rows 8s .. 8s+7; lane i writes row 8s + i/8 at chunk
    // position i % 8, i.e. global chunk (i % 8) ^ (i / 8)
    const uint32_t chunk = ((lane & 7) ^ (lane >> 3)) * 16;
    const uint32_t rowA = (uint32_t)(8 * A_SEGS * wave + (lane >> 3)) * K;
    const uint32_t rowB = (uint32_t)(8 * B_SEGS * wave + (lane >> 3)) * K;
    auto gload = [&](uint8_t *buf, int kt) MXG_INLINE {
        const uint32_t k = (uint32_t)kt * BK + chunk;
        const bool in = (int)k < K;
#pragma unroll
        for (int j = 0; j < A_SEGS; ++j)
            load16_lds(rA, buf + (A_SEGS * wave + j) * 1024, in ? rowA + (uint32_t)(8 * j) * K + k : kOob);
#pragma unroll
        for (int j = 0; j < B_SEGS; ++j)
            load16_lds(rB, buf + A_BYTES + (B_SEGS * wave + j) * 1024, in ? rowB + (uint32_t)(8 * j) * K + k : kOob);
    };
    // scale windows: thread t < 256 a row of As, thread 256 + t a row of Bs
    // (ROWS_B == 1).  Values past a row's end are of stages that do not exist.
    const bool win_a = tid < BM, win_b = ROWS_B == 1 && tid >= BM && tid < BM + BN;
    auto wload = [&](int kt) MXG_INLINE -> v4i {
        if (win_a) return load16(rAs, ((uint32_t)tid * KB + kt) * 4);
        if (win_b) return load16(rBs, ((uint32_t)(tid - BM) * KB + kt) * 4);
        return v4i{0, 0, 0, 0};
    };
    auto wstore = [&](int w, v4i x) MXG_INLINE {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int xe = x[e];  // (a bit cast of x[e] itself reads element 0 for every e)
            if (win_a) scale_a[w][e][tid] = __builtin_bit_cast(float, xe);
            if constexpr (ROWS_B == 1)
                if (win_b) scale_b[w][e][tid - BM] = __builtin_bit_cast(float, xe);
        }
    };

    v4f acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    const int sw = r16 & 7;
    const uint32_t o0 = (uint32_t)((g ^ sw) << 4), o1 = (uint32_t)(((4 + g) ^ sw) << 4);
    const uint32_t fa_off = (uint32_t)(wm * 64 + r16) * BK, fb_off = (uint32_t)(A_BYTES + (wn * 16 * NT + r16) * BK);

    auto compute = [&](const uint8_t *buf, int kt, float sb) MXG_INLINE {
        const int w = (kt >> 2) & 1, e4 = kt & 3;
        float s[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) s[i] = scale_a[w][e4][wm * 64 + 16 * i + r16];
        if constexpr (ROWS_B != 1) {
#pragma unroll
            for (int i = 0; i < MT; ++i) s[i] *= sb;
        }
        auto read = [&](uint32_t off) MXG_INLINE {
            const v4i lo = *reinterpret_cast<const v4i *>(buf + off + o0);
            const v4i hi = *reinterpret_cast<const v4i *>(buf + off + o1);
            return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        };
        auto join = [&](int j, const v4f (&t)[MT]) MXG_INLINE {
            if constexpr (ROWS_B == 1) {
                const v4f sn = *reinterpret_cast<const v4f *>(&scale_b[w][e4][wn * 16 * NT + 16 * j + 4 * g]);
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] += t[i][e] * s[i] * sn[e];
            } else {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] += t[i][e] * s[i];
            }
            // the sums are taken here: without this the compiler puts them off
            // to the end of the loop body and keeps every t until then
#pragma unroll
            for (int i = 0; i < MT; ++i) asm volatile("" : "+v"(acc[i][j]));
        };
        const v4f zero = {0.f, 0.f, 0.f, 0.f};
        // Step j: the MFMAs of column tile j, the scaling of tile j - 1's sums,
        // and the LDS reads of tile j + 1.  A step is a scheduling region of
        // its own: left to itself the compiler issues every MFMA first and
        // spills their sums.
        v4f t[2][MT];
        v8i b[2];
        b[0] = read(fb_off);
        if constexpr (NATIVE) {
            v8i a[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) a[i] = read(fa_off + i * 16 * BK);
            static_for<NT>([&](auto J) MXG_INLINE {
                constexpr int j = decltype(J)::value;
                if constexpr (j + 1 < NT) b[(j + 1) & 1] = read(fb_off + (j + 1) * 16 * BK);
#pragma unroll
                for (int i = 0; i < MT; ++i) t[j & 1][i] = mfma_f8_16<FB, FA>(b[j & 1], a[i], zero);
                if constexpr (j > 0) join(j - 1, t[(j - 1) & 1]);
                __builtin_amdgcn_sched_group_barrier(large::SG_DS_RD, 2, 0);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    __builtin_amdgcn_sched_group_barrier(large::SG_MFMA, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(large::SG_VALU, ROWS_B == 1 ? 8 : 4, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            });
        } else {
            v8bf fa[MT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const v8i x = read(fa_off + i * 16 * BK);
                decode16<FA>(v4i{x[0], x[1], x[2], x[3]}, 1.0f, fa[i][0], fa[i][1]);
                decode16<FA>(v4i{x[4], x[5], x[6], x[7]}, 1.0f, fa[i][2], fa[i][3]);
            }
            __builtin_amdgcn_sched_barrier(0);
            static_for<NT>([&](auto J) MXG_INLINE {
                constexpr int j = decltype(J)::value;
                v8bf fb[4];
                const v8i x = b[j & 1];
                if constexpr (j + 1 < NT) b[(j + 1) & 1] = read(fb_off + (j + 1) * 16 * BK);
                decode16<FB>(v4i{x[0], x[1], x[2], x[3]}, 1.0f, fb[0], fb[1]);
                decode16<FB>(v4i{x[4], x[5], x[6], x[7]}, 1.0f, fb[2], fb[3]);
#pragma unroll
                for (int i = 0; i < MT; ++i) t[j & 1][i] = zero;
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int i = 0; i < MT; ++i) t[j & 1][i] = mfma_bf16_16(fb[q], fa[i][q], t[j & 1][i]);
                if constexpr (j > 0) join(j - 1, t[(j - 1) & 1]);
                __builtin_amdgcn_sched_barrier(0);
            });
        }
        join(NT - 1, t[(NT - 1) & 1]);
    };

    // ---- main loop ----------------------------------------------------------
    gload(lds0, 0);
    v4i win = wload(0);
    wstore(0, win);
    auto sb_of = [&](int kt) MXG_INLINE -> float {
        if constexpr (ROWS_B == 1) return 0.0f;
        return scalar_load(bs + min(kt, KB - 1));
    };
    float sb = sb_of(0);
    wait_vmem();
    __syncthreads();
    auto stage = [&](int kt, uint8_t *buf, uint8_t *other) MXG_INLINE {
        gload(other, kt + 1);                       // past K: zeros, never read
        if ((kt & 3) == 0) win = wload(kt + 4);
        const float sb1 = sb_of(kt + 1);
        compute(buf, kt, sb);
        if ((kt & 3) == 3) wstore(((kt >> 2) + 1) & 1, win);
        sb = sb1;
        wait_vmem();
        __syncthreads();
    };
    int kt = 0;
    for (; kt + 2 <= KB; kt += 2) {
        stage(kt, lds0, lds1);
        stage(kt + 1, lds1, lds0);
    }
    if (kt < KB) stage(kt, lds0, lds1);

    // ---- epilogue -------------------------------------------------------------
    const int esz = p.out_bf16 ? 2 : 4;
    const rsrc_t rC = make_rsrc((uint8_t *)p.C + (size_t)m0 * p.N * esz, (uint32_t)rows_a * p.N * esz);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = wm * 64 + 16 * i + r16;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int n = n0 + wn * 16 * NT + 16 * j + 4 * g;
            store_c4(rC, (uint32_t)m * p.N + n, n, p.N, acc[i][j], p.out_bf16, p.use_acc, p.c_vec);
        }
    }
}

} // namespace block_large
} // namespace mxg

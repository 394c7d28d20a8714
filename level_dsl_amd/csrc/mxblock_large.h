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
//
// Measured (e4m3, calls behind each other until the clock has settled; traced in
// short runs right after other work they take 7 to 14 % more): native, 8192^3,
// bf16 out 457 us (2.4 PFLOP/s): one FMA per output and stage beside the MFMAs
// (128 against 32 of 16 cycles, per wave), at the clock that this load is held
// to.  Exact, 4096^3, bf16 out 121 us (1.14 PFLOP/s); with a scale per row of B
// and fp32 out 136 us: the widening (128 conversions) and the scales' 64 or 128
// instructions beside 64 MFMAs of 16 cycles.  All three wait for A at every
// stage (main loop).
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

// Workgroup barrier behind this wave's LDS reads and writes, but not its
// direct-to-LDS loads, whose landing it waits for by count.
__device__ __forceinline__ void barrier_lds()
{
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    barrier_nofence();
}

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
    // separate objects: a read of which the compiler knows the object does not
    // wait for loads into another (scale_a's reads lose that record, see the
    // main loop)
    __shared__ __attribute__((aligned(1024))) uint8_t a0[A_BYTES], a1[A_BYTES], b0[B_BYTES], b1[B_BYTES];
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
    const uint32_t offA = (uint32_t)(8 * A_SEGS * wave + (lane >> 3)) * K + chunk;
    const uint32_t offB = (uint32_t)(8 * B_SEGS * wave + (lane >> 3)) * K + chunk;
    // load j of this wave's of stage kt (past K: zeros)
    auto load_a = [&](uint8_t *buf, int kt, int j) MXG_INLINE {
        load16_lds(rA, buf + (A_SEGS * wave + j) * 1024, kt * BK + (int)chunk < K ? offA : kOob,
                   (uint32_t)(8 * j) * K + (uint32_t)kt * BK);
    };
    auto load_b = [&](uint8_t *buf, int kt, int j) MXG_INLINE {
        load16_lds(rB, buf + (B_SEGS * wave + j) * 1024, kt * BK + (int)chunk < K ? offB : kOob,
                   (uint32_t)(8 * j) * K + (uint32_t)kt * BK);
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
    const uint32_t fa_off = (uint32_t)(wm * 64 + r16) * BK, fb_off = (uint32_t)(wn * 16 * NT + r16) * BK;

    const uint32_t sn_off = opaque_v((uint32_t)(wn * 16 * NT + 4 * g) * 4);
    // step: called in each column tile's step for the loads that go there
    auto compute = [&](const uint8_t *la, const uint8_t *lb, int kt, float sb, auto &&step) MXG_INLINE {
        const int w = (kt >> 2) & 1, e4 = kt & 3;
        float s[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) s[i] = scale_a[w][e4][wm * 64 + 16 * i + r16];
        if constexpr (ROWS_B != 1) {
#pragma unroll
            for (int i = 0; i < MT; ++i) s[i] *= sb;
        }
        auto read = [&](const uint8_t *src) MXG_INLINE {
            const v4i lo = *reinterpret_cast<const v4i *>(src + o0);
            const v4i hi = *reinterpret_cast<const v4i *>(src + o1);
            return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        };
        // B's scales of column tile j, read a step before they are used.  The
        // address is the object plus two whole offsets: a longer chain loses
        // the compiler's record of which object is read, and it would wait
        // for the loads into the others.
        v4f sn[2];
        const uint32_t stage_off = opaque_s((uint32_t)(w * 4 + e4) * BN * 4);
        auto read_sn = [&](int j) MXG_INLINE {
            if constexpr (ROWS_B == 1)
                sn[j & 1] = *reinterpret_cast<const v4f *>(reinterpret_cast<const uint8_t *>(scale_b) + stage_off + sn_off +
                                                           j * 64);
        };
        // the two scales first: a block's sum times one of them may leave the fp32
        // range where their product does not
        auto join = [&](int j, const v4f (&t)[MT]) MXG_INLINE {
            if constexpr (ROWS_B == 1) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] += t[i][e] * (s[i] * sn[j & 1][e]);
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
        b[0] = read(lb + fb_off);
        if constexpr (NATIVE) {
            v8i a[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) a[i] = read(la + fa_off + i * 16 * BK);
            static_for<NT>([&](auto J) MXG_INLINE {
                constexpr int j = decltype(J)::value;
                if constexpr (j + 1 < NT) b[(j + 1) & 1] = read(lb + fb_off + (j + 1) * 16 * BK);
                read_sn(j);
                step(J);
#pragma unroll
                for (int i = 0; i < MT; ++i) t[j & 1][i] = mfma_f8_16<FB, FA>(b[j & 1], a[i], zero);
                if constexpr (j > 0) join(j - 1, t[(j - 1) & 1]);
                __builtin_amdgcn_sched_group_barrier(large::SG_DS_RD, ROWS_B == 1 ? 3 : 2, 0);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    if (i == 1) __builtin_amdgcn_sched_group_barrier(large::SG_VMEM_RD, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(large::SG_MFMA, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(large::SG_VALU, ROWS_B == 1 ? 8 : 4, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            });
        } else {
            v8bf fa[MT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const v8i x = read(la + fa_off + i * 16 * BK);
                decode16<FA>(v4i{x[0], x[1], x[2], x[3]}, 1.0f, fa[i][0], fa[i][1]);
                decode16<FA>(v4i{x[4], x[5], x[6], x[7]}, 1.0f, fa[i][2], fa[i][3]);
            }
            __builtin_amdgcn_sched_barrier(0);
            static_for<NT>([&](auto J) MXG_INLINE {
                constexpr int j = decltype(J)::value;
                v8bf fb[4];
                const v8i x = b[j & 1];
                if constexpr (j + 1 < NT) b[(j + 1) & 1] = read(lb + fb_off + (j + 1) * 16 * BK);
                read_sn(j);
                step(J);
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
    // Stage kt's first half loads B of stage kt + 1, a load a step (a burst of
    // them backs up the address path and stalls the waves behind it).  By its
    // middle every wave holds its A rows in registers, so after a barrier
    // there the second half loads A of stage kt + 2 over stage kt's.  The counted
    // wait at a stage's end lets those stay in flight; as compiled, the next
    // stage begins with a wait for all of them all the same, because its reads
    // of scale_a are taken to be of any LDS object, and because at the loop's
    // head the loads of every conditional stage count as in flight.  A thus has
    // half a stage to arrive in, not one and a half.
    auto sb_of = [&](int kt) MXG_INLINE -> float {
        if constexpr (ROWS_B == 1) return 0.0f;
        return scalar_load(bs + min(kt, KB - 1));
    };
#pragma unroll
    for (int j = 0; j < A_SEGS; ++j) load_a(a0, 0, j);
#pragma unroll
    for (int j = 0; j < B_SEGS; ++j) load_b(b0, 0, j);
    v4i win = wload(0);
    wstore(0, win);
#pragma unroll
    for (int j = 0; j < A_SEGS; ++j) load_a(a1, 1, j);
    float sb = sb_of(0);
    wait_vmcnt<A_SEGS>();
    barrier_lds();
    constexpr int HALF = NT / 2;               // steps before the middle
    constexpr int A_STEP = A_SEGS / HALF, B_STEP = B_SEGS / HALF;
    static_assert(A_STEP * HALF == A_SEGS && B_STEP * HALF == B_SEGS, "the loads divide over the steps");
    auto stage = [&](int kt, auto PH) MXG_INLINE {   // PH = kt % 4
        constexpr int ph = decltype(PH)::value;
        uint8_t *const la = ph & 1 ? a1 : a0, *const lb = ph & 1 ? b1 : b0, *const other_b = ph & 1 ? b0 : b1;
        if constexpr (ph == 0) win = wload(kt + 4);
        const float sb1 = sb_of(kt + 1);
        compute(la, lb, kt, sb, [&](auto J) MXG_INLINE {
            constexpr int j = decltype(J)::value;
            if constexpr (j < HALF) {
#pragma unroll
                for (int x = 0; x < B_STEP; ++x) load_b(other_b, kt + 1, j * B_STEP + x);
            } else {
                if constexpr (j == HALF) barrier_nofence();
#pragma unroll
                for (int x = 0; x < A_STEP; ++x) load_a(la, kt + 2, (j - HALF) * A_STEP + x);
            }
        });
        if constexpr (ph == 3) wstore(((kt >> 2) + 1) & 1, win);
        sb = sb1;
        wait_vmcnt<A_SEGS>();                  // all but A of stage kt + 2
        barrier_lds();
    };
    for (int kt = 0; kt < KB; kt += 4) {
        stage(kt, int_c<0>{});
        if (kt + 1 < KB) stage(kt + 1, int_c<1>{});
        if (kt + 2 < KB) stage(kt + 2, int_c<2>{});
        if (kt + 3 < KB) stage(kt + 3, int_c<3>{});
    }

    // ---- epilogue -------------------------------------------------------------
    const int esz = p.out_bf16 ? 2 : 4;
    const rsrc_t rC = make_rsrc((uint8_t *)p.C + (size_t)m0 * p.N * esz, (uint32_t)rows_a * p.N * esz);
    if (p.out_bf16 && p.c_vec == 2) {
        // rows of 8 bf16: column tiles j and j + 1 trade the odd lane groups of
        // one for the even groups of the other, so that a lane holds eight
        // consecutive columns of tile j (g even) or j + 1 (g odd)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int m = wm * 64 + 16 * i + r16;
#pragma unroll
            for (int j = 0; j < NT; j += 2) {
                v4f lo, hi;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = acc[i][j][e], y = acc[i][j + 1][e];
                    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x),
                                                                    __builtin_bit_cast(uint32_t, y), false, false);
                    const uint32_t r0 = r[0], r1 = r[1];
                    lo[e] = __builtin_bit_cast(float, r0);
                    hi[e] = __builtin_bit_cast(float, r1);
                }
                const int n = n0 + wn * 16 * NT + 16 * (j + (g & 1)) + 8 * (g >> 1);
                store_bf16x8(rC, (uint32_t)m * p.N + n, n, p.N, lo, hi, p.use_acc);
            }
        }
        return;
    }
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

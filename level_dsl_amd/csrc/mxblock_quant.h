// mxblock_quant.h -- quantization to codes with one fp32 scale per 128
// elements of a row, or per 128 x 128 block, with the transpose's codes from
// the same read of X.
//
// One workgroup of 256 threads holds a 128 x 128 tile of X in registers as
// fp32: a lane owns CPL consecutive columns (one 16-byte load per row) of RPT
// consecutive rows, so a load instruction of a wave reads whole 128-column
// rows.  The block maxima are integer maxima of magnitude bits (IEEE order,
// and a NaN above everything); rows by shuffles, columns and the whole tile
// through LDS.  The transpose's codes go through LDS so that they too are
// stored as whole 128-byte rows.
//
// Bound by HBM: one read of X, one write of each code.  28672 x 8192 fp32 in 128 x
// 128 blocks with the transpose: 269 us, 5.25 TB/s; 4095 x 8192 bf16 rows and
// columns: 31 us (two sets of codes, a division per row, column and block).
#pragma once

#include "mxblock.h"
#include "mxgemm_common.h"
#include "mxquant.h"

namespace mxg {
namespace block_quant {

constexpr int THREADS = 256;

// a = max(largest magnitude, 2^-100), as bits; scale a / MAX, codes x * (MAX /
// a).  a / MAX as a product with the rounded reciprocal and one correction by
// the exact remainder: correctly rounded like the division (Markstein), in
// three instructions (a NaN or an infinity gives NaN).
template <int FMT>
__device__ __forceinline__ float inverse(uint32_t m, float &scale)
{
    constexpr float MAX = FMT == 0 ? 448.0f : 57344.0f, ONE = 1.0f / MAX;
    const float a = __builtin_bit_cast(float, max(m, (uint32_t)(127 - 100) << 23));
    const float q = a * ONE;
    scale = __builtin_fmaf(__builtin_fmaf(-q, MAX, a), ONE, q);
    return MAX / a;
}

// Maximum over the 16 lanes of a row (row rotations in the ALU, no LDS).
template <int N>
__device__ __forceinline__ uint32_t max_ror(uint32_t x)
{
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + N, 0xf, 0xf, false));
}
__device__ __forceinline__ uint32_t max16(uint32_t x) { return max_ror<1>(max_ror<2>(max_ror<4>(max_ror<8>(x)))); }
// and with the neighbouring 16 lanes
__device__ __forceinline__ uint32_t max32(uint32_t x)
{
    x = max16(x);
    const auto u = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    const uint32_t u0 = u[0], u1 = u[1];
    return max(u0, u1);
}

template <int FMT, bool XBF16, bool TILE>
__global__ __launch_bounds__(THREADS) void kernel(block::QuantArgs p)
{
    constexpr int CPL = XBF16 ? 8 : 4;    // columns per lane
    constexpr int LPR = 128 / CPL;        // lanes per row
    constexpr int RPT = 64 / CPL;         // rows per lane
    constexpr int ESZ = XBF16 ? 2 : 4;
    constexpr int PITCH = 144;            // bytes per transposed row in LDS: 16-byte aligned, lanes spread over banks
    __shared__ uint32_t colmax[128];
    __shared__ uint32_t tilemax[4];
    __shared__ __attribute__((aligned(16))) uint8_t turned[128 * PITCH];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t tr = blockIdx.x / (unsigned)p.KB;
    const int tk = blockIdx.x % (unsigned)p.KB;
    const int64_t r0 = tr * 128;
    const int k0 = tk * 128, K = p.K;
    const int rows = (int)min((int64_t)128, p.R - r0);
    const rsrc_t rX = make_rsrc(p.X + (size_t)r0 * K * ESZ, (uint32_t)rows * K * ESZ);

    const int lc = lane % LPR;                                     // column group
    const int lr = wave * 32 + (lane / LPR) * RPT;                 // first row
    const bool kin = k0 + CPL * lc < K;                            // K % 16 == 0: all columns or none
    uint32_t cm[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) cm[c] = 0;
    uint32_t rm[RPT];
    v4i x[RPT];             // as loaded: bf16 takes half the registers
    auto bits = [&](int j, int c) MXG_INLINE -> uint32_t {
        if constexpr (XBF16) return c & 1 ? (uint32_t)x[j][c / 2] & 0xffff0000u : (uint32_t)x[j][c / 2] << 16;
        else return (uint32_t)x[j][c];
    };
    auto f = [&](int j, int c) MXG_INLINE { return __builtin_bit_cast(float, bits(j, c)); };
#pragma unroll
    for (int j = 0; j < RPT; ++j)
        x[j] = load16_nt(rX, kin ? ((uint32_t)(lr + j) * K + k0 + CPL * lc) * ESZ : kOob);
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
        rm[j] = 0;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            const uint32_t b = bits(j, c) & 0x7fffffffu;
            cm[c] = max(cm[c], b);
            rm[j] = max(rm[j], b);
        }
    }

    float s_tile = 0.0f, i_tile = 0.0f;
    if constexpr (TILE) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < RPT; ++j) m = max(m, rm[j]);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
        if (lane == 0) tilemax[wave] = m;
        __syncthreads();
        m = max(max(tilemax[0], tilemax[1]), max(tilemax[2], tilemax[3]));
        i_tile = inverse<FMT>(m, s_tile);
        if (tid == 0) {
            if (p.codes) p.scales[tr * p.KB + tk] = s_tile;
            if (p.codes_t) p.scales_t[(int64_t)tk * p.RB + tr] = s_tile;
        }
    } else if (p.codes_t) {
        if (tid < 128) colmax[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int c = 0; c < CPL; ++c) atomicMax(&colmax[CPL * lc + c], cm[c]);
        __syncthreads();
        if (tid < 128 && k0 + tid < K) {
            float s;
            inverse<FMT>(colmax[tid], s);
            p.scales_t[(int64_t)(k0 + tid) * p.RB + tr] = s;
        }
    }

    if (p.codes) {
        const rsrc_t rQ = make_rsrc(p.codes + (size_t)r0 * K, (uint32_t)rows * K);
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            float inv = i_tile;
            if constexpr (!TILE) {
                const uint32_t m = LPR == 16 ? max16(rm[j]) : max32(rm[j]);
                float s;
                inv = inverse<FMT>(m, s);
                if (lc == 0 && lr + j < rows) p.scales[(r0 + lr + j) * p.KB + tk] = s;
            }
            uint32_t w[CPL / 4];
#pragma unroll
            for (int q = 0; q < CPL / 4; ++q) {
                w[q] = quant::cvt_pair<FMT>(f(j, 4 * q) * inv, f(j, 4 * q + 1) * inv, 0u, false);
                w[q] = quant::cvt_pair<FMT>(f(j, 4 * q + 2) * inv, f(j, 4 * q + 3) * inv, w[q], true);
            }
            const uint32_t off = kin ? (uint32_t)(lr + j) * K + k0 + CPL * lc : kOob;
            if constexpr (XBF16)
                store8(rQ, off, v2i{(int)w[0], (int)w[1]});
            else
                store4(rQ, off, w[0]);
        }
    }

    if (p.codes_t) {
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            float inv = i_tile;
            if constexpr (!TILE) {
                float s;
                inv = inverse<FMT>(colmax[CPL * lc + c], s);
            }
            uint32_t w[RPT / 4];
#pragma unroll
            for (int q = 0; q < RPT / 4; ++q) {
                w[q] = quant::cvt_pair<FMT>(f(4 * q, c) * inv, f(4 * q + 1, c) * inv, 0u, false);
                w[q] = quant::cvt_pair<FMT>(f(4 * q + 2, c) * inv, f(4 * q + 3, c) * inv, w[q], true);
            }
            uint8_t *dst = turned + (CPL * lc + c) * PITCH + lr;
            if constexpr (XBF16)
                *reinterpret_cast<v2i *>(dst) = v2i{(int)w[0], (int)w[1]};
            else
                *reinterpret_cast<v4i *>(dst) = v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
        }
        __syncthreads();
        // 8 lanes store one transposed row of 128 codes (rows past R up to
        // its multiple of 16 are the zeros that the loads gave)
        const int chunk = tid & 7;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = q * 32 + (tid >> 3);
            const v4i v = *reinterpret_cast<const v4i *>(turned + c * PITCH + 16 * chunk);
            if (k0 + c < K && r0 + 16 * chunk < p.Rp)
                *reinterpret_cast<v4i *>(p.codes_t + (size_t)(k0 + c) * p.Rp + r0 + 16 * chunk) = v;
        }
    }
}

} // namespace block_quant
} // namespace mxg

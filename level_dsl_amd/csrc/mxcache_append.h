// mxcache_append.h -- new keys and values into the pages of the 8-bit cache.
//
// One workgroup of THREADS threads stores what one page and kv head receives of
// keys or of values (blockIdx.y: head, keys / values): 256 for whole pages, or
// one wave where max_q is at most FEW tokens (128 sequences of one token, 8
// heads: 7.0 us, 10.6 us with 256 threads).  The page's new values
// are read once into registers (at most 128 x 128 of them, 64 a thread), their
// magnitudes reduced to one scale byte, and the codes written: keys token by
// token, 8 dims a lane; values with the tokens contiguous, through LDS, where
// a thread leaves four tokens' codes of a dim as one dword and takes up 16 of
// them as one store (byte stores of single codes: 28.6 us for four prompts of
// up to 2048 tokens, 8 heads, dim 128).  Where the page held earlier tokens of
// the sequence and the byte grows, their codes are rounded to the new scale
// first (a multiplication by a power of two, then the hardware's round to
// nearest even).
//
// Bound by latency for one token per sequence, by HBM for prompts (the four of
// above: 12.5 us, a third of it the launch and the first loads).
#pragma once

#include "mxcache.h"
#include "mxgemm_common.h"

namespace mxg {
namespace cache {

constexpr int FEW = 13;  // unaligned, they touch at most 4 groups of 4 slots

// four fp32 -> four e4m3 codes, nearest even (the inputs fit the format)
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d)
{
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// four e4m3 codes times 2^e, rounded to e4m3 again
__device__ __forceinline__ uint32_t rescale4(uint32_t w, int e)
{
    return codes4(__builtin_ldexpf(__builtin_amdgcn_cvt_f32_fp8((int)w, 0), e),
                  __builtin_ldexpf(__builtin_amdgcn_cvt_f32_fp8((int)w, 1), e),
                  __builtin_ldexpf(__builtin_amdgcn_cvt_f32_fp8((int)w, 2), e),
                  __builtin_ldexpf(__builtin_amdgcn_cvt_f32_fp8((int)w, 3), e));
}

template <bool XBF16, int D, int THREADS>
__global__ __launch_bounds__(THREADS) void append_kernel(AppendArgs p)
{
    const Pages &c = p.c;
    const int head = blockIdx.y >> 1, is_v = blockIdx.y & 1;
    const int s = blockIdx.x / (unsigned)p.steps, step = blockIdx.x % (unsigned)p.steps;
    const Seq q = sequence(c, s);
    if (q.n <= 0) return;
    const int P = 1 << c.shift;
    const int last = min(q.ctx, q.first + q.n);        // end of the tokens that are stored
    const int pg = (max(q.first, 0) >> c.shift) + step;
    const int64_t base = (int64_t)pg << c.shift;
    if (base >= last) return;
    const int t0 = (int)max((int64_t)0, q.first - base);          // first new slot
    const int t1 = (int)min((int64_t)P, last - base);             // end of the new slots
    const int id = page_of(c, s, pg);
    if (id < 0) return;

    const int tid = threadIdx.x;
    const size_t at = ((size_t)id * c.kv_heads + head);
    uint8_t *const codes = (is_v ? c.v : c.k) + at * P * D;
    uint8_t *const scale = (is_v ? c.vs : c.ks) + at;
    const uint8_t *const X = is_v ? p.V : p.K;
    const int64_t row0 = q.q0 + (base + t0 - q.first);             // token matrix row of slot t0
    constexpr int ESZ = XBF16 ? 2 : 4;

    // a thread holds 8 consecutive dims of slots 4 u .. 4 u + 3, u = first + tid / (D/8) + i * UNITS
    constexpr int LPT = D / 8, UNITS = THREADS / LPT, ITERS = THREADS == 64 ? 1 : 32 / UNITS;
    static_assert(THREADS == 64 ? 4 * UNITS >= FEW + 3 : ITERS * UNITS == 32, "every new slot has a thread");
    const int dl = tid % LPT, d0 = 8 * dl, u0 = tid / LPT + (THREADS == 64 ? t0 / 4 : 0);
    float f[ITERS][4][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < ITERS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = 4 * (u0 + i * UNITS) + j;
            if (t >= t0 && t < t1) {
                const uint8_t *src = X + ((row0 + (t - t0)) * p.stride + (int64_t)head * D + d0) * ESZ;
                if constexpr (XBF16) {
                    const v4i x = *reinterpret_cast<const v4i *>(src);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        f[i][j][e] = bf16_to_f32(((uint32_t)x[e / 2] >> (16 * (e & 1))) & 0xffffu);
                } else {
                    const v4f x = *reinterpret_cast<const v4f *>(src), y = *reinterpret_cast<const v4f *>(src + 16);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        f[i][j][e] = x[e];
                        f[i][j][4 + e] = y[e];
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) m = max(m, __builtin_bit_cast(uint32_t, f[i][j][e]) & 0x7fffffffu);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[i][j][e] = 0.0f;
            }
        }
    __shared__ uint32_t part[THREADS / 64];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
    if ((tid & 63) == 0) part[tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) m = max(m, part[w]);
    // max|x| = 1.f * 2^(E-127) <= 448 * 2^(b-127) = 1.75 * 2^(b-119): b = E - 8 + (f > 0.75)
    int b = (int)(m >> 23) - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
    b = m >= 0x7f800000u ? 255 : min(max(b, 0), 254);
    const int was = *scale;
    const bool held = t0 > 0;
    if (held) b = max(b, was);
    __syncthreads();                       // every thread has read the byte
    if (tid == 0) *scale = (uint8_t)b;

    // 2^(127 - b); under the byte 255 the codes say nothing and are zero
    const int sh = 127 - b;
    auto code = [&](float x) MXG_INLINE { return b == 255 ? 0.0f : __builtin_ldexpf(x, sh); };
    if (held && b > was && b != 255) {
        const int e = was - b;
        if (is_v) {
            // rows of D tokens-contiguous codes; slots 0 .. t0 - 1 of each
            for (int i = tid; i < D * (P / 4); i += THREADS) {
                const int t = 4 * (i % (P / 4));
                if (t >= t0) continue;
                uint8_t *w = codes + (size_t)(i / (P / 4)) * P + t;
                const uint32_t o = *reinterpret_cast<uint32_t *>(w), r = rescale4(o, e);
                if (t + 4 <= t0) {
                    *reinterpret_cast<uint32_t *>(w) = r;
                } else {
                    for (int j = 0; j < t0 - t; ++j) w[j] = (uint8_t)(r >> (8 * j));
                }
            }
        } else {
            for (int i = tid; i < t0 * (D / 4); i += THREADS) {
                uint32_t *w = reinterpret_cast<uint32_t *>(codes) + i;
                *w = rescale4(*w, e);
            }
        }
    }
    if (!is_v) {
#pragma unroll
        for (int i = 0; i < ITERS; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 4 * (u0 + i * UNITS) + j;
                if (t < t0 || t >= t1) continue;
                const float *x = f[i][j];
                *reinterpret_cast<v2i *>(codes + (size_t)t * D + d0) =
                    v2i{(int)codes4(code(x[0]), code(x[1]), code(x[2]), code(x[3])),
                        (int)codes4(code(x[4]), code(x[5]), code(x[6]), code(x[7]))};
            }
        return;
    }
    // values: dword u (from the thread block's first) of dim d sits at place
    // u ^ (d / 8 % W) of its row of W, the page's dwords or the few there are
    constexpr int FEWW = UNITS;
    __shared__ uint32_t turned[THREADS == 64 ? D * FEWW : D * 32];
    const int W = THREADS == 64 ? FEWW : P / 4, ub = THREADS == 64 ? t0 / 4 : 0;
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
        const int u = u0 + i * UNITS - ub;
        if (u >= W) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            turned[(d0 + e) * W + (u ^ (dl & (W - 1)))] =
                codes4(code(f[i][0][e]), code(f[i][1][e]), code(f[i][2][e]), code(f[i][3][e]));
    }
    __syncthreads();
    const int c0 = t0 / 16, nc = (t1 + 15) / 16 - c0;      // chunks that hold new slots
    for (int i = tid; i < D * nc; i += THREADS) {
        const int d = i / nc, t = 16 * (c0 + i % nc);
        v4i x;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int u = t / 4 + w - ub;      // dwords outside hold no new slot
            x[w] = u >= 0 && u < W ? (int)turned[d * W + (u ^ (d / 8 & (W - 1)))] : 0;
        }
        uint8_t *dst = codes + (size_t)d * P + t;
        if (t >= t0 && t + 16 <= t1) {
            *reinterpret_cast<v4i *>(dst) = x;
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (t + j >= t0 && t + j < t1) dst[j] = (uint8_t)((uint32_t)x[j / 4] >> (8 * (j % 4)));
        }
    }
}

} // namespace cache
} // namespace mxg

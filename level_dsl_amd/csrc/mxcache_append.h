// mxcache_append.h -- new keys and values into the pages of the 8-bit cache.
//
// One workgroup of 256 threads stores what one page and kv head receives of
// keys or of values (blockIdx.y: head, keys / values).  The page's new
// values are read once into registers (at most 128 x 128 of them, 64 a
// thread), their magnitudes reduced to one scale byte, and the codes written:
// keys token by token, values with the tokens contiguous.  Where the page
// held earlier tokens of the sequence and the byte grows, their codes are
// rounded to the new scale first (a multiplication by a power of two, then
// the hardware's round to nearest even).
//
// Bound by latency for one token per sequence, by HBM for prompts.
#pragma once

#include "mxcache.h"
#include "mxgemm_common.h"

namespace mxg {
namespace cache {

constexpr int APPEND_THREADS = 256;

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

template <bool XBF16, int D>
__global__ __launch_bounds__(APPEND_THREADS) void append_kernel(AppendArgs p)
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

    // thread t holds 8 consecutive dims of tokens t / (D/8) + i * (256 / (D/8))
    constexpr int LPT = D / 8, TPI = APPEND_THREADS / LPT, ITERS = 128 / TPI;
    const int d0 = 8 * (tid % LPT), tt = tid / LPT;
    float f[ITERS][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
        const int t = t0 + tt + i * TPI;
        if (t < t1) {
            const uint8_t *src = X + ((row0 + (t - t0)) * p.stride + (int64_t)head * D + d0) * ESZ;
            if constexpr (XBF16) {
                const v4i x = *reinterpret_cast<const v4i *>(src);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[i][e] = bf16_to_f32(((uint32_t)x[e / 2] >> (16 * (e & 1))) & 0xffffu);
            } else {
                const v4f x = *reinterpret_cast<const v4f *>(src), y = *reinterpret_cast<const v4f *>(src + 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[i][e] = x[e];
                    f[i][4 + e] = y[e];
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max(m, __builtin_bit_cast(uint32_t, f[i][e]) & 0x7fffffffu);
        }
    }
    __shared__ uint32_t part[APPEND_THREADS / 64];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
    if ((tid & 63) == 0) part[tid >> 6] = m;
    __syncthreads();
    m = max(max(part[0], part[1]), max(part[2], part[3]));
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
            for (int i = tid; i < D * (P / 4); i += APPEND_THREADS) {
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
            for (int i = tid; i < t0 * (D / 4); i += APPEND_THREADS) {
                uint32_t *w = reinterpret_cast<uint32_t *>(codes) + i;
                *w = rescale4(*w, e);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
        const int t = t0 + tt + i * TPI;
        if (t >= t1) continue;
        const uint32_t lo = codes4(code(f[i][0]), code(f[i][1]), code(f[i][2]), code(f[i][3]));
        const uint32_t hi = codes4(code(f[i][4]), code(f[i][5]), code(f[i][6]), code(f[i][7]));
        if (is_v) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                codes[(size_t)(d0 + e) * P + t] = (uint8_t)(lo >> (8 * e));
                codes[(size_t)(d0 + 4 + e) * P + t] = (uint8_t)(hi >> (8 * e));
            }
        } else {
            *reinterpret_cast<v2i *>(codes + (size_t)t * D + d0) = v2i{(int)lo, (int)hi};
        }
    }
}

} // namespace cache
} // namespace mxg

// mxblock.hip -- host side of the operators whose codes carry one fp32 scale
// per 128 elements: argument checks, the choice of kernel and the launch.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "mxblock.h"
#include "mxgemm.h"
#include "mxgemm_ctx.h"

using mxg::overlaps;

namespace {

// The large tiles, or the small ones.  Large tiles take as long for a partly
// filled round of the 256 CUs as for a whole one, so they run at the share of
// their full rate that the outputs are of the tiles of all rounds; the small
// ones need no such care.  Measured (us, small / large exact / large native;
// N = 4096 and K = 4096 unless given, the share in brackets):
//   M = 1024  41 / 58 (50%) / 47 (25%)     M = 1280  52 / 57 (62%) / 48 (31%)
//   M = 1536  59 / 58 (75%) / 48 (37%)     M = 2304  87 / 113 (56%) / 49 (56%)
//   M = 2816  108 / 114 (69%) / 52 (69%)   M = 4352  162 / 171 (71%) / 103 (53%)
//   N = 28672, K = 8192: M = 128  94 / 121 (44%) / 103 (22%)
//                        M = 256  149 / 131 (87%) / 114 (44%)
// From 2^20 tiles of 64 x 64 on, the small ones' grid could pass 2^32 threads.
bool use_large(int variant, int64_t M, int64_t N)
{
    if (M <= 64) return false;
    if (variant == MXGEMM_VARIANT_LARGE || (M + 63) / 64 * ((N + 63) / 64) >= (int64_t)1 << 20) return true;
    if (variant == MXGEMM_VARIANT_SKINNY) return false;
    const bool native = variant == MXGEMM_VARIANT_LARGE_NATIVE;
    const int64_t bn = native ? 256 : 128;
    const int64_t rounds = ((M + 255) / 256 * ((N + bn - 1) / bn) + 255) / 256;
    return M * N >= (native ? 28 : 73) * (256 * bn * 256 / 100) * rounds;
}

} // namespace

extern "C" {

int mxgemm_validate_block128(const void *A, const float *A_scale, int fmtA, const void *B,
                             const float *B_scale, int fmtB, int b_rows, const void *C, int64_t M,
                             int64_t N, int64_t K, int use_acc, int out_dtype)
{
    if (!A || !A_scale || !B || !B_scale || !C) return MXGEMM_ERR_NULL;
    if ((fmtA != MXGEMM_FMT_E4M3 && fmtA != MXGEMM_FMT_E5M2) ||
        (fmtB != MXGEMM_FMT_E4M3 && fmtB != MXGEMM_FMT_E5M2))
        return MXGEMM_ERR_FMT;
    if ((out_dtype != MXGEMM_OUT_F32 && out_dtype != MXGEMM_OUT_BF16) || (use_acc != 0 && use_acc != 1))
        return MXGEMM_ERR_DTYPE;
    if (b_rows != 1 && b_rows != 128) return MXGEMM_ERR_SHAPE;
    if (M < 1 || N < 1 || K < 16 || M > MXGEMM_MAX_M || N > MXGEMM_MAX_N || K > MXGEMM_MAX_K ||
        K % 16 != 0 || M * N > MXGEMM_MAX_MN)
        return MXGEMM_ERR_SHAPE;
    if (((uintptr_t)A | (uintptr_t)B | (uintptr_t)C) & 15u) return MXGEMM_ERR_ALIGN;
    if (((uintptr_t)A_scale | (uintptr_t)B_scale) & 3u) return MXGEMM_ERR_ALIGN;
    const uint64_t KB = (uint64_t)(K + 127) / 128, nb = (uint64_t)(N + b_rows - 1) / b_rows;
    const uint64_t csize = (uint64_t)M * (uint64_t)N * (out_dtype == MXGEMM_OUT_F32 ? 4u : 2u);
    if (overlaps(C, csize, A, (uint64_t)(M * K)) || overlaps(C, csize, B, (uint64_t)(N * K)) ||
        overlaps(C, csize, A_scale, (uint64_t)M * KB * 4) || overlaps(C, csize, B_scale, nb * KB * 4))
        return MXGEMM_ERR_ALIAS;
    return MXGEMM_OK;
}

int mxgemm_run_block128(mxgemm_t h, const void *A, const float *A_scale, int fmtA, const void *B,
                        const float *B_scale, int fmtB, int b_rows, void *C, int64_t M, int64_t N,
                        int64_t K, int use_acc, int out_dtype, hipStream_t stream)
{
    if (!h || h->magic != mxg::kMagic) return MXGEMM_ERR_HANDLE;
    int rc = mxgemm_validate_block128(A, A_scale, fmtA, B, B_scale, fmtB, b_rows, C, M, N, K, use_acc,
                                      out_dtype);
    if (rc != MXGEMM_OK) return rc;
    if (h->variant == MXGEMM_VARIANT_SKINNY_NATIVE) return MXGEMM_ERR_VARIANT;
    rc = mxg::check_device(h);
    if (rc != MXGEMM_OK) return rc;

    mxg::block::Args a;
    a.A = (const uint8_t *)A;
    a.As = A_scale;
    a.B = (const uint8_t *)B;
    a.Bs = B_scale;
    a.C = C;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.KB = (int)((K + 127) / 128);
    a.tiles_m = a.tiles_n = 0;
    a.use_acc = use_acc;
    a.out_bf16 = out_dtype == MXGEMM_OUT_BF16;
    a.c_vec = N % 8 == 0 ? 2 : (N % 4 == 0 ? 1 : 0);
    const int f = 2 * fmtA + fmtB;
    const bool native = h->variant == MXGEMM_VARIANT_LARGE_NATIVE;
    hipError_t e;
    if (!use_large(h->variant, M, N))
        e = mxg::launch_block_small(f, b_rows, a, stream);
    else
        e = native ? mxg::launch_block_native(f, b_rows, a, stream) : mxg::launch_block_exact(f, b_rows, a, stream);
    return e == hipSuccess ? MXGEMM_OK : MXGEMM_ERR_HIP;
}

int mxgemm_validate_quantize_block128(const void *X, int x_dtype, int64_t R, int64_t K, int rows, int fmt,
                                      const uint8_t *codes, const float *scales, const uint8_t *codes_t,
                                      const float *scales_t)
{
    if (!X || (!codes != !scales) || (!codes_t != !scales_t) || (!codes && !codes_t)) return MXGEMM_ERR_NULL;
    if (fmt != MXGEMM_FMT_E4M3 && fmt != MXGEMM_FMT_E5M2) return MXGEMM_ERR_FMT;
    if (x_dtype != MXGEMM_X_F32 && x_dtype != MXGEMM_X_BF16) return MXGEMM_ERR_DTYPE;
    if (rows != 1 && rows != 128) return MXGEMM_ERR_SHAPE;
    if (R < 1 || K < 16 || R > MXGEMM_MAX_M || K > MXGEMM_MAX_K || K % 16 != 0 || R * K > MXGEMM_MAX_QELEMS ||
        (codes_t && R > MXGEMM_MAX_K) || (R + 127) / 128 * ((K + 127) / 128) >= (int64_t)1 << 24)
        return MXGEMM_ERR_SHAPE;
    if (((uintptr_t)X | (uintptr_t)codes | (uintptr_t)codes_t) & 15u) return MXGEMM_ERR_ALIGN;
    if (((uintptr_t)scales | (uintptr_t)scales_t) & 3u) return MXGEMM_ERR_ALIGN;
    const uint64_t kb = (uint64_t)(K + 127) / 128, rb = (uint64_t)(R + 127) / 128, r = (uint64_t)R, k = (uint64_t)K;
    const void *ptr[5] = {X, codes, scales, codes_t, scales_t};
    const uint64_t bytes[5] = {r * k * (x_dtype == MXGEMM_X_F32 ? 4u : 2u), r * k, (rows == 1 ? r : rb) * kb * 4,
                               k * ((r + 15) / 16 * 16), (rows == 1 ? k : kb) * rb * 4};
    for (int i = 0; i < 5; ++i)
        for (int j = 0; j < i; ++j)
            if (ptr[i] && ptr[j] && overlaps(ptr[i], bytes[i], ptr[j], bytes[j])) return MXGEMM_ERR_ALIAS;
    return MXGEMM_OK;
}

int mxgemm_quantize_block128(mxgemm_t h, const void *X, int x_dtype, int64_t R, int64_t K, int rows, int fmt,
                             uint8_t *codes, float *scales, uint8_t *codes_t, float *scales_t,
                             hipStream_t stream)
{
    if (!h || h->magic != mxg::kMagic) return MXGEMM_ERR_HANDLE;
    int rc = mxgemm_validate_quantize_block128(X, x_dtype, R, K, rows, fmt, codes, scales, codes_t, scales_t);
    if (rc != MXGEMM_OK) return rc;
    rc = mxg::check_device(h);
    if (rc != MXGEMM_OK) return rc;
    mxg::block::QuantArgs a;
    a.X = (const uint8_t *)X;
    a.codes = codes;
    a.scales = scales;
    a.codes_t = codes_t;
    a.scales_t = scales_t;
    a.R = R;
    a.Rp = (R + 15) / 16 * 16;
    a.K = (int)K;
    a.KB = (int)((K + 127) / 128);
    a.RB = (R + 127) / 128;
    const int sel = 4 * fmt + (x_dtype == MXGEMM_X_BF16 ? 2 : 0) + (rows == 128 ? 1 : 0);
    return mxg::launch_block_quant(sel, a, stream) == hipSuccess ? MXGEMM_OK : MXGEMM_ERR_HIP;
}

} // extern "C"

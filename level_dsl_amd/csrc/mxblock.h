// mxblock.h -- arguments and launchers of the operators whose codes carry one
// fp32 scale per 128 elements: the product (mxgemm_run_block128) and the
// quantization that makes its operands (mxgemm_quantize_block128).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxg {
namespace block {

struct Args {
    const uint8_t *A;
    const float *As;       // M x KB
    const uint8_t *B;
    const float *Bs;       // N x KB (rows_b == 1) or ceil(N / 128) x KB
    void *C;
    int M, N, K, KB;       // KB = ceil(K / 128)
    int tiles_m, tiles_n;
    int use_acc, out_bf16;
    int c_vec;             // 1: N % 4 == 0; 2: N % 8 == 0
};

struct QuantArgs {
    const uint8_t *X;
    uint8_t *codes;        // or NULL
    float *scales;
    uint8_t *codes_t;      // or NULL
    float *scales_t;
    int64_t R, Rp;         // rows, and rows rounded up to 16
    int K, KB;             // columns, ceil(K / 128)
    int64_t RB;            // ceil(R / 128)
};

} // namespace block

// f = 2 fmtA + fmtB
hipError_t launch_block_small(int f, int rows_b, const block::Args &a, hipStream_t s);  // k_block_small.hip
hipError_t launch_block_native(int f, int rows_b, const block::Args &a, hipStream_t s); // k_block_native.hip
hipError_t launch_block_exact(int f, int rows_b, const block::Args &a, hipStream_t s);  // k_block_exact.hip
// sel = 4 fmt + 2 (bf16 input) + (rows == 128)
hipError_t launch_block_quant(int sel, const block::QuantArgs &a, hipStream_t s);       // k_block_quant.hip

} // namespace mxg

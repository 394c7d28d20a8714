// k_block_native.hip -- large-tile product of codes with one fp32 scale per 128
// K, summed inside a block on the fp8 MFMA.
#include "mxblock_large.h"

namespace mxg {
namespace {

template <int FA, int FB>
hipError_t go(int rows_b, block::Args a, hipStream_t s)
{
    constexpr int BN = block_large::columns<true>();
    a.tiles_m = (a.M + block_large::BM - 1) / block_large::BM;
    a.tiles_n = (a.N + BN - 1) / BN;
    const dim3 grid((unsigned)((int64_t)a.tiles_m * a.tiles_n)), threads(block_large::THREADS);
    if (rows_b == 1)
        hipLaunchKernelGGL((block_large::kernel<FA, FB, 1, true>), grid, threads, 0, s, a);
    else
        hipLaunchKernelGGL((block_large::kernel<FA, FB, 128, true>), grid, threads, 0, s, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_block_native(int f, int rows_b, const block::Args &a, hipStream_t s)
{
    switch (f) {
    case 0: return go<0, 0>(rows_b, a, s);
    case 1: return go<0, 1>(rows_b, a, s);
    case 2: return go<1, 0>(rows_b, a, s);
    case 3: return go<1, 1>(rows_b, a, s);
    default: return hipErrorInvalidValue;
    }
}

} // namespace mxg

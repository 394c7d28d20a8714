// k_block_small.hip -- small-tile product of codes with one fp32 scale per
// 128 K.
#include "mxblock_small.h"

namespace mxg {
namespace {

template <int FA, int FB, int ROWS_B, int MT, int CT, int W, int R>
hipError_t go(block::Args a, hipStream_t s)
{
    a.tiles_m = (a.M + 16 * MT - 1) / (16 * MT);
    a.tiles_n = (a.N + 16 * CT - 1) / (16 * CT);
    hipLaunchKernelGGL((block_small::kernel<FA, FB, ROWS_B, MT, CT, W, R>),
                       dim3((unsigned)((int64_t)a.tiles_m * a.tiles_n)), dim3(64 * W), 0, s, a);
    return hipGetLastError();
}

template <int FA, int FB>
hipError_t pick(int rows_b, const block::Args &a, hipStream_t s)
{
    if (rows_b == 1) return a.M <= 16 ? go<FA, FB, 1, 1, 1, 8, 4>(a, s) : go<FA, FB, 1, 4, 2, 4, 3>(a, s);
    return a.M <= 16 ? go<FA, FB, 128, 1, 1, 8, 4>(a, s) : go<FA, FB, 128, 4, 2, 4, 3>(a, s);
}

} // namespace

hipError_t launch_block_small(int f, int rows_b, const block::Args &a, hipStream_t s)
{
    switch (f) {
    case 0: return pick<0, 0>(rows_b, a, s);
    case 1: return pick<0, 1>(rows_b, a, s);
    case 2: return pick<1, 0>(rows_b, a, s);
    case 3: return pick<1, 1>(rows_b, a, s);
    default: return hipErrorInvalidValue;
    }
}

} // namespace mxg

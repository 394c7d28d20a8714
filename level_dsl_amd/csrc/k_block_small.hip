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

// Rows of a tile by M; columns the widest (the fewest reads of A) that still
// give a workgroup to each of the 256 CUs.  Measured (e4m3, us; K = 8192 for
// N = 28672 and 8192, else 4096):
//   M = 64   N = 28672: 64 columns 63, 32: 85, 16: 106; N = 8192: 36, 19, 23;
//            N = 4096: 20, 10.6, 8.9
//   M = 32   N = 28672: 54, 59, 74; N = 8192: 24, 17, 16; N = 4096: 14, 7.4, 6.3
//   M = 16   N = 28672: 16 columns 50, 32: 53, 64: 52; M = 1: 39, 54, 49
// Waves and ring slots are the best of those tried for each tile (two
// workgroups on a CU beat one with a deeper ring).
template <int FA, int FB, int ROWS_B>
hipError_t pick(const block::Args &a, hipStream_t s)
{
    const int64_t mt = a.M <= 32 ? 1 : (a.M + 63) / 64;
    const bool wide = mt * ((a.N + 63) / 64) >= 256, mid = mt * ((a.N + 31) / 32) >= 256;
    if (a.M <= 16) return go<FA, FB, ROWS_B, 1, 1, 8, 2>(a, s);
    if (a.M <= 32)
        return wide ? go<FA, FB, ROWS_B, 2, 4, 2, 3>(a, s)
               : mid ? go<FA, FB, ROWS_B, 2, 2, 4, 2>(a, s)
                     : go<FA, FB, ROWS_B, 2, 1, 8, 2>(a, s);
    return wide ? go<FA, FB, ROWS_B, 4, 4, 2, 2>(a, s)
           : mid ? go<FA, FB, ROWS_B, 4, 2, 4, 2>(a, s)
                 : go<FA, FB, ROWS_B, 4, 1, 4, 2>(a, s);
}

template <int FA, int FB>
hipError_t pick_b(int rows_b, const block::Args &a, hipStream_t s)
{
    return rows_b == 1 ? pick<FA, FB, 1>(a, s) : pick<FA, FB, 128>(a, s);
}

} // namespace

hipError_t launch_block_small(int f, int rows_b, const block::Args &a, hipStream_t s)
{
    switch (f) {
    case 0: return pick_b<0, 0>(rows_b, a, s);
    case 1: return pick_b<0, 1>(rows_b, a, s);
    case 2: return pick_b<1, 0>(rows_b, a, s);
    case 3: return pick_b<1, 1>(rows_b, a, s);
    default: return hipErrorInvalidValue;
    }
}

} // namespace mxg

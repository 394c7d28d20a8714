// k_block_small.hip -- small-tile product of codes with one fp32 scale per
// 128 K.
#include <cstdint>

#include "mxblock_small.h"

namespace mxg {
namespace {

template <int FA, int FB, int ROWS_B, int MT, int CT, int W>
hipError_t go(block::Args a, hipStream_t s)
{
    a.tiles_m = (a.M + 16 * MT - 1) / (16 * MT);
    a.tiles_n = (a.N + 16 * CT - 1) / (16 * CT);
    hipLaunchKernelGGL((block_small::kernel<FA, FB, ROWS_B, MT, CT, W>),
                       dim3((unsigned)((int64_t)a.tiles_m * a.tiles_n)), dim3(64 * W), 0, s, a);
    return hipGetLastError();
}

// The tile whose rounds of the 256 CUs cost least, with a tile's cost the time
// that a CU takes for one of many (tenths of a microsecond, K = 4096).  Measured
// (e4m3, us: 64 x 64, 48 x 64, 32 x 64, 32 x 32, 32 x 16; the one taken in
// brackets):
//   333 x 3584 x 4112  24.7 [21.4] 23.9 24.7 33.5   96 x 8192 x 8192  23.2 [20.8] 24.1 24.8 32.6
//   200 x 2048 x 8192  22.8 19.9 [16.2] 15.6 21.6   64 x 4096 x 4096  13.0 11.9 9.8 [7.4] 8.1
//   32 x 4096 x 4096   13.5 12.1 9.5 7.3 [5.7]      32 x 28672 x 8192 53.7 52.2 [51.5] 58.2 68.7
//   1024 x 4096 x 4096 [40.4] 45.0 46.9 53.0        64 x 28672 x 8192 [63.1] 70.6 69.7 78.7
// M <= 16, 16 columns / 32 columns (fewer reads of A):
//   N = 28672, K = 8192: M = 1  40 / 43, M = 8  42 / 44, M = 16  51 / 46
//   M = 16: 8192 x 8192  12.2 / 11.9, 4096 x 4096  5.1 / 5.4
template <int FA, int FB, int ROWS_B>
hipError_t pick(const block::Args &a, hipStream_t s)
{
    if (a.M <= 16)
        return a.M > 8 && a.N >= 8192 ? go<FA, FB, ROWS_B, 1, 2, 8>(a, s) : go<FA, FB, ROWS_B, 1, 1, 8>(a, s);
    static constexpr struct {
        int rows, columns, cost;
    } tile[] = {{64, 64, 93}, {48, 64, 76}, {32, 64, 55}, {32, 32, 31}, {32, 16, 20}};
    int best = 0;
    int64_t least = INT64_MAX;
    for (int i = 0; i < 5; ++i) {
        const int64_t tiles = (int64_t)((a.M + tile[i].rows - 1) / tile[i].rows) *
                              ((a.N + tile[i].columns - 1) / tile[i].columns);
        const int64_t cost = (tiles + 255) / 256 * tile[i].cost;
        if (cost < least) {
            least = cost;
            best = i;
        }
    }
    switch (best) {
    case 0: return go<FA, FB, ROWS_B, 4, 4, 4>(a, s);
    case 1: return go<FA, FB, ROWS_B, 3, 4, 4>(a, s);
    case 2: return go<FA, FB, ROWS_B, 2, 4, 4>(a, s);
    case 3: return go<FA, FB, ROWS_B, 2, 2, 4>(a, s);
    default: return go<FA, FB, ROWS_B, 2, 1, 8>(a, s);
    }
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

// k_block_quant.hip -- quantization to codes with one fp32 scale per 128
// elements.
#include "mxblock_quant.h"

namespace mxg {
namespace {

template <int FMT, bool XBF16, bool TILE>
hipError_t go(const block::QuantArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL((block_quant::kernel<FMT, XBF16, TILE>), dim3((unsigned)(a.RB * a.KB)),
                       dim3(block_quant::THREADS), 0, s, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_block_quant(int sel, const block::QuantArgs &a, hipStream_t s)
{
    switch (sel) {
    case 0: return go<0, false, false>(a, s);
    case 1: return go<0, false, true>(a, s);
    case 2: return go<0, true, false>(a, s);
    case 3: return go<0, true, true>(a, s);
    case 4: return go<1, false, false>(a, s);
    case 5: return go<1, false, true>(a, s);
    case 6: return go<1, true, false>(a, s);
    case 7: return go<1, true, true>(a, s);
    default: return hipErrorInvalidValue;
    }
}

} // namespace mxg

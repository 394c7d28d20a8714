// k_attn_prompt.hip -- attention over the 8-bit cache for many query rows.
#include "mxattn_prompt.h"

namespace mxg {
namespace {

template <int D>
hipError_t go(cache::AttnArgs a, hipStream_t s)
{
    static_assert(attn_prompt::ROWS == kPromptRows, "host and kernel agree on a row tile");
    const int64_t rows = (int64_t)a.c.max_q * a.group;
    a.row_tiles = (int)((rows + attn_prompt::ROWS - 1) / attn_prompt::ROWS);
    const dim3 grid((unsigned)((int64_t)a.c.seqs * a.c.kv_heads * a.row_tiles)), block(attn_prompt::THREADS);
    if (a.c.shift < 6)
        hipLaunchKernelGGL((attn_prompt::kernel<D, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((attn_prompt::kernel<D, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_attn_prompt(int head_dim, const cache::AttnArgs &a, hipStream_t s)
{
    return head_dim == 128 ? go<128>(a, s) : go<64>(a, s);
}

} // namespace mxg

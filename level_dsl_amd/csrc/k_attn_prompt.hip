// k_attn_prompt.hip -- attention over the 8-bit cache for many query rows.
#include "mxattn_join.h"
#include "mxattn_prompt.h"

namespace mxg {
namespace {

template <int D>
hipError_t go(const cache::AttnArgs &a, hipStream_t s)
{
    static_assert(attn_prompt::ROWS == kPromptRows, "host and kernel agree on a row tile");
    const int64_t tiles = (int64_t)a.c.seqs * a.c.kv_heads * a.row_tiles;
    const dim3 grid((unsigned)(tiles * a.splits)), block(attn_prompt::THREADS);
    const bool small = a.c.shift < 6;
    if (a.splits > 1) {
        if (small) hipLaunchKernelGGL((attn_prompt::kernel<D, true, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((attn_prompt::kernel<D, false, true>), grid, block, 0, s, a);
    } else {
        if (small) hipLaunchKernelGGL((attn_prompt::kernel<D, true, false>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((attn_prompt::kernel<D, false, false>), grid, block, 0, s, a);
    }
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || a.splits == 1 ? e : attn::launch_join<D, attn_prompt::ROWS>(a, tiles, s);
}

} // namespace

hipError_t launch_attn_prompt(int head_dim, const cache::AttnArgs &a, hipStream_t s)
{
    return head_dim == 128 ? go<128>(a, s) : go<64>(a, s);
}

} // namespace mxg

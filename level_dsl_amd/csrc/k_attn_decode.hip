// k_attn_decode.hip -- attention over the 8-bit cache for few query rows.
#include "mxattn_decode.h"
#include "mxattn_join.h"

namespace mxg {
namespace {

template <int D>
hipError_t go(const cache::AttnArgs &a, hipStream_t s)
{
    static_assert(attn::ROWS == kDecodeRows, "host and kernel agree");
    const int64_t tiles = (int64_t)a.c.seqs * a.c.kv_heads * a.row_tiles;
    const dim3 grid((unsigned)(tiles * a.splits)), block(attn::THREADS);
    if (a.c.shift < 6)
        hipLaunchKernelGGL((attn::decode_kernel<D, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((attn::decode_kernel<D, false>), grid, block, 0, s, a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || a.splits == 1 ? e : attn::launch_join<D, attn::ROWS>(a, tiles, s);
}

} // namespace

hipError_t launch_attn_decode(int head_dim, const cache::AttnArgs &a, hipStream_t s)
{
    return head_dim == 128 ? go<128>(a, s) : go<64>(a, s);
}

} // namespace mxg

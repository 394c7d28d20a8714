// k_cache.hip -- storing new tokens in the 8-bit key / value cache.
#include "mxcache_append.h"

namespace mxg {

namespace {

template <bool XBF16, int D>
hipError_t go(const cache::AppendArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)((int64_t)a.c.seqs * a.steps), (unsigned)(2 * a.c.kv_heads));
    if (a.c.max_q <= cache::FEW)
        hipLaunchKernelGGL((cache::append_kernel<XBF16, D, 64>), grid, dim3(64), 0, s, a);
    else
        hipLaunchKernelGGL((cache::append_kernel<XBF16, D, 256>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_cache_append(int x_bf16, int head_dim, const cache::AppendArgs &a, hipStream_t s)
{
    if (head_dim == 128) return x_bf16 ? go<true, 128>(a, s) : go<false, 128>(a, s);
    return x_bf16 ? go<true, 64>(a, s) : go<false, 64>(a, s);
}

} // namespace mxg

// k_cache.hip -- storing new tokens in the 8-bit key / value cache.
#include "mxcache_append.h"

namespace mxg {

hipError_t launch_cache_append(int x_bf16, int head_dim, const cache::AppendArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)((int64_t)a.c.seqs * a.steps), (unsigned)(2 * a.c.kv_heads));
    const dim3 block(cache::APPEND_THREADS);
    if (head_dim == 128) {
        if (x_bf16) hipLaunchKernelGGL((cache::append_kernel<true, 128>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((cache::append_kernel<false, 128>), grid, block, 0, s, a);
    } else {
        if (x_bf16) hipLaunchKernelGGL((cache::append_kernel<true, 64>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((cache::append_kernel<false, 64>), grid, block, 0, s, a);
    }
    return hipGetLastError();
}

} // namespace mxg

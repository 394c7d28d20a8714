// mxgemm_ctx.h -- the handle behind mxgemm_t and the small host-side checks
// that every entry point shares.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "mxgemm.h"

struct mxgemm_ctx {
    uint32_t magic;
    int device;
    int variant;
    int splits;      // 0 automatic, 1 never, S >= 2 forced
    uint8_t *ws;     // caller's split-K workspace, or NULL
    size_t ws_bytes;
    int scale_layout;  // MXGEMM_SCALES_*
    uint8_t *opbuf;    // caller's buffer for widened operands, or NULL
    size_t opbuf_bytes;
};

namespace mxg {

constexpr uint32_t kMagic = 0x4d584732u;  // "MXG2"
constexpr uint32_t kDead = 0xdeadbeefu;

inline bool overlaps(const void *a, uint64_t na, const void *b, uint64_t nb)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

// MXGEMM_OK if the handle is live and its device is the current one.
inline int check_device(mxgemm_t h)
{
    if (!h || h->magic != kMagic) return MXGEMM_ERR_HANDLE;
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return MXGEMM_ERR_HIP;
    return dev == h->device ? MXGEMM_OK : MXGEMM_ERR_DEVICE;
}

} // namespace mxg

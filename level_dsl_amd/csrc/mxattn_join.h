// mxattn_join.h -- what the splits of a row tile leave in the workspace, and the
// kernel that joins them.
//
// A split's part: ROWS x D unscaled outputs, then the ROWS running maxima
// (log2), then the ROWS sums, fp32.  Rows past the sequence's are neither
// written nor joined.
#pragma once

#include "mxattn.h"

#include <algorithm>

namespace mxg {
namespace attn {

// The splits' partial sums of one row of a tile of ROWS, joined in a fixed order: lane group q
// of 256 / (D / 4) adds splits q, q + groups, ..., then the groups are added in
// turn.  The weights 2^(m_k - m) of all splits are computed once, by one wave.
constexpr int JOIN_THREADS = 256, MAX_SPLITS = 64;
template <int D, int ROWS>
__global__ __launch_bounds__(JOIN_THREADS) void join_kernel(AttnArgs p, uint32_t used)
{
    constexpr int LANES = D / 4, GROUPS = JOIN_THREADS / LANES;
    constexpr int64_t PITCH = ROWS * (D + 2);
    const Pages &c = p.c;
    const int r = (int)(blockIdx.x % used);
    uint32_t bid = blockIdx.x / used;
    const int64_t tile = bid;
    const int rt = (int)(bid % (uint32_t)p.row_tiles);
    bid /= (uint32_t)p.row_tiles;
    const int head = (int)(bid % (uint32_t)c.kv_heads), s = (int)(bid / (uint32_t)c.kv_heads);
    const Seq q = cache::sequence(c, s);
    const uint32_t G = p.group, row = (uint32_t)rt * ROWS + r;
    if (row >= (uint32_t)q.n * G) return;
    const float *const part = p.ws + tile * p.splits * PITCH;

    __shared__ float weight[MAX_SPLITS], total[2];
    __shared__ v4f sums[GROUPS][LANES];
    const int tid = threadIdx.x;
    if (tid < 64) {
        float m = kNone, l = 0.0f;
        if (tid < p.splits) {
            m = part[tid * PITCH + ROWS * D + r];
            l = part[tid * PITCH + ROWS * D + ROWS + r];
        }
        float mt = m;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) mt = fmaxf(mt, __shfl_xor(mt, d, 64));
        const float mu = mt == kNone ? 0.0f : mt;
        const float w = __builtin_amdgcn_exp2f(m - mu);
        l *= w;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d, 64);
        weight[tid] = w;
        if (tid == 0) {
            total[0] = mu;
            total[1] = l;
        }
    }
    __syncthreads();
    const int d4 = tid % LANES, g = tid / LANES;
    v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = g; k < p.splits; k += GROUPS)
        v += *reinterpret_cast<const v4f *>(part + k * PITCH + r * D + 4 * d4) * weight[k];
    sums[g][d4] = v;
    __syncthreads();
    if (g) return;
#pragma unroll
    for (int k = 1; k < GROUPS; ++k) v += sums[k][d4];
    const float l = total[1];
    v *= l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t token = q.q0 + row / G;
    const int h = head * G + (int)(row % G);
    *reinterpret_cast<v2i *>(p.O + token * p.o_stride + (int64_t)h * D + 4 * d4) =
        v2i{(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3])};
    if (tid == 0 && p.lse) p.lse[token * p.q_heads + h] = (total[0] + __builtin_log2f(l)) * kLn2;
}

// The same for few splits: a lane group of D / 4 takes a row of its own and adds
// its splits in turn, 256 / (D / 4) rows a workgroup.
template <int D, int ROWS>
__global__ __launch_bounds__(JOIN_THREADS) void join_rows_kernel(AttnArgs p, uint32_t used)
{
    constexpr int LANES = D / 4, GROUPS = JOIN_THREADS / LANES;
    constexpr int64_t PITCH = ROWS * (D + 2);
    const Pages &c = p.c;
    const uint32_t per = (used + GROUPS - 1) / GROUPS;
    const int r = (int)(blockIdx.x % per) * GROUPS + (int)(threadIdx.x / LANES);
    uint32_t bid = blockIdx.x / per;
    const int64_t tile = bid;
    const int rt = (int)(bid % (uint32_t)p.row_tiles);
    bid /= (uint32_t)p.row_tiles;
    const int head = (int)(bid % (uint32_t)c.kv_heads), s = (int)(bid / (uint32_t)c.kv_heads);
    const Seq q = cache::sequence(c, s);
    const uint32_t G = p.group, row = (uint32_t)rt * ROWS + r;
    if (r >= ROWS || row >= (uint32_t)q.n * G) return;
    const float *const part = p.ws + tile * p.splits * PITCH;
    const int d4 = threadIdx.x % LANES;
    float mt = kNone;
    for (int k = 0; k < p.splits; ++k) mt = fmaxf(mt, part[k * PITCH + ROWS * D + r]);
    const float mu = mt == kNone ? 0.0f : mt;
    float l = 0.0f;
    v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < p.splits; ++k) {
        const float *const x = part + k * PITCH;
        const float w = __builtin_amdgcn_exp2f(x[ROWS * D + r] - mu);
        l += x[ROWS * D + ROWS + r] * w;
        v += *reinterpret_cast<const v4f *>(x + r * D + 4 * d4) * w;
    }
    v *= l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t token = q.q0 + row / G;
    const int h = head * G + (int)(row % G);
    *reinterpret_cast<v2i *>(p.O + token * p.o_stride + (int64_t)h * D + 4 * d4) =
        v2i{(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3])};
    if (d4 == 0 && p.lse) p.lse[token * p.q_heads + h] = (mu + __builtin_log2f(l)) * kLn2;
}

// Joins tiles * a.splits parts of row tiles of ROWS.
template <int D, int ROWS>
inline hipError_t launch_join(const AttnArgs &a, int64_t tiles, hipStream_t s)
{
    static_assert(MAX_SPLITS == kMaxSplits, "host and kernel agree");
    constexpr int GROUPS = JOIN_THREADS / (D / 4);
    // rows of a tile that can exist
    const int64_t used = std::min((int64_t)ROWS, (int64_t)a.c.max_q * a.group);
    if (a.splits <= GROUPS)
        hipLaunchKernelGGL((join_rows_kernel<D, ROWS>), dim3((unsigned)(tiles * ((used + GROUPS - 1) / GROUPS))),
                           dim3(JOIN_THREADS), 0, s, a, (uint32_t)used);
    else
        hipLaunchKernelGGL((join_kernel<D, ROWS>), dim3((unsigned)(tiles * used)), dim3(JOIN_THREADS), 0, s, a,
                           (uint32_t)used);
    return hipGetLastError();
}

} // namespace attn
} // namespace mxg

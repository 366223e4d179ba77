// Score modifications of the scored attention calls, and the key ranges they and
// the shared-prefix decode leave of a sequence.
//
// The kernels keep scores in the log2 domain, z = log2(e) * scale * q.k.  With a
// cap c > 0 the score s becomes c tanh(s / c); since tanh x = 1 - 2 / (1 + e^(2x)),
// in the log2 domain  z' = C - 2C / (1 + 2^(z * 2/c)),  C = c log2(e):  one exp2,
// one reciprocal and one fused multiply-add.  Both SFU results are good to about
// 2^-22 relative, so z' is off by at most ~C * 2^-22 (2e-5 for c = 50), which moves a
// probability by 1.2e-5 relative, far below the 2^-9 of a 16-bit output.
// A distance bias then adds -slope * |i - j|.
#pragma once
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

struct NoScore {};

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float fast_rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// C tanh(z / C) in the log2 domain.  (2^x overflows to inf: the reciprocal gives
// 0 and the result C; it underflows to 0: -C.)
__device__ __forceinline__ float soft_cap(float z, float cap2, float cap_rate)
{
    return fmaf(-2.f * cap2, fast_rcp(1.f + fast_exp2(z * cap_rate)), cap2);
}

// Tokens of group g's prefix, in whole blocks.
__device__ __forceinline__ int prefix_tokens(const int32_t* group_prefix, int g, int block_size, int max_blocks)
{
    const int p = max(__ldg(group_prefix + g), 0) / block_size;
    return min(p, max_blocks) * block_size;
}

// First key that some of a sequence's nq query rows (the last nq of its L tokens)
// may see, clamped into [0, L] (a shared decode) or [0, L - 1].
__device__ __forceinline__ int first_visible(const ScoreParams& sc, int s, int L, int nq,
                                             int block_size, int max_blocks, unsigned* err)
{
    if (L <= 0) return 0;
    if (sc.group_of_seq) {
        const int g = __ldg(sc.group_of_seq + s);
        if (g >= sc.num_groups) set_error(err, PA_ERR_OUT_OF_RANGE);
        if (g < 0 || g >= sc.num_groups) return 0;
        return min(prefix_tokens(sc.group_prefix, g, block_size, max_blocks), L);
    }
    int lo = sc.window > 0 ? L - nq - sc.window + 1 : 0;
    if (sc.first_key) {
        int f = __ldg(sc.first_key + static_cast<int64_t>(s) * nq);
        for (int i = 1; i < nq; ++i) f = min(f, __ldg(sc.first_key + static_cast<int64_t>(s) * nq + i));
        lo = max(lo, f);
    }
    return min(max(lo, 0), L - 1);
}

// First visible key of query row i (of nq) of a sequence, at position `pos`.
__device__ __forceinline__ int row_first(const ScoreParams& sc, int s, int nq, int i, int pos)
{
    int lo = sc.window > 0 ? pos - sc.window + 1 : 0;
    if (sc.first_key) lo = max(lo, __ldg(sc.first_key + static_cast<int64_t>(s) * nq + i));
    return lo;
}

}  // namespace pa

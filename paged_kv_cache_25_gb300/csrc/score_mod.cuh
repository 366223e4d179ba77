// Score modifications of the scored attention calls, and the key ranges they and
// the shared-prefix decode leave of a sequence.
//
// The kernels keep scores in the log2 domain, z = log2(e) * scale * q.k.  With a
// cap c > 0 the score s becomes c tanh(s / c); since tanh x = 1 - 2 / (1 + e^(2x)),
// in the log2 domain  z' = C - 2C / (1 + 2^(z * 2/c)),  C = c log2(e):  one exp2,
// one reciprocal and one fused multiply-add.  Both SFU results are good to about
// 2^-22 relative and the difference is taken of numbers of size C, so z' is off by up to
// 4.4e-7 C whatever its size (5e-7 C in the prefill's form, whose quotients are products):
// 3.6e-5 for c = 50, 9e-5 for c = 128, which moves a probability by 6.4e-5 relative, far
// below the 2^-9 of a 16-bit output, but 0.7 for c = 1e6.  Caps above 128 therefore take
// kernels with the wide form (soft_cap_wide), good to 2^-20 of z' itself.
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

// The largest cap (log2 domain) whose scores are off by little enough without the series.
constexpr float kNearCap = 128.f * kLog2e;

// C tanh(z / C) for any C.  With x = z / C, for |x| < 3/8 the odd series
//   tanh x = x - x^3/3 + 2 x^5/15 - 17 x^7/315 + 62 x^9/2835 - ...,
// whose next term is at most 5e-7 of the sum there; else the form above, whose cancellation
// is then bounded by C / z' < 2.8.  e: z * cap_rate = 2 x log2(e).
__device__ __forceinline__ float soft_cap_wide(float z, float e, float cap2)
{
    const float x = e * (0.5f / kLog2e), x2 = x * x;
    float w = fmaf(62.f / 2835.f, x2, -17.f / 315.f);
    w = fmaf(w, x2, 2.f / 15.f);
    w = fmaf(w, x2, -1.f / 3.f);
    const float near = fmaf(z, w * x2, z);      // (not selected where x2 overflows)
    const float far = fmaf(-2.f * cap2, fast_rcp(1.f + fast_exp2(e)), cap2);
    return fabsf(x) < 0.375f ? near : far;
}

// The prefill's form of the cap, for four raw scores of a row at a time: with
// t_i = 1 + 2^(rate s_i) and h = -1 / (2C), z_i = C + 1 / (h t_i), and the four quotients
// share one reciprocal, r = 1 / (h t_0 h t_1 h t_2 h t_3).  The prefill is bound by the
// latency of a tile's softmax, so by the instructions of a score: sharing leaves 4.5 of
// them and 2.25 results of the exponent unit, against 5 and 3.  Mixed step's four chunks
// (bf16 / fp16 / FP8 pool): 284 / 256 / 267 us with a reciprocal each, 257 / 221 / 232 with
// one for two, 251 / 210 / 217 with one for four (193 / 153 / 149 without a cap).  Also
// measured: tanh as a rational function of degree 7/6 on the FMA pipe (330 / 286 / 301),
// and a polynomial for |x| < 3/4 behind a vote on the largest |score| (258 / 212 / 226).
// CLAMP keeps the exponents within +-kCapExp, so that the product cannot overflow (past
// it tanh is 1 to 2^-kCapExp) and a NaN, which a masked key's score may be, becomes the
// lower bound; without it the caller has checked the row's largest exponent.  (C is at
// least 0.18, so h^4 2^(4 kCapExp) stays below 2^126.)
struct CapForm {
    float rate;           // log2 of e^(2 x) for a raw score of 1
    float cap2, h;
};
constexpr float kCapExp = 30.f;

// scale_log2: log2-domain scale of the row's raw scores
__device__ __forceinline__ CapForm cap_form(float cap2, float cap_rate, float scale_log2)
{
    CapForm f;
    f.rate = scale_log2 * cap_rate;
    f.cap2 = cap2;
    f.h = -0.5f / cap2;
    return f;
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// z[i] = C tanh(x_i) + (top[i] - C)
template <bool CLAMP>
__device__ __forceinline__ void soft_cap4(const CapForm& f, const float (&s)[4], const float (&top)[4],
                                          float (&z)[4])
{
    float2 t[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float2 e;
        if constexpr (CLAMP) {
            e.x = fminf(fmaxf(s[2 * i] * f.rate, -kCapExp), kCapExp);
            e.y = fminf(fmaxf(s[2 * i + 1] * f.rate, -kCapExp), kCapExp);
        } else {
            e = fma2(make_float2(s[2 * i], s[2 * i + 1]), both(f.rate), both(0.f));
        }
        t[i] = fma2(make_float2(fast_exp2(e.x), fast_exp2(e.y)), both(f.h), both(f.h));
    }
    const float qa = t[0].x * t[0].y, qb = t[1].x * t[1].y;
    const float r = fast_rcp(qa * qb), ra = r * qb, rb = r * qa;   // 1 / qa, 1 / qb
    z[0] = fmaf(ra, t[0].y, top[0]); z[1] = fmaf(ra, t[0].x, top[1]);
    z[2] = fmaf(rb, t[1].y, top[2]); z[3] = fmaf(rb, t[1].x, top[3]);
}

// Tokens of group g's prefix, in whole blocks.
__device__ __forceinline__ int prefix_tokens(const int32_t* group_prefix, int g, int block_size, int max_blocks)
{
    const int p = max(load_input(group_prefix + g), 0) / block_size;
    return min(p, max_blocks) * block_size;
}

// First key that some of a sequence's nq query rows (the last nq of its L tokens)
// may see, clamped into [0, L] (a shared decode) or [0, L - 1].
__device__ __forceinline__ int first_visible(const ScoreParams& sc, int s, int L, int nq,
                                             int block_size, int max_blocks, unsigned* err)
{
    if (L <= 0) return 0;
    if (sc.group_of_seq) {
        const int g = load_input(sc.group_of_seq + s);
        if (g >= sc.num_groups) set_error(err, PA_ERR_OUT_OF_RANGE);
        if (g < 0 || g >= sc.num_groups) return 0;
        return min(prefix_tokens(sc.group_prefix, g, block_size, max_blocks), L);
    }
    int lo = sc.window > 0 ? L - nq - sc.window + 1 : 0;
    if (sc.first_key) {
        int f = load_input(sc.first_key + static_cast<int64_t>(s) * nq);
        for (int i = 1; i < nq; ++i) f = min(f, load_input(sc.first_key + static_cast<int64_t>(s) * nq + i));
        lo = max(lo, f);
    }
    return min(max(lo, 0), L - 1);
}

// First visible key of query row i (of nq) of a sequence, at position `pos`.
__device__ __forceinline__ int row_first(const ScoreParams& sc, int s, int nq, int i, int pos)
{
    int lo = sc.window > 0 ? pos - sc.window + 1 : 0;
    if (sc.first_key) lo = max(lo, load_input(sc.first_key + static_cast<int64_t>(s) * nq + i));
    return lo;
}

}  // namespace pa

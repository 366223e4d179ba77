#pragma once
// The 4-bit row format of PA_FP4_E2M1 pools, on the device.
//
// A row is one (token, KV head)'s d values: d / 2 bytes of E2M1 codes, element 2i in the low
// half of byte i, then d / 16 bytes of E4M3 scales, one for 16 elements.  A value is
// e2m1(code) * e4m3(scale) * S with the pool's own scale S.  The first product has at
// most 2 + 4 significant bits and lies, zero aside, in [2^-10, 2688]: fp16 holds it exactly.
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "pa_device.cuh"

namespace pa {

constexpr int kFp4Group = 16;        // elements that share a scale
__host__ __device__ constexpr int fp4_row_bytes(int d) { return d / 2 + d / kFp4Group; }

// The largest of two magnitudes, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ float e4m3_to_float(uint32_t byte)
{
    uint32_t h;
    asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(byte));
    return __low2float(*reinterpret_cast<const __half2*>(&h));
}

// Sixteen elements as codes (8 bytes, first element lowest) and their scale's code.
// scale: S; six: 6 S in fp32.  Every step is rounded to fp32 by itself (IEEE division), so the bytes
// do not depend on how the compiler contracts: s = e4m3(max|x| / (6 S)) kept in [2^-9, 448],
// codes e2m1(x / (s S)), to nearest even, saturated at 6.  (Quotients rounded as IEEE division rounds them, not
// products with a reciprocal: 16-bit inputs often lie exactly between two codes.)  A NaN among the
// sixteen becomes the scale's NaN, so that all of them read as NaN; infinities saturate.
//
// The sixteen quotients x / r share their divisor, so they are made by Markstein's method (Computation of elementary
// functions on the IBM RISC System/6000 processor, 1990) from y = 1 / r rounded to nearest: with y' = y (1 - r y), the
// rest of 1 / r, q = x y + x y' is one of the two fp32 neighbours of x / r, its remainder x - q r is
// exact, and q + (x - q r) y rounds to the quotient.  That holds while nothing over- or underflows, which
// r in [2^-60, 2^60] and |x| <= 8 r make sure of (a remainder too small to be exact comes with a
// quotient that is far below the first border, 1/4); a group outside of that divides.  The sign is x's own (-0 keeps
// its code).  The rotary write of 8192 tokens of Llama-3-8B's heads: 39.5 us, 41.7 with
// divisions; by three axes 46.5 and 48.3; the plain write 15.4 and 16.8.
__device__ __forceinline__ uint2 fp4_quantise(const float (&x)[kFp4Group], float scale, float six, uint32_t& code)
{
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < kFp4Group; ++i) a = max_nan(a, fabsf(x[i]));
    if (a != a) {
        code = 0x7Fu;
        return make_uint2(0u, 0u);
    }
    const float t = fminf(fmaxf(__fdiv_rn(a, six), 0x1p-9f), 448.f);
    code = __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
    const float r = __fmul_rn(e4m3_to_float(code), scale);
    float q[kFp4Group];
    if (r >= 0x1p-60f && r <= 0x1p60f && a <= 8.f * r) {
        const float y = __frcp_rn(r), rest = __fmul_rn(y, __fmaf_rn(-r, y, 1.f));
#pragma unroll
        for (int i = 0; i < kFp4Group; ++i) {
            const float n = __fmaf_rn(x[i], y, __fmul_rn(x[i], rest));
            q[i] = copysignf(__fmaf_rn(__fmaf_rn(-n, r, x[i]), y, n), x[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kFp4Group; ++i) q[i] = __fdiv_rn(x[i], r);
    }
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        w[h] = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[h] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(q[8 * h + 2 * i], q[8 * h + 2 * i + 1]),
                                                                   __NV_E2M1, cudaRoundNearest))
                    << (8 * i);
        }
    }
    return make_uint2(w[0], w[1]);
}

// Stores a group's codes and scale into its row (rows of 36 bytes are 4-byte aligned).
template <int D>
__device__ __forceinline__ void fp4_store(uint8_t* row, int group, uint2 codes, uint32_t scale)
{
    if constexpr (D == 128) {
        *reinterpret_cast<uint2*>(row + group * 8) = codes;
    } else {
        *reinterpret_cast<uint32_t*>(row + group * 8) = codes.x;
        *reinterpret_cast<uint32_t*>(row + group * 8 + 4) = codes.y;
    }
    row[D / 2 + group] = static_cast<uint8_t>(scale);
}

// Eight codes (a 32-bit word, first element lowest) as four f16x2 words.
__device__ __forceinline__ void fp4x8_to_h2x4(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d)
{
    asm("{\n\t.reg .b8 p, q, r, s;\n\t"
        "mov.b32 {p, q, r, s}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, p;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, q;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, r;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, s;\n\t}"
        : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
        : "r"(w));
}

// Two E4M3 codes (the low 16 bits) as f16x2.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t w)
{
    uint32_t h;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(w));
    return h;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Four rows of a matrix (box {row, 1}) into consecutive shared memory.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int r0, int r1, int r2, int r3, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(bar)
        : "memory");
}

}  // namespace pa

#pragma once
// What the chunked prefill's converter warps do for FP4 pools: 4-bit rows (fp4.cuh) widened into the
// rings that the MMAs read.
#include "fp4.cuh"
#include "pa_device.cuh"

namespace pa {

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// A staged chunk of kRows rows (K or V) into its ring stage, [keys][D] fp16 in 64-element halves of
// 128-byte swizzled rows: codes times scales, exact.  row0: the chunk's first row in the key tile of kKeys (a
// multiple of 8); rows at or past `keep` become zeros (their scales may be NaN).  One group of 16 elements a lane and
// step, 8 bytes of codes and their scale: two 16-byte pieces of the ring, of which every 8 lanes write 8 in distinct
// banks.  All loads come before the first store, which the compiler would not move them across, and the
// stores' addresses are four sums (the swizzle of a row repeats every 8) with constant offsets.
template <int D, int kRows, int kKeys>
__device__ __forceinline__ void f4_widen_chunk(const uint8_t* src, uint32_t dst, int lane, int row0, int keep)
{
    constexpr int kPer = kRows * D / 512, kStep = D == 128 ? 4 : 8;    // rows from a step to the next
    int rl, p;   // first row in the chunk, group
    if constexpr (D == 128) {
        const int gg = lane >> 3, l8 = lane & 7;
        rl = 2 * (gg >> 1) + ((l8 >> 2) ^ (gg & 1));
        p = l8;
    } else {
        rl = lane / (D / 16);
        p = lane % (D / 16);
    }
    const uint8_t* from = src + rl * fp4_row_bytes(D);
    uint2 c[kPer];
    uint32_t sc[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint8_t* at = from + i * kStep * fp4_row_bytes(D);
        if constexpr (D == 128) {
            c[i] = *reinterpret_cast<const uint2*>(at + 8 * p);
        } else {
            c[i].x = *reinterpret_cast<const uint32_t*>(at + 8 * p);
            c[i].y = *reinterpret_cast<const uint32_t*>(at + 8 * p + 4);
        }
        sc[i] = at[D / 2 + p];
    }
    if (row0 + kRows > keep) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (row0 + rl + i * kStep >= keep) {
                c[i] = make_uint2(0u, 0u);
                sc[i] = 0u;
            }
        }
    }
    const uint32_t at = dst + (p >> 2) * (kKeys * 128) + (row0 + rl) * 128 + (((2 * p & 7) ^ (rl & 7)) << 4);
    const uint32_t to[4] = {at, at ^ 16u, at ^ 64u, at ^ 80u};        // (at's bits 4 .. 6 are the piece alone)
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t s2 = e4m3x2_to_h2(sc[i] * 0x101u);
        const int odd = kStep == 4 ? 2 * (i & 1) : 0;
        uint32_t w[8];
        fp4x8_to_h2x4(c[i].x, w[0], w[1], w[2], w[3]);
        fp4x8_to_h2x4(c[i].y, w[4], w[5], w[6], w[7]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            st_shared_v4(to[odd + h] + i * kStep * 128, hmul2(w[4 * h], s2), hmul2(w[4 * h + 1], s2),
                         hmul2(w[4 * h + 2], s2), hmul2(w[4 * h + 3], s2));
    }
}

}  // namespace pa

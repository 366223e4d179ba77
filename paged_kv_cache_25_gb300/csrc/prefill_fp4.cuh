#pragma once
// What the chunked prefill's converter warps do for FP4 pools: 4-bit rows (fp4.cuh) widened into the
// rings that the MMAs read.
#include "fp4.cuh"
#include "pa_device.cuh"

namespace pa {

constexpr int kF4Converters = 3, kF4ChunkKeys = 64;

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// Converter pw of kF4Converters: every one of them runs this loop as a whole warp.
//
// A key tile of kKeys keys is four chunks of 64 rows, K's two and then V's, and chunk g of the whole sequence
// goes to converter g % 3: copied as the pool has it by one gather of four 16-row tiles into this warp's buffer, read into registers
// (after which the buffer takes the next chunk), widened, and stored into its ring stage, [keys][D] fp16 in
// 64-element halves of 128-byte swizzled rows: codes times scales, exact.  Rows at or past the context become
// zeros (their scales may be NaN).  A lane and step take one group of 16 elements, 8 bytes of codes and their
// scale: two 16-byte pieces of the ring, of which every 8 lanes write 8 in distinct banks.
//
// What bounds it: a lone warp beside four softmax warps, so the latency of its instructions, of which a chunk
// has ~24 for 16 elements and ~100 more around them (chunks of 32 rows by two untiled copies, their loads between
// the stores and the block ids loaded when they were needed: the converters took 7000 clocks a tile, the rest ~3500).
template <int D, int BS, int kKeys, int kStages>
__device__ __forceinline__ void f4_convert(const CUtensorMap* kmap, const CUtensorMap* vmap, const int32_t* table,
                                           int max_blocks, int num_blocks, int n_kv, int kvh, int L, int n_tiles, int pw,
                                           int lane, const uint8_t* buf, uint32_t buf_addr, uint32_t ring_k, uint32_t ring_v,
                                           uint32_t code_full, uint32_t k_full, uint32_t k_empty, uint32_t v_full,
                                           uint32_t v_empty, unsigned* err)
{
    constexpr int kRows = kF4ChunkKeys, kRow = fp4_row_bytes(D);
    constexpr int kStageBytes = kKeys * D * 2;
    constexpr int kPer = kRows * D / 512, kStep = D == 128 ? 4 : 8;    // steps, rows from one to the next
    static_assert(kKeys == 2 * kRows, "two chunks of K, two of V");
    const int total = (4 * n_tiles - pw + kF4Converters - 1) / kF4Converters;   // this warp's chunks
    // lane c < 8: the block id of 16-key piece c of tile t (-1: past the table; 0 for pieces at or past L)
    auto piece_id = [&](int t) -> int {
        const int key0 = t * kKeys + (lane & 7) * 16;
        if (lane >= 8 || t >= n_tiles || key0 >= L) return 0;
        return key0 / BS < max_blocks ? __ldg(table + key0 / BS) : -1;
    };
    // and that piece's tile of the pool (32 bits hold any pool's slots)
    auto piece_of = [&](int id) -> int {
        if (id < 0 || id >= num_blocks) {
            set_error(err, PA_ERR_OUT_OF_RANGE);
            id = 0;
        }
        return (id * n_kv + kvh) * (BS / 16) + (lane & (BS / 16 - 1));
    };
    // of tiles id_tile and id_tile + 1; the ids of tile id_tile + 2 are on their way
    int id_tile = 0;
    int here = piece_of(piece_id(0)), next = piece_of(piece_id(1)), id_ahead = piece_id(2);
    auto request = [&](int g) {
        const int j = g >> 2, e = g & 1;
        if (j > id_tile + 1) {                   // (three chunks on from the last: one tile at most)
            ++id_tile;
            here = next;
            next = piece_of(id_ahead);
            id_ahead = piece_id(id_tile + 2);
        }
        const int from = j == id_tile ? here : next;
        int r[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) r[x] = __shfl_sync(0xffffffffu, from, 4 * e + x);
        if (lane == 0) {
            mbar_arrive_expect_tx(code_full, kRows * kRow);
            tma_gather4(buf_addr, (g & 2) ? vmap : kmap, r[0], r[1], r[2], r[3], code_full);
        }
    };
    int rl, p;   // first row in the chunk, group
    if constexpr (D == 128) {
        const int gg = lane >> 3, l8 = lane & 7;
        rl = 2 * (gg >> 1) + ((l8 >> 2) ^ (gg & 1));
        p = l8;
    } else {
        rl = lane / (D / 16);
        p = lane % (D / 16);
    }
    const uint8_t* const from = buf + rl * kRow;
    const uint32_t off = (p >> 2) * (kKeys * 128) + rl * 128 + (((2 * p & 7) ^ (rl & 7)) << 4);

    if (total > 0) request(pw);
#pragma unroll 1
    for (int n = 0; n < total; ++n) {
        const int g = pw + kF4Converters * n, j = g >> 2, e = g & 1, st = j % kStages;
        const bool is_k = (g & 2) == 0;
        if (!__all_sync(0xffffffffu, mbar_wait(code_full, n & 1, err))) {
            mbar_wait(code_full, n & 1, err);    // the copy lands (bounded) before the CTA can exit
            return;
        }
        uint2 c[kPer];
        uint32_t sc[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint8_t* at = from + i * kStep * kRow;
            if constexpr (D == 128) {
                c[i] = *reinterpret_cast<const uint2*>(at + 8 * p);
            } else {      // (rows of 36 bytes)
                c[i].x = *reinterpret_cast<const uint32_t*>(at + 8 * p);
                c[i].y = *reinterpret_cast<const uint32_t*>(at + 8 * p + 4);
            }
            sc[i] = at[D / 2 + p];
        }
        const int keep = L - j * kKeys - e * kRows;         // rows of the chunk that exist (may exceed 64)
        if (keep < kRows) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (rl + i * kStep >= keep) {
                    c[i] = make_uint2(0u, 0u);
                    sc[i] = 0u;
                }
            }
        }
        __syncwarp();                            // every lane has read the buffer
        if (n + 1 < total) request(g + kF4Converters);
        if (j >= kStages &&
            !__all_sync(0xffffffffu, mbar_wait((is_k ? k_empty : v_empty) + 8 * st, ((j / kStages) - 1) & 1, err))) {
            if (n + 1 < total) mbar_wait(code_full, (n + 1) & 1, err);     // (likewise)
            return;
        }
        // (the pieces' place in a row lies in bits 4 .. 6 alone, and rows repeat their swizzle every 8)
        const uint32_t at = (is_k ? ring_k : ring_v) + st * kStageBytes + e * kRows * 128 + off;
        const uint32_t to[4] = {at, at ^ 16u, at ^ 64u, at ^ 80u};
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
        fence_proxy_async_smem();                // ring writes -> the MMAs' reads
        __syncwarp();
        if (lane == 0) mbar_arrive((is_k ? k_full : v_full) + 8 * st);
    }
}

}  // namespace pa

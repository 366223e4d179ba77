#pragma once
// What the chunked prefill's converter warps do for FP4 pools: 4-bit rows (fp4.cuh) widened into the
// rings that the MMAs read.
#include "fp4.cuh"
#include "pa_device.cuh"

#include <type_traits>

namespace pa {

constexpr int kF4Converters = 3;
// Keys of a converter's chunk, 4608 bytes either way (the warp's work around a chunk is the same for both head sizes; with
// chunks of 64 keys of 64 elements the converters were the slowest part there too).
template <int D>
constexpr int kF4ChunkKeys = D == 64 ? 128 : 64;

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// Converter pw of kF4Converters: every one of them runs this loop as a whole warp.
//
// A key tile of kKeys keys is chunks of K and then as many of V, and chunk g of the whole sequence
// goes to converter g % 3: copied as the pool has it by gathers of four 16-row tiles into this warp's buffer, read into registers
// (after which the buffer takes the next chunk), widened, and stored into its ring stage, [keys][D] fp16 in
// 64-element halves of 128-byte swizzled rows: codes times scales, exact.  Rows at or past the context become
// zeros (their scales may be NaN).  A lane and step take one group of 16 elements, 8 bytes of codes and their
// scale: two 16-byte pieces of the ring, of which every 8 lanes write 8 in distinct banks.
//
// What bounds it: a lone warp beside four softmax warps, so the latency of its instructions, of which a chunk
// has ~24 for 16 elements and ~100 more around them (chunks of 32 rows by two untiled copies, their loads between
// the stores and the block ids loaded when they were needed: the converters took 7000 clocks a tile, now 3500).
// Four chunks of 512 rows after 1024 - 8192 tokens of Llama-3-8B's heads: 155 us, 1060 TFLOP/s (247 at first).
template <int D, int BS, int kKeys, int kStages>
__device__ __forceinline__ void f4_convert(const CUtensorMap* kmap, const CUtensorMap* vmap, const int32_t* table,
                                           int max_blocks, int num_blocks, int n_kv, int kvh, int L, int tile0, int n_tiles,
                                           int pw, int lane, const uint8_t* buf, uint32_t buf_addr, uint32_t ring_k, uint32_t ring_v,
                                           uint32_t code_full, uint32_t k_full, uint32_t k_empty, uint32_t v_full,
                                           uint32_t v_empty, unsigned* err)
{
    constexpr int kRows = kF4ChunkKeys<D>, kRow = fp4_row_bytes(D), kBytes = kRows * kRow;
    constexpr int kHalf = kKeys / kRows, kChunks = 2 * kHalf;          // chunks of K a tile, and of K and V
    constexpr int kStageBytes = kKeys * D * 2;
    constexpr int kPer = kRows * D / 512, kStep = D == 128 ? 4 : 8;    // steps, rows from one to the next
    static_assert(kKeys % kRows == 0 && kRows % 64 == 0, "whole chunks of whole gathers");
    const int total = (kChunks * n_tiles - pw + kF4Converters - 1) / kF4Converters;   // this warp's chunks
    // lane c < 8: the block id of 16-key piece c of tile t (-1: past the table; 0 for pieces at or past L)
    auto piece_id = [&](int t) -> int {
        const int key0 = (tile0 + t) * kKeys + (lane & 7) * 16;
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
    // The block ids of the next chunk's tile are loaded with the chunk before.
    int ids = piece_id(pw / kChunks);
    auto request = [&](int g) {
        const int item = g % kChunks, first = item % kHalf * (kRows / 16), piece = piece_of(ids);
        int r[kRows / 16];
#pragma unroll
        for (int x = 0; x < kRows / 16; ++x) r[x] = __shfl_sync(0xffffffffu, piece, first + x);
        if (lane == 0) {
            const CUtensorMap* map = item < kHalf ? kmap : vmap;
            mbar_arrive_expect_tx(code_full, kBytes);
#pragma unroll
            for (int x = 0; x < kRows / 16; x += 4)
                tma_gather4(buf_addr + x * 16 * kRow, map, r[x], r[x + 1], r[x + 2], r[x + 3], code_full);
        }
        ids = piece_id((g + kF4Converters) / kChunks);
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
        const int g = pw + kF4Converters * n, j = g / kChunks, item = g % kChunks, e = item % kHalf, st = j % kStages;
        const bool is_k = item < kHalf;
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
        const int keep = L - (tile0 + j) * kKeys - e * kRows;         // rows of the chunk that exist (may exceed it)
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

// The query rows of a tile: this warp's 16 of the 32 that it shares with its pair, as fp16 in 64-element halves of
// 128-byte swizzled rows.  src(r): row r of the tile, or null (zeros).  bf16 rows are scaled into fp16 by a power of
// two (exact down to 2^-28 of the row's largest), whose exponent goes to exps[r]; fp16 rows stay as they are.  sign: flips
// the elements' signs.  Neighbouring lanes take neighbouring pieces, so a load reads whole rows (a row a lane: 14,000
// clocks a tile of bf16 rows of 128).
template <typename QT, int D, int kTileRows, typename Src>
__device__ __forceinline__ void f4_stage_queries(Src src, uint32_t dst, int first, int lane, uint32_t sign, float* exps)
{
    constexpr int kPieces = D / 8, kAtOnce = 32 / kPieces, kLoads = 16 / kAtOnce;
    const int c = lane % kPieces, r0 = first + lane / kPieces;
    uint4 v[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const QT* row = src(r0 + i * kAtOnce);
        v[i] = row ? __ldg(reinterpret_cast<const uint4*>(row) + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int r = r0 + i * kAtOnce;
        uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        if constexpr (std::is_same<QT, __nv_bfloat16>::value) {
            uint32_t top = 0;      // magnitudes compare as integers
#pragma unroll
            for (int x = 0; x < 4; ++x) top = max(top, max(w[x] & 0x7FFFu, (w[x] >> 16) & 0x7FFFu));
#pragma unroll
            for (int m = kPieces / 2; m > 0; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
            // the largest lands in [2^14, 2^15) unless tiny
            const int e = max(static_cast<int>(top >> 7) - 141, -100);
            const float down = __int_as_float((127 - e) << 23);
            if (c == 0) exps[r] = __int_as_float((127 + e) << 23);
#pragma unroll
            for (int x = 0; x < 4; ++x)
                w[x] = Cvt<__half>::pack(__uint_as_float(w[x] << 16) * down, __uint_as_float(w[x] & 0xFFFF0000u) * down);
        }
        st_shared_v4(dst + (c >> 3) * (kTileRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4), w[0] ^ sign, w[1] ^ sign,
                     w[2] ^ sign, w[3] ^ sign);
    }
}

// Half an output row of D / 2 values a lane, 16 bits each, to memory through 32 x D bytes of shared memory of this warp's
// own, so that a store writes whole half rows (straight from the registers: 6,700 clocks a tile of rows of 128).  dst(r): this
// half of the row of lane r, or null.
template <int D, typename Dst>
__device__ __forceinline__ void f4_store_rows(Dst dst, uint32_t smem, int lane, const uint4 (&w)[D / 16])
{
    constexpr int kPieces = D / 16, kAtOnce = 32 / kPieces;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
        st_shared_v4(smem + lane * D + ((i ^ (lane & (kPieces - 1))) << 4), w[i].x, w[i].y, w[i].z, w[i].w);
    __syncwarp();
    const int c = lane % kPieces;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int r = i * kAtOnce + lane / kPieces;
        uint4 x;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "r"(smem + r * D + ((c ^ (r & (kPieces - 1))) << 4))
                     : "memory");
        if (uint16_t* to = dst(r)) reinterpret_cast<uint4*>(to)[c] = x;
    }
}

}  // namespace pa

// Decode attention over FP4 pools, one query row a sequence or several (pa_decode,
// pa_decode_verify), up to 32 rows a KV head; calls of more go to the chunked prefill's kernel.
//
// Mathematics: out = softmax(scale q K^T) V over each sequence's keys, in one pass with a
// running maximum m and sum l per row; the partials (m, l, O) of key ranges merge exactly,
//   out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
//
// Work: the rows of all (sequence, KV head, up to RU of its (head, query) rows), one after another,
// are a line of 128-token granules with kRowCost more units before each row for what a piece costs
// beside its tokens (its queries and its combine take about as long as a granule); every block of a
// persistent grid takes an equal run of it.  (40 sequences of 100 - 2047 tokens and 40 KV heads, kernels
// alone: 98 us without those units, when blocks with rows of one granule came last, 72 with one, 74 with two.)
// A block's run holds whole rows, which it finishes, and at most two pieces of rows that it shares
// with its neighbours, whose partials meet in f4_merge_kernel.  A piece's four warps take 32 tokens
// of each stage and combine through shared memory.
//
// Stages of 128 tokens (32 a warp) arrive in a ring that the block's warps share, each by four
// cp.async.bulk.tensor gathers of four 16-token tiles (a tile's rows are contiguous in the pool, so
// the pool is a matrix with a tile a row), which the warps issue in turn.  (Rings of a warp's own,
// one untiled copy a tile: 174 us for 151 at the sizes below, by the instructions around the copies;
// filled by cp.async: 155 - 160.)  A warp works on its tokens transposed, on m16n8k16 fp16 MMAs:
// S^T = K q^T with tokens as the MMA rows, O^T = V^T P^T with elements of d as the rows, the unit's
// rows as the columns (NT tiles of 8).
//   - Row r of a score tile is token 4 ((r & 7) >> 1) + 2 (r >> 3) + (r & 1) of its piece; the transpose
//     of P (movmatrix) then leaves lane (g, t4) = (lane / 4, lane % 4) with tokens 4 t4 .. 4 t4 + 3, whose V
//     codes it reads in 8-byte (d 64: 4-byte) pieces without bank conflicts (rows lie 72 bytes apart).
//   - Neither K nor V is stored transposed.  K's codes lie along d, as its fragments pair them.
//     V's fragments pair tokens: the codes of two tokens are put together half byte by half
//     byte before they are widened (two shifts and two three-input logic operations for 16 codes).
//   - The k order of S is free: lane t4 holds elements (d / 4) t4 and on of its tokens, one or two
//     scales, and q is loaded to match.  Lane g holds elements (d / 8) g and on of V: one scale a token.
//   - Codes times scales are exact in fp16 (fp4.cuh).  bf16 queries are scaled by a power of two into
//     fp16 (exact down to 2^-29 of the row's largest element).
//   - P enters P V as one fp16 part, 11 bits, half a step of which is 2^-11 of P.  The exponents' reference lies 7
//     powers of two below the largest score that set it (kPRoom), so P begins at 2^7 and what fp16 rounds off below its
//     smallest normal number is at most 2^-32 of the largest weight: an output moves by at most 2^-11 of the largest |v|
//     that it averages and 2^-32 of it for each key, far below what 4 bits do to v.  (With P from 1 on, a key 17.4 nats
//     above 520,000 equal ones moved outputs by 3e-3 of |v|: each of the others is 0 in fp16, and together they are not.)
//
// Bound: HBM at 4.5 bits a value, and beside it the instructions that widen.  HBM gives an SM's
// quarter 397 clocks for 16 tokens of a head (d 128); its 64 conversions and 64 multiplies issue
// every other clock and its 16 MMAs hold the dispatch for 8 clocks each, 254 in all, of ~240
// instructions.  256 sequences of 512 - 4096 tokens of Llama-3-8B's heads: 134 us, 5.1 TB/s (0.75 of
// the copy rate), issue 60 %; 8 us pass before the first stage is there and 4 until the merge is
// done.  Eight sequences of 20,000 - 110,000 tokens: 109 us, 5.5 TB/s.  (K's products on tcgen05 with
// scores back from TMEM: 178 us, by the threads around the MMAs.)
#include "fp4.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"

#include <math.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

namespace pa {

constexpr int kF4Warps = 4;
constexpr int kF4Threads = kF4Warps * 32;
constexpr int kPieceTok = 16;             // tokens of a tile of scores, and of one copy
constexpr int kStageTok = 32;             // tokens of a stage that a warp takes: two tiles
constexpr int kGranule = kF4Warps * kStageTok;   // tokens of a stage, and of a granule
constexpr int kRowCost = 1;               // units of a row beside its granules
constexpr float kPRoom = 7.f;             // powers of two that P has left below 2^15: the reference moves only past 2^8
constexpr int kF4PrefixCap = 768;         // sequences whose lengths are kept in shared memory
static_assert(kGranule == kF4GranuleTokens, "as the workspace counts them");

struct F4Params {
    void* out;
    const void* q;
    const int32_t *block_tables, *context_lens;
    // [blocks]: a row begun and not finished here, or -1; whether the head piece goes on.  May be null
    int4* info;
    float *ws_ml, *ws_acc;                // [blocks + tails][RU] (m, l) and O
    int row_tails;                        // whether a tail's slot goes by its row (else by its block)
    unsigned* err;
    pa_dtype out_dtype;
    int max_blocks, num_seqs, n_q, nq, n_kv, group, num_blocks, bs_log;
    float scale_log2, v_scale;            // softmax scale times k_scale, in the log2 domain
};

// Resident blocks an SM and ring stages.
template <int D, int RU>
struct F4Cfg {
    static constexpr int kRow = fp4_row_bytes(D);
    static constexpr int kTile = kPieceTok * kRow;                          // bytes of a 16-token tile of K or V
    static constexpr int kTiles = kGranule / kPieceTok;                     // tiles of K, and of V, a stage
    static constexpr int kStage = 2 * kTiles * kTile;                       // K tiles, then V tiles
    // (16 rows, two tiles of accumulators: with three blocks an SM 256 sequences of 16 rows of 64 elements took 145 us for
    // 176, of 128 elements, whose accumulators spilled, 254 for 240; kernels alone)
    static constexpr int kCtas = RU == 16 ? (D == 64 ? 3 : 2) : 4;
    static constexpr int kNS = RU == 16 ? (D == 64 ? 3 : 4) : (D == 64 ? 4 : 2);
    static constexpr int kRing = kNS * kStage;
    static constexpr int kReduce = kF4Warps * RU * (D + 2) * 4;
    static constexpr int kReds = RU == 4 ? 2 : 1;      // combine buffers: two save a barrier a piece
    static constexpr int kDynBytes = kRing + kReds * kReduce + 128;         // (aligned to 128 bytes)
    static_assert(kCtas * (kDynBytes + 1024 + 3584) <= 233472, "shared memory of an SM");
    static_assert(kNS <= kF4Warps, "a warp copies at most one of the first stages");
};

__device__ __forceinline__ void f4_store4(void* out, int64_t i, float4 v, pa_dtype dt)
{
    if (dt == PA_F32)
        *reinterpret_cast<float4*>(static_cast<float*>(out) + i) = v;
    else if (dt == PA_BF16)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + i) =
            make_uint2(Cvt<__nv_bfloat16>::pack(v.x, v.y), Cvt<__nv_bfloat16>::pack(v.z, v.w));
    else
        *reinterpret_cast<uint2*>(static_cast<__half*>(out) + i) =
            make_uint2(Cvt<__half>::pack(v.x, v.y), Cvt<__half>::pack(v.z, v.w));
}

// S^T of one tile: st[n][0, 1] row g, [2, 3] row g + 8; columns 8 n + 2 t4 and the next.
template <int D, int NT>
__device__ __forceinline__ void f4_scores(const uint8_t* k, int g, int t4, const uint32_t (&q)[NT][D / 16][2],
                                          float (&st)[NT][4])
{
    constexpr int kRow = fp4_row_bytes(D), kHalves = D / 64;
    uint2 w[2][kHalves];
    uint32_t s[2][kHalves];
    const uint8_t* row = k + (4 * (g >> 1) + (g & 1)) * kRow;
#pragma unroll
    for (int i = 0; i < 2; ++i, row += 2 * kRow) {
        if constexpr (D == 128) {
#pragma unroll
            for (int h = 0; h < kHalves; ++h) w[i][h] = *reinterpret_cast<const uint2*>(row + 16 * t4 + 8 * h);
            const uint32_t both = e4m3x2_to_h2(*reinterpret_cast<const uint16_t*>(row + D / 2 + 2 * t4));
            s[i][0] = __byte_perm(both, 0, 0x1010);
            s[i][kHalves - 1] = __byte_perm(both, 0, 0x3232);
        } else {      // (rows of 36 bytes)
            w[i][0].x = *reinterpret_cast<const uint32_t*>(row + 8 * t4);
            w[i][0].y = *reinterpret_cast<const uint32_t*>(row + 8 * t4 + 4);
            s[i][0] = e4m3x2_to_h2(__byte_perm(*reinterpret_cast<const uint32_t*>(row + D / 2), 0, t4 * 0x11));
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) st[n][e] = 0.f;
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int y = 0; y < 2; ++y) {          // 8 codes: two steps of 4
            uint32_t u[4], x[4];
            fp4x8_to_h2x4(y ? w[0][h].y : w[0][h].x, u[0], u[1], u[2], u[3]);
            fp4x8_to_h2x4(y ? w[1][h].y : w[1][h].x, x[0], x[1], x[2], x[3]);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const int kk = 4 * h + 2 * y + z;
                const uint32_t a[4] = {hmul2(u[2 * z], s[0][h]), hmul2(x[2 * z], s[1][h]),
                                       hmul2(u[2 * z + 1], s[0][h]), hmul2(x[2 * z + 1], s[1][h])};
#pragma unroll
                for (int n = 0; n < NT; ++n) MmaOp<__half>::run(st[n], a, q[n][kk][0], q[n][kk][1]);
            }
        }
}

// O^T += V^T P^T of one tile.  Byte b of a lane's codes is m-tile b, its low half row g, its high half row
// g + 8.  valid: tokens of the tile that exist (kMasked; else all); the scales of the others may be
// anything, even NaN, and count as 0.
template <int D, int NT, bool kMasked>
__device__ __forceinline__ void f4_values(const uint8_t* v, int g, int t4, int valid, const uint32_t (&pt)[NT][2],
                                          float (&o)[NT][D / 16][4])
{
    constexpr int kRow = fp4_row_bytes(D), kWords = D / 64;       // words of 8 codes a token
    const uint8_t* row = v + 4 * t4 * kRow;
    uint32_t x[4][kWords], sc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (D == 128) {
            const uint2 u = *reinterpret_cast<const uint2*>(row + j * kRow + 8 * g);
            x[j][0] = u.x;
            x[j][kWords - 1] = u.y;
        } else {
            x[j][0] = *reinterpret_cast<const uint32_t*>(row + j * kRow + 4 * g);
        }
        sc[j] = row[j * kRow + D / 2 + (D == 128 ? g : g >> 1)];
    }
    if constexpr (kMasked) {
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[j] = 4 * t4 + j < valid ? sc[j] : 0u;
    }
    const uint32_t s01 = e4m3x2_to_h2(__byte_perm(sc[0], sc[1], 0x0040)), s23 = e4m3x2_to_h2(__byte_perm(sc[2], sc[3], 0x0040));
    // the low halves of a's bytes and the high halves of b's
    auto take = [](uint32_t a, uint32_t b) {
        uint32_t d;
        asm("lop3.b32 %0, %1, %2, 0x0F0F0F0F, 0xE4;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    };
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        uint32_t a0[4], a1[4], a2[4], a3[4];
        fp4x8_to_h2x4(take(x[0][w], x[1][w] << 4), a0[0], a0[1], a0[2], a0[3]);
        fp4x8_to_h2x4(take(x[0][w] >> 4, x[1][w]), a1[0], a1[1], a1[2], a1[3]);
        fp4x8_to_h2x4(take(x[2][w], x[3][w] << 4), a2[0], a2[1], a2[2], a2[3]);
        fp4x8_to_h2x4(take(x[2][w] >> 4, x[3][w]), a3[0], a3[1], a3[2], a3[3]);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint32_t a[4] = {hmul2(a0[b], s01), hmul2(a1[b], s01), hmul2(a2[b], s23), hmul2(a3[b], s23)};
#pragma unroll
            for (int n = 0; n < NT; ++n) MmaOp<__half>::run(o[n][4 * w + b], a, pt[n][0], pt[n][1]);
        }
    }
}

template <typename QT, int D, int RU, bool MQ>
__global__ void __launch_bounds__(kF4Threads, F4Cfg<D, RU>::kCtas)
f4_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ F4Params p)
{
    using Cfg = F4Cfg<D, RU>;
    constexpr int NT = RU == 16 ? 2 : 1, NS = Cfg::kNS, kTiles = kStageTok / kPieceTok;   // kTiles: a warp's of a stage
    constexpr bool kBf16 = std::is_same<QT, __nv_bfloat16>::value;

    __shared__ int s_table[kF4PrefixCap];        // the sequences' lengths
    __shared__ int s_scan[kF4Warps], s_begin[3];
    __shared__ __align__(8) uint64_t s_full[NS], s_empty[NS];
    extern __shared__ uint8_t dyn_smem[];
    uint8_t* const smem = dyn_smem + (-smem_u32(dyn_smem) & 127u);     // (an offset, so that it stays a shared address)

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int nq = MQ ? p.nq : 1;
    const int rows_kv = p.group * nq;                        // rows of a KV head, head-major
    const int n_groups = p.n_kv * ((rows_kv + RU - 1) / RU);
    const int max_ctx = p.max_blocks << p.bs_log;
    if (tid < NS) {
        mbar_init(smem_u32(&s_full[tid]), 1);
        mbar_init(smem_u32(&s_empty[tid]), kF4Warps);
    }
    fence_mbar_init();
    if (tid == 0) {
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    grid_dependency_wait();      // launched as a programmatic dependent: every input may come from the kernel before

    // ---- this block's run of units.  A thread takes `mine` neighbouring sequences, and the one in
    // whose rows the run begins finds the place.
    auto granules = [&](int L) { return L < nq || L <= 0 ? 0 : (min(L, max_ctx) + kGranule - 1) / kGranule; };
    auto units = [&](int L) { const int J = granules(L); return J ? J + kRowCost : 0; };      // of a row
    const bool tabled = p.num_seqs <= kF4PrefixCap;
    int left;                                    // units of the run that are not in a piece yet
    int at_s, at_unit, at_grp;                   // where the next piece begins
    {
        const int mine = (p.num_seqs + kF4Threads - 1) / kF4Threads;
        const int s0 = min(p.num_seqs, tid * mine), s1 = min(p.num_seqs, s0 + mine);
        int local = 0;
        for (int s = s0; s < s1; ++s) {
            const int L = __ldg(p.context_lens + s);
            if (L > 0 && L < nq) set_error(p.err, PA_ERR_OUT_OF_RANGE);   // fewer keys than query rows
            if (tabled) s_table[s] = L;
            local += units(L);
        }
        int run = local;
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, run, w);
            if (lane >= w) run += up;
        }
        if (lane == 31) s_scan[warp] = run;
        __syncthreads();
        run -= local;
        int sum = 0;
#pragma unroll
        for (int i = 0; i < kF4Warps; ++i) {
            if (i < warp) run += s_scan[i];
            sum += s_scan[i];
        }
        const int total = sum * n_groups, blocks = gridDim.x;
        const int base = total / blocks, more = total - base * blocks, b = blockIdx.x;
        const int begin = b * base + min(b, more);
        left = base + (b < more ? 1 : 0);
        if (left == 0) {                         // uniform over the block
            if (tid == 0 && p.info) p.info[blockIdx.x] = make_int4(-1, 0, 0, 0);
            return;
        }
        const int x = begin / n_groups;
        if (run <= x && x < run + local) {       // one thread
            int s = s0, n = units(__ldg(p.context_lens + s));
            while (run + n <= x) {
                run += n;
                n = units(__ldg(p.context_lens + ++s));
            }
            const int off = begin - run * n_groups, grp = off / n;
            s_begin[0] = s;
            s_begin[1] = grp;
            s_begin[2] = off - grp * n;
        }
        __syncthreads();
        at_s = s_begin[0];
        at_grp = s_begin[1];
        at_unit = s_begin[2];
    }
    auto len_of = [&](int s) { return tabled ? s_table[s] : __ldg(p.context_lens + s); };

    // A piece: tokens [t0, t1) of the rows r0 .. r0 + nh - 1 of a KV head of sequence s, in n stages.
    struct Piece {
        int s, L, grp, kvh, r0, nh, t0, t1, n;
        bool live, tail;                         // tail: the rows' keys go on past t1
    };
    auto next_piece = [&]() {
        Piece x{};
        int J = 0, g0 = 0, g1 = 0;               // the row's granules, and the piece's
        while (true) {
            if (left <= 0) return x;             // (not live)
            if (at_grp == n_groups) {
                at_grp = 0;
                ++at_s;
            }
            x.L = len_of(at_s);
            J = granules(x.L);
            if (J == 0) {                        // a sequence without keys
                ++at_s;
                continue;
            }
            const int n = min(left, J + kRowCost - at_unit);
            g0 = max(0, at_unit - kRowCost);
            g1 = max(0, at_unit + n - kRowCost);
            left -= n;
            at_unit = 0;
            x.grp = at_grp++;
            if (g1 > g0) break;                  // (else the run ends before the row's first granule)
        }
        x.live = true;
        x.s = at_s;
        const int n_sub = n_groups / p.n_kv;
        x.kvh = n_sub == 1 ? x.grp : x.grp / n_sub;
        x.r0 = (x.grp - x.kvh * n_sub) * RU;
        x.nh = min(RU, rows_kv - x.r0);
        const int end = min(x.L, max_ctx);
        x.n = g1 - g0;
        x.t0 = g0 * kGranule;
        x.t1 = min(end, g1 * kGranule);
        x.tail = x.t1 < end;
        return x;
    };
    const uint32_t ring32 = smem_u32(smem), full0 = smem_u32(s_full), empty0 = smem_u32(s_empty);

    // query fragments: columns 8 n + g; step kk is elements (d / 4) t4 + 4 kk and on.  A negative
    // softmax scale is applied as -q, so the largest raw score is the largest score.
    const uint32_t qsign = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    uint32_t q[NT][D / 16][2];
    float c_q[NT];            // softmax scale of column 8 n + g (log2 domain)
    auto load_q = [&](const Piece& x) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = 8 * n + g;
            if (r >= x.nh) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) q[n][kk][0] = q[n][kk][1] = 0u;
                continue;
            }
            const int hh = (x.r0 + r) / nq, qi = x.r0 + r - hh * nq;
            const QT* row = static_cast<const QT*>(p.q) +
                            ((static_cast<int64_t>(x.s) * nq + qi) * p.n_q + x.kvh * p.group + hh) * D + D / 4 * t4;
#pragma unroll
            for (int kk = 0; kk < D / 16; kk += 2) {
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + 4 * kk));
                q[n][kk][0] = u.x;
                q[n][kk][1] = u.y;
                q[n][kk + 1][0] = u.z;
                q[n][kk + 1][1] = u.w;
            }
        }
    };
    // Once the piece starts (so that the loads' latency overlaps the combine): signs, and bf16 -> fp16.  A quad holds
    // a row; the row is scaled by 2^-e so that its largest magnitude lands in [2^14, 2^15), and
    // 2^e goes into its softmax scale.
    auto scale_q = [&]() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            c_q[n] = fabsf(p.scale_log2);
            if constexpr (kBf16) {
                uint32_t top = 0;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        top = max(top, max(q[n][kk][h] & 0x7FFFu, (q[n][kk][h] >> 16) & 0x7FFFu));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = top == 0u ? 0 : max(static_cast<int>((top >> 7) & 0xFFu) - 141, -100);
                c_q[n] *= __int_as_float((127 + e) << 23);
                const float down = __int_as_float((127 - e) << 23);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 f = Cvt<__nv_bfloat16>::unpack(q[n][kk][h]);
                        q[n][kk][h] = Cvt<__half>::pack(f.x * down, f.y * down);
                    }
            }
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                q[n][kk][0] ^= qsign;
                q[n][kk][1] ^= qsign;
            }
        }
    };

    Piece cu = next_piece();
    if (!cu.live) {                              // uniform over the block
        if (tid == 0 && p.info) p.info[blockIdx.x] = make_int4(-1, 0, 0, 0);
        return;
    }
    const bool head = cu.t0 > 0;                 // the run begins inside a row
    bool first = true;
    Piece nx{};

    // ---- the block's stages, numbered on through its pieces.  The first NS are copied by warps 0 .. NS - 1; then,
    // as the warps begin on stage n, warp n % 4 copies stage n - 1 + NS into the slot of the stage before, which all
    // have left by then or are about to.  (Every warp waits for every stage's data, its own tokens among them or not:
    // so none can leave a slot, or wait for its next stage, before the slot's present stage has come.)
    // `duty` is the stage that this warp copies next; lanes 0 .. 7 hold the block ids of its tiles where
    // those are loaded already (id_stage).  A stage past the next piece has to wait until its piece is known.
    int duty = warp, id_stage = -1, id = 0;
    int first_n = 0;                             // number of the current piece's first stage
    bool timed_out = false;
    const int first_duty = (warp == 0 ? kF4Warps : warp) - 1 + NS;
    if (duty >= NS) duty = first_duty;
    auto load_ids = [&]() {                      // false: the stage's piece is not known
        int i = duty - first_n;
        const bool later = i >= cu.n;
        if (later) i -= cu.n;
        if (later && (!nx.live || i >= nx.n)) return false;
        const int tok = (later ? nx.t0 : cu.t0) + i * kGranule + lane * kPieceTok;
        if (lane < Cfg::kTiles && tok < (later ? nx.t1 : cu.t1))
            id = __ldg(p.block_tables + static_cast<int64_t>(later ? nx.s : cu.s) * p.max_blocks + (tok >> p.bs_log));
        id_stage = duty;
        return true;
    };
    auto copy_duty = [&]() {                     // whole warp
        if (id_stage != duty && !load_ids()) return;
        const int slot = duty % NS, round = duty / NS;
        // (a wait that has run out is not waited for again: the outputs are flagged)
        if (round > 0 && !timed_out) timed_out = !mbar_wait(empty0 + slot * 8, (round - 1) & 1, p.err);
        __syncwarp();
        int i = duty - first_n;
        const bool later = i >= cu.n;
        if (later) i -= cu.n;
        const int begin = (later ? nx.t0 : cu.t0) + i * kGranule, end = later ? nx.t1 : cu.t1;
        const int tok = begin + lane * kPieceTok;
        const bool there = lane < Cfg::kTiles && tok < end;
        int b = there ? id : 0;
        if (b < 0 || b >= p.num_blocks) {
            set_error(p.err, PA_ERR_OUT_OF_RANGE);
            b = 0;                               // keep the ring moving; the outputs are flagged
        }
        // (tiles past the end: any row; their tokens are masked)
        const int sub = (1 << (p.bs_log - 4)) - 1;
        const int row = there ? ((b * p.n_kv + (later ? nx.kvh : cu.kvh)) << (p.bs_log - 4)) + ((tok >> 4) & sub) : 0;
        const bool both = begin + 4 * kPieceTok < end;      // else only the first four tiles
        int r[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) r[k] = __shfl_sync(0xffffffffu, row, k);
        if (lane == 0) {
            const uint32_t bar = full0 + slot * 8, dst = ring32 + slot * Cfg::kStage;
            mbar_arrive_expect_tx(bar, (both ? 16 : 8) * Cfg::kTile);
            tma_gather4(dst, &kmap, r[0], r[1], r[2], r[3], bar);
            tma_gather4(dst + 8 * Cfg::kTile, &vmap, r[0], r[1], r[2], r[3], bar);
            if (both) {
                tma_gather4(dst + 4 * Cfg::kTile, &kmap, r[4], r[5], r[6], r[7], bar);
                tma_gather4(dst + 12 * Cfg::kTile, &vmap, r[4], r[5], r[6], r[7], bar);
            }
        }
        __syncwarp();
        duty = duty < NS ? first_duty : duty + kF4Warps;
        load_ids();                              // (in flight until the duty comes)
    };
    static_assert(Cfg::kTiles == 8, "two gathers of four tiles");
    if (duty < NS) load_ids();                   // (in flight over the queries' loads)
    load_q(cu);
    nx = next_piece();
    if (duty < NS) copy_duty();
    int number = 0, slot = 0;                         // the next stage, its slot and the slot's phase
    uint32_t phase = 0;

    float o[NT][D / 16][4];
    int buf = 0;
    while (cu.live) {
        scale_q();
        // this lane's columns 8 n + 2 t4 + e: softmax scales c, sums, and of the reference m of the exponents (a raw
        // score near the largest so far) kPRoom - m c and the raw score past which it moves
        float c[NT][2], ref[NT][2], bar_z[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                c[n][e] = __shfl_sync(0xffffffffu, c_q[n], 8 * t4 + 4 * e);
                ref[n][e] = 0.f;
                bar_z[n][e] = -INFINITY;
                l[n][e] = 0.f;
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) o[n][mt][e] = o[n][mt][2 + e] = 0.f;
            }
        // One stage of this warp, 32 tokens from pos0.  Masked: some of its keys are not there, or not visible to every row.
        auto stage = [&](auto masked, const uint8_t* st_k, const uint8_t* st_v, int pos0) {
            constexpr bool kMasked = decltype(masked)::value;
            float z[kTiles][NT][4];
#pragma unroll
            for (int i = 0; i < kTiles; ++i) f4_scores<D, NT>(st_k + i * Cfg::kTile, g, t4, q, z[i]);
            if constexpr (kMasked) {
                const int tA = pos0 + 4 * (g >> 1) + (g & 1);       // this lane's tokens of a tile: tA and tA + 2
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int col = 8 * n + 2 * t4 + e;
                        const int lim = min(MQ && col < cu.nh ? cu.L - nq + (cu.r0 + col) % nq + 1 : cu.L, cu.t1);
#pragma unroll
                        for (int i = 0; i < kTiles; ++i) {
                            z[i][n][e] = tA + i * kPieceTok < lim ? z[i][n][e] : -INFINITY;
                            z[i][n][2 + e] = tA + i * kPieceTok + 2 < lim ? z[i][n][2 + e] : -INFINITY;
                        }
                    }
            }
            // the columns' largest raw scores, met over the eight lanes of each t4.  The reference moves only
            // when the first key sets it or the largest is more than 2^8 past it (lazily: P stays below 2^(8 + kPRoom)).
            float mx[NT][2];
            bool moved = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(z[0][n][e], z[0][n][2 + e]);
#pragma unroll
                    for (int i = 1; i < kTiles; ++i) x = max3f(x, z[i][n][e], z[i][n][2 + e]);
                    mx[n][e] = x;
                    moved = moved || x > bar_z[n][e];
                }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = mx[n][e];
#pragma unroll
                        for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
                        if (x > bar_z[n][e]) {
                            // (scores so large that the products' rounding would use that room up keep it free)
                            const float far = -x * c[n][e], r = fabsf(far) < 0x1p20f ? far + kPRoom : far;
                            const float f = bar_z[n][e] == -INFINITY ? 0.f : fast_exp2(r - ref[n][e]);
                            ref[n][e] = r;
                            bar_z[n][e] = x + 8.f / c[n][e];      // (a scale of 0: never again)
                            l[n][e] *= f;
#pragma unroll
                            for (int mt = 0; mt < D / 16; ++mt) {
                                o[n][mt][e] *= f;
                                o[n][mt][2 + e] *= f;
                            }
                        }
                    }
            }
            uint32_t pt[kTiles][NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] = fast_exp2(fmaf(z[i][n][e], c[n][e & 1], ref[n][e & 1]));
                        // (even with scale 0, where the exponent is NaN)
                        if constexpr (kMasked) x[e] = z[i][n][e] == -INFINITY ? 0.f : x[e];
                    }
                    l[n][0] += x[0] + x[2];
                    l[n][1] += x[1] + x[3];
                    pt[i][n][0] = movmatrix_trans(Cvt<__half>::pack(x[0], x[1]));
                    pt[i][n][1] = movmatrix_trans(Cvt<__half>::pack(x[2], x[3]));
                }
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
                f4_values<D, NT, kMasked>(st_v + i * Cfg::kTile, g, t4, cu.t1 - pos0 - i * kPieceTok, pt[i], o);
        };
        const int open = min(cu.L - nq + 1, cu.t1);      // keys below it are there and visible to every row
#pragma unroll 1
        for (; number < first_n + cu.n; ++number) {
            const int pos0 = cu.t0 + (number - first_n) * kGranule + warp * kStageTok;
            if (!timed_out) timed_out = !mbar_wait(full0 + slot * 8, phase, p.err);
            __syncwarp();
            if (duty <= number - 1 + NS) copy_duty();
            const uint8_t* st_k = smem + slot * Cfg::kStage + warp * kTiles * Cfg::kTile;
            if (pos0 + kStageTok <= open) stage(std::false_type{}, st_k, st_k + Cfg::kTiles * Cfg::kTile, pos0);
            else if (pos0 < cu.t1) stage(std::true_type{}, st_k, st_k + Cfg::kTiles * Cfg::kTile, pos0);
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + slot * 8);
            slot = slot + 1 == NS ? 0 : slot + 1;
            phase ^= slot == 0 ? 1u : 0u;
        }
        // ---- this warp's partials: O of lane g's D / 8 elements and its columns, then (m, l)
        float* const red_o = reinterpret_cast<float*>(smem + Cfg::kRing + buf * Cfg::kReduce);   // [warps][RU][D]
        float* const red_m = red_o + kF4Warps * RU * D;                                 // [warps][RU], log2 domain
        float* const red_l = red_m + kF4Warps * RU;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], w);
                const int col = 8 * n + 2 * t4 + e;
                if (col < RU) {
                    float4* dst = reinterpret_cast<float4*>(red_o + (warp * RU + col) * D + D / 8 * g);
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
                        dst[i] = make_float4(o[n][2 * i][e], o[n][2 * i][2 + e], o[n][2 * i + 1][e], o[n][2 * i + 1][2 + e]);
                    if (g == 0) {
                        red_m[warp * RU + col] = bar_z[n][e] == -INFINITY ? -INFINITY : -ref[n][e];
                        red_l[warp * RU + col] = l[n][e];
                    }
                }
            }
        if (nx.live) load_q(nx);                     // its latency overlaps the combine
        else if (!timed_out) allow_dependent_launch();   // this block's last piece
        if (__syncthreads_or(timed_out)) {           // (else every warp's partials are written)
            // the copies still in flight land first, as far as a limit allows
            for (int i = 0; tid == 0 && i < NS; ++i)
                for (uint32_t ph = 0; ph < 2; ++ph) mbar_wait(full0 + i * 8, ph, p.err, 10000000ull);
            timed_out = true;
            break;
        }
        // pieces that are not whole rows go to the workspace: slot b (the run's head), or one behind those (its tail)
        const bool shared_head = first && head, to_ws = shared_head || cu.tail;
        for (int idx = tid; idx < cu.nh * (D / 4); idx += kF4Threads) {
            const int r = idx / (D / 4), dd = idx % (D / 4) * 4;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kF4Warps; ++w) M = fmaxf(M, red_m[w * RU + r]);
            // M = -inf: no key of this piece is visible to the row (keys of later rows only)
            const float M_use = MQ && M == -INFINITY ? 0.f : M;
            float lsum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kF4Warps; ++w) {
                const float f = exp2f(red_m[w * RU + r] - M_use);
                lsum += f * red_l[w * RU + r];
                const float4 x = *reinterpret_cast<const float4*>(red_o + (w * RU + r) * D + dd);
                acc.x = fmaf(f, x.x, acc.x);
                acc.y = fmaf(f, x.y, acc.y);
                acc.z = fmaf(f, x.z, acc.z);
                acc.w = fmaf(f, x.w, acc.w);
            }
            if (!to_ws) {
                const int hh = MQ ? (cu.r0 + r) / nq : cu.r0 + r, qi = MQ ? cu.r0 + r - hh * nq : 0;
                const int64_t at = (static_cast<int64_t>(cu.s) * nq + qi) * p.n_q + cu.kvh * p.group + hh;
                const float inv = p.v_scale / lsum;
                f4_store4(p.out, at * D + dd, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv), p.out_dtype);
            } else {
                const int64_t w = (shared_head ? static_cast<int64_t>(blockIdx.x)
                                               : static_cast<int64_t>(gridDim.x) +
                                                     (p.row_tails ? cu.s * n_groups + cu.grp : blockIdx.x)) * RU + r;
                *reinterpret_cast<float4*>(p.ws_acc + w * D + dd) = acc;
                if (dd == 0) *reinterpret_cast<float2*>(p.ws_ml + 2 * w) = make_float2(M, lsum);
            }
        }
        if (!nx.live && tid == 0 && p.info)
            p.info[blockIdx.x] = make_int4(cu.tail && !shared_head ? cu.s * n_groups + cu.grp : -1,
                                           shared_head && cu.tail ? 1 : 0, 0, 0);
        // (two buffers: the next piece's partials go to the other; the one after meets a barrier first)
        if constexpr (Cfg::kReds == 1) __syncthreads();
        else buf ^= 1;
        first = false;
        first_n += cu.n;
        cu = nx;
        if (cu.live) {
            nx = next_piece();
            if (duty <= number - 1 + NS) copy_duty();      // (one that waited for its piece)
        }
    }
    if (timed_out && tid == 0 && p.info) p.info[blockIdx.x] = make_int4(-1, 0, 0, 0);
}

// Merges the pieces of rows that several blocks shared: block b takes the rows that decode block b began and did not
// finish, whose pieces are b's tail and the heads of the blocks after it, up to the first that does not go on.
// A thread has four neighbouring elements of a row; four slices of threads take the pieces in turn.
constexpr int kMergeThreads = 512, kMergeSlices = 4;

template <int D, int RU>
__global__ void __launch_bounds__(kMergeThreads) f4_merge_kernel(const __grid_constant__ F4Params p, int blocks)
{
    constexpr int kPer = kMergeThreads / kMergeSlices, kRows = kPer / (D / 4);      // rows at a time
    __shared__ float4 s_acc[kMergeSlices][kPer];
    __shared__ float s_m[kMergeSlices][kPer], s_l[kMergeSlices][kPer];
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.x;
    grid_dependency_wait();
    const int row = p.info[b].x;
    if (row < 0) return;
    if (tid < 32) {                           // pieces after b's
        int n = 0;
        for (int i0 = b + 1;; i0 += 32) {
            const unsigned ends = __ballot_sync(0xffffffffu, i0 + lane >= blocks || p.info[i0 + lane].y == 0);
            if (ends) {
                n = i0 - b + __ffs(ends) - 1;
                break;
            }
        }
        if (lane == 0) s_n = min(n, blocks - 1 - b);
    }
    __syncthreads();
    const int n = s_n;
    const int rows_kv = p.group * p.nq, n_sub = (rows_kv + RU - 1) / RU, n_groups = p.n_kv * n_sub;
    const int s = row / n_groups, grp = row - s * n_groups, kvh = grp / n_sub, r0 = (grp - kvh * n_sub) * RU;
    const int slice = tid / kPer, j = tid % kPer, dd = j % (D / 4) * 4;
    for (int ra = 0; ra < min(RU, rows_kv - r0); ra += kRows) {
        const int r = ra + j / (D / 4);
        const bool mine = r < min(RU, rows_kv - r0);
        auto slot = [&](int i) {              // of piece i
            return (i == 0 ? static_cast<int64_t>(blocks) + (p.row_tails ? row : b) : static_cast<int64_t>(b) + i) * RU + r;
        };
        float M = -INFINITY, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (mine) {
            for (int i = slice; i <= n; i += kMergeSlices) M = fmaxf(M, p.ws_ml[2 * slot(i)]);
            // (rows of several queries may see no key of a piece, or of all that this slice has)
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll 4
            for (int i = slice; i <= n; i += kMergeSlices) {
                const int64_t w = slot(i);
                const float2 ml = *reinterpret_cast<const float2*>(p.ws_ml + 2 * w);
                const float4 x = *reinterpret_cast<const float4*>(p.ws_acc + w * D + dd);
                const float f = exp2f(ml.x - ref);
                sum = fmaf(f, ml.y, sum);
                acc.x = fmaf(f, x.x, acc.x);
                acc.y = fmaf(f, x.y, acc.y);
                acc.z = fmaf(f, x.z, acc.z);
                acc.w = fmaf(f, x.w, acc.w);
            }
        }
        s_acc[slice][j] = acc;
        s_m[slice][j] = M;
        s_l[slice][j] = sum;
        __syncthreads();
        if (slice == 0 && mine) {
#pragma unroll
            for (int w = 1; w < kMergeSlices; ++w) M = fmaxf(M, s_m[w][j]);
            sum = 0.f;
            acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kMergeSlices; ++w) {
                const float f = exp2f(s_m[w][j] - M);
                const float4 x = s_acc[w][j];
                sum = fmaf(f, s_l[w][j], sum);
                acc.x = fmaf(f, x.x, acc.x);
                acc.y = fmaf(f, x.y, acc.y);
                acc.z = fmaf(f, x.z, acc.z);
                acc.w = fmaf(f, x.w, acc.w);
            }
            const int hh = (r0 + r) / p.nq, qi = r0 + r - hh * p.nq;
            const int64_t at = (static_cast<int64_t>(s) * p.nq + qi) * p.n_q + kvh * p.group + hh;
            const float inv = p.v_scale / sum;
            f4_store4(p.out, at * D + dd, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv), p.out_dtype);
        }
        __syncthreads();                      // (the next rows' partials)
    }
}

static cudaError_t f4_resident(int* sms)
{
    static std::mutex mu;
    static int cache[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!cache[dev]) e = cudaDeviceGetAttribute(&cache[dev], cudaDevAttrMultiProcessorCount, dev);
    *sms = cache[dev];
    return e;
}

template <typename QT, int D, int RU, bool MQ>
static cudaError_t run_f4(F4Params p, const DecodeArgs& a, void* workspace, size_t workspace_bytes, cudaStream_t s)
{
    using Cfg = F4Cfg<D, RU>;
    auto kern = f4_decode_kernel<QT, D, RU, MQ>;
    static SmemOptIn opt_in;
    const cudaError_t attr_err = opt_in(reinterpret_cast<const void*>(kern), Cfg::kDynBytes);
    if (attr_err != cudaSuccess) return attr_err;
    int sms = 0;
    cudaError_t e = f4_resident(&sms);
    if (e != cudaSuccess) return e;
    // no more blocks than granules that the tables can hold, nor than the workspace has room for
    const int max_ctx = p.max_blocks << p.bs_log;
    const int64_t most = f4_granules(p.num_seqs, p.nq, p.group, p.n_kv, max_ctx);
    int blocks = static_cast<int>(std::min<int64_t>(most, sms * Cfg::kCtas));
    while (blocks > 1 && f4_workspace_bytes(p.num_seqs, p.nq, p.group, p.n_kv, D, max_ctx, blocks) > workspace_bytes)
        blocks -= std::max(1, blocks / 64);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const bool split = max_ctx > kGranule;    // (rows of one granule are never shared)
    if (split) {
        p.info = reinterpret_cast<int4*>(ws);
        p.ws_ml = reinterpret_cast<float*>(ws + 16ll * blocks);
        const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.n_kv * ((p.group * p.nq + RU - 1) / RU);
        p.row_tails = rows <= blocks;
        p.ws_acc = p.ws_ml + (blocks + std::min<int64_t>(rows, blocks)) * RU * 2;
    }
    CUtensorMap kmap{}, vmap{};
    const uint64_t tiles = static_cast<uint64_t>(p.num_blocks) * p.n_kv << (p.bs_log - 4);
    if (encode_byte_rows(&kmap, a.k_cache, Cfg::kTile, tiles) != PA_OK || encode_byte_rows(&vmap, a.v_cache, Cfg::kTile, tiles) != PA_OK)
        return cudaErrorInvalidValue;
    cudaEvent_t ev0 = nullptr, ev1 = nullptr;
    profile_events(&ev0, &ev1);
    if (ev0) cudaEventRecord(ev0, s);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kF4Threads);
    cfg.dynamicSmemBytes = Cfg::kDynBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, kmap, vmap, p);
    if (ev1) cudaEventRecord(ev1, s);
    if (e != cudaSuccess || !split) return e;
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, f4_merge_kernel<D, RU>, p, blocks);
}

template <typename QT, int D>
static cudaError_t run_f4_rows(const F4Params& p, const DecodeArgs& a, void* ws, size_t ws_bytes, cudaStream_t s)
{
    switch (f4_unit_rows(p.nq * p.group)) {
        case 4: return p.nq == 1 ? run_f4<QT, D, 4, false>(p, a, ws, ws_bytes, s) : run_f4<QT, D, 4, true>(p, a, ws, ws_bytes, s);
        case 8: return p.nq == 1 ? run_f4<QT, D, 8, false>(p, a, ws, ws_bytes, s) : run_f4<QT, D, 8, true>(p, a, ws, ws_bytes, s);
        default: return p.nq == 1 ? run_f4<QT, D, 16, false>(p, a, ws, ws_bytes, s) : run_f4<QT, D, 16, true>(p, a, ws, ws_bytes, s);
    }
}

// Rows of a KV head past which the chunked prefill's kernel takes the call, its sequences as chunks of
// q_per_seq rows: one pass over the keys, on tcgen05, for up to 128 rows a tile, where the kernel above reads and widens them
// again for every 16.  64 sequences of 512 - 4096 tokens of 8 KV heads of 128 elements: 132 us for any
// number of rows up to 128, against 133 with 32 rows here, 177 - 188 with 40, 236 - 254 with 64, 458 with 128.
// The rule looks at rows alone, and a few long sequences lose by it: their row blocks, each cut over a cluster of at most
// eight, leave most of the GPU idle, where the line of work above fills it.  One of 60,000 tokens on one KV head 104 us
// with 40 rows against 34, on eight KV heads 107 against 69; eight of 20,000 - 110,000 on eight 701 against 475.
constexpr int kF4DecodeRows = 32;

cudaError_t launch_decode_fp4(const DecodeArgs& a, void* workspace, size_t workspace_bytes, cudaStream_t s)
{
    if (a.n_q / a.cache.n_kv_heads * a.q_per_seq > kF4DecodeRows) {
        PrefillArgs c{};
        c.out = a.out; c.out_dtype = a.out_dtype; c.q = a.q;
        c.k_cache = a.k_cache; c.v_cache = a.v_cache; c.cache = a.cache;
        c.block_tables = a.block_tables; c.max_blocks = a.max_blocks; c.context_lens = a.context_lens;
        c.num_reqs = a.num_seqs; c.max_q = a.q_per_seq; c.n_q = a.n_q; c.scale = a.scale; c.err = a.err;
        cudaEvent_t ev0 = nullptr, ev1 = nullptr;
        profile_events(&ev0, &ev1);
        if (ev0) cudaEventRecord(ev0, s);
        const cudaError_t e = launch_prefill_fp4(c, s);
        if (ev1) cudaEventRecord(ev1, s);
        return e;
    }
    F4Params p{};
    p.out = a.out; p.q = a.q; p.block_tables = a.block_tables; p.context_lens = a.context_lens;
    p.err = a.err; p.out_dtype = a.out_dtype;
    p.max_blocks = a.max_blocks; p.num_seqs = a.num_seqs; p.n_q = a.n_q; p.nq = a.q_per_seq;
    p.n_kv = a.cache.n_kv_heads; p.group = a.n_q / a.cache.n_kv_heads; p.num_blocks = a.cache.num_blocks;
    p.bs_log = a.cache.block_size == 32 ? 5 : 4;
    p.scale_log2 = a.scale * 1.4426950408889634f * a.cache.k_scale; p.v_scale = a.cache.v_scale;
    const int D = a.cache.head_dim;
    if (D != 64 && D != 128) return cudaErrorInvalidValue;
    if (a.cache.act_dtype == PA_BF16)
        return D == 64 ? run_f4_rows<__nv_bfloat16, 64>(p, a, workspace, workspace_bytes, s) : run_f4_rows<__nv_bfloat16, 128>(p, a, workspace, workspace_bytes, s);
    return D == 64 ? run_f4_rows<__half, 64>(p, a, workspace, workspace_bytes, s) : run_f4_rows<__half, 128>(p, a, workspace, workspace_bytes, s);
}

}  // namespace pa

// Rotary position embedding fused with the cache write: q and k are rotated by
// the angle of their token's position, q goes to its output and k (rotated) and
// v into their slots of the paged pool, in one pass over the projections.
//
// Mathematics: with angle a = position * base^(-2i/rot), i < rot/2, pair i of a
// head turns as  (x, y) -> (x cos a - y sin a, y cos a + x sin a).  The pair is
// elements (i, i + rot/2) of the head, or (2i, 2i + 1) in the interleaved form;
// elements at and past `rot` pass unchanged.  cos and sin come from the caller's
// fp32 table, the products are fp32 and each result is rounded once, to the
// dtype it is stored in (an E4M3 code of the value over the scale for FP8 pools, 4-bit rows for
// FP4 pools: fp4.cuh).
// With several position axes (time, height, width of a video's tokens) every pair has an axis of
// its own, whose position of the token is the one that turns it; all axes share one table.
//
// Bound: HBM for long chunks (every element is read once and written once,
// 3 flops each), launch latency for a decode step; for FP4 pools also the ~390 instructions of a group
// of 16 (K and V of 8192 tokens of 8 heads of 128 elements: 24 us, issue 46 %, HBM floor 6).  The forms with several
// axes of 16-bit types spill 48 - 56 bytes a thread at 64 registers, as they hold two loops over the tokens; the others none.
#include <cuda_fp8.h>
#include <algorithm>
#include <cmath>

#include "fp4.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

// Elements of one 16-byte piece as floats and back.
template <typename T>
struct Piece {
    static constexpr int kN = 16 / static_cast<int>(sizeof(T));
    __device__ __forceinline__ static uint4 fetch(const T* p)
    {
        return __ldcs(reinterpret_cast<const uint4*>(p));   // read once: streaming
    }
    __device__ __forceinline__ static void widen(uint4 u, float (&x)[kN])
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                x[i] = __uint_as_float(w[i]);
            } else {
                const float2 f = Cvt<T>::unpack(w[i]);
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            }
        }
    }
    __device__ __forceinline__ static void store(T* p, const float (&x)[kN])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(x[i]);
            else w[i] = Cvt<T>::pack(x[2 * i], x[2 * i + 1]);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Four values as E4M3 codes of x / scale (IEEE division, rounded to nearest
// even, saturated), first value in the low byte.  inv: 1 / scale where that is exact
// (a power of two: the product is then the quotient), else 0.
__device__ __forceinline__ uint32_t codes4(const float* x, float scale, float inv)
{
    float y[4];
    if (inv != 0.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = x[i] * inv;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __fdiv_rn(x[i], scale);
    }
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
    return (lo & 0xFFFFu) | (hi << 16);
}

struct RopeParams {
    const void *q, *k, *v;
    void *q_out, *k_cache, *v_cache;
    int64_t q_out_stride, q_stride, k_stride, v_stride;   // elements from token to token
    const int32_t* positions;
    const float* cos_sin;
    const int64_t* slots;
    int64_t num_slots;
    int num_tokens, max_position, rot, interleaved;
    int n_q, n_kv, head_dim, block_size;
    float k_scale, v_scale, k_inv, v_inv;
    unsigned* err;
    // several axes: positions of axis a at positions + a * axis_stride; the axis of pair i is
    // bits 2 (i % 16) and up of axis[i / 16]
    int64_t axis_stride;
    int axes;
    uint32_t axis[PA_MAX_ROPE_PAIRS / 16];
};

// A token's slot and position (AX: one for each axis).
template <bool AX = false>
struct Place {
    int64_t slot;
    int pos[AX ? PA_MAX_ROPE_AXES : 1];
};
template <bool AX = false>
__device__ __forceinline__ Place<AX> rope_place(const RopeParams& p, int t)
{
    Place<AX> w;
    w.slot = __ldg(p.slots + t);
    if constexpr (AX) {
#pragma unroll
        for (int a = 0; a < PA_MAX_ROPE_AXES; ++a)
            w.pos[a] = a < p.axes ? __ldg(p.positions + a * p.axis_stride + t) : 0;
    } else {
        w.pos[0] = __ldg(p.positions + t);
    }
    return w;
}
// Whether the token is written at all: not if it is padding or (flagged) its slot
// or its position is out of range.
template <bool AX>
__device__ __forceinline__ bool rope_written(const RopeParams& p, const Place<AX>& w)
{
    if (w.slot < 0) return false;
    bool ok = w.slot < p.num_slots;
#pragma unroll
    for (int pos : w.pos) ok = ok && pos >= 0 && pos < p.max_position;
    if (!ok) set_error(p.err, PA_ERR_OUT_OF_RANGE);
    return ok;
}

// Cosines and sines of pairs i0 .. i0 + N - 1 (i0 a multiple of 4).
template <int N, bool AX>
__device__ __forceinline__ void rope_angles(const RopeParams& p, const Place<AX>& at, int i0, float (&co)[N],
                                            float (&si)[N])
{
    int pos = at.pos[0];
    if constexpr (AX) {
        static_assert(N <= 16, "the pairs' axes lie in one word");
        const uint32_t bits = (p.axis[i0 / 16] >> (2 * (i0 % 16))) & ((1ull << (2 * N)) - 1u);
        auto pick = [&](uint32_t a) { return a < 2 ? (a ? at.pos[1] : at.pos[0]) : (a == 2 ? at.pos[2] : at.pos[3]); };
        if (bits != (bits & 3u) * (0x55555555u & ((1ull << (2 * N)) - 1u))) {   // pairs of several axes
#pragma unroll
            for (int x = 0; x < N; ++x) {
                const float* row = p.cos_sin + static_cast<int64_t>(pick((bits >> (2 * x)) & 3u)) * p.rot + i0 + x;
                co[x] = __ldg(row);
                si[x] = __ldg(row + p.rot / 2);
            }
            return;
        }
        pos = pick(bits & 3u);
    }
    const float4* cs = reinterpret_cast<const float4*>(p.cos_sin + static_cast<int64_t>(pos) * p.rot + i0);
    const float4* sn = cs + p.rot / 8;
#pragma unroll
    for (int x = 0; x < N / 4; ++x) {
        const float4 f = __ldg(cs + x), g = __ldg(sn + x);
        co[4 * x] = f.x; co[4 * x + 1] = f.y; co[4 * x + 2] = f.z; co[4 * x + 3] = f.w;
        si[4 * x] = g.x; si[4 * x + 1] = g.y; si[4 * x + 2] = g.z; si[4 * x + 3] = g.w;
    }
}

constexpr int kRopeThreads = 256;
// Blocks of a grid that covers more: four an SM (64 registers a thread).  8192 tokens
// of Llama-3-8B heads, bf16: 34.6 us (5.9 TB/s), against 50.2 with a block for every 256
// items and no next token in flight, 43.6 and 39.5 with grids of five and six an SM.
constexpr int kRopeBlocksPerSm = 4;
constexpr int kVTok = 16;             // FP8: tokens of one transposed V tile

// A thread moves two 16-byte pieces of one head: in the rotated part the two that
// its pairs lie in (pieces c and c + rot/2, or 2c and 2c + 1 interleaved: either way
// pairs c * kN .. + kN - 1), else two neighbours.  Consecutive threads take consecutive
// pieces, then heads, then tokens; a thread keeps its head and pieces and goes from
// token to token in steps of what the grid covers at once, the next token's pieces,
// slot and position in flight while it works on one.
template <typename T, bool F8>
struct RopeItem {
    static constexpr int N = Piece<T>::kN;
    int h, c, e0, e1;          // head of its tensor; pieces, and their elements
    bool is_q, is_v, turn;
    const T* src;              // the head's elements of token 0
    int64_t stride;
    __device__ __forceinline__ RopeItem(const RopeParams& p, int head, int c_) : c(c_)
    {
        is_q = head < p.n_q;
        is_v = head >= p.n_q + p.n_kv;
        turn = !is_v && c < p.rot / (2 * N);
        e0 = turn && !p.interleaved ? c * N : 2 * c * N;                 // first piece's element
        e1 = turn && !p.interleaved ? p.rot / 2 + c * N : e0 + N;        // second piece's
        h = is_q ? head : (is_v ? head - p.n_q - p.n_kv : head - p.n_q);
        src = static_cast<const T*>(is_q ? p.q : (is_v ? p.v : p.k)) + static_cast<int64_t>(h) * p.head_dim;
        stride = is_q ? p.q_stride : (is_v ? p.v_stride : p.k_stride);
    }
    // Turns the pieces by the cosines and sines that angles(co, si) gives and stores them as token t's, in slot `slot`.
    template <typename Angles>
    __device__ __forceinline__ void finish(const RopeParams& p, uint4 ra, uint4 rb, int t, int64_t slot, Angles angles) const
    {
        using Pc = Piece<T>;
        float a[N], b[N];
        Pc::widen(ra, a);
        Pc::widen(rb, b);
        if (turn) {
            float co[N], si[N];
            angles(co, si);
            if (p.interleaved) {
#pragma unroll
                for (int x = 0; x < N / 2; ++x) {
                    const float u = a[2 * x], w = a[2 * x + 1];
                    a[2 * x] = u * co[x] - w * si[x];
                    a[2 * x + 1] = w * co[x] + u * si[x];
                    const float u1 = b[2 * x], w1 = b[2 * x + 1];
                    b[2 * x] = u1 * co[N / 2 + x] - w1 * si[N / 2 + x];
                    b[2 * x + 1] = w1 * co[N / 2 + x] + u1 * si[N / 2 + x];
                }
            } else {
#pragma unroll
                for (int x = 0; x < N; ++x) {
                    const float u = a[x], w = b[x];
                    a[x] = u * co[x] - w * si[x];
                    b[x] = w * co[x] + u * si[x];
                }
            }
        }
        if (is_q) {
            T* dst = static_cast<T*>(p.q_out) + t * p.q_out_stride + static_cast<int64_t>(h) * p.head_dim;
            Pc::store(dst + e0, a);
            Pc::store(dst + e1, b);
        } else {
            // (the pool has fewer than 2^31 rows)
            const unsigned sl = static_cast<unsigned>(slot), bs = p.block_size, blk = sl / bs;
            const int64_t row = static_cast<int64_t>((blk * p.n_kv + h) * bs + sl % bs) * p.head_dim;
            if constexpr (F8) {   // K codes (V has its own tiles)
                uint8_t* dst = static_cast<uint8_t*>(p.k_cache) + row;
#pragma unroll
                for (int x = 0; x < N; x += 4) {
                    *reinterpret_cast<uint32_t*>(dst + e0 + x) = codes4(a + x, p.k_scale, p.k_inv);
                    *reinterpret_cast<uint32_t*>(dst + e1 + x) = codes4(b + x, p.k_scale, p.k_inv);
                }
            } else {
                T* dst = static_cast<T*>(is_v ? p.v_cache : p.k_cache) + row;
                Pc::store(dst + e0, a);
                Pc::store(dst + e1, b);
            }
        }
    }
};

// Several axes, where a warp's items are of one token and the table's row has at most 128 values: the lanes load
// the angles of two pairs each and share them through shared memory, the next token's in flight with its pieces, the
// positions (one axis a lane) two tokens ahead.  (With every thread picking its own pairs' positions and angles, 8192
// tokens of Llama-3-8B's heads and three axes took 48 us into an FP8 pool, now 41, 48.6 into an FP4 pool, now 46.5.)
template <typename T, bool F8>
__device__ __forceinline__ void rope_warp(const RopeParams& p, const RopeItem<T, F8>& w, int t, int step, uint4 ra, uint4 rb)
{
    using Pc = Piece<T>;
    constexpr int N = Pc::kN;
    __shared__ __align__(16) float s_angle[kRopeThreads / 32][128];
    float* const own = s_angle[threadIdx.x / 32];
    const int lane = threadIdx.x & 31, half = p.rot / 2;
    int axis[2];                        // of pairs lane and lane + 32
#pragma unroll
    for (int x = 0; x < 2; ++x) axis[x] = (p.axis[(lane + 32 * x) / 16] >> (2 * (lane % 16))) & 3u;
    auto position = [&](int i) { return lane < p.axes && i < p.num_tokens ? __ldg(p.positions + lane * p.axis_stride + i) : 0; };
    auto load = [&](int pos, float (&f)[4]) {      // cosines, then sines, of the two pairs
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int at = __shfl_sync(0xffffffffu, pos, axis[x]), pair = lane + 32 * x;
            const bool ok = pair < half && at >= 0 && at < p.max_position;
            const float* row = p.cos_sin + static_cast<int64_t>(at) * p.rot + pair;
            f[x] = ok ? __ldg(row) : 0.f;
            f[2 + x] = ok ? __ldg(row + half) : 0.f;
        }
    };
    int pos = position(t), next_pos = position(t + step);
    int64_t slot = __ldg(p.slots + t);
    float f[4];
    load(pos, f);
    while (true) {
        const int next = t + step;
        const bool more = next < p.num_tokens;
        uint4 na = ra, nb = rb;
        int64_t next_slot = slot;
        int far_pos = 0;
        if (more) {                     // (before this token's angles are waited for)
            na = Pc::fetch(w.src + next * w.stride + w.e0);
            nb = Pc::fetch(w.src + next * w.stride + w.e1);
            next_slot = __ldg(p.slots + next);
            far_pos = position(next + step);
        }
        const bool bad = __any_sync(0xffffffffu, pos < 0 || pos >= p.max_position) || slot >= p.num_slots;
        if (bad && slot >= 0) set_error(p.err, PA_ERR_OUT_OF_RANGE);
        const bool written = slot >= 0 && !bad;
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (lane + 32 * x < half) {
                own[lane + 32 * x] = f[x];
                own[half + lane + 32 * x] = f[2 + x];
            }
        __syncwarp();
        if (more) load(next_pos, f);
        if (written)
            w.finish(p, ra, rb, t, slot, [&](float (&co)[N], float (&si)[N]) {
#pragma unroll
                for (int x = 0; x < N; x += 4) {
                    const float4 a = *reinterpret_cast<const float4*>(own + w.c * N + x);
                    const float4 b = *reinterpret_cast<const float4*>(own + half + w.c * N + x);
                    co[x] = a.x; co[x + 1] = a.y; co[x + 2] = a.z; co[x + 3] = a.w;
                    si[x] = b.x; si[x + 1] = b.y; si[x + 2] = b.z; si[x + 3] = b.w;
                }
            });
        if (!more) return;
        __syncwarp();                   // every lane has read the angles
        t = next;
        ra = na;
        rb = nb;
        slot = next_slot;
        pos = next_pos;
        next_pos = far_pos;
    }
}

template <typename T, bool F8, bool AX>
__device__ __forceinline__ void rope_rows(const RopeParams& p, unsigned index, unsigned threads, int heads)
{
    using Pc = Piece<T>;
    constexpr int N = Pc::kN;
    const int per_head = p.head_dim / (2 * N);
    const unsigned per_token = static_cast<unsigned>(heads * per_head);
    const int step = static_cast<int>(threads / per_token);      // (the host gives at least one token)
    int t = static_cast<int>(index / per_token);
    if (t >= step || t >= p.num_tokens) return;
    const unsigned rem = index % per_token;
    const RopeItem<T, F8> w(p, static_cast<int>(rem / per_head), static_cast<int>(rem % per_head));

    uint4 ra = Pc::fetch(w.src + t * w.stride + w.e0), rb = Pc::fetch(w.src + t * w.stride + w.e1);
    if (AX && per_token % 32 == 0 && p.rot <= 128) {
        rope_warp(p, w, t, step, ra, rb);
        return;
    }
    Place<AX> at = rope_place<AX>(p, t);
    while (true) {
        const int next = t + step;                               // (below 2^31: tokens and grid are)
        const bool more = next < p.num_tokens;
        uint4 na = ra, nb = rb;
        Place<AX> next_at = at;
        if (more) {
            na = Pc::fetch(w.src + next * w.stride + w.e0);
            nb = Pc::fetch(w.src + next * w.stride + w.e1);
            next_at = rope_place<AX>(p, next);
        }
        if (rope_written(p, at))
            w.finish(p, ra, rb, t, at.slot, [&](float (&co)[N], float (&si)[N]) { rope_angles<N, AX>(p, at, w.c * N, co, si); });
        if (!more) return;
        t = next;
        ra = na;
        rb = nb;
        at = next_at;
    }
}

// 16-bit and fp32 pools: q, k and v heads alike.
template <typename T, bool AX>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocksPerSm) rope_kernel(const RopeParams p)
{
    grid_dependency_wait();     // a programmatic dependent: scheduled while the kernel before drains
    allow_dependent_launch();   // a decode launched next waits for this grid before it reads
    rope_rows<T, false, AX>(p, blockIdx.x * kRopeThreads + threadIdx.x, gridDim.x * kRopeThreads,
                        p.n_q + 2 * p.n_kv);
}

// FP8 pools: blocks v0 .. v0 + v_blocks - 1 take a V tile each, the others the q and k
// heads.  A tile is 16 tokens of 256 / D heads, whose codes are transposed through shared
// memory and written in the pool's V layout ([d][16 tokens] per piece): 16-byte rows when
// the 16 tokens fill one piece (a prompt's chunk), 4-byte words for aligned runs of 4, single
// bytes else (a decode step's tokens lie in 16 blocks).
template <typename T, int D, bool AX>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocksPerSm) rope_f8_kernel(const RopeParams p, unsigned v0, unsigned v_blocks)
{
    grid_dependency_wait();
    allow_dependent_launch();
    if (blockIdx.x < v0 || blockIdx.x >= v0 + v_blocks) {
        const unsigned blk = blockIdx.x < v0 ? blockIdx.x : blockIdx.x - v_blocks;
        rope_rows<T, true, AX>(p, blk * kRopeThreads + threadIdx.x, (gridDim.x - v_blocks) * kRopeThreads,
                           p.n_q + p.n_kv);
        return;
    }
    constexpr int kHeads = kRopeThreads / D;      // V heads of a tile
    constexpr int kPieces = D / 16;               // 16-element pieces of a row
    constexpr int kItems = kVTok * kPieces * kHeads;   // = threads
    static_assert(kItems == kRopeThreads, "one 16-element piece a thread");
    __shared__ __align__(16) uint8_t vt[kHeads][D][kVTok];
    __shared__ int64_t s_slot[kVTok], s_byte[kVTok];   // token's slot; its byte of head 0, row 0
    const int tid = threadIdx.x;
    const int head_tiles = (p.n_kv + kHeads - 1) / kHeads;
    const unsigned tile = blockIdx.x - v0;
    const int t0 = static_cast<int>(tile / head_tiles) * kVTok;
    const int h0 = static_cast<int>(tile % head_tiles) * kHeads;
    if (tid < kVTok) {
        s_slot[tid] = -1;
        if (t0 + tid < p.num_tokens) {
            const Place<AX> w = rope_place<AX>(p, t0 + tid);
            if (rope_written(p, w)) {
                const int64_t b = w.slot / p.block_size, o = w.slot - b * p.block_size;
                s_slot[tid] = w.slot;
                s_byte[tid] = (b * p.n_kv * (p.block_size / 16) + o / 16) * (D * 16) + (o & 15);
            }
        }
    }
    {
        // (tokens fastest: the bytes of a warp's stores into vt share words or banks' rows)
        const int hh = tid / (kVTok * kPieces), tt = tid % kVTok, c = tid / kVTok % kPieces;
        const int t = t0 + tt, h = h0 + hh;
        if (t < p.num_tokens && h < p.n_kv) {
            const T* src = static_cast<const T*>(p.v) + t * p.v_stride + static_cast<int64_t>(h) * D + c * 16;
            constexpr int N = Piece<T>::kN;
#pragma unroll
            for (int x = 0; x < 16; x += N) {
                float f[N];
                Piece<T>::widen(Piece<T>::fetch(src + x), f);
#pragma unroll
                for (int y = 0; y < N; y += 4) {
                    const uint32_t w = codes4(f + y, p.v_scale, p.v_inv);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        vt[hh][c * 16 + x + y + e][tt] = static_cast<uint8_t>(w >> (8 * e));
                }
            }
        }
    }
    __syncthreads();
    const int hh = tid / D, d = tid % D, h = h0 + hh;
    if (h >= p.n_kv) return;
    const uint8_t* row = vt[hh][d];
    uint8_t* const out = static_cast<uint8_t*>(p.v_cache) +
                         (static_cast<int64_t>(h) * (p.block_size / 16) * D + d) * 16;
    const int64_t s0 = s_slot[0];
    bool whole = s0 >= 0 && s0 % kVTok == 0;
#pragma unroll
    for (int i = 1; i < kVTok; ++i) whole = whole && s_slot[i] == s0 + i;
    if (whole) {
        *reinterpret_cast<uint4*>(out + s_byte[0]) = *reinterpret_cast<const uint4*>(row);
        return;
    }
#pragma unroll
    for (int q4 = 0; q4 < kVTok; q4 += 4) {
        const int64_t a = s_slot[q4];
        if (a >= 0 && a % 4 == 0 && s_slot[q4 + 1] == a + 1 && s_slot[q4 + 2] == a + 2 &&
            s_slot[q4 + 3] == a + 3) {
            *reinterpret_cast<uint32_t*>(out + s_byte[q4]) = *reinterpret_cast<const uint32_t*>(row + q4);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (s_slot[q4 + i] >= 0) out[s_byte[q4 + i]] = row[q4 + i];
        }
    }
}

// FP4 pools: blocks v0 .. v0 + v_blocks - 1 take a tile of K and V groups each (16 elements that
// share a scale), the others the q heads.  A thread quantises one group; a K group is rotated
// first, with its pairs' other elements read beside it (they come from the first-level cache:
// the neighbouring threads read the same rows).  The products of the rotation are rounded to
// fp32 before they are added, here alone: a sum contracted one way or another could move a
// value over the border between two codes.
template <typename T, int D, bool AX>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocksPerSm) rope_f4_kernel(const RopeParams p, unsigned v0, unsigned v_blocks)
{
    grid_dependency_wait();
    allow_dependent_launch();
    if (blockIdx.x < v0 || blockIdx.x >= v0 + v_blocks) {
        const unsigned blk = blockIdx.x < v0 ? blockIdx.x : blockIdx.x - v_blocks;
        rope_rows<T, false, AX>(p, blk * kRopeThreads + threadIdx.x, (gridDim.x - v_blocks) * kRopeThreads, p.n_q);
        return;
    }
    constexpr int kGroups = D / kFp4Group, kTok = kRopeThreads / (2 * kGroups);
    constexpr int N = 8;
    const int tid = threadIdx.x, c = tid % kGroups, tt = tid / kGroups % kTok;
    const bool is_v = tid / (kGroups * kTok) != 0;
    const unsigned tile = blockIdx.x - v0;
    const int t = static_cast<int>(tile / p.n_kv) * kTok + tt, h = static_cast<int>(tile % p.n_kv);
    if (t >= p.num_tokens) return;
    const Place<AX> at = rope_place<AX>(p, t);
    if (!rope_written(p, at)) return;
    const T* src = static_cast<const T*>(is_v ? p.v : p.k) + t * (is_v ? p.v_stride : p.k_stride) +
                   static_cast<int64_t>(h) * D;
    auto load8 = [&](int e, float (&x)[N]) {
        constexpr int n = Piece<T>::kN;
#pragma unroll
        for (int i = 0; i < N; i += n) {
            float f[n];
            Piece<T>::widen(__ldg(reinterpret_cast<const uint4*>(src + e + i)), f);
#pragma unroll
            for (int j = 0; j < n; ++j) x[i + j] = f[j];
        }
    };
    float x[kFp4Group];
#pragma unroll
    for (int hf = 0; hf < kFp4Group / N; ++hf) {
        const int e = c * kFp4Group + hf * N;
        float a[N];
        load8(e, a);
        if (!is_v && e < p.rot) {
            if (p.interleaved) {
                float co[N / 2], si[N / 2];
                rope_angles<N / 2, AX>(p, at, e / 2, co, si);
#pragma unroll
                for (int i = 0; i < N / 2; ++i) {
                    const float u = a[2 * i], w = a[2 * i + 1];
                    a[2 * i] = __fsub_rn(__fmul_rn(u, co[i]), __fmul_rn(w, si[i]));
                    a[2 * i + 1] = __fadd_rn(__fmul_rn(w, co[i]), __fmul_rn(u, si[i]));
                }
            } else {
                const bool second = e >= p.rot / 2;
                const int i0 = second ? e - p.rot / 2 : e;
                float b[N], co[N], si[N];
                load8(second ? i0 : e + p.rot / 2, b);
                rope_angles<N, AX>(p, at, i0, co, si);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float m = __fmul_rn(a[i], co[i]), o = __fmul_rn(b[i], si[i]);
                    a[i] = second ? __fadd_rn(m, o) : __fsub_rn(m, o);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) x[hf * N + i] = a[i];
    }
    const float scale = is_v ? p.v_scale : p.k_scale;
    uint32_t s;
    const uint2 codes = fp4_quantise(x, scale, __fmul_rn(6.f, scale), s);
    const unsigned sl = static_cast<unsigned>(at.slot), bs = p.block_size, blk = sl / bs;
    fp4_store<D>(static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) +
                     (static_cast<int64_t>(blk) * p.n_kv * bs + h * bs + sl % bs) * fp4_row_bytes(D),
                 c, codes, s);
}

template <typename T, bool AX>
static cudaError_t run_rope(const RopeParams& p, pa_dtype pool, cudaStream_t s)
{
    const bool f8 = pool == PA_FP8_E4M3, f4 = pool == PA_FP4_E2M1;
    const int per_head = p.head_dim / (2 * Piece<T>::kN);
    const int64_t per_token = static_cast<int64_t>(p.n_q + (f8 ? 1 : (f4 ? 0 : 2)) * p.n_kv) * per_head;
    const int64_t items = p.num_tokens * per_token;
    // as many blocks as the GPU holds, but at least one token's threads
    const int64_t most = std::max<int64_t>(152 * kRopeBlocksPerSm, (per_token + kRopeThreads - 1) / kRopeThreads);
    const unsigned blocks = static_cast<unsigned>(std::min(most, (items + kRopeThreads - 1) / kRopeThreads));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (f4) {
        const int tok = kRopeThreads / (2 * (p.head_dim / kFp4Group));
        const unsigned kv_blocks = static_cast<unsigned>((p.num_tokens + tok - 1) / tok) * static_cast<unsigned>(p.n_kv);
        const unsigned first = kv_blocks <= 152 * kRopeBlocksPerSm / 2 ? 0 : blocks;   // (as the V tiles below)
        cfg.gridDim = dim3(blocks + kv_blocks);
        if (p.head_dim == 128) return cudaLaunchKernelEx(&cfg, rope_f4_kernel<T, 128, AX>, p, first, kv_blocks);
        if (p.head_dim == 64) return cudaLaunchKernelEx(&cfg, rope_f4_kernel<T, 64, AX>, p, first, kv_blocks);
        return cudaErrorInvalidValue;
    }
    if (!f8) return cudaLaunchKernelEx(&cfg, rope_kernel<T, AX>, p);
    const int tile_heads = kRopeThreads / p.head_dim;
    const unsigned v_blocks = static_cast<unsigned>((p.num_tokens + kVTok - 1) / kVTok) *
                              static_cast<unsigned>((p.n_kv + tile_heads - 1) / tile_heads);
    // V tiles, whose chain of steps is the longer one, go first while they leave room for the
    // others beside them (512 scattered tokens 7.3 -> 5.5 us), else last (8192 tokens: 37 against 39)
    const unsigned v0 = v_blocks <= 152 * kRopeBlocksPerSm / 2 ? 0 : blocks;
    cfg.gridDim = dim3(blocks + v_blocks);
    if (p.head_dim == 128) return cudaLaunchKernelEx(&cfg, rope_f8_kernel<T, 128, AX>, p, v0, v_blocks);
    if (p.head_dim == 64) return cudaLaunchKernelEx(&cfg, rope_f8_kernel<T, 64, AX>, p, v0, v_blocks);
    return cudaErrorInvalidValue;
}

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s)
{
    RopeParams p;
    p.q = a.q; p.k = a.k; p.v = a.v; p.q_out = a.q_out;
    p.k_cache = a.k_cache; p.v_cache = a.v_cache;
    p.q_out_stride = a.q_out_stride; p.q_stride = a.q_stride;
    p.k_stride = a.k_stride; p.v_stride = a.v_stride;
    p.positions = a.positions; p.cos_sin = a.cos_sin; p.slots = a.slots;
    p.num_slots = static_cast<int64_t>(a.cache.num_blocks) * a.cache.block_size;
    p.num_tokens = a.num_tokens; p.max_position = a.max_position;
    p.rot = a.rot_dim; p.interleaved = a.interleaved;
    p.n_q = a.n_q; p.n_kv = a.cache.n_kv_heads; p.head_dim = a.cache.head_dim;
    p.block_size = a.cache.block_size;
    p.k_scale = a.cache.k_scale; p.v_scale = a.cache.v_scale; p.err = a.err;
    // exact reciprocals only: a power of two whose inverse is a normal float
    auto inverse = [](float x) {
        int e = 0;
        return std::frexp(x, &e) == 0.5f && e > -120 && e < 120 ? 1.f / x : 0.f;
    };
    p.k_inv = inverse(a.cache.k_scale);
    p.v_inv = inverse(a.cache.v_scale);
    p.axes = a.axes;
    p.axis_stride = a.axis_stride;
    std::copy(a.axis, a.axis + PA_MAX_ROPE_PAIRS / 16, p.axis);
    auto run = [&](auto zero) {
        using T = decltype(zero);
        return a.axes > 1 ? run_rope<T, true>(p, a.cache.dtype, s) : run_rope<T, false>(p, a.cache.dtype, s);
    };
    switch (a.in_dtype) {
        case PA_BF16: return run(__nv_bfloat16{});
        case PA_F16: return run(__half{});
        case PA_F32: return run(0.f);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa

// How the prefix pass of a shared decode is dealt to thread blocks, decided on the
// device from the groups as they are (no host round trip, so a captured graph follows
// groups that change between replays).
//
// A unit is (group, tile of 256 (member, query head) rows of one KV head, KV head, range
// of the prefix's 128-key tiles).  The prefix is cut into at most S ranges, S chosen by a
// model of the pass: waves of thread blocks times (key tiles of the longest range + 2,
// the tiles' worth of time that a block spends before its first and after its last tile).
#pragma once
#include "score_mod.cuh"

#include <limits.h>

namespace pa {

struct PrefixUnit {
    int group, kvh, split, tile0, tiles, row0, rows, first_seq, prefix;
    bool live;
};

constexpr int kUnitRows = 256, kUnitKeys = 128;
constexpr int kUnitMembers = kUnitRows + 1;   // members that a row tile can touch
constexpr float kUnitOverhead = 2.f;

// Every thread of the block calls it.  scratch: 4 * num_groups ints of shared memory;
// members: kUnitMembers ints, filled with the sequences of the unit's rows (member
// m of the tile serves rows m * group - row0 .. of it, from member row0 / group on).
__device__ __forceinline__ void plan_prefix_unit(const ScoreParams& sc, const PrefixPass& sp, int n_kv,
                                                 int group, int block_size, int max_blocks,
                                                 const int32_t* context_lens, int* scratch,
                                                 int* members, PrefixUnit* unit, unsigned* err)
{
    __shared__ int s_warp[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x;
    const int G = sc.num_groups;
    int* count = scratch;
    int* first = scratch + G;
    int* prefix = scratch + 2 * G;
    int* context = scratch + 3 * G;    // longest member's: nothing of the prefix lies past it
    const int mine0 = tid < sp.num_seqs ? __ldg(sc.group_of_seq + tid) : -1;   // in flight meanwhile
    const int len0 = tid < sp.num_seqs ? __ldg(context_lens + tid) : 0;
    for (int g = tid; g < G; g += threads) {
        count[g] = 0;
        first[g] = INT_MAX;
        context[g] = 0;
        prefix[g] = prefix_tokens(sc.group_prefix, g, block_size, max_blocks);
    }
    __syncthreads();
    for (int s = tid; s < sp.num_seqs; s += threads) {
        const int g = s == tid ? mine0 : __ldg(sc.group_of_seq + s);
        if (g >= G) set_error(err, PA_ERR_OUT_OF_RANGE);   // (such a sequence shares nothing)
        if (g < 0 || g >= G) continue;
        atomicAdd(&count[g], 1);
        atomicMin(&first[g], s);
        atomicMax(&context[g], s == tid ? len0 : __ldg(context_lens + s));
    }
    __syncthreads();
    auto prefix_of = [&](int g) { return min(prefix[g], context[g]); };
    auto row_tiles = [&](int g) { return (count[g] * group + kUnitRows - 1) / kUnitRows; };
    auto key_tiles = [&](int g) {
        return count[g] ? (prefix_of(g) + kUnitKeys - 1) / kUnitKeys : 0;
    };
    if (warp == 0) {
        int longest = 0;
        for (int g = lane; g < G; g += 32) longest = max(longest, key_tiles(g));
        longest = __reduce_max_sync(0xffffffffu, longest);
        // lane i tries i + 1 ranges of the longest prefix
        const int range = (longest + lane) / (lane + 1);
        float cost = INFINITY;
        if (longest > 0 && lane < sp.max_splits) {
            int units = 0;
            for (int g = 0; g < G; ++g) units += row_tiles(g) * n_kv * ((key_tiles(g) + range - 1) / range);
            if (lane == 0 || units <= static_cast<int>(gridDim.x))
                cost = ceilf(static_cast<float>(units) / sp.target) * (range + kUnitOverhead);
        }
        float best = cost;
        for (int w = 16; w > 0; w >>= 1) best = fminf(best, __shfl_xor_sync(0xffffffffu, best, w));
        const int pick = __ffs(__ballot_sync(0xffffffffu, cost == best)) - 1;   // fewest ranges of the best
        const int keys = __shfl_sync(0xffffffffu, range, pick);
        if (lane == 0) {
            PrefixUnit u{};
            int left = blockIdx.x;
            for (int g = 0; longest > 0 && g < G; ++g) {
                const int kt = key_tiles(g), n = (kt + keys - 1) / keys, tr = row_tiles(g);
                if (left >= tr * n_kv * n) {
                    left -= tr * n_kv * n;
                    continue;
                }
                u.live = true;
                u.group = g;
                u.row0 = left % tr * kUnitRows;        // row tiles of one K/V range are neighbours
                u.kvh = left / tr % n_kv;
                u.split = left / tr / n_kv;
                u.tile0 = u.split * kt / n;            // (kt <= 2^23, n <= 32)
                u.tiles = (u.split + 1) * kt / n - u.tile0;
                u.rows = count[g] * group;
                u.first_seq = first[g];
                u.prefix = prefix_of(g);
                if (left == 0) sp.splits[g] = n;       // for the merge
                break;
            }
            *unit = u;
        }
    }
    __syncthreads();
    if (!unit->live) return;
    const int m0 = unit->row0 / group;
    const int m1 = (min(unit->rows, unit->row0 + kUnitRows) - 1) / group;
    for (int base = 0, run = 0; base < sp.num_seqs && run <= m1; base += threads) {
        const int s = base + tid;
        const bool mine = s < sp.num_seqs &&
                          (base == 0 ? mine0 : __ldg(sc.group_of_seq + s)) == unit->group;
        const unsigned mask = __ballot_sync(0xffffffffu, mine);
        if (lane == 0) s_warp[warp] = __popc(mask);
        __syncthreads();
        int at = run + __popc(mask & ((1u << lane) - 1u));
        for (int w = 0; w < threads / 32; ++w) {
            if (w < warp) at += s_warp[w];
            run += s_warp[w];
        }
        if (mine && at >= m0 && at <= m1) members[at - m0] = s;
        __syncthreads();
    }
}

}  // namespace pa

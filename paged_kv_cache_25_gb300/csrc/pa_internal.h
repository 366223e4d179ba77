// Host-side internals shared by the library's translation units.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/pa.h"
#include "smem_opt_in.h"

namespace pa {

// Tokens per decode partition for a launch: every partition of a sequence but
// its last covers exactly this many tokens (a multiple of the block size).
int decode_partition_tokens(int64_t seq_groups, int block_size, int max_context_len);

// Records a host-side failure message for pa_last_error_message().
pa_status fail(pa_status st, const char* fmt, ...);
pa_status cuda_fail(cudaError_t e, const char* what);

// Device address of this device's error word (cached per device).
unsigned* device_error_word();

// Encodes a 2-D tiled tensor map over a pool viewed as rows of head_dim
// elements: dims {head_dim, rows}, box {box_x, box_y}, 128-byte swizzle.
// swizzle: 0 none, 64 or 128 (bytes); row_elems = elements per row of the view
pa_status encode_pool_map(CUtensorMap* map, const void* base, pa_dtype dt, int row_elems,
                          uint64_t rows, int box_x, int box_y, int swizzle = 128);

// Encodes a tensor map over `rows` rows of row_bytes bytes (a multiple of 16, at most 2048), box of one
// row, no swizzle: for gathers of rows.
pa_status encode_byte_rows(CUtensorMap* map, const void* base, int row_bytes, uint64_t rows);

// Profiling events around the decode's attention kernels (may be null).
void profile_events(cudaEvent_t* start, cudaEvent_t* stop);

// (of pools other than 4-bit ones)
inline int elem_bytes(pa_dtype d) { return d == PA_F32 ? 4 : (d == PA_FP8_E4M3 ? 1 : 2); }
// bytes of one token's row of one KV head, K or V
inline int row_bytes(const pa_cache_desc& c)
{
    return c.dtype == PA_FP4_E2M1 ? c.head_dim / 2 + c.head_dim / 16 : c.head_dim * elem_bytes(c.dtype);
}

// ---- launchers (defined next to their kernels) ----
cudaError_t launch_cache_write(const void* k, const void* v, void* kc, void* vc,
                               const int64_t* slots, int T, const pa_cache_desc& c,
                               unsigned* err, cudaStream_t s);
cudaError_t launch_cache_write_fp8(const void* k, const void* v, pa_dtype in_dtype, void* kc,
                                   void* vc, const int64_t* slots, int T, const pa_cache_desc& c,
                                   unsigned* err, cudaStream_t s);

cudaError_t launch_cache_write_fp4(const void* k, const void* v, pa_dtype in_dtype, void* kc,
                                   void* vc, const int64_t* slots, int T, const pa_cache_desc& c,
                                   unsigned* err, cudaStream_t s);
cudaError_t launch_gather(void* k_out, void* v_out, pa_dtype out, const void* kc, const void* vc,
                          const int64_t* slots, int T, const pa_cache_desc& c, unsigned* err,
                          cudaStream_t s);

struct RopeArgs {
    void* q_out; const void *q, *k, *v; pa_dtype in_dtype;
    int64_t q_out_stride, q_stride, k_stride, v_stride;   // elements between tokens
    const int32_t* positions; const float* cos_sin; int max_position; int rot_dim; int interleaved;
    void* k_cache; void* v_cache; const int64_t* slots; int num_tokens; int n_q;
    pa_cache_desc cache; unsigned* err;
    // position axes (1: positions is one row); the axis of pair i is bits 2 (i % 16) of axis[i / 16]
    int axes; int64_t axis_stride; uint32_t axis[PA_MAX_ROPE_PAIRS / 16];
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s);

cudaError_t launch_copy_blocks(const void* src_k, const void* src_v, int src_blocks, void* dst_k,
                               void* dst_v, int dst_blocks, const pa_cache_desc& layout,
                               const int32_t* mapping, int pairs, unsigned* err, cudaStream_t s);

// What the scored and shared-prefix kernels take besides a decode's or prefill's
// arguments (device functions: score_mod.cuh).
struct ScoreParams {
    float cap2;                  // C = softcap * log2(e); 0: no cap
    float cap_rate;              // 2 / softcap
    const float* slopes;         // [n_q] distance slopes, or null
    int window;                  // 0: none
    const int32_t* first_key;    // first visible key of every query row, or null
    const int32_t* prefix_lens;  // prefill: keys below it are visible to every row, or null
    // shared-prefix decode: a member sequence's own pass starts after its group's prefix
    const int32_t* group_of_seq; // null: not a shared decode
    const int32_t* group_prefix;
    const int32_t* group_splits; // partials of each group's prefix pass (written by that pass)
    int num_groups;
    // partial slots of an output row: [0, slot0) the prefix pass's, then the partitions'
    int slots, slot0;
};

// The prefix pass of a shared decode: partials of every member row and prefix range.
struct PrefixPass {
    int num_seqs;
    float* ml;          // [B][n_q][slots][2]
    float* acc;         // [B][n_q][slots][d]
    int32_t* splits;    // [num_groups], written by the pass
    unsigned* ticket;   // work counter of the decode kernel that follows, cleared by the pass
    int max_splits;     // ranges a prefix may be cut into (at most 32, at most slot0)
    int target;         // thread blocks that run at once
};

struct DecodeArgs {
    void* out; pa_dtype out_dtype; const void* q;
    const void* k_cache; const void* v_cache; pa_cache_desc cache;
    const int32_t* block_tables; int max_blocks;
    const int32_t* context_lens; int num_seqs; int n_q; float scale;
    int q_per_seq;     // query rows per sequence (1 for decode; k+1 to verify k drafts)
    float* ws_ml;      // [B][q_per_seq][n_q][J][2] (m, l) or null
    float* ws_acc;     // [B][q_per_seq][n_q][J][d] or null
    int part_tokens;   // tokens per partition
    int max_parts;     // J: partitions of the longest possible sequence
    unsigned* ticket;  // work counter in the workspace's control area; null: units are
                       // dealt round robin (unit blockIdx.x + k * gridDim.x), no counter
    unsigned* err;
    const ScoreParams* score;   // scored or shared-prefix decode (host memory); else null
};
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t s);
// attention kernel of a scored or shared-prefix call (decode_scored.cu)
cudaError_t launch_decode_scored(const DecodeArgs& a, cudaStream_t s, float scale_log2);
cudaError_t launch_decode_wide(const DecodeArgs& a, cudaStream_t s, float scale_log2);   // (caps above kNearCap)
cudaError_t launch_decode_scored_simt(const DecodeArgs& a, cudaStream_t s, float scale_log2);
// a call on an FP4 pool, its merge included (decode_fp4.cu), and what its workspace holds: for each of its blocks
// (at most f4_grid and f4_granules; fewer where there is no room, but room for half of f4_grid is asked
// for) the head of its run of f4_unit_rows rows and, as far as there are so many such rows, the tail
constexpr int kF4GranuleTokens = 128, kF4Sms = 152;
inline int f4_unit_rows(int rows_kv) { return rows_kv <= 4 ? 4 : (rows_kv <= 8 ? 8 : 16); }
inline int64_t f4_granules(int num_seqs, int nq, int group, int n_kv, int max_ctx)
{
    const int ru = f4_unit_rows(group * nq);
    return static_cast<int64_t>(num_seqs) * n_kv * ((group * nq + ru - 1) / ru) *
           ((max_ctx + kF4GranuleTokens - 1) / kF4GranuleTokens);
}
inline int f4_grid(int rows_kv, int D)      // blocks of the GPU
{
    return kF4Sms * (f4_unit_rows(rows_kv) == 16 ? (D == 64 ? 3 : 2) : 4);
}
inline size_t f4_workspace_bytes(int num_seqs, int nq, int group, int n_kv, int D, int max_ctx, int64_t blocks)
{
    if (max_ctx <= kF4GranuleTokens) return 0;    // (no shared pieces)
    const int ru = f4_unit_rows(group * nq);
    const int64_t most = f4_granules(num_seqs, nq, group, n_kv, max_ctx);
    blocks = most < blocks ? most : blocks;
    const int64_t rows = static_cast<int64_t>(num_seqs) * n_kv * ((group * nq + ru - 1) / ru);
    return blocks * 16 + static_cast<size_t>(blocks + (rows < blocks ? rows : blocks)) * ru * (D + 2) * sizeof(float);
}
cudaError_t launch_decode_fp4(const DecodeArgs& a, void* workspace, size_t workspace_bytes, cudaStream_t s);
// prefix pass of a shared-prefix call (prefix_pass.cu)
cudaError_t launch_prefix_pass(const DecodeArgs& a, const PrefixPass& pass, cudaStream_t s);
// attention kernel of a call with q_per_seq > 1 (decode_verify.cu)
cudaError_t launch_decode_mq(const DecodeArgs& a, cudaStream_t s, float scale_log2);

struct PrefillArgs {
    void* out; pa_dtype out_dtype; const void* q;
    const void* k_cache; const void* v_cache; pa_cache_desc cache;
    const int32_t* block_tables; int max_blocks;
    const int32_t* q_start; const int32_t* context_lens;
    int num_reqs; int max_q; int n_q; float scale;
    unsigned* err;
    const ScoreParams* score;   // scored prefill (host memory); else null
};
cudaError_t launch_prefill_tc(const PrefillArgs& a, cudaStream_t s);
cudaError_t launch_prefill_fp4(const PrefillArgs& a, cudaStream_t s);
cudaError_t launch_prefill_scored(const PrefillArgs& a, cudaStream_t s);
cudaError_t launch_prefill_bias(const PrefillArgs& a, cudaStream_t s);   // (its forms with a bias)
cudaError_t launch_prefill_wide(const PrefillArgs& a, cudaStream_t s);   // (its caps above kNearCap)
cudaError_t launch_prefill_split(const PrefillArgs& a, cudaStream_t s);
cudaError_t launch_prefill_split_bias(const PrefillArgs& a, cudaStream_t s);

}  // namespace pa

// Chunked prefill over FP4 pools (pa_prefill_chunk): the tcgen05 prefill kernel, whose
// converter warps widen 4-bit rows into its rings (prefill_fp4.cuh).  Calls of few row blocks over long contexts split
// their key tiles over clusters as scored calls do, by the same rule (prefill_splits): one chunk of 512 rows after
// 3584 tokens of Llama-3-8B's heads, 64 blocks: 45 us in clusters of two, 67 not split, 132 in clusters of eight; four such
// chunks, 256 blocks: 130 not split, as they run, 470 in clusters of eight.
#include "prefill_tc.cuh"

namespace pa {

cudaError_t launch_prefill_fp4(const PrefillArgs& a, cudaStream_t s)
{
    const float sl2 = a.scale * kLog2e;
    const ScoreParams plain{};
    PrefillArgs split = a;
    split.score = &plain;
    if (prefill_splits(split) > 1)
        return a.cache.act_dtype == PA_BF16
                   ? run_prefill_tc_dt<__half, __nv_bfloat16, true, kPfScored | kPfSplit, true>(split, s, sl2)
                   : run_prefill_tc_dt<__half, __half, true, kPfScored | kPfSplit, true>(split, s, sl2);
    return a.cache.act_dtype == PA_BF16 ? run_prefill_tc_dt<__half, __nv_bfloat16, true, 0, true>(a, s, sl2)
                                        : run_prefill_tc_dt<__half, __half, true, 0, true>(a, s, sl2);
}

}  // namespace pa

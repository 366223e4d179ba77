// Scored chunked prefill of few rows over a long context, its key tiles split over a
// cluster (prefill_splits in prefill_tc.cuh), in a translation unit of its own to compile
// in parallel.  Two chunks of 155 rows, 2 KV heads, 5,800 tokens, FP8, cap and bias: 41 us
// against 242 with a block for each row block (12 blocks of 46 key tiles).
#include "prefill_tc.cuh"

namespace pa {

cudaError_t launch_prefill_split(const PrefillArgs& a, cudaStream_t s)
{
    if (a.score->slopes) return launch_prefill_split_bias(a, s);
    return a.score->cap2 > 0.f ? run_prefill_any<kPfScored | kPfCap | kPfSplit>(a, s)
                               : run_prefill_any<kPfScored | kPfSplit>(a, s);
}

}  // namespace pa

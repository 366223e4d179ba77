// Scored chunked prefill of few rows over a long context, its key tiles split over a
// cluster (prefill_splits in prefill_tc.cuh), in a translation unit of its own to compile
// in parallel.  Two chunks of 149 and 160 rows after 2,617 and 5,852 tokens, 8 heads on 2 of
// 64 elements, FP8, cap and bias: 41 us against 242 with a block for each row block (12 blocks
// of up to 47 key tiles), floor 1.5; two of 155 after 5,645 42 us, of 128 elements 54.5.
#include "prefill_tc.cuh"

namespace pa {

cudaError_t launch_prefill_split(const PrefillArgs& a, cudaStream_t s)
{
    if (a.score->slopes) return launch_prefill_split_bias(a, s);
    return a.score->cap2 > 0.f ? run_prefill_any<kPfScored | kPfCap | kPfSplit>(a, s)
                               : run_prefill_any<kPfScored | kPfSplit>(a, s);
}

}  // namespace pa

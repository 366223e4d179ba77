// Scored chunked prefill with a distance bias (see prefill_scored.cu), in a
// translation unit of its own to compile in parallel.
#include "prefill_tc.cuh"

namespace pa {

cudaError_t launch_prefill_bias(const PrefillArgs& a, cudaStream_t s)
{
    return a.score->cap2 > 0.f ? run_prefill_any<kPfScored | kPfCap | kPfBias>(a, s)
                               : run_prefill_any<kPfScored | kPfBias>(a, s);
}

}  // namespace pa

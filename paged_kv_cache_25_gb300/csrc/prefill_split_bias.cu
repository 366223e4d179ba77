// As prefill_split.cu, with a distance bias.
#include "prefill_tc.cuh"

namespace pa {

cudaError_t launch_prefill_split_bias(const PrefillArgs& a, cudaStream_t s)
{
    return a.score->cap2 > 0.f ? run_prefill_any<kPfScored | kPfCap | kPfBias | kPfSplit>(a, s)
                               : run_prefill_any<kPfScored | kPfBias | kPfSplit>(a, s);
}

}  // namespace pa

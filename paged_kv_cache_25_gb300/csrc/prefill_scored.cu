// Scored chunked prefill: the kernel of prefill_tc.cuh with masks of every row's
// own, and with a cap on the scores or without.  (Forms with a distance bias:
// prefill_scored_bias.cu; with caps above kNearCap: prefill_wide.cu; split over a cluster: prefill_split.cu, prefill_split_bias.cu.)
#include "prefill_tc.cuh"

namespace pa {

cudaError_t launch_prefill_scored(const PrefillArgs& a, cudaStream_t s)
{
    if (a.score->cap2 > kNearCap) return launch_prefill_wide(a, s);
    if (prefill_splits(a) > 1) return launch_prefill_split(a, s);
    if (a.score->slopes) return launch_prefill_bias(a, s);
    return a.score->cap2 > 0.f ? run_prefill_any<kPfScored | kPfCap>(a, s) : run_prefill_any<kPfScored>(a, s);
}

}  // namespace pa

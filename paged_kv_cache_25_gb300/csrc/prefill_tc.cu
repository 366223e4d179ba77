// Plain causal chunked prefill: the kernel of prefill_tc.cuh without modifications.
#include "prefill_tc.cuh"

namespace pa {

cudaError_t launch_prefill_tc(const PrefillArgs& a, cudaStream_t s)
{
    return run_prefill_any<0>(a, s);
}

}  // namespace pa

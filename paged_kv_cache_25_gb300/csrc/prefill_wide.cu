// Scored chunked prefill with a cap above kNearCap (score_mod.cuh), with a distance bias or
// without, in instantiations of its own: as a run-time branch of the capped kernels the wide
// form cost caps in use 2 - 8 % (mixed step's four chunks, bf16 250.5 -> 255.9 us, FP8 220.4 ->
// 237.8, bf16 with a bias 453 -> 486).  No model in use caps that high: one form serves all of
// them, also few rows over a long context.
#include "prefill_tc.cuh"

namespace pa {

cudaError_t launch_prefill_wide(const PrefillArgs& a, cudaStream_t s)
{
    return run_prefill_any<kPfScored | kPfCap | kPfBias | kPfWide>(a, s);
}

}  // namespace pa

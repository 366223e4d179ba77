// Scored decode and the sequences' own part of the shared-prefix decode: the
// tensor-core decode kernel with score modifications and a first key per sequence
// (SC, see decode_mma.cuh).  Kept in its own translation unit, so the plain decode
// kernels carry none of it and compile in parallel.
#include "decode_mma.cuh"

namespace pa {

cudaError_t launch_decode_scored(const DecodeArgs& a, cudaStream_t s, float scale_log2)
{
    if (a.score->cap2 > kNearCap) return launch_decode_wide(a, s, scale_log2);
    return a.q_per_seq > 1 ? run_mma_any<true, true>(a, s, scale_log2)
                           : run_mma_any<false, true>(a, s, scale_log2);
}

}  // namespace pa

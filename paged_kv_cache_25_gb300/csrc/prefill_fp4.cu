// Chunked prefill over FP4 pools (pa_prefill_chunk): the tcgen05 prefill kernel, whose
// converter warps widen 4-bit rows into its rings (prefill_tc.cuh).
#include "prefill_tc.cuh"

namespace pa {

cudaError_t launch_prefill_fp4(const PrefillArgs& a, cudaStream_t s)
{
    const float sl2 = a.scale * kLog2e;
    return a.cache.act_dtype == PA_BF16 ? run_prefill_tc_dt<__half, __nv_bfloat16, true, 0, true>(a, s, sl2)
                                        : run_prefill_tc_dt<__half, __half, true, 0, true>(a, s, sl2);
}

}  // namespace pa

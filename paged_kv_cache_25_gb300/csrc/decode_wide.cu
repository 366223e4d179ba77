// Scored decode with a cap above kNearCap (score_mod.cuh): every score then pays for both
// sides of the wide form, so such calls have instantiations of their own.  As a run-time
// branch of the scored kernels the form cost the others up to 2.7 % (256 sequences of four rows,
// FP8 pool: 342.3 -> 351.3 us).  No model in use caps that high: one form, 8-row units of any
// number of query rows, serves all of them.
#include "decode_mma.cuh"

namespace pa {

template <typename T, typename QT, bool F8>
static cudaError_t run_wide(const DecodeArgs& a, cudaStream_t s, float sl2)
{
    const int D = a.cache.head_dim, BS = a.cache.block_size;
    if (D == 64 && BS == 16) return run_mma<T, QT, 64, 16, F8, true, 8, true, true>(a, s, sl2);
    if (D == 64 && BS == 32) return run_mma<T, QT, 64, 32, F8, true, 8, true, true>(a, s, sl2);
    if (D == 128 && BS == 16) return run_mma<T, QT, 128, 16, F8, true, 8, true, true>(a, s, sl2);
    if (D == 128 && BS == 32) return run_mma<T, QT, 128, 32, F8, true, 8, true, true>(a, s, sl2);
    return cudaErrorNotSupported;
}

cudaError_t launch_decode_wide(const DecodeArgs& a, cudaStream_t s, float sl2)
{
    switch (a.cache.dtype) {
        case PA_BF16: return run_wide<__nv_bfloat16, __nv_bfloat16, false>(a, s, sl2);
        case PA_F16: return run_wide<__half, __half, false>(a, s, sl2);
        case PA_FP8_E4M3:
            return a.cache.act_dtype == PA_BF16 ? run_wide<__half, __nv_bfloat16, true>(a, s, sl2)
                                                : run_wide<__half, __half, true>(a, s, sl2);
        default: return cudaErrorNotSupported;
    }
}

}  // namespace pa

// Cache write into 4-bit pools ("Life of a prompt", "Back to the queue, and into vLLM
// proper": every new token's K and V vector is appended into the next free slot): rows of
// fp32, fp16 or bf16 become 4-bit rows (format and rounding: fp4.cuh).
//
// One thread quantises one group of 16 elements of a row; the groups of a row, then
// the tokens of a 16-token tile, then K and V are neighbours, so that a prompt's chunk is read in
// whole rows and written as one run of bytes a (block, head).
//
// Bound: instructions (a group's quotients and conversions, fp4.cuh) and HBM: 8192 tokens of 8 heads of
// 128 bf16 elements 15.4 us, HBM floor 6.3.
#include "fp4.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

template <typename T, int D>
__global__ void __launch_bounds__(256)
cache_write_fp4_kernel(const T* __restrict__ k, const T* __restrict__ v, uint8_t* __restrict__ kc,
                       uint8_t* __restrict__ vc, const int64_t* __restrict__ slots, int T_, int n_kv,
                       int block_size, int64_t num_slots, float k_scale, float v_scale, unsigned* err)
{
    constexpr int kGroups = D / kFp4Group;
    constexpr int kTok = 256 / (2 * kGroups);      // tokens of a tile
    allow_dependent_launch();   // the decode launched next waits for this grid before it reads the pool
    const int tid = threadIdx.x;
    const int c = tid % kGroups, t = blockIdx.x * kTok + tid / kGroups % kTok;
    const bool is_v = tid / (kGroups * kTok) != 0;
    const int h = blockIdx.y;
    if (t >= T_) return;
    const int64_t slot = __ldg(slots + t);
    if (slot < 0) return;                          // padding token
    if (slot >= num_slots) {
        set_error(err, PA_ERR_OUT_OF_RANGE);
        return;
    }
    const T* src = (is_v ? v : k) + (static_cast<int64_t>(t) * n_kv + h) * D + c * kFp4Group;
    float x[kFp4Group];
    constexpr int N = 16 / static_cast<int>(sizeof(T));
#pragma unroll
    for (int i = 0; i < kFp4Group; i += N) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(src + i));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (sizeof(T) == 4) {
                x[i + e] = __uint_as_float(w[e]);
            } else {
                const float2 f = Cvt<T>::unpack(w[e]);
                x[i + 2 * e] = f.x;
                x[i + 2 * e + 1] = f.y;
            }
        }
    }
    const float scale = is_v ? v_scale : k_scale;
    uint32_t s;
    const uint2 codes = fp4_quantise(x, scale, __fmul_rn(6.f, scale), s);
    const int64_t b = slot / block_size, o = slot - b * block_size;
    fp4_store<D>((is_v ? vc : kc) + ((b * n_kv + h) * block_size + o) * fp4_row_bytes(D), c, codes, s);
}

cudaError_t launch_cache_write_fp4(const void* k, const void* v, pa_dtype in_dtype, void* kc, void* vc,
                                   const int64_t* slots, int T, const pa_cache_desc& c, unsigned* err,
                                   cudaStream_t s)
{
    if (T == 0) return cudaSuccess;
    const int64_t ns = static_cast<int64_t>(c.num_blocks) * c.block_size;
    if (c.head_dim != 64 && c.head_dim != 128) return cudaErrorInvalidValue;
    const int tok = 256 / (2 * c.head_dim / kFp4Group);
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(T) + tok - 1) / tok), static_cast<unsigned>(c.n_kv_heads));
    auto run = [&](auto zero) {
        using TI = decltype(zero);
        auto go = [&](auto kern) {
            kern<<<grid, 256, 0, s>>>(static_cast<const TI*>(k), static_cast<const TI*>(v), static_cast<uint8_t*>(kc),
                                      static_cast<uint8_t*>(vc), slots, T, c.n_kv_heads, c.block_size, ns, c.k_scale,
                                      c.v_scale, err);
        };
        if (c.head_dim == 128) go(cache_write_fp4_kernel<TI, 128>);
        else go(cache_write_fp4_kernel<TI, 64>);
    };
    if (in_dtype == PA_BF16) run(__nv_bfloat16{});
    else if (in_dtype == PA_F16) run(__half{});
    else if (in_dtype == PA_F32) run(0.f);
    else return cudaErrorInvalidValue;
    return cudaGetLastError();
}

}  // namespace pa

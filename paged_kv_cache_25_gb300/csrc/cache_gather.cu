// Rows of slots read back out of a paged pool as values, the inverse of the cache write:
// token t's K and V rows, of the slot that it names, become contiguous rows of fp32, fp16 or
// bf16.
//
// Bound: HBM (each row is read once and written once) or launch latency.  One thread makes
// 16 elements of a row.  V of an FP8 pool lies transposed in 16-token pieces, so a token's
// 16 codes are 16 single bytes, 16 apart; neighbouring threads take neighbouring tokens there, whose
// bytes share the same sectors.
// 32,768 tokens of 8 heads of 128 elements out of an FP4 pool into bf16: 32.6 us, 5.3 TB/s (0.78 of the copy
// rate), issue 60 %; out of an FP8 pool 47.7, by V's single bytes, of a bf16 pool 42.5 (floors 25, 30, 40).
#include <algorithm>

#include "fp4.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kGatherThreads = 256;
constexpr int kGatherElems = 16;
constexpr int kGatherTok = 16;      // tokens of a tile

struct GatherParams {
    void *k_out, *v_out;
    const uint8_t *k_cache, *v_cache;
    const int64_t* slots;
    int64_t num_slots;
    int num_tokens, n_kv, block_size;
    float k_scale, v_scale;
    unsigned* err;
};

// Sixteen values to p, rounded once.
template <typename TO>
__device__ __forceinline__ void store16(TO* p, const float (&x)[kGatherElems])
{
    constexpr int kWords = kGatherElems * static_cast<int>(sizeof(TO)) / 4;
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        if constexpr (sizeof(TO) == 4) w[i] = __float_as_uint(x[i]);
        else w[i] = Cvt<TO>::pack(x[2 * i], x[2 * i + 1]);
    }
#pragma unroll
    for (int i = 0; i < kWords; i += 4)
        __stcs(reinterpret_cast<uint4*>(p) + i / 4, make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]));
}

__device__ __forceinline__ void widen_e4m3(uint32_t w, float* x)   // four codes
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t u = e4m3x2_to_h2(w >> (16 * h));
        const float2 f = Cvt<__half>::unpack(u);
        x[2 * h] = f.x;
        x[2 * h + 1] = f.y;
    }
}

// DT: the pool's type.  A tile is 16 tokens of one head; its items are (K or V, piece of 16
// elements, token), pieces fastest, but for V of FP8 pools the tokens.
template <pa_dtype DT, typename TO, int D>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const GatherParams p)
{
    constexpr int kPieces = D / kGatherElems, kItems = 2 * kPieces * kGatherTok;
    const int h = blockIdx.y;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kGatherTok;
    grid_dependency_wait();      // a programmatic dependent of the write before it
    allow_dependent_launch();
#pragma unroll
    for (int item = threadIdx.x; item < kItems; item += kGatherThreads) {
        const bool is_v = item >= kItems / 2;
        const int i = is_v ? item - kItems / 2 : item;
        const bool by_token = DT == PA_FP8_E4M3 && is_v;
        const int c = by_token ? i / kGatherTok : i % kPieces;
        const int64_t t = t0 + (by_token ? i % kGatherTok : i / kPieces);
        if (t >= p.num_tokens) continue;
        const int64_t slot = __ldg(p.slots + t);
        if (slot < 0) continue;                    // padding: its output row stays as it is
        if (slot >= p.num_slots) {
            set_error(p.err, PA_ERR_OUT_OF_RANGE);
            continue;
        }
        const unsigned sl = static_cast<unsigned>(slot), bs = p.block_size, blk = sl / bs, o = sl % bs;
        const int64_t head = static_cast<int64_t>(blk) * p.n_kv + h;
        const uint8_t* pool = is_v ? p.v_cache : p.k_cache;
        const float scale = is_v ? p.v_scale : p.k_scale;
        float x[kGatherElems];
        if constexpr (DT == PA_FP4_E2M1) {
            const uint8_t* row = pool + (head * bs + o) * fp4_row_bytes(D);
            uint32_t w[2];
            if constexpr (D == 128) {
                const uint2 u = __ldg(reinterpret_cast<const uint2*>(row + c * 8));
                w[0] = u.x;
                w[1] = u.y;
            } else {
                w[0] = __ldg(reinterpret_cast<const uint32_t*>(row + c * 8));
                w[1] = __ldg(reinterpret_cast<const uint32_t*>(row + c * 8 + 4));
            }
            const float s = e4m3_to_float(__ldg(row + D / 2 + c));
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t u[4];
                fp4x8_to_h2x4(w[q], u[0], u[1], u[2], u[3]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = Cvt<__half>::unpack(u[e]);
                    x[8 * q + 2 * e] = f.x * s * scale;             // (f * s is exact)
                    x[8 * q + 2 * e + 1] = f.y * s * scale;
                }
            }
        } else if constexpr (DT == PA_FP8_E4M3) {
            uint32_t w[4];
            if (!is_v) {
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(pool + (head * bs + o) * D) + c);
                w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
            } else {
                const uint8_t* piece = pool + (head * (bs / 16) + o / 16) * (D * 16) + c * 256 + o % 16;
                uint8_t b[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) b[e] = __ldg(piece + e * 16);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = b[4 * e] | (b[4 * e + 1] << 8) | (b[4 * e + 2] << 16) | (static_cast<uint32_t>(b[4 * e + 3]) << 24);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) widen_e4m3(w[e], x + 4 * e);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] *= scale;
        } else {
            using TI = std::conditional_t<DT == PA_F32, float, std::conditional_t<DT == PA_F16, __half, __nv_bfloat16>>;
            const uint4* row = reinterpret_cast<const uint4*>(reinterpret_cast<const TI*>(pool) + (head * bs + o) * D +
                                                             c * kGatherElems);
            constexpr int N = 16 / static_cast<int>(sizeof(TI));
#pragma unroll
            for (int q = 0; q < kGatherElems / N; ++q) {
                const uint4 u = __ldcs(row + q);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (sizeof(TI) == 4) {
                        x[q * N + e] = __uint_as_float(w[e]);
                    } else {
                        const float2 f = Cvt<TI>::unpack(w[e]);
                        x[q * N + 2 * e] = f.x;
                        x[q * N + 2 * e + 1] = f.y;
                    }
                }
            }
        }
        store16(static_cast<TO*>(is_v ? p.v_out : p.k_out) + (t * p.n_kv + h) * D + c * kGatherElems, x);
    }
}

template <pa_dtype DT, typename TO>
static cudaError_t run_gather(const GatherParams& p, int d, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(p.num_tokens) + kGatherTok - 1) / kGatherTok),
                       static_cast<unsigned>(p.n_kv));
    cfg.blockDim = dim3(kGatherThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (d == 64) return cudaLaunchKernelEx(&cfg, gather_kernel<DT, TO, 64>, p);
    if (d == 128) return cudaLaunchKernelEx(&cfg, gather_kernel<DT, TO, 128>, p);
    if constexpr (DT != PA_FP4_E2M1 && DT != PA_FP8_E4M3) {
        if (d == 32) return cudaLaunchKernelEx(&cfg, gather_kernel<DT, TO, 32>, p);
        if (d == 96) return cudaLaunchKernelEx(&cfg, gather_kernel<DT, TO, 96>, p);
        if (d == 256) return cudaLaunchKernelEx(&cfg, gather_kernel<DT, TO, 256>, p);
    }
    return cudaErrorInvalidValue;
}

template <pa_dtype DT>
static cudaError_t run_gather_to(const GatherParams& p, pa_dtype out, int d, cudaStream_t s)
{
    switch (out) {
        case PA_F32: return run_gather<DT, float>(p, d, s);
        case PA_F16: return run_gather<DT, __half>(p, d, s);
        case PA_BF16: return run_gather<DT, __nv_bfloat16>(p, d, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_gather(void* k_out, void* v_out, pa_dtype out, const void* kc, const void* vc,
                          const int64_t* slots, int T, const pa_cache_desc& c, unsigned* err, cudaStream_t s)
{
    GatherParams p{};
    p.k_out = k_out; p.v_out = v_out;
    p.k_cache = static_cast<const uint8_t*>(kc); p.v_cache = static_cast<const uint8_t*>(vc);
    p.slots = slots; p.num_slots = static_cast<int64_t>(c.num_blocks) * c.block_size;
    p.num_tokens = T; p.n_kv = c.n_kv_heads; p.block_size = c.block_size;
    p.k_scale = c.k_scale; p.v_scale = c.v_scale; p.err = err;
    switch (c.dtype) {
        case PA_F32: return run_gather_to<PA_F32>(p, out, c.head_dim, s);
        case PA_F16: return run_gather_to<PA_F16>(p, out, c.head_dim, s);
        case PA_BF16: return run_gather_to<PA_BF16>(p, out, c.head_dim, s);
        case PA_FP8_E4M3: return run_gather_to<PA_FP8_E4M3>(p, out, c.head_dim, s);
        case PA_FP4_E2M1: return run_gather_to<PA_FP4_E2M1>(p, out, c.head_dim, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa

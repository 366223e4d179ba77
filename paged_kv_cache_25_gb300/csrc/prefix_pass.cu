// Prefix pass of the shared-prefix decode: attention of every member of a prefix
// group over the group's common prefix, read once for all of them.
//
// Mathematics: softmax partials over disjoint key sets merge exactly.  For the rows of
// one (sequence, head) the pass gives (m, l, O) = (max z, sum 2^(z - m), sum 2^(z - m) v)
// per range of the prefix, the decode kernel the same over the sequence's own keys, and
// the merge out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
//
// The members' rows against one KV head are a dense product (members * heads per KV
// head rows, prefix keys), so it runs on the fifth-generation tensor cores with the
// chunked prefill's kernel: 256 rows a thread block, 128-key tiles, the prefix cut into
// ranges so that the blocks fill the GPU (prefix_plan.cuh).
#include "prefill_tc.cuh"

namespace pa {

template <typename T, typename QT, int D, int BS, bool F8>
static cudaError_t run_prefix(const DecodeArgs& a, const PrefixPass& pass, cudaStream_t s, float sl2)
{
    constexpr bool kBq = std::is_same<QT, __nv_bfloat16>::value;
    using Ly = PfLayout<T, D, F8, kBq>;
    auto kern = prefill_tc_kernel<T, QT, D, BS, F8, kPfShared>;
    static SmemOptIn opt_in;
    const cudaError_t attr_err = opt_in(reinterpret_cast<const void*>(kern), static_cast<int>(Ly::kDynBytes));
    if (attr_err != cudaSuccess) return attr_err;
    CUtensorMap kmap{}, vmap{};
    const cudaError_t map_err = prefill_maps<T, D, BS, F8, kBq>(a.cache, a.k_cache, a.v_cache, &kmap, &vmap);
    if (map_err != cudaSuccess) return map_err;
    const int n_kv = a.cache.n_kv_heads, group = a.n_q / n_kv;
    // one range of every prefix always fits the grid: the groups' row tiles are at most this many
    const int64_t rows = static_cast<int64_t>(a.num_seqs) * group;
    const int64_t row_tiles = rows / kUnitRows + (a.score->num_groups < a.num_seqs ? a.score->num_groups : a.num_seqs);
    const int64_t units = row_tiles * n_kv;
    const unsigned grid = static_cast<unsigned>(units > pass.target ? units : pass.target);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(PfWarps<F8, D, kBq>::kThreads);
    cfg.dynamicSmemBytes = Ly::kDynBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(
        &cfg, kern, kmap, vmap, static_cast<const uint8_t*>(a.k_cache), static_cast<const uint8_t*>(a.v_cache),
        static_cast<void*>(nullptr), PA_F32, static_cast<const QT*>(a.q), a.block_tables, a.max_blocks,
        static_cast<const int32_t*>(nullptr), a.context_lens, 0, a.n_q, n_kv, group, a.cache.num_blocks,
        F8 ? sl2 * a.cache.k_scale : sl2, F8 ? a.cache.v_scale : 1.f, a.err, *a.score, pass);
}

template <typename T, typename QT, bool F8>
static cudaError_t run_prefix_dt(const DecodeArgs& a, const PrefixPass& p, cudaStream_t s, float sl2)
{
    const int D = a.cache.head_dim, BS = a.cache.block_size;
    if (D == 64 && BS == 16) return run_prefix<T, QT, 64, 16, F8>(a, p, s, sl2);
    if (D == 64 && BS == 32) return run_prefix<T, QT, 64, 32, F8>(a, p, s, sl2);
    if (D == 128 && BS == 16) return run_prefix<T, QT, 128, 16, F8>(a, p, s, sl2);
    if (D == 128 && BS == 32) return run_prefix<T, QT, 128, 32, F8>(a, p, s, sl2);
    return cudaErrorInvalidValue;
}

cudaError_t launch_prefix_pass(const DecodeArgs& a, const PrefixPass& pass, cudaStream_t s)
{
    const float sl2 = a.scale * kLog2e;
    PrefixPass p = pass;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&p.target, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (a.cache.dtype == PA_BF16) return run_prefix_dt<__nv_bfloat16, __nv_bfloat16, false>(a, p, s, sl2);
    if (a.cache.dtype == PA_F16) return run_prefix_dt<__half, __half, false>(a, p, s, sl2);
    if (a.cache.dtype == PA_FP8_E4M3)
        return a.cache.act_dtype == PA_BF16 ? run_prefix_dt<__half, __nv_bfloat16, true>(a, p, s, sl2)
                                            : run_prefix_dt<__half, __half, true>(a, p, s, sl2);
    return cudaErrorInvalidValue;
}

}  // namespace pa

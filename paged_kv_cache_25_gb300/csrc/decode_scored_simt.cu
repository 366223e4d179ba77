// Scored decode on the CUDA cores: fp32 pools, and 16-bit pools of the head dims that the
// tensor-core kernel does not take.  A thread block serves HG query heads of one KV head over
// one partition of a sequence, whose keys start at its first visible block; its eight warps
// take kTok keys at a time in turn.
//
// Mathematics: one pass with the running maximum m and sum l of the softmax.  A lane holds
// D / 32 elements of every row, so the HG * kTok dot products of a step are sums over the
// lanes.  They are added up by halves: at each step a lane hands the half of its partial
// sums that its partner keeps over and keeps the other half, so N sums take about N shuffles
// (31 for 32) instead of 5 N and end up spread over the lanes, which then work out cap,
// bias, mask and exponential of one (head, key) each.  The warps merge (m, l, O) in
// shared memory at the end.
//
// Bound: HBM for large batches, latency for small ones.  fp32, 128 elements, 32 heads on 8:
// 256 sequences of 64 - 1000 tokens 173 us (floor 166), 97 of 112 with a cap 17.9 (13.7).  With
// a warp for each (partition, head), every sum in every lane: 747 and 88.7; sums spread: 318
// and 35.7; eight warps a partition, one head each: 335 and 33.1 (64 sequences of 500 - 1500
// tokens, 8 heads on 8 of 64 elements: 298, 131, 50).
#include "decode_mma.cuh"

namespace pa {

constexpr int kSimtWarps = 8;

// The sum over the warp of every lane's v[u], u = lane / (32 / N).
template <int N>
__device__ __forceinline__ float sum_spread(float (&v)[N], int lane)
{
    int w = 16;
#pragma unroll
    for (int n = N / 2; n >= 1; n /= 2, w /= 2) {
        const bool upper = lane & w;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
        }
    }
#pragma unroll
    for (; w > 0; w /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], w);
    return v[0];
}

template <typename T, int DPL, int HG>
__global__ void __launch_bounds__(kSimtWarps * 32)
decode_scored_simt_kernel(void* __restrict__ out, pa_dtype out_dtype, const T* __restrict__ q,
                          const T* __restrict__ kc, const T* __restrict__ vc,
                          const int32_t* __restrict__ block_tables, int max_blocks,
                          const int32_t* __restrict__ context_lens, int n_q, int n_kv, int group,
                          int num_blocks, int block_size, float scale_log2, float* __restrict__ ws_ml,
                          float* __restrict__ ws_acc, int part_tokens, int max_parts, unsigned* err,
                          const __grid_constant__ ScoreParams sc)
{
    constexpr int D = DPL * 32;
    constexpr int V = DPL % 4 == 0 ? 4 : (DPL % 2 == 0 ? 2 : 1);   // elements of one load
    // keys of a step, a divisor of the block sizes: as many as the registers hold
    constexpr int kTok = DPL <= 4 ? 8 : 4;
    constexpr int kSpread = 32 / (HG * kTok);                      // lanes that hold one score
    static_assert(HG * kTok <= 32, "a lane holds one score");
    struct alignas(sizeof(T) * V) Run {
        T x[V];
    };
    struct alignas(4 * V) FloatRun {
        float x[V];
    };
    __shared__ float s_ml[kSimtWarps][HG][2];
    __shared__ __align__(16) float s_acc[kSimtWarps][HG][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int j = blockIdx.x;
    const int chunks = (group + HG - 1) / HG;
    const int kvh = blockIdx.y / chunks;
    const int g0 = blockIdx.y % chunks * HG;            // the block's first head of the KV head's
    const int live = min(HG, group - g0);               // its heads (the others repeat the last one)
    const int s = blockIdx.z;
    const int L = __ldg(context_lens + s);
    const int lo = first_visible(sc, s, L, 1, block_size, max_blocks, err);
    const int base = lo / block_size * block_size;
    const int tok0 = base + j * part_tokens;
    if (tok0 >= L) return;
    const int tok1 = min(L, tok0 + part_tokens);
    const int nparts = min((L - base + part_tokens - 1) / part_tokens, max_parts);
    const int first = max(lo, row_first(sc, s, 1, 0, L - 1));   // (past the row's position: it sees none)
    const int64_t row_q = static_cast<int64_t>(s) * n_q + kvh * group + g0;   // first head's row of q, out

    // element i of a lane's part of a row
    auto at = [&](int i) { return (i / V * 32 + lane) * V + i % V; };
    auto fetch = [&](const T* row, float (&x)[DPL]) {
#pragma unroll
        for (int c = 0; c < DPL / V; ++c) {
            const Run r = *reinterpret_cast<const Run*>(row + at(c * V));
#pragma unroll
            for (int e = 0; e < V; ++e) x[c * V + e] = Cvt<T>::to_f(r.x[e]);
        }
    };
    float qv[HG][DPL], acc[HG][DPL];
#pragma unroll
    for (int g = 0; g < HG; ++g) {
        fetch(q + (row_q + min(g, live - 1)) * D, qv[g]);
#pragma unroll
        for (int i = 0; i < DPL; ++i) acc[g][i] = 0.f;
    }
    // this lane's score: head my_g of the block, key my_u of the step
    const int my_g = lane / (kSpread * kTok), my_u = lane / kSpread % kTok;
    const float slope = sc.slopes ? __ldg(sc.slopes + kvh * group + g0 + min(my_g, live - 1)) * kLog2e : 0.f;
    float m_run = -INFINITY, l_run = 0.f;   // of head my_g; l_run: of this lane's keys
    const int32_t* table = block_tables + static_cast<int64_t>(s) * max_blocks;
    auto block_of = [&](int p) {
        const int lb = p / block_size;
        return lb < max_blocks ? __ldg(table + lb) : -1;
    };
    constexpr int kStep = kSimtWarps * kTok;
    int p0 = first < tok1 ? max(tok0, first / kTok * kTok) + warp * kTok : tok1;
    int b = p0 < tok1 ? block_of(p0) : 0;
    bool bad = false;
    while (p0 < tok1) {
        if (b < 0 || b >= num_blocks) {     // the same id in every lane
            bad = true;
            break;
        }
        const int64_t row0 = ((static_cast<int64_t>(b) * n_kv + kvh) * block_size + p0 % block_size) * D;
        float kf[kTok][DPL], vf[kTok][DPL];
#pragma unroll
        for (int u = 0; u < kTok; ++u) {
            if (p0 + u >= first && p0 + u < tok1) {
                fetch(kc + row0 + u * D, kf[u]);
                fetch(vc + row0 + u * D, vf[u]);
            } else {
#pragma unroll
                for (int i = 0; i < DPL; ++i) kf[u][i] = vf[u][i] = 0.f;
            }
        }
        const int b_next = p0 + kStep < tok1 ? block_of(p0 + kStep) : 0;
        float dot[HG * kTok];
#pragma unroll
        for (int u = 0; u < kTok; ++u)
#pragma unroll
            for (int g = 0; g < HG; ++g) {
                float d = 0.f;
#pragma unroll
                for (int i = 0; i < DPL; ++i) d = fmaf(qv[g][i], kf[u][i], d);
                dot[g * kTok + u] = d;
            }
        float z = sum_spread(dot, lane) * scale_log2;
        const int p = p0 + my_u;
        if (sc.cap2 > 0.f) z = sc.cap2 * tanhf(z / sc.cap2);
        z = fmaf(slope, static_cast<float>(p + 1 - L), z);
        z = p >= first && p < tok1 ? z : -INFINITY;
        float m_new = z;
#pragma unroll
        for (int w = kSpread * kTok / 2; w >= kSpread; w /= 2)
            m_new = fmaxf(m_new, __shfl_xor_sync(0xffffffffu, m_new, w));
        m_new = fmaxf(m_run, m_new);
        const float m_use = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = exp2f(m_run - m_use);   // 0 on the first keys (m_run = -inf)
        const float pz = exp2f(z - m_use);          // 0 for a masked key (z = -inf)
        l_run = fmaf(l_run, alpha, pz);
        m_run = m_new;
#pragma unroll
        for (int g = 0; g < HG; ++g) {
            const float down = HG > 1 ? __shfl_sync(0xffffffffu, alpha, g * kTok * kSpread) : alpha;
#pragma unroll
            for (int i = 0; i < DPL; ++i) acc[g][i] *= down;
#pragma unroll
            for (int u = 0; u < kTok; ++u) {
                const float w = __shfl_sync(0xffffffffu, pz, (g * kTok + u) * kSpread);
#pragma unroll
                for (int i = 0; i < DPL; ++i) acc[g][i] = fmaf(w, vf[u][i], acc[g][i]);
            }
        }
        p0 += kStep;
        b = b_next;
    }
    if (bad) set_error(err, PA_ERR_OUT_OF_RANGE);

    // ---- the warps' (m, l, O) of each head
#pragma unroll
    for (int w = kSpread * kTok / 2; w >= kSpread; w /= 2) l_run += __shfl_xor_sync(0xffffffffu, l_run, w);
    if (lane % (kSpread * kTok) == 0) {
        s_ml[warp][my_g][0] = m_run;
        s_ml[warp][my_g][1] = l_run;
    }
#pragma unroll
    for (int g = 0; g < HG; ++g)
#pragma unroll
        for (int c = 0; c < DPL / V; ++c) {
            FloatRun r;
#pragma unroll
            for (int e = 0; e < V; ++e) r.x[e] = acc[g][c * V + e];
            *reinterpret_cast<FloatRun*>(&s_acc[warp][g][at(c * V)]) = r;
        }
    if (__syncthreads_or(bad)) return;                  // a partition with a bad block is dropped
    for (int i = threadIdx.x; i < live * D; i += kSimtWarps * 32) {
        const int g = i / D, d = i % D;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kSimtWarps; ++w) m = fmaxf(m, s_ml[w][g][0]);
        const float m_use = m == -INFINITY ? 0.f : m;
        float l = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < kSimtWarps; ++w) {
            const float weight = exp2f(s_ml[w][g][0] - m_use);
            l = fmaf(weight, s_ml[w][g][1], l);
            o = fmaf(weight, s_acc[w][g][d], o);
        }
        if (nparts == 1) {
            store_any(out, (row_q + g) * D + d, l > 0.f ? o / l : 0.f, out_dtype);   // (no visible key: 0)
        } else {
            const int64_t u = (row_q + g) * sc.slots + sc.slot0 + j;
            ws_acc[u * D + d] = o;
            if (d == 0) {
                ws_ml[2 * u] = m;
                ws_ml[2 * u + 1] = l;
            }
        }
    }
}

template <typename T, int DPL, int HG>
static cudaError_t run_scored_simt(const DecodeArgs& a, cudaStream_t s, float scale_log2)
{
    const int group = a.n_q / a.cache.n_kv_heads;
    const dim3 grid(a.max_parts, a.cache.n_kv_heads * ((group + HG - 1) / HG), a.num_seqs);
    decode_scored_simt_kernel<T, DPL, HG><<<grid, kSimtWarps * 32, 0, s>>>(
        a.out, a.out_dtype, static_cast<const T*>(a.q), static_cast<const T*>(a.k_cache),
        static_cast<const T*>(a.v_cache), a.block_tables, a.max_blocks, a.context_lens, a.n_q,
        a.cache.n_kv_heads, group, a.cache.num_blocks, a.cache.block_size, scale_log2, a.ws_ml, a.ws_acc,
        a.part_tokens, a.max_parts, a.err, *a.score);
    return cudaGetLastError();
}

// Heads a block: the KV head's where they are at most four (two for 256 elements, whose q
// and O rows fill the registers), else four at a time.
template <typename T, int DPL>
static cudaError_t run_scored_simt_heads(const DecodeArgs& a, cudaStream_t s, float sl2)
{
    const int group = a.n_q / a.cache.n_kv_heads;
    if (group == 1) return run_scored_simt<T, DPL, 1>(a, s, sl2);
    if (group == 2 || DPL > 4) return run_scored_simt<T, DPL, 2>(a, s, sl2);
    if constexpr (DPL <= 4) return run_scored_simt<T, DPL, 4>(a, s, sl2);
    return cudaErrorInvalidValue;
}

template <typename T>
static cudaError_t run_scored_simt_dt(const DecodeArgs& a, cudaStream_t s, float sl2)
{
    switch (a.cache.head_dim) {
        case 32: return run_scored_simt_heads<T, 1>(a, s, sl2);
        case 96: return run_scored_simt_heads<T, 3>(a, s, sl2);
        case 256: return run_scored_simt_heads<T, 8>(a, s, sl2);
    }
    if constexpr (sizeof(T) == 4) {    // (16-bit rows of 64 and 128 elements go to the tensor cores)
        if (a.cache.head_dim == 64) return run_scored_simt_heads<T, 2>(a, s, sl2);
        if (a.cache.head_dim == 128) return run_scored_simt_heads<T, 4>(a, s, sl2);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_decode_scored_simt(const DecodeArgs& a, cudaStream_t s, float sl2)
{
    switch (a.cache.dtype) {
        case PA_BF16: return run_scored_simt_dt<__nv_bfloat16>(a, s, sl2);
        case PA_F16: return run_scored_simt_dt<__half>(a, s, sl2);
        case PA_F32: return run_scored_simt_dt<float>(a, s, sl2);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa

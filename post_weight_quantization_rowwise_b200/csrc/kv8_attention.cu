// kv8_attention.cu -- causal attention over the paged int8 key/value cache, on sm_100a.
//
// One warp a (row, head): scores of 32 keys at a time (a lane a key), one pass with the running
// maximum and sum of the softmax, then the values of the 32 keys (a lane four or two dimensions).
#include <math.h>

#include "kv8.cuh"

namespace {

using iqq::Kv8;
using iqq::Span;

constexpr int kThreads = 128;

struct Args {
    const void* q;
    void* out;
    float* lse;
    int64_t q_token_stride, q_head_stride;
    int32_t heads, group;
    float scale;
};

template <class T, int D>
__global__ void __launch_bounds__(kThreads)
attention_kernel(const Kv8 C, const Args A, uint32_t* __restrict__ flags)
{
    constexpr int kE = D / 32;  // output dimensions a lane
    __shared__ float sq[kThreads / 32][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    iqq::check_spans(C, false, flags);
    const int64_t row = blockIdx.x;
    const int h = blockIdx.y * (kThreads / 32) + warp;
    if (h >= A.heads) return;
    const int b = iqq::seq_of_slot(C, row, 1, 1, 0);
    const Span s = iqq::span_of(C, b);
    if (row < s.first || row >= s.first + s.n) return;
    const T* q = static_cast<const T*>(A.q) + row * A.q_token_stride + h * A.q_head_stride;
    for (int i = lane; i < D; i += 32) sq[warp][i] = iqq::to_f32(q[i]) * A.scale;
    __syncwarp();
    int64_t seen = s.start + (row - s.first) + 1;  // tokens 0 .. seen-1 are attended to
    if (seen > C.capacity) seen = C.capacity;
    const int kvh = h / A.group, page = 1 << C.page_log2;
    float m = -INFINITY, sum = 0.0f, acc[kE] = {};
    for (int64_t j0 = 0; j0 < seen; j0 += 32) {
        // page_size >= 16: the 32 keys lie in at most two pages
        const int64_t j = j0 + lane;
        int p = j < seen ? iqq::page_at(C, b, j >> C.page_log2) : -1;
        if (j < seen && p < 0) iqq::raise_flags(flags, IQQ_FLAG_BAD_INDEX);
        const int64_t cell = static_cast<int64_t>(p) * C.heads + kvh;
        const int64_t at = ((cell << C.page_log2) + (j & (page - 1))) * D;
        float score = -INFINITY, vs = 0.0f;
        if (p >= 0) {
            float dot = 0.0f;
            const uint4* k = reinterpret_cast<const uint4*>(C.codes[0] + at);
            for (int i = 0; i < D / 16; ++i) {
                const uint4 w = __ldg(k + i);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    dot = fmaf(sq[warp][16 * i + e], static_cast<float>(static_cast<int8_t>(u[e >> 2] >> (8 * (e & 3)))), dot);
            }
            score = dot * __ldg(C.scales[0] + cell);
            vs = __ldg(C.scales[1] + cell);
        }
        float top = score;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float next = fmaxf(m, top);
        const float base = next == -INFINITY ? 0.0f : next;
        const float keep = expf(m - base), w = p >= 0 ? expf(score - base) : 0.0f;
        m = next;
        sum = sum * keep;
#pragma unroll
        for (int e = 0; e < kE; ++e) acc[e] *= keep;
        sum += w;
        for (int i = 0; i < 32; ++i) {
            const int pi = __shfl_sync(0xffffffffu, p, i);
            const float wi = __shfl_sync(0xffffffffu, p >= 0 ? w * vs : 0.0f, i);
            const int64_t ai = __shfl_sync(0xffffffffu, at, i);
            if (pi < 0) continue;
            const int8_t* v = C.codes[1] + ai + lane * kE;
#pragma unroll
            for (int e = 0; e < kE; ++e) acc[e] = fmaf(wi, static_cast<float>(v[e]), acc[e]);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    T* out = static_cast<T*>(A.out) + (row * A.heads + h) * D + lane * kE;
    const bool none = m == -INFINITY && sum == 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e) out[e] = iqq::from_f32<T>(none ? 0.0f : acc[e] / sum);
    if (A.lse != nullptr && lane == 0) A.lse[row * A.heads + h] = none ? -INFINITY : m + logf(sum);
}

}  // namespace

extern "C" size_t iqq_kv8_attention_workspace_bytes(const iqq_kv8_cache*, const iqq_kv8_seqs*, int64_t, int64_t)
{
    return 0;
}

extern "C" iqq_status iqq_kv8_attention(const iqq_kv8_cache* cache, const iqq_kv8_seqs* seqs, int dtype, const void* q,
                                        int64_t q_token_stride, int64_t q_head_stride, int64_t n_heads,
                                        int64_t n_tokens, void* out, float* lse, float scale, void* workspace,
                                        size_t workspace_bytes, uint32_t* d_flags, void* stream)
{
    if (dtype != IQQ_BF16 && dtype != IQQ_F16) return IQQ_ERR_ARG;
    if (!isfinite(scale)) return IQQ_ERR_ARG;
    Kv8 C;
    const iqq_status c = iqq::kv8_check(cache, seqs, n_tokens, C);
    if (c != IQQ_OK) return c;
    if (n_tokens == 1) q_token_stride = 0;
    if (n_heads == 1) q_head_stride = 0;
    if (n_heads < 1 || n_heads % C.heads != 0 || n_heads > 65535 || q_token_stride < 0 || q_head_stride < 0)
        return IQQ_ERR_SHAPE;
    if (n_tokens == 0 || C.n_seqs == 0) return IQQ_OK;
    const size_t need = iqq_kv8_attention_workspace_bytes(cache, seqs, n_heads, n_tokens);
    if (q == nullptr || out == nullptr || (need > 0 && workspace == nullptr)) return IQQ_ERR_NULL;
    if (workspace_bytes < need) return IQQ_ERR_SHAPE;
    if (!iqq::aligned(q, 16) || !iqq::aligned(out, 16) || !iqq::aligned(lse, 4) || q_token_stride % 8 != 0 ||
        q_head_stride % 8 != 0 || !iqq::aligned(workspace, 16) || !iqq::aligned(d_flags, 4))
        return IQQ_ERR_ALIGN;
    const Args A = {q, out, lse, q_token_stride, q_head_stride, static_cast<int32_t>(n_heads),
                    static_cast<int32_t>(n_heads / C.heads), scale};
    const dim3 grid(static_cast<unsigned>(n_tokens), static_cast<unsigned>((n_heads + 3) / 4));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool wide = cache->head_dim == 128;
    if (dtype == IQQ_BF16)
        (wide ? attention_kernel<__nv_bfloat16, 128> : attention_kernel<__nv_bfloat16, 64>)<<<grid, kThreads, 0, st>>>(C, A, d_flags);
    else
        (wide ? attention_kernel<__half, 128> : attention_kernel<__half, 64>)<<<grid, kThreads, 0, st>>>(C, A, d_flags);
    return iqq::launch_status();
}

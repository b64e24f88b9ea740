// kv8_cache.cu -- writing and reading back the paged int8 key/value cache, on sm_100a.
//
// Append.  One CTA (a warp, where a sequence has few new tokens) takes one (page, head) of the keys or
// of the values: the new tokens of the page set its scale, so whoever quantizes them is the only one
// that reads the page's old scale and rewrites its old codes.  d = max(d_old, fl32(amax/127)); the new
// values wait in registers, as they were read, between the maximum and the rounding (what a page of
// 128 tokens does not fit is read again, from L2).  HBM-bound on prompts (2 or 4 B in, 1 B out a
// value); a decoding step is one token and, when the scale grows, the page's old codes, and takes the
// five dependent reads (cu, the span, the table, the scale, the codes) that lead to its store.
//
// Measured: 12 prompts of up to 1500 tokens, 8 heads of 128 dimensions, bfloat16: 21.8 us (2.2 TB/s);
// 96 sequences of one token: 4.8 us.
//
// Gather.  One warp a packed row: fl32(d * q) of all heads, 8 codes in and 16 or 32 B out a lane.
// The same prompts back: 9.1 us (5.5 TB/s).
#include "kv8.cuh"

namespace {

using iqq::Kv8;
using iqq::Span;

constexpr int kThreads = 256;        // of a gathering CTA
constexpr int kAppendThreads = 128;

struct New {
    const void* p[2];
    int64_t token_stride[2], head_stride[2];
};

// G threads (a warp, or the CTA) take slot, head and which (keys or values) together.
template <class T, int D, int G>
__global__ void __launch_bounds__(kAppendThreads, 8)
append_kernel(const Kv8 C, const New N, uint32_t* __restrict__ flags)
{
    constexpr int kRow = D / 8;                        // units of eight values of a token
    constexpr int kUnits = sizeof(T) == 2 ? 8 : 4;     // units a thread keeps
    __shared__ uint32_t part[kAppendThreads / 32];
    const int tid = threadIdx.x % G, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    iqq::check_spans(C, true, flags);
    const int page = 1 << C.page_log2;
    const int item = (blockIdx.y * kAppendThreads + threadIdx.x) / G;  // head and which, which first
    if (item >= 2 * C.heads) return;
    const int head = item >> 1, which = item & 1;
    const int64_t slot = blockIdx.x;
    const int b = iqq::seq_of_slot(C, slot, 1, page, 2);
    const Span s = iqq::span_of(C, b);
    const int64_t j = slot - iqq::slot_base(C, b, 1, page, 2);  // the sequence's j-th page reached
    if (j < 0 || !s.ok || s.start < 0) return;  // (a slot before the first sequence's, where cu begins above 0)
    const int64_t index = (s.start >> C.page_log2) + j, t0 = index << C.page_log2;
    if (s.n == 0 || t0 >= s.len) return;
    const int p = t0 < C.capacity ? iqq::page_at(C, b, index) : -1;
    // tokens lo .. hi-1 of the page are new
    const int lo = s.start > t0 ? static_cast<int>(s.start - t0) : 0;
    const int hi = s.len - t0 < page ? static_cast<int>(s.len - t0) : page;
    const int64_t row0 = s.first + (t0 + lo - s.start);
    const int64_t ts = N.token_stride[which];
    const T* x = static_cast<const T*>(N.p[which]) + row0 * ts + head * N.head_stride[which];
    const int units = (hi - lo) * kRow;
    const auto at = [&](int u) { return x + (u / kRow) * ts + (u % kRow) * 8; };

    typename iqq::Raw<T>::type v[kUnits];
    uint32_t m = 0u;
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        v[k] = {};
        if (tid + k * G < units) iqq::fetch(at(tid + k * G), v[k]);
    }
    if (p < 0) {
        if (tid == 0) iqq::raise_flags(flags, IQQ_FLAG_BAD_INDEX);
        return;
    }
    float* scale = C.scales[which] + static_cast<int64_t>(p) * C.heads + head;
    const float held = lo > 0 ? *scale : 0.0f;
#pragma unroll
    for (int k = 0; k < kUnits; ++k) m = iqq::amax8(x, v[k], m);
    for (int u = tid + kUnits * G; u < units; u += G) {
        typename iqq::Raw<T>::type t;
        iqq::fetch(at(u), t);
        m = iqq::amax8(x, t, m);
    }
    m = __reduce_max_sync(0xffffffffu, iqq::amax_bits(x, m));
    if constexpr (G > 32) {
        if (lane == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();  // every thread has read the old scale, too
        m = __reduce_max_sync(0xffffffffu, part[lane % (G / 32)]);
    } else {
        __syncwarp();
    }
    const float need = iqq::i8_scale(m);
    const float d = need != need || held != held ? __uint_as_float(0x7fc00000u) : fmaxf(held, need);
    const float inv = d > 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
    if (tid == 0) {
        *scale = d;
        if (m >= iqq::kInfBits) iqq::raise_flags(flags, IQQ_FLAG_NONFINITE_INPUT);
    }
    uint2* tile = reinterpret_cast<uint2*>(C.codes[which] + ((static_cast<int64_t>(p) * C.heads + head) << C.page_log2) * D);
    const auto store = [&](int u, const typename iqq::Raw<T>::type& r) {
        float t[8];
        iqq::widen(x, r, t);
        tile[lo * kRow + u] = d > 0.0f ? iqq::codes8(t, d, inv) : make_uint2(0u, 0u);
    };
#pragma unroll
    for (int k = 0; k < kUnits; ++k)
        if (tid + k * G < units) store(tid + k * G, v[k]);
    for (int u = tid + kUnits * G; u < units; u += G) {
        typename iqq::Raw<T>::type t;
        iqq::fetch(at(u), t);
        store(u, t);
    }
    if (d > held) {  // the tokens already in the page, to the new scale
        const float ratio = held * inv;
#pragma unroll 4
        for (int u = tid; u < lo * kRow; u += G) {
            const uint2 w = tile[u];
            int c[8];
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = static_cast<int8_t>((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
                t[i] = static_cast<float>(c[i]);
            }
            tile[u] = iqq::codes8(t, ratio, [&](int i, float q) { return iqq::exact_code(held, c[i], d, q); });
        }
    }
}

__device__ __forceinline__ void put8(float* p, const float (&v)[8])
{
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <class T>
__device__ __forceinline__ void put8(T* p, const float (&v)[8])
{
    __align__(16) T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = iqq::from_f32<T>(v[i]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(t);
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads)
gather_kernel(const Kv8 C, T* __restrict__ ko, T* __restrict__ vo, uint32_t* __restrict__ flags)
{
    constexpr int kRow = D / 8, kFlight = 4;
    const int lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    iqq::check_spans(C, true, flags);
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= C.n_tokens) return;
    const int b = iqq::seq_of_slot(C, row, 1, 1, 0);
    const Span s = iqq::span_of(C, b);
    if (row < s.first || row >= s.first + s.n) return;  // a row of no sequence (s.n is 0 for a bad span)
    const int64_t pos = s.start + (row - s.first);
    int p = -1;
    if (pos >= 0 && pos < C.capacity) p = iqq::page_at(C, b, pos >> C.page_log2);
    if (p < 0 && lane == 0) iqq::raise_flags(flags, IQQ_FLAG_BAD_INDEX);
    const int off = static_cast<int>(pos & ((1 << C.page_log2) - 1));
    const int units = C.heads * kRow;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        T* out = (which == 0 ? ko : vo) + row * units * 8;
        // four units' loads before their stores (which may not pass one another)
        for (int u0 = lane; u0 < units; u0 += 32 * kFlight) {
            float d[kFlight];
            uint2 w[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const int u = u0 + 32 * i;
                d[i] = 0.0f;
                w[i] = make_uint2(0u, 0u);
                if (p >= 0 && u < units) {
                    const int64_t cell = static_cast<int64_t>(p) * C.heads + u / kRow;
                    d[i] = iqq::ld(C.scales[which] + cell);
                    w[i] = iqq::ld(reinterpret_cast<const uint2*>(C.codes[which] + ((cell << C.page_log2) + off) * D + (u % kRow) * 8));
                }
            }
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                if (u0 + 32 * i >= units) break;
                float t[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    t[e] = __fmul_rn(d[i], static_cast<float>(static_cast<int8_t>((e < 4 ? w[i].x : w[i].y) >> (8 * (e & 3)))));
                put8(out + (u0 + 32 * i) * 8, t);
            }
        }
    }
}

template <class K, class... A>
iqq_status launch(K kernel, dim3 grid, int threads, cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kernel, args...);
    return iqq::launch_status();
}

}  // namespace

iqq_status iqq::kv8_check(const iqq_kv8_cache* cache, const iqq_kv8_seqs* seqs, int64_t n_tokens, Kv8& C)
{
    if (cache == nullptr || seqs == nullptr) return IQQ_ERR_NULL;
    const int64_t ps = cache->page_size, d = cache->head_dim;
    if (ps != 16 && ps != 32 && ps != 64 && ps != 128) return IQQ_ERR_SHAPE;
    if (d != 64 && d != 128) return IQQ_ERR_SHAPE;
    if (cache->n_pages < 0 || cache->n_pages > 0x7fffffffLL || cache->n_kv_heads < 1 || cache->n_kv_heads > 65535 ||
        n_tokens < 0 || n_tokens > 0x7fffffffLL || seqs->n_seqs < 0 || seqs->n_seqs > (1LL << 24) ||
        seqs->table_width < 0 || seqs->table_width > 0x7fffffffLL || !size_ok(cache->n_pages * cache->n_kv_heads, ps * d, 1))
        return IQQ_ERR_SHAPE;
    if (seqs->n_seqs > 1 && seqs->table_stride < seqs->table_width) return IQQ_ERR_SHAPE;
    if (seqs->n_seqs > 0 && n_tokens > 0) {
        if (cache->n_pages == 0) return IQQ_ERR_SHAPE;
        if (cache->k_codes == nullptr || cache->v_codes == nullptr || cache->k_scales == nullptr || cache->v_scales == nullptr)
            return IQQ_ERR_NULL;
        if (seqs->seq_lens == nullptr || seqs->cu_tokens == nullptr ||
            (seqs->table_width > 0 && seqs->block_tables == nullptr))
            return IQQ_ERR_NULL;
        if (!aligned(cache->k_codes, 16) || !aligned(cache->v_codes, 16) || !aligned(cache->k_scales, 4) ||
            !aligned(cache->v_scales, 4) || !aligned(seqs->block_tables, 4) || !aligned(seqs->seq_lens, 4) ||
            !aligned(seqs->cu_tokens, 4))
            return IQQ_ERR_ALIGN;
    }
    C.codes[0] = cache->k_codes;
    C.codes[1] = cache->v_codes;
    C.scales[0] = cache->k_scales;
    C.scales[1] = cache->v_scales;
    C.tables = seqs->block_tables;
    C.lens = seqs->seq_lens;
    C.cu = seqs->cu_tokens;
    C.table_stride = seqs->table_stride;
    C.n_pages = static_cast<int32_t>(cache->n_pages);
    C.heads = static_cast<int32_t>(cache->n_kv_heads);
    C.page_log2 = ps == 16 ? 4 : (ps == 32 ? 5 : (ps == 64 ? 6 : 7));
    C.n_seqs = static_cast<int32_t>(seqs->n_seqs);
    C.n_tokens = static_cast<int32_t>(n_tokens);
    C.capacity = seqs->table_width * ps;
    return IQQ_OK;
}

extern "C" iqq_status iqq_kv8_append(const iqq_kv8_cache* cache, const iqq_kv8_seqs* seqs, int dtype, const void* k,
                                     int64_t k_token_stride, int64_t k_head_stride, const void* v,
                                     int64_t v_token_stride, int64_t v_head_stride, int64_t n_tokens,
                                     uint32_t* d_flags, void* stream)
{
    if (!iqq::dtype_ok(dtype)) return IQQ_ERR_ARG;
    Kv8 C;
    const iqq_status c = iqq::kv8_check(cache, seqs, n_tokens, C);
    if (c != IQQ_OK) return c;
    if (n_tokens == 0 || C.n_seqs == 0) return IQQ_OK;
    const int64_t each = 16 / iqq::dtype_bytes(dtype);
    if (n_tokens == 1) k_token_stride = v_token_stride = 0;
    if (C.heads == 1) k_head_stride = v_head_stride = 0;
    if (k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0) return IQQ_ERR_SHAPE;
    if (k == nullptr || v == nullptr) return IQQ_ERR_NULL;
    if (!iqq::aligned(k, 16) || !iqq::aligned(v, 16) || k_token_stride % each != 0 || k_head_stride % each != 0 ||
        v_token_stride % each != 0 || v_head_stride % each != 0 || !iqq::aligned(d_flags, 4))
        return IQQ_ERR_ALIGN;
    const New N = {{k, v}, {k_token_stride, v_token_stride}, {k_head_stride, v_head_stride}};
    // n tokens reach at most floor(n / page) + 2 pages of a sequence
    const int64_t slots = n_tokens / cache->page_size + 2LL * C.n_seqs;
    // A warp a page and head while a sequence has up to four new tokens (96 sequences of one token, 8
    // heads: 4.6 us; with a CTA of 256 threads each it took 27), else a CTA.
    const bool few = n_tokens <= 4LL * C.n_seqs;
    const int64_t items = 2LL * C.heads, held = few ? kAppendThreads / 32 : 1, groups = (items + held - 1) / held;
    if (slots > 0x7fffffffLL || groups > 65535) return IQQ_ERR_SHAPE;
    const dim3 grid(static_cast<unsigned>(slots), static_cast<unsigned>(groups));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const auto go = [&](auto zero) -> iqq_status {
        using T = decltype(zero);
        if (cache->head_dim == 128)
            return few ? launch(append_kernel<T, 128, 32>, grid, kAppendThreads, st, C, N, d_flags)
                       : launch(append_kernel<T, 128, kAppendThreads>, grid, kAppendThreads, st, C, N, d_flags);
        return few ? launch(append_kernel<T, 64, 32>, grid, kAppendThreads, st, C, N, d_flags)
                   : launch(append_kernel<T, 64, kAppendThreads>, grid, kAppendThreads, st, C, N, d_flags);
    };
    switch (dtype) {
    case IQQ_F32: return go(float{});
    case IQQ_BF16: return go(__nv_bfloat16{});
    default: return go(__half{});
    }
}

extern "C" iqq_status iqq_kv8_gather(const iqq_kv8_cache* cache, const iqq_kv8_seqs* seqs, int dtype, void* k_out,
                                     void* v_out, int64_t n_tokens, uint32_t* d_flags, void* stream)
{
    if (!iqq::dtype_ok(dtype)) return IQQ_ERR_ARG;
    Kv8 C;
    const iqq_status c = iqq::kv8_check(cache, seqs, n_tokens, C);
    if (c != IQQ_OK) return c;
    if (n_tokens == 0 || C.n_seqs == 0) return IQQ_OK;
    if (k_out == nullptr || v_out == nullptr) return IQQ_ERR_NULL;
    if (!iqq::aligned(k_out, 16) || !iqq::aligned(v_out, 16) || !iqq::aligned(d_flags, 4)) return IQQ_ERR_ALIGN;
    constexpr int kRows = kThreads / 32;
    const dim3 grid(static_cast<unsigned>((n_tokens + kRows - 1) / kRows));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto go = [&](auto* k, auto* v) -> iqq_status {
        using T = std::remove_pointer_t<decltype(k)>;
        return launch(cache->head_dim == 128 ? gather_kernel<T, 128> : gather_kernel<T, 64>, grid, kThreads, st, C, k, v, d_flags);
    };
    switch (dtype) {
    case IQQ_F32: return go(static_cast<float*>(k_out), static_cast<float*>(v_out));
    case IQQ_BF16: return go(static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out));
    default: return go(static_cast<__half*>(k_out), static_cast<__half*>(v_out));
    }
}

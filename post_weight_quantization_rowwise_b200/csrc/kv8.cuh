// kv8.cuh -- the paged int8 key/value cache as its kernels see it (iqq_kv8_cache and
// iqq_kv8_seqs in iqq.h), and the checks its entry points share.
#pragma once

#include "i8_code.cuh"

namespace iqq {

struct Kv8 {
    int8_t* codes[2];   // keys, values
    float* scales[2];
    const int32_t* tables;
    const int32_t* lens;
    const int32_t* cu;
    int64_t table_stride;
    int32_t n_pages, heads, page_log2, n_seqs, n_tokens;
    int64_t capacity;   // table_width * page_size
};

// A sequence's part of a call: `first` its first packed row, `n` its rows, `start` the position
// of the first of them (below 0 when there are more rows than tokens), `len` its cached tokens.
struct Span {
    int32_t first, n;
    int64_t start, len;
    bool ok;
};

__device__ __forceinline__ Span span_of(const Kv8& C, int b)
{
    Span s;
    const int32_t c0 = __ldg(C.cu + b), c1 = __ldg(C.cu + b + 1), len = __ldg(C.lens + b);
    s.ok = c0 >= 0 && c1 >= c0 && c1 <= C.n_tokens && len >= 0;
    s.first = c0;
    s.n = s.ok ? c1 - c0 : 0;
    s.len = len;
    s.start = static_cast<int64_t>(len) - s.n;
    return s;
}

// The first CTA of a launch looks over every span, whether or not its rows get work: a bad span
// or length raises the flag once, and the others need only leave it out.  `places`: every new
// token needs a place in the cache.
__device__ __forceinline__ void check_spans(const Kv8& C, bool places, uint32_t* flags)
{
    if (blockIdx.x != 0 || blockIdx.y != 0 || blockIdx.z != 0) return;
    bool bad = false;
    for (int b = threadIdx.x; b < C.n_seqs; b += blockDim.x) {
        const Span s = span_of(C, b);
        bad |= !s.ok || s.len > C.capacity || (places && s.start < 0);
    }
    if (bad) raise_flags(flags, IQQ_FLAG_BAD_INDEX);
}

// Work laid out by sequence without a pass over the spans: sequence b's slots begin at
// slot_base(b) = floor(cu[b] * per / unit) + extra * b, so slots of every sequence fit between its
// base and the next one's, and the sequence of a slot is found by bisection over cu.  (cu is
// clamped, so arrays that are not monotone give some sequence in range, which span_of checks.)
__device__ __forceinline__ int64_t slot_base(const Kv8& C, int b, int per, int unit, int extra)
{
    const int32_t c = max(0, min(__ldg(C.cu + b), C.n_tokens));
    return static_cast<int64_t>(c) * per / unit + static_cast<int64_t>(extra) * b;
}

__device__ __forceinline__ int seq_of_slot(const Kv8& C, int64_t slot, int per, int unit, int extra)
{
    int lo = 0, hi = C.n_seqs;  // base(lo) <= slot < base(hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (slot_base(C, mid, per, unit, extra) <= slot) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The page of tokens pos >> page_log2 of sequence b, or -1 when the table's entry is no page.
__device__ __forceinline__ int page_at(const Kv8& C, int b, int64_t index)
{
    const int p = __ldg(C.tables + b * C.table_stride + index);
    return p >= 0 && p < C.n_pages ? p : -1;
}

// Host checks shared by the entry points; fills C.
iqq_status kv8_check(const iqq_kv8_cache* cache, const iqq_kv8_seqs* seqs, int64_t n_tokens, Kv8& C);

}  // namespace iqq

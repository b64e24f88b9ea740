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
    const int32_t c0 = ld(C.cu + b), c1 = ld(C.cu + b + 1), len = ld(C.lens + b);
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
// base and the next one's, and the sequence of a slot is found by a search over cu.  (cu is
// clamped, so arrays that are not monotone give some sequence in range, which span_of checks.)
__device__ __forceinline__ int64_t slot_base(const Kv8& C, int b, int per, int unit, int extra)
{
    const int32_t c = max(0, min(ld(C.cu + b), C.n_tokens));
    return static_cast<int64_t>(c) * per / unit + static_cast<int64_t>(extra) * b;
}

// All lanes of a warp together, 32 places of cu looked at each time.
__device__ __forceinline__ int seq_of_slot(const Kv8& C, int64_t slot, int per, int unit, int extra)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = C.n_seqs;  // base(lo) <= slot < base(hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
        const uint32_t past = __ballot_sync(0xffffffffu, at < hi && slot_base(C, at, per, unit, extra) <= slot);
        lo += step * (past == 0xffffffffu ? 32 : __ffs(~past) - 1);
        hi = min(hi, lo + step);
    }
    return lo;
}

// The page of tokens pos >> page_log2 of sequence b, or -1 when the table's entry is no page.
__device__ __forceinline__ int page_at(const Kv8& C, int b, int64_t index)
{
    const int p = ld(C.tables + b * C.table_stride + index);
    return p >= 0 && p < C.n_pages ? p : -1;
}

// Whether one of the keys j0 .. j1-1 of sequence b (j1 within its table) has a page.  Asked where a row's
// sum of weights is 0 or NaN: its scores may all be -Inf (an infinity in q, products beyond binary32),
// whose softmax is NaN, or it saw no key.
__device__ __forceinline__ bool any_page(const Kv8& C, int b, int64_t j0, int64_t j1)
{
    for (int64_t index = j0 >> C.page_log2; (index << C.page_log2) < j1; ++index)
        if (page_at(C, b, index) >= 0) return true;
    return false;
}

// What both attention kernels take: q, the outputs, and n_heads = group * key/value heads.
struct Attend {
    const void* q;
    void* out;
    float* lse;
    int64_t q_token_stride, q_head_stride;
    int32_t heads, group;
    float scale;
    // Parts of rows, where the keys of a row are split over CTAs: normalized outputs, log-sums (base 2).
    int32_t splits;
    float* part;
    float* part_lse;
};

constexpr float kLog2e = 1.4426950408889634f;
// The maximum of no score: below every finite one.  As a part's log-sum it says that the part's scores are
// all -Inf: it has no weight beside a part with finite ones, and where all parts say so the row is NaN
// (a part that saw no key says -Inf).
constexpr float kNone = -3.4028234663852886e38f;

constexpr float kTinyScale = 8.077935669463161e-28f;  // 2^-90: a value scale below it counts as 0, so denominators stay finite

// The weights 2^(y - m) go to the products in binary16, where a value below 2^-14 rounds by an
// absolute 2^-25.  So the reference m is kept kLift below the largest y when it moves, and moves
// only when a y comes kMove further: the largest weight is 2^7 to 2^15 (of 65504), and a weight
// rounds by 2^-11 of itself or 2^-32 of the largest.
constexpr float kLift = 7.0f, kMove = 8.0f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t sub_h2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
// A row of q becomes binary16 exactly when it is multiplied by a power of two that brings its
// largest magnitude `top` near 2^14 (values below 2^-38 of it round, which is beyond the binary32
// sums): the exponent of the power's reciprocal, kept where both are normal.
__device__ __forceinline__ int row_exponent(float top)
{
    return max(-126, min(126, static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14));
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Many rows a sequence (kv8_prompt.cu): how many CTAs share the keys of 256 rows, the workspace's bytes
// (0 for one), and the launch.
int prompt_splits(const iqq_kv8_cache* cache, const iqq_kv8_seqs* seqs, int64_t n_heads, int64_t n_tokens);
size_t prompt_part_bytes(const iqq_kv8_cache* cache, const iqq_kv8_seqs* seqs, int64_t n_heads, int64_t n_tokens,
                         int splits, size_t* lse_bytes);
iqq_status launch_prompt(const iqq_kv8_cache* cache, const Kv8& C, const Attend& A, int dtype, uint32_t* flags,
                         cudaStream_t st);

// Host checks shared by the entry points; fills C.
iqq_status kv8_check(const iqq_kv8_cache* cache, const iqq_kv8_seqs* seqs, int64_t n_tokens, Kv8& C);

}  // namespace iqq

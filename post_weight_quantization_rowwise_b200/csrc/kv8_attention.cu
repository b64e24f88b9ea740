// kv8_attention.cu -- causal attention over the paged int8 key/value cache, on sm_100a.
//
// For a row (a query token and head) with scores s_j = scale * q . k_j:
//     out = sum_j p_j v_j / sum_j p_j,  p_j = exp(s_j - m),
// in one pass over the keys with the running maximum m and sum of the softmax.  The rows of a
// sequence that share a key/value head are packed together (row r is token r / group, head
// r % group of the group), so a page is read once for all of them.
//
// decode kernel (few rows a sequence).  Bound by the cache's bytes.  A warp takes 16 keys at a
// time straight from global memory into the operand registers of mma.m16n8k16:
//     S^T = K Q^T (16 keys x 8 rows),  O^T = V^T P^T (16 dimensions x 8 rows).
// The order of the dimensions in a dot product, and of the rows of V^T, is free, so each lane
// loads 16 contiguous bytes and no transposition through shared memory is needed; P^T goes from
// the accumulators' layout to the operand's by movmatrix.  int8 codes become binary16 exactly:
// the byte b of a code c, in the low byte of 0x6400, is the binary16 1152 + c after b ^= 0x80,
// and 1152 is subtracted.  Rows of q become binary16 exactly as well, by a power of two for each
// row that brings its largest value near 2^14 (values below 2^-38 of it round, which is beyond
// the binary32 sums).  The weights p_j are rounded to binary16, times the page's value scale over
// a power of two that follows the largest such scale: 2^-11 each, as fine as the output's type or
// finer.  The running maximum moves only when a score passes it by 2^8, so a block costs one vote.
//
// The keys of a sequence are split over CTAs (and the four warps of one) so that the machine is
// filled; partial results, each with its log-sum, meet in the workspace and combine_kernel joins
// them.
#include <math.h>

#include <algorithm>

#include "kv8.cuh"

namespace {

using iqq::Kv8;
using iqq::Span;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSegment = 2048;   // keys whose pages are looked up at a time
constexpr int kMinChunk = 256;   // keys a CTA takes at least
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
    const void* q;
    void* out;
    float* lse;
    int64_t q_token_stride, q_head_stride;
    int32_t heads, group, splits;
    float scale;
    float* part;      // [n_tokens * heads][splits][head_dim], then the log-sums [..][splits]
    float* part_lse;
};

// The keys of a CTA: a sequence's length divided by the launch's splits, whole multiples of 64.
__device__ __forceinline__ int64_t chunk_of(int64_t len, int splits)
{
    const int64_t c = ((len + splits - 1) / splits + 63) / 64 * 64;
    return c < kMinChunk ? kMinChunk : c;
}

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
// Bytes 0 and 2, and bytes 1 and 3, of four codes as binary16 pairs.
__device__ __forceinline__ uint32_t codes_even(uint32_t w) { return sub_h2((w & 0x00ff00ffu) ^ 0x64806480u, 0x64806480u); }
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) { return codes_even(w >> 8); }

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 keys of a page for this lane: keys g and g+8 (dimensions 16t.. of each 64), and the values
// of keys 2t, 2t+1, 2t+8, 2t+9 (dimensions D/8 * g ..); g = lane / 4, t = lane % 4.
template <int D>
struct Block {
    uint32_t k[2][D / 16];
    uint32_t v[4][D / 32];
};

template <int D>
__device__ __forceinline__ void load_block(Block<D>& B, const Kv8& C, int page, int kvh, int off, int g, int t)
{
    const int64_t at = (((static_cast<int64_t>(page) * C.heads + kvh) << C.page_log2) + off) * D;
    const int8_t* k = C.codes[0] + at;
    const int8_t* v = C.codes[1] + at;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(k + (g + 8 * h) * D + 64 * i + 16 * t));
            B.k[h][4 * i] = w.x; B.k[h][4 * i + 1] = w.y; B.k[h][4 * i + 2] = w.z; B.k[h][4 * i + 3] = w.w;
        }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int8_t* p = v + (2 * t + (i & 1) + 8 * (i >> 1)) * D + D / 8 * g;
        if constexpr (D == 128) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
            B.v[i][0] = w.x; B.v[i][1] = w.y; B.v[i][2] = w.z; B.v[i][3] = w.w;
        } else {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
            B.v[i][0] = w.x; B.v[i][1] = w.y;
        }
    }
}

template <class T, int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? (D == 64 ? 4 : 3) : 2)
decode_kernel(const Kv8 C, const Args A, uint32_t* __restrict__ flags)
{
    constexpr int kRows = 8 * NT, kK = D / 16, kM = D / 16;  // k steps of S, 16-row tiles of O^T
    __shared__ int s_page[kSegment / 16];
    __shared__ float s_ks[kSegment / 16], s_vs[kSegment / 16];
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
    __shared__ __align__(16) float s_o[kWarps][kRows][D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    iqq::check_spans(C, false, flags);

    const int64_t slot = blockIdx.x;
    const int split = blockIdx.y;
    const int kvh = blockIdx.z;
    const int b = iqq::seq_of_slot(C, slot, A.group, kRows, 1);
    const Span s = iqq::span_of(C, b);
    const int64_t first_row = (slot - iqq::slot_base(C, b, A.group, kRows, 1)) * kRows;
    const int64_t rows = static_cast<int64_t>(s.n) * A.group;  // 0 for a bad span
    if (first_row >= rows) return;
    // keys this tile's rows can see at all, and this CTA's part of them
    const int64_t len = s.len < C.capacity ? s.len : C.capacity;
    const int64_t last_row = first_row + kRows < rows ? first_row + kRows - 1 : rows - 1;
    const int64_t seen = min(len, s.start + last_row / A.group + 1);
    const int64_t chunk = chunk_of(len, A.splits);
    const int64_t j0 = split * chunk;
    if (split > 0 && j0 >= len) return;
    const int64_t j1 = min(seen, j0 + chunk);

    // the rows of q this lane feeds (row g of each 8), as binary16 times 2^-e
    uint32_t bq[NT][kK][2];
    float unscale[NT][2];  // of rows 2t, 2t+1: scale * 2^e * log2(e)
    int limit[NT][2];      // keys of this CTA (from j0) below it are seen
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int64_t r = first_row + 8 * n + g;
        float v[D / 4];
        if (r < rows) {
            const T* q = static_cast<const T*>(A.q) + (s.first + r / A.group) * A.q_token_stride +
                         (kvh * A.group + r % A.group) * A.q_head_stride;
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float u[8];
                    iqq::load8(q + 64 * i + 16 * t + 8 * h, u);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[16 * i + 8 * h + e] = u[e];
                }
        } else {
#pragma unroll
            for (int i = 0; i < D / 4; ++i) v[i] = 0.0f;
        }
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(v[i]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // e = exponent of top - 14, kept where 2^e and 2^-e are normal
        int e = static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14;
        e = max(-110, min(110, e));
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
        for (int j = 0; j < kK; ++j) {
            // dimensions 64 (j/4) + 16 t + 4 (j%4) + {0, 2} and {1, 3}: as codes_even and codes_odd
            const int i = 16 * (j >> 2) + 4 * (j & 3);
            bq[n][j][0] = pack_h2(v[i] * down, v[i + 2] * down);
            bq[n][j][1] = pack_h2(v[i + 1] * down, v[i + 3] * down);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            unscale[n][h] = __shfl_sync(0xffffffffu, up, (2 * t + h) * 4) * A.scale * kLog2e;
            const int64_t row = first_row + 8 * n + 2 * t + h;
            const int64_t lim = row < rows ? min(len, s.start + row / A.group + 1) - j0 : 0;
            limit[n][h] = static_cast<int>(max(int64_t{0}, min(lim, int64_t{0x7fffffff})));
        }
    }
    // below this key (from j0) no row of the tile needs a mask
    const int64_t clear64 = min(len, s.start + first_row / A.group + 1) - j0;
    const int clear = last_row - first_row + 1 == kRows ? static_cast<int>(max(int64_t{0}, min(clear64, int64_t{0x7fffffff}))) : 0;

    float m[NT][2], l[NT][2], o[NT][kM][4], vref = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            m[n][h] = -INFINITY;
            l[n][h] = 0.0f;
        }
#pragma unroll
        for (int d = 0; d < kM; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][d][i] = 0.0f;
    }

    const int page_size = 1 << C.page_log2;
    for (int64_t seg = j0; seg < j1; seg += kSegment) {
        const int64_t seg_end = min(j1, seg + kSegment);
        const int64_t p0 = seg >> C.page_log2;
        const int pages = static_cast<int>(((seg_end - 1) >> C.page_log2) - p0) + 1;
        if (seg > j0) __syncthreads();
        if (tid < pages) {
            const int p = iqq::page_at(C, b, p0 + tid);
            s_page[tid] = p;
            const int64_t cell = static_cast<int64_t>(p) * C.heads + kvh;
            s_ks[tid] = p < 0 ? 0.0f : __ldg(C.scales[0] + cell);
            s_vs[tid] = p < 0 ? 0.0f : __ldg(C.scales[1] + cell);
            if (p < 0) iqq::raise_flags(flags, IQQ_FLAG_BAD_INDEX);
        }
        __syncthreads();
        const int blocks = static_cast<int>((seg_end - seg + 15) >> 4);
        auto place = [&](int i) { return static_cast<int>(((seg + 16 * i) >> C.page_log2) - p0); };
        auto fetch = [&](int i, Block<D>& B) {
            const int p = s_page[place(i)];
            if (p >= 0) load_block<D>(B, C, p, kvh, static_cast<int>((seg + 16 * i) & (page_size - 1)), g, t);
        };
        Block<D> cur, next;
        if (warp < blocks) fetch(warp, cur);
        for (int i = warp; i < blocks; i += kWarps) {
            if (i + kWarps < blocks) fetch(i + kWarps, next);
            const int at = place(i);
            const int key0 = static_cast<int>(seg - j0) + 16 * i;  // from j0
            if (s_page[at] >= 0) {
                const float ks = s_ks[at], vs = s_vs[at];
                float x[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[n][e] = 0.0f;
#pragma unroll
                for (int j = 0; j < kK; ++j) {
                    const uint32_t a0 = codes_even(cur.k[0][j]), a2 = codes_odd(cur.k[0][j]);
                    const uint32_t a1 = codes_even(cur.k[1][j]), a3 = codes_odd(cur.k[1][j]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma(x[n], a0, a1, a2, a3, bq[n][j][0], bq[n][j][1]);
                }
                const bool masked = key0 + 16 > clear;
                bool moved = false;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float f = unscale[n][h] * ks;
                        x[n][h] *= f;
                        x[n][2 + h] *= f;
                        if (masked) {
                            if (key0 + g >= limit[n][h]) x[n][h] = -INFINITY;
                            if (key0 + g + 8 >= limit[n][h]) x[n][2 + h] = -INFINITY;
                        }
                        moved |= fmaxf(x[n][h], x[n][2 + h]) > m[n][h] + 8.0f;
                    }
                }
                if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float top = fmaxf(x[n][h], x[n][2 + h]);
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                            top = fmaxf(top, m[n][h]);
                            const float f = top == -INFINITY ? 1.0f : ex2(m[n][h] - top);
                            m[n][h] = top;
                            l[n][h] *= f;
#pragma unroll
                            for (int d = 0; d < kM; ++d) {
                                o[n][d][h] *= f;
                                o[n][d][2 + h] *= f;
                            }
                        }
                }
                if (vs > vref) {  // (uniform) the next power of two above vs
                    const float up = __uint_as_float((__float_as_uint(vs) & 0x7f800000u) + 0x00800000u);
                    const float f = vref == 0.0f ? 1.0f : __fdiv_rn(vref, up);
                    vref = up;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int d = 0; d < kM; ++d)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[n][d][e] *= f;
                }
                const float vf = vs == 0.0f ? 0.0f : __fdiv_rn(vs, vref == 0.0f ? 1.0f : vref);
                uint32_t bp[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float p[4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float mu = m[n][h] == -INFINITY ? 0.0f : m[n][h];
                        p[h] = ex2(x[n][h] - mu);
                        p[2 + h] = ex2(x[n][2 + h] - mu);
                        l[n][h] += p[h] + p[2 + h];
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = x[n][e] == -INFINITY ? 0.0f : p[e] * vf;
                    bp[n][0] = transpose8(pack_h2(p[0], p[1]));
                    bp[n][1] = transpose8(pack_h2(p[2], p[3]));
                }
#pragma unroll
                for (int d = 0; d < kM; d += 2) {
                    // bytes 2d .. 2d+3 of the lane's dimensions: tiles d and d+1
                    const uint32_t w01a = __byte_perm(cur.v[0][d / 2], cur.v[1][d / 2], 0x5410);
                    const uint32_t w23a = __byte_perm(cur.v[2][d / 2], cur.v[3][d / 2], 0x5410);
                    const uint32_t w01b = __byte_perm(cur.v[0][d / 2], cur.v[1][d / 2], 0x7632);
                    const uint32_t w23b = __byte_perm(cur.v[2][d / 2], cur.v[3][d / 2], 0x7632);
                    const uint32_t a0 = codes_even(w01a), a1 = codes_odd(w01a), a2 = codes_even(w23a), a3 = codes_odd(w23a);
                    const uint32_t c0 = codes_even(w01b), c1 = codes_odd(w01b), c2 = codes_even(w23b), c3 = codes_odd(w23b);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma(o[n][d], a0, a1, a2, a3, bp[n][0], bp[n][1]);
                        mma(o[n][d + 1], c0, c1, c2, c3, bp[n][0], bp[n][1]);
                    }
                }
            }
            cur = next;
        }
    }

    // the warps' parts meet: rows 2t, 2t+1 of each 8, dimensions D/8 * g + 2d, + 1 of tile d
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], 4);
            l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], 8);
            l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], 16);
            const int r = 8 * n + 2 * t + h;
            if (g == 0) {
                s_m[warp][r] = m[n][h];
                s_l[warp][r] = l[n][h];
            }
#pragma unroll
            for (int d = 0; d < kM; ++d)
                *reinterpret_cast<float2*>(&s_o[warp][r][D / 8 * g + 2 * d]) = make_float2(o[n][d][h] * vref, o[n][d][2 + h] * vref);
        }
    __syncthreads();
    const bool whole = chunk >= len;  // this CTA has every key
    for (int i = tid; i < kRows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        const int64_t row = first_row + r;
        if (row >= rows) continue;
        float top = s_m[0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
        const float mu = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(s_m[w][r] - mu);
            sum = fmaf(s_l[w][r], f, sum);
            const float4 v = *reinterpret_cast<const float4*>(&s_o[w][r][d]);
            acc.x = fmaf(v.x, f, acc.x);
            acc.y = fmaf(v.y, f, acc.y);
            acc.z = fmaf(v.z, f, acc.z);
            acc.w = fmaf(v.w, f, acc.w);
        }
        const bool none = top == -INFINITY && sum == 0.0f;
        const float inv = none ? 0.0f : __fdiv_rn(1.0f, sum);
        acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
        const float lse = none ? -INFINITY : top + log2f(sum);
        const int64_t at = (s.first + row / A.group) * A.heads + kvh * A.group + row % A.group;
        if (whole) {
            T* out = static_cast<T*>(A.out) + at * D + d;
            out[0] = iqq::from_f32<T>(acc.x);
            out[1] = iqq::from_f32<T>(acc.y);
            out[2] = iqq::from_f32<T>(acc.z);
            out[3] = iqq::from_f32<T>(acc.w);
            if (A.lse != nullptr && d == 0) A.lse[at] = lse / kLog2e;
        } else {
            *reinterpret_cast<float4*>(A.part + (at * A.splits + split) * D + d) = acc;
            if (d == 0) A.part_lse[at * A.splits + split] = lse;
        }
    }
}

// Joins a row's parts, each normalized and with its log-sum (base 2): a CTA a row and head, its
// warps taking the parts in turn.
template <class T, int D>
__global__ void __launch_bounds__(kThreads)
combine_kernel(const Kv8 C, const Args A)
{
    constexpr int kE = D / 32;
    __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t token = blockIdx.x, at = token * A.heads + blockIdx.y;
    const int b = iqq::seq_of_slot(C, token, 1, 1, 0);
    const Span s = iqq::span_of(C, b);
    if (token < s.first || token >= s.first + s.n) return;
    const int64_t len = s.len < C.capacity ? s.len : C.capacity;
    const int64_t chunk = chunk_of(len, A.splits);
    if (chunk >= len) return;  // written by its one CTA
    // parts that hold keys this token sees (the first always exists)
    const int64_t seen = max(int64_t{1}, min(len, s.start + (token - s.first) + 1));
    const int parts = static_cast<int>((seen + chunk - 1) / chunk);
    const float* lse = A.part_lse + at * A.splits;
    float m = -INFINITY, l = 0.0f, o[kE] = {};
    for (int p = warp; p < parts; p += kWarps) {
        const float x = lse[p];
        if (x == -INFINITY) continue;
        const float top = fmaxf(m, x);  // (a NaN part keeps m and makes the weight NaN)
        const float keep = m == -INFINITY ? 0.0f : ex2(m - top), w = ex2(x - (top == -INFINITY ? 0.0f : top));
        m = top;
        l = fmaf(l, keep, w);
        const float* v = A.part + (at * A.splits + p) * D + lane * kE;
#pragma unroll
        for (int e = 0; e < kE; ++e) o[e] = fmaf(o[e], keep, w * v[e]);
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) s_o[warp][lane * kE + e] = o[e];
    __syncthreads();
    const int d = threadIdx.x;
    if (d >= D) return;
    float top = s_m[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
    const float mu = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, acc = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(s_m[w] - mu);
        sum = fmaf(s_l[w], f, sum);
        acc = fmaf(s_o[w][d], f, acc);
    }
    const bool none = top == -INFINITY && sum == 0.0f;
    static_cast<T*>(A.out)[at * D + d] = iqq::from_f32<T>(none ? 0.0f : acc / sum);
    if (A.lse != nullptr && d == 0) A.lse[at] = none ? -INFINITY : (top + log2f(sum)) / kLog2e;
}

struct Plan {
    int row_tile;     // rows a CTA
    int64_t slots;    // row tiles of all sequences
    int splits;
};

// The launch goes by shapes alone (lengths are on the device).  Row tiles of 8 while a sequence's
// share of the tokens fits, else of 16.  Splits fill the machine about four CTAs an SM deep when
// every sequence is as long as the table is wide, but leave a CTA kMinChunk keys.
Plan plan_of(const iqq_kv8_cache* cache, const iqq_kv8_seqs* seqs, int64_t n_heads, int64_t n_tokens)
{
    Plan p;
    const int64_t group = n_heads / cache->n_kv_heads;
    const int64_t each = (n_tokens + seqs->n_seqs - 1) / seqs->n_seqs * group;
    p.row_tile = each <= 8 ? 8 : 16;
    p.slots = n_tokens * group / p.row_tile + seqs->n_seqs;
    const int64_t ctas = p.slots * cache->n_kv_heads, capacity = seqs->table_width * cache->page_size;
    const int64_t want = (4LL * iqq::sm_count() + ctas - 1) / ctas, most = (capacity + kMinChunk - 1) / kMinChunk;
    p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want, most, 1024})));
    return p;
}

template <class K>
iqq_status start(K kernel, dim3 grid, cudaStream_t st, const Kv8& C, const Args& A, uint32_t* flags)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if constexpr (std::is_invocable_v<K, Kv8, Args, uint32_t*>)
        cudaLaunchKernelEx(&cfg, kernel, C, A, flags);
    else
        cudaLaunchKernelEx(&cfg, kernel, C, A);
    return iqq::launch_status();
}

template <class T, int D>
iqq_status launch(const Kv8& C, const Args& A, const Plan& p, cudaStream_t st, uint32_t* flags)
{
    const dim3 grid(static_cast<unsigned>(p.slots), static_cast<unsigned>(p.splits), static_cast<unsigned>(C.heads));
    const iqq_status s = p.row_tile == 8 ? start(decode_kernel<T, D, 1>, grid, st, C, A, flags)
                                         : start(decode_kernel<T, D, 2>, grid, st, C, A, flags);
    if (s != IQQ_OK || p.splits == 1) return s;
    return start(combine_kernel<T, D>, dim3(static_cast<unsigned>(C.n_tokens), static_cast<unsigned>(A.heads)), st, C, A, flags);
}

bool shapes_ok(const iqq_kv8_cache* cache, const iqq_kv8_seqs* seqs, int64_t n_heads, int64_t n_tokens)
{
    return cache != nullptr && seqs != nullptr && cache->n_kv_heads >= 1 && n_heads >= 1 && n_heads <= 65535 &&
           n_heads % cache->n_kv_heads == 0 && n_tokens >= 1 && n_tokens <= 0x7fffffffLL && seqs->n_seqs >= 1 &&
           seqs->n_seqs <= (1LL << 24) && cache->page_size >= 1 && seqs->table_width >= 0;
}

}  // namespace

extern "C" size_t iqq_kv8_attention_workspace_bytes(const iqq_kv8_cache* cache, const iqq_kv8_seqs* seqs, int64_t n_heads,
                                                    int64_t n_tokens)
{
    if (!shapes_ok(cache, seqs, n_heads, n_tokens)) return 0;
    const Plan p = plan_of(cache, seqs, n_heads, n_tokens);
    if (p.splits == 1) return 0;
    return static_cast<size_t>(n_tokens) * n_heads * p.splits * (cache->head_dim + 1) * sizeof(float);
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
    const Plan p = plan_of(cache, seqs, n_heads, n_tokens);
    if (p.slots > 0x7fffffffLL) return IQQ_ERR_SHAPE;
    const size_t need = iqq_kv8_attention_workspace_bytes(cache, seqs, n_heads, n_tokens);
    if (q == nullptr || out == nullptr || (need > 0 && workspace == nullptr)) return IQQ_ERR_NULL;
    if (workspace_bytes < need) return IQQ_ERR_SHAPE;
    if (!iqq::aligned(q, 16) || !iqq::aligned(out, 16) || !iqq::aligned(lse, 4) || q_token_stride % 8 != 0 ||
        q_head_stride % 8 != 0 || !iqq::aligned(workspace, 16) || !iqq::aligned(d_flags, 4))
        return IQQ_ERR_ALIGN;
    Args A = {};
    A.q = q;
    A.out = out;
    A.lse = lse;
    A.q_token_stride = q_token_stride;
    A.q_head_stride = q_head_stride;
    A.heads = static_cast<int32_t>(n_heads);
    A.group = static_cast<int32_t>(n_heads / C.heads);
    A.splits = p.splits;
    A.scale = scale;
    A.part = static_cast<float*>(workspace);
    if (need > 0) A.part_lse = A.part + n_tokens * n_heads * p.splits * cache->head_dim;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool wide = cache->head_dim == 128;
    if (dtype == IQQ_BF16)
        return wide ? launch<__nv_bfloat16, 128>(C, A, p, st, d_flags) : launch<__nv_bfloat16, 64>(C, A, p, st, d_flags);
    return wide ? launch<__half, 128>(C, A, p, st, d_flags) : launch<__half, 64>(C, A, p, st, d_flags);
}

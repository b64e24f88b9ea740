// kv8_attention.cu -- causal attention over the paged int8 key/value cache, on sm_100a.
//
// For a row (a query token and head) with scores s_j = scale * q . k_j:
//     out = sum_j p_j v_j / sum_j p_j,  p_j = exp(s_j - m),
// in one pass over the keys with the running maximum m and sum of the softmax.  The rows of a
// sequence that share a key/value head are packed together (row r is token r / group, head
// r % group of the group), so a page is read once for all of them.
//
// decode kernel (few rows a sequence).  Bound by the cache's bytes.  One warp streams the pages'
// tiles into a ring of stages (cp.async.bulk, the scales beside them by cp.async); four warps
// take 16 keys of a stage each, straight into the operand registers of mma.m16n8k16:
//     S^T = K Q^T (16 keys x 8 rows),  O^T = V^T P^T (16 dimensions x 8 rows).
// The order of the dimensions in a dot product, and of the rows of V^T, is free, so each lane
// reads 16 contiguous bytes and nothing is transposed through shared memory; P^T goes from the
// accumulators' layout to the operand's by movmatrix.  int8 codes become binary16 exactly: the
// byte b of a code c, in the low byte of 0x6400, is the binary16 1152 + c after b ^= 0x80, and
// 1152 is subtracted.  Rows of q become binary16 exactly as well, by a power of two for each row
// that brings its largest value near 2^14 (values below 2^-38 of it round, which is beyond the
// binary32 sums).  The weights p_j are rounded to binary16, times the page's value scale over a
// power of two that follows the largest such scale: 2^-11 each, as fine as the output's type or
// finer.  The running maximum moves only when a score passes it by 2^8, so a block costs one vote.
//
// The keys of a sequence are split over CTAs (and the four warps of one) so that the machine is
// filled; partial results, each with its log-sum, meet in the workspace and combine_kernel joins
// them.
#include <math.h>

#include <algorithm>

#include "kv8.cuh"
#include "sm100.cuh"

namespace {

using iqq::Kv8;
using iqq::Span;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;       // that compute; one more warp loads
constexpr int kStageBytes = 16384;          // keys and values of a stage
constexpr int kStages = 4;
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

// The keys of a CTA: a sequence's length divided by the launch's splits, a multiple of every page size.
__device__ __forceinline__ int64_t chunk_of(int64_t len, int splits)
{
    const int64_t c = ((len + splits - 1) / splits + 127) / 128 * 128;
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

// Shared memory of the decode kernel.  A stage holds kKeys keys' codes, then their values', in
// the order of the keys, and the scales of each 16 keys.
template <int D, int NT>
struct Smem {
    static constexpr int kRows = 8 * NT, kKeys = kStageBytes / (2 * D);
    union {
        uint8_t stage[kStages][kStageBytes];
        float o[kWarps][kRows][D];  // the warps' parts, once the stages are done with
    };
    float ks[kStages][kKeys / 16], vs[kStages][kKeys / 16];
    int live[kStages];              // which 16 keys have a page, a bit each
    uint64_t full[kStages], empty[kStages];
    float m[kWarps][kRows], l[kWarps][kRows];
};

// Copies `bytes` (a multiple of 16) to shared memory, counted by the barrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void async_load4(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on the barrier when this thread's cp.async so far are done.
__device__ __forceinline__ void async_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// The loading warp: keys j0 .. j1-1 of sequence b, a stage at a time.  A lane takes the pieces of
// one page within a stage (kKeys or page_size keys, whichever is less), 32 pieces at a time.
template <int D, int NT>
__device__ __forceinline__ bool feed(Smem<D, NT>& S, const Kv8& C, int b, int kvh, int64_t j0, int64_t j1, uint32_t* flags)
{
    constexpr int kKeys = Smem<D, NT>::kKeys;
    const int lane = threadIdx.x & 31;
    const int piece = min(kKeys, 1 << C.page_log2), per = kKeys / piece;  // keys a piece, pieces a stage
    const int batch = 32 / per;                                         // stages whose pages are looked up at once
    const int stages = static_cast<int>((j1 - j0 + kKeys - 1) / kKeys);
    const auto page_of = [&](int st0) {
        const int64_t key = j0 + static_cast<int64_t>(st0) * kKeys + lane * piece;
        return key < j1 ? iqq::page_at(C, b, key >> C.page_log2) : -2;
    };
    int s = 0, issued = 0, page = page_of(0);
    uint32_t ph = 0;
    bool late = false;
    for (int st0 = 0; st0 < stages && !late; st0 += batch) {
        const int here = page;
        if (st0 + batch < stages) page = page_of(st0 + batch);
        if (here == -1) iqq::raise_flags(flags, IQQ_FLAG_BAD_INDEX);
        const uint32_t live = __ballot_sync(0xffffffffu, here >= 0);
        for (int i = 0; i < batch && st0 + i < stages; ++i) {
            late = !iqq::bar_wait(iqq::smem_u32(&S.empty[s]), ph ^ 1u);
            if (__any_sync(0xffffffffu, late)) break;
            const uint32_t bar = iqq::smem_u32(&S.full[s]);
            const uint32_t mine = (live >> (i * per)) & ((1u << per) - 1u);
            if (lane == 0) {
                uint32_t keys = 0;  // a bit for each 16 keys
                for (int u = 0; u < per; ++u)
                    if (mine >> u & 1u) keys |= ((1u << (piece / 16)) - 1u) << (u * (piece / 16));
                S.live[s] = static_cast<int>(keys);
                iqq::bar_expect(bar, static_cast<uint32_t>(__popc(mine)) * piece * D * 2);
            }
            __syncwarp();
            const int u = lane - i * per;
            if (u >= 0 && u < per && here >= 0) {
                const int64_t key = j0 + static_cast<int64_t>(st0) * kKeys + lane * piece;
                const int64_t cell = static_cast<int64_t>(here) * C.heads + kvh;
                const int64_t at = ((cell << C.page_log2) + (key & ((1 << C.page_log2) - 1))) * D;
                const uint32_t to = iqq::smem_u32(&S.stage[s][0]) + u * piece * D;
                bulk_load(to, C.codes[0] + at, piece * D, bar);
                bulk_load(to + kKeys * D, C.codes[1] + at, piece * D, bar);
                for (int k = 0; k < piece / 16; ++k) {
                    async_load4(iqq::smem_u32(&S.ks[s][u * (piece / 16) + k]), C.scales[0] + cell);
                    async_load4(iqq::smem_u32(&S.vs[s][u * (piece / 16) + k]), C.scales[1] + cell);
                }
            }
            async_arrive(bar);
            ++issued;
            if (++s == kStages) {
                s = 0;
                ph ^= 1u;
            }
        }
    }
    // every copy has landed (somebody waited for it) unless a wait ran out
    for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
        late |= !iqq::bar_wait(iqq::smem_u32(&S.full[i % kStages]), static_cast<uint32_t>(i / kStages) & 1u);
    return !late;
}

template <class T, int D, int NT>
__global__ void __launch_bounds__(kThreads + 32, NT == 1 ? 3 : 2)
decode_kernel(const Kv8 C, const Args A, uint32_t* __restrict__ flags)
{
    constexpr int kRows = 8 * NT, kK = D / 16, kM = D / 16;  // k steps of S, 16-row tiles of O^T
    constexpr int kKeys = Smem<D, NT>::kKeys;
    extern __shared__ __align__(128) uint8_t raw[];
    Smem<D, NT>& S = *reinterpret_cast<Smem<D, NT>*>(raw);
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

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            iqq::bar_init(iqq::smem_u32(&S.full[i]), 33);        // expect_tx, and the lanes' scales
            iqq::bar_init(iqq::smem_u32(&S.empty[i]), kWarps);
        }
        iqq::bar_init_fence();
    }
    __syncthreads();
    if (warp == kWarps) {
        if (j1 > j0 && !feed<D, NT>(S, C, b, kvh, j0, j1, flags)) iqq::raise_flags(flags, IQQ_FLAG_WAIT_TIMEOUT);
        __syncwarp();
        __syncthreads();
        __syncthreads();
        return;
    }

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

    const int stages = j1 > j0 ? static_cast<int>((j1 - j0 + kKeys - 1) / kKeys) : 0;
    int st = 0;
    uint32_t ph = 0;
    for (int i = 0; i < stages; ++i) {
        const bool late = !iqq::bar_wait(iqq::smem_u32(&S.full[st]), ph);
        if (__any_sync(0xffffffffu, late)) {
            iqq::raise_flags(flags, IQQ_FLAG_WAIT_TIMEOUT);
            break;
        }
        const int live = S.live[st];
#pragma unroll
        for (int u = 0; u < kKeys / (16 * kWarps); ++u) {
            const int at = u * kWarps + warp;        // which 16 keys of the stage
            const int key0 = i * kKeys + 16 * at;    // from j0
            if (live >> at & 1) {
                const float ks = S.ks[st][at], vs = S.vs[st][at];
                const uint8_t* kp = &S.stage[st][16 * at * D + g * D + 16 * t];
                const uint8_t* vp = &S.stage[st][kKeys * D + 16 * at * D + 2 * t * D + D / 8 * g];
                float x[NT][4], x2[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[n][e] = x2[n][e] = 0.0f;
                // keys g and g+8, dimensions 16t .. of each 64; two chains of sums
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    const uint4 k0 = *reinterpret_cast<const uint4*>(kp + 64 * h);
                    const uint4 k1 = *reinterpret_cast<const uint4*>(kp + 8 * D + 64 * h);
                    const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int j = 4 * h + c;
                        const uint32_t a0 = codes_even(w0[c]), a2 = codes_odd(w0[c]);
                        const uint32_t a1 = codes_even(w1[c]), a3 = codes_odd(w1[c]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma(c & 1 ? x2[n] : x[n], a0, a1, a2, a3, bq[n][j][0], bq[n][j][1]);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[n][e] += x2[n][e];
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
                // keys 2t, 2t+1, 2t+8, 2t+9, dimensions D/8 * g ..: 16-row tile d is bytes 2d, 2d+1
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    uint2 v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = *reinterpret_cast<const uint2*>(vp + ((e & 1) + 8 * (e >> 1)) * D + 8 * h);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t w0 = c ? v[0].y : v[0].x, w1 = c ? v[1].y : v[1].x;
                        const uint32_t w2 = c ? v[2].y : v[2].x, w3 = c ? v[3].y : v[3].x;
                        const uint32_t lo01 = __byte_perm(w0, w1, 0x5410), hi01 = __byte_perm(w0, w1, 0x7632);
                        const uint32_t lo23 = __byte_perm(w2, w3, 0x5410), hi23 = __byte_perm(w2, w3, 0x7632);
                        const uint32_t a0 = codes_even(lo01), a1 = codes_odd(lo01), a2 = codes_even(lo23), a3 = codes_odd(lo23);
                        const uint32_t c0 = codes_even(hi01), c1 = codes_odd(hi01), c2 = codes_even(hi23), c3 = codes_odd(hi23);
                        const int d = 4 * h + 2 * c;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma(o[n][d], a0, a1, a2, a3, bp[n][0], bp[n][1]);
                            mma(o[n][d + 1], c0, c1, c2, c3, bp[n][0], bp[n][1]);
                        }
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) iqq::bar_arrive(iqq::smem_u32(&S.empty[st]));
        if (++st == kStages) {
            st = 0;
            ph ^= 1u;
        }
    }
    __syncthreads();  // the stages' memory is free

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
                S.m[warp][r] = m[n][h];
                S.l[warp][r] = l[n][h];
            }
#pragma unroll
            for (int d = 0; d < kM; ++d)
                *reinterpret_cast<float2*>(&S.o[warp][r][D / 8 * g + 2 * d]) = make_float2(o[n][d][h] * vref, o[n][d][2 + h] * vref);
        }
    __syncthreads();
    const bool whole = chunk >= len;  // this CTA has every key
    for (int i = tid; i < kRows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        const int64_t row = first_row + r;
        if (row >= rows) continue;
        float top = S.m[0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, S.m[w][r]);
        const float mu = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(S.m[w][r] - mu);
            sum = fmaf(S.l[w][r], f, sum);
            const float4 v = *reinterpret_cast<const float4*>(&S.o[w][r][d]);
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
    const int64_t want = (8LL * iqq::sm_count() + ctas - 1) / ctas, most = (capacity + kMinChunk - 1) / kMinChunk;
    p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want, most, 1024})));
    return p;
}

template <class K>
iqq_status start(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, const Kv8& C, const Args& A, uint32_t* flags)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
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

template <class T, int D, int NT>
iqq_status start_decode(const Kv8& C, const Args& A, const Plan& p, cudaStream_t st, uint32_t* flags)
{
    static std::atomic<uint64_t> done{0};
    constexpr size_t smem = sizeof(Smem<D, NT>);
    const iqq_status s = iqq::opt_in_smem(reinterpret_cast<const void*>(decode_kernel<T, D, NT>), smem, done);
    if (s != IQQ_OK) return s;
    const dim3 grid(static_cast<unsigned>(p.slots), static_cast<unsigned>(p.splits), static_cast<unsigned>(C.heads));
    return start(decode_kernel<T, D, NT>, grid, kThreads + 32, smem, st, C, A, flags);
}

template <class T, int D>
iqq_status launch(const Kv8& C, const Args& A, const Plan& p, cudaStream_t st, uint32_t* flags)
{
    const iqq_status s = p.row_tile == 8 ? start_decode<T, D, 1>(C, A, p, st, flags) : start_decode<T, D, 2>(C, A, p, st, flags);
    if (s != IQQ_OK || p.splits == 1) return s;
    return start(combine_kernel<T, D>, dim3(static_cast<unsigned>(C.n_tokens), static_cast<unsigned>(A.heads)), kThreads, 0,
                 st, C, A, flags);
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

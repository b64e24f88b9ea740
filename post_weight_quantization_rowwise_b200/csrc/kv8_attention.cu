// kv8_attention.cu -- causal attention over the paged int8 key/value cache, on sm_100a.
//
// For a row (a query token and head) with scores s_j = scale * q . k_j:
//     out = sum_j p_j v_j / sum_j p_j,  p_j = exp(s_j - m),
// in one pass over the keys with the running maximum m and sum of the softmax.  The rows of a
// sequence that share a key/value head are packed together (row r is token r / group, head
// r % group of the group), so a page is read once for all of them.
//
// decode kernel (few rows a sequence).  Bound by the cache's bytes.  One warp streams the pages'
// tiles into a ring of stages (TMA, the scales beside them by cp.async); four warps
// take 32 keys of a stage each, straight into the operand registers of mma.m16n8k16:
//     S^T = K Q^T (16 keys x 8 rows),  O^T = V^T P^T (16 dimensions x 8 rows).
// The order of the dimensions in a dot product, and of the rows of V^T, is free, so each lane
// reads 16 contiguous bytes and nothing is transposed through shared memory; P^T goes from the
// accumulators' layout to the operand's by movmatrix.  int8 codes become binary16 exactly: the
// byte b of a code c, in the low byte of 0x6400, is the binary16 1152 + c after b ^= 0x80, and
// 1152 is subtracted.  Rows of q become binary16 exactly as well, by a power of two for each row
// that brings its largest value near 2^14 (values below 2^-38 of it round, which is beyond the
// binary32 sums).  With vs = f 2^v the page's value scale, f from 1/2 to 1, the weights that meet the
// codes are f 2^(y - m), y = s log2(e) + v, rounded to binary16: 2^-11 of each, as fine as the output's
// type or finer.  m is the running maximum of y less 7 (see kLift), so large values without weight cost
// the others no bits; it moves only when a weight passes 2^15, so a block costs one vote.  The
// denominator is the sum of 2^(y - m) 2^-v, in binary32.
//
// Every launch is one wave of CTAs, and each takes an equal share of the work: the stages of all
// sequences, heads and row tiles laid end to end, in an order that every CTA works out from the
// lengths by one scan.  So a ragged batch, one long sequence and many short ones all fill the
// machine evenly.  A tile that lies in one share is finished there; of the others each share
// leaves a part, normalized and with its log-sum, in the workspace (two a CTA at most: where its
// share begins and where it ends), and combine_kernel joins them.  Where the tables are short and the
// tiles few, each CTA takes a whole tile instead: no parts, no workspace, one launch.
//
// Measured with inputs larger than L2: 32 sequences of 4096 tokens, 32 heads over 32 of 128 dimensions
// 168 us (6.4 TB/s of 6.55); 64 up to 8000, 32 over 8: 97 us (5.5); one of 131000, 32 over 4: 37 us
// (3.6; the scan, the ring's filling and the joining launch are 10 us of any call).
#include <math.h>

#include <algorithm>

#include "kv8.cuh"
#include "sm100.cuh"

namespace {

using iqq::ex2;
using iqq::kLog2e;
using iqq::kNone;
using iqq::Kv8;
using iqq::pack_h2;
using iqq::Span;
using iqq::sub_h2;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;       // that compute; one more warp loads
constexpr int kKeys = 128;                  // keys of a stage: 32 a warp
constexpr int kMaxCtas = 1024;

struct Args : iqq::Attend {
    // [gridDim.x]; parts are [gridDim.x][2][row tile][head_dim], log-sums [..][2][row tile].  Null: a tile a CTA.
    struct Mark* marks;
};

// The launch's stages in equal shares: `each`, and one more for the first `more` CTAs.
struct Shares {
    int64_t each;
    int32_t more;
    __device__ __forceinline__ Shares() {}
    __device__ __forceinline__ Shares(int64_t total, int32_t ctas)
    {
        if (total >> 31 == 0) {  // (64-bit division is a long call)
            each = static_cast<uint32_t>(total) / static_cast<uint32_t>(ctas);
        } else {
            each = total / ctas;
        }
        more = static_cast<int32_t>(total - each * ctas);
    }
    __device__ __forceinline__ int64_t start(int c) const { return each * c + min(c, more); }
    __device__ __forceinline__ bool empty(int c) const { return each == 0 && c >= more; }
};

// What a CTA's share begins in: the tile (sequence, key/value head, row tile) whose stages are
// t0 .. t1-1 of the launch's.
struct Mark {
    int64_t t0, t1;
    Shares shares;
    int32_t token, head, row0, rows;  // the sequence's first packed row; the tile's first row, and how many
};

// A sequence as the launch sees it.  (n_tokens * heads < 2^31, so a sequence's rows and, with its
// length below 2^31, its stages fit 32 bits; the stages of all its tiles need not.)
template <int ROWS>
struct Seq {
    Span s;
    int32_t rows, tiles, len, stages;
    int64_t all;  // stages of every head and row tile
    __device__ __forceinline__ Seq(const Kv8& C, int b, int group)
    {
        s = iqq::span_of(C, b);
        rows = s.n * group;  // 0 for a bad span
        tiles = (rows + ROWS - 1) / ROWS;
        len = static_cast<int32_t>(s.len < C.capacity ? s.len : C.capacity);
        // One more than the keys fill, the first: what a tile costs beside its keys (its rows of q,
        // joining the warps' parts, storing) is about a stage's time, and without it CTAs whose share
        // is many short sequences finish last (64 sequences of 50 to 8000 tokens: SMs apart by 20%).
        // It also is the one stage of a sequence without keys, whose rows get zeros.
        stages = 1 + static_cast<int32_t>((static_cast<uint32_t>(max(len, 0)) + kKeys - 1) / kKeys);
        all = static_cast<int64_t>(tiles) * stages * C.heads;
    }
    // Tile and stage within it of the sequence's stage `at`.
    __device__ __forceinline__ void place(int64_t at, int32_t& head, int32_t& row_tile, int32_t& stage) const
    {
        int64_t tile;
        if (at >> 31 == 0) tile = static_cast<uint32_t>(at) / static_cast<uint32_t>(stages);
        else tile = at / stages;
        stage = static_cast<int32_t>(at - tile * stages);
        head = static_cast<int32_t>(static_cast<uint32_t>(tile) / static_cast<uint32_t>(tiles));  // (heads * tiles < 2^31)
        row_tile = static_cast<int32_t>(tile - static_cast<int64_t>(head) * tiles);
    }
};

// Bytes 0 and 2, and bytes 1 and 3, of four codes as binary16 pairs.
__device__ __forceinline__ uint32_t codes_even(uint32_t w) { return sub_h2((w & 0x00ff00ffu) ^ 0x64806480u, 0x64806480u); }
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) { return codes_even(w >> 8); }

__device__ __forceinline__ uint32_t transpose8(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Shared memory of the decode kernel.  A stage holds kKeys keys' codes, then their values', in
// the order of the keys, as rows of 128 bytes with TMA's 128-byte swizzle (16-byte unit c of row r
// at c ^ (r & 7)), so the operand reads below meet no bank twice; and the scales of each 16 keys.
template <int D, int NT>
struct Smem {
    static constexpr int kRows = 8 * NT, kStages = D == 128 ? (NT == 1 ? 2 : 3) : 4, kHalf = kKeys * D;
    uint8_t stage[kStages][2 * kHalf];
    float4 o[2][NT * D / 16][32];   // accumulators of two warps, as their lanes hold them
    float m[2][kRows], l[2][kRows];
    float ks[kStages][kKeys / 16], vs[kStages][kKeys / 16];
    int live[kStages];              // which 16 keys have a page, a bit each
    uint64_t full[kStages], empty[kStages];
    int64_t scan[kWarps + 1], offset, left;
    int first, abort;
};

// The stages from..to-1 (of its `stages`) of one tile: a CTA's work between two stores.
struct Piece {
    int32_t b, head, row_tile, from, to;
    __device__ __forceinline__ int64_t first_key() const { return static_cast<int64_t>(max(from - 1, 0)) * kKeys; }
    __device__ __forceinline__ int64_t end_key() const { return static_cast<int64_t>(to - 1) * kKeys; }
};

// A CTA's walk through its share: sequence b, `at` stages into it, `left` to go.
template <int ROWS>
struct Walk {
    int b;
    int64_t at, left;
    __device__ __forceinline__ bool next(const Kv8& C, int group, Piece& P)
    {
        while (left > 0 && b < C.n_seqs) {
            const Seq<ROWS> q(C, b, group);
            if (at >= q.all) {
                at = 0;
                ++b;
                continue;
            }
            P.b = b;
            q.place(at, P.head, P.row_tile, P.from);
            P.to = left < q.stages - P.from ? P.from + static_cast<int32_t>(left) : q.stages;
            at += P.to - P.from;
            left -= P.to - P.from;
            return true;
        }
        return false;
    }
};


// The loading warp's ring, over all pieces of its share.
template <int D, int NT>
struct Feed {
    static constexpr int kStages = Smem<D, NT>::kStages;
    Smem<D, NT>& S;
    int s = 0;
    uint32_t ph = 0;
    int64_t issued = 0;

    // Keys j0 .. j1-1 of sequence b.  A lane takes what a stage has of one page (kKeys or
    // page_size keys, whichever is less), 32 of these at a time.
    __device__ __forceinline__ bool keys(const CUtensorMap* kmap, const CUtensorMap* vmap, const Kv8& C, int b, int kvh,
                                         int64_t j0, int64_t j1, uint32_t* flags)
    {
        const int lane = threadIdx.x & 31;
        const int piece = min(kKeys, 1 << C.page_log2), per = kKeys / piece;  // keys of a lane, lanes of a stage
        const int batch = 32 / per;                                           // stages looked up at once
        const int64_t stages = (j1 - j0 + kKeys - 1) / kKeys;
        const auto page_of = [&](int64_t st0) {
            const int64_t key = j0 + st0 * kKeys + lane * piece;
            return key < j1 ? iqq::page_at(C, b, key >> C.page_log2) : -2;
        };
        int page = page_of(0);
        for (int64_t st0 = 0; st0 < stages; st0 += batch) {
            const int here = page;
            if (st0 + batch < stages) page = page_of(st0 + batch);
            if (here == -1) iqq::raise_flags(flags, IQQ_FLAG_BAD_INDEX);
            const uint32_t live = __ballot_sync(0xffffffffu, here >= 0);
            for (int i = 0; i < batch && st0 + i < stages; ++i) {
                const bool late = !iqq::bar_wait(iqq::smem_u32(&S.empty[s]), ph ^ 1u);
                if (__any_sync(0xffffffffu, late)) return false;
                const uint32_t bar = iqq::smem_u32(&S.full[s]);
                const uint32_t mine = (live >> (i * per)) & (per == 32 ? 0xffffffffu : (1u << per) - 1u);
                if (lane == 0) {
                    uint32_t with = 0;  // a bit for each 16 keys
                    for (int u = 0; u < per; ++u)
                        if (mine >> u & 1u) with |= ((1u << (piece / 16)) - 1u) << (u * (piece / 16));
                    S.live[s] = static_cast<int>(with);
                    iqq::bar_expect(bar, static_cast<uint32_t>(__popc(mine)) * piece * D * 2);
                }
                __syncwarp();
                const int u = lane - i * per;
                if (u >= 0 && u < per && here >= 0) {
                    const int64_t key = j0 + st0 * kKeys + lane * piece;
                    const int64_t cell = static_cast<int64_t>(here) * C.heads + kvh;
                    // the map's rows are 128 bytes; a page's 16 keys are whole groups of eight
                    const int row = static_cast<int>(((cell << C.page_log2) + (key & ((1 << C.page_log2) - 1))) * D / 128);
                    const uint32_t to = iqq::smem_u32(&S.stage[s][0]) + u * piece * D;
                    iqq::tma_load(to, kmap, 0, row, bar);
                    iqq::tma_load(to + Smem<D, NT>::kHalf, vmap, 0, row, bar);
                    for (int k = 0; k < piece / 16; ++k) {
                        iqq::async_load4(iqq::smem_u32(&S.ks[s][u * (piece / 16) + k]), C.scales[0] + cell);
                        iqq::async_load4(iqq::smem_u32(&S.vs[s][u * (piece / 16) + k]), C.scales[1] + cell);
                    }
                }
                iqq::async_arrive(bar);
                ++issued;
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        return true;
    }

    // Every copy has landed (somebody waited for it) unless a wait ran out.
    __device__ __forceinline__ bool drain()
    {
        bool ok = true;
        for (int64_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
            ok &= iqq::bar_drain(iqq::smem_u32(&S.full[i % kStages]), static_cast<uint32_t>(i / kStages) & 1u);
        return ok;
    }
};

// The four computing warps.
__device__ __forceinline__ void meet() { asm volatile("barrier.sync 1, 128;" ::: "memory"); }

template <class T, int D, int NT>
__global__ void __launch_bounds__(kThreads + 32, NT == 1 ? 3 : 2)
decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const Kv8 C, const Args A,
              uint32_t* __restrict__ flags)
{
    using Sm = Smem<D, NT>;
    constexpr int kRows = Sm::kRows, kK = D / 16, kM = D / 16;  // k steps of S, 16-row tiles of O^T
    extern __shared__ __align__(1024) uint8_t raw[];
    Sm& S = *reinterpret_cast<Sm*>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    if (tid == 0) {
        for (int i = 0; i < Sm::kStages; ++i) {
            iqq::bar_init(iqq::smem_u32(&S.full[i]), 33);        // expect_tx, and the lanes' scales
            iqq::bar_init(iqq::smem_u32(&S.empty[i]), kWarps);
        }
        iqq::bar_init_fence();
        S.first = -1;
        S.abort = 0;
        iqq::tma_prefetch_map(&kmap);
        iqq::tma_prefetch_map(&vmap);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // Where this CTA's share begins: a scan over the sequences, a run of them a thread, in stages (or in
    // tiles, where a CTA takes one).
    Walk<kRows> walk;
    {
        const bool whole = A.marks == nullptr;
        const auto parts_of = [&](const Seq<kRows>& q) { return whole ? static_cast<int64_t>(q.tiles) * C.heads : q.all; };
        const int run = (C.n_seqs + kThreads + 31) / (kThreads + 32), b0 = min(C.n_seqs, tid * run), b1 = min(C.n_seqs, b0 + run);
        int64_t sum = 0;
        bool bad = false;
        for (int b = b0; b < b1; ++b) {
            const Seq<kRows> q(C, b, A.group);
            sum += parts_of(q);
            bad |= !q.s.ok || q.s.len > C.capacity;
        }
        if (bad && blockIdx.x == 0) iqq::raise_flags(flags, IQQ_FLAG_BAD_INDEX);
        int64_t before = sum;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int64_t v = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += v;
        }
        if (lane == 31) S.scan[warp] = before;
        __syncthreads();
        int64_t total = 0;
#pragma unroll
        for (int w = 0; w <= kWarps; ++w) {
            if (w < warp) before += S.scan[w];
            total += S.scan[w];
        }
        before -= sum;
        const Shares shares(total, gridDim.x);
        const int64_t start = whole ? blockIdx.x : shares.start(blockIdx.x);
        if (start >= before && start < before + sum) {
            int64_t at = start - before;
            int b = b0;
            Seq<kRows> q(C, b, A.group);
            while (at >= parts_of(q)) {
                at -= parts_of(q);
                q = Seq<kRows>(C, ++b, A.group);
            }
            S.first = b;
            S.offset = whole ? at * q.stages : at;
            S.left = whole ? q.stages : shares.start(blockIdx.x + 1) - start;
            if (!whole) {
                Mark M;
                int32_t stage, row_tile;
                q.place(at, M.head, row_tile, stage);
                M.t0 = start - stage;
                M.t1 = M.t0 + q.stages;
                M.shares = shares;
                M.token = q.s.first;
                M.row0 = row_tile * kRows;
                M.rows = min(kRows, q.rows - M.row0);
                A.marks[blockIdx.x] = M;
            }
        } else if (!whole && start >= total && tid == 0) {  // more CTAs than stages: an empty share at the end
            A.marks[blockIdx.x].t0 = A.marks[blockIdx.x].t1 = start;
        }
        __syncthreads();
        walk.b = S.first;
        walk.at = S.offset;
        walk.left = walk.b < 0 ? 0 : S.left;
    }

    Piece P;
    if (warp == kWarps) {
        Feed<D, NT> feed{S};
        bool ok = true;
        while (ok && walk.next(C, A.group, P)) {
            const Seq<kRows> q(C, P.b, A.group);
            const int last_row = min(q.rows, (P.row_tile + 1) * kRows) - 1;
            const int64_t seen = min(static_cast<int64_t>(q.len), q.s.start + last_row / A.group + 1);
            const int64_t j0 = P.first_key(), j1 = min(seen, P.end_key());
            if (j1 > j0) ok = feed.keys(&kmap, &vmap, C, P.b, P.head, j0, j1, flags);
        }
        if (!feed.drain() || !ok) iqq::raise_flags(flags, IQQ_FLAG_WAIT_TIMEOUT);
        return;
    }

    int st = 0, turn = 0;
    uint32_t ph = 0;
    while (walk.next(C, A.group, P)) {
    const Seq<kRows> Q(C, P.b, A.group);
    const Span s = Q.s;
    const int kvh = P.head;
    const int32_t rows = Q.rows, first_row = P.row_tile * kRows;
    const int64_t len = Q.len;
    const int32_t last_row = min(rows, first_row + kRows) - 1;
    const int64_t seen = min(len, s.start + last_row / A.group + 1);  // keys this tile's rows can see at all
    const int64_t j0 = P.first_key(), j1 = min(seen, P.end_key());

    // the rows of q this lane feeds (row g of each 8), as binary16 times 2^-e
    uint32_t bq[NT][kK][2];
    float unscale[NT][2];  // of rows 2t, 2t+1: scale * 2^e * log2(e)
    int limit[NT][2];      // keys of this CTA (from j0) below it are seen
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int32_t r = first_row + 8 * n + g;
        float v[D / 4];
        if (r < rows) {
            const int32_t token = r / A.group;
            const T* q = static_cast<const T*>(A.q) + (s.first + token) * A.q_token_stride +
                         (kvh * A.group + r - token * A.group) * A.q_head_stride;
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float u[8];
                    iqq::load8(q + D / 4 * t + 16 * i + 8 * h, u);
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
        const int e = iqq::row_exponent(top);
        const float down = iqq::power_of_two(-e), up = iqq::power_of_two(e);
#pragma unroll
        for (int j = 0; j < kK; ++j) {
            // dimensions D/4 t + 4 j + {0, 2} and {1, 3}: as codes_even and codes_odd
            const int i = 4 * j;
            bq[n][j][0] = pack_h2(v[i] * down, v[i + 2] * down);
            bq[n][j][1] = pack_h2(v[i + 1] * down, v[i + 3] * down);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            unscale[n][h] = __shfl_sync(0xffffffffu, up, (2 * t + h) * 4) * A.scale * kLog2e;
            const int32_t row = first_row + 8 * n + 2 * t + h;
            const int64_t lim = row < rows ? min(len, s.start + row / A.group + 1) - j0 : 0x7fffffff;  // (padding: no mask)
            limit[n][h] = static_cast<int>(max(int64_t{0}, min(lim, int64_t{0x7fffffff})));
        }
    }
    // below this key (from j0) no row of the tile needs a mask
    const int64_t clear64 = min(len, s.start + first_row / A.group + 1) - j0;
    const int clear = static_cast<int>(max(int64_t{0}, min(clear64, int64_t{0x7fffffff})));

    float m[NT][2], l[NT][2], o[NT][kM][4];
    uint32_t sees = 0;  // rows that had a key here, a bit each
    int hi = 86;  // biased exponent of the largest value scale so far
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            m[n][h] = kNone;
            l[n][h] = 0.0f;
        }
#pragma unroll
        for (int d = 0; d < kM; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][d][i] = 0.0f;
    }

    const int64_t stages = j1 > j0 ? (j1 - j0 + kKeys - 1) / kKeys : 0;
    for (int64_t i = 0; i < stages; ++i) {
        const bool late = !iqq::bar_wait(iqq::smem_u32(&S.full[st]), ph);
        if (__any_sync(0xffffffffu, late)) {
            S.abort = 1;
            break;
        }
        const int key0 = static_cast<int>(i) * kKeys + 32 * warp;  // from j0
        const uint8_t* kp = &S.stage[st][32 * warp * D];
        const uint8_t* vp = kp + Sm::kHalf;
        // scores: x[u][n] of keys 16u + g and 16u + g + 8 (elements 0, 1 and 2, 3), rows 2t, 2t+1
        const int live = S.live[st] >> (2 * warp);
        float x[2][NT][4], vf[2], rv[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[u][n][e] = 0.0f;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                // keys g and g+8, dimensions D/4 t ..
                uint4 k0, k1;
                const uint8_t* k = kp + 16 * u * D;
                if constexpr (D == 128) {
                    k0 = *reinterpret_cast<const uint4*>(k + g * 128 + (((2 * t + h) ^ g) << 4));
                    k1 = *reinterpret_cast<const uint4*>(k + g * 128 + (((2 * t + h) ^ g) << 4) + 1024);
                } else {  // two keys a row of 128 bytes
                    k0 = *reinterpret_cast<const uint4*>(k + (g >> 1) * 128 + ((((g & 1) * 4 + t) ^ (g >> 1)) << 4));
                    k1 = *reinterpret_cast<const uint4*>(k + (4 + (g >> 1)) * 128 + ((((g & 1) * 4 + t) ^ (4 + (g >> 1))) << 4));
                }
                const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t a0 = codes_even(w0[c]), a2 = codes_odd(w0[c]);
                    const uint32_t a1 = codes_even(w1[c]), a3 = codes_odd(w1[c]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma(x[u][n], a0, a1, a2, a3, bq[n][4 * h + c][0], bq[n][4 * h + c][1]);
                }
            }
            const float ks = S.ks[st][2 * warp + u], vs = live >> u & 1 ? S.vs[st][2 * warp + u] : 1.0f;
            int exp = static_cast<int>(__float_as_uint(vs) >> 23);  // of vs = vf 2^(exp - 126)
            vf[u] = __uint_as_float((__float_as_uint(vs) & 0x007fffffu) | 0x3f000000u);
            if (vs >= iqq::kTinyScale) {  // (all of this is the same in all lanes)
                hi = max(hi, exp);
            } else {
                // Codes of a scale that counts as 0 have no part in the sums, so any scale does in their
                // weights, if it neither moves m above what other pages need (2^-40) nor takes the weights
                // out of binary32 beside the largest scale (2^-100 of it).
                exp = max(86, hi - 100);
                vf[u] = 0.0f;
            }
            rv[u] = __uint_as_float(static_cast<uint32_t>(253 - exp) << 23);
            const float v = vs == vs ? static_cast<float>(exp - 126) : vs;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[u][n][e] = fmaf(x[u][n][e], unscale[n][e & 1] * ks, v);
        }
        const bool masked = key0 + 32 > clear || (live & 3) != 3;
        if (masked) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bool dead = !(live >> u & 1);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (dead || key0 + 16 * u + g + (e & 2) * 4 >= limit[n][e & 1]) x[u][n][e] = -INFINITY;
                        else sees |= 1u << (2 * n + (e & 1));
            }
        } else {
            sees = ~0u;
        }
        bool moved = false;
        float top[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                top[n][h] = fmaxf(fmaxf(x[0][n][h], x[0][n][2 + h]), fmaxf(x[1][n][h], x[1][n][2 + h]));
                moved |= top[n][h] > m[n][h] + (iqq::kLift + iqq::kMove);
            }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v = fmaxf(top[n][h] - iqq::kLift, m[n][h]);
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    const float root = ex2(0.5f * (m[n][h] - v)), f = root * root;
                    m[n][h] = v;
                    l[n][h] = l[n][h] * root * root;  // (f may be below binary32, where zero pages made l large)
#pragma unroll
                    for (int d = 0; d < kM; ++d) {
                        o[n][d][h] *= f;
                        o[n][d][2 + h] *= f;
                    }
                }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t bp[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = ex2(x[u][n][e] - m[n][e & 1]);
                l[n][0] = fmaf(p[0] + p[2], rv[u], l[n][0]);
                l[n][1] = fmaf(p[1] + p[3], rv[u], l[n][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] *= vf[u];
                bp[n][0] = transpose8(pack_h2(p[0], p[1]));
                bp[n][1] = transpose8(pack_h2(p[2], p[3]));
            }
            // keys 2t, 2t+1, 2t+8, 2t+9, dimensions D/8 g ..: 16-row tile d is bytes 2d, 2d+1
            uint32_t v[4][D / 32];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint8_t* w = vp + 16 * u * D;
                if constexpr (D == 128) {
                    const int r = 2 * t + (e & 1);
                    const uint4 c = *reinterpret_cast<const uint4*>(w + (r + 8 * (e >> 1)) * 128 + ((g ^ r) << 4));
                    v[e][0] = c.x; v[e][1] = c.y; v[e][2] = c.z; v[e][3] = c.w;
                } else {
                    const int r = t + 4 * (e >> 1);
                    const uint2 c = *reinterpret_cast<const uint2*>(w + r * 128 + ((((e & 1) * 4 + (g >> 1)) ^ r) << 4) + 8 * (g & 1));
                    v[e][0] = c.x; v[e][1] = c.y;
                }
            }
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const uint32_t lo01 = __byte_perm(v[0][c], v[1][c], 0x5410), hi01 = __byte_perm(v[0][c], v[1][c], 0x7632);
                const uint32_t lo23 = __byte_perm(v[2][c], v[3][c], 0x5410), hi23 = __byte_perm(v[2][c], v[3][c], 0x7632);
                const uint32_t a0 = codes_even(lo01), a1 = codes_odd(lo01), a2 = codes_even(lo23), a3 = codes_odd(lo23);
                const uint32_t c0 = codes_even(hi01), c1 = codes_odd(hi01), c2 = codes_even(hi23), c3 = codes_odd(hi23);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma(o[n][2 * c], a0, a1, a2, a3, bp[n][0], bp[n][1]);
                    mma(o[n][2 * c + 1], c0, c1, c2, c3, bp[n][0], bp[n][1]);
                }
            }
        }
        __syncwarp();
        if (lane == 0) iqq::bar_arrive(iqq::smem_u32(&S.empty[st]));
        if (++st == Sm::kStages) {
            st = 0;
            ph ^= 1u;
        }
    }

    // the warps' parts meet: 2 and 3 with 0 and 1, then 1 with 0; lane g, t holds rows 2t, 2t+1 of
    // each 8, dimensions D/8 g + 2d, + 1 of tile d
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // Keys without a weight: next to nothing, lost in any other sum.  Where all scores of a row are
            // -Inf it stays the sum, with m still kNone.
            if (l[n][h] == 0.0f && (sees >> (2 * n + h) & 1)) l[n][h] = 0x1p-149f;
            l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], 4);
            l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], 8);
            l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], 16);
        }
    bool stop = false;
#pragma unroll
    for (int step = 2; step > 0; step /= 2) {
        if (warp >= step && warp < 2 * step) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (g == 0) {
                        S.m[warp - step][8 * n + 2 * t + h] = m[n][h];
                        S.l[warp - step][8 * n + 2 * t + h] = l[n][h];
                    }
#pragma unroll
                for (int d = 0; d < kM; ++d)
                    S.o[warp - step][n * kM + d][lane] = make_float4(o[n][d][0], o[n][d][1], o[n][d][2], o[n][d][3]);
            }
        }
        meet();
        // All four warps stop together: what they set before this barrier they see here, and none gets past the
        // next one to set it for another piece before all have looked.
        if (step == 2) stop = S.abort != 0;
        if (stop) break;
        if (warp < step) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float own[2], other[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float mo = S.m[warp][8 * n + 2 * t + h], v = fmaxf(m[n][h], mo);
                    const float r = ex2(0.5f * (m[n][h] - v)), ro = ex2(0.5f * (mo - v));
                    l[n][h] = l[n][h] * r * r + S.l[warp][8 * n + 2 * t + h] * ro * ro;
                    m[n][h] = v;
                    own[h] = r * r;
                    other[h] = ro * ro;
                }
#pragma unroll
                for (int d = 0; d < kM; ++d) {
                    const float4 v = S.o[warp][n * kM + d][lane];
                    o[n][d][0] = fmaf(o[n][d][0], own[0], v.x * other[0]);
                    o[n][d][1] = fmaf(o[n][d][1], own[1], v.y * other[1]);
                    o[n][d][2] = fmaf(o[n][d][2], own[0], v.z * other[0]);
                    o[n][d][3] = fmaf(o[n][d][3], own[1], v.w * other[1]);
                }
            }
        }
        meet();
    }
    if (stop) {
        iqq::raise_flags(flags, IQQ_FLAG_WAIT_TIMEOUT);
        break;
    }
    if (warp == 0) {
        const bool whole = P.from == 0 && P.to == Q.stages;  // this CTA has every key
        const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + (turn > 0)) * kRows;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int32_t r = 8 * n + 2 * t + h, row = first_row + r;
                if (row >= rows) continue;
                const bool none = l[n][h] == 0.0f, flat = m[n][h] == kNone;
                const float inv = none || (flat && !whole) ? 0.0f : (flat ? NAN : __fdiv_rn(1.0f, l[n][h]));
                const float lse = none ? -INFINITY : (flat && whole ? NAN : m[n][h] + log2f(l[n][h]));
                const int32_t token = row / A.group;
                const int64_t at = static_cast<int64_t>(s.first + token) * A.heads + kvh * A.group + row - token * A.group;
                if (whole) {
                    __align__(16) T v[D / 8];
#pragma unroll
                    for (int d = 0; d < kM; ++d) {
                        v[2 * d] = iqq::from_f32<T>(o[n][d][h] * inv);
                        v[2 * d + 1] = iqq::from_f32<T>(o[n][d][2 + h] * inv);
                    }
                    uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(A.out) + at * D + D / 8 * g);
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) out[i] = reinterpret_cast<const uint4*>(v)[i];
                    if (A.lse != nullptr && g == 0) A.lse[at] = lse / kLog2e;
                } else {
                    float2* out = reinterpret_cast<float2*>(A.part + (part + r) * D + D / 8 * g);
#pragma unroll
                    for (int d = 0; d < kM; ++d) out[d] = make_float2(o[n][d][h] * inv, o[n][d][2 + h] * inv);
                    if (g == 0) A.part_lse[part + r] = lse;
                }
            }
    }
    ++turn;
    }
}

// Joins the parts of a tile that shares c-1, c, c+1 .. cut: CTA c takes it when its share is the
// first to begin inside the tile.  Share c-1's part is its last piece (its first, if it begins with
// the tile); the others begin inside, so it is their first.  Four warps a row, eight
// parts in flight each, and two rows a CTA: a long sequence leaves a hundred parts of few tiles,
// and one SM would take several microseconds to read them.
template <class T, int D, int ROWS>
__global__ void __launch_bounds__(256)
combine_kernel(const Args A, const int ctas)
{
    constexpr int kE = D / 32, kFlight = 8;
    __shared__ float s_m[2][4], s_l[2][4], s_o[2][4][D];
    const int lane = threadIdx.x & 31, half = threadIdx.x >> 7, warp = (threadIdx.x >> 5) & 3, c = blockIdx.x + 1;
    const int r = blockIdx.y * 2 + half;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Mark M = A.marks[c];
    if (M.t0 == M.t1 || static_cast<int>(blockIdx.y) * 2 >= M.rows) return;
    const int64_t prev = M.shares.start(c - 1);
    if (M.shares.start(c) <= M.t0 || prev > M.t0) return;
    // the shares c-1 .. end-1 have parts
    int end;
    {
        int lo = c, hi = ctas;  // share lo begins before t1, share hi does not (or is none)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (M.shares.start(mid) < M.t1) lo = mid;
            else hi = mid;
        }
        end = hi;
    }
    const int parts = end - c + 1;
    float m = kNone, l = 0.0f, o[kE] = {};
    if (r < M.rows) {
        for (int p0 = warp; p0 < parts; p0 += 4 * kFlight) {
            float x[kFlight], v[kFlight][kE];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {  // (loads without a branch, so that they overlap)
                const int p = min(p0 + 4 * i, parts - 1), from = c - 1 + p;
                const int at = (from * 2 + (p == 0 && prev < M.t0)) * ROWS + r;
                x[i] = A.part_lse[at];
                if (p0 + 4 * i >= parts || M.shares.empty(from)) x[i] = -INFINITY;
                if constexpr (D == 128) {
                    const float4 w = *reinterpret_cast<const float4*>(A.part + static_cast<int64_t>(at) * D + lane * 4);
                    v[i][0] = w.x; v[i][1] = w.y; v[i][2] = w.z; v[i][3] = w.w;
                } else {
                    const float2 w = *reinterpret_cast<const float2*>(A.part + static_cast<int64_t>(at) * D + lane * 2);
                    v[i][0] = w.x; v[i][1] = w.y;
                }
            }
            float top = m;
#pragma unroll
            for (int i = 0; i < kFlight; ++i) top = fmaxf(top, x[i]);  // (skips NaN, whose part makes everything NaN)
            const float keep = ex2(m - top);
            m = top;
            l *= keep;
#pragma unroll
            for (int e = 0; e < kE; ++e) o[e] *= keep;
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                if (x[i] == -INFINITY) continue;  // (its values may be anything)
                const float w = ex2(x[i] - top);
                l += w;
#pragma unroll
                for (int e = 0; e < kE; ++e) o[e] = fmaf(w, v[i][e], o[e]);
            }
        }
    }
    if (lane == 0) {
        s_m[half][warp] = m;
        s_l[half][warp] = l;
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) s_o[half][warp][lane * kE + e] = o[e];
    __syncthreads();
    const int d = threadIdx.x & 127;
    if (d >= D || r >= M.rows) return;
    float top = s_m[half][0];
#pragma unroll
    for (int w = 1; w < 4; ++w) top = fmaxf(top, s_m[half][w]);
    float sum = 0.0f, acc = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float f = ex2(s_m[half][w] - top);
        sum = fmaf(s_l[half][w], f, sum);
        acc = fmaf(s_o[half][w][d], f, acc);
    }
    const bool none = top == kNone && sum == 0.0f;
    if (top == kNone && !none) sum = NAN;  // parts whose scores are all -Inf
    const int32_t row = M.row0 + r, token = row / A.group;
    const int64_t at = static_cast<int64_t>(M.token + token) * A.heads + M.head * A.group + row - token * A.group;
    static_cast<T*>(A.out)[at * D + d] = iqq::from_f32<T>(none ? 0.0f : __fdiv_rn(acc, sum));
    if (A.lse != nullptr && d == 0) A.lse[at] = none ? -INFINITY : (top + log2f(sum)) / kLog2e;
}

// Rows a sequence (its share of the tokens, times the group) from which the prompt kernel is taken: it
// makes 256 rows' operands for any number, this one 16 rows' at a time.  Decode and prompt kernel, us:
//   128 dimensions  24 sequences up to 5000: 32 rows 82, 101; 40 rows 110, 102.  64 of 2000: 32 rows 144, 155; 40 rows 200, 156
//    64 dimensions  24 sequences up to 5000: 48 rows 76, 83; 62 rows 97, 82.     64 of 2000: 48 rows 124, 127; 62 rows 158, 127
constexpr int64_t prompt_rows(int64_t head_dim) { return head_dim == 128 ? 33 : 49; }

// Tables up to this many keys, and tiles that fit the machine at once: a CTA takes a whole tile; of one
// sequence whose tiles are less than a quarter of the SMs, up to kFewKeys.  Shares and whole tiles, us on
// the device (128 dimensions), by keys:
//   1 sequence    1 tile 512: 8.3, 8.0; 768: 8.6, 9.8    8 tiles 640: 9.5, 9.1; 704: 9.6, 10.0; 1024: 10.1, 11.7
//                32 tiles 640: 10.2, 9.9; 1024: 11.5, 12.6    64 tiles 1024: 13.7, 12.9
//   sequences x heads   2 x 32 1024: 13.8, 12.9   8 x 8 1024: 15.2, 13.7; 1536: 17.0, 17.8   32 x 8 1024: 24.9, 22.6
// Few sequences of few tiles lose on the device between the two limits (3 x 2 heads 1024: 9.8, 11.7) and
// win in a call that the host makes each time, where the second launch and the workspace take 4 us.
constexpr int64_t kWholeKeys = 1024, kFewKeys = 704;

struct Plan {
    bool prompt;
    bool whole;       // a tile a CTA
    int splits;       // of the prompt kernel
    int row_tile;     // rows a CTA
    int64_t ctas;     // shares
    size_t marks, part, lse;  // bytes of the workspace's parts
};

// The launch goes by shapes alone (lengths are on the device): row tiles of 8 while a sequence's
// share of the tokens fits, else of 16; as many CTAs as fit the machine, or fewer where the tables
// leave less than a stage each.
Plan plan_of(const iqq_kv8_cache* cache, const iqq_kv8_seqs* seqs, int64_t n_heads, int64_t n_tokens)
{
    Plan p = {};
    const int64_t group = n_heads / cache->n_kv_heads;
    const int64_t each = (n_tokens + seqs->n_seqs - 1) / seqs->n_seqs * group;
    p.prompt = each >= prompt_rows(cache->head_dim);
    if (p.prompt) {
        p.splits = iqq::prompt_splits(cache, seqs, n_heads, n_tokens);
        p.part = iqq::prompt_part_bytes(cache, seqs, n_heads, n_tokens, p.splits, &p.lse);
        return p;
    }
    p.row_tile = each <= 8 ? 8 : 16;
    const int64_t tiles = (n_tokens * group / p.row_tile + seqs->n_seqs) * cache->n_kv_heads;
    const int64_t stages = 1 + (seqs->table_width * cache->page_size + kKeys - 1) / kKeys;
    const int64_t most = std::min<int64_t>(kMaxCtas, (p.row_tile == 8 ? 3 : 2) * iqq::sm_count());
    const bool few = seqs->n_seqs == 1 && tiles < iqq::sm_count() / 4;
    p.whole = tiles <= most && seqs->table_width * cache->page_size <= (few ? kFewKeys : kWholeKeys);
    if (p.whole) {
        p.ctas = tiles;
        return p;
    }
    p.ctas = tiles >= most ? most : std::min<int64_t>(most, tiles * std::min<int64_t>(stages, most));
    p.marks = (static_cast<size_t>(p.ctas) * sizeof(Mark) + 15) / 16 * 16;
    p.part = static_cast<size_t>(p.ctas) * 2 * p.row_tile * cache->head_dim * sizeof(float);
    p.lse = static_cast<size_t>(p.ctas) * 2 * p.row_tile * sizeof(float);
    return p;
}

template <class... P, class... A>
iqq_status start(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args)
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
    cudaLaunchKernelEx(&cfg, kernel, args...);
    return iqq::launch_status();
}

template <class T, int D, int NT>
iqq_status launch(const Kv8& C, const Args& A, const Plan& p, cudaStream_t st, uint32_t* flags)
{
    static std::atomic<uint64_t> done{0};
    constexpr size_t smem = sizeof(Smem<D, NT>);
    iqq_status s = iqq::opt_in_smem(reinterpret_cast<const void*>(decode_kernel<T, D, NT>), smem, done);
    if (s != IQQ_OK) return s;
    // the codes as rows of 128 bytes, read as much of a page at a time as a stage takes
    CUtensorMap maps[2];
    const int64_t rows = (static_cast<int64_t>(C.n_pages) * C.heads << C.page_log2) * D / 128;
    const int box = std::min(kKeys, 1 << C.page_log2) * D / 128;
    for (int i = 0; i < 2; ++i) {
        s = iqq::byte_map(&maps[i], C.codes[i], 128, rows, 128, box);
        if (s != IQQ_OK) return s;
    }
    s = start(decode_kernel<T, D, NT>, dim3(static_cast<unsigned>(p.ctas)), kThreads + 32, smem, st, maps[0], maps[1], C, A, flags);
    if (s != IQQ_OK || p.whole || p.ctas == 1) return s;
    return start(combine_kernel<T, D, 8 * NT>, dim3(static_cast<unsigned>(p.ctas - 1), 4 * NT), 256, 0, st, A,
                 static_cast<int>(p.ctas));
}

bool shapes_ok(const iqq_kv8_cache* cache, const iqq_kv8_seqs* seqs, int64_t n_heads, int64_t n_tokens)
{
    return cache != nullptr && seqs != nullptr && cache->n_kv_heads >= 1 && n_heads >= 1 && n_heads <= 65535 &&
           n_heads % cache->n_kv_heads == 0 && n_tokens >= 1 && n_tokens <= 0x7fffffffLL / n_heads && seqs->n_seqs >= 1 &&
           seqs->n_seqs <= (1LL << 24) && cache->page_size >= 1 && cache->page_size <= 128 && seqs->table_width >= 0 &&
           seqs->table_width <= 0x7fffffffLL;
}

}  // namespace

extern "C" size_t iqq_kv8_attention_workspace_bytes(const iqq_kv8_cache* cache, const iqq_kv8_seqs* seqs, int64_t n_heads,
                                                    int64_t n_tokens)
{
    if (!shapes_ok(cache, seqs, n_heads, n_tokens)) return 0;
    const Plan p = plan_of(cache, seqs, n_heads, n_tokens);
    return p.marks + p.part + p.lse;
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
    if (n_heads < 1 || n_heads % C.heads != 0 || n_heads > 65535 || q_token_stride < 0 || q_head_stride < 0 ||
        n_tokens * n_heads > 0x7fffffffLL)
        return IQQ_ERR_SHAPE;
    // (a tile's row is 32 bits; more than 274 GB of codes are refused)
    if (cache->n_pages * cache->n_kv_heads > 0x7fffffffLL * 128 / (cache->page_size * cache->head_dim)) return IQQ_ERR_SHAPE;
    if (n_tokens == 0 || C.n_seqs == 0) return IQQ_OK;
    const Plan p = plan_of(cache, seqs, n_heads, n_tokens);
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
    A.scale = scale;
    char* ws = static_cast<char*>(workspace);
    A.splits = p.splits;
    A.marks = p.whole ? nullptr : reinterpret_cast<Mark*>(ws);
    A.part = reinterpret_cast<float*>(ws + p.marks);
    A.part_lse = reinterpret_cast<float*>(ws + p.marks + p.part);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p.prompt) return iqq::launch_prompt(cache, C, A, dtype, d_flags, st);
    const auto go = [&](auto zero) {
        using T = decltype(zero);
        if (cache->head_dim == 128)
            return p.row_tile == 8 ? launch<T, 128, 1>(C, A, p, st, d_flags) : launch<T, 128, 2>(C, A, p, st, d_flags);
        return p.row_tile == 8 ? launch<T, 64, 1>(C, A, p, st, d_flags) : launch<T, 64, 2>(C, A, p, st, d_flags);
    };
    return dtype == IQQ_BF16 ? go(__nv_bfloat16{}) : go(__half{});
}

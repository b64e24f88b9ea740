// kv8_prompt.cu -- causal attention over the paged int8 key/value cache for many rows a sequence
// (prompts and their chunks), on sm_100a.
//
// out = sum_j p_j v_j / sum_j p_j, p_j = exp(s_j - m), s_j = scale * q . k_j, one pass with the
// running maximum m.  A CTA takes 256 rows of one sequence and key/value head (row r is token
// r / group, head r % group of the group) as two tiles of 128, over 128 keys at a time:
//     S = Q K^T and O += P V on tcgen05 (binary16 operands, binary32 sums in tensor memory).
// While one tile's scores go through the softmax, the other's products run.  One warp loads, one turns
// the pages' scales into factors.  Four warps make the operands: codes become binary16 exactly (the
// byte b of a code c, in the low byte of 0x6400, is the binary16 1152 + c after b ^= 0x80), rows of q
// by a power of two for each row.  Four warps a tile do the softmax, a thread a row, so maximum and
// sum need no other thread.
//
// The scales stay out of the operands: with f = (the row's and the page's key scale) and the page's
// value scale vs, the thread computes y = s f + log2(vs) for 16 keys at a time, P = 2^(y - m) with
// m the running maximum of y less 7 (see kLift), in binary16 (2^-11, as fine as the output's type or
// finer), and the denominator as sum P / vs in binary32.  m moves only when a P passes 2^15, and only
// then O is rescaled.  Bound by the tensor cores and, as nearly, by the exponentials (16 an SM and clock).
// Measured: 8192 tokens, 32 heads over 8 of 128 dimensions 520 us (1057 TFLOP/s of 1650); chunks of 2000
// and 1700 tokens after 3000 and 6300: 354 us (932); 16 prompts of 1000: 270 us (486: a CTA's
// lookups, first loads and output are half of its time there).
#include <math.h>

#include <algorithm>

#include "kv8.cuh"
#include "sm100.cuh"

namespace {

using iqq::Attend;
using iqq::ex2;
using iqq::kLog2e;
using iqq::kNone;
using iqq::kTinyScale;
using iqq::Kv8;
using iqq::pack_h2;
using iqq::Span;
using iqq::sub_h2;

constexpr int kRows = 128, kTiles = 2, kKeys = 128, kStages = 2 /* a power of two */, kScales = 4;
// First warp that makes operands; the ones that multiply, load and turn the pages' scales into factors.
constexpr int kMakers = 8, kMma = 12, kLoader = 13, kScaler = 14;
constexpr int kThreads = 32 * 16;
// Registers a thread of the softmax, the makers and the rest (the launch's are shared out anew); where
// the rest spill, so does the time (8192 tokens of 32 heads over 8: 650 us with 40 for them).
constexpr int kSoftmaxRegs = 192, kMakerRegs = 72, kOtherRegs = 56;
constexpr int kRegs = 128 * (2 * kSoftmaxRegs + kMakerRegs + kOtherRegs);

// Operands in rows of 64 dimensions (128 bytes), 128-byte swizzle: block b of 64 dimensions of a
// tile is 128 rows at b * 16384.
template <int D>
struct Smem {
    static constexpr int kOperand = 128 * D * 2;
    uint8_t v[kStages][kOperand];
    uint8_t k[kStages][kOperand];
    uint8_t q[kTiles][kOperand];
    uint8_t raw[2][128 * D];                    // the codes of a tile of keys, and of values
    float rawks[kKeys / 16], rawvs[kKeys / 16];  // their scales, beside the keys
    int live[2];                                // which 16 keys have a page, a bit each
    // of each 16 keys: the key scale, log2 of the value scale and its reciprocal
    float ks[kScales][kKeys / 16], lv[kScales][kKeys / 16], rv[kScales][kKeys / 16];
    uint64_t rfull[2], rempty[2];
    uint64_t kfull[kStages], kempty[kStages], vfull[kStages], vempty[kStages];
    uint64_t scaled[kScales], qfull[kTiles], sfull[kTiles], pfull[kTiles], ofull[kTiles], done;
    uint32_t tmem;
};

// 16-byte unit u (of 8) of row r of a 64-dimension block.
__device__ __forceinline__ uint32_t unit(int r, int u) { return static_cast<uint32_t>(r * 128 + ((u ^ (r & 7)) << 4)); }

// Four codes as two binary16 pairs, in order.
__device__ __forceinline__ uint2 codes4(uint32_t w)
{
    w ^= 0x80808080u;
    return make_uint2(sub_h2(__byte_perm(w, 0x64646464u, 0x4140), 0x64806480u),
                      sub_h2(__byte_perm(w, 0x64646464u, 0x4342), 0x64806480u));
}

template <int N>
__device__ __forceinline__ void more_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A warp's arrival, after its threads' writes to an operand.
__device__ __forceinline__ void warp_arrive(uint64_t* bar)
{
    proxy_fence();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) iqq::bar_arrive(iqq::smem_u32(bar));
}

// The work of a CTA.
struct Work {
    int32_t b, head, row0, rows;  // sequence, key/value head, first row, rows of the sequence
    int64_t start, len;           // position of the sequence's first token here, its keys
    int32_t first;                // its first packed row
    int32_t tile0;                // the first key tile of this CTA's part
    int64_t part;                 // where its rows' parts go
    int32_t tiles[kTiles];        // key tiles of the part that the row tile sees
    __device__ __forceinline__ int key_tiles() const { return max(tiles[0], tiles[1]); }
    __device__ __forceinline__ int64_t sees(int row, int group) const { return min(len, start + row / group + 1); }
};

// ---- the warp that loads ----

// Key tiles 0 .. n-1 into `raw`, keys and values in turn.  A lane takes what a tile has of one page
// (all or page_size of its keys, whichever is less); 32 of these are looked up at a time.
template <int D>
__device__ __forceinline__ bool load(Smem<D>& S, const Kv8& C, const Work& W, int n, int64_t end, uint32_t* flags)
{
    const int lane = threadIdx.x & 31;
    const int piece = min(kKeys, 1 << C.page_log2), per = kKeys / piece, batch = 32 / per;
    const auto page_of = [&](int j) {
        const int64_t key = (static_cast<int64_t>(W.tile0) + j) * kKeys + lane * piece;
        return key < end ? iqq::page_at(C, W.b, key >> C.page_log2) : -2;
    };
    bool ok = true;
    int page = page_of(0), j = 0, sent[2] = {0, 0};
    for (int j0 = 0; j0 < n && ok; j0 += batch) {
        const int here = page;
        if (j0 + batch < n) page = page_of(j0 + batch);
        if (here == -1) iqq::raise_flags(flags, IQQ_FLAG_BAD_INDEX);
        const uint32_t live = __ballot_sync(0xffffffffu, here >= 0);
        for (int i = 0; i < batch && j < n && ok; ++i, ++j) {
            const uint32_t mine = (live >> (i * per)) & ((1u << per) - 1u);
            const int u = lane - i * per;
            const bool my = u >= 0 && u < per && here >= 0;
            const int64_t cell = static_cast<int64_t>(here) * C.heads + W.head;
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                const bool late = !iqq::bar_wait(iqq::smem_u32(&S.rempty[which]), (j & 1) ^ 1u);
                if (__any_sync(0xffffffffu, late)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = iqq::smem_u32(&S.rfull[which]);
                if (lane == 0) {
                    uint32_t with = 0;
                    for (int x = 0; x < per; ++x)
                        if (mine >> x & 1u) with |= ((1u << (piece / 16)) - 1u) << (x * (piece / 16));
                    S.live[which] = static_cast<int>(with);
                    iqq::bar_expect(bar, static_cast<uint32_t>(__popc(mine)) * piece * D);
                }
                __syncwarp();
                if (my) {
                    const int64_t key = (static_cast<int64_t>(W.tile0) + j) * kKeys + u * piece;
                    iqq::bulk_load(iqq::smem_u32(S.raw[which]) + u * piece * D,
                                   C.codes[which] + ((cell << C.page_log2) + (key & ((1 << C.page_log2) - 1))) * D, piece * D, bar);
                    if (which == 0)
                        for (int x = 0; x < piece / 16; ++x) {
                            iqq::async_load4(iqq::smem_u32(&S.rawks[u * (piece / 16) + x]), C.scales[0] + cell);
                            iqq::async_load4(iqq::smem_u32(&S.rawvs[u * (piece / 16) + x]), C.scales[1] + cell);
                        }
                }
                iqq::async_arrive(bar);
                ++sent[which];
            }
        }
    }
    // every copy has landed (the makers waited for it) unless a wait ran out
#pragma unroll
    for (int which = 0; which < 2; ++which)
        if (sent[which] > 0) ok &= iqq::bar_drain(iqq::smem_u32(&S.rfull[which]), (sent[which] - 1) & 1);
    return ok;
}

// ---- the warp that makes the scales' factors ----

// Codes of a value scale that counts as 0 are made 0, so any scale does in their weights, if it neither
// moves m above what other pages need (as low as 2^-40, or as the lowest seen) nor takes the weights out
// of binary32 beside the largest (2^-100 of it).
template <int D>
__device__ __forceinline__ bool make_scales(Smem<D>& S, int n)
{
    const int lane = threadIdx.x & 31;
    float lo = -40.0f, hi = -40.0f;  // log2 of the smallest and the largest value scale so far
    for (int j = 0; j < n; ++j) {
        const int c = j % kScales;  // (its last reader is four tiles back: that tile's weights met their values before this one was loaded)
        const bool late = !iqq::bar_wait(iqq::smem_u32(&S.rfull[0]), j & 1);
        if (__any_sync(0xffffffffu, late)) return false;
        const bool has = lane < kKeys / 16 && (S.live[0] >> lane & 1);
        const float vs = has ? S.rawvs[lane] : 0.0f, ks = has ? S.rawks[lane] : 0.0f;
        __syncwarp();
        if (lane == 0) iqq::bar_arrive(iqq::smem_u32(&S.rempty[0]));
        float here = vs;
        if (vs >= kTinyScale) {
            here = log2f(vs);
            lo = fminf(lo, here);
            hi = fmaxf(hi, here);
        }
        if (__any_sync(0xffffffffu, has && vs < kTinyScale)) {
#pragma unroll
            for (int o = 1; o < kKeys / 16; o *= 2) {
                lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
                hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
            }
            if (vs < kTinyScale) here = fmaxf(lo, hi - 100.0f);
        }
        if (lane < kKeys / 16) {
            S.ks[c][lane] = ks;
            S.lv[c][lane] = has ? here : -INFINITY;                       // no page: hidden
            S.rv[c][lane] = has ? (vs == vs ? ex2(-here) : 1.0f) : 0.0f;  // (0 weights of NaN pages stay 0)
        }
        __syncwarp();
        if (lane == 0) iqq::bar_arrive(iqq::smem_u32(&S.scaled[c]));
    }
    return true;
}

// ---- the warps that make the operands ----

// This thread's pieces of a raw tile, to binary16, swizzled.
template <int D>
__device__ __forceinline__ void convert(const uint4 (&w)[D / 16], int tid, uint8_t* to)
{
    constexpr int kChunks = D / 16;
    const int c = tid % kChunks, block = c >> 2, u = 2 * (c & 3), swap = block & 1;
    to += block * 16384;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int key = (i * 128 + tid) / kChunks;
        const uint2 a = codes4(w[i].x), b = codes4(w[i].y), d = codes4(w[i].z), e = codes4(w[i].w);
        const uint4 lo = make_uint4(a.x, a.y, b.x, b.y), hi = make_uint4(d.x, d.y, e.x, e.y);
        // the two blocks' threads write their halves in opposite order, so they meet no bank
        *reinterpret_cast<uint4*>(to + unit(key, u + swap)) = swap ? hi : lo;
        *reinterpret_cast<uint4*>(to + unit(key, u + 1 - swap)) = swap ? lo : hi;
    }
}

template <int D>
__device__ __forceinline__ bool make_operands(Smem<D>& S, int n)
{
    constexpr int kChunks = D / 16;  // 16-byte pieces of a token, and a thread's of a tile
    const int tid = threadIdx.x - 32 * kMakers, lane = tid & 31;
    for (int j = 0; j < n; ++j) {
        const int s = j % kStages;
        const uint32_t ph = (j / kStages) & 1;
        uint32_t zero = 0;  // the 16 keys whose value scale is 0
#pragma unroll 1  // (the code of all roles together has to stay in the instruction caches)
        for (int which = 0; which < 2; ++which) {
            bool late = !iqq::bar_wait(iqq::smem_u32(&S.rfull[which]), j & 1);
            if (__any_sync(0xffffffffu, late)) return false;
            uint32_t live = S.live[which];
            if (which == 0) {
                zero = __ballot_sync(0xffffffffu, lane < kKeys / 16 && S.rawvs[lane & 7] < kTinyScale);
            } else {
                live &= ~zero;
            }
            uint4 w[kChunks];
#pragma unroll
            for (int i = 0; i < kChunks; ++i) w[i] = *reinterpret_cast<const uint4*>(&S.raw[which][(i * 128 + tid) * 16]);
            __syncwarp();
            if (lane == 0) iqq::bar_arrive(iqq::smem_u32(&S.rempty[which]));
            if (live != 0xffu) {
#pragma unroll
                for (int i = 0; i < kChunks; ++i)
                    if (!(live >> ((i * 128 + tid) / kChunks / 16) & 1)) w[i] = make_uint4(0, 0, 0, 0);
            }
            late = !iqq::bar_wait(iqq::smem_u32(which == 0 ? &S.kempty[s] : &S.vempty[s]), ph ^ 1u);
            if (__any_sync(0xffffffffu, late)) return false;
            convert<D>(w, tid, which == 0 ? S.k[s] : S.v[s]);
            warp_arrive(which == 0 ? &S.kfull[s] : &S.vfull[s]);
        }
    }
    return true;
}

// ---- the warp that multiplies ----
// Its path from a tile's weights to the next products is every step's: it is one loop, not unrolled
// over the tiles, within its registers, and descriptors are a 32-bit sum (8192 tokens of 32 heads
// over 8: 590 us before, 541 us so).  All lanes run it, on values that are the same in all, and one
// issues, so the operands stay in uniform registers; the weights are waited for last (514 us then).

template <int D>
__device__ __forceinline__ bool multiply(Smem<D>& S, const Work& W, uint32_t base)
{
    const uint32_t tmem = __shfl_sync(0xffffffffu, base, 0);
    const int tiles0 = __shfl_sync(0xffffffffu, W.tiles[0], 0), tiles1 = __shfl_sync(0xffffffffu, W.tiles[1], 0);
    constexpr uint32_t kQk = iqq::idesc_f16(kRows, kKeys, false), kPv = iqq::idesc_f16(kRows, D, true);
    const int n = max(tiles0, tiles1);
    bool late = false;
    for (int t = 0; t < kTiles; ++t)
        if ((t == 0 ? tiles0 : tiles1) > 0) late |= !iqq::bar_wait(iqq::smem_u32(&S.qfull[t]), 0);
    for (int j = -1; j < n; ++j) {
        const int sv = j & (kStages - 1), sk = (j + 1) & (kStages - 1);
#pragma unroll 1
        for (int t = 0; t < kTiles; ++t) {
            const int mine = t == 0 ? tiles0 : tiles1;
            const bool weigh = j >= 0 && j < mine, score = j + 1 < mine;
            // the operands first, which are ready early: then nothing but the weights is waited for
            if (weigh) late |= !iqq::bar_wait(iqq::smem_u32(&S.vfull[sv]), (j / kStages) & 1);
            if (score) late |= !iqq::bar_wait(iqq::smem_u32(&S.kfull[sk]), ((j + 1) / kStages) & 1);
            if (weigh) late |= !iqq::bar_wait(iqq::smem_u32(&S.pfull[t]), j & 1);
            if (__any_sync(0xffffffffu, late)) return false;
            iqq::tc_fence_after();
            const uint32_t s = tmem + t * kKeys, o = tmem + kTiles * kKeys + t * 128;
            const uint32_t q = iqq::desc_lo(iqq::smem_u32(S.q[t]), 16), k = iqq::desc_lo(iqq::smem_u32(S.k[sk]), 16);
            const uint32_t v = iqq::desc_lo(iqq::smem_u32(S.v[sv]), 16384);
            if (iqq::elect()) {
                if (weigh) {
#pragma unroll
                    for (int i = 0; i < kKeys / 16; ++i) iqq::mma_f16_t(o, s + 8 * i, v + i * 128, kPv, j > 0 || i > 0);
                    if (j + 1 == mine) iqq::tc_commit<1>(iqq::smem_u32(&S.ofull[t]));
                }
                if (score) {  // (over this tile's weights: the products run in order)
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint32_t at = ((i >> 2) * 16384 + (i & 3) * 32) >> 4;
                        iqq::mma_f16(s, q + at, k + at, kQk, i > 0);
                    }
                    iqq::tc_commit<1>(iqq::smem_u32(&S.sfull[t]));
                }
            }
        }
        if (iqq::elect()) {
            if (j + 1 < n) iqq::tc_commit<1>(iqq::smem_u32(&S.kempty[sk]));
            if (j >= 0) iqq::tc_commit<1>(iqq::smem_u32(&S.vempty[sv]));
        }
    }
    return true;
}

// ---- the warps of a row tile (a thread a row) ----

// The largest y = s f + log2(vs) of this thread's row.  (A NaN, of a hidden run whose factor is 0 or
// of a page whose scale is NaN, is passed over.)
template <bool MASKED>
__device__ __forceinline__ float row_top(uint32_t s_at, const float* ks, const float* lv, float unscale, int limit)
{
    float top = kNone;
    uint32_t x[2][32];
    iqq::tmem_ld32(s_at, x[0]);
#pragma unroll
    for (int i = 0; i < kKeys / 32; ++i) {
        iqq::tmem_wait_ld(x[i & 1]);
        if (i + 1 < kKeys / 32) iqq::tmem_ld32(s_at + 32 * (i + 1), x[(i + 1) & 1]);
        float most[4];  // independent chains
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            float v = __uint_as_float(x[i & 1][e]);
            if (MASKED && 32 * i + e >= limit) v = -INFINITY;
            most[e >> 3] = (e & 7) == 0 ? v : fmaxf(most[e >> 3], v);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            top = fmaxf(top, fmaf(fmaxf(most[2 * h], most[2 * h + 1]), unscale * ks[2 * i + h], lv[2 * i + h]));
    }
    return top;
}

// P = 2^(y - m), as binary16 pairs; returns the row's sum of P / vs.  `over`: whether a weight is
// above 2^15.
template <bool MASKED>
__device__ __forceinline__ float row_weights(uint32_t s_at, const float* ks, const float* lv, const float* rv, float unscale,
                                             float m, int limit, uint32_t (&p)[kKeys / 32][16], bool& over)
{
    float l = 0.0f;
    uint32_t x[2][32], most[2] = {0u, 0u};
    iqq::tmem_ld32(s_at, x[0]);
#pragma unroll
    for (int i = 0; i < kKeys / 32; ++i) {
        iqq::tmem_wait_ld(x[i & 1]);
        if (i + 1 < kKeys / 32) iqq::tmem_ld32(s_at + 32 * (i + 1), x[(i + 1) & 1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float f = unscale * ks[2 * i + h], b = lv[2 * i + h] - m;
            const uint64_t f2 = iqq::pack_f2(f, f), b2 = iqq::pack_f2(b, b);
            uint64_t sum[2];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                float y0, y1;
                iqq::unpack_f2(iqq::fma_f2(iqq::pack_f2(__uint_as_float(x[i & 1][16 * h + e]), __uint_as_float(x[i & 1][16 * h + e + 1])),
                                           f2, b2), y0, y1);
                if (MASKED) {
                    if (32 * i + 16 * h + e >= limit) y0 = -INFINITY;
                    if (32 * i + 16 * h + e + 1 >= limit) y1 = -INFINITY;
                }
                const float p0 = ex2(y0), p1 = ex2(y1);
                const uint64_t p2 = iqq::pack_f2(p0, p1);
                sum[e / 2 & 1] = e < 4 ? p2 : iqq::add_f2(sum[e / 2 & 1], p2);
                p[i][8 * h + e / 2] = pack_h2(p0, p1);
                most[e / 2 & 1] = iqq::max_h2(most[e / 2 & 1], p[i][8 * h + e / 2]);
            }
            float s0, s1;
            iqq::unpack_f2(iqq::add_f2(sum[0], sum[1]), s0, s1);
            l = fmaf(s0 + s1, rv[2 * i + h], l);
        }
    }
    const uint32_t top = iqq::max_h2(most[0], most[1]);
    over = max(top & 0xffffu, top >> 16) > 0x7800u;  // 2^15 (the weights are not negative; a NaN was passed over)
    return l;
}

// A row is D/8 units of 16 bytes, in q and in the output: as many lanes take a row of global memory,
// so a warp's access is whole rows (a thread for each row took 7 us for q and 2 us for the output).
template <int D>
struct Rows {
    static constexpr int kUnits = D / 8, kAtOnce = 32 / kUnits;
    // where the lane's unit of the i-th access lies: the row within the warp's 32, and the unit
    __device__ __forceinline__ static int row(int i) { return kAtOnce * i + static_cast<int>(threadIdx.x & 31) / kUnits; }
    __device__ __forceinline__ static int unit_of() { return static_cast<int>(threadIdx.x & 31) % kUnits; }
    // ... and in the tile's operand
    __device__ __forceinline__ static uint32_t at(int r, int u) { return static_cast<uint32_t>(u >> 3) * 16384 + unit(r, u & 7); }
};

// This warp's 32 rows of q on their way into the operand's place, as they are.
template <class T, int D>
__device__ __forceinline__ void fetch_q(Smem<D>& S, const Attend& A, const Work& W, int t)
{
    using R = Rows<D>;
    const int r0 = static_cast<int>(threadIdx.x & 96), row = W.row0 + t * kRows + r0 + static_cast<int>(threadIdx.x & 31);
    const int token = row / A.group;
    const int64_t from = row < W.rows ? (W.first + token) * A.q_token_stride +
                                            (W.head * A.group + row - token * A.group) * A.q_head_stride
                                      : -1;
#pragma unroll
    for (int i = 0; i < R::kUnits; ++i) {
        const int r = R::row(i), u = R::unit_of();
        const int64_t at = __shfl_sync(0xffffffffu, from, r);
        iqq::async_load16(iqq::smem_u32(S.q[t] + R::at(r0 + r, u)), static_cast<const T*>(A.q) + (at < 0 ? 0 : at + u * 8),
                          at < 0 ? 0u : 16u);
    }
}

// This warp's 32 rows of sums times `by`, out: staged in q's place, which no product reads any more.
// `to` is this thread's row (null: none).
template <class V, int D>
__device__ __forceinline__ void put_rows(Smem<D>& S, int t, uint32_t o_at, float by, bool none, V* to)
{
    using R = Rows<D>;
    constexpr int kRound = R::kUnits * 16 / static_cast<int>(sizeof(V)), kPer = 16 / static_cast<int>(sizeof(V));
    const int r = static_cast<int>(threadIdx.x & 127), r0 = r & 96;
#pragma unroll
    for (int d = 0; d < D; d += kRound) {
#pragma unroll
        for (int i = 0; i < kRound; i += 32) {
            uint32_t x[32];
            iqq::tmem_ld32(o_at + d + i, x);
            iqq::tmem_wait_ld(x);
            __align__(16) V v[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = iqq::from_f32<V>(none ? 0.0f : __uint_as_float(x[e]) * by);
#pragma unroll
            for (int e = 0; e < 32 / kPer; ++e)
                *reinterpret_cast<uint4*>(S.q[t] + R::at(r, i / kPer + e)) = reinterpret_cast<const uint4*>(v)[e];
        }
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < R::kUnits; ++i) {
            const int row = R::row(i), u = R::unit_of();
            V* out = reinterpret_cast<V*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), row));
            const uint4 w = *reinterpret_cast<const uint4*>(S.q[t] + R::at(r0 + row, u));
            if (out != nullptr) reinterpret_cast<uint4*>(out + d)[u] = w;
        }
        __syncwarp();
    }
}

template <class T, int D>
__device__ __forceinline__ bool attend(Smem<D>& S, const Kv8& C, const Attend& A, const Work& W, uint32_t tmem, int t)
{
    const int r = threadIdx.x & 127, row = W.row0 + t * kRows + r;
    const bool real = row < W.rows;
    const int token = row / A.group;
    const int64_t at = static_cast<int64_t>(W.first + token) * A.heads + W.head * A.group + row - token * A.group;
    const int n = t == 0 ? W.tiles[0] : W.tiles[1];
    const int64_t part = W.part + t * kRows + r;
    if (n == 0) {  // nothing to see: zeros
        if (real && A.splits > 1) {
            A.part_lse[part] = -INFINITY;
        } else if (real) {
            uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(A.out) + at * D);
            for (int i = 0; i < D / 8; ++i) out[i] = make_uint4(0, 0, 0, 0);
            if (A.lse != nullptr) A.lse[at] = -INFINITY;
        }
        return true;
    }
    // the row of q that fetch_q brought: its largest value, then the operand
    float unscale;
    iqq::async_wait_all();
    __syncwarp();
    {
        const T* q = nullptr;  // (of its type)
        uint4 raw[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) raw[i] = *reinterpret_cast<const uint4*>(S.q[t] + Rows<D>::at(r, i));
        float top = 0.0f, v[8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            iqq::widen8(q, raw[i], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
        }
        const int e = iqq::row_exponent(top);
        // the scale's sign goes with q, so that the largest score is the largest product
        const float down = A.scale < 0.0f ? -iqq::power_of_two(-e) : iqq::power_of_two(-e);
        unscale = iqq::power_of_two(e) * fabsf(A.scale) * kLog2e;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            iqq::widen8(q, raw[i], v);
            *reinterpret_cast<uint4*>(S.q[t] + Rows<D>::at(r, i)) =
                make_uint4(pack_h2(v[0] * down, v[1] * down), pack_h2(v[2] * down, v[3] * down),
                           pack_h2(v[4] * down, v[5] * down), pack_h2(v[6] * down, v[7] * down));
        }
        warp_arrive(&S.qfull[t]);
    }
    // keys below `limit` are seen by this row, below `clear` by every row of the tile
    const int64_t limit64 = real ? W.sees(row, A.group) : W.len, clear64 = W.sees(W.row0 + t * kRows, A.group);
    const uint32_t lanes = static_cast<uint32_t>((threadIdx.x >> 5) & 3) * 32 << 16;
    const uint32_t s_at = tmem + lanes + t * kKeys, o_at = tmem + lanes + kTiles * kKeys + t * 128;
    float m = kNone, l = 0.0f;
    for (int j = 0; j < n; ++j) {
        const int c = j % kScales;
        bool late = !iqq::bar_wait(iqq::smem_u32(&S.scaled[c]), (j / kScales) & 1);
        late |= !iqq::bar_wait(iqq::smem_u32(&S.sfull[t]), j & 1);
        if (__any_sync(0xffffffffu, late)) return false;
        iqq::tc_fence_after();
        const int64_t first_key = (static_cast<int64_t>(W.tile0) + j) * kKeys;
        const bool masked = clear64 < first_key + kKeys;
        const int limit = static_cast<int>(max(int64_t{0}, min(limit64 - first_key, int64_t{kKeys})));
        // One pass with the maximum as it is; where a weight came out above 2^15 (rare after the first
        // tiles), or a row has seen nothing yet, the maximum is taken and the weights anew.
        uint32_t p[kKeys / 32][16];
        const float *ks = S.ks[c], *lv = S.lv[c], *rv = S.rv[c];
        bool over = m == kNone;
        float sum = 0.0f;
        for (int turn = __any_sync(0xffffffffu, over) ? 1 : 0; turn < 3; ++turn) {
            if (turn == 1) {
                if (!__any_sync(0xffffffffu, over)) break;
                const float top = masked ? row_top<true>(s_at, ks, lv, unscale, limit) : row_top<false>(s_at, ks, lv, unscale, limit);
                const float to = top - iqq::kLift, next = over || to > m + iqq::kMove ? fmaxf(m, to) : m, f = ex2(m - next);
                const float root = ex2(0.5f * (m - next));  // (f may be below binary32, where zero pages made l large)
                m = next;
                l = l * root * root;
                if (j > 0) {
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        uint32_t x[32];
                        iqq::tmem_ld32(o_at + 32 * i, x);
                        iqq::tmem_wait_ld(x);
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                        iqq::tmem_st32(o_at + 32 * i, x);
                    }
                }
            } else {
                sum = masked ? row_weights<true>(s_at, ks, lv, rv, unscale, m, limit, p, over)
                             : row_weights<false>(s_at, ks, lv, rv, unscale, m, limit, p, over);
            }
        }
        l += sum;
#pragma unroll
        for (int i = 0; i < kKeys / 32; ++i) iqq::tmem_st16(s_at + 16 * i, p[i]);
        iqq::tmem_wait_st();
        iqq::tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) iqq::bar_arrive(iqq::smem_u32(&S.pfull[t]));
    }
    const bool late = !iqq::bar_wait(iqq::smem_u32(&S.ofull[t]), 0);
    if (__any_sync(0xffffffffu, late)) return false;
    iqq::tc_fence_after();
    float inv = __fdiv_rn(1.0f, l), lse = m + log2f(l);
    bool none = false;
    if (real && !(l > 0.0f)) {  // (a NaN may come of q alone, where no key has a page)
        const int64_t first_key = static_cast<int64_t>(W.tile0) * kKeys;
        const bool sees = iqq::any_page(C, W.b, first_key, min(limit64, first_key + static_cast<int64_t>(n) * kKeys));
        if (!sees || l == 0.0f) {
            none = !sees || A.splits > 1;
            inv = NAN;
            lse = !sees ? -INFINITY : (A.splits > 1 ? kNone : NAN);
        }
    }
    if (A.splits > 1) put_rows<float, D>(S, t, o_at, inv, none, real ? A.part + part * D : nullptr);
    else put_rows<T, D>(S, t, o_at, inv, none, real ? static_cast<T*>(A.out) + at * D : nullptr);
    if (real && A.splits > 1) A.part_lse[part] = lse;
    else if (real && A.lse != nullptr) A.lse[at] = lse / kLog2e;
    return true;
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const Kv8 C, const Attend A, uint32_t* __restrict__ flags)
{
    extern __shared__ __align__(1024) uint8_t raw[];
    Smem<D>& S = *reinterpret_cast<Smem<D>*>(raw);
    const int warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    iqq::check_spans(C, false, flags);

    // later slots first, in all heads: the last rows of a sequence see the most keys
    const uint32_t split = blockIdx.x % static_cast<uint32_t>(A.splits), item = (gridDim.x - 1 - blockIdx.x) / static_cast<uint32_t>(A.splits);
    const int64_t slot = item / static_cast<uint32_t>(C.heads);
    Work W;
    W.b = iqq::seq_of_slot(C, slot, A.group, kTiles * kRows, 1);
    W.head = static_cast<int32_t>(item % static_cast<uint32_t>(C.heads));
    const Span s = iqq::span_of(C, W.b);
    const int64_t row0 = (slot - iqq::slot_base(C, W.b, A.group, kTiles * kRows, 1)) * (kTiles * kRows);
    W.rows = s.n * A.group;  // 0 for a bad span
    if (row0 < 0 || row0 >= W.rows) return;  // (below 0: before the first sequence's, where cu begins above 0)
    W.row0 = static_cast<int32_t>(row0);
    W.first = s.first;
    W.start = s.start;
    W.len = s.len < C.capacity ? s.len : C.capacity;
    W.part = (static_cast<int64_t>(item) * A.splits + split) * (kTiles * kRows);
    int64_t end = 0;  // keys that some row sees
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const int first = W.row0 + t * kRows, last = min(W.rows, first + kRows) - 1;
        const int64_t sees = first < W.rows ? max(int64_t{0}, W.sees(last, A.group)) : 0;
        W.tiles[t] = static_cast<int32_t>((sees + kKeys - 1) / kKeys);
        end = max(end, sees);
    }
    {  // this CTA's part of the key tiles
        const int n = W.key_tiles(), to = static_cast<int>(static_cast<int64_t>(n) * (split + 1) / A.splits);
        W.tile0 = static_cast<int32_t>(static_cast<int64_t>(n) * split / A.splits);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) W.tiles[t] = max(0, min(W.tiles[t], to) - W.tile0);
    }
    if (warp < kMakers && (warp < 4 ? W.tiles[0] : W.tiles[1]) > 0) fetch_q<T, D>(S, A, W, warp >> 2);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            iqq::bar_init(iqq::smem_u32(&S.kfull[i]), 4);
            iqq::bar_init(iqq::smem_u32(&S.vfull[i]), 4);
            iqq::bar_init(iqq::smem_u32(&S.kempty[i]), 1);
            iqq::bar_init(iqq::smem_u32(&S.vempty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            iqq::bar_init(iqq::smem_u32(&S.rfull[i]), 33);  // expect_tx, and the lanes' scales
            iqq::bar_init(iqq::smem_u32(&S.rempty[i]), i == 0 ? 5 : 4);  // the makers; of the keys the scales' warp, too
        }
        for (int i = 0; i < kScales; ++i) iqq::bar_init(iqq::smem_u32(&S.scaled[i]), 1);
        for (int i = 0; i < kTiles; ++i) {
            iqq::bar_init(iqq::smem_u32(&S.qfull[i]), 4);
            iqq::bar_init(iqq::smem_u32(&S.sfull[i]), 1);
            iqq::bar_init(iqq::smem_u32(&S.pfull[i]), 4);
            iqq::bar_init(iqq::smem_u32(&S.ofull[i]), 1);
        }
        iqq::bar_init(iqq::smem_u32(&S.done), 1);
        iqq::bar_init_fence();
    }
    if (warp == kMma) iqq::tmem_alloc<1>(iqq::smem_u32(&S.tmem), 512);
    iqq::tc_fence_before();
    __syncthreads();
    iqq::tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = S.tmem;

    bool ok = true;
    if (warp < kMakers) {
        more_registers<kSoftmaxRegs>();
        ok = attend<T, D>(S, C, A, W, tmem, warp >> 2);
    } else if (warp < kMma) {
        fewer_registers<kMakerRegs>();
        ok = make_operands<D>(S, W.key_tiles());
    } else {
        fewer_registers<kOtherRegs>();
        if (warp == kLoader) {
            ok = load<D>(S, C, W, W.key_tiles(), end, flags);
        } else if (warp == kScaler) {
            ok = make_scales<D>(S, W.key_tiles());
        } else if (warp == kMma) {
            ok = multiply<D>(S, W, tmem);
            // nothing is left running when the tensor memory goes
            if (iqq::elect()) iqq::tc_commit<1>(iqq::smem_u32(&S.done));
            ok &= iqq::bar_drain(iqq::smem_u32(&S.done), 0);
        }
    }
    if (!ok) iqq::raise_flags(flags, IQQ_FLAG_WAIT_TIMEOUT);
    __syncwarp();
    iqq::tc_fence_before();
    __syncthreads();
    iqq::tc_fence_after();
    if (warp == kMma) iqq::tmem_free<1>(tmem, 512);
}

// Joins a row's parts: a warp a row.
template <class T, int D>
__global__ void __launch_bounds__(256)
join_kernel(const Kv8 C, const Attend A)
{
    constexpr int kE = D / 32;
    const int lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t item = id / (kTiles * kRows), slot = item / C.heads;
    const int r = static_cast<int>(id % (kTiles * kRows)), head = static_cast<int>(item % C.heads);
    const int b = iqq::seq_of_slot(C, slot, A.group, kTiles * kRows, 1);
    const Span s = iqq::span_of(C, b);
    const int64_t row = (slot - iqq::slot_base(C, b, A.group, kTiles * kRows, 1)) * (kTiles * kRows) + r;
    if (row < 0 || row >= static_cast<int64_t>(s.n) * A.group) return;
    const int64_t part = item * A.splits * (kTiles * kRows) + r;
    float m = kNone, l = 0.0f, o[kE] = {};
#pragma unroll 4
    for (int p = 0; p < A.splits; ++p) {
        const int64_t at = part + static_cast<int64_t>(p) * (kTiles * kRows);
        const float x = A.part_lse[at];
        float v[kE];
#pragma unroll
        for (int e = 0; e < kE; ++e) v[e] = A.part[at * D + lane * kE + e];
        if (x == -INFINITY) continue;  // (its values may be anything)
        const float top = fmaxf(m, x), keep = ex2(m - top), w = ex2(x - top);  // (a NaN part makes everything NaN)
        m = top;
        l = fmaf(l, keep, w);
#pragma unroll
        for (int e = 0; e < kE; ++e) o[e] = fmaf(o[e], keep, w * v[e]);
    }
    const bool none = m == kNone && l == 0.0f;
    if (m == kNone && !none) l = NAN;  // parts whose scores are all -Inf
    const int64_t token = row / A.group, at = (s.first + token) * A.heads + head * A.group + row - token * A.group;
#pragma unroll
    for (int e = 0; e < kE; ++e)
        static_cast<T*>(A.out)[at * D + lane * kE + e] = iqq::from_f32<T>(none ? 0.0f : __fdiv_rn(o[e], l));
    if (A.lse != nullptr && lane == 0) A.lse[at] = none ? -INFINITY : (m + log2f(l)) / kLog2e;
}

int64_t slots_of(int64_t n_tokens, int64_t group, int64_t n_seqs) { return n_tokens * group / (kTiles * kRows) + n_seqs; }

template <class... P, class... A>
iqq_status start(void (*kernel)(P...), int64_t grid, int threads, size_t smem, cudaStream_t st, const A&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
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

template <class T, int D>
iqq_status launch(const Kv8& C, const Attend& A, uint32_t* flags, cudaStream_t st)
{
    static std::atomic<uint64_t> done{0};
    constexpr size_t smem = 226 * 1024;  // the whole SM's: it takes the whole tensor memory
    static_assert(sizeof(Smem<D>) <= smem, "shared memory");
    iqq_status s = iqq::opt_in_smem(reinterpret_cast<const void*>(prompt_kernel<T, D>), smem, done);
    if (s != IQQ_OK) return s;
    // The warps' shares have to fit what the launch gives, or they would wait for registers for good.
    static std::atomic<int> known{0};  // registers a thread, once they could be asked for
    int regs = known.load(std::memory_order_relaxed);
    if (regs == 0) {
        cudaFuncAttributes at = {};
        if (cudaFuncGetAttributes(&at, prompt_kernel<T, D>) != cudaSuccess) return iqq::launch_status();
        regs = at.numRegs;
        known.store(regs, std::memory_order_relaxed);
    }
    if (regs * kThreads < kRegs) {
        iqq::set_last_cuda_error(cudaErrorLaunchOutOfResources);
        return IQQ_ERR_CUDA;
    }
    const int64_t items = slots_of(C.n_tokens, A.group, C.n_seqs) * C.heads;
    if (items * A.splits > 0x7fffffffLL || items * kTiles * kRows / 8 > 0x7fffffffLL) return IQQ_ERR_SHAPE;
    s = start(prompt_kernel<T, D>, items * A.splits, kThreads, smem, st, C, A, flags);
    if (s != IQQ_OK || A.splits == 1) return s;
    return start(join_kernel<T, D>, items * kTiles * kRows / 8, 256, 0, st, C, A);
}

}  // namespace

// The keys of 256 rows are split while the row tiles alone leave SMs idle and a part keeps at least four
// key tiles (64 tokens after 16000, 32 heads over 8: 47 us, and 315 us in 16 CTAs; 50 tokens of 8 heads
// over one of 64 dimensions after 60000: 44 us, and 1000 us in two).
int iqq::prompt_splits(const iqq_kv8_cache* cache, const iqq_kv8_seqs* seqs, int64_t n_heads, int64_t n_tokens)
{
    const int64_t group = n_heads / cache->n_kv_heads, items = slots_of(n_tokens, group, seqs->n_seqs) * cache->n_kv_heads;
    const int64_t most = seqs->table_width * cache->page_size / (4 * kKeys);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({sm_count() / items, most, 128})));
}

size_t iqq::prompt_part_bytes(const iqq_kv8_cache* cache, const iqq_kv8_seqs* seqs, int64_t n_heads, int64_t n_tokens,
                              int splits, size_t* lse_bytes)
{
    *lse_bytes = 0;
    if (splits == 1) return 0;
    const int64_t group = n_heads / cache->n_kv_heads;
    const size_t rows = static_cast<size_t>(slots_of(n_tokens, group, seqs->n_seqs) * cache->n_kv_heads) * splits * kTiles * kRows;
    *lse_bytes = rows * sizeof(float);
    return rows * cache->head_dim * sizeof(float);
}

iqq_status iqq::launch_prompt(const iqq_kv8_cache* cache, const Kv8& C, const Attend& A, int dtype, uint32_t* flags,
                              cudaStream_t st)
{
    if (dtype == IQQ_BF16)
        return cache->head_dim == 128 ? launch<__nv_bfloat16, 128>(C, A, flags, st) : launch<__nv_bfloat16, 64>(C, A, flags, st);
    return cache->head_dim == 128 ? launch<__half, 128>(C, A, flags, st) : launch<__half, 64>(C, A, flags, st);
}

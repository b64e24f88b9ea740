// i8_gemm.cu -- matrix product of int8 rows with a scale for each token and each output
// channel, on sm_100a.
//
// y[t][r] = ((float(sum_j a[t][j] w[r][j]) * a_scales[t]) * w_scales[r]) + bias[r], the
// integer sum exact in 32 bits, so neither the order of the sum nor its split changes a value.
//
// Both kernels run tcgen05.mma.kind::i8 from 128-byte-swizzled tiles that TMA brings in (k and
// edge rows beyond the matrices arrive as zeros), with the output channels along the tensor
// memory's lanes and the tokens along its columns: a warp of the epilogue then holds 32
// neighbouring channels of one token and writes them as one run, whatever y's pitch and
// alignment.  One warp loads, one issues the products, four carry the sums out.
//
//  pair kernel   tiles of 256 channels x up to 256 tokens by a pair of CTAs (cta_group::2: each
//                holds half of both operands), persistent, two accumulators, so a tile's sums
//                are carried out while the next one's products run.  Bound by the tensor cores.
//  split kernel  tiles of 128 channels x up to 256 tokens, the k axis split over a cluster of up
//                to 8 CTAs whose partial sums meet in shared memory: when tokens are few, the
//                weights' bytes bound the product and every SM has to read its share of them.
//
// Measured with weights larger than L2 in turn (tokens x channels x k): 4096 x 11008 x 4096 117 us
// (3170 TOPS; twice the bfloat16 rate would be 3299), 777 x 4099 x 11000 30 us (2340 TOPS), 192 x 4096
// x 14336 21 us, 16 x 11008 x 4096 11.2 us (4.1 TB/s of weights), 1 x 4096 x 4096 6.5 us.
#include <math.h>

#include <algorithm>

#include "i8_code.cuh"
#include "sm100.cuh"

namespace {

constexpr int kThreads = 192;        // warp 0 loads, warp 1 multiplies, warps 2..5 finish
constexpr int kStep = 128;           // bytes of k a stage: one swizzle row
constexpr int kRows = 128;           // channels a CTA
constexpr int kABytes = kRows * kStep;
constexpr int kMaxStages = 12;
constexpr int kScales = 4 * 256 * 4;      // shared memory for the tokens' scales, a copy a finishing warp
constexpr int kSmem = 227 * 1024 - 1024;  // beside the static shared memory
constexpr int kSmemHalf = 112 * 1024;     // two CTAs an SM

struct Args {
    const float* as;
    const float* ws;
    const float* bias;
    void* y;
    uint32_t* flags;
    int64_t ldy, n_tok, n_out;
    int64_t m_tiles, t_tiles;
    int kblocks, tn, stages, split;
};

struct Bars {
    uint64_t full[kMaxStages], empty[kMaxStages], done[2], taken[2];
    uint32_t tmem;
};

__device__ __forceinline__ float finish(int sum, float da, float dw, float bias)
{
    return __fadd_rn(__fmul_rn(__fmul_rn(static_cast<float>(sum), da), dw), bias);
}

// 32 sums of this lane's channel, of n tokens with the scales da, from y on.
template <class T>
__device__ __forceinline__ void put32(const uint32_t (&x)[32], const float* da, float dw, float bias, T* y, int64_t ldy, int n)
{
    if (n >= 32) {  // (checked apart: a test a token took as long as its arithmetic)
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const float4 d = *reinterpret_cast<const float4*>(da + i);
            y[0] = iqq::from_f32<T>(finish(static_cast<int>(x[i]), d.x, dw, bias));
            y += ldy;
            y[0] = iqq::from_f32<T>(finish(static_cast<int>(x[i + 1]), d.y, dw, bias));
            y += ldy;
            y[0] = iqq::from_f32<T>(finish(static_cast<int>(x[i + 2]), d.z, dw, bias));
            y += ldy;
            y[0] = iqq::from_f32<T>(finish(static_cast<int>(x[i + 3]), d.w, dw, bias));
            y += ldy;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < n) y[i * ldy] = iqq::from_f32<T>(finish(static_cast<int>(x[i]), da[i], dw, bias));
    }
}

// This lane's channel r of tokens t0 .. t0 + cols - 1, from the tensor memory's columns at `at`: 32 at
// a time, the next ones on the way while these are finished.  `da`: the warp's own 256 floats of
// shared memory, for the tokens' scales.
template <class T>
__device__ __forceinline__ void put(const Args& P, uint32_t at, int64_t t0, int cols, int64_t r, float dw, float bias, float* da)
{
    const int lane = threadIdx.x & 31;
    const bool real = r < P.n_out;
    T* y = static_cast<T*>(P.y) + t0 * P.ldy + r;
    uint32_t v0[32], v1[32];
    iqq::tmem_ld32(at, v0);
    __syncwarp();
    for (int c = lane; c < cols; c += 32) da[c] = iqq::ld(P.as + t0 + c);
    __syncwarp();
    for (int c = 0; c < cols; c += 64) {
        iqq::tmem_wait_ld(v0);
        if (c + 32 < cols) iqq::tmem_ld32(at + c + 32, v1);
        if (real) put32<T>(v0, da + c, dw, bias, y + c * P.ldy, P.ldy, cols - c);
        if (c + 32 >= cols) break;
        __syncwarp();
        iqq::tmem_wait_ld(v1);
        if (c + 64 < cols) iqq::tmem_ld32(at + c + 64, v0);
        if (real) put32<T>(v1, da + c + 32, dw, bias, y + (c + 32) * P.ldy, P.ldy, cols - c - 32);
        __syncwarp();
    }
}

// (0 + bias and no bias differ for no value but -0, which the product of a zero sum may have)
__device__ __forceinline__ float bias_of(const Args& P, int64_t r)
{
    return P.bias != nullptr && r < P.n_out ? iqq::ld(P.bias + r) : 0.0f;
}

template <class T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
pair_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap, const Args P)
{
    extern __shared__ uint8_t raw[];
    __shared__ Bars S;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = (iqq::smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t rank = iqq::cluster_rank();
    const int half = P.tn >> 1;
    const uint32_t stage_bytes = kABytes + static_cast<uint32_t>(half) * kStep;
    const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, tiles = P.m_tiles * P.t_tiles;
    bool late = false;  // a wait of this thread ran out

    if (threadIdx.x == 0) {
        for (int i = 0; i < P.stages; ++i) {
            iqq::bar_init(iqq::smem_u32(&S.full[i]), 1);
            iqq::bar_init(iqq::smem_u32(&S.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            iqq::bar_init(iqq::smem_u32(&S.done[i]), 1);
            iqq::bar_init(iqq::smem_u32(&S.taken[i]), 8);
        }
        iqq::bar_init_fence();
        iqq::tma_prefetch_map(&wmap);
        iqq::tma_prefetch_map(&amap);
    }
    if (warp == 1) iqq::tmem_alloc<2>(iqq::smem_u32(&S.tmem), 512);
    iqq::tc_fence_before();
    iqq::cluster_sync();
    iqq::tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t tmem = S.tmem;

    if (warp == 0 && lane == 0) {
        int64_t issued = 0;
        int s = 0;
        uint32_t ph = 0;
        for (int64_t i = pair; i < tiles && !late; i += pairs) {
            const int m0 = static_cast<int>(i / P.t_tiles) * 2 * kRows + static_cast<int>(rank) * kRows;
            const int t0 = static_cast<int>(i % P.t_tiles) * P.tn + static_cast<int>(rank) * half;
            for (int kb = 0; kb < P.kblocks; ++kb) {
                if (!iqq::bar_wait_long<true>(iqq::smem_u32(&S.empty[s]), ph ^ 1u)) {
                    late = true;
                    break;
                }
                const uint32_t bar = iqq::map_rank(iqq::smem_u32(&S.full[s]), 0), at = base + s * stage_bytes;
                if (rank == 0) iqq::bar_expect(iqq::smem_u32(&S.full[s]), 2 * stage_bytes);
                iqq::tma_load_pair(at, &wmap, kb * kStep, m0, bar);
                iqq::tma_load_pair(at + kABytes, &amap, kb * kStep, t0, bar);
                ++issued;
                if (++s == P.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        // every copy has landed (the products waited for them) unless a wait ran out: then the two CTAs may have
        // stopped at different stages, whose barriers never complete, and the copies get 1 ms to land
        if (rank == 0)
            for (int64_t i = issued > P.stages ? issued - P.stages : 0; i < issued && !late; ++i)
                late = !iqq::bar_drain<true>(iqq::smem_u32(&S.full[i % P.stages]), static_cast<uint32_t>(i / P.stages) & 1u);
        if (late)
            for (const long long t0 = clock64(); clock64() - t0 < 2000000LL;) {}
    } else if (warp == 1 && lane == 0 && rank == 0) {
        const uint32_t idesc = iqq::idesc_i8(2 * kRows, P.tn);
        int s = 0, turn = 0;
        uint32_t ph = 0;
        for (int64_t i = pair; i < tiles && !late; i += pairs, ++turn) {
            const int buf = turn & 1;
            late = !iqq::bar_wait_long<true>(iqq::smem_u32(&S.taken[buf]), (static_cast<uint32_t>(turn >> 1) & 1u) ^ 1u);
            iqq::tc_fence_after();
            for (int kb = 0; kb < P.kblocks && !late; ++kb) {
                if (!iqq::bar_wait_long<true>(iqq::smem_u32(&S.full[s]), ph)) {
                    late = true;
                    break;
                }
                iqq::tc_fence_after();
                const uint32_t at = base + s * stage_bytes;
                const uint64_t a = iqq::desc_k128(at), b = iqq::desc_k128(at + kABytes);
#pragma unroll
                for (int u = 0; u < kStep / 32; ++u)
                    iqq::mma_i8<2>(tmem + buf * 256, a + 2 * u, b + 2 * u, idesc, kb > 0 || u > 0);
                iqq::tc_commit<2>(iqq::smem_u32(&S.empty[s]));
                if (++s == P.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            iqq::tc_commit<2>(iqq::smem_u32(&S.done[buf]));
        }
        // (the tensor memory goes after the last products, also where the epilogue gave up)
        if (turn > 0) late |= !iqq::bar_drain<true>(iqq::smem_u32(&S.done[(turn - 1) & 1]), static_cast<uint32_t>((turn - 1) >> 1) & 1u);
    } else if (warp >= 2) {
        const int quad = warp & 3;
        float* scales = reinterpret_cast<float*>(raw + (base - iqq::smem_u32(raw)) + P.stages * stage_bytes) + (warp - 2) * 256;
        int turn = 0;
        for (int64_t i = pair; i < tiles; i += pairs, ++turn) {
            const int buf = turn & 1;
            const int64_t r = (i / P.t_tiles) * 2 * kRows + rank * kRows + quad * 32 + lane, t0 = (i % P.t_tiles) * P.tn;
            const float dw = r < P.n_out ? iqq::ld(P.ws + r) : 0.0f, bias = bias_of(P, r);
            late = !iqq::bar_wait_long<true>(iqq::smem_u32(&S.done[buf]), static_cast<uint32_t>(turn >> 1) & 1u);
            if (__any_sync(0xffffffffu, late)) break;
            iqq::tc_fence_after();
            const uint32_t at = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * 256;
            const int cols = P.n_tok - t0 < P.tn ? static_cast<int>(P.n_tok - t0) : P.tn;
            put<T>(P, at, t0, cols, r, dw, bias, scales);
            iqq::tc_fence_before();
            __syncwarp();
            if (lane == 0) iqq::bar_arrive_cluster(iqq::map_rank(iqq::smem_u32(&S.taken[buf]), 0));
        }
    }
    if (late) iqq::raise_flags(P.flags, IQQ_FLAG_WAIT_TIMEOUT);
    __syncwarp();
    iqq::tc_fence_before();
    iqq::cluster_sync();  // the pair is done with each other's barriers and tensor memory
    iqq::tc_fence_after();
    if (warp == 1) iqq::tmem_free<2>(tmem, 512);
}

template <class T>
__global__ void __launch_bounds__(kThreads, 2)
split_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap, const Args P,
             const uint32_t columns)
{
    extern __shared__ uint8_t raw[];
    __shared__ Bars S;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = (iqq::smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t rank = P.split > 1 ? iqq::cluster_rank() : 0u;
    const uint32_t stage_bytes = kABytes + static_cast<uint32_t>(P.tn) * kStep;
    const int64_t tile = blockIdx.x / static_cast<uint32_t>(P.split);
    const int64_t m0 = (tile / P.t_tiles) * kRows, t0 = (tile % P.t_tiles) * P.tn;
    // this CTA's part of the k axis
    const int kb0 = static_cast<int>(static_cast<int64_t>(P.kblocks) * rank / P.split);
    const int kb1 = static_cast<int>(static_cast<int64_t>(P.kblocks) * (rank + 1) / P.split);
    bool late = false;

    if (threadIdx.x == 0) {
        for (int i = 0; i < P.stages; ++i) {
            iqq::bar_init(iqq::smem_u32(&S.full[i]), 1);
            iqq::bar_init(iqq::smem_u32(&S.empty[i]), 1);
        }
        iqq::bar_init(iqq::smem_u32(&S.done[0]), 1);
        iqq::bar_init_fence();
        iqq::tma_prefetch_map(&wmap);
        iqq::tma_prefetch_map(&amap);
    }
    if (warp == 1) iqq::tmem_alloc<1>(iqq::smem_u32(&S.tmem), columns);
    iqq::tc_fence_before();
    __syncthreads();
    iqq::tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = S.tmem;

    if (warp == 0) {
        if (lane == 0) {
            // into L2 while the kernel before still runs (a line it then writes is written there)
            for (int kb = kb0; kb < kb1 && kb < kb0 + 16; ++kb)
                iqq::tma_prefetch_l2(&wmap, kb * kStep, static_cast<int>(m0));
            asm volatile("griddepcontrol.wait;" ::: "memory");
            int s = 0;
            uint32_t ph = 0;
            int issued = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!iqq::bar_wait_long(iqq::smem_u32(&S.empty[s]), ph ^ 1u)) {
                    late = true;
                    break;
                }
                const uint32_t bar = iqq::smem_u32(&S.full[s]), at = base + s * stage_bytes;
                iqq::bar_expect(bar, stage_bytes);
                iqq::tma_load(at, &wmap, kb * kStep, static_cast<int>(m0), bar);
                iqq::tma_load(at + kABytes, &amap, kb * kStep, static_cast<int>(t0), bar);
                ++issued;
                if (++s == P.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            // every copy has landed (the products waited for them) unless a wait ran out
            for (int i = issued > P.stages ? issued - P.stages : 0; i < issued; ++i)
                late |= !iqq::bar_drain(iqq::smem_u32(&S.full[i % P.stages]), static_cast<uint32_t>(i / P.stages) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            asm volatile("griddepcontrol.wait;" ::: "memory");  // (its waits are limited, as the copies they wait for begin here)
            const uint32_t idesc = iqq::idesc_i8(kRows, P.tn);
            int s = 0;
            uint32_t ph = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!iqq::bar_wait_long(iqq::smem_u32(&S.full[s]), ph)) {
                    late = true;
                    break;
                }
                iqq::tc_fence_after();
                const uint32_t at = base + s * stage_bytes;
                const uint64_t a = iqq::desc_k128(at), b = iqq::desc_k128(at + kABytes);
#pragma unroll
                for (int u = 0; u < kStep / 32; ++u)
                    iqq::mma_i8<1>(tmem, a + 2 * u, b + 2 * u, idesc, kb > kb0 || u > 0);
                iqq::tc_commit<1>(iqq::smem_u32(&S.empty[s]));
                if (++s == P.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            iqq::tc_commit<1>(iqq::smem_u32(&S.done[0]));
        }
    }
    __syncwarp();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    late |= !iqq::bar_drain(iqq::smem_u32(&S.done[0]), 0);
    __syncwarp();
    iqq::tc_fence_after();

    const int quad = warp & 3, row = quad * 32 + lane;
    const int cols = P.n_tok - t0 < P.tn ? static_cast<int>(P.n_tok - t0) : P.tn;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    if (P.split == 1) {
        if (warp >= 2) {
            float* scales = reinterpret_cast<float*>(raw + (base - iqq::smem_u32(raw))) + (warp - 2) * 256;  // (the stages are free)
            const int64_t r = m0 + row;
            const float dw = r < P.n_out ? iqq::ld(P.ws + r) : 0.0f, bias = bias_of(P, r);
            put<T>(P, lanes, t0, cols, r, dw, bias, scales);
        }
    } else {
        // Groups of four columns per * o .. belong to the cluster's CTA o: everybody sends it its part,
        // 16 bytes a lane, into the stages' memory (free once every CTA's products are done).
        const int groups = (cols + 3) / 4, per = (groups + P.split - 1) / P.split;
        iqq::cluster_sync();
        if (warp >= 2) {
            const uint32_t mine = base + ((rank * per * kRows + row) << 4);
            int owner = 0, local = 0;
            uint32_t to = iqq::map_rank(mine, 0);
            for (int q = 0; q < groups; q += 4) {
                uint32_t v[16];
                iqq::tmem_ld16(lanes + 4 * q, v);
                iqq::tmem_wait_ld(v);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (q + i >= groups) break;
                    iqq::st_cluster(to + ((local * kRows) << 4), v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    if (++local == per && q + i + 1 < groups) {
                        local = 0;
                        to = iqq::map_rank(mine, static_cast<uint32_t>(++owner));
                    }
                }
            }
        }
        __syncwarp();
        iqq::cluster_sync();
        const int first = static_cast<int>(rank) * per, mine = min(per, groups - first);
        const uint4* part = reinterpret_cast<const uint4*>(raw + (base - iqq::smem_u32(raw)));
        for (int i = threadIdx.x; i < mine * kRows; i += kThreads) {
            const int64_t t = t0 + 4 * (first + i / kRows), r = m0 + i % kRows;
            if (r >= P.n_out) continue;
            const float dw = iqq::ld(P.ws + r), bias = bias_of(P, r);
            float da[4];  // (before the stores, which loads may not pass)
#pragma unroll
            for (int u = 0; u < 4; ++u) da[u] = t + u < P.n_tok ? iqq::ld(P.as + t + u) : 0.0f;
            uint4 sum = make_uint4(0, 0, 0, 0);
            for (int src = 0; src < P.split; ++src) {
                const uint4 v = part[src * per * kRows + i];
                sum = make_uint4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
            }
            T* y = static_cast<T*>(P.y) + t * P.ldy + r;
            const uint32_t each[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (t + u < P.n_tok) y[u * P.ldy] = iqq::from_f32<T>(finish(static_cast<int>(each[u]), da[u], dw, bias));
        }
    }
    if (late) iqq::raise_flags(P.flags, IQQ_FLAG_WAIT_TIMEOUT);
    iqq::tc_fence_before();
    __syncthreads();
    iqq::tc_fence_after();
    if (warp == 1) iqq::tmem_free<1>(tmem, columns);
}

// k == 0: the empty sums.
template <class T>
__global__ void __launch_bounds__(256) empty_kernel(const Args P)
{
    const int64_t n = P.n_tok * P.n_out, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) {
        const int64_t t = i / P.n_out, r = i % P.n_out;
        static_cast<T*>(P.y)[t * P.ldy + r] = iqq::from_f32<T>(finish(0, P.as[t], P.ws[r], bias_of(P, r)));
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The launch is the one that this estimate of its time (in microseconds, from measurements on one
// B200) finds shortest: which kernel, its token tile and its parts of the k axis.
//   An SM takes in 0.14 MB of operands a microsecond, 0.1 MB when most SMs do; HBM gives 6 MB, and
//   0.057 MB an SM when few ask; tensor cores take tn/256 * 0.27 a 128-byte step; a launch has 3.3,
//   its finish 0.008 a token, joining parts 0.5 + 0.012 a token.
// Both sides of its turns, tokens x channels x k: 192 x 11008 x 4096: pairs with 192 tokens 14.9 us,
// with 64 tokens 20.1, split kernel 15.7; 16 x 11008 x 4096: 3 parts 11.2, 2 parts 13.0, 1 part 12.6;
// 192 x 4096 x 14336: 4 parts of 192 tokens 21.1, one part of 128 tokens 29.5, pairs 31.0;
// 64 x 11008 x 4096: pairs 12.8, 3 parts 13.6; 200 x 512 x 8192: 8 parts of 64 tokens 7.9, pairs 12.1.
struct Choice {
    double us = 1e300;
    bool pair = false;
    int tn = 0, split = 1;
};

Choice choose(int64_t n_tok, int64_t n_out, int64_t k, int kblocks, int sms)
{
    const double bytes = (static_cast<double>(n_out) + static_cast<double>(n_tok)) * static_cast<double>(k) / 1e6;
    Choice best;
    const auto consider = [&](bool pair, int tn, int split) {
        const int64_t tiles = ceil_div(n_out, pair ? 2 * kRows : kRows) * ceil_div(n_tok, tn);
        const int64_t ctas = tiles * (pair ? 2 : split), per = ceil_div(kblocks, split);
        if (split > 1 && ctas > (tn <= 64 ? 2 : 1) * sms) return;  // the parts of a tile run at once
        const double stage = (kABytes + tn / (pair ? 2 : 1) * kStep) / 1e6;
        // steps of the SM that has most; CTAs of up to 64 tokens run two an SM, but share what it takes in
        const double steps = static_cast<double>(ceil_div(ctas, sms) * per);
        const double use = static_cast<double>(ctas) / static_cast<double>(ceil_div(ctas, sms) * sms);
        const double hbm = ctas <= sms ? std::min(6.0, 0.057 * static_cast<double>(ctas)) : 6.0 * std::sqrt(use);
        double us = std::max(steps * stage / (ctas > 64 || pair ? 0.1 : 0.14), std::max(bytes / hbm, steps * tn * 0.00105));
        us += 3.3 + 0.008 * tn + (split > 1 ? 0.5 + 0.012 * tn : 0.0);
        if (us < best.us) {
            best.us = us;
            best.pair = pair;
            best.tn = tn;
            best.split = split;
        }
    };
    const int most = n_tok >= 256 ? 256 : static_cast<int>(ceil_div(n_tok, 16) * 16);
    for (int split = std::min(8, kblocks); split >= 1; --split) {
        consider(false, most, split);
        if (most > 128) consider(false, 128, split);
        if (most > 64) consider(false, 64, split);
    }
    if (n_tok > 32)
        for (int tn = 32; tn <= 256 && tn < n_tok + 32; tn += 32) consider(true, tn, 1);
    return best;
}

template <class T>
iqq_status launch(Args P, const int8_t* a, int64_t lda, const int8_t* w, int64_t ldw, int64_t k, cudaStream_t st)
{
    static std::atomic<uint64_t> pair_done{0}, split_done{0};
    if (k == 0) {
        empty_kernel<T><<<static_cast<unsigned>(std::min<int64_t>(ceil_div(P.n_tok * P.n_out, 256), 4096)), 256, 0, st>>>(P);
        return iqq::launch_status();
    }
    const int sms = iqq::sm_count();
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    CUtensorMap wmap, amap;
    iqq_status s = iqq::byte_map(&wmap, w, k, P.n_out, ldw, kRows);
    if (s != IQQ_OK) return s;
    const Choice plan = choose(P.n_tok, P.n_out, k, P.kblocks, sms);
    P.tn = plan.tn;
    P.split = plan.split;
    P.m_tiles = ceil_div(P.n_out, plan.pair ? 2 * kRows : kRows);
    P.t_tiles = ceil_div(P.n_tok, P.tn);
    if (plan.pair) {
        s = iqq::byte_map(&amap, a, k, P.n_tok, lda, P.tn / 2);
        if (s == IQQ_OK) s = iqq::opt_in_smem(reinterpret_cast<const void*>(pair_kernel<T>), kSmem, pair_done);
        if (s != IQQ_OK) return s;
        P.stages = std::min<int>(kMaxStages, (kSmem - 1024 - kScales - static_cast<int>(sizeof(Bars))) / (kABytes + P.tn / 2 * kStep));
        const int64_t pairs = std::min<int64_t>(P.m_tiles * P.t_tiles, sms / 2);
        cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
        cfg.dynamicSmemBytes = kSmem - sizeof(Bars);  // the whole SM's: it takes the whole tensor memory
        cudaLaunchKernelEx(&cfg, pair_kernel<T>, wmap, amap, P);
        return iqq::launch_status();
    }
    const int64_t tiles = P.m_tiles * P.t_tiles;
    if (tiles * P.split > 0x7fffffffLL) return IQQ_ERR_SHAPE;
    // Small stages: two CTAs an SM where there are so many, and where a CTA has few steps anyway (16 x
    // 4096 x 4096 in 4 parts: 6.9 us, with an SM's memory each 7.6; clusters of 8 then find room as
    // well); else all of an SM's memory for stages (64 x 11008 x 4096 in one part: 12.9, with half 16.4).
    const bool two = P.tn <= 64 && (tiles * P.split > sms || ceil_div(P.kblocks, P.split) <= 8);
    const int stage = kABytes + P.tn * kStep, room = (two ? kSmemHalf : kSmem - static_cast<int>(sizeof(Bars))) - 1024;
    P.stages = std::min(kMaxStages, room / stage);
    uint32_t columns = 32;
    while (columns < static_cast<uint32_t>(P.tn)) columns *= 2;
    s = iqq::byte_map(&amap, a, k, P.n_tok, lda, P.tn);
    if (s == IQQ_OK) s = iqq::opt_in_smem(reinterpret_cast<const void*>(split_kernel<T>), kSmem, split_done);
    if (s != IQQ_OK) return s;
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * P.split));
    cfg.dynamicSmemBytes = static_cast<size_t>(P.stages * stage + 1024);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(P.split);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = P.split > 1 ? 2 : 1;
    cudaLaunchKernelEx(&cfg, split_kernel<T>, wmap, amap, P, columns);
    return iqq::launch_status();
}

}  // namespace

extern "C" iqq_status iqq_gemm_i8(const int8_t* a, int64_t lda, const float* a_scales, const int8_t* w, int64_t ldw,
                                  const float* w_scales, const float* bias, int y_dtype, void* y, int64_t ldy,
                                  int64_t n_tok, int64_t n_out, int64_t k, uint32_t* d_flags, void* stream)
{
    if (!iqq::dtype_ok(y_dtype)) return IQQ_ERR_ARG;
    if (n_tok < 0 || n_out < 0 || k < 0 || k > IQQ_GEMM_I8_MAX_K) return IQQ_ERR_SHAPE;
    if (n_tok == 0 || n_out == 0) return IQQ_OK;
    const int64_t pitch = (k + 15) / 16 * 16;
    // the distance of rows is not looked at where there is one row, or nothing in them
    if (n_tok == 1 || k == 0) lda = pitch;
    if (n_tok == 1) ldy = n_out;
    if (n_out == 1 || k == 0) ldw = pitch;
    constexpr int64_t kMost = 0x7fffffff - 1024, kFar = (1LL << 40) - 16;  // a tile's coordinates and pitch
    if (lda < k || ldw < k || ldy < n_out || n_tok > kMost || n_out > kMost || lda > kFar || ldw > kFar ||
        !iqq::size_ok(n_tok, lda > 0 ? lda : 1, 1) || !iqq::size_ok(n_out, ldw > 0 ? ldw : 1, 1) ||
        !iqq::size_ok(n_tok, ldy, 4))
        return IQQ_ERR_SHAPE;
    if (y == nullptr || a_scales == nullptr || w_scales == nullptr) return IQQ_ERR_NULL;
    if (k > 0 && (a == nullptr || w == nullptr)) return IQQ_ERR_NULL;
    if (!iqq::aligned(a, 16) || !iqq::aligned(w, 16) || lda % 16 != 0 || ldw % 16 != 0 || !iqq::aligned(a_scales, 4) ||
        !iqq::aligned(w_scales, 4) || !iqq::aligned(bias, 4) || !iqq::aligned(d_flags, 4) ||
        !iqq::aligned(y, static_cast<uintptr_t>(iqq::dtype_bytes(y_dtype))))
        return IQQ_ERR_ALIGN;
    Args P = {};
    P.as = a_scales;
    P.ws = w_scales;
    P.bias = bias;
    P.y = y;
    P.flags = d_flags;
    P.ldy = ldy;
    P.n_tok = n_tok;
    P.n_out = n_out;
    P.kblocks = static_cast<int>(ceil_div(k, kStep));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (y_dtype) {
    case IQQ_F32: return launch<float>(P, a, lda, w, ldw, k, st);
    case IQQ_BF16: return launch<__nv_bfloat16>(P, a, lda, w, ldw, k, st);
    default: return launch<__half>(P, a, lda, w, ldw, k, st);
    }
}

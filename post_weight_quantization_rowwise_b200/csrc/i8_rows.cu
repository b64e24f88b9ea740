// i8_rows.cu -- 8-bit integer rows with one binary32 scale each (the operands of the int8
// matrix product) on sm_100a.
//
// Per row: d = fl32(max|x| / 127), q = rint(x / d).  Two dependent passes over a row, one
// read of it: a CTA takes a row, each thread keeps NV units of eight values in registers
// while the CTA agrees on the maximum, and a row wider than the CTA's registers has its rest
// read again (from L2).  HBM-bound for many rows (2 or 4 B read + 1 B written a value); for
// few rows it is the latency of one load, one block reduction and one store, so the CTA gets
// one unit per thread and up to 1024 threads.
#include <atomic>

#include "i8_code.cuh"

namespace {

constexpr int kMaxWarps = 32;

template <class T, bool VEC>
__device__ __forceinline__ void load_unit(const T* row, int64_t j, int64_t n, float (&v)[8])
{
    if (VEC && j + 8 <= n) {
        iqq::load8(row + j, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = j + i < n ? iqq::to_f32(row[j + i]) : 0.0f;
    }
}

__device__ __forceinline__ uint32_t amax8(const float (&v)[8], uint32_t m)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}

__device__ __forceinline__ void store_unit(int8_t* row, int64_t j, int64_t n, const float (&v)[8], float d, float inv)
{
    uint2 q = make_uint2(0u, 0u);
    if (d > 0.0f) q = iqq::codes8(v, d, inv);  // (NaN > 0 is false)
    if (j + 8 <= n) {
        *reinterpret_cast<uint2*>(row + j) = q;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (j + i < n) row[j + i] = static_cast<int8_t>((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
    }
}

template <class T, int NV, bool VEC>
__global__ void __launch_bounds__(1024)
i8_rows_kernel(const T* __restrict__ x, int64_t ldx, int8_t* __restrict__ codes, int64_t ldc,
               float* __restrict__ scales, int64_t nrows, int64_t n, uint32_t* __restrict__ flags)
{
    __shared__ uint32_t part[2][kMaxWarps];
    const int tid = threadIdx.x, lane = tid & 31, warps = blockDim.x >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t step = 8LL * blockDim.x;
    int turn = 0;
    for (int64_t r = blockIdx.x; r < nrows; r += gridDim.x, turn ^= 1) {
        const T* row = x + r * ldx;
        float v[NV][8];
        uint32_t m = 0u;
#pragma unroll
        for (int u = 0; u < NV; ++u) load_unit<T, VEC>(row, 8LL * tid + u * step, n, v[u]);
#pragma unroll
        for (int u = 0; u < NV; ++u) m = amax8(v[u], m);
        for (int64_t j = 8LL * tid + NV * step; j < n; j += step) {
            float t[8];
            load_unit<T, VEC>(row, j, n, t);
            m = amax8(t, m);
        }
        m = __reduce_max_sync(0xffffffffu, m);
        // two sets of slots in turn: a warp can be at most one row ahead of another
        if (lane == 0) part[turn][tid >> 5] = m;
        __syncthreads();
        m = __reduce_max_sync(0xffffffffu, lane < warps ? part[turn][lane] : 0u);
        const float d = iqq::i8_scale(m);
        const float inv = d > 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
        if (tid == 0) {
            scales[r] = d;
            if (m >= iqq::kInfBits) iqq::raise_flags(flags, IQQ_FLAG_NONFINITE_INPUT);
        }
        int8_t* out = codes + r * ldc;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int64_t j = 8LL * tid + u * step;
            if (j < n) store_unit(out, j, n, v[u], d, inv);
        }
        for (int64_t j = 8LL * tid + NV * step; j < n; j += step) {
            float t[8];
            load_unit<T, VEC>(row, j, n, t);
            store_unit(out, j, n, t, d, inv);
        }
    }
}

template <class T, int NV, bool VEC>
iqq_status launch(const void* x, int64_t ldx, int8_t* codes, int64_t ldc, float* scales, int64_t nrows, int64_t n,
                  uint32_t* flags, cudaStream_t st)
{
    const int64_t units = (n + 7) / 8, per = (units + NV - 1) / NV;
    const int threads = static_cast<int>(per >= 1024 ? 1024 : (per <= 64 ? 64 : (per + 31) / 32 * 32));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(nrows < 0x7fffffffLL ? nrows : 0x7fffffffLL));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, i8_rows_kernel<T, NV, VEC>, static_cast<const T*>(x), ldx, codes, ldc, scales, nrows, n,
                       flags);
    return iqq::launch_status();
}

template <class T>
iqq_status launch_type(const void* x, int64_t ldx, int8_t* codes, int64_t ldc, float* scales, int64_t nrows, int64_t n,
                       uint32_t* flags, cudaStream_t st)
{
    const bool vec = iqq::aligned(x, 16) && (ldx * static_cast<int64_t>(sizeof(T))) % 16 == 0;
    // Few rows (less than two CTAs an SM): one unit a thread, the shortest chain.  Many rows:
    // four units in flight a thread.
    const bool few = nrows < 2LL * iqq::sm_count();
    if (vec) return few ? launch<T, 1, true>(x, ldx, codes, ldc, scales, nrows, n, flags, st)
                        : launch<T, 4, true>(x, ldx, codes, ldc, scales, nrows, n, flags, st);
    return few ? launch<T, 1, false>(x, ldx, codes, ldc, scales, nrows, n, flags, st)
               : launch<T, 4, false>(x, ldx, codes, ldc, scales, nrows, n, flags, st);
}

}  // namespace

int iqq::sm_count()
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

extern "C" iqq_status iqq_quantize_i8_rows(int dtype, const void* x, int64_t ldx, int8_t* codes, int64_t ldc,
                                           float* scales, int64_t nrows, int64_t n, uint32_t* d_flags, void* stream)
{
    if (!iqq::dtype_ok(dtype)) return IQQ_ERR_ARG;
    if (!iqq::size_ok(nrows, n, 4)) return IQQ_ERR_SHAPE;
    if (nrows == 0 || n == 0) return IQQ_OK;
    if (nrows == 1) {
        ldx = (n + 15) / 16 * 16;
        ldc = ldx;
    }
    if (ldx < n || ldc < n || !iqq::size_ok(nrows, ldx, 4) || !iqq::size_ok(nrows, ldc, 1)) return IQQ_ERR_SHAPE;
    if (x == nullptr || codes == nullptr || scales == nullptr) return IQQ_ERR_NULL;
    if (!iqq::aligned(x, static_cast<uintptr_t>(iqq::dtype_bytes(dtype))) || !iqq::aligned(codes, 16) ||
        ldc % 16 != 0 || !iqq::aligned(scales, 4) || !iqq::aligned(d_flags, 4))
        return IQQ_ERR_ALIGN;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dtype) {
    case IQQ_F32: return launch_type<float>(x, ldx, codes, ldc, scales, nrows, n, d_flags, st);
    case IQQ_BF16: return launch_type<__nv_bfloat16>(x, ldx, codes, ldc, scales, nrows, n, d_flags, st);
    default: return launch_type<__half>(x, ldx, codes, ldc, scales, nrows, n, d_flags, st);
    }
}

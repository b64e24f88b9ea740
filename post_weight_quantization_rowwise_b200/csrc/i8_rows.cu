// i8_rows.cu -- 8-bit integer rows with one binary32 scale each (the operands of the int8
// matrix product) on sm_100a.
//
// Per row: d = fl32(max|x| / 127), q = rint(x / d).  Two dependent passes over a row, one
// read of it: a CTA takes a row, each thread keeps NV units of eight values in registers
// while the CTA agrees on the maximum, and a row wider than the CTA's registers has its rest
// read again (from L2).  HBM-bound for many rows (2 or 4 B read + 1 B written a value); for
// few rows it is the latency of one load, one block reduction and one store, so the CTA gets
// one unit per thread and up to 1024 threads.
// Measured: 4096 x 4096 bfloat16 15.5 us (3.2 TB/s; the exact rounding's arithmetic is as long as the
// copy), 777 x 11000 binary32 11.5 us (3.7 TB/s), one row of 4096 1.8 us.
#include <atomic>

#include "i8_code.cuh"

namespace {

constexpr int kMaxWarps = 32;

// Rows of whole units of eight values on 16-byte boundaries.
template <class T, int NV>
__global__ void __launch_bounds__(1024)
i8_rows_kernel(const T* x, int64_t ldx, int8_t* codes, int64_t ldc,
               float* scales, int64_t nrows, int64_t n, uint32_t* flags)
{
    __shared__ uint32_t part[2][kMaxWarps];
    const int tid = threadIdx.x, lane = tid & 31, warps = blockDim.x >> 5;
    const int64_t units = n / 8, beyond = static_cast<int64_t>(NV) * blockDim.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int turn = 0;
    for (int64_t r = blockIdx.x; r < nrows; r += gridDim.x, turn ^= 1) {
        const T* row = x + r * ldx;
        typename iqq::Raw<T>::type v[NV];
        uint32_t m = 0u;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            v[u] = {};
            if (tid + u * static_cast<int>(blockDim.x) < units) iqq::fetch(row + 8 * (tid + u * blockDim.x), v[u]);
        }
#pragma unroll
        for (int u = 0; u < NV; ++u) m = iqq::amax8(row, v[u], m);
        for (int64_t u = tid + beyond; u < units; u += blockDim.x) {
            typename iqq::Raw<T>::type t;
            iqq::fetch(row + 8 * u, t);
            m = iqq::amax8(row, t, m);
        }
        m = __reduce_max_sync(0xffffffffu, iqq::amax_bits(row, m));
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
        uint2* out = reinterpret_cast<uint2*>(codes + r * ldc);
        if (d > 0.0f) {  // (NaN > 0 is false)
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                float w[8];
                iqq::widen(row, v[u], w);
                if (tid + u * static_cast<int>(blockDim.x) < units) out[tid + u * blockDim.x] = iqq::codes8(w, d, inv);
            }
            for (int64_t u = tid + beyond; u < units; u += blockDim.x) {
                typename iqq::Raw<T>::type t;
                float w[8];
                iqq::fetch(row + 8 * u, t);
                iqq::widen(row, t, w);
                out[u] = iqq::codes8(w, d, inv);
            }
        } else {
            for (int64_t u = tid; u < units; u += blockDim.x) out[u] = make_uint2(0u, 0u);
        }
    }
}

// Any rows, a value at a time; the second pass reads them again.
template <class T>
__global__ void __launch_bounds__(1024)
i8_rows_any_kernel(const T* x, int64_t ldx, int8_t* codes, int64_t ldc,
                   float* scales, int64_t nrows, int64_t n, uint32_t* flags)
{
    __shared__ uint32_t part[2][kMaxWarps];
    const int tid = threadIdx.x, lane = tid & 31, warps = blockDim.x >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int turn = 0;
    for (int64_t r = blockIdx.x; r < nrows; r += gridDim.x, turn ^= 1) {
        const T* row = x + r * ldx;
        uint32_t m = 0u;
#pragma unroll 8
        for (int64_t j = tid; j < n; j += blockDim.x) m = max(m, __float_as_uint(iqq::to_f32(row[j])) & 0x7fffffffu);
        m = __reduce_max_sync(0xffffffffu, m);
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
        // four codes a thread, a word where there are four (rows of codes begin on 16-byte boundaries)
        for (int64_t j = 4LL * tid; j < n; j += 4LL * blockDim.x) {
            int q[4] = {0, 0, 0, 0};
            const int most = n - j < 4 ? static_cast<int>(n - j) : 4;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = i < most ? iqq::to_f32(row[j + i]) : 0.0f;
                if (d > 0.0f) q[i] = iqq::rint_code(v, 1, d, v * inv);
            }
            if (most == 4) {
                *reinterpret_cast<uint32_t*>(out + j) = iqq::pack4(q[0], q[1], q[2], q[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (i < most) out[j + i] = static_cast<int8_t>(q[i]);
            }
        }
    }
}

iqq_status start(void (*kernel)(), int64_t per, int64_t nrows, cudaStream_t st, void** args)
{
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
    cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), args);
    return iqq::launch_status();
}

template <class T>
iqq_status launch_type(const void* x, int64_t ldx, int8_t* codes, int64_t ldc, float* scales, int64_t nrows, int64_t n,
                       uint32_t* flags, cudaStream_t st)
{
    const T* from = static_cast<const T*>(x);
    void* args[] = {&from, &ldx, &codes, &ldc, &scales, &nrows, &n, &flags};
    const int64_t units = (n + 7) / 8;
    if (n % 8 != 0 || !iqq::aligned(x, 16) || (ldx * static_cast<int64_t>(sizeof(T))) % 16 != 0)
        return start(reinterpret_cast<void (*)()>(i8_rows_any_kernel<T>), units, nrows, st, args);
    // Few rows (less than two CTAs an SM): one unit a thread, the shortest chain.  Many rows: four
    // units in flight a thread.
    if (nrows < 2LL * iqq::sm_count())
        return start(reinterpret_cast<void (*)()>(i8_rows_kernel<T, 1>), units, nrows, st, args);
    return start(reinterpret_cast<void (*)()>(i8_rows_kernel<T, 4>), (units + 3) / 4, nrows, st, args);
}

}  // namespace

int iqq::sm_count()
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();  // (not the next launch's)
        return 148;
    }
    if (dev < 0 || dev >= 64) return 148;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
            cudaGetLastError();
            return 148;
        }
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

extern "C" iqq_status iqq_quantize_i8_rows(int dtype, const void* x, int64_t ldx, int8_t* codes, int64_t ldc,
                                           float* scales, int64_t nrows, int64_t n, uint32_t* d_flags, void* stream)
{
    if (!iqq::dtype_ok(dtype)) return IQQ_ERR_ARG;
    if (!iqq::size_ok(nrows, n, 4)) return IQQ_ERR_SHAPE;
    if (nrows == 0) return IQQ_OK;
    if (n == 0) {
        if (!iqq::aligned(scales, 4)) return IQQ_ERR_ALIGN;
        if (scales != nullptr &&
            cudaMemsetAsync(scales, 0, static_cast<size_t>(nrows) * sizeof(float), static_cast<cudaStream_t>(stream)) != cudaSuccess)
            return iqq::launch_status();
        return IQQ_OK;
    }
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

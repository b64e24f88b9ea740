// i8_gemm.cu -- matrix product of int8 rows with a scale for each token and each output
// channel, on sm_100a.
//
// y[t][r] = ((float(sum_j a[t][j] w[r][j]) * a_scales[t]) * w_scales[r]) + bias[r], the
// integer sum exact in 32 bits.
#include "i8_code.cuh"

namespace {

constexpr int kTile = 64, kStep = 64;  // 64x64 outputs a CTA, 64 bytes of k a step

struct Args {
    const int8_t* a;
    const float* as;
    const int8_t* w;
    const float* ws;
    const float* bias;
    void* y;
    int64_t lda, ldw, ldy, n_tok, n_out;
    int k;
};

// 16 bytes of a row from byte j, zeros behind k.
__device__ __forceinline__ uint4 load16(const int8_t* row, int j, int k)
{
    if (j + 16 <= k) return __ldg(reinterpret_cast<const uint4*>(row + j));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = 0u;
#pragma unroll
        for (int b = 0; b < 4; ++b)
            if (j + 4 * i + b < k) w[i] |= static_cast<uint32_t>(static_cast<uint8_t>(row[j + 4 * i + b])) << (8 * b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <class T>
__global__ void __launch_bounds__(256) i8_gemm_kernel(const Args P)
{
    __shared__ uint32_t sa[kTile][kStep / 4 + 1], sw[kTile][kStep / 4 + 1];
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kTile, t0 = static_cast<int64_t>(blockIdx.y) * kTile;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int lr = tid >> 2, lj = (tid & 3) * 16;
    int acc[4][4] = {};
    for (int j0 = 0; j0 < P.k; j0 += kStep) {
        uint4 va = make_uint4(0, 0, 0, 0), vw = va;
        if (t0 + lr < P.n_tok) va = load16(P.a + (t0 + lr) * P.lda, j0 + lj, P.k);
        if (r0 + lr < P.n_out) vw = load16(P.w + (r0 + lr) * P.ldw, j0 + lj, P.k);
        const int c = lj / 4;
        sa[lr][c] = va.x; sa[lr][c + 1] = va.y; sa[lr][c + 2] = va.z; sa[lr][c + 3] = va.w;
        sw[lr][c] = vw.x; sw[lr][c + 1] = vw.y; sw[lr][c + 2] = vw.z; sw[lr][c + 3] = vw.w;
        __syncthreads();
#pragma unroll 4
        for (int i = 0; i < kStep / 4; ++i) {
            int a[4], w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                a[u] = static_cast<int>(sa[ty + 16 * u][i]);
                w[u] = static_cast<int>(sw[tx + 16 * u][i]);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[u][v] = __dp4a(a[u], w[v], acc[u][v]);
        }
        __syncthreads();
    }
    T* y = static_cast<T*>(P.y);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t t = t0 + ty + 16 * u;
        if (t >= P.n_tok) continue;
        const float da = __ldg(P.as + t);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int64_t r = r0 + tx + 16 * v;
            if (r >= P.n_out) continue;
            float o = __fmul_rn(__fmul_rn(static_cast<float>(acc[u][v]), da), __ldg(P.ws + r));
            if (P.bias != nullptr) o = __fadd_rn(o, __ldg(P.bias + r));
            y[t * P.ldy + r] = iqq::from_f32<T>(o);
        }
    }
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
    if (n_tok == 1) {
        lda = pitch;
        ldy = n_out;
    }
    if (n_out == 1) ldw = pitch;
    if (lda < k || ldw < k || ldy < n_out || !iqq::size_ok(n_tok, lda > 0 ? lda : 1, 1) ||
        !iqq::size_ok(n_out, ldw > 0 ? ldw : 1, 1) || !iqq::size_ok(n_tok, ldy, 4) || n_tok > 64LL * 65535 ||
        n_out > 64LL * 0x7fffffff)
        return IQQ_ERR_SHAPE;
    if (y == nullptr || a_scales == nullptr || w_scales == nullptr) return IQQ_ERR_NULL;
    if (k > 0 && (a == nullptr || w == nullptr)) return IQQ_ERR_NULL;
    if (!iqq::aligned(a, 16) || !iqq::aligned(w, 16) || lda % 16 != 0 || ldw % 16 != 0 || !iqq::aligned(a_scales, 4) ||
        !iqq::aligned(w_scales, 4) || !iqq::aligned(bias, 4) || !iqq::aligned(d_flags, 4) ||
        !iqq::aligned(y, static_cast<uintptr_t>(iqq::dtype_bytes(y_dtype))))
        return IQQ_ERR_ALIGN;
    const Args P = {a, a_scales, w, w_scales, bias, y, lda, ldw, ldy, n_tok, n_out, static_cast<int>(k)};
    const dim3 grid(static_cast<unsigned>((n_out + kTile - 1) / kTile), static_cast<unsigned>((n_tok + kTile - 1) / kTile));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (y_dtype) {
    case IQQ_F32: i8_gemm_kernel<float><<<grid, 256, 0, st>>>(P); break;
    case IQQ_BF16: i8_gemm_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(P); break;
    default: i8_gemm_kernel<__half><<<grid, 256, 0, st>>>(P); break;
    }
    return iqq::launch_status();
}

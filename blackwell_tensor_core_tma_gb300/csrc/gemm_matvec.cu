// Matrix-vector products with 4-bit weights (gemm_matvec_run in include/gb300gemm.h): the form of
// the block-scaled e2m1 product for 1 to 16 rows of A, on the plans' own B and SFB buffers, with
// 16-bit activations.
//
//   D[m][n] = C[m][n] + sum_k x[m][k] * B[k][n] * sf(SFB[n][k / blk])
//
// One warp per column n: each lane takes 32 consecutive k of it (16 bytes of weights) at a time,
// multiplies them with the M rows and adds in fp32; the lanes' sums are joined by shuffles.
#include <initializer_list>

#include "gemm_rows.cuh"

namespace gb300 {
namespace {

constexpr int MAX_M = 16;
constexpr int64_t MAX_K = 32768;

struct MatvecParams {
    const void *x;
    const uint8_t *b, *sfb;
    const float *c;
    void *d;
    int M, N, K;
};

__device__ __forceinline__ float2 e2m1x2(uint32_t byte) {
    uint32_t h;
    asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(byte));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
__device__ __forceinline__ float2 pair_of(const __nv_bfloat16 *, uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 pair_of(const __half *, uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ float ue8m0(uint32_t c) {
    return c == 255u ? __uint_as_float(0x7FC00000u) : rows::scale_value(c);
}
__device__ __forceinline__ float ue4m3(uint32_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(c & 0x7Fu)));
    return __half2float(__low2half(*reinterpret_cast<const __half2 *>(&h)));
}

template <typename XT, int MODE, bool OUT_BF16>
__global__ void __launch_bounds__(256) matvec_kernel(MatvecParams p) {
    const int lane = threadIdx.x & 31;
    const int n = blockIdx.x * 8 + threadIdx.x / 32;
    if (n >= p.N) return;
    const int groups = p.K / 32;
    float acc[MAX_M];
#pragma unroll
    for (int m = 0; m < MAX_M; ++m) acc[m] = 0.f;
    for (int j = lane; j < groups; j += 32) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p.b + (int64_t)n * (p.K / 2) + j * 16);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        float s[2];
        if (MODE == GEMM_SCALE_UE8M0_32) {
            s[0] = s[1] = ue8m0(p.sfb[(int64_t)n * groups + j]);
        } else {
            s[0] = ue4m3(p.sfb[((int64_t)n * groups + j) * 2]);
            s[1] = ue4m3(p.sfb[((int64_t)n * groups + j) * 2 + 1]);
        }
#pragma unroll
        for (int m = 0; m < MAX_M; ++m) {
            if (m >= p.M) break;
            const uint32_t *x = reinterpret_cast<const uint32_t *>(static_cast<const XT *>(p.x) + (int64_t)m * p.K + j * 32);
            float part[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 v = e2m1x2((w[i / 4] >> (8 * (i & 3))) & 0xFFu), a = pair_of((const XT *)nullptr, x[i]);
                part[i / 8] = fmaf(v.x, a.x, fmaf(v.y, a.y, part[i / 8]));
            }
            acc[m] = fmaf(part[0], s[0], fmaf(part[1], s[1], acc[m]));
        }
    }
#pragma unroll
    for (int m = 0; m < MAX_M; ++m) {
        if (m >= p.M) break;
        float v = acc[m];
        for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        if (lane == 0) {
            const int64_t at = (int64_t)m * p.N + n;
            if (p.c) v += p.c[at];
            if (OUT_BF16) static_cast<__nv_bfloat16 *>(p.d)[at] = __float2bfloat16_rn(v);
            else static_cast<float *>(p.d)[at] = v;
        }
    }
}

template <typename XT, int MODE>
cudaError_t launch(gemm_dtype d, const MatvecParams &p, cudaStream_t stream) {
    const unsigned ctas = (unsigned)((p.N + 7) / 8);
    if (d == GEMM_BF16) matvec_kernel<XT, MODE, true><<<ctas, 256, 0, stream>>>(p);
    else matvec_kernel<XT, MODE, false><<<ctas, 256, 0, stream>>>(p);
    return cudaGetLastError();
}
template <typename XT>
cudaError_t launch(int mode, gemm_dtype d, const MatvecParams &p, cudaStream_t stream) {
    return mode == GEMM_SCALE_UE8M0_32 ? launch<XT, GEMM_SCALE_UE8M0_32>(d, p, stream)
                                       : launch<XT, GEMM_SCALE_UE4M3_16>(d, p, stream);
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" gemm_status gemm_matvec_run(int64_t M, int64_t N, int64_t K, gemm_dtype x, gemm_dtype d, int block_scaled,
                                       const void *X, const void *B, const uint8_t *SFB, const float *C, void *D,
                                       void *cuda_stream) {
    if (M < 0 || N <= 0 || K <= 0 || N > INT32_MAX / 16) return GEMM_ERR_INVALID_ARG;
    if (block_scaled < GEMM_SCALE_NONE || block_scaled > GEMM_SCALE_UE4M3_16) return GEMM_ERR_INVALID_ARG;
    if ((x != GEMM_F16 && x != GEMM_BF16) || (d != GEMM_F32 && d != GEMM_BF16) || block_scaled == GEMM_SCALE_NONE ||
        M > MAX_M || K > MAX_K)
        return GEMM_ERR_UNSUPPORTED;
    if (K % 32 != 0) return GEMM_ERR_ALIGNMENT;
    if (M == 0) return GEMM_OK;
    if (!X || !B || !SFB || !D) return GEMM_ERR_INVALID_ARG;
    for (const void *p : {X, B, (const void *)SFB, (const void *)C, (const void *)D})
        if (!rows::aligned16(p)) return GEMM_ERR_ALIGNMENT;
    int sms = 0;
    gemm_status st = rows::device_sms(&sms);
    if (st != GEMM_OK) return st;
    const MatvecParams p{X, static_cast<const uint8_t *>(B), SFB, C, D, (int)M, (int)N, (int)K};
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = x == GEMM_F16 ? launch<__half>(block_scaled, d, p, stream)
                                        : launch<__nv_bfloat16>(block_scaled, d, p, stream);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

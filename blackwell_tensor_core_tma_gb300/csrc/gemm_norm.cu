// Root-mean-square norm with the residual's addition, and its gradient (gemm_norm_run,
// gemm_norm_backward in include/gb300gemm.h).
//
//   h = round(x + r),  rstd = 1 / sqrt(mean_k h^2 + eps),  y = h * rstd * w
//   n = h * rstd,  g = dy * w,  dx = dh + rstd * (g - n * mean_k(g * n)),  dw = sum_rows dy * n
//
// One pass over memory: a row lives in the registers of its threads (U units of eight elements each)
// between the sum that the statistics need and the outputs that use them.
#include <initializer_list>
#include <mutex>

#include "gemm_rows.cuh"

namespace gb300 {
namespace rows {

gemm_status device_sms(int *sms) {
    constexpr int MAX_DEVICES = 64;
    static int known[MAX_DEVICES];          // 0: not asked yet, -1: not a GB300
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) return GEMM_ERR_CUDA;
    std::lock_guard<std::mutex> lock(mu);
    if (known[dev] == 0) {
        int major = 0, minor = 0, n = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            return GEMM_ERR_CUDA;
        known[dev] = major == 10 && minor == 3 ? n : -1;
    }
    if (known[dev] < 0) return GEMM_ERR_UNSUPPORTED;
    *sms = known[dev];
    return GEMM_OK;
}

}  // namespace rows

namespace {

using namespace rows;

constexpr int MAX_K = 32768;         // a row in registers: 1024 threads x 4 units
constexpr int MAX_WARPS = 32;

// How a row is spread over threads: U units per thread, `tpr` threads per row (a power of two up to
// 32, else whole warps), `rpc` rows per CTA.
struct RowShape {
    int u, tpr, rpc;
};
RowShape row_shape(int K) {
    const int units = K / UNIT;
    RowShape s;
    s.u = units <= 512 ? 1 : units <= 1024 ? 2 : 4;
    const int need = (units + s.u - 1) / s.u;
    if (need <= 32) {
        s.tpr = 4;
        while (s.tpr < need) s.tpr *= 2;
    } else {
        s.tpr = (need + 31) / 32 * 32;
    }
    s.rpc = s.tpr >= 256 ? 1 : 256 / s.tpr;
    return s;
}

// Sum over the threads of a row (threadIdx.y), the same in each of them and in a fixed order.  Every
// thread of the CTA takes part.  `red` holds one float per warp; it may be written again after the
// next __syncthreads.
__device__ __forceinline__ float row_sum(float v, float *red) {
    const int tpr = blockDim.x;
    for (int o = min(tpr, 32) / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (tpr <= 32) return v;
    const int tid = threadIdx.y * tpr + threadIdx.x, warps = tpr / 32;
    if ((tid & 31) == 0) red[tid / 32] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < warps; ++i) s += red[threadIdx.y * warps + i];
    return s;
}

struct NormParams {
    const void *x, *r;
    const float *w;
    void *h, *y;
    uint8_t *sf;
    float *rstd;
    int64_t M;
    int K;
    float eps;
};

template <typename XT, typename HT, typename YT, int U>
__global__ void __launch_bounds__(U == 4 ? 1024 : 512) norm_kernel(NormParams p) {
    __shared__ float red[MAX_WARPS];
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < p.M;
    const int units = p.K / UNIT, tpr = blockDim.x;
    const XT *x = static_cast<const XT *>(p.x) + row * p.K;
    const HT *r = p.r ? static_cast<const HT *>(p.r) + row * p.K : nullptr;
    HT *h = p.h ? static_cast<HT *>(p.h) + row * p.K : nullptr;

    float v[U][UNIT];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const int u = threadIdx.x + j * tpr;
#pragma unroll
        for (int i = 0; i < UNIT; ++i) v[j][i] = 0.f;
        if (live && u < units) {
            load_unit(x + u * UNIT, v[j]);
            if (r) {
                float a[UNIT];
                load_unit(r + u * UNIT, a);
#pragma unroll
                for (int i = 0; i < UNIT; ++i) v[j][i] += a[i];
            }
            // the norm takes the rounded h, so that the gradient from a stored h is the gradient of
            // what was computed
#pragma unroll
            for (int i = 0; i < UNIT; ++i) {
                v[j][i] = round_as((const HT *)nullptr, v[j][i]);
                sum = fmaf(v[j][i], v[j][i], sum);
            }
            if (h) store_unit(h + u * UNIT, v[j]);
        }
    }
    sum = row_sum(sum, red);
    const float rstd = 1.f / sqrtf(sum / (float)p.K + p.eps);
    if (live && threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;

#pragma unroll
    for (int j = 0; j < U; ++j) {
        const int u = threadIdx.x + j * tpr;
        const bool on = live && u < units;
        if (on) {
            float w[UNIT];
            load_unit(p.w + u * UNIT, w);
#pragma unroll
            for (int i = 0; i < UNIT; ++i) v[j][i] = v[j][i] * rstd * w[i];
        }
        if constexpr (sizeof(YT) == 1) {
            uint32_t code;
            const uint2 q = quantise_unit(v[j], code);
            if (on) {
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.y) + row * p.K + u * UNIT) = q;
                if ((u & 3) == 0) p.sf[row * ((p.K + BLOCK - 1) / BLOCK) + u / 4] = (uint8_t)code;
            }
        } else if (on) {
            store_unit(static_cast<YT *>(p.y) + row * p.K + u * UNIT, v[j]);
        }
    }
}

struct NormBackParams {
    const void *dy, *dh, *h;
    const float *rstd, *w;
    void *dx, *y;
    float *parts;        // one row of K per CTA, or null when dw is not wanted
    int64_t M;
    int K;
};

template <typename GT, typename HT, typename YT, int U>
__global__ void __launch_bounds__(U == 4 ? 1024 : 512) norm_back_kernel(NormBackParams p) {
    extern __shared__ float shared[];                  // rpc rows of K sums (rpc > 1)
    __shared__ float red[2][MAX_WARPS];
    const int units = p.K / UNIT, tpr = blockDim.x;
    float dw[U][UNIT];
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
        for (int i = 0; i < UNIT; ++i) dw[j][i] = 0.f;

    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * blockDim.y; first < p.M; first += step, turn ^= 1) {
        const int64_t row = first + threadIdx.y;
        const bool live = row < p.M;
        const float rstd = live ? p.rstd[row] : 0.f;
        float g[U][UNIT], n[U][UNIT];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int u = threadIdx.x + j * tpr;
            if (live && u < units) {
                float w[UNIT];
                load_unit(static_cast<const GT *>(p.dy) + row * p.K + u * UNIT, g[j]);
                load_unit(static_cast<const HT *>(p.h) + row * p.K + u * UNIT, n[j]);
                load_unit(p.w + u * UNIT, w);
#pragma unroll
                for (int i = 0; i < UNIT; ++i) {
                    n[j][i] *= rstd;
                    dw[j][i] = fmaf(g[j][i], n[j][i], dw[j][i]);
                    g[j][i] *= w[i];
                    sum = fmaf(g[j][i], n[j][i], sum);
                }
                if (p.y) {
                    float y[UNIT];
#pragma unroll
                    for (int i = 0; i < UNIT; ++i) y[i] = n[j][i] * w[i];
                    store_unit(static_cast<YT *>(p.y) + row * p.K + u * UNIT, y);
                }
            }
        }
        const float c = row_sum(sum, red[turn]) / (float)p.K;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int u = threadIdx.x + j * tpr;
            if (live && u < units) {
                float d[UNIT];
#pragma unroll
                for (int i = 0; i < UNIT; ++i) d[i] = 0.f;
                if (p.dh) load_unit(static_cast<const HT *>(p.dh) + row * p.K + u * UNIT, d);
#pragma unroll
                for (int i = 0; i < UNIT; ++i) d[i] += rstd * (g[j][i] - n[j][i] * c);
                store_unit(static_cast<HT *>(p.dx) + row * p.K + u * UNIT, d);
            }
        }
    }
    if (!p.parts) return;

    // the CTA's sums in a fixed order: rows of threads first, then (norm_dw_kernel) CTAs
    float *part = p.parts + (int64_t)blockIdx.x * p.K;
    if (blockDim.y == 1) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int u = threadIdx.x + j * tpr;
            if (u < units) store_unit(part + u * UNIT, dw[j]);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const int u = threadIdx.x + j * tpr;
        if (u < units) store_unit(shared + threadIdx.y * p.K + u * UNIT, dw[j]);
    }
    __syncthreads();
    for (int k = threadIdx.y * tpr + threadIdx.x; k < p.K; k += tpr * blockDim.y) {
        float s = 0.f;
        for (int y = 0; y < (int)blockDim.y; ++y) s += shared[y * p.K + k];
        part[k] = s;
    }
}

// dw[k] = sum of the CTAs' rows, in order: 32 columns per CTA, its warps share the rows out
__global__ void __launch_bounds__(256) norm_dw_kernel(const float *__restrict__ parts, int n, int K, float *__restrict__ dw) {
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, k = blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (k < K)
        for (int i = warp; i < n; i += 8) sum += parts[(int64_t)i * K + k];
    s[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && k < K) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += s[i][lane];
        dw[k] = t;
    }
}

template <typename XT, typename HT, typename YT>
cudaError_t norm_launch(const RowShape &s, const NormParams &p, cudaStream_t stream) {
    const dim3 block(s.tpr, s.rpc);
    const int64_t ctas = (p.M + s.rpc - 1) / s.rpc;
    if (s.u == 1) norm_kernel<XT, HT, YT, 1><<<(unsigned)ctas, block, 0, stream>>>(p);
    else if (s.u == 2) norm_kernel<XT, HT, YT, 2><<<(unsigned)ctas, block, 0, stream>>>(p);
    else norm_kernel<XT, HT, YT, 4><<<(unsigned)ctas, block, 0, stream>>>(p);
    return cudaGetLastError();
}
template <typename XT, typename HT>
cudaError_t norm_launch(gemm_dtype y, const RowShape &s, const NormParams &p, cudaStream_t stream) {
    if (y == GEMM_E4M3) return norm_launch<XT, HT, uint8_t>(s, p, stream);
    if (y == GEMM_BF16) return norm_launch<XT, HT, __nv_bfloat16>(s, p, stream);
    return norm_launch<XT, HT, __half>(s, p, stream);
}
template <typename XT>
cudaError_t norm_launch(gemm_dtype h, gemm_dtype y, const RowShape &s, const NormParams &p, cudaStream_t stream) {
    return h == GEMM_F32 ? norm_launch<XT, float>(y, s, p, stream) : norm_launch<XT, __nv_bfloat16>(y, s, p, stream);
}

template <typename GT, typename HT, typename YT>
cudaError_t back_launch(const RowShape &s, int ctas, const NormBackParams &p, cudaStream_t stream) {
    const dim3 block(s.tpr, s.rpc);
    const size_t smem = s.rpc > 1 && p.parts ? (size_t)s.rpc * p.K * sizeof(float) : 0;
    if (s.u == 1) norm_back_kernel<GT, HT, YT, 1><<<ctas, block, smem, stream>>>(p);
    else if (s.u == 2) norm_back_kernel<GT, HT, YT, 2><<<ctas, block, smem, stream>>>(p);
    else norm_back_kernel<GT, HT, YT, 4><<<ctas, block, smem, stream>>>(p);
    return cudaGetLastError();
}
template <typename GT, typename HT>
cudaError_t back_launch(gemm_dtype y, const RowShape &s, int ctas, const NormBackParams &p, cudaStream_t stream) {
    return y == GEMM_F16 ? back_launch<GT, HT, __half>(s, ctas, p, stream)
                         : back_launch<GT, HT, __nv_bfloat16>(s, ctas, p, stream);
}
template <typename GT>
cudaError_t back_launch(gemm_dtype h, gemm_dtype y, const RowShape &s, int ctas, const NormBackParams &p,
                        cudaStream_t stream) {
    return h == GEMM_F32 ? back_launch<GT, float>(y, s, ctas, p, stream)
                         : back_launch<GT, __nv_bfloat16>(y, s, ctas, p, stream);
}

bool real(gemm_dtype t) { return t == GEMM_F32 || t == GEMM_BF16; }
gemm_status check_sizes(int64_t M, int64_t K) {
    if (M < 0 || K <= 0 || M > INT32_MAX) return GEMM_ERR_INVALID_ARG;
    if (K > MAX_K) return GEMM_ERR_UNSUPPORTED;
    return K % 16 == 0 ? GEMM_OK : GEMM_ERR_ALIGNMENT;
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" gemm_status gemm_norm_run(int64_t M, int64_t K, gemm_dtype x, gemm_dtype h, gemm_dtype y, float eps,
                                     const void *X, const void *R, const float *W, void *H, void *Y, uint8_t *SFY,
                                     float *RSTD, void *cuda_stream) {
    if (!(eps >= 0.f)) return GEMM_ERR_INVALID_ARG;
    gemm_status st = check_sizes(M, K);
    if (st == GEMM_ERR_INVALID_ARG) return st;
    if (!real(x) || !real(h) || (y != GEMM_E4M3 && y != GEMM_BF16 && y != GEMM_F16)) return GEMM_ERR_UNSUPPORTED;
    if (st != GEMM_OK) return st;
    if (M == 0) return GEMM_OK;
    if (!X || !W || !Y || (y == GEMM_E4M3 && !SFY)) return GEMM_ERR_INVALID_ARG;
    for (const void *p : {X, R, (const void *)W, (const void *)H, (const void *)Y})
        if (!rows::aligned16(p)) return GEMM_ERR_ALIGNMENT;
    int sms = 0;
    st = rows::device_sms(&sms);
    if (st != GEMM_OK) return st;
    const NormParams p{X, R, W, H, Y, SFY, RSTD, M, (int)K, eps};
    const RowShape s = row_shape((int)K);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = x == GEMM_F32 ? norm_launch<float>(h, y, s, p, stream)
                                        : norm_launch<__nv_bfloat16>(h, y, s, p, stream);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

extern "C" gemm_status gemm_norm_backward(int64_t M, int64_t K, gemm_dtype dy, gemm_dtype h, gemm_dtype y,
                                          const void *DY, const void *DH, const void *H, const float *RSTD,
                                          const float *W, void *DX, float *DW, void *Y, void *workspace,
                                          size_t workspace_bytes, void *cuda_stream) {
    gemm_status st = check_sizes(M, K);
    if (st == GEMM_ERR_INVALID_ARG) return st;
    if (!real(dy) || !real(h) || (Y && y != GEMM_BF16 && y != GEMM_F16)) return GEMM_ERR_UNSUPPORTED;
    if (st != GEMM_OK) return st;
    if (M > 0 && (!DY || !H || !RSTD || !W || !DX)) return GEMM_ERR_INVALID_ARG;
    const int64_t parts_max = M < GEMM_NORM_PARTS ? M : GEMM_NORM_PARTS;
    if (DW && M > 0 && (!workspace || workspace_bytes < (size_t)parts_max * K * sizeof(float))) return GEMM_ERR_INVALID_ARG;
    for (const void *p : {DY, DH, H, (const void *)W, (const void *)DX, (const void *)DW, (const void *)Y,
                          (const void *)workspace})
        if (!rows::aligned16(p)) return GEMM_ERR_ALIGNMENT;
    if (M == 0 && !DW) return GEMM_OK;
    int sms = 0;
    st = rows::device_sms(&sms);
    if (st != GEMM_OK) return st;

    cudaStream_t stream = reinterpret_cast<cudaStream_t>(cuda_stream);
    const RowShape s = row_shape((int)K);
    const int64_t groups = (M + s.rpc - 1) / s.rpc;
    const int64_t most = (int64_t)sms * 2 < GEMM_NORM_PARTS ? sms * 2 : GEMM_NORM_PARTS;
    const int ctas = (int)(groups < most ? groups : most);
    if (M > 0) {
        const NormBackParams p{DY, DH, H, RSTD, W, DX, Y, DW ? static_cast<float *>(workspace) : nullptr, M, (int)K};
        const cudaError_t e = dy == GEMM_F32 ? back_launch<float>(h, y, s, ctas, p, stream)
                                             : back_launch<__nv_bfloat16>(h, y, s, ctas, p, stream);
        if (e != cudaSuccess) return GEMM_ERR_CUDA;
    }
    if (DW) {
        norm_dw_kernel<<<(unsigned)((K + 31) / 32), 256, 0, stream>>>(static_cast<const float *>(workspace), ctas,
                                                                      (int)K, DW);
        if (cudaGetLastError() != cudaSuccess) return GEMM_ERR_CUDA;
    }
    return GEMM_OK;
}

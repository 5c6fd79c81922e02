// The gated unit between a feed-forward block's two products, with an 8-bit checkpoint for its
// gradient (gemm_gate_run, gemm_gate_backward in include/gb300gemm.h).
//
//   z = [g | u],  s = 1 / (1 + exp(-g)),  a = g * s * u
//   dg = da * u * s * (1 + g * (1 - s)),  du = da * g * s
//
// The checkpoint keeps g and u as e4m3 codes with a UE8M0 scale per 32: a quarter of fp32's bytes.
// The gradient is that of the unit at the checkpoint's values.  Both kernels are one pass over
// memory: a thread takes eight consecutive elements of each half of a row.
#include <initializer_list>

#include "gemm_rows.cuh"

namespace gb300 {
namespace {

using namespace rows;

// s * g and s itself; exp(-g) infinite gives s = 0
__device__ __forceinline__ float sigmoid(float g) { return 1.f / (1.f + __expf(-g)); }

struct GateParams {
    const void *z;
    void *a;
    uint8_t *sfa, *ck, *sfck;
    int64_t M;
    int F;
};

// Units are counted as if every row had whole blocks of four, so that a block never straddles the
// lanes of two rows; the units past a row's end do nothing.
__device__ __forceinline__ bool place(int64_t i, int per_row, int F, int64_t M, int64_t &row, int &u) {
    row = i / per_row;
    u = (int)(i - row * per_row);
    return row < M && u * UNIT < F;
}

template <typename ZT, typename AT>
__global__ void __launch_bounds__(256) gate_kernel(GateParams p) {
    const int blocks = (p.F + BLOCK - 1) / BLOCK, per_row = blocks * 4;
    int64_t row;
    int u;
    const bool on = place((int64_t)blockIdx.x * 256 + threadIdx.x, per_row, p.F, p.M, row, u);
    float g[UNIT], v[UNIT], a[UNIT];
#pragma unroll
    for (int i = 0; i < UNIT; ++i) g[i] = v[i] = 0.f;
    if (on) {
        const ZT *z = static_cast<const ZT *>(p.z) + row * 2 * p.F + u * UNIT;
        load_unit(z, g);
        load_unit(z + p.F, v);
    }
#pragma unroll
    for (int i = 0; i < UNIT; ++i) a[i] = g[i] * sigmoid(g[i]) * v[i];
    uint32_t code;
    if constexpr (sizeof(AT) == 1) {
        const uint2 q = quantise_unit(a, code);
        if (on) {
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.a) + row * p.F + u * UNIT) = q;
            if ((u & 3) == 0) p.sfa[row * blocks + u / 4] = (uint8_t)code;
        }
    } else if (on) {
        store_unit(static_cast<AT *>(p.a) + row * p.F + u * UNIT, a);
    }
    if (p.ck) {
        uint8_t *ck = p.ck + row * 2 * p.F + u * UNIT, *sf = p.sfck + row * 2 * blocks + u / 4;
        uint2 q = quantise_unit(g, code);
        if (on) {
            *reinterpret_cast<uint2 *>(ck) = q;
            if ((u & 3) == 0) sf[0] = (uint8_t)code;
        }
        q = quantise_unit(v, code);
        if (on) {
            *reinterpret_cast<uint2 *>(ck + p.F) = q;
            if ((u & 3) == 0) sf[blocks] = (uint8_t)code;
        }
    }
}

struct GateBackParams {
    const void *da;
    const uint8_t *ck, *sfck;
    void *dz, *a;
    int64_t M;
    int F;
};

template <typename GT, typename ZT, typename AT>
__global__ void __launch_bounds__(256) gate_back_kernel(GateBackParams p) {
    const int blocks = (p.F + BLOCK - 1) / BLOCK;
    int64_t row;
    int u;
    if (!place((int64_t)blockIdx.x * 256 + threadIdx.x, p.F / UNIT, p.F, p.M, row, u)) return;
    const uint8_t *ck = p.ck + row * 2 * p.F + u * UNIT, *sf = p.sfck + row * 2 * blocks + u / 4;
    float g[UNIT], v[UNIT], d[UNIT], a[UNIT];
    load_unit(static_cast<const GT *>(p.da) + row * p.F + u * UNIT, d);
    decode_unit(*reinterpret_cast<const uint2 *>(ck), scale_value(sf[0]), g);
    decode_unit(*reinterpret_cast<const uint2 *>(ck + p.F), scale_value(sf[blocks]), v);
#pragma unroll
    for (int i = 0; i < UNIT; ++i) {
        const float s = sigmoid(g[i]), gs = g[i] * s, dgs = s * (1.f + g[i] * (1.f - s));
        a[i] = gs * v[i];
        g[i] = d[i] * v[i] * dgs;
        d[i] *= gs;
    }
    ZT *dz = static_cast<ZT *>(p.dz) + row * 2 * p.F + u * UNIT;
    store_unit(dz, g);
    store_unit(dz + p.F, d);
    if (p.a) store_unit(static_cast<AT *>(p.a) + row * p.F + u * UNIT, a);
}

// CTAs for n threads' work
unsigned ctas(int64_t n) { return (unsigned)((n + 255) / 256); }

template <typename ZT>
cudaError_t gate_launch(gemm_dtype a, unsigned n, const GateParams &p, cudaStream_t stream) {
    if (a == GEMM_E4M3) gate_kernel<ZT, uint8_t><<<n, 256, 0, stream>>>(p);
    else if (a == GEMM_BF16) gate_kernel<ZT, __nv_bfloat16><<<n, 256, 0, stream>>>(p);
    else gate_kernel<ZT, __half><<<n, 256, 0, stream>>>(p);
    return cudaGetLastError();
}
template <typename GT, typename ZT>
cudaError_t back_launch(gemm_dtype a, unsigned n, const GateBackParams &p, cudaStream_t stream) {
    if (a == GEMM_F16) gate_back_kernel<GT, ZT, __half><<<n, 256, 0, stream>>>(p);
    else gate_back_kernel<GT, ZT, __nv_bfloat16><<<n, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

bool real(gemm_dtype t) { return t == GEMM_F32 || t == GEMM_BF16; }
gemm_status check_sizes(int64_t M, int64_t F) {
    if (M < 0 || F <= 0 || M > INT32_MAX || F > (1 << 20)) return GEMM_ERR_INVALID_ARG;
    if (M * ((F + BLOCK - 1) / BLOCK * 4) / 256 >= INT32_MAX) return GEMM_ERR_UNSUPPORTED;   // more CTAs than a launch holds
    return F % 16 == 0 ? GEMM_OK : GEMM_ERR_ALIGNMENT;
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" gemm_status gemm_gate_run(int64_t M, int64_t F, gemm_dtype z, gemm_dtype a, const void *Z, void *A,
                                     uint8_t *SFA, uint8_t *CK, uint8_t *SFCK, void *cuda_stream) {
    gemm_status st = check_sizes(M, F);
    if (st == GEMM_ERR_INVALID_ARG || st == GEMM_ERR_UNSUPPORTED) return st;
    if (!real(z) || (a != GEMM_E4M3 && a != GEMM_BF16 && a != GEMM_F16)) return GEMM_ERR_UNSUPPORTED;
    if (st != GEMM_OK || M == 0) return st;
    if (!Z || !A || (a == GEMM_E4M3 && !SFA) || (CK && !SFCK)) return GEMM_ERR_INVALID_ARG;
    for (const void *p : {Z, (const void *)A, (const void *)CK})
        if (!rows::aligned16(p)) return GEMM_ERR_ALIGNMENT;
    int sms = 0;
    st = rows::device_sms(&sms);
    if (st != GEMM_OK) return st;
    const GateParams p{Z, A, SFA, CK, SFCK, M, (int)F};
    const unsigned n = ctas(M * ((F + BLOCK - 1) / BLOCK * 4));
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = z == GEMM_F32 ? gate_launch<float>(a, n, p, stream)
                                        : gate_launch<__nv_bfloat16>(a, n, p, stream);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

extern "C" gemm_status gemm_gate_backward(int64_t M, int64_t F, gemm_dtype da, gemm_dtype dz, gemm_dtype a,
                                          const void *DA, const uint8_t *CK, const uint8_t *SFCK, void *DZ, void *A,
                                          void *cuda_stream) {
    gemm_status st = check_sizes(M, F);
    if (st == GEMM_ERR_INVALID_ARG || st == GEMM_ERR_UNSUPPORTED) return st;
    if (!real(da) || !real(dz) || (A && a != GEMM_BF16 && a != GEMM_F16)) return GEMM_ERR_UNSUPPORTED;
    if (st != GEMM_OK || M == 0) return st;
    if (!DA || !CK || !SFCK || !DZ) return GEMM_ERR_INVALID_ARG;
    for (const void *p : {DA, (const void *)CK, (const void *)DZ, (const void *)A})
        if (!rows::aligned16(p)) return GEMM_ERR_ALIGNMENT;
    int sms = 0;
    st = rows::device_sms(&sms);
    if (st != GEMM_OK) return st;
    const GateBackParams p{DA, CK, SFCK, DZ, A, M, (int)F};
    const unsigned n = ctas(M * (F / UNIT));
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(cuda_stream);
    cudaError_t e;
    if (da == GEMM_F32)
        e = dz == GEMM_F32 ? back_launch<float, float>(a, n, p, stream) : back_launch<float, __nv_bfloat16>(a, n, p, stream);
    else
        e = dz == GEMM_F32 ? back_launch<__nv_bfloat16, float>(a, n, p, stream)
                           : back_launch<__nv_bfloat16, __nv_bfloat16>(a, n, p, stream);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

// The gated unit between a feed-forward block's two products, with an 8-bit checkpoint for its
// gradient (gemm_gate_run, gemm_gate_backward in include/gb300gemm.h).
//
//   z = [g | u],  s = 1 / (1 + exp(-g)),  a = g * s * u
//   dg = da * u * s * (1 + g * (1 - s)),  du = da * g * s
//
// The checkpoint keeps g and u as e4m3 codes with a UE8M0 scale per 32: a quarter of fp32's bytes.
// The gradient is that of the unit at the checkpoint's values.  Both kernels are one pass over
// memory: a thread takes 16 (forward) or 8 (backward) consecutive elements of each half of a row.
#include <initializer_list>

#include "gemm_rows.cuh"

namespace gb300 {
namespace {

using namespace rows;

// s = 1 / (1 + exp(-g)) and t = 1 - s = exp(-g) s, which a subtraction would leave few digits of.  With p = 2^-16 exp(-g / 2)
// both come from r = 1 / (p^2 + 2^-32) = 2^32 s, which is a normal number wherever s is not zero: s goes down to fp32's
// smallest number, at g = -103, and t to 2^-117.  (Where s is zero t is no matter, but has to be finite.)  The fast
// exponential and reciprocal (p^2: 4 + 1.173 |g| units in the last place, r: 1) are what the outputs' 8 or 16 bits, or a
// comparison at 1e-6, have room for.
__device__ __forceinline__ void sigmoid(float g, float &s, float &t) {
    float p, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(g * -0.72134752f));                     // log2(e) / 2
    p *= 0x1p-16f;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(p, p, 0x1p-32f)));
    s = r * 0x1p-32f;
    t = fminf(p * p, 0x1p126f) * r;
}

struct GateParams {
    const void *z;
    void *a;
    uint8_t *sfa, *ck, *sfck;
    Units units;
    int F;
};

// Bound by memory: z in, a and the checkpoint out, once each.  A thread takes half a scale's block, so that two lanes
// settle its largest magnitude and the units are as wide as 64 registers allow: four CTAs per SM.  4096 x 8192, bf16 to
// e4m3 with checkpoint: 37.7 us, 6320 GB/s (93% of a copy's rate); three CTAs per SM take 41.0 us, five spill: 46.7.
// 1 x 8192: 1.5 us, a launch and one trip to memory.
template <typename ZT, typename AT>
__global__ void __launch_bounds__(256, 4) gate_kernel(const __grid_constant__ GateParams p) {
    constexpr int N = 16;
    const int blocks = (p.F + BLOCK - 1) / BLOCK;
    int64_t row;
    int u;
    const bool on = p.units.place(blockIdx.x * 256 + threadIdx.x, row, u) && u * N < p.F;
    float g[N], v[N], a[N];
    wait_for_previous();
    let_next_launch();
    {
        uint4 gq[PIECES<ZT, N>], vq[PIECES<ZT, N>];
        const ZT *z = static_cast<const ZT *>(p.z) + row * 2 * p.F + u * N;
        load_pieces(z, on, gq);
        load_pieces(z + p.F, on, vq);
        unpack(z, gq, g);
        unpack(z, vq, v);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s, t;
        sigmoid(g[i], s, t);
        a[i] = g[i] * s * v[i];
    }
    const bool first = on && (u & 1) == 0;           // of its block
    uint32_t code;
    if constexpr (sizeof(AT) == 1) {
        code = quantise(a, static_cast<uint8_t *>(p.a) + row * p.F + u * N, on);
        if (first) p.sfa[row * blocks + u / 2] = (uint8_t)code;
    } else if (on) {
        store(static_cast<AT *>(p.a) + row * p.F + u * N, a);
    }
    if (p.ck) {
        uint8_t *ck = p.ck + row * 2 * p.F + u * N, *sf = p.sfck + row * 2 * blocks + u / 2;
        code = quantise(g, ck, on);
        if (first) sf[0] = (uint8_t)code;
        code = quantise(v, ck + p.F, on);
        if (first) sf[blocks] = (uint8_t)code;
    }
}

struct GateBackParams {
    const void *da;
    const uint8_t *ck, *sfck;
    void *dz, *a;
    Units units;
    int F;
};

// Bound by memory: da and the checkpoint in, dz (and a) out.  4096 x 8192, bf16 with a again: 50.0 us, 6750 GB/s (a
// copy's rate).  77 x 2064, fp32: 1.75 us, a launch and one trip to memory.
template <typename GT, typename ZT, typename AT>
__global__ void __launch_bounds__(256) gate_back_kernel(const __grid_constant__ GateBackParams p) {
    constexpr int N = 8;             // no block is shared: the smaller unit keeps each access of a warp contiguous
    const int blocks = (p.F + BLOCK - 1) / BLOCK;
    int64_t row;
    int u;
    wait_for_previous();
    let_next_launch();
    if (!p.units.place(blockIdx.x * 256 + threadIdx.x, row, u)) return;
    const uint8_t *ck = p.ck + row * 2 * p.F + u * N, *sf = p.sfck + row * 2 * blocks + u / 4;
    float g[N], v[N], d[N], a[N];
    load(static_cast<const GT *>(p.da) + row * p.F + u * N, d);
    decode(*reinterpret_cast<const uint2 *>(ck), scale_value(sf[0]), g);
    decode(*reinterpret_cast<const uint2 *>(ck + p.F), scale_value(sf[blocks]), v);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s, t;
        sigmoid(g[i], s, t);
        const float gs = g[i] * s, dgs = s * (1.f + g[i] * t);
        a[i] = gs * v[i];
        g[i] = d[i] * v[i] * dgs;
        d[i] *= gs;
    }
    ZT *dz = static_cast<ZT *>(p.dz) + row * 2 * p.F + u * N;
    store(dz, g);
    store(dz + p.F, d);
    if (p.a) store(static_cast<AT *>(p.a) + row * p.F + u * N, a);
}

template <typename ZT>
cudaError_t gate_launch(gemm_dtype a, unsigned n, const GateParams &p, cudaStream_t stream) {
    if (a == GEMM_E4M3) return launch(gate_kernel<ZT, uint8_t>, (int)n, 256, 0, stream, p);
    if (a == GEMM_BF16) return launch(gate_kernel<ZT, __nv_bfloat16>, (int)n, 256, 0, stream, p);
    return launch(gate_kernel<ZT, __half>, (int)n, 256, 0, stream, p);
}
template <typename GT, typename ZT>
cudaError_t back_launch(gemm_dtype a, unsigned n, const GateBackParams &p, cudaStream_t stream) {
    return a == GEMM_F16 ? launch(gate_back_kernel<GT, ZT, __half>, (int)n, 256, 0, stream, p)
                         : launch(gate_back_kernel<GT, ZT, __nv_bfloat16>, (int)n, 256, 0, stream, p);
}

bool real(gemm_dtype t) { return t == GEMM_F32 || t == GEMM_BF16; }
gemm_status check_sizes(int64_t M, int64_t F) {
    if (M < 0 || F <= 0 || M > INT32_MAX || F > (1 << 20)) return GEMM_ERR_INVALID_ARG;
    return F % 16 == 0 ? GEMM_OK : GEMM_ERR_ALIGNMENT;
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" gemm_status gemm_gate_run(int64_t M, int64_t F, gemm_dtype z, gemm_dtype a, const void *Z, void *A,
                                     uint8_t *SFA, uint8_t *CK, uint8_t *SFCK, void *cuda_stream) {
    gemm_status st = check_sizes(M, F);
    if (st == GEMM_ERR_INVALID_ARG) return st;
    if (!real(z) || (a != GEMM_E4M3 && a != GEMM_BF16 && a != GEMM_F16)) return GEMM_ERR_UNSUPPORTED;
    if (st != GEMM_OK || M == 0) return st;
    if (!Z || !A || (a == GEMM_E4M3 && !SFA) || (CK && !SFCK)) return GEMM_ERR_INVALID_ARG;
    for (const void *p : {Z, (const void *)A, (const void *)CK})
        if (!rows::aligned16(p)) return GEMM_ERR_ALIGNMENT;
    int sms = 0;
    st = rows::device_sms(&sms);
    if (st != GEMM_OK) return st;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(cuda_stream);
    GateParams p{Z, A, SFA, CK, SFCK, Units{}, (int)F};
    // whole blocks of two units per row, so that no block straddles the lanes of two rows
    return over_rows(M, (int)((F + BLOCK - 1) / BLOCK * 2), [&](const Units &units, unsigned n) {
        p.units = units;
        return z == GEMM_F32 ? gate_launch<float>(a, n, p, stream) : gate_launch<__nv_bfloat16>(a, n, p, stream);
    });
}

extern "C" gemm_status gemm_gate_backward(int64_t M, int64_t F, gemm_dtype da, gemm_dtype dz, gemm_dtype a,
                                          const void *DA, const uint8_t *CK, const uint8_t *SFCK, void *DZ, void *A,
                                          void *cuda_stream) {
    gemm_status st = check_sizes(M, F);
    if (st == GEMM_ERR_INVALID_ARG) return st;
    if (!real(da) || !real(dz) || (A && a != GEMM_BF16 && a != GEMM_F16)) return GEMM_ERR_UNSUPPORTED;
    if (st != GEMM_OK || M == 0) return st;
    if (!DA || !CK || !SFCK || !DZ) return GEMM_ERR_INVALID_ARG;
    for (const void *p : {DA, (const void *)CK, (const void *)DZ, (const void *)A})
        if (!rows::aligned16(p)) return GEMM_ERR_ALIGNMENT;
    int sms = 0;
    st = rows::device_sms(&sms);
    if (st != GEMM_OK) return st;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(cuda_stream);
    GateBackParams p{DA, CK, SFCK, DZ, A, Units{}, (int)F};
    return over_rows(M, (int)(F / 8), [&](const Units &units, unsigned n) {
        p.units = units;
        if (da == GEMM_F32)
            return dz == GEMM_F32 ? back_launch<float, float>(a, n, p, stream)
                                  : back_launch<float, __nv_bfloat16>(a, n, p, stream);
        return dz == GEMM_F32 ? back_launch<__nv_bfloat16, float>(a, n, p, stream)
                              : back_launch<__nv_bfloat16, __nv_bfloat16>(a, n, p, stream);
    });
}

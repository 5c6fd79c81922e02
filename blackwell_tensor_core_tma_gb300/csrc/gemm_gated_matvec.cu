// The gated product for 1 to 16 rows (gemm_gated_matvec_run in include/gb300gemm.h): one token, or a few, through
// the weights of a gated plan.
//
//   g = x·Wgᵀ, u = x·Wuᵀ, a = g / (1 + exp(-g)) * u
//
// Bound by the weights' bytes, which pass once from memory to registers.  The product runs on mma.sync m16n8k16: its 16
// rows are 8 rows of Wg and the same 8 of Wu, its 8 columns tokens, so that an element's g and u end up in one thread and
// the tokens that are not there cost nothing but idle lanes of an otherwise idle unit.  The order of k within an MMA is
// free as long as both operands agree on it: a lane takes 16 consecutive bytes of a weight row, whatever k they are, and the
// same k of its token.
//
// A CTA takes 8 G columns of A; its eight warps, and the CTAs of a cluster where columns are few, share K out in
// chunks and join their sums through shared memory, always in the same order.
//
// e4m3 weights become bf16 exactly: the code's exponent and mantissa bits stand at the bottom of a bf16's, which is the
// value times 2^-120, and one multiplication by 2^120 times the block's scale makes it the weight.  fp16 activations are
// split into two bf16 values whose sum they are.
#include <type_traits>

#include "gemm_rows.cuh"

namespace gb300 {
namespace {

using namespace rows;

constexpr int WARPS = 8;
constexpr int MAX_ROWS = 16;
constexpr int MAX_CLUSTER = 8;

struct FewParams {
    const void *x;
    const uint8_t *w, *sfw;
    void *a;
    int M, F, K;
    int chunks;              // of K
};

template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// weights: read once, not kept in L1 beside the activations
__device__ __forceinline__ uint4 load_once(const void *p, bool on) {
    uint4 q = make_uint4(0, 0, 0, 0);
    if (on)
        asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                     : "l"(p));
    return q;
}

// The factors that make a scaled weight of an e4m3 code's bits: 2^(120 + c - 127), which passes bf16's range from
// c = 135 on, and then the rest
__device__ __forceinline__ uint32_t low_factor(uint32_t c) { return (min(c, 134u) + 120u) << 7; }
__device__ __forceinline__ uint32_t high_factor(uint32_t c) { return (c > 134u ? c - 134u + 127u : 127u) << 7; }
__device__ __forceinline__ uint32_t times(uint32_t v, uint32_t f) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(f | f << 16));
    return r;
}
// codes 0 and 2 (even) or 1 and 3 (odd) of a word, in bf16, times the factors
__device__ __forceinline__ uint32_t widen_even(uint32_t w) { return (w << 4 & 0x07F007F0u) | (w << 8 & 0x80008000u); }
__device__ __forceinline__ uint32_t widen_odd(uint32_t w) { return (w >> 4 & 0x07F007F0u) | (w & 0x80008000u); }

// bit 7 of each byte: the code is NaN (bits besides those may be set too)
__device__ __forceinline__ uint32_t not_a_number(uint32_t w) { return (w & 0x7F7F7F7Fu) + 0x01010101u; }

__device__ __forceinline__ uint32_t lane_of(const uint4 &q, int i) { return i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w; }

// two fp16 values as two pairs of bf16 values that sum to them
__device__ __forceinline__ void split(uint32_t h, uint32_t &hi, uint32_t &lo) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    hi = pack2(static_cast<const __nv_bfloat16 *>(nullptr), f.x, f.y);
    lo = pack2(static_cast<const __nv_bfloat16 *>(nullptr), f.x - __uint_as_float(hi << 16), f.y - __uint_as_float(hi & 0xFFFF0000u));
}

// U loads of 16 bytes per weight row, chunk and lane: their k, four lanes side by side
template <bool E4M3>
constexpr int STEP_K = E4M3 ? 64 : 32;

template <typename XT, bool E4M3, int NG, int G, int U>
__global__ void __launch_bounds__(WARPS * 32) few_kernel(const __grid_constant__ FewParams p) {
    constexpr bool X_BF16 = sizeof(XT) == 2 && std::is_same<XT, __nv_bfloat16>::value;
    constexpr int CHUNK = STEP_K<E4M3> * U, WB = E4M3 ? 1 : 2, XP = E4M3 ? 2 : 1;
    constexpr int OUTPUTS = 64 * G * NG;
    __shared__ float part[WARPS][G][NG][4][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, r = lane / 4, t = lane % 4;
    uint32_t rank, ranks;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    const int f0 = (int)(blockIdx.x / ranks) * 8 * G;
    const int64_t row_bytes = (int64_t)p.K * WB;
    const int blocks = (p.K + BLOCK - 1) / BLOCK;
    wait_for_previous();
    let_next_launch();

    float acc[G][NG][4] = {};
    uint32_t nan[G][2] = {};                              // bits 7, 15, 23, 31: a code or scale of the row is NaN
    const XT *x = static_cast<const XT *>(p.x);
    for (int c = warp + WARPS * (int)rank; c < p.chunks; c += WARPS * (int)ranks) {
        uint4 w[U][G][2], xq[U][NG][XP];
        uint32_t sf[U][G][2];
#pragma unroll
        for (int s = 0; s < U; ++s) {
            const int k = c * CHUNK + s * STEP_K<E4M3> + t * (16 / WB);
            const bool in = k < p.K;
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const int f = f0 + 8 * i + r;
                const bool on = in && f < p.F;
                const uint8_t *g = p.w + f * row_bytes + (int64_t)k * WB;
                w[s][i][0] = load_once(g, on);
                w[s][i][1] = load_once(g + p.F * row_bytes, on);
                if constexpr (E4M3) {
                    const uint8_t *q = p.sfw + (int64_t)f * blocks + k / BLOCK;
                    sf[s][i][0] = on ? __ldg(q) : 127u;
                    sf[s][i][1] = on ? __ldg(q + (int64_t)p.F * blocks) : 127u;
                }
            }
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const int m = 8 * j + r;
#pragma unroll
                for (int h = 0; h < XP; ++h)
                    xq[s][j][h] = in && m < p.M ? __ldg(reinterpret_cast<const uint4 *>(x + (int64_t)m * p.K + k) + h)
                                                : make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int s = 0; s < U; ++s) {
            if constexpr (!E4M3) {
#pragma unroll
                for (int i = 0; i < G; ++i)
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        const uint4 &g = w[s][i][0], &u = w[s][i][1], &v = xq[s][j][0];
                        mma<X_BF16>(acc[i][j], g.x, u.x, g.y, u.y, v.x, v.y);
                        mma<X_BF16>(acc[i][j], g.z, u.z, g.w, u.w, v.z, v.w);
                    }
            } else {
                uint32_t most = 0;
#pragma unroll
                for (int i = 0; i < G; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 &q = w[s][i][h];
                        const uint32_t n0 = not_a_number(q.x) | not_a_number(q.y), n1 = not_a_number(q.z) | not_a_number(q.w);
                        nan[i][h] |= n0 | n1 | ((sf[s][i][h] + 1u) & 0x100u) >> 1;
                        most = max(most, sf[s][i][h]);
                    }
                const bool far = __any_sync(0xFFFFFFFFu, most > 134u);
#pragma unroll
                for (int o = 0; o < 4; ++o) {             // four k of each lane at a time
                    uint32_t b[NG][X_BF16 ? 1 : 2][2];
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        const uint4 &v = xq[s][j][o / 2];
                        const uint32_t v0 = o % 2 ? v.z : v.x, v1 = o % 2 ? v.w : v.y;
                        const uint32_t even = __byte_perm(v0, v1, 0x5410), odd = __byte_perm(v0, v1, 0x7632);
                        if constexpr (X_BF16) {
                            b[j][0][0] = even;
                            b[j][0][1] = odd;
                        } else {
                            split(even, b[j][0][0], b[j][1][0]);
                            split(odd, b[j][0][1], b[j][1][1]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < G; ++i) {
                        uint32_t a[4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t q = lane_of(w[s][i][h], o), f = low_factor(sf[s][i][h]);
                            a[h] = times(widen_even(q), f);
                            a[2 + h] = times(widen_odd(q), f);
                            if (far) {
                                const uint32_t rest = high_factor(sf[s][i][h]);
                                a[h] = times(a[h], rest);
                                a[2 + h] = times(a[2 + h], rest);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < NG; ++j)
#pragma unroll
                            for (int h = 0; h < (X_BF16 ? 1 : 2); ++h)
                                mma<true>(acc[i][j], a[0], a[1], a[2], a[3], b[j][h][0], b[j][h][1]);
                    }
                }
            }
        }
    }
    if constexpr (E4M3) {                                 // a row with such a weight has no other sum
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t n = nan[i][h] & 0x80808080u;
                n |= __shfl_xor_sync(0xFFFFFFFFu, n, 1);
                n |= __shfl_xor_sync(0xFFFFFFFFu, n, 2);
                if (n)
#pragma unroll
                    for (int j = 0; j < NG; ++j) acc[i][j][2 * h] = acc[i][j][2 * h + 1] = __int_as_float(0x7FFFFFFF);
            }
    }
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
        for (int j = 0; j < NG; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[warp][i][j][e][lane] = acc[i][j][e];
    __syncthreads();
    // output o: column f0 + 8 i + r of token 8 j + 2 t + e; elements e of a thread's sums are g, e + 2 are u
    float sums[(OUTPUTS + WARPS * 32 - 1) / (WARPS * 32)][2];
#pragma unroll
    for (int n = 0; n < (OUTPUTS + WARPS * 32 - 1) / (WARPS * 32); ++n) {
        const int o = n * WARPS * 32 + threadIdx.x;
        if (o >= OUTPUTS) break;
        const int i = o / (64 * NG), j = o / 64 % NG, e = o / 32 % 2, l = o % 32;
        sums[n][0] = sums[n][1] = 0.f;
#pragma unroll
        for (int k = 0; k < WARPS; ++k) {
            sums[n][0] += part[k][i][j][e][l];
            sums[n][1] += part[k][i][j][e + 2][l];
        }
    }
    float *own = &part[0][0][0][0][0];                    // the CTA's sums, once the warps' have been read
    if (ranks > 1) {
        __syncthreads();
#pragma unroll
        for (int n = 0; n < (OUTPUTS + WARPS * 32 - 1) / (WARPS * 32); ++n) {
            const int o = n * WARPS * 32 + threadIdx.x;
            if (o >= OUTPUTS) break;
            own[2 * o] = sums[n][0];
            own[2 * o + 1] = sums[n][1];
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
#pragma unroll
    for (int n = 0; n < (OUTPUTS + WARPS * 32 - 1) / (WARPS * 32); ++n) {
        const int o = n * WARPS * 32 + threadIdx.x;
        if (o >= OUTPUTS) break;
        if (ranks > 1) {                                  // each CTA of the cluster finishes a share of the outputs
            if ((uint32_t)(o / 32) % ranks != rank) continue;
            sums[n][0] = sums[n][1] = 0.f;
            for (uint32_t q = 0; q < ranks; ++q) {
                uint32_t at;
                const uint32_t here = (uint32_t)__cvta_generic_to_shared(own + 2 * o);
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(here), "r"(q));
                float vg, vu;
                asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(vg), "=f"(vu) : "r"(at) : "memory");
                sums[n][0] += vg;
                sums[n][1] += vu;
            }
        }
        const int i = o / (64 * NG), j = o / 64 % NG, e = o / 32 % 2, l = o % 32;
        const int f = f0 + 8 * i + l / 4, m = 8 * j + 2 * (l % 4) + e;
        if (f < p.F && m < p.M) {
            float s1, s0;
            sigmoid(sums[n][0], s1, s0);
            const float v = sums[n][0] * s1 * sums[n][1];
            if constexpr (X_BF16) static_cast<__nv_bfloat16 *>(p.a)[(int64_t)m * p.F + f] = __float2bfloat16_rn(v);
            else static_cast<__half *>(p.a)[(int64_t)m * p.F + f] = __float2half_rn(v);
        }
    }
    // no CTA leaves while another may still read its sums
    if (ranks > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename XT, bool E4M3, int NG, int G, int U>
cudaError_t few_launch(FewParams p, int sms, cudaStream_t stream) {
    constexpr int CHUNK = STEP_K<E4M3> * U;
    p.chunks = (p.K + CHUNK - 1) / CHUNK;
    const int groups = (p.F + 8 * G - 1) / (8 * G);
    int cluster = 1;
    while (cluster < MAX_CLUSTER && groups * cluster * 2 <= 2 * sms && p.chunks > WARPS * cluster) cluster *= 2;
    const Launch l(groups * cluster, WARPS * 32, 0, cluster, stream);
    return cudaLaunchKernelEx(&l.config, few_kernel<XT, E4M3, NG, G, U>, p);
}

template <typename XT, bool E4M3>
cudaError_t few(const FewParams &p, int sms, cudaStream_t stream) {
    if (p.M <= 8) return few_launch<XT, E4M3, 1, 1, E4M3 ? 2 : 4>(p, sms, stream);
    return few_launch<XT, E4M3, 2, 2, 2>(p, sms, stream);
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" gemm_status gemm_gated_matvec_run(int64_t M, int64_t F, int64_t K, gemm_dtype x, gemm_dtype w, gemm_dtype a,
                                             const void *X, const void *W, const uint8_t *SFW, void *A, void *cuda_stream) {
    if (M < 0 || F <= 0 || K <= 0 || F > (1 << 20)) return GEMM_ERR_INVALID_ARG;
    if (M > MAX_ROWS || K > 32768) return GEMM_ERR_UNSUPPORTED;
    if ((x != GEMM_BF16 && x != GEMM_F16) || (w != x && w != GEMM_E4M3) || a != x) return GEMM_ERR_UNSUPPORTED;
    if (K % (w == GEMM_E4M3 ? 16 : 8) != 0) return GEMM_ERR_ALIGNMENT;
    if (M == 0) return GEMM_OK;
    if (!X || !W || !A || (w == GEMM_E4M3 && !SFW)) return GEMM_ERR_INVALID_ARG;
    for (const void *q : {X, W, (const void *)A})
        if (!rows::aligned16(q)) return GEMM_ERR_ALIGNMENT;
    int sms = 0;
    const gemm_status st = rows::device_sms(&sms);
    if (st != GEMM_OK) return st;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(cuda_stream);
    const FewParams p{X, static_cast<const uint8_t *>(W), SFW, A, (int)M, (int)F, (int)K, 0};
    cudaError_t e;
    if (x == GEMM_BF16) e = w == x ? few<__nv_bfloat16, false>(p, sms, stream) : few<__nv_bfloat16, true>(p, sms, stream);
    else e = w == x ? few<__half, false>(p, sms, stream) : few<__half, true>(p, sms, stream);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

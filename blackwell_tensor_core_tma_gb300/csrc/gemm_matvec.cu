// Matrix-vector products with 4-bit weights (gemm_matvec_run in include/gb300gemm.h): the form of
// the block-scaled e2m1 product for 1 to 16 rows of A, on the plans' own B and SFB buffers, with
// 16-bit activations.
//
//   D[m][n] = C[m][n] + sum_k x[m][k] * B[k][n] * sf(SFB[n][k / blk])
//
// The bound is the weights' bytes: half a byte per weight leaves an SM under three issue slots per
// weight at full HBM rate, which unpacking and multiplying in fp32 would pass several times over for
// more than one row.  So the weights become fp16 (one conversion for two of them, exact) and meet the
// activations in m16n8k16 MMAs with fp32 accumulators: 16 columns of B by 8 rows of X per MMA, and the cost per
// weight does not depend on M up to 8.  (tcgen05 would want 128-row operand tiles in shared or tensor
// memory, that is every weight written there once more; the tensor rate is not what bounds this.)
//
// A warp owns 16 columns (n) and a slice of K, which it walks in chunks of 128: lane (g, t) holds k =
// 32 t .. 32 t + 31 of columns g and g + 8, one 128-bit load each, straight from global memory (each
// weight is used by one lane: shared memory would only add a copy).  The order of k inside an MMA is free
// as long as both operands agree, so word j of a lane's four gives the A operand of MMAs 2j and 2j + 1, and
// the activations are laid out in shared memory in that order when the CTA starts.
//
// Scales.  UE4M3 (per 16): the product with an e2m1 value has at most six significant bits and
// lies within 2^-10 .. 2688, so it is exact in fp16: weights are scaled before the MMA.  UE8M0 (per 32): a
// lane's 32 k are one block; its weights are multiplied by 2^(c - max c of the column's four blocks in the
// chunk), exact in fp16 down to 2^-14, and the chunk's sum by 2^(max c - 127) in fp32.
// Activations.  fp16 goes in as it is.  bf16 is multiplied per row and chunk by the power of two that brings
// the largest magnitude to 2^15 .. 2^16, which is exact in fp16 for elements down to 2^-32 of it.
// What these rules do not hold exactly (scales further apart, activations too far apart, infinities, NaN)
// takes products_fp32 for that chunk: the same sums in fp32 from the original values.
//
// A CTA's eight warps are R row tiles (of 16 columns of B) by S slices of K, and `c` CTAs of a cluster split K
// further; the partial sums are joined in a fixed order through shared memory, the cluster's through
// distributed shared memory.
#include <initializer_list>
#include <mutex>
#include <type_traits>

#include "gemm_rows.cuh"
#include "ptx.cuh"

namespace gb300 {
namespace {

constexpr int MAX_M = 16;
constexpr int64_t MAX_K = 32768;
constexpr int WARPS = 8;
constexpr int CHUNK = 128;           // k per step of a warp
constexpr int AHEAD = 4;             // chunks in flight per warp: 1 KB of weights each

struct MatvecParams {
    const void *x;
    const uint8_t *b, *sfb;
    const float *c;
    void *d;
    int M, N, K;
    int out_bf16;
    int slices;          // slices of K per CTA (S)
    int chunk_room;      // chunks the activations' shared memory holds
};

// eight packed e2m1 values (k ascending from the low nibble) to four pairs of halves
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// two UE4M3 codes (bit 7 is not part of the format) to halves
__device__ __forceinline__ uint32_t ue4m3x2(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(codes & 0x7F7Fu)));
    return h;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float2 halves(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2 *>(&h)); }

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// weights: read once, not kept in L1; a request brings its whole line to L2
__device__ __forceinline__ uint4 load_weights(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ float load_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float2 pair_of(const __nv_bfloat16 *, uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 pair_of(const __half *, uint32_t w) { return halves(w); }

// One chunk's products in fp32 from the original values, for eight rows of X from m0: what lane (g, t) adds to
// its accumulators (columns g, g, g + 8, g + 8 by rows 2t, 2t + 1).  codes: the lane's scale codes of the two
// columns (UE8M0: one each, UE4M3: two each).
template <typename XT, int MODE>
__device__ __noinline__ float4 products_fp32(const void *x, int K, int M, int m0, int k0, uint4 qa, uint4 qb,
                                             uint32_t code_a, uint32_t code_b) {
    const int t = threadIdx.x & 3;
    float4 out = make_float4(0.f, 0.f, 0.f, 0.f);
    const uint32_t w[2][4] = {{qa.x, qa.y, qa.z, qa.w}, {qb.x, qb.y, qb.z, qb.w}};
    for (int m = 0; m < 8; ++m) {
        if (m0 + m >= M) break;
        float sum[2] = {0.f, 0.f};
        if (k0 < K) {
            const uint32_t *a = reinterpret_cast<const uint32_t *>(static_cast<const XT *>(x) + (int64_t)(m0 + m) * K + k0);
            for (int col = 0; col < 2; ++col) {
                const uint32_t code = col ? code_b : code_a;
                float part[2] = {0.f, 0.f};
                for (int i = 0; i < 4; ++i) {
                    uint32_t h[4];
                    e2m1x8(w[col][i], h);
                    for (int j = 0; j < 4; ++j) {
                        const float2 v = halves(h[j]), xv = pair_of((const XT *)nullptr, a[4 * i + j]);
                        part[i / 2] = fmaf(v.x, xv.x, fmaf(v.y, xv.y, part[i / 2]));
                    }
                }
                if (MODE == GEMM_SCALE_UE8M0_32) {
                    sum[col] = code == 255u ? __uint_as_float(0x7FC00000u) : ldexpf(part[0] + part[1], (int)code - 127);
                } else {
                    const float2 s = halves(ue4m3x2(code));
                    sum[col] = fmaf(part[0], s.x, part[1] * s.y);
                }
            }
        }
        for (int col = 0; col < 2; ++col) {
            sum[col] += __shfl_xor_sync(0xFFFFFFFFu, sum[col], 1);
            sum[col] += __shfl_xor_sync(0xFFFFFFFFu, sum[col], 2);
        }
        if (m / 2 == t) {
            (m & 1 ? out.y : out.x) += sum[0];
            (m & 1 ? out.w : out.z) += sum[1];
        }
    }
    return out;
}

// The CTA's chunks [lo, hi) of X into shared memory as the MMA's B operand: eight consecutive k (one 128-bit word)
// of row m, chunk lc at word ((lc * 4 + j) * M + m) * 4 + t for k = 32 t + 8 j.  bf16: scaled per (row, chunk);
// scale[lc * rows + m] undoes it, or is negative where the chunk of some row does not convert exactly.
template <typename XT>
__device__ __forceinline__ void stage_x(const MatvecParams &p, int lo, int hi, int rows_x, uint4 *xf, float *scale) {
    const int l = threadIdx.x & 15, j = l & 3, t = l >> 2;
    const int pairs = (hi - lo) * p.M;
    // every lane takes the same number of turns: the shuffles below need both halves of the warp
    for (int first = (threadIdx.x >> 5) * 2; first < pairs; first += WARPS * 2) {
        const int i = first + ((threadIdx.x >> 4) & 1);
        const int lc = i / p.M, m = i - lc * p.M, k = (lo + lc) * CHUNK + l * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (i < pairs && k < p.K)
            v = *reinterpret_cast<const uint4 *>(static_cast<const XT *>(p.x) + (int64_t)m * p.K + k);
        if constexpr (sizeof(XT) == 2 && !std::is_same<XT, __half>::value) {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                    __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
            top = max(top >> 16, top & 0xFFFFu);
#pragma unroll
            for (int o = 8; o > 0; o /= 2) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            const int e = top ? (int)(top >> 7) : 142;              // biased exponent; a chunk of zeros keeps scale 1
            // within 2^-60 .. 2^60 the factors of the sums stay away from fp32's ends
            bool fine = e >= 82 && e <= 202;
            const float up = __uint_as_float((uint32_t)(142 - e + 127) << 23);
            uint32_t h[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 f = pair_of((const XT *)nullptr, w[q]);
                const __half2 r = __floats2half2_rn(f.x * up, f.y * up);
                const float2 back = __half22float2(r);
                fine = fine && back.x == f.x * up && back.y == f.y * up;
                h[q] = *reinterpret_cast<const uint32_t *>(&r);
            }
            v = make_uint4(h[0], h[1], h[2], h[3]);
            const uint32_t all = __ballot_sync(0xFFFFFFFFu, fine) >> (threadIdx.x & 16) & 0xFFFFu;
            if (l == 0 && i < pairs)
                scale[lc * rows_x + m] = all == 0xFFFFu ? __uint_as_float((uint32_t)(e - 142 + 127) << 23) : -1.f;
        }
        if (i < pairs) xf[((lc * 4 + j) * p.M + m) * 4 + t] = v;
    }
}

template <typename XT, int MODE, int NT>
__global__ void __launch_bounds__(WARPS * 32, 2) matvec_kernel(MatvecParams p) {
    constexpr bool SCALED_X = !std::is_same<XT, __half>::value;
    constexpr int ROWS_X = NT * 8;
    extern __shared__ uint4 smem[];
    uint4 *xf = smem;
    float *xscale = reinterpret_cast<float *>(xf + (size_t)p.chunk_room * p.M * 16);
    float *parts = xscale + (SCALED_X ? p.chunk_room * ROWS_X : 0);     // [2][WARPS][NT][16][8]
    constexpr int PART = NT * 16 * 8;

    uint32_t cluster = 1, rank = 0, cluster_id = blockIdx.x, clusters = gridDim.x;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cluster));
    rank = cluster_ctarank();
    cluster_id = blockIdx.x / cluster;
    clusters = gridDim.x / cluster;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int S = p.slices, R = WARPS / S, tl = warp / S, sl = warp - tl * S;
    const int chunks = (p.K + CHUNK - 1) / CHUNK, T = (int)cluster * S;
    const int lo = chunks * (int)(rank * S) / T, hi = chunks * (int)(rank * S + S) / T;
    const int c0 = chunks * (int)(rank * S + sl) / T, c1 = chunks * (int)(rank * S + sl + 1) / T;
    const int tiles = (p.N + 15) / 16, groups = (tiles + R - 1) / R;
    const int blocks = p.K / 32;                        // 32-k blocks of a column

    // weights in flight: the slots hold chunks c .. c + AHEAD - 1 of a tile
    uint4 q[AHEAD][2];
    uint32_t code[AHEAD][2];
    auto fetch = [&](int j, int grp, int ch) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int n = (grp * R + tl) * 16 + g + 8 * r;
            q[j][r] = make_uint4(0, 0, 0, 0);
            code[j][r] = 0;
            if (ch < c1 && n < p.N && ch * 4 + t < blocks) {
                const int64_t block = (int64_t)n * blocks + ch * 4 + t;
                q[j][r] = load_weights(p.b + block * 16);
                if (MODE == GEMM_SCALE_UE8M0_32) code[j][r] = __ldg(p.sfb + block);
                else code[j][r] = __ldg(reinterpret_cast<const uint16_t *>(p.sfb) + block);
            }
        }
    };
    int grp = (int)cluster_id;
    if (grp < groups) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) fetch(j, grp, c0 + j);
    }
    if (SCALED_X)
        for (int i = threadIdx.x; i < (hi - lo) * ROWS_X; i += WARPS * 32) xscale[i] = 0.f;
    __syncthreads();
    stage_x<XT>(p, lo, hi, ROWS_X, xf, xscale);
    __syncthreads();

    for (int turn = 0; grp < groups; grp += clusters, turn ^= 1) {
        float total[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) total[nt][i] = 0.f;

        for (int base = c0; base < c1; base += AHEAD) {
            const bool last = base + AHEAD >= c1;
            const int next_grp = last ? grp + (int)clusters : grp, next = last ? c0 : base + AHEAD;
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const int ch = base + j, lc = ch - lo;
                if (ch < c1) {
                    float acc[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
                    float2 xs[NT];
                    bool fine = true;
                    if (SCALED_X) {
                        float worst = 1.f;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            xs[nt] = *reinterpret_cast<const float2 *>(xscale + lc * ROWS_X + nt * 8 + 2 * t);
                            worst = fminf(worst, fminf(xs[nt].x, xs[nt].y));
                        }
                        fine = worst >= 0.f;
                    }
                    uint32_t mul[2][2];                       // scales of the two columns' halves of 16 k
                    float row_scale[2];
                    if (MODE == GEMM_SCALE_UE8M0_32) {
                        const uint32_t both = code[j][0] | code[j][1] << 16;
                        uint32_t top = __vmaxu2(both, __shfl_xor_sync(0xFFFFFFFFu, both, 1));
                        top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const uint32_t ref = top >> (16 * r) & 0xFFFFu, down = ref - code[j][r];
                            // (columns past N and blocks past K have weights 0 and code 0)
                            const bool zero = ((q[j][r].x | q[j][r].y | q[j][r].z | q[j][r].w) & 0x77777777u) == 0 &&
                                              code[j][r] != 255u;
                            fine = fine && (zero || (down <= 14u && ref >= 64u && ref <= 190u));
                            mul[r][0] = mul[r][1] = (15u - min(down, 14u)) * 0x04000400u;
                            row_scale[r] = __uint_as_float(ref << 23);
                        }
                    } else {
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const uint32_t s = ue4m3x2(code[j][r]);
                            mul[r][0] = __byte_perm(s, s, 0x1010);
                            mul[r][1] = __byte_perm(s, s, 0x3232);
                        }
                    }
                    if (__all_sync(0xFFFFFFFFu, fine)) {
                        const uint32_t w[2][4] = {{q[j][0].x, q[j][0].y, q[j][0].z, q[j][0].w},
                                                  {q[j][1].x, q[j][1].y, q[j][1].z, q[j][1].w}};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t a[2][4];
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                e2m1x8(w[r][i], a[r]);
#pragma unroll
                                for (int e = 0; e < 4; ++e) a[r][e] = mul2(a[r][e], mul[r][i / 2]);
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                uint4 x = make_uint4(0, 0, 0, 0);
                                if (nt * 8 + g < p.M) x = xf[((lc * 4 + i) * p.M + nt * 8 + g) * 4 + t];
                                mma_16816(acc[nt], a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y);
                                mma_16816(acc[nt], a[0][2], a[1][2], a[0][3], a[1][3], x.z, x.w);
                            }
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float f = SCALED_X ? (i & 1 ? xs[nt].y : xs[nt].x) : 1.f;
                                if (MODE == GEMM_SCALE_UE8M0_32) f *= row_scale[i / 2];
                                total[nt][i] = fmaf(acc[nt][i], f, total[nt][i]);
                            }
                    } else {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const float4 add = products_fp32<XT, MODE>(p.x, p.K, p.M, nt * 8, ch * CHUNK + t * 32, q[j][0],
                                                                       q[j][1], code[j][0], code[j][1]);
                            total[nt][0] += add.x;
                            total[nt][1] += add.y;
                            total[nt][2] += add.z;
                            total[nt][3] += add.w;
                        }
                    }
                }
                if (next_grp < groups) fetch(j, next_grp, next + j);
            }
        }

        // join the slices of K: the CTA's, and the cluster's, always in the same order.  The two buffers
        // take turns, so the barrier of the next tile also says that this one's sums have been read.
        float *mine = parts + (turn * WARPS + warp) * PART;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            *reinterpret_cast<float2 *>(mine + (nt * 16 + g) * 8 + 2 * t) = make_float2(total[nt][0], total[nt][1]);
            *reinterpret_cast<float2 *>(mine + (nt * 16 + g + 8) * 8 + 2 * t) = make_float2(total[nt][2], total[nt][3]);
        }
        if (cluster == 1) __syncthreads();
        else {
            __syncwarp();
            cluster_sync();
        }
        const int outputs = R * 16 * p.M;
        for (int i = rank * WARPS * 32 + threadIdx.x; i < outputs; i += (int)cluster * WARPS * 32) {
            const int row = i & 15, m = (i >> 4) % p.M, tile = (i >> 4) / p.M;
            const int n = (grp * R + tile) * 16 + row;
            if (n >= p.N) continue;
            const int at = (turn * WARPS + tile * S) * PART + ((m >> 3) * 16 + row) * 8 + (m & 7);
            float v = 0.f;
            if (cluster == 1) {
                for (int s = 0; s < S; ++s) v += parts[at + s * PART];
            } else {
                for (uint32_t r = 0; r < cluster; ++r) {
                    const uint32_t from = mapa_shared(smem_addr(parts + at), r);
                    for (int s = 0; s < S; ++s) v += load_cluster(from + s * PART * 4);
                }
            }
            const int64_t o = (int64_t)m * p.N + n;
            if (p.c) v += p.c[o];
            if (p.out_bf16) static_cast<__nv_bfloat16 *>(p.d)[o] = __float2bfloat16_rn(v);
            else static_cast<float *>(p.d)[o] = v;
        }
    }
    __syncwarp();
    if (cluster != 1) cluster_sync();        // no CTA's shared memory goes while another may read it
}

// How the product is cut (see the head of this file)
struct MatvecShape {
    int slices, cluster, chunk_room, smem, grid;
};
MatvecShape matvec_shape(int M, int N, int K, bool scaled_x, int sms) {
    constexpr int X_ROOM = 88 * 1024;                    // activations in shared memory with two CTAs per SM
    const int nt = M > 8 ? 2 : 1, chunks = (K + CHUNK - 1) / CHUNK, tiles = (N + 15) / 16;
    const int per_chunk = M * CHUNK * 2 + (scaled_x ? nt * 8 * 4 : 0);
    const int warps = sms * 2 * WARPS;
    const int most = M <= 4 ? 8 : M <= 8 ? 4 : 2;        // slices: each needs the activations in its own CTA
    MatvecShape s;
    s.cluster = 1;
    while (s.cluster < 8 && s.cluster * 2 <= chunks && (chunks + s.cluster - 1) / s.cluster * per_chunk > X_ROOM) s.cluster *= 2;
    s.slices = 1;
    while (s.slices < most && s.slices * 2 * s.cluster <= chunks && (int64_t)tiles * s.slices * s.cluster < warps) s.slices *= 2;
    while (s.cluster < 8 && s.slices * s.cluster * 4 <= chunks && (int64_t)tiles * s.slices * s.cluster < warps) s.cluster *= 2;
    // a CTA's chunks: slices [rank S, rank S + S) of S c equal ones
    s.chunk_room = (chunks + s.cluster - 1) / s.cluster + 1;
    s.smem = s.chunk_room * per_chunk + 2 * WARPS * nt * 16 * 8 * 4;
    const int groups = (tiles + WARPS / s.slices - 1) / (WARPS / s.slices);
    const int resident = sms * (s.smem <= 112 * 1024 ? 2 : 1) / s.cluster;
    s.grid = (groups < resident ? groups : resident) * s.cluster;
    return s;
}

template <typename XT, int MODE, int NT>
cudaError_t launch(const MatvecShape &s, const MatvecParams &p, cudaStream_t stream) {
    static std::mutex mu;
    static bool ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev & 63]) {
            e = cudaFuncSetAttribute(matvec_kernel<XT, MODE, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
            if (e != cudaSuccess) return e;
            ready[dev & 63] = true;
        }
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)s.grid);
    cfg.blockDim = dim3(WARPS * 32);
    cfg.dynamicSmemBytes = (size_t)s.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)s.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, matvec_kernel<XT, MODE, NT>, p);
}
template <typename XT, int MODE>
cudaError_t launch(const MatvecShape &s, const MatvecParams &p, cudaStream_t stream) {
    return p.M > 8 ? launch<XT, MODE, 2>(s, p, stream) : launch<XT, MODE, 1>(s, p, stream);
}
template <typename XT>
cudaError_t launch(int mode, const MatvecShape &s, const MatvecParams &p, cudaStream_t stream) {
    return mode == GEMM_SCALE_UE8M0_32 ? launch<XT, GEMM_SCALE_UE8M0_32>(s, p, stream)
                                       : launch<XT, GEMM_SCALE_UE4M3_16>(s, p, stream);
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
    const MatvecShape s = matvec_shape((int)M, (int)N, (int)K, x == GEMM_BF16, sms);
    const MatvecParams p{X, static_cast<const uint8_t *>(B), SFB, C, D, (int)M, (int)N, (int)K, d == GEMM_BF16, s.slices, s.chunk_room};
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = x == GEMM_F16 ? launch<__half>(block_scaled, s, p, stream)
                                        : launch<__nv_bfloat16>(block_scaled, s, p, stream);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

// The gated product for 1 to 16 rows (gemm_gated_matvec_run in include/gb300gemm.h): one token, or a few, through
// the weights of a gated plan.
//
//   g = x·Wgᵀ, u = x·Wuᵀ, a = g / (1 + exp(-g)) * u
//
// Bound by the weights' bytes, which pass once from memory to registers.  The product runs on mma.sync m16n8k16: its 16
// rows are 8 rows of Wg and the same 8 of Wu, its 8 columns tokens, so that an element's g and u end up in one thread and
// the tokens that are not there cost nothing but idle lanes of an otherwise idle unit.  The order of k within an MMA is
// free as long as both operands agree on it: a lane takes consecutive bytes of a weight row, whatever k they are, and the
// same k of its token.
//
// A CTA takes 8 G columns of A; its eight warps, and the CTAs of a cluster where columns are few, share K out in chunks of
// 128 bytes of a weight row and join their sums through shared memory, always in the same order.  Each warp has a ring in
// shared memory of its own, filled with asynchronous copies some chunks ahead: the weights' 128-byte lines, the
// activations' and the scales; it runs on from one tile of columns to the next, so that memory does not wait for the sums.
#include <algorithm>
#include <atomic>
#include <mutex>
#include <type_traits>

#include "gemm_rows.cuh"

namespace gb300 {
namespace {

using namespace rows;

constexpr int WARPS = 8;
constexpr int MAX_ROWS = 16;
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_DEVICES = 64;                            // device_sms knows no more

struct FewParams {
    const void *x;
    const uint8_t *w, *sfw;
    void *a;
    int M, F, K;
    int chunks;              // of K
    int tiles;               // of 8 G columns
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

// the same from nothing: d = a b
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 16 or 4 bytes to shared memory; zeros where not `on` (the address is then any valid one)
__device__ __forceinline__ void copy16(uint32_t to, const void *from, bool on) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(on ? 16 : 0) : "memory");
}
// the same by way of L1
__device__ __forceinline__ void copy16_l1(uint32_t to, const void *from, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }
__device__ __forceinline__ uint4 shared16(uint32_t at) {
    uint4 q;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(at) : "memory");
    return q;
}
__device__ __forceinline__ uint2 shared8(uint32_t at) {
    uint2 q;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(q.x), "=r"(q.y) : "r"(at) : "memory");
    return q;
}
__device__ __forceinline__ uint32_t shared4(uint32_t at) {
    uint32_t q;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(q) : "r"(at) : "memory");
    return q;
}

__device__ __forceinline__ uint4 load_row(const void *p, bool on) {
    return on ? *static_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
struct Place {
    int lane, warp, r, t;    // r: a weight row of eight, and a token of eight; t: a lane of the four that share a row
    uint32_t rank, ranks;    // in the cluster
    __device__ __forceinline__ Place() {
        lane = threadIdx.x & 31;
        warp = threadIdx.x / 32;
        r = lane / 4;
        t = lane % 4;
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    }
};

__device__ __forceinline__ float2 load_cluster(const float *here, uint32_t rank) {     // the same place in another CTA
    uint32_t from;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"((uint32_t)__cvta_generic_to_shared(here)), "r"(rank));
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(from) : "memory");
    return v;
}
// a of column f and token m, where there are such
template <typename XT>
__device__ __forceinline__ void put(void *a, int M, int F, int f, int m, float g, float u) {
    if (f >= F || m >= M) return;
    float s1, s0;
    sigmoid(g, s1, s0);
    const float v = g * s1 * u;
    if constexpr (std::is_same<XT, __nv_bfloat16>::value) static_cast<__nv_bfloat16 *>(a)[(int64_t)m * F + f] = __float2bfloat16_rn(v);
    else static_cast<__half *>(a)[(int64_t)m * F + f] = __float2half_rn(v);
}

// The warps' sums acc[G][NG][g of two tokens, u of them] of the columns from f0 on joined over the CTA and the cluster, and
// the columns of A
template <typename XT, int NG, int G>
__device__ __forceinline__ void finish(const FewParams &p, const Place &at, int f0, const float (&acc)[G][NG][4]) {
    constexpr int OUTPUTS = 64 * G * NG, TURNS = (OUTPUTS + WARPS * 32 - 1) / (WARPS * 32);
    __shared__ float part[WARPS][G][NG][4][32];
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
        for (int j = 0; j < NG; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[at.warp][i][j][e][at.lane] = acc[i][j][e];
    __syncthreads();
    // output o: column f0 + 8 i + r of token 8 j + 2 t + e; elements e of a thread's sums are g, e + 2 are u
    float sums[TURNS][2];
#pragma unroll
    for (int n = 0; n < TURNS; ++n) {
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
    if (at.ranks > 1) {
        __syncthreads();
#pragma unroll
        for (int n = 0; n < TURNS; ++n) {
            const int o = n * WARPS * 32 + threadIdx.x;
            if (o >= OUTPUTS) break;
            own[2 * o] = sums[n][0];
            own[2 * o + 1] = sums[n][1];
        }
        cluster_barrier();
    }
#pragma unroll
    for (int n = 0; n < TURNS; ++n) {
        const int o = n * WARPS * 32 + threadIdx.x;
        if (o >= OUTPUTS) break;
        if (at.ranks > 1) {                               // each CTA of the cluster finishes a share of the outputs
            if ((uint32_t)(o / 32) % at.ranks != at.rank) continue;
            sums[n][0] = sums[n][1] = 0.f;
            for (uint32_t q = 0; q < at.ranks; ++q) {
                const float2 v = load_cluster(own + 2 * o, q);
                sums[n][0] += v.x;
                sums[n][1] += v.y;
            }
        }
        const int i = o / (64 * NG), j = o / 64 % NG, e = o / 32 % 2, l = o % 32;
        put<XT>(p.a, p.M, p.F, f0 + 8 * i + l / 4, 8 * j + 2 * (l % 4) + e, sums[n][0], sums[n][1]);
    }
    if (at.ranks > 1) cluster_barrier();                  // no CTA leaves, or begins anew, while another may still read its sums
    else __syncthreads();
}

// ------------------------------------------------------------------------------------------- 16-bit weights

// A piece of 16 bytes in a line of 128, eight of them.  Its place depends on the line's row so that a warp's reads meet every
// bank once: 16-byte reads take the same half of two rows at a time, 8-byte reads (e4m3) the same quarter of four.
__device__ __forceinline__ int half(int row, int piece) { return piece ^ ((row & 1) << 2); }
__device__ __forceinline__ int quarter(int row, int piece) { return piece ^ ((row & 3) << 1); }

// A warp's ring: DEPTH stages, each 64 of k of 16 G weight rows (8 of g, 8 of u, the next 8 ...) and of 8 NG tokens
template <int NG, int G, int DEPTH>
struct Ring {
    static constexpr int OFF_X = 16 * G * 128;
    static constexpr int STAGE = OFF_X + 8 * NG * 128;
    static constexpr int WARP_BYTES = DEPTH * STAGE;
    static constexpr int BYTES = WARPS * WARP_BYTES;
    static constexpr int PART = 4 * WARPS * G * NG * 128;                           // finish()'s
    static constexpr int CTAS_PER_SM = BYTES + PART <= 112 * 1024 ? 2 : 1;
    static_assert(BYTES + PART <= 226 * 1024, "shared memory");
};

// A lane's 16 bytes are 8 k of its row, the four lanes of a row have 32 k side by side.  Bound by memory: 1 x 8192 x 4096 bf16
// 20.8 to 21.2 us, 6350 to 6450 GB/s (93 to 95 % of a copy's rate), 8 rows 21.3, 16 rows 23.2.  (Loads to registers, as many as fit, leave memory
// waiting while a warp computes: 23.3, 23.9 and 28.6.)  Eight columns per CTA and four stages for up to eight rows, sixteen
// columns for more, whose lines are half of a stage: 16 columns and one row 21.1, 8 columns and 16 rows 27.8.
template <typename XT, int NG, int G, int DEPTH>
__global__ void __launch_bounds__(WARPS * 32) few_kernel(const __grid_constant__ FewParams p) {
    using R = Ring<NG, G, DEPTH>;
    constexpr bool BF16 = std::is_same<XT, __nv_bfloat16>::value;
    extern __shared__ __align__(128) uint8_t rings[];
    const Place at;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(rings) + at.warp * R::WARP_BYTES;
    const int64_t row_bytes = (int64_t)p.K * 2, half_bytes = p.F * row_bytes;
    wait_for_previous();
    let_next_launch();

    // Rows of X that begin inside a sector of 32 bytes come by way of L1, where a sector that two copies share is read once:
    // 8 x 8000 x 1000 8.9 us, 14.0 past it, 8 x 8192 x 4104 26.8 and 34.0; rows of whole sectors 8 x 8192 x 8192 44.2, 40.1 past it.
    const bool whole_sectors = p.K % 16 == 0;
    // fills stage s with chunk c of the tile whose columns begin at f0: lane l has piece l % 8 of every fourth line from l / 8 on
    const int piece = at.lane % 8, line0 = at.lane / 8;
    auto fill = [&](int s, int c, int f0) {
        const uint32_t to = ring + s * R::STAGE;
        const int64_t byte = (int64_t)c * 128 + piece * 16;
        const bool in = byte < row_bytes;
#pragma unroll
        for (int i = 0; i < 4 * G; ++i) {
            const int line = line0 + 4 * i, f = f0 + 8 * (i / 4) + line0 + 4 * (i % 2);        // g: i % 4 < 2, then u
            const bool on = in && f < p.F;
            const uint8_t *from = p.w + (on ? f * row_bytes + (i % 4 < 2 ? 0 : half_bytes) + byte : 0);
            copy16(to + line * 128 + 16 * half(line, piece), from, on);
        }
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i) {
            const int m = line0 + 4 * i;
            if (m >= p.M) break;                          // zero from the start
            const uint32_t x_to = to + R::OFF_X + m * 128 + 16 * half(m, piece);
            const uint8_t *from = static_cast<const uint8_t *>(p.x) + (in ? m * row_bytes + byte : 0);
            if (whole_sectors) copy16(x_to, from, in);
            else copy16_l1(x_to, from, in);
        }
    };
    // tokens that are not there are zero in every stage
    for (int i = at.lane; i < DEPTH * 8 * NG * 8; i += 32) {
        const int s = i / (8 * NG * 8), o = i % (8 * NG * 8);
        if (o / 8 >= p.M)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(ring + s * R::STAGE + R::OFF_X + o * 16), "r"(0) : "memory");
    }

    // This warp's chunks: every (WARPS * ranks)-th of each of the CTA's (or cluster's) tiles, which are every turn-th of all.
    // The ring runs on from tile to tile: the next one's chunks are under way while this one's sums are joined.
    const int first = at.warp + WARPS * (int)at.rank, step = WARPS * (int)at.ranks;
    const int tile0 = (int)(blockIdx.x / at.ranks), turn = (int)(gridDim.x / at.ranks);
    int fill_tile = tile0, fill_chunk = first;
    auto fill_next = [&](int s) {
        if (fill_chunk >= p.chunks) {                     // the tile has no more: on to the next
            fill_chunk = first;
            fill_tile += turn;
        }
        if (fill_tile < p.tiles && fill_chunk < p.chunks) fill(s, fill_chunk, fill_tile * 8 * G);
        fill_chunk += step;
        commit_copies();
    };
#pragma unroll
    for (int n = 0; n < DEPTH - 1; ++n) fill_next(n);
    int s = 0, ahead = DEPTH - 1;                         // the stage at hand, and the one filled next
    for (int tile = tile0; tile < p.tiles; tile += turn) {
        float acc[G][NG][4] = {};
        for (int c = first; c < p.chunks; c += step) {
            wait_copies<DEPTH - 2>();
            __syncwarp();                                 // all lanes' copies are here, and all have read the stage before
            fill_next(ahead);
            const uint32_t from = ring + s * R::STAGE;
            if (++s == DEPTH) s = 0;
            if (++ahead == DEPTH) ahead = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int q = 16 * half(at.r, 4 * h + at.t);
                uint4 x[NG];
#pragma unroll
                for (int j = 0; j < NG; ++j) x[j] = shared16(from + R::OFF_X + (8 * j + at.r) * 128 + q);
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    const uint32_t line = from + (16 * i + at.r) * 128 + q;
                    const uint4 g = shared16(line), u = shared16(line + 8 * 128);
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        mma<BF16>(acc[i][j], g.x, u.x, g.y, u.y, x[j].x, x[j].y);
                        mma<BF16>(acc[i][j], g.z, u.z, g.w, u.w, x[j].z, x[j].w);
                    }
                }
            }
        }
        finish<XT>(p, at, tile * 8 * G, acc);
    }
    wait_copies<0>();
}

template <typename Kernel>
cudaError_t allow_shared(Kernel kernel, std::atomic<bool> *ready, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || ready[dev].load(std::memory_order_acquire)) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);      // (twice does no harm)
    if (e == cudaSuccess) ready[dev].store(true, std::memory_order_release);
    return e;
}

// A cluster's CTAs share K where there are fewer CTAs than the GPU runs and chunks for all their warps
template <typename XT, int NG, int G, int DEPTH>
cudaError_t few_launch(FewParams p, int sms, cudaStream_t stream) {
    using R = Ring<NG, G, DEPTH>;
    const auto kernel = few_kernel<XT, NG, G, DEPTH>;
    static std::atomic<bool> ready[MAX_DEVICES];
    const cudaError_t e = allow_shared(kernel, ready, R::BYTES);
    if (e != cudaSuccess) return e;
    const int slots = R::CTAS_PER_SM * sms;
    p.chunks = (p.K + 63) / 64;
    p.tiles = (p.F + 8 * G - 1) / (8 * G);
    int cluster = 1;
    while (cluster < MAX_CLUSTER && p.tiles * cluster * 2 <= slots && p.chunks > WARPS * cluster) cluster *= 2;
    // as many CTAs as run at once, or fewer that all have as many tiles
    const int rounds = (p.tiles + slots - 1) / slots, ctas = (p.tiles + rounds - 1) / rounds;
    const Launch l(ctas * cluster, WARPS * 32, R::BYTES, cluster, stream);
    return cudaLaunchKernelEx(&l.config, kernel, p);
}

// ------------------------------------------------------------------------------------------- e4m3 weights

// four e4m3 codes as four fp16 values, exactly
__device__ __forceinline__ void widen(uint32_t codes, uint32_t &low, uint32_t &high) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(low), "=r"(high)
        : "r"(codes));
}
// four UE8M0 codes as fp32 values, 255 as a NaN
__device__ __forceinline__ void scales(uint32_t codes, float (&v)[4]) {
    uint32_t low, high;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.bf16x2.ue8m0x2 %0, a;\n\tcvt.rn.bf16x2.ue8m0x2 %1, b;\n\t}"
        : "=r"(low), "=r"(high)
        : "r"(codes));
    v[0] = __uint_as_float(low << 16);
    v[1] = __uint_as_float(low & 0xFFFF0000u);
    v[2] = __uint_as_float(high << 16);
    v[3] = __uint_as_float(high & 0xFFFF0000u);
}
// two bf16 values times a power of two, as two fp16 values
__device__ __forceinline__ uint32_t narrow(uint32_t v, uint32_t factor) {
    uint32_t s, h;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(s) : "r"(v), "r"(factor));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(__uint_as_float(s & 0xFFFF0000u)), "f"(__uint_as_float(s << 16)));
    return h;
}
__device__ __forceinline__ uint32_t largest2(uint32_t a, uint32_t b) {             // of bf16 magnitudes, NaN left out
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&a), __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&b)));
    return *reinterpret_cast<const uint32_t *>(&m);
}

// The weights are a power of two per 32 of k times codes, which become fp16, which holds them all, by one conversion for two.
// A lane's 8 bytes are 8 codes, the four lanes of a row have one scale's block side by side, so that two MMAs sum a block, whose
// sum takes the scale.
// fp16 activations meet the codes as they are.  bf16 ones are brought to fp16 by a power of two for each token's 128 of k,
// which puts the largest of them at 2^14 to 2^15: those down to 2^-31 of it are exact, smaller ones off by 2^-39 of it at
// most.  That is done once for all columns of a CTA: its sixteen warps have 8 columns each of up to 128, or share
// K between them; the activations lie in shared memory, a phase of K's chunks ahead.  1 x 8192 x 8192 24.4 to 25 us (5600 GB/s), 8 rows
// 28, 16 rows 35.2: the weights' way through shared memory and the chains of MMAs behind it (16 rows with no weights loaded take
// 27, without the products with scales 32.6, without conversions or reads of activations no less).  Tried, for 1, 8 and 16 rows:
// each warp a part of K, its activations converted by itself 28.4, 29.1 and 46; weights made bf16 by their bits and a product, from
// registers 35, 36 and 43; 24 warps with 80 registers 25.8, 30.2 and 41.8; weights by tensor boxes, one per chunk 25.9, 29 and
// 37.9; for 16 rows a stage more 38, a stage less 37.7.
constexpr int CHUNK = 128;                                 // of k: a line of a weight row
constexpr int STAGE = 16 * 128 + 16 * 4;                   // 8 rows of g, 8 of u, and their scales
constexpr int WIDE_WARPS = 16;
// bf16 activations: a chunk's sum of up to 2^15 |w| for each of 128 k takes the weights' scales before the token's power of two, so
// 2^-22 goes with the scales, and no weight that fp32 holds takes it past fp32.  The power of two has 2^14 of that back, the
// joined sums 2^8.  (Far below, a block's sum is off by up to 2^-142 of the largest activation.)
constexpr float SCALE_DOWN = 0x1p-22f, SUMS_UP = 0x1p8f;
template <int NG>
struct Wide {
    static constexpr int DEPTH = NG == 1 ? 4 : 3;                                   // stages of a warp's ring
    static constexpr int RINGS = WIDE_WARPS * DEPTH * STAGE;
    // activations held at once, twice: (chunk, token)s of 128 k, and their powers of two
    // (what the first sums wait for: 4 x 2048 x 2048 3.8 us with two pieces, 4.2 with four; 16 x 8192 x 8192 36.9 and 35.3)
    static constexpr int PIECES = NG == 1 ? 2 : 4;                                  // of sixteen lanes
    static constexpr int HELD = PIECES * WIDE_WARPS * 2;
    static constexpr int OFF_FX = HELD * 256;
    static constexpr int X_BYTES = OFF_FX + (HELD + 16) * 4;
    static constexpr int BYTES = RINGS + 2 * X_BYTES;
    static_assert(BYTES + WIDE_WARPS * NG * 512 <= 227 * 1024, "shared memory");
};

struct WideParams {
    const void *x;
    const uint8_t *w, *sfw;
    void *a;
    int M, F, K;
    int chunks;              // of K
    int tiles;               // of 8 * groups columns
    int groups;              // of 8 columns side by side in a CTA
    int shares;              // warps that share a group's K; those behind the last group's have none
};

template <typename XT, int NG>
__global__ void __launch_bounds__(WIDE_WARPS * 32) few_scaled_kernel(const __grid_constant__ WideParams p) {
    using W = Wide<NG>;
    constexpr bool BF16 = std::is_same<XT, __nv_bfloat16>::value;
    constexpr int TURNS = 2 * NG, DEPTH = W::DEPTH;
    extern __shared__ __align__(128) uint8_t shared[];
    __shared__ float part[WIDE_WARPS][NG][4][32];
    const Place at;
    // shared memory: the warps' rings, then two buffers of activations, lines [chunk][token][2], and their powers of two
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(shared), ring = base + at.warp * DEPTH * STAGE;
    const int blocks = (p.K + BLOCK - 1) / BLOCK;
    const bool whole_scales = blocks % 4 == 0 && (reinterpret_cast<uintptr_t>(p.sfw) & 3) == 0;
    const int shares = p.shares, group = at.warp % p.groups, share = at.warp / p.groups < shares ? at.warp / p.groups : p.chunks;
    // the CTA's slice: chunks [c0, c1), every shares-th of them this warp's
    const int c0 = (int)((int64_t)p.chunks * at.rank / at.ranks), c1 = (int)((int64_t)p.chunks * (at.rank + 1) / at.ranks);
    const int rows = min(p.M, 8 * NG), phase_chunks = W::HELD / rows, phases = (c1 - c0 + phase_chunks - 1) / phase_chunks;
    const uint32_t inverse = (65535u + rows) / rows;      // n / rows = n * inverse >> 16 for n < HELD
    const int tile0 = (int)(blockIdx.x / at.ranks), turn = (int)(gridDim.x / at.ranks);
    wait_for_previous();
    let_next_launch();

    // Fills stage s with chunk c of the columns from f0 on: lane l has piece l % 8 of rows l / 8 and l / 8 + 4 of g and of u.
    // Away from the matrix's edges a lane's four addresses are one and three constants.
    const int piece = at.lane % 8, line0 = at.lane / 8;
    const uint32_t piece_to = ring + line0 * 128 + 16 * quarter(line0, piece), scale_to = ring + 16 * 128 + 4 * at.lane;
    const int64_t four = (int64_t)4 * p.K, half_bytes = (int64_t)p.F * p.K;
    auto fill = [&](int s, int c, int f0) {
        const uint32_t to = piece_to + s * STAGE, sf_to = scale_to + s * STAGE;
        const uint8_t *g = p.w + (int64_t)(f0 + line0) * p.K + (c * CHUNK + piece * 16);
        const int f = f0 + at.lane % 8;
        const uint8_t *sf = p.sfw + (int64_t)(f + (at.lane < 8 ? 0 : p.F)) * blocks + 4 * c;
        if (whole_scales && f0 + 8 <= p.F && (c + 1) * CHUNK <= p.K) {
            copy16(to, g, true);
            copy16(to + 512, g + four, true);
            copy16(to + 1024, g + half_bytes, true);
            copy16(to + 1536, g + half_bytes + four, true);
            if (at.lane < 16) copy4(sf_to, sf);
            return;
        }
        const bool in = c * CHUNK + piece * 16 < p.K, on0 = in && f0 + line0 < p.F, on4 = in && f0 + line0 + 4 < p.F;
        copy16(to, on0 ? g : p.w, on0);
        copy16(to + 512, on4 ? g + four : p.w, on4);
        copy16(to + 1024, on0 ? g + half_bytes : p.w, on0);
        copy16(to + 1536, on4 ? g + half_bytes + four : p.w, on4);
        if (at.lane < 16) {
            uint32_t w = 0x7F7F7F7Fu;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (f < p.F && 4 * c + b < blocks) w = (w & ~(0xFFu << 8 * b)) | (uint32_t)sf[b] << 8 * b;
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(sf_to), "r"(w) : "memory");
        }
    };
    int fill_tile = tile0, fill_chunk = c0 + share;
    auto fill_next = [&](int s) {
        if (fill_chunk >= c1) {                           // the tile has no more: on to the next
            fill_chunk = c0 + share;
            fill_tile += turn;
        }
        if (fill_tile < p.tiles && fill_chunk < c1) fill(s, fill_chunk, (fill_tile * p.groups + group) * 8);
        fill_chunk += shares;
        commit_copies();
    };
#pragma unroll
    for (int n = 0; n < DEPTH - 1; ++n) fill_next(n);

    // A phase's activations: sixteen lanes have a token's 128 of k.  They are loaded while the phase before is summed, and
    // put into the other buffer behind it.  Tokens that are not there are read as the last one: no sum of another token
    // knows of them.
    const int l16 = at.lane % 16, half_warp = at.warp * 2 + at.lane / 16;
    uint4 raw[W::PIECES];
    auto load_x = [&](int phase) {
#pragma unroll
        for (int i = 0; i < W::PIECES; ++i) {
            const int n = half_warp + i * WIDE_WARPS * 2, o = (int)(n * inverse >> 16), m = n - o * rows;
            const int c = phase * phase_chunks + o, k = (c0 + c) * CHUNK + 8 * l16;
            raw[i] = load_row(static_cast<const XT *>(p.x) + (int64_t)m * p.K + k, c0 + c < c1 && k < p.K);
        }
    };
    auto store_x = [&](int buffer) {
        const uint32_t to = base + W::RINGS + buffer * W::X_BYTES;
#pragma unroll
        for (int i = 0; i < W::PIECES; ++i) {
            const int n = half_warp + i * WIDE_WARPS * 2, m = n - (int)(n * inverse >> 16) * rows;
            uint4 q = raw[i];
            if constexpr (BF16) {
                uint32_t top = largest2(largest2(largest2(largest2(0, q.x), q.y), q.z), q.w);
                top = max(top >> 16, top & 0xFFFFu);      // magnitudes order as their bits do
#pragma unroll
                for (int o = 1; o < 16; o *= 2) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                // exponent fields: of the factor, within 2^-114 (beside an infinity) and 2^127, and of its inverse times 2^14
                const uint32_t e = max(top >> 7, 14u), up = (268u - e) << 7, factor = up | up << 16;
                q = make_uint4(narrow(q.x, factor), narrow(q.y, factor), narrow(q.z, factor), narrow(q.w, factor));
                if (l16 == 0)
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + W::OFF_FX + 4 * n), "r"(e << 23) : "memory");
            }
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + n * 256 + 128 * (l16 / 8) + 16 * half(m, l16 % 8)),
                         "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w)
                         : "memory");
        }
    };
    load_x(0);
    store_x(0);
    __syncthreads();

    // where a lane reads in a stage and in a chunk's activations
    uint32_t wo[4], xo[NG][2];
#pragma unroll
    for (int b = 0; b < 4; ++b) wo[b] = at.r * 128 + 16 * quarter(at.r, 2 * b + at.t / 2) + 8 * (at.t % 2);
#pragma unroll
    for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int m = min(8 * j + at.r, rows - 1);
            xo[j][b] = m * 256 + 16 * half(m, 4 * b + at.t);
        }
    int s = 0, ahead = DEPTH - 1, buffer = 0;             // the stage at hand, the one filled next, the activations at hand
    for (int tile = tile0; tile < p.tiles; tile += turn) {
        float acc[NG][4] = {};
        int c = c0 + share;
        for (int phase = 0; phase < phases; ++phase) {
            const bool more = phase + 1 < phases || tile + turn < p.tiles, renew = more && phases > 1;
            if (renew) load_x(phase + 1 < phases ? phase + 1 : 0);
            const int begin = c0 + phase * phase_chunks, end = min(c1, begin + phase_chunks);
            const uint32_t xs = base + W::RINGS + buffer * W::X_BYTES;
            for (; c < end; c += shares) {
                wait_copies<DEPTH - 2>();
                __syncwarp();                             // all lanes' copies are here, and all have read the stage before
                fill_next(ahead);
                const uint32_t from = ring + s * STAGE, xc = xs + (c - begin) * rows * 256;
                if (++s == DEPTH) s = 0;
                if (++ahead == DEPTH) ahead = 0;
                float sum[NG][4] = {}, scale[2][4];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    scales(shared4(from + 16 * 128 + 32 * z + 4 * at.r), scale[z]);
                    if constexpr (BF16) {
#pragma unroll
                        for (int b = 0; b < 4; ++b) scale[z][b] *= SCALE_DOWN;
                    }
                }
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    uint4 x[NG];
#pragma unroll
                    for (int j = 0; j < NG; ++j) x[j] = shared16(xc + xo[j][b % 2] + 128 * (b / 2));
                    uint32_t h[2][4];
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const uint2 q = shared8(from + wo[b] + z * 8 * 128);
                        widen(q.x, h[z][0], h[z][1]);
                        widen(q.y, h[z][2], h[z][3]);
                    }
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        float d[4];
                        mma_first(d, h[0][0], h[1][0], h[0][1], h[1][1], x[j].x, x[j].y);
                        mma<false>(d, h[0][2], h[1][2], h[0][3], h[1][3], x[j].z, x[j].w);
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum[j][e] = fmaf(d[e], scale[e / 2][b], sum[j][e]);
                    }
                }
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    uint2 f = make_uint2(0x3F800000u, 0x3F800000u);
                    if constexpr (BF16) {
                        const uint32_t fx = xs + W::OFF_FX + ((c - begin) * rows + 8 * j + 2 * at.t) * 4;
                        f = make_uint2(shared4(fx), shared4(fx + 4));
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(sum[j][e], __uint_as_float(e % 2 ? f.y : f.x), acc[j][e]);
                }
            }
            if (renew) {
                buffer ^= 1;                              // (read last before the barrier that stands behind the phase before)
                store_x(buffer);
                __syncthreads();
            }
        }
        // Output o of the CTA: column group o / (64 NG), token group o / 64 % NG, and of those column r of token 2 t + e.  A group's
        // warps are added in order, then the cluster's CTAs.
#pragma unroll
        for (int j = 0; j < NG; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[at.warp][j][e][at.lane] = BF16 ? acc[j][e] * SUMS_UP : acc[j][e];
        __syncthreads();
        const int outputs = p.groups * 64 * NG;
        float sums[TURNS][2];
#pragma unroll
        for (int n = 0; n < TURNS; ++n) {
            const int o = n * WIDE_WARPS * 32 + threadIdx.x;
            sums[n][0] = sums[n][1] = 0.f;
            if (o >= outputs) break;
            const int w = o / (64 * NG), j = o / 64 % NG, e = o / 32 % 2, l = o % 32;
            for (int k = w; k < p.groups * shares; k += p.groups) {
                sums[n][0] += part[k][j][e][l];
                sums[n][1] += part[k][j][e + 2][l];
            }
        }
        float *own = &part[0][0][0][0];
        if (at.ranks > 1) {
            __syncthreads();
#pragma unroll
            for (int n = 0; n < TURNS; ++n) {
                const int o = n * WIDE_WARPS * 32 + threadIdx.x;
                if (o >= outputs) break;
                own[2 * o] = sums[n][0];
                own[2 * o + 1] = sums[n][1];
            }
            cluster_barrier();
        }
#pragma unroll
        for (int n = 0; n < TURNS; ++n) {
            const int o = n * WIDE_WARPS * 32 + threadIdx.x;
            if (o >= outputs) break;
            if (at.ranks > 1) {                           // each CTA of the cluster finishes a share of the outputs
                if ((uint32_t)(o / 32) % at.ranks != at.rank) continue;
                sums[n][0] = sums[n][1] = 0.f;
                for (uint32_t q = 0; q < at.ranks; ++q) {
                    const float2 v = load_cluster(own + 2 * o, q);
                    sums[n][0] += v.x;
                    sums[n][1] += v.y;
                }
            }
            const int w = o / (64 * NG), j = o / 64 % NG, e = o / 32 % 2, l = o % 32;
            put<XT>(p.a, p.M, p.F, (tile * p.groups + w) * 8 + l / 4, 8 * j + 2 * (l % 4) + e, sums[n][0], sums[n][1]);
        }
        if (at.ranks > 1) cluster_barrier();              // no CTA leaves, or begins anew, while another may still read its sums
        else __syncthreads();
    }
    wait_copies<0>();
}

// How columns and K are shared out: `groups` column groups per CTA, the warps that are left and the CTAs of a cluster sharing K.
// The estimate in microseconds, but for what every shape costs, is fitted to 2900 times of 85 sizes (M 1 to 16, F 333 to 65 536, K
// 512 to 32 768) in every shape; the shape that it takes is 1.1 % slower than the fastest on average, 21 % at most.  For
// example 16 x 8192 x 8192: 14 groups and clusters of two 35.3 us, 16 and two 36.9, 7 and one 37.1, 16 and four 46; 1 x 14336 x
// 4096: 12 or 6 groups 22.4, 13 25.3, 16 31.
struct WideShape {
    int groups, cluster, slots;                            // slots: clusters that run at once
};
constexpr int CLUSTERS = 4;                                // of 1, 2, 4 and 8 CTAs
WideShape wide_shape(int M, int F, int K, const int (&slots)[CLUSTERS]) {
    const bool few = M <= 8;
    const float cluster_us = few ? 0.16f : 0.74f, round_us = few ? 0.38f : 0.54f, cluster_round_us = few ? 1.19f : 1.49f;
    const float step_us = few ? 0.111f : 0.365f, warp_us = few ? 0.036f : 0.0437f, x_us = few ? 0.0038f : 0.0073f;
    const uint32_t columns = (uint32_t)(F + 7) / 8, chunks = (uint32_t)(K + CHUNK - 1) / CHUNK;
    WideShape best{};
    float least = 0.f;
    for (int i = 0; i < CLUSTERS && (1u << i) <= chunks; ++i) {
        const uint32_t slice = (chunks + (1u << i) - 1) >> i;
        if (slots[i] < 1) continue;
        for (uint32_t groups = 2; groups <= WIDE_WARPS; ++groups) {
            const uint32_t tiles = (columns + groups - 1) / groups, rounds = (tiles + slots[i] - 1) / slots[i];
            const uint32_t shares = WIDE_WARPS / groups, steps = (slice + shares - 1) / shares;
            const uint32_t warps = groups * std::min(shares, slice);
            const float us = (i > 0 ? cluster_us : 0.f) +
                             (float)rounds * (round_us + (i > 0 ? cluster_round_us : 0.f) + (float)steps * (step_us + warp_us * (float)warps) +
                                              x_us * (float)(slice * (uint32_t)M));
            if (best.groups == 0 || us < least) {
                least = us;
                best = WideShape{(int)groups, 1 << i, slots[i]};
            }
        }
    }
    return best;
}

template <typename XT, int NG>
cudaError_t few_scaled_launch(const FewParams &q, int sms, cudaStream_t stream) {
    const auto kernel = few_scaled_kernel<XT, NG>;
    static std::mutex mu;
    static int known[MAX_DEVICES][CLUSTERS];               // clusters that run at once; they are asked for once
    static thread_local struct {
        int dev, M, F, K;
        WideShape shape;
    } last{-1, 0, 0, 0, {}};                               // the shape is a microsecond's work
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (last.dev != dev || last.M != q.M || last.F != q.F || last.K != q.K) {
        std::lock_guard<std::mutex> lock(mu);
        int(&slots)[CLUSTERS] = known[dev];
        if (slots[0] == 0) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Wide<NG>::BYTES);
            for (int i = CLUSTERS - 1; i > 0 && e == cudaSuccess; --i) {
                const Launch l(1 << i, WIDE_WARPS * 32, Wide<NG>::BYTES, 1 << i, nullptr, false);
                e = cudaOccupancyMaxActiveClusters(&slots[i], kernel, &l.config);
            }
            if (e != cudaSuccess) return e;
            slots[0] = sms;
        }
        last = {dev, q.M, q.F, q.K, wide_shape(q.M, q.F, q.K, slots)};
    }
    const WideShape &s = last.shape;
    const int columns = (q.F + 7) / 8, tiles = (columns + s.groups - 1) / s.groups;
    const WideParams p{q.x, q.w, q.sfw, q.a, q.M, q.F, q.K, (q.K + CHUNK - 1) / CHUNK, tiles, s.groups, WIDE_WARPS / s.groups};
    const int rounds = (tiles + s.slots - 1) / s.slots, ctas = (tiles + rounds - 1) / rounds;
    const Launch l(ctas * s.cluster, WIDE_WARPS * 32, Wide<NG>::BYTES, s.cluster, stream);
    return cudaLaunchKernelEx(&l.config, kernel, p);
}

template <typename XT>
cudaError_t few(const FewParams &p, int sms, cudaStream_t stream) {
    if (p.sfw) return p.M <= 8 ? few_scaled_launch<XT, 1>(p, sms, stream) : few_scaled_launch<XT, 2>(p, sms, stream);
    return p.M <= 8 ? few_launch<XT, 1, 1, 4>(p, sms, stream) : few_launch<XT, 2, 2, 4>(p, sms, stream);
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
    const FewParams p{X, static_cast<const uint8_t *>(W), w == GEMM_E4M3 ? SFW : nullptr, A, (int)M, (int)F, (int)K, 0};
    const cudaError_t e = x == GEMM_BF16 ? few<__nv_bfloat16>(p, sms, stream) : few<__half>(p, sms, stream);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

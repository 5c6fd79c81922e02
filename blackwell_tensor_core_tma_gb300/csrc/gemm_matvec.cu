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
// A warp owns 16 columns (n) and a slice of K, which it walks in chunks of 256 through a ring of its own in
// shared memory, filled AHEAD - 1 chunks early with asynchronous copies: 128 contiguous bytes of each column and
// its scale codes.  The order of k inside an MMA is free as long as both operands agree: in 32-block i of a chunk
// lane (g, t) takes k = 32 i + 8 t .. + 7 of columns g and g + 8, one 32-bit word each, as the A operand of two
// MMAs, and the activations are laid out in shared memory in that order when the CTA starts.  Those words are what
// ldmatrix deals out of 8 x 16-byte matrices; a column's eight pieces of 16 bytes are permuted by its number, so
// that a matrix covers the 32 banks.
//
// Scales, more than four rows.  UE8M0 (per 32): the two MMAs of a block start from zero and their sum is scaled
// in fp32.  UE4M3 (per 16): the product with an e2m1 value has at most six significant bits and lies within
// 2^-10 .. 2688, so it is exact in fp16: weights are scaled before the MMA.
// Scales, up to four rows.  An MMA has eight columns of activations, so a row of X is given 8 / FORM of them and its
// k are dealt out so that each column sees one scale only: a block's halves of 16 k (UE4M3) or two blocks
// (UE8M0) to neighbouring columns, and 4 / FORM such pairs to the rest; everything else in the
// column is zero.  MMAs then run on through 4 / FORM pairs into one accumulator, whose two values per lane
// and row are scaled by the lane's own pair of codes with one packed fp32 multiply-add: nothing is scaled per
// weight, and no lane decodes a code that another one decodes too.
// Activations.  fp16 goes in as it is.  bf16 is multiplied per row and chunk by the power of two that brings
// the largest magnitude to 2^15 .. 2^16, which is exact in fp16 for elements down to 2^-29 of it.
// What these rules do not hold (bf16 activations too far apart within a chunk, outside 2^-50 .. 2^40, infinite or
// NaN; UE8M0 scales from 2^33, NaN among them) takes products_by_band for that chunk.
//
// A CTA (one per SM) is 16 warps: R tiles of 16 columns by S slices of K, and `c` CTAs of a cluster split K
// further; the partial sums are joined in a fixed order through shared memory, the cluster's through
// distributed shared memory.
//
// Measured (of 6775 GB/s, a copy's rate): 1 x 32768 x 8192 (M x N x K, UE4M3, bf16) 25.2 us, 5990 GB/s, 88%, the rest
// being the start (X's and the first weights' trip from memory, 1.6 us), the last groups' imbalance and the join.
// 8 x 16384 x 16384 (UE8M0) 32.5 us, 65%: a step's chain of loads, conversions and MMAs, 0.84 us for four warps per
// scheduler.  16 x 8192 x 16384 (UE8M0) 28.5 us, 2555 GB/s, 38%: converting X for every CTA (4 us), then 1.15 us per step;
// no pipe is full (while active: issue slots 50%, ALU 44%, tensor 30%, shared memory 44%).  Of the 8 cycles that one of a
// scheduler's four warps takes for an instruction 2.3 are fixed latencies, 1.3 shared memory and 1.0 the ALU's turn: a chain
// that more warps would hide, for which there are no registers.
// 1 x 4096 x 4096 4.0 us, 5 x 1000 x 2080 4.0 us: launch, trips to memory and the join.
#include <algorithm>
#include <atomic>
#include <initializer_list>
#include <mutex>
#include <type_traits>

#include "gb300gemm_testing.h"
#include "gemm_rows.cuh"
#include "ptx.cuh"

namespace gb300 {
namespace {

constexpr int MAX_M = 16;
constexpr int64_t MAX_K = 32768;
constexpr int LOG_WARPS = 4, WARPS = 1 << LOG_WARPS;
constexpr int CHUNK = 256;           // k per step of a warp
constexpr int BLOCKS = CHUNK / 32;   // 32-k blocks of a chunk: a column's 16-byte pieces
// Ring slots per warp, by the form (below).  Sixteen rows are bound by shared memory and issue, not by the requests in
// flight, and their activations need the room: 16 x 8192 x 16384 (UE8M0) 31.5 us with two slots, 39.1 with three.
__host__ __device__ constexpr int ahead_of(int form) { return form == 16 ? 2 : 3; }
constexpr int MOST_CLUSTER = 8;
constexpr int MOST_SMEM = 226 * 1024;
constexpr int W_BYTES = 16 * CHUNK / 2;        // weights of a slot

// A column's scale codes of a chunk, and the 32-bit words that a slot keeps for them: with K a multiple of 256
// every chunk's codes are aligned to their size and come in one copy; otherwise the aligned words that
// hold them do, and the codes are shifted out of those.
template <int MODE>
constexpr int CODES = MODE == GEMM_SCALE_UE8M0_32 ? BLOCKS : 2 * BLOCKS;
template <int MODE, bool ALIGNED>
constexpr int SF_WORDS = CODES<MODE> / 4 + (ALIGNED ? 0 : 1);
template <int MODE, bool ALIGNED>
constexpr int SF_STRIDE = ALIGNED ? CODES<MODE> : (SF_WORDS<MODE, ALIGNED> + 1) / 2 * 8;
template <int MODE, bool ALIGNED>
constexpr int SLOT = W_BYTES + 16 * SF_STRIDE<MODE, ALIGNED>;

// Forms of the kernel: the most rows of X
int form_of(int M) { return M <= 2 ? M : M <= 4 ? 4 : M <= 8 ? 8 : 16; }

struct MatvecParams {
    const void *x;
    const uint8_t *b, *sfb;
    const float *c;
    void *d;
    int M, N, K;
    uint32_t inverse_m, inverse_x, inverse_c;        // ceil(2^16 / d): of M, X's rows in shared memory, the cluster
    uint32_t inverse_t;  // ceil(2^32 / (cluster * slices)), or 0 for 2^32
    int out_bf16;
    int cluster, clusters;
    int log_slices;      // slices of K per CTA: S = 2^log_slices
    int x_stride;        // bytes of shared memory per row of X
    int held;            // tiles of a warp whose sums are kept before they are joined
};

// Divisions by what a launch fixes, as multiplications: integer division would be a third of a small product's time.
uint32_t inverse16(int d) { return (65536u + (uint32_t)d - 1) / (uint32_t)d; }
// i / d for i < 4096, d <= 16
__device__ __forceinline__ int over(int i, uint32_t inverse) { return (int)((uint32_t)i * inverse >> 16); }
// i / T for i < 2^24, T <= 128 (0 stands for T = 1)
uint32_t inverse32(int T) { return (uint32_t)(((1ull << 32) + (uint32_t)T - 1) / (uint32_t)T); }
__device__ __forceinline__ int over_t(int i, uint32_t inverse) { return inverse ? (int)__umulhi((uint32_t)i, inverse) : i; }

// eight packed e2m1 values (k ascending from the low nibble) to four pairs of halves
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// two UE4M3 codes (bit 7, which is not part of the format, clear) to halves
__device__ __forceinline__ uint32_t ue4m3x2(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return h;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    const __half2 d = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&d);
}
// bytes of (a, b) by four-bit selectors, whose top bit takes the byte's sign instead (__byte_perm has no such bit)
__device__ __forceinline__ uint32_t permute(uint32_t a, uint32_t b, uint32_t selector) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(selector));
    return d;
}
__device__ __forceinline__ float2 halves(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2 *>(&h)); }

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the same from zero
__device__ __forceinline__ void mma_16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// (a.x * b.x + c.x, a.y * b.y + c.y)
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// asynchronous copies of 16, 4 or BYTES bytes to shared memory: the first `bytes` of them from src, the rest zero
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const uint8_t *src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void copy_codes(uint32_t dst, const uint8_t *src, uint32_t bytes) {
    if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// four 8 x 16-byte matrices, one row address per lane; lane (g, t) gets bytes 4 t .. 4 t + 3 of row g of each
__device__ __forceinline__ void matrices(uint32_t addr, uint32_t (&v)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ uint32_t load_shared(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 load_shared2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t load_shared_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t load_shared_u16(uint32_t addr) {
    uint32_t v;
    asm volatile("{\n\t.reg .u16 h;\n\tld.shared.u16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// into v where `on`; elsewhere v stays as it is
__device__ __forceinline__ void load_shared4_if(bool on, uint4 &v, uint32_t addr) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t@p ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
                 : "r"(addr), "r"((uint32_t)on)
                 : "memory");
}
__device__ __forceinline__ uint4 load_shared4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float4 load_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void add4(float4 &a, float4 b) {
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
}
// Where the sums of row m of X and four of a tile's columns lie, in floats: a row's four quads swapped about by the row,
// so that neither the MMAs' layout of them nor rows of them meet in the banks more than twice
__device__ __forceinline__ int quad_of(int m, int quad) { return m * 16 + ((quad ^ (m >> 1)) & 3) * 4; }

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t min_s16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.s16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// 0xFFFF where a half of a is less than b's, as bf16 numbers that are not negative
__device__ __forceinline__ uint32_t less2(uint32_t a, uint32_t b) {
    return __hlt2_mask(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
}

// v * 2^e for e of -240 .. 254 (and what is above: infinity either way), in two steps that are factors of fp32
__device__ __forceinline__ float times_power(float v, int e) {
    e = min(e, 254);
    const int half = e >> 1;
    return v * __uint_as_float((uint32_t)(half + 127) << 23) * __uint_as_float((uint32_t)(e - half + 127) << 23);
}

// One chunk's products for eight rows of X from m0, where the chunk's one power of two per row does not hold them or a
// scale code is from 160 on: what lane (g, t) adds to its accumulators (columns n0 + g, n0 + g, n0 + g + 8, n0 + g + 8
// by rows 2t, 2t + 1; with FEW row t in x and z).  `w` is the chunk's slot, `shift` the columns' bits within the first words
// of their codes.
//
// bf16: X is read again and taken in bands of thirty exponents, the lowest first: band b holds biased exponents 30 b + 1 ..
// 30 b + 30 (band 0 also 0, the subnormal numbers), which are fp16's with 30 b subtracted, exactly.  Each band that
// the chunk spans runs through the MMAs as above, the rest being zeros, and its sums are scaled back in fp32.  Infinities and
// NaN go with the first band.  A gated unit's output spans two or three bands when its gates are far apart, and a
// chunk then takes about ten times as long: 16 x 8192 x 16384 (UE8M0) with gates of deviation 8 297 us instead of 28.1,
// 1 x 32768 x 8192 (UE4M3) 205 instead of 24.9 (with the sums in 64 bits on the CUDA cores 17164 and 1636).
template <typename XT, int MODE, bool FEW, bool ALIGNED>
__device__ __noinline__ float4 products_by_band(const MatvecParams &p, uint32_t w, uint2 shift, int chunk, int m0) {
    constexpr bool BF16 = !std::is_same<XT, __half>::value;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, m = m0 + g;
    const XT *x = static_cast<const XT *>(p.x) + (int64_t)m * p.K + chunk * CHUNK + t * 8;
    // the lane's eight values of block i
    auto load_x = [&](int i) {
        return m < p.M && chunk * CHUNK + i * 32 < p.K ? *reinterpret_cast<const uint4 *>(x + i * 32) : make_uint4(0, 0, 0, 0);
    };
    int band = 0, last = 0;
    bool special = false;                                // infinities or NaN
    if (BF16) {
        uint32_t low = 0x7FFF7FFFu, high = 0;
#pragma unroll
        for (int i = 0; i < BLOCKS; ++i) {
            const uint4 v = load_x(i);
            const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                low = min_s16x2(low, (q[k] | 0x80008000u) - 0x00010001u);       // |x| - 1 - 2^15, of zeros 2^15 - 1
                high = max_u16x2(high, q[k] & 0x7FFF7FFFu);
            }
        }
        const int top = (int)__reduce_max_sync(0xFFFFFFFFu, max(high >> 16, high & 0xFFFFu));
        const int least = __reduce_min_sync(0xFFFFFFFFu, min((int)low >> 16, (int)(int16_t)low)) + 32769;
        special = top >= 0x7F80;
        last = (max(min(top >> 7, 254), 1) - 1) / 30;
        band = min(max((least >> 7) - 1, 0) / 30, last);             // (a chunk of zeros meets its scale codes all the same)
    }
    float out[4] = {0.f, 0.f, 0.f, 0.f};
    for (; band <= last; ++band) {
        const uint32_t base = (uint32_t)(30 * band) * 0x00800080u, from = base + 0x00800080u, to = base + 31 * 0x00800080u;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int i = 0; i < BLOCKS; ++i) {
            const uint4 v = load_x(i);
            uint32_t b[4] = {v.x, v.y, v.z, v.w};
            if (BF16) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t a = b[k] & 0x7FFF7FFFu, sign = b[k] & 0x80008000u;
                    uint32_t in = band == 8 ? less2(a, 0x7F807F80u) : less2(a, to);
                    if (band != 0) in &= ~less2(a, from);
                    b[k] = sign | ((max_u16x2(a, base) - base) & in) << 3;
                    if (special) {
                        if ((a >> 16) >= 0x7F80u) b[k] |= (a >> 16) > 0x7F80u ? 0x7E000000u : 0x7C000000u;
                        if ((a & 0xFFFFu) >= 0x7F80u) b[k] |= (a & 0xFFFFu) > 0x7F80u ? 0x7E00u : 0x7C00u;
                    }
                }
            }
            uint32_t q[4], h[2][4];                      // words of columns g and g + 8 in the even block, then the odd one
            matrices(w + (lane & 15) * 128 + ((((i & ~1) + (lane >> 4)) ^ lane) & 7) * 16, q);
            int code[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                e2m1x8(i & 1 ? q[2 + r] : q[r], h[r]);
                const uint32_t at = w + W_BYTES + (g + 8 * r) * SF_STRIDE<MODE, ALIGNED> + (ALIGNED ? 0 : (r ? shift.y : shift.x) / 8);
                if (MODE == GEMM_SCALE_UE8M0_32) {
                    code[r] = (int)load_shared_u8(at + i);
                } else {
                    const uint32_t c = load_shared_u8(at + 2 * i + t / 2) & 0x7Fu, f = ue4m3x2(c * 0x0101u);
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[r][e] = mul2(h[r][e], f);
                }
            }
            if (MODE == GEMM_SCALE_UE8M0_32) {
                float acc[4];
                mma_16816_zero(acc, h[0][0], h[1][0], h[0][1], h[1][1], b[0], b[1]);
                mma_16816(acc, h[0][2], h[1][2], h[0][3], h[1][3], b[2], b[3]);
                const int e = (BF16 ? 30 * band - 112 : 0) - 127;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    out[k] += code[k / 2] == 255 ? __uint_as_float(0x7FC00000u) : times_power(acc[k], e + code[k / 2]);
            } else {
                mma_16816(sum, h[0][0], h[1][0], h[0][1], h[1][1], b[0], b[1]);
                mma_16816(sum, h[0][2], h[1][2], h[0][3], h[1][3], b[2], b[3]);
            }
        }
        special = false;
        if (MODE != GEMM_SCALE_UE8M0_32)
#pragma unroll
            for (int k = 0; k < 4; ++k) out[k] += times_power(sum[k], BF16 ? 30 * band - 112 : 0);
    }
    if (!FEW) return make_float4(out[0], out[1], out[2], out[3]);
    float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {                        // row t is lane t / 2's
        const float v = __shfl_sync(0xFFFFFFFFu, out[k], g * 4 + t / 2);
        if (t < p.M && (t & 1) == (k & 1)) (k < 2 ? d.x : d.z) = v;
    }
    return d;
}

// Rows of X in shared memory: forms 8 and 16 have zeros where X has no row
__host__ __device__ constexpr int x_rows(int form, int M) { return form > 4 ? form : M; }

// The CTA's chunks [lo, hi) of X into shared memory as the MMA's B operand: row by row, k ascending; lane (g, t) reads
// the eight k of 32 i + 8 t as one 128-bit word.  A row's stride is 64 bytes past a multiple of 128, so that two rows'
// words come from different banks.  BATCH loads are in flight per lane, and `then` runs behind the first of them.
//
// bf16: scaled per (row, chunk) by the power of two that takes the largest magnitude's exponent to 30, the top of
// f16's normal numbers; scale[lc * form + m] undoes it (times unbias), or is negative where the row's chunk does not
// convert exactly.  Two values are converted at once on their bits: the exponent less the largest's plus 30, three
// places up.  That is exact for zeros and what is within 2^-29 of the largest.
template <typename XT, int BATCH, typename Then>
__device__ __forceinline__ void stage_x(const MatvecParams &p, int lo, int hi, int form, float unbias, uint8_t *xf, float *scale,
                                        Then then) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = x_rows(form, p.M), all = (hi - lo) * rows;
#pragma unroll 1
    for (int first = warp; first == warp || first < all; first += WARPS * BATCH) {
        uint4 in[BATCH];
        int lc[BATCH], m[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int i = first + j * WARPS;
            lc[j] = over(i, p.inverse_x);
            m[j] = i - lc[j] * rows;
            const int k = (lo + lc[j]) * CHUNK + lane * 8;
            in[j] = make_uint4(0, 0, 0, 0);
            if (i < all && m[j] < p.M && k < p.K)
                in[j] = *reinterpret_cast<const uint4 *>(static_cast<const XT *>(p.x) + (int64_t)m[j] * p.K + k);
        }
        if (first == warp) then();
        // (no branch between the batch's members: their chains of reductions overlap)
        if constexpr (!std::is_same<XT, __half>::value) {
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                uint32_t w[4] = {in[j].x, in[j].y, in[j].z, in[j].w}, low = 0x7FFF7FFFu, high = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    low = min_s16x2(low, (w[q] | 0x80008000u) - 0x00010001u);       // |x| - 1 - 2^15, of zeros 2^15 - 1
                    high = max_u16x2(high, w[q] & 0x7FFF7FFFu);
                }
                const int top = (int)__reduce_max_sync(0xFFFFFFFFu, max(high >> 16, high & 0xFFFFu));
                const int least = min((int)low >> 16, (int)(int16_t)low) + 32769;
                const int e = top ? top >> 7 : 142;              // biased exponent; a chunk of zeros keeps scale 1
                const int base = (e - 30) << 7;
                // magnitudes within 2^-50 .. 2^40: what underflows before the factor is applied is below 2^-100 after
                const bool exact = __all_sync(0xFFFFFFFFu, least >= base + 128) && e >= 77 && e <= 167;
                const uint32_t both = (uint32_t)base * 0x10001u;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    w[q] = (w[q] & 0x80008000u) | (max_u16x2(w[q] & 0x7FFF7FFFu, both) - both) << 3;
                in[j] = make_uint4(w[0], w[1], w[2], w[3]);
                if (lane == 0 && first + j * WARPS < all)
                    scale[lc[j] * form + m[j]] = exact ? __uint_as_float((uint32_t)(e - 142 + 127) << 23) * unbias : -1.f;
            }
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
            if (first + j * WARPS < all)
                *reinterpret_cast<uint4 *>(xf + m[j] * p.x_stride + lc[j] * CHUNK * 2 + lane * 16) = in[j];
    }
}

// Joins the slices of K, the CTA's and the cluster's, always in the same order, and writes D: the `turns` groups of tiles
// from `group` on.
template <int FORM>
__device__ __forceinline__ void join_slices(const MatvecParams &p, float *parts, int group, int turns, int rank) {
    constexpr int PART = 16 * FORM;
    const int S = 1 << p.log_slices, R = WARPS >> p.log_slices, cluster = p.cluster;
    const int quads = R * 4 * p.M;                       // of a turn's outputs: n ascending, then row of X, then tile
    int from = 0, to = quads;
    if (cluster != 1) {
        for (int i = threadIdx.x; i < turns * quads && S > 1; i += WARPS * 32) {
            const int b = i / quads, q = i - b * quads, tile = over(q >> 2, p.inverse_m), m = (q >> 2) - tile * p.M;
            float4 *first = reinterpret_cast<float4 *>(parts + (b * WARPS + tile * S) * PART + quad_of(m, q & 3)), v = first[0];
            for (int s = 1; s < S; ++s) add4(v, first[s * PART / 4]);
            first[0] = v;
        }
        __syncwarp();
        cluster_sync();
        const int share = over(R * p.M + cluster - 1, p.inverse_c) * 4;        // whole rows of a tile
        from = min(rank * share, quads);
        to = min(from + share, quads);
    }
    const int each = to - from;
    const bool whole = p.N % 4 == 0;
    for (int i = threadIdx.x; i < turns * each; i += WARPS * 32) {
        const int b = i / each, q = from + i - b * each, tile = over(q >> 2, p.inverse_m), m = (q >> 2) - tile * p.M;
        const int n = ((group + b * p.clusters) * R + tile) * 16 + (q & 3) * 4;
        const float4 *first = reinterpret_cast<const float4 *>(parts + (b * WARPS + tile * S) * PART + quad_of(m, q & 3));
        if (n >= p.N) continue;
        const int64_t o = (int64_t)m * p.N + n;
        float4 c = make_float4(0.f, 0.f, 0.f, 0.f), v = c;
        if (p.c && whole) {
            c = *reinterpret_cast<const float4 *>(p.c + o);
        } else if (p.c) {
            c.x = p.c[o];
            if (n + 1 < p.N) c.y = p.c[o + 1];
            if (n + 2 < p.N) c.z = p.c[o + 2];
            if (n + 3 < p.N) c.w = p.c[o + 3];
        }
        if (cluster == 1) {
            for (int s = 0; s < S; ++s) add4(v, first[s * PART / 4]);
        } else {
            constexpr int AT_ONCE = FORM > 4 ? 8 : 4;        // (the registers of the loop over K are kept meanwhile)
            static_assert(MOST_CLUSTER % AT_ONCE == 0, "");
#pragma unroll 1
            for (int r0 = 0; r0 < cluster; r0 += AT_ONCE) {
                float4 part[AT_ONCE];
#pragma unroll
                for (int r = 0; r < AT_ONCE; ++r)
                    if (r0 + r < cluster) part[r] = load_cluster4(mapa_shared(smem_addr(first), r0 + r));
#pragma unroll
                for (int r = 0; r < AT_ONCE; ++r)
                    if (r0 + r < cluster) add4(v, part[r]);
            }
        }
        add4(v, c);
        if (p.out_bf16) {
            __nv_bfloat16 *d = static_cast<__nv_bfloat16 *>(p.d) + o;
            const __nv_bfloat162 low = __floats2bfloat162_rn(v.x, v.y), high = __floats2bfloat162_rn(v.z, v.w);
            if (whole) {
                *reinterpret_cast<uint2 *>(d) =
                    make_uint2(*reinterpret_cast<const uint32_t *>(&low), *reinterpret_cast<const uint32_t *>(&high));
            } else {
                d[0] = low.x;
                if (n + 1 < p.N) d[1] = low.y;
                if (n + 2 < p.N) d[2] = high.x;
                if (n + 3 < p.N) d[3] = high.y;
            }
        } else {
            float *d = static_cast<float *>(p.d) + o;
            if (whole) {
                *reinterpret_cast<float4 *>(d) = v;
            } else {
                d[0] = v.x;
                if (n + 1 < p.N) d[1] = v.y;
                if (n + 2 < p.N) d[2] = v.z;
                if (n + 3 < p.N) d[3] = v.w;
            }
        }
    }
}

template <typename XT, int MODE, int FORM, bool ALIGNED>
__global__ void __launch_bounds__(WARPS * 32, 1) matvec_kernel(const __grid_constant__ MatvecParams p) {
    constexpr bool SCALED_X = !std::is_same<XT, __half>::value;
    constexpr bool FEW = FORM <= 4;
    constexpr int NT = FORM == 16 ? 2 : 1;               // MMAs' columns of eight rows of X
    // FEW: blocks whose MMAs share an accumulator, and how often a chunk's sums are scaled
    constexpr int SPREAD = FEW ? 4 / FORM * (MODE == GEMM_SCALE_UE8M0_32 ? 2 : 1) : 1, FLUSHES = BLOCKS / SPREAD;
    // UE8M0 factors are taken 2^60 too large: code 0 (2^-127) is then a normal number, and a sum of 256 products
    // under codes below 160 still stays below 2^121
    constexpr uint32_t BIAS = MODE == GEMM_SCALE_UE8M0_32 ? 60 : 0;
    constexpr float UNBIAS = MODE == GEMM_SCALE_UE8M0_32 ? 0x1p-60f : 1.f;
    constexpr int PART = 16 * FORM, AHEAD = ahead_of(FORM);
    // each warp's ring; the sums to be joined [held][WARPS][16][FORM]; X; its scales
    extern __shared__ __align__(128) uint4 smem[];
    uint8_t *rings = reinterpret_cast<uint8_t *>(smem);
    float *parts = reinterpret_cast<float *>(rings + WARPS * AHEAD * SLOT<MODE, ALIGNED>);
    uint8_t *xf = reinterpret_cast<uint8_t *>(parts + p.held * WARPS * PART);
    float *xscale = reinterpret_cast<float *>(xf + x_rows(FORM, p.M) * p.x_stride);

    const int cluster = p.cluster, first_group = over(blockIdx.x, p.inverse_c), group_step = p.clusters;
    const int rank = blockIdx.x - first_group * cluster;              // in the cluster

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int S = 1 << p.log_slices, R = WARPS >> p.log_slices, tl = warp >> p.log_slices, sl = warp - (tl << p.log_slices);
    const int chunks = (p.K + CHUNK - 1) / CHUNK, first_slice = rank << p.log_slices;
    const int c0 = over_t(chunks * (first_slice + sl), p.inverse_t), c1 = over_t(chunks * (first_slice + sl + 1), p.inverse_t);
    const int lo = over_t(chunks * first_slice, p.inverse_t), hi = over_t(chunks * (first_slice + S), p.inverse_t);
    const int tiles = (p.N + 15) / 16, groups = (tiles + R - 1) >> (LOG_WARPS - p.log_slices);
    const int blocks = p.K / 32;                        // 32-k blocks of a column
    const int codes = blocks / BLOCKS * CODES<MODE> + blocks % BLOCKS * (CODES<MODE> / BLOCKS);       // of a column
    const uint32_t ring = smem_addr(rings) + warp * AHEAD * SLOT<MODE, ALIGNED>;

    // The next chunk to request.  A copy of weights takes four columns: lane l brings piece l & 7 of columns
    // l / 8, l / 8 + 4, + 8, + 12; `w_next` and `sf_next` are the lane's addresses in the next chunk.
    const int piece = lane & 7, col = lane >> 3;
    int next_group = first_group, next_chunk = c0, next_slot = 0, live = 0;
    bool full = false;
    const int64_t four = (int64_t)blocks * 64;               // four columns on
    const uint8_t *w_next = p.b, *sf_next = p.sfb;
    int sf_left = 0;
    auto enter_tile = [&]() {
        const int n0 = (next_group * R + tl) * 16;
        live = (p.N - n0 - col + 3) / 4;                        // the lane's columns inside the matrix
        full = n0 + 16 <= p.N;
        w_next = p.b + ((int64_t)(n0 + col) * blocks + c0 * BLOCKS + piece) * 16;
        const int n = n0 + (ALIGNED ? lane : lane >> 1);
        const int64_t at = (int64_t)n * codes + c0 * CODES<MODE>;
        sf_next = p.sfb + (ALIGNED ? at : (at & ~(int64_t)3) + (lane & 1) * 4);
        // codes of the column from here on, in bytes past sf_next
        sf_left = n >= p.N ? 0 : ALIGNED ? CODES<MODE> : codes - c0 * CODES<MODE> + (int)(at & 3) - (lane & 1) * 4;
    };
    auto request = [&]() {
        if (next_group < groups) {
            const uint32_t slot = ring + next_slot * SLOT<MODE, ALIGNED>;
            const uint32_t to = slot + col * 128, even = (piece ^ col) * 16, odd = even ^ 64;
            if (ALIGNED && full) {
                copy16(to + even, w_next, 16);
                copy16(to + 512 + odd, w_next + four, 16);
                copy16(to + 1024 + even, w_next + 2 * four, 16);
                copy16(to + 1536 + odd, w_next + 3 * four, 16);
            } else {
                const bool on = next_chunk * BLOCKS + piece < blocks;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool here = on && r < live;
                    copy16(to + r * 512 + (r & 1 ? odd : even), here ? w_next + r * four : p.b, here ? 16 : 0);
                }
            }
            const uint32_t sf = slot + W_BYTES;
            if (ALIGNED) {
                if (lane < 16) copy_codes<CODES<MODE>>(sf + lane * CODES<MODE>, sf_left ? sf_next : p.sfb, sf_left);
            } else {
                // bytes of this chunk that the column still has, from sf_next on
                const int most = CODES<MODE> + 3 - (lane & 1) * 4, left = min(sf_left, most);
#pragma unroll
                for (int i = 0; i < SF_STRIDE<MODE, ALIGNED> / 4; i += 2) {
                    const int bytes = max(0, min(left - 4 * i, 4));
                    copy4(sf + (lane >> 1) * SF_STRIDE<MODE, ALIGNED> + (lane & 1) * 4 + i * 4, bytes ? sf_next + i * 4 : p.sfb,
                          (uint32_t)bytes);
                }
                sf_left -= CODES<MODE>;
            }
            w_next += CHUNK / 2;
            sf_next += CODES<MODE>;
            next_slot = next_slot + 1 == AHEAD ? 0 : next_slot + 1;
            if (++next_chunk == c1) {
                next_chunk = c0;
                next_group += group_step;
                enter_tile();
            }
        }
        copies_commit();
    };
    enter_tile();
    rows::wait_for_previous();
    rows::let_next_launch();
    // X's first loads go out before the weights', which take longer
    stage_x<XT, FORM == 16 ? 8 : FORM == 8 ? 4 : 2>(p, lo, hi, FORM, UNBIAS, xf, xscale, [&]() {
#pragma unroll 1
        for (int j = 0; j < AHEAD - 1; ++j) request();
    });
    if (SCALED_X && FEW)
        for (int i = threadIdx.x; i < (hi - lo) * FORM; i += WARPS * 32)
            if (i % FORM >= p.M) xscale[i] = 0.f;
    __syncthreads();

    // The lane's word of X in block 0 of the CTA's first chunk, and whether it has one (in which blocks of SPREAD).
    // Lanes without keep zeros in the registers that the others load.
    uint32_t x_lane[NT];
    bool x_on[NT];
    int x_turn = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int m = FEW ? g / 2 % FORM : nt * 8 + g;
        x_on[nt] = !FEW || (m < p.M && (MODE == GEMM_SCALE_UE8M0_32 || (g & 1) == t / 2));
        x_lane[nt] = smem_addr(xf + (x_on[nt] ? m : 0) * p.x_stride + t * 16);
    }
    if (FEW) x_turn = MODE == GEMM_SCALE_UE8M0_32 ? g / 2 / FORM * 2 + (g & 1) : g / 2 / FORM;
    // the lane's row address for ldmatrix: lanes 0-7 columns 0-7 of block i, 8-15 columns 8-15, 16-31 the same of
    // block i + 1
    uint32_t w_lane[BLOCKS / 2];
#pragma unroll
    for (int i = 0; i < BLOCKS / 2; ++i) w_lane[i] = (lane & 15) * 128 + (((2 * i + (lane >> 4)) ^ lane) & 7) * 16;
    int slot = 0;
    for (int grp = first_group, turn = 0; grp < groups; grp += group_step) {
        float total[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) total[nt][i] = 0.f;
        uint4 x[SPREAD * NT];
#pragma unroll
        for (int i = 0; i < SPREAD * NT; ++i) x[i] = make_uint4(0, 0, 0, 0);
        const int n0 = (grp * R + tl) * 16;
        // where a column's codes begin within their first word, in bits
        const uint32_t shift[2] = {(uint32_t)((n0 + g) * (codes & 3) & 3) * 8, (uint32_t)((n0 + g + 8) * (codes & 3) & 3) * 8};

#pragma unroll 1
        for (int ch = c0; ch < c1; ++ch) {
            copies_wait<AHEAD - 2>();
            __syncwarp();            // every lane's copies have landed, and every lane is done with the slot before this
            request();
            const uint32_t w = ring + slot * SLOT<MODE, ALIGNED>;
            slot = slot + 1 == AHEAD ? 0 : slot + 1;
            const int lc = ch - lo;
            float2 xs[NT];               // of rows 2t and 2t + 1; FEW: of row t % FORM
            bool fine = true;
            if (SCALED_X) {
                float worst = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float *at = xscale + lc * FORM + (FEW ? t % FORM : nt * 8 + 2 * t);
                    xs[nt] = FEW ? make_float2(at[0], 0.f) : *reinterpret_cast<const float2 *>(at);
                    worst = fminf(worst, fminf(xs[nt].x, xs[nt].y));
                }
                fine = worst >= 0.f;
            }
            // FEW: the lane's pair of codes for each flush, of columns g and g + 8; else those columns' codes
            constexpr int CODE_WORDS = FEW ? FLUSHES : CODES<MODE> / 4;
            uint32_t code[2][CODE_WORDS];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t sf = w + W_BYTES + (g + 8 * r) * SF_STRIDE<MODE, ALIGNED>;
                if constexpr (FEW && FORM < 4) {
#pragma unroll
                    for (int f = 0; f < FLUSHES; ++f) {
                        const uint32_t at = sf + (f * (4 / FORM) + t / FORM) * 2;
                        code[r][f] = ALIGNED ? load_shared_u16(at)
                                             : load_shared_u8(at + shift[r] / 8) | load_shared_u8(at + shift[r] / 8 + 1) << 8;
                    }
                } else {
                    uint32_t v[CODES<MODE> / 4 + 1];
                    if constexpr (ALIGNED && MODE == GEMM_SCALE_UE8M0_32) {
                        const uint2 l = load_shared2(sf);
                        v[0] = l.x;
                        v[1] = l.y;
                    } else if constexpr (ALIGNED) {
                        const uint4 l = load_shared4(sf);
                        v[0] = l.x;
                        v[1] = l.y;
                        v[2] = l.z;
                        v[3] = l.w;
                    } else {
                        uint32_t l[SF_WORDS<MODE, ALIGNED>];
#pragma unroll
                        for (int i = 0; i < SF_WORDS<MODE, ALIGNED>; ++i) l[i] = load_shared(sf + 4 * i);
#pragma unroll
                        for (int i = 0; i < CODES<MODE> / 4; ++i) v[i] = __funnelshift_r(l[i], l[i + 1], shift[r]);
                    }
#pragma unroll
                    for (int f = 0; f < CODE_WORDS; ++f) code[r][f] = !FEW ? v[f] : f & 1 ? v[f / 2] >> 16 : v[f / 2] & 0xFFFFu;
                }
                // a code from 160 on has its top bit and one of the next two set
                if (MODE == GEMM_SCALE_UE8M0_32) {
                    uint32_t high = 0;
#pragma unroll
                    for (int f = 0; f < CODE_WORDS; ++f) high |= code[r][f] & (code[r][f] << 1 | code[r][f] << 2);
                    fine = fine && (high & 0x80808080u) == 0;
                }
            }
            if ((SCALED_X || MODE == GEMM_SCALE_UE8M0_32) && !__all_sync(0xFFFFFFFFu, fine)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float4 add = products_by_band<XT, MODE, FEW, ALIGNED>(p, w, make_uint2(shift[0], shift[1]), ch, nt * 8);
                    total[nt][0] += add.x;
                    total[nt][1] += add.y;
                    total[nt][2] += add.z;
                    total[nt][3] += add.w;
                }
                continue;
            }
            float sum[NT][4];            // the chunk's, before the activations' scale
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[nt][i] = 0.f;
            uint32_t mul[2][BLOCKS];     // UE4M3 with more than four rows: the lane's scale in each block, twice
            if constexpr (MODE == GEMM_SCALE_UE4M3_16 && !FEW) {
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int i = 0; i < BLOCKS; i += 2) {
                        // even codes for lanes t = 0, 1 (a block's first 16 k), odd ones for t = 2, 3, each twice
                        const uint32_t twice = __byte_perm(code[r][i / 2], 0, t < 2 ? 0x2200u : 0x3311u) & 0x7F7F7F7Fu;
                        mul[r][i] = ue4m3x2(twice);
                        mul[r][i + 1] = ue4m3x2(twice >> 16);
                    }
            }
            // UE8M0 with more than four rows: the codes plus BIAS, cut where a float's third and fourth byte meet
            uint32_t high7[2][2], low1[2][2];
            if constexpr (MODE == GEMM_SCALE_UE8M0_32 && !FEW) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t c = code[i / 2][i % 2] + BIAS * 0x01010101u;
                    high7[i / 2][i % 2] = c >> 1 & 0x7F7F7F7Fu;
                    low1[i / 2][i % 2] = c << 7 & 0x80808080u;
                }
            }
            uint32_t q[4];               // words of (block i, columns g and g + 8), (block i + 1, the same)
            // sums that long chains of MMAs add to are kept twice, for every other MMA
            constexpr int CHAINS = SPREAD >= 4 ? 2 : 1;
            float acc[CHAINS][NT][4];
#pragma unroll
            for (int i = 0; i < BLOCKS; ++i) {
                if (i % 2 == 0) matrices(w + w_lane[i / 2], q);
                uint32_t a[2][4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    e2m1x8(q[(i & 1) * 2 + r], a[r]);
                    if constexpr (MODE == GEMM_SCALE_UE4M3_16 && !FEW) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) a[r][e] = mul2(a[r][e], mul[r][i]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint4 &b = x[i % SPREAD * NT + nt];
                    const uint32_t at = x_lane[nt] + lc * (CHUNK * 2) + i * 64;
                    if constexpr (FEW) load_shared4_if(x_on[nt] && x_turn == i % SPREAD, b, at);
                    else b = load_shared4(at);
                    if constexpr (MODE == GEMM_SCALE_UE4M3_16 && !FEW) {
                        mma_16816(sum[nt], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
                        mma_16816(sum[nt], a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
                        continue;
                    }
                    if (i % SPREAD == 0) mma_16816_zero(acc[0][nt], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
                    else mma_16816(acc[0][nt], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
                    if (CHAINS == 2 && i % SPREAD == 0) mma_16816_zero(acc[1][nt], a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
                    else mma_16816(acc[CHAINS - 1][nt], a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
                    if (i % SPREAD != SPREAD - 1) continue;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        // the factors of a row's two sums
                        float2 s;
                        if constexpr (MODE == GEMM_SCALE_UE4M3_16) {
                            s = halves(ue4m3x2(code[r][i / SPREAD] & 0x7F7Fu));
                        } else if constexpr (FEW) {
                            // 2^(code - 127 + BIAS)
                            const uint32_t pair = code[r][i / SPREAD];
                            s.x = __uint_as_float(((pair & 0xFFu) << 23) + (BIAS << 23));
                            s.y = __uint_as_float(((pair & 0xFF00u) << 15) + (BIAS << 23));
                        } else {
                            // the same in one permutation: selector 8 takes a byte's top bit, which is 0 in high7
                            const int k = i % 4;
                            s.x = s.y = __uint_as_float(permute(high7[r][i / 4], low1[r][i / 4], k << 12 | (4 + k) << 8 | 0x88));
                        }
                        float2 v = make_float2(acc[0][nt][2 * r], acc[0][nt][2 * r + 1]);
                        if (CHAINS == 2) {
                            v.x += acc[1][nt][2 * r];
                            v.y += acc[1][nt][2 * r + 1];
                        }
                        const float2 d = fma2(v, s, make_float2(sum[nt][2 * r], sum[nt][2 * r + 1]));
                        sum[nt][2 * r] = d.x;
                        sum[nt][2 * r + 1] = d.y;
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float factor = !SCALED_X ? UNBIAS : i & 1 && !FEW ? xs[nt].y : xs[nt].x;
                    total[nt][i] = fmaf(sum[nt][i], factor, total[nt][i]);
                }
        }

        float *mine = parts + (turn * WARPS + warp) * PART;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int quad = 2 * r + (g >> 2);
                if constexpr (FEW) {                     // a row's columns of the MMA
                    float v = total[nt][2 * r] + total[nt][2 * r + 1];
                    if (FORM <= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
                    if (FORM <= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
                    if (t < FORM) mine[quad_of(t, quad) + (g & 3)] = v;
                } else {
                    float *at = mine + quad_of(nt * 8 + 2 * t, quad) + (g & 3);         // (the next row's is 16 on)
                    at[0] = total[nt][2 * r];
                    at[16] = total[nt][2 * r + 1];
                }
            }
        if (++turn < p.held && grp + group_step < groups) continue;

        __syncthreads();
        join_slices<FORM>(p, parts, grp - (turn - 1) * group_step, turn, rank);
        turn = 0;
        if (grp + group_step < groups) {                 // the sums have been read before others take their place
            __syncwarp();
            if (cluster == 1) __syncthreads();
            else cluster_sync();
        }
    }
    __syncwarp();
    // No CTA's shared memory goes while another may read it.  (Relaxed: this is not to wait for the stores of D.)
    if (cluster != 1)
        asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

int slot_bytes(int mode, int K) {
    if (K % CHUNK == 0) return mode == GEMM_SCALE_UE8M0_32 ? SLOT<GEMM_SCALE_UE8M0_32, true> : SLOT<GEMM_SCALE_UE4M3_16, true>;
    return mode == GEMM_SCALE_UE8M0_32 ? SLOT<GEMM_SCALE_UE8M0_32, false> : SLOT<GEMM_SCALE_UE4M3_16, false>;
}

// How the product is cut (see the head of this file)
struct MatvecShape {
    int log_slices, cluster, x_stride, held, smem, grid;
};
// resident[c]: clusters of c CTAs that run at once
MatvecShape search_shape(int M, int N, int K, bool scaled_x, int slot, const int *resident) {
    const int chunks = (K + CHUNK - 1) / CHUNK, tiles = (N + 15) / 16, form = form_of(M);
    const int ring = WARPS * ahead_of(form) * slot, part = WARPS * 16 * form * 4;
    MatvecShape best{};
    double best_cost = 0;
    for (int c = 1; c <= MOST_CLUSTER && c <= chunks; ++c)
        for (int log_s = 0; log_s <= LOG_WARPS && (c << log_s) <= chunks; ++log_s) {
            const int S = 1 << log_s;
            MatvecShape s;
            s.cluster = c;
            s.log_slices = log_s;
            const int room = (chunks + c - 1) / c;
            s.x_stride = room * CHUNK * 2 + 64;
            const int base = ring + x_rows(form, M) * s.x_stride + (scaled_x ? room * form * 4 : 0);
            if (base + part > MOST_SMEM || resident[c] == 0) continue;
            const int R = WARPS / S, groups = (tiles + R - 1) / R, clusters = groups < resident[c] ? groups : resident[c];
            const int turns = (groups + clusters - 1) / clusters, fit = (MOST_SMEM - base) / part;
            s.held = turns < fit ? turns : fit;
            s.smem = base + s.held * part;
            s.grid = clusters * c;
            // Microseconds, fitted to 3170 measured products (all shapes of 123 sizes of 1 to 16 rows; the shape taken is
            // within 1.1% of the best one on average, 13% at worst): a warp's steps, at the rate of its weights or of
            // its arithmetic; the turns' ends; a warp's share of X; the joins.
            const int joins = (turns + s.held - 1) / s.held;
            const double copy = WARPS * slot / std::min(46e3, 6.63e6 / s.grid);
            const double step = form == 16 ? std::max(copy, 1.15) : form == 8 ? std::max(copy, 0.84) : copy;
            const double turn = form == 16 ? 0.5 : form == 8 ? 0.09 : 0.14, join = c == 1 ? 0.58 : 1.22 + 0.16 * c;
            const double cost = turns * ((chunks + c * S - 1) / (c * S) * step + turn) + 0.32 * x_rows(form, M) * room / WARPS +
                                joins * join;
            if (best.grid == 0 || cost < best_cost) {
                best = s;
                best_cost = cost;
            }
        }
    return best;
}

// The search is a microsecond of the caller's time: each thread keeps the last few sizes' results.
MatvecShape matvec_shape(int M, int N, int K, bool scaled_x, int slot, const int *resident) {
    struct Known {
        int M, N, K, scaled_x, slot;
        const int *resident;
        MatvecShape shape;
    };
    constexpr int KNOWN = 8;
    static thread_local Known known[KNOWN];
    static thread_local int next;
    for (const Known &k : known)
        if (k.M == M && k.N == N && k.K == K && k.scaled_x == scaled_x && k.slot == slot && k.resident == resident) return k.shape;
    known[next] = Known{M, N, K, scaled_x, slot, resident, search_shape(M, N, K, scaled_x, slot, resident)};
    const MatvecShape s = known[next].shape;
    next = (next + 1) % KNOWN;
    return s;
}

constexpr int MAX_DEVICES = 64;

template <typename XT, int MODE, int FORM, bool ALIGNED>
cudaError_t launch(const MatvecShape &s, const MatvecParams &p, cudaStream_t stream) {
    static std::atomic<bool> ready[MAX_DEVICES];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!ready[dev].load(std::memory_order_acquire)) {               // (setting it twice does no harm)
        e = cudaFuncSetAttribute(matvec_kernel<XT, MODE, FORM, ALIGNED>, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST_SMEM);
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_release);
    }
    const rows::Launch l(s.grid, WARPS * 32, s.smem, s.cluster, stream);
    return cudaLaunchKernelEx(&l.config, matvec_kernel<XT, MODE, FORM, ALIGNED>, p);
}

// How many clusters of 1 .. 8 CTAs run at once on the current device (asked once: one CTA fills an SM whatever
// the instance, and a cluster stays within a group of SMs whose size is not a multiple of every c)
cudaError_t resident_clusters(const int **out) {
    static std::mutex mu;
    static int known[MAX_DEVICES][MOST_CLUSTER + 1];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (known[dev][1] == 0) {
        const auto kernel = matvec_kernel<__half, GEMM_SCALE_UE4M3_16, 16, true>;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST_SMEM);
        int found[MOST_CLUSTER + 1] = {};
        for (int c = 1; c <= MOST_CLUSTER && e == cudaSuccess; ++c) {
            const rows::Launch l(c, WARPS * 32, MOST_SMEM, c, nullptr, false);
            e = cudaOccupancyMaxActiveClusters(&found[c], kernel, &l.config);
        }
        if (e != cudaSuccess) return e;
        for (int c = 1; c <= MOST_CLUSTER; ++c) known[dev][c] = found[c];
    }
    *out = known[dev];
    return cudaSuccess;
}

template <typename XT, int MODE, bool ALIGNED>
cudaError_t launch(const MatvecShape &s, const MatvecParams &p, cudaStream_t stream) {
    switch (form_of(p.M)) {
        case 1: return launch<XT, MODE, 1, ALIGNED>(s, p, stream);
        case 2: return launch<XT, MODE, 2, ALIGNED>(s, p, stream);
        case 4: return launch<XT, MODE, 4, ALIGNED>(s, p, stream);
        case 8: return launch<XT, MODE, 8, ALIGNED>(s, p, stream);
        default: return launch<XT, MODE, 16, ALIGNED>(s, p, stream);
    }
}
template <typename XT, int MODE>
cudaError_t launch(const MatvecShape &s, const MatvecParams &p, cudaStream_t stream) {
    return p.K % CHUNK == 0 ? launch<XT, MODE, true>(s, p, stream) : launch<XT, MODE, false>(s, p, stream);
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
    const int *resident = nullptr;
    if (resident_clusters(&resident) != cudaSuccess) return GEMM_ERR_CUDA;
    const MatvecShape s = matvec_shape((int)M, (int)N, (int)K, x == GEMM_BF16, slot_bytes(block_scaled, (int)K), resident);
    if (s.grid == 0) return GEMM_ERR_UNSUPPORTED;        // (clusters of eight hold the activations of every M and K)
    const int T = s.cluster << s.log_slices;
    const MatvecParams p{X,
                         static_cast<const uint8_t *>(B),
                         SFB,
                         C,
                         D,
                         (int)M,
                         (int)N,
                         (int)K,
                         inverse16((int)M),
                         inverse16(x_rows(form_of((int)M), (int)M)),
                         inverse16(s.cluster),
                         T == 1 ? 0u : inverse32(T),
                         d == GEMM_BF16,
                         s.cluster,
                         s.grid / s.cluster,
                         s.log_slices,
                         s.x_stride,
                         s.held};
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = x == GEMM_F16 ? launch<__half>(block_scaled, s, p, stream)
                                        : launch<__nv_bfloat16>(block_scaled, s, p, stream);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

// Test hook (declared in include/gb300gemm_testing.h): the launch's shape.
extern "C" gemm_status gemm_testing_matvec_shape(int64_t M, int64_t N, int64_t K, gemm_dtype x, int block_scaled,
                                                 int largest_cluster, int *out) {
    if (!out || M < 1 || M > MAX_M || N < 1 || N > INT32_MAX / 16 || K < 32 || K > MAX_K || K % 32 != 0 || largest_cluster < 1 ||
        largest_cluster > MOST_CLUSTER || (x != GEMM_F16 && x != GEMM_BF16) ||
        (block_scaled != GEMM_SCALE_UE8M0_32 && block_scaled != GEMM_SCALE_UE4M3_16))
        return GEMM_ERR_INVALID_ARG;
    int resident[MOST_CLUSTER + 1] = {};
    for (int c = 1; c <= largest_cluster; ++c) resident[c] = 152 / c;
    const MatvecShape s = search_shape((int)M, (int)N, (int)K, x == GEMM_BF16, slot_bytes(block_scaled, (int)K), resident);
    if (s.grid == 0) return GEMM_ERR_UNSUPPORTED;
    out[0] = s.grid;
    out[1] = s.cluster;
    out[2] = 1 << s.log_slices;
    out[3] = s.smem;
    return GEMM_OK;
}

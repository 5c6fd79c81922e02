// Shared pieces of the row operators (gemm_norm.cu, gemm_gate.cu): vectors of consecutive elements in every element
// type, the e4m3 block scale rule, the row and unit a thread of many rows takes, and the per-device facts of a launch.
//
// A thread works on units of N consecutive elements of a row, N = 8 or 16.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gb300gemm.h"

namespace gb300 {
namespace rows {

constexpr int BLOCK = 32;         // elements per scale

// ------------------------------------------------------------------ launches

// Every kernel of these operators may begin while the one before it in the stream ends (a programmatic launch).  It
// touches memory only after its own wait, which is for the whole of what came before, and then (the norm's gradient when
// its rows are done) lets the next one begin.  It reads with ordinary loads: those for data that stays the same all through a
// kernel (__ldg) may be moved ahead of the wait, and what an earlier kernel writes does not stay the same.
// Letting the next one begin before the wait has kernels queue up on the SMs: a row of small calls then takes longer (the norm of
// 333 x 2048 3.8 us instead of 2.3, the gate of it 2.7 instead of 2.0; of one row 0.3 us less).
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A launch's configuration: programmatic, and with a cluster where there is one; a query's has the cluster alone
struct Launch {
    cudaLaunchAttribute attributes[2];
    cudaLaunchConfig_t config;
    Launch(int ctas, dim3 block, int smem, int cluster, cudaStream_t stream, bool programmatic = true) : attributes{}, config{} {
        unsigned n = 0;
        if (programmatic) {
            attributes[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attributes[n++].val.programmaticStreamSerializationAllowed = 1;
        }
        if (cluster > 1 || !programmatic) {
            attributes[n].id = cudaLaunchAttributeClusterDimension;
            attributes[n].val.clusterDim.x = (unsigned)cluster;
            attributes[n].val.clusterDim.y = attributes[n].val.clusterDim.z = 1;
            ++n;
        }
        config.gridDim = dim3((unsigned)ctas);
        config.blockDim = block;
        config.dynamicSmemBytes = (size_t)smem;
        config.stream = stream;
        config.attrs = attributes;
        config.numAttrs = n;
    }
    Launch(const Launch &) = delete;
};
template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int ctas, dim3 block, int smem, cudaStream_t stream, const Args &...args) {
    const Launch l(ctas, block, smem, 1, stream);
    return cudaLaunchKernelEx(&l.config, kernel, args...);
}

// ------------------------------------------------------------------ elements

// 16-byte pieces of N elements
template <typename T, int N>
constexpr int PIECES = sizeof(T) * N / 16;

template <int P>
__device__ __forceinline__ void load_pieces(const void *p, bool on, uint4 (&q)[P]) {       // zeros where not `on`
#pragma unroll
    for (int i = 0; i < P; ++i) q[i] = on ? static_cast<const uint4 *>(p)[i] : make_uint4(0, 0, 0, 0);
}

template <int N>
__device__ __forceinline__ void unpack(const float *, const uint4 *q, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        v[4 * i] = __uint_as_float(q[i].x);
        v[4 * i + 1] = __uint_as_float(q[i].y);
        v[4 * i + 2] = __uint_as_float(q[i].z);
        v[4 * i + 3] = __uint_as_float(q[i].w);
    }
}
template <int N>
__device__ __forceinline__ void unpack(const __nv_bfloat16 *, const uint4 *q, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
        const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
            v[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
    }
}

__device__ __forceinline__ uint32_t pack2(const __nv_bfloat16 *, float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint32_t pack2(const __half *, float lo, float hi) {
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}
template <typename T16>
__device__ __forceinline__ uint4 pack8(const T16 *t, const float *v) {
    return make_uint4(pack2(t, v[0], v[1]), pack2(t, v[2], v[3]), pack2(t, v[4], v[5]), pack2(t, v[6], v[7]));
}

template <int N>
__device__ __forceinline__ void load(const float *p, float (&v)[N]) {
    uint4 q[N / 4];
    load_pieces(p, true, q);
    unpack(p, q, v);
}
template <int N>
__device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&v)[N]) {
    uint4 q[N / 8];
    load_pieces(p, true, q);
    unpack(p, q, v);
}
template <int N>
__device__ __forceinline__ void store(float *p, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) reinterpret_cast<float4 *>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
template <typename T16, int N>
__device__ __forceinline__ void store(T16 *p, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) reinterpret_cast<uint4 *>(p)[i] = pack8(p, v + 8 * i);
}

// v rounded to the type of p, stored there where `on`, and kept in fp32
template <int N>
__device__ __forceinline__ void round_store(float *p, bool on, float (&v)[N]) {
    if (on) store(p, v);
}
template <int N>
__device__ __forceinline__ void round_store(__nv_bfloat16 *p, bool on, float (&v)[N]) {
    uint4 q[N / 8];
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
        q[i] = pack8(p, v + 8 * i);
        if (on) reinterpret_cast<uint4 *>(p)[i] = q[i];
    }
    unpack(p, q, v);
}

// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// ------------------------------------------------------------- the gated unit

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

// The same for two values, operation by operation
__device__ __forceinline__ void sigmoid2(float2 g, float2 &s, float2 &t) {
    float2 p = mul2(g, both(-0.72134752f)), r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p.x) : "f"(p.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p.y) : "f"(p.y));
    p = mul2(p, both(0x1p-16f));
    const float2 d = fma2(p, p, both(0x1p-32f)), q = mul2(p, p);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
    s = mul2(r, both(0x1p-32f));
    t = mul2(make_float2(fminf(q.x, 0x1p126f), fminf(q.y, 0x1p126f)), r);
}

// ------------------------------------------------------------- e4m3 with UE8M0

// Scale code of a block with maximum magnitude amax: s = 2^(code - 127) is the smallest power of two
// (not below 2^-127) with amax <= 448 s.  448 = 1.75 * 2^8, so the exponent field minus 8 is the code,
// plus one when the mantissa passes 1.75: adding 2^23 - 0x600000 - 1 carries into the exponent
// exactly then.  An infinite amax gives 247: 448 * 2^120 is past fp32's largest value, so the
// saturated element still decodes to infinity.
__device__ __forceinline__ uint32_t scale_code(float amax) {
    const int e = (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 8;
    return (uint32_t)max(e, 0);
}
__device__ __forceinline__ float scale_inverse(uint32_t code) { return __uint_as_float((254u - code) << 23); }   // 2^(127 - code)
// 2^(code - 127); code 0 is fp32's subnormal 2^-127
__device__ __forceinline__ float scale_value(uint32_t code) {
    return __uint_as_float(code ? code << 23 : 0x400000u);
}

// two values to e4m3 (round to nearest even; the scale keeps finite values within 448), lo in the low byte
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Quantise 16 or 8 elements of a block (the rest is with the neighbouring one or three lanes; all of them are active, and
// pass zeros past a row's end): stores the codes at p where `on`; returns the block's scale code.
template <int N>
__device__ __forceinline__ uint32_t quantise(const float (&v)[N], uint8_t *p, bool on) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) amax = fmaxf(amax, fabsf(v[i]));      // fmaxf drops NaN
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    if (N == 8) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    const uint32_t code = scale_code(amax);
    const float inv = scale_inverse(code);
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        w[i] = e4m3x2(v[4 * i] * inv, v[4 * i + 1] * inv) | e4m3x2(v[4 * i + 2] * inv, v[4 * i + 3] * inv) << 16;
    if constexpr (N == 16) {
        if (on) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        if (on) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
    return code;
}

// eight e4m3 codes times a scale
__device__ __forceinline__ void decode(uint2 q, float s, float (&v)[8]) {
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;                                   // two halves: every e4m3 value is exact in f16
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[i / 2] >> (16 * (i & 1)))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        const float2 m = mul2(f, both(s));
        v[2 * i] = m.x;
        v[2 * i + 1] = m.y;
    }
}

// -------------------------------------------------------------- units of many rows

// Which unit of which row thread i of a launch takes: i / per_row by a multiplication, exact for i < 2^31.
struct Units {
    int64_t row0;            // the launch's first row
    int rows, per_row;
    uint32_t inverse, shift; // ceil(2^(32 + shift) / per_row), shift = floor(log2(per_row - 1))

    __device__ __forceinline__ bool place(uint32_t i, int64_t &row, int &u) const {
        const uint32_t r = per_row == 1 ? i : __umulhi(i, inverse) >> shift;
        row = row0 + r;
        u = (int)(i - r * per_row);
        return r < (uint32_t)rows;
    }
};

// Launch over M rows of per_row units each, 256 threads per CTA: one launch, or more where the units number 2^31 or
// over.  launch(units, ctas) returns its cudaError_t.
template <typename F>
gemm_status over_rows(int64_t M, int per_row, F launch) {
    Units u{};
    u.per_row = per_row;
    while (((per_row - 1) >> (u.shift + 1)) != 0) ++u.shift;
    if (per_row > 1) u.inverse = (uint32_t)((((uint64_t)1 << (32 + u.shift)) + per_row - 1) / per_row);
    const int64_t most = ((int64_t)INT32_MAX - 255) / per_row;
    for (; u.row0 < M; u.row0 += most) {
        u.rows = (int)(M - u.row0 < most ? M - u.row0 : most);
        const unsigned ctas = (unsigned)(((int64_t)u.rows * per_row + 255) / 256);
        if (launch(u, ctas) != cudaSuccess) return GEMM_ERR_CUDA;
    }
    return GEMM_OK;
}

// ------------------------------------------------------------------ host side

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The current device's SM count; GEMM_ERR_UNSUPPORTED for anything but compute capability 10.3.
gemm_status device_sms(int *sms);      // gemm_norm.cu

}  // namespace rows
}  // namespace gb300

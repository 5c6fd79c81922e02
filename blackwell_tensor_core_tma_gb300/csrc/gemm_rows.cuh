// Shared pieces of the row operators (gemm_norm.cu, gemm_gate.cu): eight-element vectors in every
// element type, the e4m3 block scale rule, and the per-device facts their launches need.
//
// A "unit" is eight consecutive elements of a row: 16 bytes of a 16-bit type (one 128-bit access per
// thread, consecutive threads on consecutive units), 32 bytes of fp32, 8 bytes of e4m3.  A scale
// block (32 elements) is four units, held by four consecutive lanes of a warp.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gb300gemm.h"

namespace gb300 {
namespace rows {

constexpr int UNIT = 8;           // elements per unit
constexpr int BLOCK = 32;         // elements per scale

// ------------------------------------------------------------------ elements

__device__ __forceinline__ void load_unit(const float *p, float (&v)[UNIT]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ void load_unit(const __nv_bfloat16 *p, float (&v)[UNIT]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
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

__device__ __forceinline__ void store_unit(float *p, const float (&v)[UNIT]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <typename T16>
__device__ __forceinline__ void store_unit(T16 *p, const float (&v)[UNIT]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack2(p, v[0], v[1]), pack2(p, v[2], v[3]), pack2(p, v[4], v[5]),
                                               pack2(p, v[6], v[7]));
}

// v rounded to the type's values, in fp32
__device__ __forceinline__ float round_as(const float *, float v) { return v; }
__device__ __forceinline__ float round_as(const __nv_bfloat16 *, float v) {
    return __bfloat162float(__float2bfloat16_rn(v));
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

// Quantise a unit against its block (four consecutive lanes, all of them active; lanes past the row's
// end pass zeros): returns the codes, and the block's scale code in every lane.
__device__ __forceinline__ uint2 quantise_unit(const float (&v)[UNIT], uint32_t &code) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < UNIT; ++i) amax = fmaxf(amax, fabsf(v[i]));     // fmaxf drops NaN
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    code = scale_code(amax);
    const float inv = scale_inverse(code);
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = e4m3x2(v[2 * i] * inv, v[2 * i + 1] * inv);
    return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

// eight e4m3 codes times a scale
__device__ __forceinline__ void decode_unit(uint2 q, float s, float (&v)[UNIT]) {
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;                                   // two halves: every e4m3 value is exact in f16
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[i / 2] >> (16 * (i & 1)))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        v[2 * i] = f.x * s;
        v[2 * i + 1] = f.y * s;
    }
}

// ------------------------------------------------------------------ host side

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The current device's SM count; GEMM_ERR_UNSUPPORTED for anything but compute capability 10.3.
gemm_status device_sms(int *sms);      // gemm_norm.cu

}  // namespace rows
}  // namespace gb300

// Device helpers of the block-scaled 8-bit form: the scale rule, fp8
// conversions, and element types widened to fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "../../include/vnm.h"
#include "vnm_internal.h"

namespace vnm {

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// 8 fp32 values rounded, in pairs.
__device__ __forceinline__ void narrow8(const float (&f)[8], float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = f[j];
}
__device__ __forceinline__ void narrow8(const float (&f)[8], __half (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) *reinterpret_cast<__half2*>(&v[j]) = __floats2half2_rn(f[j], f[j + 1]);
}
__device__ __forceinline__ void narrow8(const float (&f)[8], __nv_bfloat16 (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) *reinterpret_cast<__nv_bfloat162*>(&v[j]) = __floats2bfloat162_rn(f[j], f[j + 1]);
}

// Largest finite values of the two formats.
constexpr float kMaxE4m3 = 448.f;
constexpr float kMaxE5m2 = 57344.f;
// Smallest scale: a group of zeros (or of values below 2^-100 of the format's
// range) keeps a finite reciprocal.
constexpr float kMinScale = 0x1p-100f;

// Magnitudes compare as the integers of their bits, which orders
// finite < Inf < NaN: one integer maximum then finds both the largest magnitude
// of a group and whether it holds a non-finite value.
__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The larger magnitude, NaN if either is one.
__device__ __forceinline__ float max_magnitude(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

// Scale of a group of largest magnitude m, m * (1 / F) but at least 2^-100, and
// its reciprocal, correctly rounded (both NaN for a group with a non-finite value,
// so that its q are NaN too).
__device__ __forceinline__ float group_scale(float m, bool e5m2, float& inv) {
    float s = m * (e5m2 ? 1.f / kMaxE5m2 : 1.f / kMaxE4m3);
    s = s < kMinScale ? kMinScale : s;  // (false for NaN)
    if (m == __uint_as_float(0x7F800000u)) s = __uint_as_float(0x7FC00000u);
    inv = __frcp_rn(s);
    return s;
}
__device__ __forceinline__ float group_scale(uint32_t bits, bool e5m2, float& inv) {
    return group_scale(__uint_as_float(bits), e5m2, inv);
}

// v / s correctly rounded, from s's reciprocal: the rounded product is within an ulp, and its
// remainder, exact in one fused multiply-add, times the reciprocal corrects it (P. Markstein,
// Computation of elementary functions on the IBM RISC System/6000 processor, IBM J. Res.
// Dev. 34, 1990; the remainder may lose bits for s below 2^-85). The product alone sends an
// element near the middle between two fp8 values to either. The remainder's sign keeps -0.
// The quantiser's 8192 x 4096 bf16 to both forms takes 31.4 us so, 27.8 with the product
// alone, 31.5 with two elements an instruction (f32x2: moving them into pairs costs as much).
__device__ __forceinline__ float quotient(float v, float s, float inv) {
    const float q = v * inv;
    return fmaf(fmaf(q, s, -v), -inv, q);
}

// Two fp32 values to fp8 (nearest even, saturating, NaN kept), `lo` in the low byte.
__device__ __forceinline__ uint32_t to_fp8x2(float lo, float hi, bool e5m2) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, e5m2 ? __NV_E5M2 : __NV_E4M3);
}

__device__ __forceinline__ uint32_t to_fp8x4(float a, float b, float c, float d, bool e5m2) {
    return to_fp8x2(a, b, e5m2) | (to_fp8x2(c, d, e5m2) << 16);
}

// An element of a vnm_dtype array.
__device__ __forceinline__ float load_any(const void* p, int type, int64_t i) {
    if (type == VNM_F32) return static_cast<const float*>(p)[i];
    if (type == VNM_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ void store_any(void* p, int type, int64_t i, float v) {
    if (type == VNM_F32)
        static_cast<float*>(p)[i] = v;
    else if (type == VNM_F16)
        static_cast<__half*>(p)[i] = __float2half_rn(v);
    else
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ float activate(int act, float v) {
    // a comparison rather than fmaxf, which would turn NaN into 0
    if (act == VNM_ACT_RELU) return v < 0.f ? 0.f : v;
    if (act == VNM_ACT_GELU) return gelu(v);
    return v;
}

}  // namespace vnm

// Device parts that the dense 16-bit kernels share: activations and their
// slopes, and an output's last steps, eight neighbouring columns at a time.
#pragma once

#include "vnm_dense16.h"
#include "vnm_fp8.cuh"
#include "vnm_umma.cuh"

namespace vnm {

// 1 / (1 + e^-v). The quotient is off by 2 ulp; for v < -87 (e^-v above 2^126) it may
// be 0, where the value is below 2^-126.
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + expf(-v)); }

__device__ __forceinline__ void activate8(int act, float (&v)[8]) {
    if (act == VNM_ACT_NONE) return;
    if (act == VNM_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= sigmoid(v[j]);
    } else if (act == VNM_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = gelu(v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = activate(VNM_ACT_RELU, v[j]);
    }
}

// A 16-bit element's or pair's fp32 values.
__device__ __forceinline__ float2 widen2(uint32_t w, bool bf16) {
    if (bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ void widen8(const uint4& w, bool bf16, float (&v)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 p = widen2(u[j], bf16);
        v[2 * j] = p.x;
        v[2 * j + 1] = p.y;
    }
}

__device__ __forceinline__ uint4 pack16x8(const float (&v)[8], bool bf16) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = bf16 ? to_bf16x2(v[2 * j], v[2 * j + 1]) : to_f16x2(v[2 * j], v[2 * j + 1]);
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// v to elements at .. at + 7 of a vnm_dtype array, the first `left` of them; vec: they are
// 16-byte aligned.
__device__ __forceinline__ void store8(void* p, int type, int64_t at, bool vec, int64_t left, const float (&v)[8]) {
    if (vec && left >= 8) {
        if (type == VNM_F32) {
            float4* to = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
            to[0] = make_float4(v[0], v[1], v[2], v[3]);
            to[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = pack16x8(v, type == VNM_BF16);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) store_any(p, type, at + j, v[j]);
    }
}

__device__ __forceinline__ void load8(const void* p, int type, int64_t at, bool vec, int64_t left, float (&v)[8]) {
    if (vec && left >= 8) {
        if (type == VNM_F32) {
            const float4* from = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
            const float4 a = from[0], b = from[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            widen8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at), type == VNM_BF16, v);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < left ? load_any(p, type, at + j) : 0.f;
    }
}

// v / s in 8 bits (the quotient correctly rounded) to 8 bytes, the first `left` of them.
__device__ __forceinline__ void store_fp8x8(uint8_t* p, bool vec, int64_t left, const float (&v)[8], float s, float inv,
                                            bool e5m2) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = quotient(v[j], s, inv);
    const uint32_t lo = to_fp8x4(q[0], q[1], q[2], q[3], e5m2), hi = to_fp8x4(q[4], q[5], q[6], q[7], e5m2);
    if (vec && left >= 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) p[j] = static_cast<uint8_t>((j < 4 ? lo : hi) >> (8 * (j & 3)));
    }
}

// Where a product's results go.
struct OutArgs {
    int64_t T, R;
    void* y[2];
    const void* res[2];
    const void* bias;
    int64_t ld_y, ld_res;
    int y_type, bias_type, act;
    bool y_vec, res_vec;  // rows start on 16 bytes
    int keep;             // a KeepKind
    bool e5m2, g_vec, u_vec;
    Kept g, u;
};

// Row t, columns r .. r + 7 of a gated pair from the sums g and u: the checkpoints,
// then y = act(g) * u. The scales and their reciprocals are of the row's group (kKeep8).
__device__ __forceinline__ void finish_gated8(const OutArgs& o, int64_t t, int64_t r, float (&g)[8], const float (&u)[8],
                                              float gs, float ginv, float us, float uinv) {
    const int64_t left = o.R - r;
    if (left <= 0) return;
    if (o.keep == kKeep16) {
        store8(o.g.p, o.y_type, t * o.g.ld + r, o.g_vec, left, g);
        store8(o.u.p, o.y_type, t * o.u.ld + r, o.u_vec, left, u);
    } else if (o.keep == kKeep8) {
        store_fp8x8(static_cast<uint8_t*>(o.g.p) + t * o.g.ld + r, o.g_vec, left, g, gs, ginv, o.e5m2);
        store_fp8x8(static_cast<uint8_t*>(o.u.p) + t * o.u.ld + r, o.u_vec, left, u, us, uinv, o.e5m2);
    }
    activate8(o.act, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] *= u[j];
    store8(o.y[0], o.y_type, t * o.ld_y + r, o.y_vec, left, g);
}

}  // namespace vnm

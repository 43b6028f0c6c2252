// Element-wise part of the gated pair's backward pass:
//
//   dg = dy * u * act'(g), du = dy * act(g), h = act(g) * u
//
// with g and u as the forward pass kept them, in 16 bits or in the block-scaled
// 8-bit form. Bound by memory traffic: 8 neighbouring columns a thread, 16-byte loads
// and stores (8 bytes of an 8-bit checkpoint) where the rows allow them. dg and du are
// rounded once to 16 bits: the tensor cores take no wider operands at this rate.
//   silu'(g) = s (1 + g (1 - s)), s = 1 / (1 + e^-g); gelu'(g) = Phi(g) + g phi(g).
#include <algorithm>

#include "vnm_dense16.cuh"
#include "vnm_internal.h"

namespace vnm {
namespace {

// act(g) and act'(g)
__device__ __forceinline__ float2 with_slope(int act, float g) {
    if (act == VNM_ACT_SILU) {
        const float s = sigmoid(g);
        return make_float2(g * s, s * (1.f + g * (1.f - s)));
    }
    if (act == VNM_ACT_GELU) {
        const float cdf = 0.5f * (1.f + erff(g * 0.70710678118654752f));
        return make_float2(g * cdf, cdf + g * (0.39894228040143268f * expf(-0.5f * g * g)));
    }
    // (a NaN passes through both)
    if (act == VNM_ACT_RELU) return make_float2(g < 0.f ? 0.f : g, g > 0.f ? 1.f : g <= 0.f ? 0.f : g);
    return make_float2(g, 1.f);
}

__device__ __forceinline__ void load_kept8(const GatedGradArgs& a, const Kept& k, int type, int64_t t, int64_t f, bool vec,
                                           int64_t left, float (&v)[8]) {
    if (a.keep == kKeep16) {
        load8(k.p, type, t * k.ld + f, vec, left, v);
        return;
    }
    const uint8_t* p = static_cast<const uint8_t*>(k.p) + t * k.ld + f;
    const float s = k.s[t * k.s_rs + (f >> 7) * k.s_cs];
    uint32_t w[2] = {0u, 0u};
    if (vec && left >= 8) {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        w[0] = q.x;
        w[1] = q.y;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) w[j >> 2] |= static_cast<uint32_t>(p[j]) << (8 * (j & 3));
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[j >> 2] >> (8 * (j & 3))),
                                                         a.e5m2 ? __NV_E5M2 : __NV_E4M3);
        const float2 q = __half22float2(__half2(h));
        v[j] = q.x * s;
        v[j + 1] = q.y * s;
    }
}

__global__ void __launch_bounds__(256) gated_grad_kernel(const GatedGradArgs a, bool dy_vec, bool g_vec, bool u_vec, bool d_vec,
                                                         bool h_vec) {
    const int64_t per_row = (a.F + 7) / 8;
    const int type = a.bf16 ? VNM_BF16 : VNM_F16;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < a.T * per_row;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t t = i / per_row, f = 8 * (i - t * per_row), left = a.F - f;
        float dy[8] = {}, g[8], u[8];
        if (a.dy != nullptr) load8(a.dy, type, t * a.ld_dy + f, dy_vec, left, dy);
        load_kept8(a, a.g, type, t, f, g_vec, left, g);
        load_kept8(a, a.u, type, t, f, u_vec, left, u);
        float h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 s = with_slope(a.act, g[j]);
            h[j] = s.x * u[j];
            g[j] = dy[j] * u[j] * s.y;
            u[j] = dy[j] * s.x;
        }
        if (a.dg != nullptr) {
            store8(a.dg, type, t * a.ld_d + f, d_vec, left, g);
            store8(a.du, type, t * a.ld_d + f, d_vec, left, u);
        }
        if (a.h != nullptr) store8(a.h, type, t * a.ld_h + f, h_vec, left, h);
    }
}

}  // namespace

cudaError_t launch_gated_grad(const GatedGradArgs& a, int sm_count, cudaStream_t stream) {
    auto rows_aligned = [](const void* p, int64_t ld_bytes, int n) {
        return reinterpret_cast<uintptr_t>(p) % n == 0 && ld_bytes % n == 0;
    };
    const int k = a.keep == kKeep8 ? 1 : 2;
    const int64_t n = a.T * ((a.F + 7) / 8);
    const int64_t blocks = std::min<int64_t>((n + 255) / 256, static_cast<int64_t>(sm_count) * 8);
    gated_grad_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
        a, rows_aligned(a.dy, a.ld_dy * 2, 16), rows_aligned(a.g.p, a.g.ld * k, 8 * k), rows_aligned(a.u.p, a.u.ld * k, 8 * k),
        rows_aligned(a.dg, a.ld_d * 2, 16) && rows_aligned(a.du, a.ld_d * 2, 16), rows_aligned(a.h, a.ld_h * 2, 16));
    return cudaGetLastError();
}

}  // namespace vnm

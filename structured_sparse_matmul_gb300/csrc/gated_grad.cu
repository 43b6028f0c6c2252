// Element-wise part of the gated pair's backward pass:
//
//   dg = dy * u * act'(g), du = dy * act(g), h = act(g) * u
//
// with g and u as the forward pass kept them, in 16 bits or in the block-scaled
// 8-bit form. Bound by memory traffic: a warp takes 256 columns of a row, 8 neighbours a lane,
// 16-byte loads and stores (8 bytes of an 8-bit checkpoint) where the rows allow them, a unit's loads ahead of the
// work; rows of another alignment go element by element, neighbours to neighbouring lanes. dg and du
// are rounded once to 16 bits: the tensor cores take no wider operands at this rate.
// Measured: 8192 x 11008, SiLU, 8-bit checkpoints 141 us (0.9 GB, 135 us at a copy's rate; 42 instructions an element);
// 1024 x 4096, GELU, 16-bit checkpoints 10 us.
//   silu'(g) = s (1 + g (1 - s)), s = 1 / (1 + e^-g); gelu'(g) = Phi(g) + g phi(g).
#include <algorithm>

#include "vnm_dense16.cuh"
#include "vnm_internal.h"

namespace vnm {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 256;  // columns of a row that a warp takes at a time

// act(g) and act'(g)
template <int ACT>
__device__ __forceinline__ float2 with_slope(float g) {
    if (ACT == VNM_ACT_SILU) {
        const float s = sigmoid(g);
        return make_float2(g * s, s * (1.f + g * (1.f - s)));
    }
    if (ACT == VNM_ACT_GELU) {
        // Phi's tail as e^(-g^2 / 2) times a polynomial in 1 / (1 + 0.3275911 |g| / sqrt 2) (M. Abramowitz and
        // I. A. Stegun, Handbook of Mathematical Functions, 7.1.26): phi shares the exponential, where erff has one of its own
        // and two branches. The formula is within 7e-8; evaluated in fp32 the cdf is within 3e-7 (near g = 0, where terms of
        // 1.4 cancel), 6e-7 with e and t at their bounds of 2 and 1 ulp, and 1e-7 beyond |g| = 3: below a rounding to fp16.
        const float e = exp2_fast(-0.5f * kLog2E * g * g), t = reciprocal_fast(fmaf(0.23164189f, fabsf(g), 1.f));
        const float poly = fmaf(fmaf(fmaf(fmaf(1.061405429f, t, -1.453152027f), t, 1.421413741f), t, -0.284496736f), t, 0.254829592f);
        const float tail = 0.5f * e * t * poly, cdf = g < 0.f ? tail : 1.f - tail;
        return make_float2(g * cdf, cdf + g * (0.39894228040143268f * e));
    }
    // (a NaN passes through both)
    if (ACT == VNM_ACT_RELU) return make_float2(g < 0.f ? 0.f : g, g > 0.f ? 1.f : g <= 0.f ? 0.f : g);
    return make_float2(g, 1.f);
}

// A lane's eight elements of a matrix, as they are stored, and their scales: of columns 0 to 3 and of 4 to 7.
struct Part {
    uint32_t w[4];
    float s[2];
};

template <bool FP8>
__device__ __forceinline__ Part load_part(const Kept& k, int64_t t, const Cols& c) {
    Part p{{0u, 0u, 0u, 0u}, {1.f, 1.f}};
    if (FP8) {
        p.s[0] = p.s[1] = k.s[t * k.s_rs + (min(c.first, c.end - 1) >> 7) * k.s_cs];
        if (!c.vec) p.s[1] = k.s[t * k.s_rs + (min(c.at(4), c.end - 1) >> 7) * k.s_cs];
        const uint8_t* row = static_cast<const uint8_t*>(k.p) + t * k.ld;
        if (c.whole()) {
            const uint2 q = __ldcs(reinterpret_cast<const uint2*>(row + c.first));
            p.w[0] = q.x;
            p.w[1] = q.y;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c.at(j) < c.end) p.w[j >> 2] |= static_cast<uint32_t>(row[c.at(j)]) << (8 * (j & 3));
        }
    } else {
        const uint16_t* row = static_cast<const uint16_t*>(k.p) + t * k.ld;
        if (c.whole()) {
            const uint4 q = __ldcs(reinterpret_cast<const uint4*>(row + c.first));
            p.w[0] = q.x;
            p.w[1] = q.y;
            p.w[2] = q.z;
            p.w[3] = q.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c.at(j) < c.end) p.w[j >> 1] |= static_cast<uint32_t>(row[c.at(j)]) << (16 * (j & 1));
        }
    }
    return p;
}

template <bool FP8>
__device__ __forceinline__ void widen_part(const Part& p, bool bf16, bool e5m2, float (&v)[8]) {
    if constexpr (!FP8) {
        widen8(make_uint4(p.w[0], p.w[1], p.w[2], p.w[3]), bf16, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(p.w[j >> 2] >> (8 * (j & 3))),
                                                             e5m2 ? __NV_E5M2 : __NV_E4M3);
            const float2 q = __half22float2(__half2(h));
            v[j] = q.x * p.s[j >> 2];
            v[j + 1] = q.y * p.s[j >> 2];
        }
    }
}

// VEC: the rows of every matrix start on 16 bytes (8-bit checkpoints: 8); a lane then takes 8 neighbours.
template <int ACT, bool FP8, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) gated_grad_kernel(const GatedGradArgs a) {
    const int lane = threadIdx.x & 31, type = a.bf16 ? VNM_BF16 : VNM_F16;
    const int64_t per_row = (a.F + kUnit - 1) / kUnit, warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    // units warp, warp + warps, ...; the place of the next one without a division
    const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t dt = warps / per_row, dn = warps - dt * per_row;
    int64_t t = warp / per_row, n = warp - t * per_row;
    const Kept kdy{const_cast<void*>(a.dy), a.ld_dy, nullptr, 0, 0};
    auto columns = [&](int64_t at) { return Cols{at * kUnit + (VEC ? 8 * lane : lane), a.F, VEC ? 1 : 32, VEC}; };
    Part g_next, u_next, d_next;  // of the unit (t, n): a unit's loads are in flight while the one before it is worked on
    auto fetch = [&] {
        const Cols c = columns(n);
        if (t >= a.T || c.none()) return;
        g_next = load_part<FP8>(a.g, t, c);
        u_next = load_part<FP8>(a.u, t, c);
        d_next = Part{{0u, 0u, 0u, 0u}, {1.f, 1.f}};
        if (a.dy != nullptr) d_next = load_part<false>(kdy, t, c);
    };
    after_previous_grid();
    let_next_grid_start();
    fetch();
#pragma unroll 1
    while (t < a.T) {
        const Part pg = g_next, pu = u_next, pd = d_next;
        const Cols c = columns(n);
        const int64_t row = t;
        t += dt;
        n += dn;
        if (n >= per_row) {
            n -= per_row;
            ++t;
        }
        fetch();
        if (c.none()) continue;
        float dy[8], g[8], u[8], h[8];
        widen_part<false>(pd, a.bf16, false, dy);
        widen_part<FP8>(pg, a.bf16, a.e5m2, g);
        widen_part<FP8>(pu, a.bf16, a.e5m2, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 s = with_slope<ACT>(g[j]);
            h[j] = s.x * u[j];
            g[j] = dy[j] * u[j] * s.y;
            u[j] = dy[j] * s.x;
        }
        if (a.dg != nullptr) {
            store8(a.dg, type, row * a.ld_d, c, g);
            store8(a.du, type, row * a.ld_d, c, u);
        }
        if (a.h != nullptr) store8(a.h, type, row * a.ld_h, c, h);
    }
}

template <int ACT, bool FP8>
cudaError_t launch(const GatedGradArgs& a, bool vec, int sm_count, cudaStream_t stream) {
    const int64_t units = a.T * ((a.F + kUnit - 1) / kUnit);
    const int64_t blocks = std::min<int64_t>((units + kThreads / 32 - 1) / (kThreads / 32), static_cast<int64_t>(sm_count) * 8);
    return vec ? launch_early(gated_grad_kernel<ACT, FP8, true>, blocks, kThreads, 0, 1, stream, a)
               : launch_early(gated_grad_kernel<ACT, FP8, false>, blocks, kThreads, 0, 1, stream, a);
}

template <int ACT>
cudaError_t launch(const GatedGradArgs& a, bool vec, int sm_count, cudaStream_t stream) {
    return a.keep == kKeep8 ? launch<ACT, true>(a, vec, sm_count, stream) : launch<ACT, false>(a, vec, sm_count, stream);
}

}  // namespace

cudaError_t launch_gated_grad(const GatedGradArgs& a, int sm_count, cudaStream_t stream) {
    auto rows_aligned = [](const void* p, int64_t ld_bytes, int n) {
        return p == nullptr || (reinterpret_cast<uintptr_t>(p) % n == 0 && ld_bytes % n == 0);
    };
    const int k = a.keep == kKeep8 ? 1 : 2;
    const bool vec = rows_aligned(a.dy, a.ld_dy * 2, 16) && rows_aligned(a.g.p, a.g.ld * k, 8 * k) &&
                     rows_aligned(a.u.p, a.u.ld * k, 8 * k) && rows_aligned(a.dg, a.ld_d * 2, 16) &&
                     rows_aligned(a.du, a.ld_d * 2, 16) && rows_aligned(a.h, a.ld_h * 2, 16);
    switch (a.act) {
        case VNM_ACT_SILU: return launch<VNM_ACT_SILU>(a, vec, sm_count, stream);
        case VNM_ACT_GELU: return launch<VNM_ACT_GELU>(a, vec, sm_count, stream);
        case VNM_ACT_RELU: return launch<VNM_ACT_RELU>(a, vec, sm_count, stream);
        default: return launch<VNM_ACT_NONE>(a, vec, sm_count, stream);
    }
}

}  // namespace vnm

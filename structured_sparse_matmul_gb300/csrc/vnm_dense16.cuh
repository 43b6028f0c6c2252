// Device parts that the dense 16-bit kernels share: activations and their
// slopes, and an output's last steps, eight neighbouring columns at a time.
#pragma once

#include "vnm_dense16.h"
#include "vnm_fp8.cuh"
#include "vnm_umma.cuh"

namespace vnm {

// The launches let this grid start while the stream's previous one drains: nothing of global memory is
// touched before its end.
__device__ __forceinline__ void after_previous_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The same of a grid that may run beside the one before: what came before that one has ended then. What such a grid reads
// by way of L1 (`l1`) must not be what an earlier grid read there before its other CTAs wrote it.
__device__ __forceinline__ void after_the_one_before(bool beside, bool l1) {
    if (!beside)
        after_previous_grid();
    else if (l1)
        __threadfence();
}
// From here on the next such grid may start (it waits for our end in the same way). Called after the wait: only one
// grid is ahead at a time.
__device__ __forceinline__ void let_next_grid_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// 2^v and 1 / v by the special-function unit, within 2 ulp and 1 ulp; subnormal arguments and results are 0.
__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float reciprocal_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
constexpr float kLog2E = 1.4426950408889634f;

// 1 / (1 + e^-v). 2^(-v log2 e) is off by a relative 2^-22 (1 + |v|) or so (the product's rounding), which 1 + e^-v
// damps by s e^-v <= 1 and, where v is far below 0, v's own factor s; the reciprocal by 1 ulp, and for v < -87
// (e^-v above 2^126) it is 0, where the value is below 2^-126. v * sigmoid(v) is within 8 * 2^-23 |v|.
__device__ __forceinline__ float sigmoid(float v) { return reciprocal_fast(1.f + exp2_fast(-kLog2E * v)); }

template <int N>
__device__ __forceinline__ void activate_all(int act, float (&v)[N]) {
    if (act == VNM_ACT_NONE) return;
    if (act == VNM_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] *= sigmoid(v[j]);
    } else if (act == VNM_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = gelu(v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = activate(VNM_ACT_RELU, v[j]);
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

// Eight columns of a row that a lane handles: neighbours (step 1), whose loads and stores are of 16
// bytes where the rows are aligned; or, where they are not, columns `step` lanes apart, so that
// the warp's accesses of single elements are of neighbours.
struct Cols {
    int64_t first, end;  // the first column; the matrix's columns
    int step;
    bool vec;            // the rows start on 16 bytes (and step is 1)
    __device__ __forceinline__ int64_t at(int j) const { return first + j * step; }
    __device__ __forceinline__ bool whole() const { return vec && first + 8 <= end; }
    __device__ __forceinline__ bool none() const { return first >= end; }
};

// Eight elements as they are stored: of a 16-bit type in w[0 .. 3]. Loading them apart from widening
// them lets several rows' loads be in flight.
struct Raw8 {
    uint32_t w[8];
};

__device__ __forceinline__ Raw8 load_raw8(const void* p, int type, int64_t row, const Cols& c) {
    Raw8 r;
    const bool f32 = type == VNM_F32;
    if (c.whole()) {
        const uint4* from = f32 ? reinterpret_cast<const uint4*>(static_cast<const float*>(p) + row + c.first)
                                : reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + row + c.first);
        const uint4 a = from[0];
        r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
        if (f32) {
            const uint4 b = from[1];
            r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
        }
    } else if (f32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.w[j] = c.at(j) < c.end ? static_cast<const uint32_t*>(p)[row + c.at(j)] : 0u;
    } else {
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = c.at(j) < c.end ? static_cast<const uint16_t*>(p)[row + c.at(j)] : 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) r.w[j] = h[2 * j] | (h[2 * j + 1] << 16);
    }
    return r;
}

__device__ __forceinline__ void widen_raw8(const Raw8& r, int type, float (&v)[8]) {
    if (type == VNM_F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r.w[j]);
    } else {
        widen8(make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]), type == VNM_BF16, v);
    }
}

// v to the row's columns, `row` being the index of its first element.
__device__ __forceinline__ void store8(void* p, int type, int64_t row, const Cols& c, const float (&v)[8]) {
    if (type == VNM_F32) {
        float* to = static_cast<float*>(p) + row;
        if (c.whole()) {
            reinterpret_cast<float4*>(to + c.first)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(to + c.first)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c.at(j) < c.end) to[c.at(j)] = v[j];
        }
        return;
    }
    uint16_t* to = static_cast<uint16_t*>(p) + row;
    const uint4 w = pack16x8(v, type == VNM_BF16);
    if (c.whole()) {
        *reinterpret_cast<uint4*>(to + c.first) = w;
    } else {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c.at(j) < c.end) to[c.at(j)] = static_cast<uint16_t>(u[j >> 1] >> (16 * (j & 1)));
    }
}

// v / s in 8 bits (the quotient correctly rounded) to a row's columns.
__device__ __forceinline__ void store_fp8x8(uint8_t* row, const Cols& c, const float (&v)[8], float s, float inv, bool e5m2) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = quotient(v[j], s, inv);
    const uint32_t lo = to_fp8x4(q[0], q[1], q[2], q[3], e5m2), hi = to_fp8x4(q[4], q[5], q[6], q[7], e5m2);
    if (c.whole()) {
        *reinterpret_cast<uint2*>(row + c.first) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c.at(j) < c.end) row[c.at(j)] = static_cast<uint8_t>((j < 4 ? lo : hi) >> (8 * (j & 3)));
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
    int keep;                         // a KeepKind
    bool y_vec, res_vec, keep_vec;    // rows start on 16 bytes (8-bit checkpoints: 8)
    bool y_tma, keep_tma;             // rows start on 16 bytes
    bool e5m2;
    Kept g, u;
};

// A scale of the 8-bit form and its reciprocal, of G's and of U's group.
struct Scales {
    float g, g_inv, u, u_inv;
};

// Some columns of row t of a gated pair's checkpoints.
__device__ __forceinline__ void keep_gated8(const OutArgs& o, int64_t t, const Cols& c, const float (&g)[8], const float (&u)[8],
                                            const Scales& s) {
    if (o.keep == kKeep16) {
        store8(o.g.p, o.y_type, t * o.g.ld, c, g);
        store8(o.u.p, o.y_type, t * o.u.ld, c, u);
    } else if (o.keep == kKeep8) {
        store_fp8x8(static_cast<uint8_t*>(o.g.p) + t * o.g.ld, c, g, s.g, s.g_inv, o.e5m2);
        store_fp8x8(static_cast<uint8_t*>(o.u.p) + t * o.u.ld, c, u, s.u, s.u_inv, o.e5m2);
    }
}

// Some columns of row t of a gated pair: y = act(g) * u.
__device__ __forceinline__ void finish_gated8(const OutArgs& o, int64_t t, const Cols& c, float (&g)[8], const float (&u)[8]) {
    activate_all(o.act, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] *= u[j];
    store8(o.y[0], o.y_type, t * o.ld_y, c, g);
}

// The bias of a lane's columns (0 without one).
__device__ __forceinline__ void bias8(const OutArgs& o, const Cols& c, float (&b)[8]) {
    if (o.bias == nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = 0.f;
        return;
    }
    widen_raw8(load_raw8(o.bias, o.bias_type, 0, Cols{c.first, c.end, c.step, false}), o.bias_type, b);
}

// Some columns of row t of one product from their sums, the bias's columns b and the residual's r.
__device__ __forceinline__ void finish8(const OutArgs& o, int seg, int64_t t, const Cols& c, float (&v)[8], const float (&b)[8],
                                        const Raw8& r) {
    if (c.none()) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += b[j];
    activate_all(o.act, v);
    if (o.res[seg] != nullptr) {
        float w[8];
        widen_raw8(r, o.y_type, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += w[j];
    }
    store8(o.y[seg], o.y_type, t * o.ld_y, c, v);
}

// The largest magnitudes of g and u over LANES neighbouring lanes that hold 8 each (NaN if one is).
template <int LANES>
__device__ __forceinline__ float2 largest_of(const float (&g)[8], const float (&u)[8]) {
    float2 m = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        m.x = max_magnitude(m.x, g[j]);
        m.y = max_magnitude(m.y, u[j]);
    }
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) {
        m.x = max_magnitude(m.x, __shfl_xor_sync(0xFFFFFFFFu, m.x, d));
        m.y = max_magnitude(m.y, __shfl_xor_sync(0xFFFFFFFFu, m.y, d));
    }
    return m;
}

// The scales of group n of row t with these largest magnitudes, stored where `write` says.
__device__ __forceinline__ Scales scales_of(const OutArgs& o, float2 largest, int64_t t, int64_t n, bool write) {
    Scales s;
    s.g = group_scale(largest.x, o.e5m2, s.g_inv);
    s.u = group_scale(largest.y, o.e5m2, s.u_inv);
    if (write) {
        o.g.s[t * o.g.s_rs + n * o.g.s_cs] = s.g;
        o.u.s[t * o.u.s_rs + n * o.u.s_cs] = s.u;
    }
    return s;
}

}  // namespace vnm

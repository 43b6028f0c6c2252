// The block-scaled 8-bit form of a matrix, plain and transposed, in one pass.
//
//   s = max(max |x| / F, 2^-100) over a group of 128 (or a 128 x 128 block),
//   q = fp8(x * (1 / s))
//
// Bound by memory traffic (2 or 4 bytes read, 1 or 2 written for an element)
// as long as the instructions for an element stay few. A CTA takes a 128 x 128
// tile, a thread 8 rows x 8 columns of it in registers: it holds 8 neighbours of
// every row (8 bytes of q) and 8 neighbours of every column (8 bytes of qt), so
// neither form passes through shared memory element by element. Row maxima are
// reduced over the 16 lanes of a row, column maxima over the 16 row groups
// through shared memory; the transposed bytes cross one 16 KB tile in
// shared memory, in 8-byte units whose index is XORed with the column group so
// that writing 16 columns and reading 16 rows both touch every bank once.
#include "vnm_dense.h"
#include "vnm_fp8.cuh"

namespace vnm {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct Raw8;  // 8 elements as 16-byte words
template <>
struct Raw8<float> {
    static constexpr int kWords = 2;
};
template <>
struct Raw8<__half> {
    static constexpr int kWords = 1;
};
template <>
struct Raw8<__nv_bfloat16> {
    static constexpr int kWords = 1;
};

__device__ __forceinline__ uint2 pack8(const float (&v)[8], float inv, bool e5m2) {
    return make_uint2(to_fp8x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv, e5m2),
                      to_fp8x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv, e5m2));
}

// 8 bytes to p[0 .. 7], the first `n` of them.
__device__ __forceinline__ void store8(uint8_t* p, uint2 v, int64_t n, bool vec) {
    if (vec && n >= 8) {
        *reinterpret_cast<uint2*>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = static_cast<uint8_t>((i < 4 ? v.x : v.y) >> (8 * (i & 3)));
    }
}

// vec: rows of x are 16-byte aligned, vec_q / vec_qt: rows of q / qt 8-byte aligned.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    fp8_quantize_kernel(const QuantArgs a, int64_t tiles_c, bool vec, bool vec_q, bool vec_qt) {
    __shared__ uint32_t colmax[8][kGroup];
    __shared__ uint2 turned[kGroup][16];
    const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
    const int64_t r0 = tr * kGroup, c0 = tc * kGroup;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cg = threadIdx.x & 15;   // column group: columns 8 cg .. 8 cg + 7
    const int rg = threadIdx.x >> 4;   // row group: rows 8 rg .. 8 rg + 7
    const int64_t col = c0 + 8 * cg, row = r0 + 8 * rg;
    const int64_t ncol = a.C - col, nrow = a.R - row;  // how many of the 8 exist (may be <= 0)

    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const T* p = static_cast<const T*>(a.x) + (row + i) * a.ld_x + col;
        if (vec && ncol >= 8 && i < nrow) {
            uint4 raw[Raw8<T>::kWords];
#pragma unroll
            for (int k = 0; k < Raw8<T>::kWords; ++k) raw[k] = reinterpret_cast<const uint4*>(p)[k];
            const T* e = reinterpret_cast<const T*>(raw);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = widen(e[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = i < nrow && j < ncol ? widen(p[j]) : 0.f;
        }
    }

    // largest magnitude of each of the 8 rows, over its 16 lanes
    uint32_t rmax[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, magnitude_bits(v[i][j]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        rmax[i] = m;
    }

    if (a.block) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, rmax[i]);
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
        if (lane == 0) colmax[warp][0] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, colmax[i][0]);
#pragma unroll
        for (int i = 0; i < 8; ++i) rmax[i] = m;
        float inv;
        const float s = group_scale(m, a.e5m2, inv);
        if (threadIdx.x == 0) {
            if (a.s) a.s[tr * a.s_rs + tc * a.s_cs] = s;
            if (a.st) a.st[tc * a.st_rs + tr * a.st_cs] = s;
        }
    }
    if (a.q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float inv;
            const float s = group_scale(rmax[i], a.e5m2, inv);
            if (!a.block && cg == 0 && i < nrow) a.s[(row + i) * a.s_rs + tc * a.s_cs] = s;
            if (i < nrow) store8(a.q + (row + i) * a.ld_q + col, pack8(v[i], inv, a.e5m2), ncol, vec_q);
        }
    }
    if (!a.qt) return;

    float inv[8];
    if (a.block) {
        group_scale(rmax[0], a.e5m2, inv[0]);
#pragma unroll
        for (int j = 1; j < 8; ++j) inv[j] = inv[0];
    } else {
        // largest magnitude of each of the 8 columns: the thread's 8 rows, the
        // warp's two row groups, then the 8 warps
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, magnitude_bits(v[i][j]));
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
            if (lane < 16) colmax[warp][8 * cg + j] = m;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) m = max(m, colmax[k][8 * cg + j]);
            const float s = group_scale(m, a.e5m2, inv[j]);
            if (rg == 0 && j < ncol) a.st[(col + j) * a.st_rs + tr * a.st_cs] = s;
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = v[i][j];
        turned[8 * cg + j][rg ^ cg] = pack8(t, inv[j], a.e5m2);
    }
    __syncthreads();
    // rows of qt: 16 lanes a column, 8 bytes each
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int c = 16 * k + (threadIdx.x >> 4);
        const int u = threadIdx.x & 15;
        if (c0 + c < a.C)
            store8(a.qt + (c0 + c) * a.ld_qt + r0 + 8 * u, turned[c][u ^ (c >> 3)], a.R - (r0 + 8 * u), vec_qt);
    }
}

template <typename T>
cudaError_t run(const QuantArgs& a, cudaStream_t stream) {
    const int64_t tiles_r = (a.R + kGroup - 1) / kGroup, tiles_c = (a.C + kGroup - 1) / kGroup;
    if (tiles_r * tiles_c > INT32_MAX) return cudaErrorInvalidValue;
    auto rows_aligned = [](const void* p, int64_t ld_bytes, int n) {
        return reinterpret_cast<uintptr_t>(p) % n == 0 && ld_bytes % n == 0;
    };
    fp8_quantize_kernel<T><<<static_cast<unsigned>(tiles_r * tiles_c), kThreads, 0, stream>>>(
        a, tiles_c, rows_aligned(a.x, a.ld_x * static_cast<int64_t>(sizeof(T)), 16), rows_aligned(a.q, a.ld_q, 8),
        rows_aligned(a.qt, a.ld_qt, 8));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_quantize(const QuantArgs& a, vnm_dtype type, cudaStream_t stream) {
    switch (type) {
        case VNM_F16: return run<__half>(a, stream);
        case VNM_BF16: return run<__nv_bfloat16>(a, stream);
        default: return run<float>(a, stream);
    }
}

}  // namespace vnm

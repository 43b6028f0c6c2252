// The block-scaled 8-bit form of a matrix, plain and transposed, in one pass.
//
//   s = max(max |x| / F, 2^-100) over a group of 128 (or a 128 x 128 block),
//   q = fp8(x / s)
//
// Bound by memory traffic (2 or 4 bytes read, 1 or 2 written for an element)
// as long as the instructions for an element stay few. A CTA takes a 128 x 128
// tile, a thread 8 rows x 8 columns of it in registers, as they came (16-bit
// types stay packed in pairs, whose magnitudes compare as 16-bit integers): it
// holds 8 neighbours of every row (8 bytes of q) and 8 neighbours of every column
// (8 bytes of qt), so neither form passes through shared memory element by
// element. A row's maximum is reduced over its 16 lanes by halving (each step a
// lane keeps half of its rows), which leaves each lane one row's scale to work
// out; a column's goes through shared memory, one thread a column. The
// transposed bytes cross one 16 KB tile in shared memory, in 8-byte units whose
// index is XORed with the column group so that writing 16 columns and reading
// 16 rows both touch every bank once.
//
// Measured: 8192 x 4096 bf16 to both forms 31.4 us, 4.3 TB/s, 0.64 of a copy's rate;
// 11008 x 4096 fp16 in blocks 35.0 us, 5.2 TB/s, 0.76 (issue 66 and 60 % active). Widths
// that 8 does not divide go by single elements: 8192 x 4095 bf16 55 us.
#include <type_traits>

#include "vnm_dense.h"
#include "vnm_fp8.cuh"

namespace vnm {
namespace {

constexpr int kThreads = 256;

// A thread's 8 x 8 elements.
template <typename T>
struct Part {
    static constexpr bool kPacked = sizeof(T) == 2;
    static constexpr int kWords = kPacked ? 4 : 8;  // 32-bit words of 8 elements
    uint32_t w[8][kWords];

    // Rows of 16-byte words from `p`, `ld` elements apart: all loads before any use.
    __device__ __forceinline__ void load(const T* p, int64_t ld) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < kWords; k += 4)
                *reinterpret_cast<uint4*>(&w[i][k]) = *reinterpret_cast<const uint4*>(p + i * ld + k * (kPacked ? 2 : 1));
    }
    // Any alignment, nrow x ncol elements inside the matrix, 0 elsewhere.
    __device__ __forceinline__ void load_edge(const T* p, int64_t ld, int64_t nrow, int64_t ncol) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                if (kPacked) {
                    const uint32_t lo = i < nrow && 2 * k < ncol ? bits(p[i * ld + 2 * k]) : 0u;
                    const uint32_t hi = i < nrow && 2 * k + 1 < ncol ? bits(p[i * ld + 2 * k + 1]) : 0u;
                    w[i][k] = lo | (hi << 16);
                } else {
                    w[i][k] = i < nrow && k < ncol ? bits(p[i * ld + k]) : 0u;
                }
            }
    }
    static __device__ __forceinline__ uint32_t bits(float v) { return __float_as_uint(v); }
    static __device__ __forceinline__ uint32_t bits(__half v) { return __half_as_ushort(v); }
    static __device__ __forceinline__ uint32_t bits(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }

    __device__ __forceinline__ float get(int i, int j) const {
        if (!kPacked) return __uint_as_float(w[i][j]);
        return half_of(w[i][j / 2], j & 1);
    }
    static __device__ __forceinline__ float half_of(uint32_t word, int hi) {
        if (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(hi ? word & 0xFFFF0000u : word << 16);
        const __half2 h = *reinterpret_cast<const __half2*>(&word);
        return hi ? __high2float(h) : __low2float(h);
    }

    // Magnitudes as integers: of one element (fp32), or of a pair (16-bit types).
    static __device__ __forceinline__ uint32_t mag(uint32_t word) { return word & (kPacked ? 0x7FFF7FFFu : 0x7FFFFFFFu); }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return kPacked ? __vmaxu2(a, b) : max(a, b); }
    // fp32 magnitude bits of a word's larger element.
    static __device__ __forceinline__ uint32_t widened(uint32_t m) {
        if (!kPacked) return m;
        return magnitude_bits(half_of(max(m & 0xFFFFu, m >> 16), 0));
    }
};

__device__ __forceinline__ uint2 pack8(const float (&v)[8], bool e5m2) {
    return make_uint2(to_fp8x4(v[0], v[1], v[2], v[3], e5m2), to_fp8x4(v[4], v[5], v[6], v[7], e5m2));
}

// 8 bytes to p[0 .. 7], the first `n` of them.
__device__ __forceinline__ void store8(uint8_t* p, uint2 v, int64_t n, bool vec) {
    if (vec && n >= 8) {
        *reinterpret_cast<uint2*>(p) = v;
    } else {
#pragma unroll 1
        for (int i = 0; i < 8 && i < n; ++i) p[i] = static_cast<uint8_t>((i < 4 ? v.x : v.y) >> (8 * (i & 3)));
    }
}

// vec: rows of x are 16-byte aligned, vec_q / vec_qt: rows of q / qt 8-byte aligned.
template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2)
    fp8_quantize_kernel(const QuantArgs a, int64_t tiles_c, bool vec, bool vec_q, bool vec_qt) {
    using P = Part<T>;
    constexpr int kColWords = kGroup * P::kWords / 8;  // words of the tile's 128 columns
    __shared__ __align__(16) uint32_t colmax[8][kColWords];
    __shared__ __align__(16) float2 colscale[kGroup];  // a column's scale and its reciprocal
    __shared__ uint2 turned[kGroup][16];
    const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
    const int64_t r0 = tr * kGroup, c0 = tc * kGroup;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cg = threadIdx.x & 15;   // column group: columns 8 cg .. 8 cg + 7
    const int rg = threadIdx.x >> 4;   // row group: rows 8 rg .. 8 rg + 7
    const int64_t col = c0 + 8 * cg, row = r0 + 8 * rg;
    const int64_t ncol = a.C - col, nrow = a.R - row;  // how many of the 8 exist (may be <= 0)

    P x;
    const T* src = static_cast<const T*>(a.x) + row * a.ld_x + col;
    if (vec && ncol >= 8 && nrow >= 8)
        x.load(src, a.ld_x);
    else
        x.load_edge(src, a.ld_x, nrow, ncol);

    uint32_t rmax[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t m = P::mag(x.w[i][0]);
#pragma unroll
        for (int k = 1; k < P::kWords; ++k) m = P::larger(m, P::mag(x.w[i][k]));
        rmax[i] = m;
    }
    float rscale, rinv;  // of row lane & 7 of the lane's 8 rows (of the block: of all)
    if (a.block) {
        uint32_t m = rmax[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) m = P::larger(m, rmax[i]);
        m = __reduce_max_sync(0xFFFFFFFFu, P::widened(m));
        if (lane == 0) colmax[warp][0] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, colmax[i][0]);
        rscale = group_scale(m, a.e5m2, rinv);
        if (threadIdx.x == 0) {
            if (a.s) a.s[tr * a.s_rs + tc * a.s_cs] = rscale;
            if (a.st) a.st[tc * a.st_rs + tr * a.st_cs] = rscale;
        }
    } else {
        // rows 0..7 over lanes of the same half-warp: bits 2, 1, 0 of the lane number
        // choose the rows it keeps, bit 3 is reduced in full
        uint32_t h[4], u[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t keep = lane & 4 ? rmax[i + 4] : rmax[i], give = lane & 4 ? rmax[i] : rmax[i + 4];
            h[i] = P::larger(keep, __shfl_xor_sync(0xFFFFFFFFu, give, 4));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t keep = lane & 2 ? h[i + 2] : h[i], give = lane & 2 ? h[i] : h[i + 2];
            u[i] = P::larger(keep, __shfl_xor_sync(0xFFFFFFFFu, give, 2));
        }
        uint32_t m = P::larger(lane & 1 ? u[1] : u[0], __shfl_xor_sync(0xFFFFFFFFu, lane & 1 ? u[0] : u[1], 1));
        m = P::larger(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
        rscale = group_scale(P::widened(m), a.e5m2, rinv);
        if (a.s && !(lane & 8) && (lane & 7) < nrow) a.s[(row + (lane & 7)) * a.s_rs + tc * a.s_cs] = rscale;
    }
    if (a.q) {
        uint8_t* q = a.q + row * a.ld_q + col;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = a.block ? rscale : __shfl_sync(0xFFFFFFFFu, rscale, (lane & 16) | i);
            const float inv = a.block ? rinv : __shfl_sync(0xFFFFFFFFu, rinv, (lane & 16) | i);
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = quotient(x.get(i, j), s, inv);
            if (i < nrow) store8(q + i * a.ld_q, pack8(v, a.e5m2), ncol, vec_q);
        }
    }
    if (!a.qt) return;

    if (!a.block) {
        // columns: the thread's 8 rows, the warp's two row groups, then the 8 warps, a
        // thread a column
#pragma unroll
        for (int k = 0; k < P::kWords; k += 4) {
            uint32_t m[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                m[e] = P::mag(x.w[0][k + e]);
#pragma unroll
                for (int i = 1; i < 8; ++i) m[e] = P::larger(m[e], P::mag(x.w[i][k + e]));
                m[e] = P::larger(m[e], __shfl_xor_sync(0xFFFFFFFFu, m[e], 16));
            }
            if (lane < 16)
                *reinterpret_cast<uint4*>(&colmax[warp][cg * P::kWords + k]) = make_uint4(m[0], m[1], m[2], m[3]);
        }
        __syncthreads();
        if (threadIdx.x < kGroup) {
            const int c = threadIdx.x, word = P::kPacked ? c / 2 : c;
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) m = P::larger(m, colmax[k][word]);
            if (P::kPacked) m = c & 1 ? m >> 16 : m & 0xFFFFu;
            float ci;
            const float s = group_scale(P::widened(m), a.e5m2, ci);
            colscale[c] = make_float2(s, ci);
            if (c0 + c < a.C) a.st[(c0 + c) * a.st_rs + tr * a.st_cs] = s;
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        float4 c = make_float4(rscale, rinv, rscale, rinv);
        if (!a.block) c = *reinterpret_cast<const float4*>(&colscale[8 * cg + j]);
        float v[2][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[0][i] = quotient(x.get(i, j), c.x, c.y);
            v[1][i] = quotient(x.get(i, j + 1), c.z, c.w);
        }
        turned[8 * cg + j][rg ^ cg] = pack8(v[0], a.e5m2);
        turned[8 * cg + j + 1][rg ^ cg] = pack8(v[1], a.e5m2);
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

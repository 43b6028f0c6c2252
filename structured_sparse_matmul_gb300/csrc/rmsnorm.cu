// RMS norm with the residual's addition and an 8-bit output, and its backward
// pass.
//
//   h = x + residual, rstd = 1 / sqrt(mean h^2 + eps), y = h rstd w
//   q, s = block-scaled 8-bit form of y in groups of 128 columns
//   backward, g = dy w:  dh = dres + rstd (g - h rstd^2 mean(g h)),
//                        dw = sum over rows of dy h rstd
//
// Both are bound by memory traffic: a row is read once, kept in registers
// while its sum is formed, and written once. The unit of work is a warp on a
// group of 128 columns: 4 elements a lane, so that a group's largest magnitude
// is one warp reduction and its 8-bit values one 128-byte store, whatever the
// type. A row takes `warps` warps with CPT groups each; rows of one warp share
// a CTA of four. The row's sum crosses warps through shared memory in a fixed
// order, so results do not depend on timing.
#include "vnm_dense.h"
#include "vnm_fp8.cuh"

namespace vnm {
namespace {

constexpr int kMaxWarps = 32;
// Warps of a row that keeps `cpt` groups a warp in registers: 64 registers a
// thread hold two groups, 128 hold eight.
constexpr int max_warps(int cpt) { return cpt <= 2 ? kMaxWarps : 16; }
constexpr int min_ctas(int cpt) { return cpt == 4 ? 2 : 1; }
constexpr int grad_min_ctas(int) { return 1; }

// 4 elements of a lane as one vector access.
template <typename T>
struct Vec4;
template <>
struct Vec4<float> {
    using type = uint4;
};
template <>
struct Vec4<__half> {
    using type = uint2;
};
template <>
struct Vec4<__nv_bfloat16> {
    using type = uint2;
};

// Column of element j of a lane in group g: 4 neighbours for vector accesses,
// 32 apart for scalar ones (each access of the warp is then contiguous).
template <bool VEC>
__device__ __forceinline__ int64_t column(int64_t g, int lane, int j) {
    return g * kGroup + (VEC ? 4 * lane + j : lane + 32 * j);
}

// The lane's elements of group g of a row; columns from D on read as 0.
template <typename T, bool VEC>
__device__ __forceinline__ void load4(const T* row, int64_t g, int lane, int64_t D, T (&v)[4]) {
    if (VEC) {  // D % 4 == 0: the lane's 4 are inside or outside together
        typename Vec4<T>::type raw{};
        const int64_t c = column<VEC>(g, lane, 0);
        if (c < D) raw = *reinterpret_cast<const typename Vec4<T>::type*>(row + c);
        *reinterpret_cast<typename Vec4<T>::type*>(v) = raw;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t c = column<VEC>(g, lane, j);
            v[j] = c < D ? row[c] : narrow<T>(0.f);
        }
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store4(T* row, int64_t g, int lane, int64_t D, const T (&v)[4]) {
    if (VEC) {
        const int64_t c = column<VEC>(g, lane, 0);
        if (c < D) *reinterpret_cast<typename Vec4<T>::type*>(row + c) = *reinterpret_cast<const typename Vec4<T>::type*>(v);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t c = column<VEC>(g, lane, j);
            if (c < D) row[c] = v[j];
        }
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the `warps` warps of a row (a whole CTA; every thread calls it).
// `slot` alternates between calls so that one barrier a call is enough.
__device__ __forceinline__ float row_sum(float v, int warps, int warp, int lane, float (*buf)[kMaxWarps], int slot) {
    v = warp_sum(v);
    if (warps == 1) return v;
    if (lane == 0) buf[slot][warp] = v;
    __syncthreads();
    return warp_sum(lane < warps ? buf[slot][lane] : 0.f);
}

// One 8-bit group: the scale and the lane's 4 values.
template <bool VEC>
__device__ __forceinline__ void store_group(const RmsNormArgs& a, int64_t t, int64_t g, int lane, const float (&y)[4]) {
    uint32_t m = max(max(magnitude_bits(y[0]), magnitude_bits(y[1])), max(magnitude_bits(y[2]), magnitude_bits(y[3])));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    float inv;
    const float s = group_scale(m, a.e5m2, inv);
    if (lane == 0) a.s[t * a.s_rs + g * a.s_cs] = s;
    const uint32_t q = to_fp8x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv, a.e5m2);
    uint8_t* row = static_cast<uint8_t*>(a.q) + t * a.ld_q;
    if (VEC) {
        const int64_t c = column<VEC>(g, lane, 0);
        if (c < a.D) *reinterpret_cast<uint32_t*>(row + c) = q;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t c = column<VEC>(g, lane, j);
            if (c < a.D) row[c] = static_cast<uint8_t>(q >> (8 * j));
        }
    }
}

// Forward. A CTA takes the rows blockIdx.x, + gridDim.x, ... CPT > 0: the row's
// groups stay in registers, its weights too, and the next row's loads are issued
// before this row's sum is waited for. CPT = 0: rows longer than the registers
// hold; h is formed twice from the inputs (or read back where it was stored).
template <typename T, bool VEC, int CPT>
__global__ void __launch_bounds__(32 * max_warps(CPT), min_ctas(CPT)) rmsnorm_kernel(const RmsNormArgs a, int warps, int rows_per_cta) {
    __shared__ float buf[2][kMaxWarps];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int warp = warps == 1 ? 0 : wid;
    const int64_t groups = (a.D + kGroup - 1) / kGroup;
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows_per_cta;
    const T* w = static_cast<const T*>(a.w);
    constexpr int N = CPT > 0 ? CPT : 1;
    T xv[N][4], rv[N][4], hv[N][4], wv[N][4];
    auto load_row = [&](int64_t t) {
        const T* x = static_cast<const T*>(a.x) + t * a.ld_x;
#pragma unroll
        for (int i = 0; i < N; ++i) load4<T, VEC>(x, warp + static_cast<int64_t>(i) * warps, lane, a.D, xv[i]);
        if (a.res) {
            const T* r = static_cast<const T*>(a.res) + t * a.ld_res;
#pragma unroll
            for (int i = 0; i < N; ++i) load4<T, VEC>(r, warp + static_cast<int64_t>(i) * warps, lane, a.D, rv[i]);
        }
    };
    // h of the loaded elements
    auto add = [&](const T(&x4)[4], const T(&r4)[4], T(&h4)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) h4[j] = a.res ? narrow<T>(widen(x4[j]) + widen(r4[j])) : x4[j];
    };
    int slot = 0;
    int64_t t = static_cast<int64_t>(blockIdx.x) * rows_per_cta + (warps == 1 ? wid : 0);
    if (CPT > 0) {
        if (t < a.T) load_row(t);
        if (w) {
#pragma unroll
            for (int i = 0; i < N; ++i) load4<T, VEC>(w, warp + static_cast<int64_t>(i) * warps, lane, a.D, wv[i]);
        }
    }
    for (; t < a.T; t += step) {
        const T* x = static_cast<const T*>(a.x) + t * a.ld_x;
        const T* r = a.res ? static_cast<const T*>(a.res) + t * a.ld_res : nullptr;
        T* hrow = a.h ? static_cast<T*>(a.h) + t * a.ld_h : nullptr;
        float sum = 0.f;
        if (CPT > 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                add(xv[i], rv[i], hv[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) sum = fmaf(widen(hv[i][j]), widen(hv[i][j]), sum);
            }
            if (t + step < a.T) load_row(t + step);
            if (hrow) {
#pragma unroll
                for (int i = 0; i < N; ++i) store4<T, VEC>(hrow, warp + static_cast<int64_t>(i) * warps, lane, a.D, hv[i]);
            }
        } else {
            for (int64_t g = warp; g < groups; g += warps) {
                load4<T, VEC>(x, g, lane, a.D, xv[0]);
                if (r) load4<T, VEC>(r, g, lane, a.D, rv[0]);
                add(xv[0], rv[0], hv[0]);
                if (hrow) store4<T, VEC>(hrow, g, lane, a.D, hv[0]);
#pragma unroll
                for (int j = 0; j < 4; ++j) sum = fmaf(widen(hv[0][j]), widen(hv[0][j]), sum);
            }
        }
        sum = row_sum(sum, warps, warp, lane, buf, slot);
        slot ^= 1;
        const float rstd = 1.f / sqrtf(sum / static_cast<float>(a.D) + a.eps);
        if (a.rstd && warp == 0 && lane == 0) a.rstd[t] = rstd;
        T* yrow = a.y ? static_cast<T*>(a.y) + t * a.ld_y : nullptr;
        auto out_group = [&](int64_t g, const T(&h4)[4], const T(&w4)[4]) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = widen(h4[j]) * rstd * (w ? widen(w4[j]) : 1.f);
            if (a.q) store_group<VEC>(a, t, g, lane, y);
            if (yrow) {
                T yv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) yv[j] = narrow<T>(y[j]);
                store4<T, VEC>(yrow, g, lane, a.D, yv);
            }
        };
        if (CPT > 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int64_t g = warp + static_cast<int64_t>(i) * warps;
                if (g < groups) out_group(g, hv[i], wv[i]);  // the same for the whole warp
            }
        } else {
            for (int64_t g = warp; g < groups; g += warps) {
                // the lane reads back what it wrote itself, or forms h again
                if (hrow) {
                    load4<T, VEC>(hrow, g, lane, a.D, hv[0]);
                } else {
                    load4<T, VEC>(x, g, lane, a.D, xv[0]);
                    if (r) load4<T, VEC>(r, g, lane, a.D, rv[0]);
                    add(xv[0], rv[0], hv[0]);
                }
                if (w) load4<T, VEC>(w, g, lane, a.D, wv[0]);
                out_group(g, hv[0], wv[0]);
            }
        }
    }
}

// Backward. A CTA takes the rows t = blockIdx.x, + gridDim.x, ...; a thread owns
// the same columns in all of them, so its share of dweight stays in registers
// and is written once, to the CTA's row of `partial`. The next row's loads are
// issued before this row's sum is waited for. CPT = 0: no dweight here (long
// rows, see rmsnorm_dw_kernel), dy and h read twice.
template <typename T, bool VEC, int CPT>
__global__ void __launch_bounds__(32 * max_warps(CPT), grad_min_ctas(CPT)) rmsnorm_grad_kernel(const RmsNormGradArgs a, int warps, bool with_dw) {
    __shared__ float buf[2][kMaxWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t groups = (a.D + kGroup - 1) / kGroup;
    const T* w = static_cast<const T*>(a.w);
    constexpr int N = CPT > 0 ? CPT : 1;
    float acc[N][4];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    T dyv[N][4], hv[N][4], rv[N][4], wv[N][4];
    float rstd_next = 0.f;
    auto load_row = [&](int64_t t) {
        const T* dy = static_cast<const T*>(a.dy) + t * a.ld_dy;
        const T* h = static_cast<const T*>(a.h) + t * a.ld_h;
        rstd_next = a.rstd[t];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            load4<T, VEC>(dy, warp + static_cast<int64_t>(i) * warps, lane, a.D, dyv[i]);
            load4<T, VEC>(h, warp + static_cast<int64_t>(i) * warps, lane, a.D, hv[i]);
        }
    };
    int64_t t = blockIdx.x;
    if (CPT > 0) {
        if (t < a.T) load_row(t);
        if (w) {
#pragma unroll
            for (int i = 0; i < N; ++i) load4<T, VEC>(w, warp + static_cast<int64_t>(i) * warps, lane, a.D, wv[i]);
        }
    }
    int slot = 0;
    for (; t < a.T; t += gridDim.x) {
        const T* dy = static_cast<const T*>(a.dy) + t * a.ld_dy;
        const T* h = static_cast<const T*>(a.h) + t * a.ld_h;
        const T* dr = a.dres && a.dh ? static_cast<const T*>(a.dres) + t * a.ld_dres : nullptr;
        T* dh = a.dh ? static_cast<T*>(a.dh) + t * a.ld_dh : nullptr;
        const float rstd = CPT > 0 ? rstd_next : a.rstd[t];
        float g[N][4], hf[N][4];  // dy w and h of the row
        float dot = 0.f;
        auto take = [&](const T(&d4)[4], const T(&h4)[4], const T(&w4)[4], float(&g4)[4], float(&f4)[4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                g4[j] = widen(d4[j]) * (w ? widen(w4[j]) : 1.f);
                f4[j] = widen(h4[j]);
                dot = fmaf(g4[j], f4[j], dot);
            }
        };
        if (CPT > 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                take(dyv[i], hv[i], wv[i], g[i], hf[i]);
                if (with_dw) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(widen(dyv[i][j]), hf[i][j] * rstd, acc[i][j]);
                }
            }
            if (dr) {
#pragma unroll
                for (int i = 0; i < N; ++i) load4<T, VEC>(dr, warp + static_cast<int64_t>(i) * warps, lane, a.D, rv[i]);
            }
            if (t + gridDim.x < a.T) load_row(t + gridDim.x);
        } else {
            for (int64_t k = warp; k < groups; k += warps) {
                load4<T, VEC>(dy, k, lane, a.D, dyv[0]);
                load4<T, VEC>(h, k, lane, a.D, hv[0]);
                if (w) load4<T, VEC>(w, k, lane, a.D, wv[0]);
                take(dyv[0], hv[0], wv[0], g[0], hf[0]);
            }
        }
        if (!dh) continue;  // dweight alone needs no row sum
        dot = row_sum(dot, warps, warp, lane, buf, slot);
        slot ^= 1;
        const float c = rstd * rstd * (dot / static_cast<float>(a.D));
        auto out_group = [&](int64_t k, const float(&g4)[4], const float(&f4)[4], const T(&r4)[4]) {
            T ov[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float v = rstd * (g4[j] - f4[j] * c);
                ov[j] = narrow<T>(dr ? v + widen(r4[j]) : v);
            }
            store4<T, VEC>(dh, k, lane, a.D, ov);
        };
        if (CPT > 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int64_t k = warp + static_cast<int64_t>(i) * warps;
                if (k < groups) out_group(k, g[i], hf[i], rv[i]);
            }
        } else {
            for (int64_t k = warp; k < groups; k += warps) {
                load4<T, VEC>(dy, k, lane, a.D, dyv[0]);
                load4<T, VEC>(h, k, lane, a.D, hv[0]);
                if (w) load4<T, VEC>(w, k, lane, a.D, wv[0]);
                if (dr) load4<T, VEC>(dr, k, lane, a.D, rv[0]);
                take(dyv[0], hv[0], wv[0], g[0], hf[0]);
                out_group(k, g[0], hf[0], rv[0]);
            }
        }
    }
    if (CPT > 0 && with_dw) {
        float* part = a.partial + static_cast<int64_t>(blockIdx.x) * a.D;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t c = column<VEC>(warp + static_cast<int64_t>(i) * warps, lane, j);
                if (c < a.D) part[c] = acc[i][j];
            }
    }
}

// dweight of long rows: a thread a column, the rows dealt to gridDim.y parts.
template <typename T>
__global__ void rmsnorm_dw_kernel(const RmsNormGradArgs a) {
    const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (c >= a.D) return;
    float acc = 0.f;
    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y)
        acc = fmaf(widen(static_cast<const T*>(a.dy)[t * a.ld_dy + c]),
                   widen(static_cast<const T*>(a.h)[t * a.ld_h + c]) * a.rstd[t], acc);
    a.partial[static_cast<int64_t>(blockIdx.y) * a.D + c] = acc;
}

// dw[c] = sum over the parts, in order within each of 8 slices, then the slices.
__global__ void rmsnorm_dw_reduce_kernel(const float* partial, int64_t parts, int64_t D, float* dw) {
    __shared__ float sum[8][33];
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    float v = 0.f;
    if (c < D)
        for (int64_t p = threadIdx.y; p < parts; p += 8) v += partial[p * D + c];
    sum[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += sum[i][threadIdx.x];
        dw[c] = v;
    }
}

bool vec_ok(const void* p, int64_t ld, int elem) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % (4 * elem) == 0 && ld % 4 == 0);
}

// Groups a warp keeps in registers, for a row of `groups` groups: the fewest that
// cover it (0: none does, the row is read twice). With enough rows to fill the
// GPU, fewer and busier warps a row.
int groups_per_warp(int64_t groups, bool many_rows) {
    int c = 1;
    while (c <= 8 && groups > static_cast<int64_t>(c) * max_warps(c)) c *= 2;
    if (c > 8) return 0;
    while (many_rows && c < 4 && groups > c) c *= 2;
    return c;
}

template <typename T, bool VEC>
cudaError_t run_forward(const RmsNormArgs& a, int sm_count, cudaStream_t stream) {
    const int64_t groups = (a.D + kGroup - 1) / kGroup;
    const int cpt = groups_per_warp(groups, a.T > 2 * sm_count);
    const int warps = cpt == 0 ? kMaxWarps : static_cast<int>((groups + cpt - 1) / cpt);
    const int rows_per_cta = warps == 1 ? 4 : 1;
    const int threads = warps == 1 ? 128 : 32 * warps;
    const int64_t ctas = (a.T + rows_per_cta - 1) / rows_per_cta;
    // persistent: as many CTAs as fit the SMs at 64 registers a thread
    const int64_t fit = static_cast<int64_t>(sm_count) * (1024 / threads > 0 ? 1024 / threads : 1);
    const unsigned grid = static_cast<unsigned>(ctas < fit ? ctas : fit);
    switch (cpt) {
        case 0: rmsnorm_kernel<T, VEC, 0><<<grid, threads, 0, stream>>>(a, warps, rows_per_cta); break;
        case 1: rmsnorm_kernel<T, VEC, 1><<<grid, threads, 0, stream>>>(a, warps, rows_per_cta); break;
        case 2: rmsnorm_kernel<T, VEC, 2><<<grid, threads, 0, stream>>>(a, warps, rows_per_cta); break;
        case 4: rmsnorm_kernel<T, VEC, 4><<<grid, threads, 0, stream>>>(a, warps, rows_per_cta); break;
        default: rmsnorm_kernel<T, VEC, 8><<<grid, threads, 0, stream>>>(a, warps, rows_per_cta); break;
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t forward_of(const RmsNormArgs& a, int sm_count, cudaStream_t stream) {
    const int e = sizeof(T);
    const bool vec = a.D % 4 == 0 && vec_ok(a.x, a.ld_x, e) && vec_ok(a.res, a.ld_res, e) && vec_ok(a.w, 0, e) &&
                     vec_ok(a.h, a.ld_h, e) && vec_ok(a.y, a.ld_y, e) && vec_ok(a.q, a.ld_q, 1);
    return vec ? run_forward<T, true>(a, sm_count, stream) : run_forward<T, false>(a, sm_count, stream);
}

constexpr int64_t kGradParts = 304;  // two CTAs for each of 152 SMs

template <typename T, bool VEC>
cudaError_t run_grad(const RmsNormGradArgs& a, cudaStream_t stream) {
    const int64_t groups = (a.D + kGroup - 1) / kGroup;
    const int cpt = groups_per_warp(groups, a.T > kGradParts);
    const int warps = cpt == 0 ? kMaxWarps : static_cast<int>((groups + cpt - 1) / cpt);
    const int64_t parts = rmsnorm_grad_parts(a.T, a.D);
    const bool dw = a.dw != nullptr;
    if (a.T > 0) {
        const unsigned grid = static_cast<unsigned>(parts);
        if (dw && cpt == 0) {  // before dh is written: dh may be dy
            const dim3 g2(static_cast<unsigned>((a.D + 127) / 128), static_cast<unsigned>(parts));
            rmsnorm_dw_kernel<T><<<g2, 128, 0, stream>>>(a);
            const cudaError_t e = cudaGetLastError();
            if (e != cudaSuccess) return e;
        }
        switch (cpt) {
            case 0: rmsnorm_grad_kernel<T, VEC, 0><<<grid, 32 * warps, 0, stream>>>(a, warps, false); break;
            case 1: rmsnorm_grad_kernel<T, VEC, 1><<<grid, 32 * warps, 0, stream>>>(a, warps, dw); break;
            case 2: rmsnorm_grad_kernel<T, VEC, 2><<<grid, 32 * warps, 0, stream>>>(a, warps, dw); break;
            case 4: rmsnorm_grad_kernel<T, VEC, 4><<<grid, 32 * warps, 0, stream>>>(a, warps, dw); break;
            default: rmsnorm_grad_kernel<T, VEC, 8><<<grid, 32 * warps, 0, stream>>>(a, warps, dw); break;
        }
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (dw) {
        rmsnorm_dw_reduce_kernel<<<static_cast<unsigned>((a.D + 31) / 32), dim3(32, 8), 0, stream>>>(
            a.partial, a.T > 0 ? parts : 0, a.D, a.dw);
        return cudaGetLastError();
    }
    return cudaSuccess;
}

template <typename T>
cudaError_t grad_of(const RmsNormGradArgs& a, cudaStream_t stream) {
    const int e = sizeof(T);
    const bool vec = a.D % 4 == 0 && vec_ok(a.dy, a.ld_dy, e) && vec_ok(a.h, a.ld_h, e) && vec_ok(a.w, 0, e) &&
                     vec_ok(a.dres, a.ld_dres, e) && vec_ok(a.dh, a.ld_dh, e);
    return vec ? run_grad<T, true>(a, stream) : run_grad<T, false>(a, stream);
}

}  // namespace

cudaError_t launch_rmsnorm(const RmsNormArgs& a, vnm_dtype type, int sm_count, cudaStream_t stream) {
    switch (type) {
        case VNM_F16: return forward_of<__half>(a, sm_count, stream);
        case VNM_BF16: return forward_of<__nv_bfloat16>(a, sm_count, stream);
        default: return forward_of<float>(a, sm_count, stream);
    }
}

int64_t rmsnorm_grad_parts(int64_t T, int64_t) { return T < kGradParts ? T : kGradParts; }

cudaError_t launch_rmsnorm_grad(const RmsNormGradArgs& a, vnm_dtype type, cudaStream_t stream) {
    switch (type) {
        case VNM_F16: return grad_of<__half>(a, stream);
        case VNM_BF16: return grad_of<__nv_bfloat16>(a, stream);
        default: return grad_of<float>(a, stream);
    }
}

}  // namespace vnm

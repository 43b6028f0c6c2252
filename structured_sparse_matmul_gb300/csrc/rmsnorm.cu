// RMS norm with the residual's addition and an 8-bit output, and its backward
// pass.
//
//   h = x + residual, rstd = 1 / sqrt(mean h^2 + eps), y = h rstd w
//   q, s = block-scaled 8-bit form of y in groups of 128 columns
//   backward, g = dy w:  dh = dres + rstd (g - h rstd^2 mean(g h)),
//                        dw = sum over rows of dy h rstd
//
// Both are bound by memory traffic: a row is read once, kept in registers
// while its sum is formed, and written once. The unit of work is a warp on two
// groups of 128 columns, 8 elements a lane (16 bytes of a 16-bit type), so that a
// group's largest magnitude is a reduction over half a warp whatever the type,
// and the scale's arithmetic is shared by 8 elements. A CTA takes a row at a time,
// its warps CPT units each. CTAs are persistent, keep their weights, and load the
// next row before they wait for this one's sum.
// The sum crosses warps through shared memory in a fixed order, so results do not
// depend on timing.
//
// Measured: forward 8192 x 4096 bf16 with residual and 8-bit output 45.5 us, 5.2 TB/s,
// 0.76 of a copy's rate; what is left is instruction issue (72 % active, 39 for an
// element). Backward 8192 x 4096 bf16 52.1 us, 5.2 TB/s, 0.76 (53 % issue active, loads
// of one row ahead in flight). One row of 4096: 2.5 us, the launch and one round trip.
#include <algorithm>
#include <type_traits>

#include "vnm_dense.h"
#include "vnm_fp8.cuh"

namespace vnm {
namespace {

constexpr int kMaxWarps = 32;
constexpr int kUnit = 2 * kGroup;  // columns of a warp's unit of work
// Warps of a row that keeps `cpt` units a warp in registers: 64 registers a
// thread hold one, 128 hold two or four.
constexpr int max_warps(int cpt) { return cpt <= 1 ? kMaxWarps : 16; }

// A lane's elements of a unit: 8 neighbours for vector accesses, 16 apart for
// scalar ones (each access of a half-warp is then contiguous). first_column is the
// lane's first; element j is at first_column + j * kStep.
template <bool VEC>
constexpr int kStep = VEC ? 1 : 16;
template <bool VEC>
__device__ __forceinline__ int64_t first_column(int64_t u, int lane) {
    return u * kUnit + (lane >> 4) * kGroup + (lane & 15) * (VEC ? 8 : 1);
}

// A lane's 8 elements of a unit, as they came.
template <typename T>
struct alignas(16) Elems {
    T v[8];
};

// The lane's elements of a row, `left` = D less the lane's first column: past the
// row's end they read as 0. p: the row's element at that column.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int64_t left, Elems<T>& e) {
    if (VEC) {  // D % 8 == 0: the lane's 8 are inside or outside together
        uint4* raw = reinterpret_cast<uint4*>(&e);
#pragma unroll
        for (int k = 0; k < static_cast<int>(sizeof(T)) / 2; ++k)
            raw[k] = left > 0 ? reinterpret_cast<const uint4*>(p)[k] : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) e.v[j] = left > j * kStep<VEC> ? p[j * kStep<VEC>] : narrow<T>(0.f);
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int64_t left, const Elems<T>& e) {
    if (VEC) {
        const uint4* raw = reinterpret_cast<const uint4*>(&e);
        if (left > 0) {
#pragma unroll
            for (int k = 0; k < static_cast<int>(sizeof(T)) / 2; ++k) reinterpret_cast<uint4*>(p)[k] = raw[k];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (left > j * kStep<VEC>) p[j * kStep<VEC>] = e.v[j];
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

// 1 / sqrt(v) to fp32 accuracy: the approximation and one Newton step.
__device__ __forceinline__ float inverse_root(float v) {
    const float r = rsqrtf(v);
    const float e = fmaf(-v * r, r, 1.f);
    const float n = fmaf(0.5f * r, e, r);
    return isfinite(n) ? n : r;  // v = 0, Inf, or too small or large for the step
}

// The unit's two 8-bit groups: the scale of the half-warp's, and the lane's 8
// values. q: the row's byte at the lane's first column, s: the group's scale.
template <bool VEC>
__device__ __forceinline__ void store_groups(const float (&y)[8], bool e5m2, uint8_t* q, float* s, int64_t left, int lane) {
    float m = max_magnitude(y[0], y[1]);
#pragma unroll
    for (int j = 2; j < 8; ++j) m = max_magnitude(m, y[j]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max_magnitude(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    float inv;
    const float scale = group_scale(m, e5m2, inv);
    if ((lane & 15) == 0 && left > 0) *s = scale;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = quotient(y[j], scale, inv);
    const uint32_t lo = to_fp8x4(v[0], v[1], v[2], v[3], e5m2);
    const uint32_t hi = to_fp8x4(v[4], v[5], v[6], v[7], e5m2);
    if (VEC) {
        if (left > 0) *reinterpret_cast<uint2*>(q) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (left > j * kStep<VEC>) q[j * kStep<VEC>] = static_cast<uint8_t>((j < 4 ? lo : hi) >> (8 * (j & 3)));
    }
}

// Forward. A CTA takes the rows t = blockIdx.x, + gridDim.x, ... CPT > 0: the row's
// units stay in registers. CPT = 0: rows longer than the registers hold; h is
// formed twice from the inputs (or read back where it was stored).
template <typename T, bool VEC, int CPT>
__global__ void __launch_bounds__(32 * max_warps(CPT), 1) rmsnorm_kernel(const __grid_constant__ RmsNormArgs a) {
    using Off = std::conditional_t<(CPT > 0), int, int64_t>;  // columns: rows in registers are short
    __shared__ float buf[2][kMaxWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    constexpr int N = CPT > 0 ? CPT : 1;
    const Off D = static_cast<Off>(a.D);
    const Off c0 = static_cast<Off>(first_column<VEC>(warp, lane));  // of the lane's first unit
    const Off across = static_cast<Off>(warps) * kUnit;              // to the warp's next unit
    const Off own = (D + across - 1 - warp * kUnit) / across;        // units of this warp
    const T* w = static_cast<const T*>(a.w);
    const float inv_d = 1.f / static_cast<float>(a.D);

    Elems<T> x8[N], r8[N];
    float hf[N][8], wf[N][8];
    // (a row's address is the same for the whole CTA: only columns are a lane's own)
    auto load_row = [&](int64_t t) {
        const T* x = static_cast<const T*>(a.x) + t * a.ld_x;
#pragma unroll
        for (int i = 0; i < N; ++i) load8<T, VEC>(x + (c0 + i * across), D - c0 - i * across, x8[i]);
        if (a.res) {
            const T* r = static_cast<const T*>(a.res) + t * a.ld_res;
#pragma unroll
            for (int i = 0; i < N; ++i) load8<T, VEC>(r + (c0 + i * across), D - c0 - i * across, r8[i]);
        }
    };
    auto load_weight = [&](Off c, float(&f)[8]) {
        Elems<T> e;
        if (w) load8<T, VEC>(w + c, D - c, e);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = w ? widen(e.v[j]) : 1.f;
    };
    float sum = 0.f;
    // h of the loaded elements as it is stored, widened, and its squares
    auto add = [&](const Elems<T>& xe, const Elems<T>& re, float(&f)[8], T* h, Off c) {
        if (a.res) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = widen(xe.v[j]) + widen(re.v[j]);
            Elems<T> he;
            narrow8(f, he.v);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = widen(he.v[j]);
            if (h) store8<T, VEC>(h + c, D - c, he);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = widen(xe.v[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
    };
    auto out_unit = [&](int64_t t, Off u, float rstd, const float(&f)[8], const float(&wt)[8]) {
        const Off c = c0 + u * across;
        float yf[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) yf[j] = f[j] * rstd * wt[j];
        if (a.q)
            store_groups<VEC>(yf, a.e5m2, static_cast<uint8_t*>(a.q) + t * a.ld_q + c,
                              a.s + t * a.s_rs + (c / kGroup) * a.s_cs, D - c, lane);
        if (a.y) {
            Elems<T> ye;
            narrow8(yf, ye.v);
            store8<T, VEC>(static_cast<T*>(a.y) + t * a.ld_y + c, D - c, ye);
        }
    };
    if (CPT > 0) {
        load_row(blockIdx.x);
#pragma unroll
        for (int i = 0; i < N; ++i) load_weight(c0 + i * across, wf[i]);
    }
    int slot = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        T* h = a.h ? static_cast<T*>(a.h) + t * a.ld_h : nullptr;
        sum = 0.f;
        if (CPT > 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) add(x8[i], r8[i], hf[i], h, c0 + i * across);
            if (t + gridDim.x < a.T) load_row(t + gridDim.x);
        } else {
            const T* x = static_cast<const T*>(a.x) + t * a.ld_x;
            const T* r = a.res ? static_cast<const T*>(a.res) + t * a.ld_res : nullptr;
            for (Off u = 0; u < own; ++u) {
                const Off c = c0 + u * across;
                load8<T, VEC>(x + c, D - c, x8[0]);
                if (r) load8<T, VEC>(r + c, D - c, r8[0]);
                add(x8[0], r8[0], hf[0], h, c);
            }
        }
        const float total = row_sum(sum, warps, warp, lane, buf, slot);
        slot ^= 1;
        const float rstd = inverse_root(fmaf(total, inv_d, a.eps));
        if (a.rstd && threadIdx.x == 0) a.rstd[t] = rstd;
        if (CPT > 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < own) out_unit(t, i, rstd, hf[i], wf[i]);  // the same for the whole warp
        } else {
            const T* x = static_cast<const T*>(a.x) + t * a.ld_x;
            const T* r = a.res ? static_cast<const T*>(a.res) + t * a.ld_res : nullptr;
            for (Off u = 0; u < own; ++u) {
                const Off c = c0 + u * across;
                // the lane reads back what it wrote itself, or forms h again
                load8<T, VEC>((h ? h : x) + c, D - c, x8[0]);
                if (r && !h) {
                    load8<T, VEC>(r + c, D - c, r8[0]);
                    add(x8[0], r8[0], hf[0], nullptr, c);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) hf[0][j] = widen(x8[0].v[j]);
                }
                load_weight(c, wf[0]);
                out_unit(t, u, rstd, hf[0], wf[0]);
            }
        }
    }
}

// Backward. A CTA takes the rows t = blockIdx.x, + gridDim.x, ...; a thread owns
// the same columns in all of them, so its share of dweight stays in registers
// and is written once, to the CTA's row of `partial`. CPT = 0: no dweight here
// (long rows, see rmsnorm_dw_kernel; launched for dh only), dy and h read twice.
template <typename T, bool VEC, int CPT>
__global__ void __launch_bounds__(32 * max_warps(CPT), 1)
    rmsnorm_grad_kernel(const __grid_constant__ RmsNormGradArgs a, bool with_dw) {
    using Off = std::conditional_t<(CPT > 0), int, int64_t>;
    __shared__ float buf[2][kMaxWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    constexpr int N = CPT > 0 ? CPT : 1;
    // The next row's loads are in flight (four units leave no registers for it) and a
    // row's elements stay in registers until dh. Four units of a 32-bit type, or by
    // scalar accesses, read dy and h again from the caches instead of spilling (2048 x
    // 16383 bf16: 123 us, 148 with them kept; 2048 x 8704 fp16, vectors: 73.6, kept 48.1).
    constexpr bool kAhead = CPT == 1 || CPT == 2, kKeep = kAhead || (CPT == 4 && VEC && sizeof(T) == 2);
    constexpr int M = kKeep ? N : 1;
    const Off D = static_cast<Off>(a.D);
    const Off c0 = static_cast<Off>(first_column<VEC>(warp, lane));
    const Off across = static_cast<Off>(warps) * kUnit;
    const Off own = (D + across - 1 - warp * kUnit) / across;  // units of this warp
    const T* w = static_cast<const T*>(a.w);
    const float inv_d = 1.f / static_cast<float>(a.D);
    float acc[N][8];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    Elems<T> dn[kAhead ? N : 1], hn[kAhead ? N : 1], d8[M], h8[M], r8[M], w8[M];  // dn, hn: the next row's dy and h
    float rstd_next = 0.f;
    auto load_row = [&](int64_t t, Elems<T>* de, Elems<T>* he) {
        const T* dy = static_cast<const T*>(a.dy) + t * a.ld_dy;
        const T* h = static_cast<const T*>(a.h) + t * a.ld_h;
        rstd_next = a.rstd[t];
#pragma unroll
        for (int i = 0; i < M; ++i) {
            load8<T, VEC>(dy + (c0 + i * across), D - c0 - i * across, de[i]);
            load8<T, VEC>(h + (c0 + i * across), D - c0 - i * across, he[i]);
        }
    };
    auto load_unit = [&](int64_t t, Off c) {
        load8<T, VEC>(static_cast<const T*>(a.dy) + t * a.ld_dy + c, D - c, d8[0]);
        load8<T, VEC>(static_cast<const T*>(a.h) + t * a.ld_h + c, D - c, h8[0]);
        if (w) load8<T, VEC>(w + c, D - c, w8[0]);
    };
    if (CPT > 0) {
        if (kAhead) load_row(blockIdx.x, dn, hn);
        if (kKeep && w) {
#pragma unroll
            for (int i = 0; i < M; ++i) load8<T, VEC>(w + (c0 + i * across), D - c0 - i * across, w8[i]);
        }
    }
    // dy w
    auto scaled = [&](const Elems<T>& de, const Elems<T>& we, int j) {
        return widen(de.v[j]) * (w ? widen(we.v[j]) : 1.f);
    };
    const bool add_res = a.dres && a.dh;
    float rstd = 0.f, k = 0.f;  // k = rstd^2 mean(g h)
    auto out_unit = [&](T* dh, Off c, const Elems<T>& de, const Elems<T>& he, const Elems<T>& we, const Elems<T>& re) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = fmaf(-widen(he.v[j]), k, scaled(de, we, j));
            f[j] = add_res ? fmaf(rstd, v, widen(re.v[j])) : rstd * v;
        }
        Elems<T> oe;
        narrow8(f, oe.v);
        store8<T, VEC>(dh + c, D - c, oe);
    };
    int slot = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const T* dr = static_cast<const T*>(a.dres) + (add_res ? t * a.ld_dres : 0);
        T* dh = static_cast<T*>(a.dh) + (a.dh ? t * a.ld_dh : 0);
        float dot = 0.f;
        if (CPT > 0) {
            if (kKeep && add_res) {
#pragma unroll
                for (int i = 0; i < M; ++i) load8<T, VEC>(dr + (c0 + i * across), D - c0 - i * across, r8[i]);
            }
            if (kAhead) {
                rstd = rstd_next;
#pragma unroll
                for (int i = 0; i < (kAhead ? N : 1); ++i) {
                    d8[i] = dn[i];
                    h8[i] = hn[i];
                }
                if (t + gridDim.x < a.T) load_row(t + gridDim.x, dn, hn);
            } else {
                if (kKeep) load_row(t, d8, h8);
                rstd = a.rstd[t];
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int m = kKeep ? i : 0;
                if (!kKeep) load_unit(t, c0 + i * across);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float hj = widen(h8[m].v[j]);
                    dot = fmaf(scaled(d8[m], w8[m], j), hj, dot);
                    acc[i][j] = fmaf(widen(d8[m].v[j]), hj * rstd, acc[i][j]);
                }
            }
        } else {
            const T* dy = static_cast<const T*>(a.dy) + t * a.ld_dy;
            const T* h = static_cast<const T*>(a.h) + t * a.ld_h;
            rstd = a.rstd[t];
            for (Off u = 0; u < own; ++u) {
                const Off c = c0 + u * across;
                load8<T, VEC>(dy + c, D - c, d8[0]);
                load8<T, VEC>(h + c, D - c, h8[0]);
                if (w) load8<T, VEC>(w + c, D - c, w8[0]);
#pragma unroll
                for (int j = 0; j < 8; ++j) dot = fmaf(scaled(d8[0], w8[0], j), widen(h8[0].v[j]), dot);
            }
        }
        if (!a.dh) continue;  // dweight alone needs no row sum
        const float total = row_sum(dot, warps, warp, lane, buf, slot);
        slot ^= 1;
        k = rstd * rstd * (total * inv_d);
        if (CPT > 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int m = kKeep ? i : 0;
                if (i >= own) continue;  // the same for the whole warp
                if (!kKeep) {
                    load_unit(t, c0 + i * across);
                    if (add_res) load8<T, VEC>(dr + (c0 + i * across), D - c0 - i * across, r8[0]);
                }
                out_unit(dh, c0 + i * across, d8[m], h8[m], w8[m], r8[m]);
            }
        } else {
            const T* dy = static_cast<const T*>(a.dy) + t * a.ld_dy;
            const T* h = static_cast<const T*>(a.h) + t * a.ld_h;
            for (Off u = 0; u < own; ++u) {
                const Off c = c0 + u * across;
                load8<T, VEC>(dy + c, D - c, d8[0]);
                load8<T, VEC>(h + c, D - c, h8[0]);
                if (w) load8<T, VEC>(w + c, D - c, w8[0]);
                if (add_res) load8<T, VEC>(dr + c, D - c, r8[0]);
                out_unit(dh, c, d8[0], h8[0], w8[0], r8[0]);
            }
        }
    }
    if (CPT > 0 && with_dw) {
        float* part = a.partial + static_cast<int64_t>(blockIdx.x) * a.D + c0;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (D - c0 - i * across > j * kStep<VEC>) part[i * across + j * kStep<VEC>] = acc[i][j];
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

// dw[c] = sum over the parts: in order within each of 32 slices, then the slices.
__global__ void __launch_bounds__(1024) rmsnorm_dw_reduce_kernel(const float* partial, int64_t parts, int64_t D, float* dw) {
    __shared__ float sum[32][33];
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    float v = 0.f;
    if (c < D) {
#pragma unroll 4
        for (int64_t p = threadIdx.y; p < parts; p += 32) v += partial[p * D + c];
    }
    sum[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 32; ++i) v += sum[i][threadIdx.x];
        dw[c] = v;
    }
}

// Rows of 8 elements on 8 * elem bytes (16 at most).
bool vec_ok(const void* p, int64_t ld, int elem) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % (elem == 1 ? 8 : 16) == 0 && ld % 8 == 0);
}

// Units a warp keeps in registers for a row of `units` (0: too many, the row is
// read twice), and the row's warps. Forward (pair = false): one unit a warp as long
// as 32 warps reach (8192 x 4096 with 8-bit output, by a product with the reciprocal in place
// of the quotient: 42.9 us; two units a warp 54.4).
// Backward: two units where there are rows enough to fill the GPU, so that the sum
// across warps and the row's scalars are shared by 16 elements a lane (8192 x 4096:
// 51.3 us; one unit 56.2).
int units_per_warp(int64_t units, bool pair, int& warps) {
    const int cpt = pair && units >= 4 && units <= 2 * max_warps(2) ? 2
                    : units <= max_warps(1)                        ? 1
                    : units <= 4 * max_warps(4)                    ? 4
                                                                   : 0;
    warps = cpt == 0 ? kMaxWarps : static_cast<int>((units + cpt - 1) / cpt);
    return cpt;
}

template <typename T, bool VEC>
cudaError_t run_forward(const RmsNormArgs& a, int sm_count, cudaStream_t stream) {
    int warps;
    const int cpt = units_per_warp((a.D + kUnit - 1) / kUnit, false, warps);
    const int threads = 32 * warps;
    // persistent: the CTAs that fit at 64 (one unit) or 128 registers a thread
    const int64_t fit = static_cast<int64_t>(sm_count) * std::max(1, std::min(32, (cpt == 1 ? 1024 : 512) / threads));
    const unsigned grid = static_cast<unsigned>(std::min(a.T, fit));
    switch (cpt) {
        case 0: rmsnorm_kernel<T, VEC, 0><<<grid, threads, 0, stream>>>(a); break;
        case 1: rmsnorm_kernel<T, VEC, 1><<<grid, threads, 0, stream>>>(a); break;
        default: rmsnorm_kernel<T, VEC, 4><<<grid, threads, 0, stream>>>(a); break;
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t forward_of(const RmsNormArgs& a, int sm_count, cudaStream_t stream) {
    const int e = sizeof(T);
    const bool vec = a.D % 8 == 0 && vec_ok(a.x, a.ld_x, e) && vec_ok(a.res, a.ld_res, e) && vec_ok(a.w, 0, e) &&
                     vec_ok(a.h, a.ld_h, e) && vec_ok(a.y, a.ld_y, e) && vec_ok(a.q, a.ld_q, 1);
    return vec ? run_forward<T, true>(a, sm_count, stream) : run_forward<T, false>(a, sm_count, stream);
}

// Rows of partial sums of dweight, and CTAs, at most: four for each of 152 SMs
// where a row's warps leave room for them, two (of 512 threads or more)
// elsewhere, one for rows of four units a warp, whose partial sums cost more traffic
// than a second CTA in turn gains (300 x 12000 bf16: 24.7 us, with two 34.0; 2048 x
// 16384: 90.6 and 98.7).
int64_t grad_parts_of(int64_t D) {
    return D <= 8 * kUnit ? 608 : D > kMaxWarps * kUnit && D <= 4 * max_warps(4) * kUnit ? 152 : 304;
}

template <typename T, bool VEC>
cudaError_t run_grad(const RmsNormGradArgs& a, cudaStream_t stream) {
    int warps;
    const int cpt = units_per_warp((a.D + kUnit - 1) / kUnit, a.T >= 608, warps);
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
            case 0:
                if (a.dh != nullptr) rmsnorm_grad_kernel<T, VEC, 0><<<grid, 32 * warps, 0, stream>>>(a, false);
                break;
            case 1: rmsnorm_grad_kernel<T, VEC, 1><<<grid, 32 * warps, 0, stream>>>(a, dw); break;
            case 2: rmsnorm_grad_kernel<T, VEC, 2><<<grid, 32 * warps, 0, stream>>>(a, dw); break;
            default: rmsnorm_grad_kernel<T, VEC, 4><<<grid, 32 * warps, 0, stream>>>(a, dw); break;
        }
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (dw) {
        rmsnorm_dw_reduce_kernel<<<static_cast<unsigned>((a.D + 31) / 32), dim3(32, 32), 0, stream>>>(
            a.partial, a.T > 0 ? parts : 0, a.D, a.dw);
        return cudaGetLastError();
    }
    return cudaSuccess;
}

template <typename T>
cudaError_t grad_of(const RmsNormGradArgs& a, cudaStream_t stream) {
    const int e = sizeof(T);
    const bool vec = a.D % 8 == 0 && vec_ok(a.dy, a.ld_dy, e) && vec_ok(a.h, a.ld_h, e) && vec_ok(a.w, 0, e) &&
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

int64_t rmsnorm_grad_parts(int64_t T, int64_t D) { return std::min(T, grad_parts_of(D)); }

cudaError_t launch_rmsnorm_grad(const RmsNormGradArgs& a, vnm_dtype type, cudaStream_t stream) {
    switch (type) {
        case VNM_F16: return grad_of<__half>(a, stream);
        case VNM_BF16: return grad_of<__nv_bfloat16>(a, stream);
        default: return grad_of<float>(a, stream);
    }
}

}  // namespace vnm

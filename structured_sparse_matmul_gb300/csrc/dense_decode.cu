// The dense 16-bit layers for a few tokens.
//
//   Y[t][r] = act(sum_k X[t][k] W[r][k] + bias[r]) + residual[t][r]
//   Y[t][r] = act(G) * U,  G = X . Wg^T, U = X . Wu^T
//
// Bound by reading the weights once. Every warp streams them from global memory straight
// into the operand registers of mma.sync (m16n8k16, fp32 sums): 16 rows of W by 8 tokens;
// a gated pair takes 16 rows of Wg and the same 16 of Wu against the same tokens. The
// MMA's k positions may be dealt in any order as long as both operands agree: lane
// (g, i) = (lane / 4, lane % 4) reads 16 bytes of rows g and g + 8 at column 32 h + 8 i of
// a block of 64, and the same columns of token g, which are the operands of two MMAs with
// no shuffle. A CTA takes 16 rows, its warps deal the K blocks among themselves and
// meet once in shared memory, in a fixed order. The loads of W run kRing blocks ahead,
// those of x (from L2) one; a last block shorter than 64 is worked on while the first ones are on their way (1500 rows of 500,
// one token: 4.2 us behind the others and byte by byte, 2.1 so). After every round of the ring the MMAs' sums, which
// truncate, are added up in fp32. Measured, fp16, one token (us; in brackets the weights at a copy's rate, which is
// below what reads alone reach): 4096 rows of 11008 15.8 (13.5), 11008 x 2 rows of 4096 27.8 (27.0); what is left is
// the launch and the first loads' round trip.
#include <type_traits>

#include "vnm_dense16.cuh"
#include "vnm_internal.h"
#include "vnm_stream.cuh"

namespace vnm {
namespace {

constexpr int kRows = 16;  // rows of W of a CTA
constexpr int kBlockK = 64;

// 8 warps a CTA, two CTAs an SM; where there are no more CTAs than SMs, 16 warps, as many loads in flight, if K gives each
// two blocks; or, where those do not hold all rows of W at once, 4 warps, five CTAs, with fewer loads in flight a warp.
// 1 and 8 tokens, fp16 (us): 1024 rows of 11008 (64 CTAs) 11.4 and 12.1 with 8 warps, 7.6 and 8.1 with 16, 1024 of 1024
// 2.13 and 2.24, 2.11 and 2.28; 4096 rows of 11008 (256 CTAs) 15.8 and 16.9 with 8 warps, 31.6 and 31.9 with 4; 11008 rows of 4096 (688
// CTAs) 18.7 and 20.1, 16.3 and 16.4; gated 32.5 and 33.3, 27.8 and 27.9.
template <int WARPS, bool GATED>
struct Cfg {
    static constexpr int kCtas = WARPS == 16 ? 1 : WARPS == 8 ? 2 : 5;
    static constexpr int kRing = WARPS >= 8 ? (GATED ? 2 : 4) : (GATED ? 1 : 3);
};

struct FewArgs {
    const uint8_t *x, *w[2];
    int64_t ld_x, ld_w[2];  // bytes
    int64_t T, R, K;
    const void *bias, *res;
    int bias_type, act;
    int64_t ld_res;
    void* y;
    int64_t ld_y;
    int y_type;
};
// (kept apart: with these in the struct the dense kernel took 19.3 us instead of 16.1 for 4096 rows of 11008)
struct FewGatedArgs : FewArgs {
    void *g, *u;  // checkpoints of y_type, or NULL
    int64_t ld_g, ld_u;
};
template <bool GATED>
using ArgsOf = std::conditional_t<GATED, FewGatedArgs, FewArgs>;

// d += A (16 x 16, W) x B (16 x 8, X)
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes of X, which the SM's other warps read too. (Past L1, 8 tokens took 16.8 to 18.8 us through 4096 rows of 11008.)
__device__ __forceinline__ uint4 load_shared_row(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// 16 bytes of a row's last block, `left` bytes (an even number, any) before the row's end; what lies past it is not read. By
// loads that do not wait for each other: `in_place` puts the pieces there.
__device__ __forceinline__ uint4 load_end(const uint8_t* p, int left) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    const int n = left >= 16 || left < 0 ? 0 : left;
    asm volatile(
        "{\n\t.reg .pred w, a, b, c;\n\t"
        "setp.ge.s32 w, %5, 16;\n\tsetp.ne.s32 a, %6, 0;\n\tsetp.ne.s32 b, %7, 0;\n\tsetp.ne.s32 c, %8, 0;\n\t"
        "@w ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t"
        "@a ld.global.v2.u32 {%0, %1}, [%4];\n\t"
        "@b ld.global.u32 %2, [%9];\n\t"
        "@c ld.global.u16 %3, [%10];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "l"(p), "r"(left), "r"(n & 8), "r"(n & 4), "r"(n & 2), "l"(p + (n & 8)), "l"(p + (n & 12)));
    return v;
}
__device__ __forceinline__ uint4 in_place(const uint4& v, int left) {
    if (left >= 16 || left <= 0) return v;
    const uint32_t first = left & 4 ? v.z : v.w, second = left & 4 ? v.w : 0u;
    return left & 8 ? make_uint4(v.x, v.y, first, second) : make_uint4(first, second, 0u, 0u);
}

template <int NW>
struct Weights {
    uint4 v[NW][2][2];  // [matrix][row g, g + 8][step]
};
template <int NT>
struct Tokens {
    uint4 v[NT][2];  // of tokens g, g + 8
};

// Registers spill with 9 to 16 tokens of a gated pair: 164 bytes of stores and 192 of loads, with TAIL 552 and 520; and up to
// 60 and 60 in the other variants with TAIL that hold two matrices or two groups of tokens.
// NT: groups of 8 tokens. TAIL: K is no multiple of kBlockK (the code for its last block costs the others registers: 16
// tokens, gated, 1024 x 1024 took 3.2 us without it and 3.5 with it).
template <bool BF16, bool GATED, int NT, int kWarps, bool TAIL>
__global__ void __launch_bounds__(32 * kWarps, Cfg<kWarps, GATED>::kCtas) dense_decode_kernel(const ArgsOf<GATED> a) {
    constexpr int NW = GATED ? 2 : 1, kRing = Cfg<kWarps, GATED>::kRing;
    __shared__ float part[NW][kWarps][8 * NT][kRows + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, i = lane & 3;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows;
    // rows and tokens past the edges: the last ones again (their sums are not stored)
    const int64_t row0 = min(r0 + g, a.R - 1), row1 = min(r0 + g + 8, a.R - 1), last = a.T - 1;
    const int full = static_cast<int>(a.K / kBlockK);
    const uint8_t *w0[NW], *w1[NW], *x0[NT];
#pragma unroll
    for (int m = 0; m < NW; ++m) {
        w0[m] = a.w[m] + row0 * a.ld_w[m] + 16 * i;
        w1[m] = a.w[m] + row1 * a.ld_w[m] + 16 * i;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) x0[n] = a.x + min(static_cast<int64_t>(g + 8 * n), last) * a.ld_x + 16 * i;
    float sum[NW][NT][4], d[NW][NT][4];
#pragma unroll
    for (int m = 0; m < NW; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[m][n][e] = d[m][n][e] = 0.f;

    auto load_w = [&](Weights<NW>& w, int b) {
        const int64_t at = static_cast<int64_t>(b) * 128;
#pragma unroll
        for (int m = 0; m < NW; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w.v[m][0][h] = load_once_coherent(w0[m] + at + 64 * h);
                w.v[m][1][h] = load_once_coherent(w1[m] + at + 64 * h);
            }
    };
    auto load_x = [&](Tokens<NT>& x, int b) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                x.v[n][h] = load_shared_row(x0[n] + static_cast<int64_t>(b) * 128 + 64 * h);
    };
    auto multiply = [&](const Weights<NW>& w, const Tokens<NT>& x) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int m = 0; m < NW; ++m) {
                const uint4 &p = w.v[m][0][h], &q = w.v[m][1][h];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma<BF16>(d[m][n], p.x, q.x, p.y, q.y, x.v[n][h].x, x.v[n][h].y);
                    mma<BF16>(d[m][n], p.z, q.z, p.w, q.w, x.v[n][h].z, x.v[n][h].w);
                }
            }
    };
    auto take = [&] {  // the MMAs' sums: d[0], d[1]: row g, tokens 2i and 2i + 1; d[2], d[3]: row g + 8
#pragma unroll
        for (int m = 0; m < NW; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sum[m][n][e] += d[m][n][e];
                    d[m][n][e] = 0.f;
                }
    };
    Weights<NW> ring[kRing];
    Tokens<NT> cur, next;
    after_previous_grid();
    let_next_grid_start();
#pragma unroll
    for (int u = 0; u < kRing; ++u)
        if (warp + u * kWarps < full) load_w(ring[u], warp + u * kWarps);
    if (warp < full) load_x(next, warp);
    if (TAIL && full % kWarps == warp) {  // the last, shorter block, whose loads are in flight with the first ones
        const int64_t at = static_cast<int64_t>(full) * 128;
        const int left = static_cast<int>(2 * a.K - at) - 16 * i;
        Weights<NW> w;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int m = 0; m < NW; ++m) {
                w.v[m][0][h] = load_end(w0[m] + at + 64 * h, left - 64 * h);
                w.v[m][1][h] = load_end(w1[m] + at + 64 * h, left - 64 * h);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) cur.v[n][h] = load_end(x0[n] + at + 64 * h, left - 64 * h);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int m = 0; m < NW; ++m) {
                w.v[m][0][h] = in_place(w.v[m][0][h], left - 64 * h);
                w.v[m][1][h] = in_place(w.v[m][1][h], left - 64 * h);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) cur.v[n][h] = in_place(cur.v[n][h], left - 64 * h);
        }
        multiply(w, cur);
        take();
    }
#pragma unroll 1
    for (int b0 = warp; b0 < full; b0 += kRing * kWarps) {
#pragma unroll
        for (int u = 0; u < kRing; ++u) {
            const int b = b0 + u * kWarps;
            if (b >= full) break;  // the same for the whole warp
            cur = next;
            if (b + kWarps < full) load_x(next, b + kWarps);
            multiply(ring[u], cur);
            if (b + kRing * kWarps < full) load_w(ring[u], b + kRing * kWarps);
        }
        take();
    }
#pragma unroll
    for (int m = 0; m < NW; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[m][warp][8 * n + 2 * i + (e & 1)][g + 8 * (e >> 1)] = sum[m][n][e];
    __syncthreads();
    for (int k = threadIdx.x; k < 8 * NT * kRows; k += 32 * kWarps) {
        const int t = k / kRows, j = k % kRows;
        if (t >= a.T || r0 + j >= a.R) continue;
        float v[NW];
#pragma unroll
        for (int m = 0; m < NW; ++m) {
            v[m] = part[m][0][t][j];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) v[m] += part[m][w][t][j];
        }
        if constexpr (GATED) {
            if (a.g) {
                store_any(a.g, a.y_type, t * a.ld_g + r0 + j, v[0]);
                store_any(a.u, a.y_type, t * a.ld_u + r0 + j, v[1]);
            }
        }
        if (a.bias) v[0] += load_any(a.bias, a.bias_type, r0 + j);
        float y = a.act == VNM_ACT_SILU ? v[0] * sigmoid(v[0]) : activate(a.act, v[0]);
        if (GATED) y *= v[NW - 1];
        if (a.res) y += load_any(a.res, a.y_type, t * a.ld_res + r0 + j);
        store_any(a.y, a.y_type, t * a.ld_y + r0 + j, y);
    }
}

template <bool BF16, bool GATED, int NT, int WARPS>
cudaError_t launch(const FewGatedArgs& all, int64_t blocks, cudaStream_t stream) {
    const ArgsOf<GATED>& a = all;
    return a.K % kBlockK == 0 ? launch_early(dense_decode_kernel<BF16, GATED, NT, WARPS, false>, blocks, 32 * WARPS, 0, 1, stream, a)
                              : launch_early(dense_decode_kernel<BF16, GATED, NT, WARPS, true>, blocks, 32 * WARPS, 0, 1, stream, a);
}

template <bool BF16, bool GATED, int NT>
cudaError_t launch(const FewGatedArgs& a, int sm_count, cudaStream_t stream) {
    const int64_t blocks = (a.R + kRows - 1) / kRows;
    if (blocks <= sm_count && a.K >= 32 * kBlockK) return launch<BF16, GATED, NT, 16>(a, blocks, stream);
    if constexpr (NT == 1) {  // (with more than 8 tokens, more rows go to the narrow tiles)
        if (blocks > 2 * sm_count) return launch<BF16, GATED, NT, 4>(a, blocks, stream);
    }
    return launch<BF16, GATED, NT, 8>(a, blocks, stream);
}

template <bool BF16, bool GATED>
cudaError_t launch(const FewGatedArgs& all, int sm_count, cudaStream_t stream) {
    return all.T <= 8 ? launch<BF16, GATED, 1>(all, sm_count, stream) : launch<BF16, GATED, 2>(all, sm_count, stream);
}

}  // namespace

cudaError_t launch_few_tokens(const ProductArgs& p, int sm_count, cudaStream_t stream) {
    const bool gated = p.kind == kGatedPair;
    FewGatedArgs a{};
    a.x = static_cast<const uint8_t*>(p.x[0].p);
    a.ld_x = 2 * p.x[0].ld;
    for (int m = 0; m < (gated ? 2 : 1); ++m) {
        a.w[m] = static_cast<const uint8_t*>(p.w[m].p);
        a.ld_w[m] = 2 * p.w[m].ld;
    }
    a.T = p.T;
    a.R = p.R;
    a.K = p.K;
    a.bias = p.bias;
    a.res = p.residual[0];
    a.bias_type = p.bias_type;
    a.act = p.act;
    a.ld_res = p.ld_residual;
    a.y = p.y[0];
    a.ld_y = p.ld_y;
    a.y_type = p.y_type;
    if (p.keep == kKeep16) {
        a.g = p.g.p;
        a.u = p.u.p;
        a.ld_g = p.g.ld;
        a.ld_u = p.u.ld;
    }
    if (gated) return p.bf16 ? launch<true, true>(a, sm_count, stream) : launch<false, true>(a, sm_count, stream);
    return p.bf16 ? launch<true, false>(a, sm_count, stream) : launch<false, false>(a, sm_count, stream);
}

}  // namespace vnm

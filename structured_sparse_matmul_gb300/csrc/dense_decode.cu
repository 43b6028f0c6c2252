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
// no shuffle. A CTA takes 16 rows, its 8 warps deal the K blocks among themselves and
// meet once in shared memory, in a fixed order. The loads of W run kRing blocks ahead,
// those of x (from L2) one. After every round of the ring the MMAs' sums, which
// truncate, are added up in fp32.
#include "vnm_dense16.cuh"
#include "vnm_internal.h"
#include "vnm_stream.cuh"

namespace vnm {
namespace {

constexpr int kRows = 16;  // rows of W of a CTA
constexpr int kWarps = 8;
constexpr int kBlockK = 64;

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

template <int NW>
struct Weights {
    uint4 v[NW][2][2];  // [matrix][row g, g + 8][step]
};
struct Tokens {
    uint4 v[2];  // of token g
};

template <bool BF16, bool GATED>
__global__ void __launch_bounds__(32 * kWarps, 2) dense_decode_kernel(const FewArgs a) {
    constexpr int NW = GATED ? 2 : 1, kRing = GATED ? 2 : 4;
    __shared__ float part[NW][kWarps][kFewTokens][kRows + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, i = lane & 3;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows;
    // rows and tokens past the edges: the last ones again (their sums are not stored)
    const int64_t row0 = min(r0 + g, a.R - 1), row1 = min(r0 + g + 8, a.R - 1), last = a.T - 1;
    const int full = static_cast<int>(a.K / kBlockK);
    const uint8_t *w0[NW], *w1[NW];
#pragma unroll
    for (int m = 0; m < NW; ++m) {
        w0[m] = a.w[m] + row0 * a.ld_w[m] + 16 * i;
        w1[m] = a.w[m] + row1 * a.ld_w[m] + 16 * i;
    }
    const uint8_t* x0 = a.x + min(static_cast<int64_t>(g), last) * a.ld_x + 16 * i;
    float sum[NW][4], d[NW][4];
#pragma unroll
    for (int m = 0; m < NW; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[m][e] = d[m][e] = 0.f;

    auto load_w = [&](Weights<NW>& w, int b) {
        const int64_t at = static_cast<int64_t>(b) * 128;
#pragma unroll
        for (int m = 0; m < NW; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w.v[m][0][h] = load_once(w0[m] + at + 64 * h);
                w.v[m][1][h] = load_once(w1[m] + at + 64 * h);
            }
    };
    auto load_x = [&](Tokens& x, int b) {
#pragma unroll
        for (int h = 0; h < 2; ++h) x.v[h] = __ldg(reinterpret_cast<const uint4*>(x0 + static_cast<int64_t>(b) * 128 + 64 * h));
    };
    auto multiply = [&](const Weights<NW>& w, const Tokens& x) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int m = 0; m < NW; ++m) {
                const uint4 &p = w.v[m][0][h], &q = w.v[m][1][h];
                mma<BF16>(d[m], p.x, q.x, p.y, q.y, x.v[h].x, x.v[h].y);
                mma<BF16>(d[m], p.z, q.z, p.w, q.w, x.v[h].z, x.v[h].w);
            }
    };
    auto take = [&] {  // the MMAs' sums: d[0], d[1]: row g, tokens 2i and 2i + 1; d[2], d[3]: row g + 8
#pragma unroll
        for (int m = 0; m < NW; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sum[m][e] += d[m][e];
                d[m][e] = 0.f;
            }
    };
    Weights<NW> ring[kRing];
    Tokens cur, next;
    let_next_grid_start();
    after_previous_grid();
#pragma unroll
    for (int u = 0; u < kRing; ++u)
        if (warp + u * kWarps < full) load_w(ring[u], warp + u * kWarps);
    if (warp < full) load_x(next, warp);
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
    if (a.K % kBlockK != 0 && full % kWarps == warp) {
        const int64_t at = static_cast<int64_t>(full) * 128 + 16 * i, end = 2 * a.K;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int m = 0; m < NW; ++m) {
                ring[0].v[m][0][h] = load_edge(w0[m] - 16 * i, at + 64 * h, end, row0 == a.R - 1);
                ring[0].v[m][1][h] = load_edge(w1[m] - 16 * i, at + 64 * h, end, row1 == a.R - 1);
            }
            cur.v[h] = load_edge(x0 - 16 * i, at + 64 * h, end, g >= last);
        }
        multiply(ring[0], cur);
        take();
    }
#pragma unroll
    for (int m = 0; m < NW; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[m][warp][2 * i + (e & 1)][g + 8 * (e >> 1)] = sum[m][e];
    __syncthreads();
    const int t = threadIdx.x / kRows, j = threadIdx.x % kRows;
    if (t >= kFewTokens || t >= a.T || r0 + j >= a.R) return;
    float v[NW];
#pragma unroll
    for (int m = 0; m < NW; ++m) {
        v[m] = part[m][0][t][j];
#pragma unroll
        for (int k = 1; k < kWarps; ++k) v[m] += part[m][k][t][j];
    }
    if (a.bias) v[0] += load_any(a.bias, a.bias_type, r0 + j);
    float y = a.act == VNM_ACT_SILU ? v[0] * sigmoid(v[0]) : activate(a.act, v[0]);
    if (GATED) y *= v[NW - 1];
    if (a.res) y += load_any(a.res, a.y_type, t * a.ld_res + r0 + j);
    store_any(a.y, a.y_type, t * a.ld_y + r0 + j, y);
}

template <bool BF16, bool GATED>
cudaError_t launch(const FewArgs& a, cudaStream_t stream) {
    return launch_early(dense_decode_kernel<BF16, GATED>, (a.R + kRows - 1) / kRows, 32 * kWarps, 0, 1, stream, a);
}

}  // namespace

cudaError_t launch_few_tokens(const ProductArgs& p, cudaStream_t stream) {
    const bool gated = p.kind == kGatedPair;
    FewArgs a{};
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
    if (gated) return p.bf16 ? launch<true, true>(a, stream) : launch<false, true>(a, stream);
    return p.bf16 ? launch<true, false>(a, stream) : launch<false, false>(a, stream);
}

}  // namespace vnm

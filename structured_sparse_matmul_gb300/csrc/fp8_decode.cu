// The block-scaled 8-bit Linear layer for a few tokens.
//
//   Y[t][r] = act(sum_b xs[t, b] ws[r', b] (sum_{k in b} xq[t][k] wq[r][k]) + bias[r])
//
// Bound by reading W once. The tiled tensor-core kernel's setup (TMEM, a TMA
// pipeline, a cluster's sum) takes as long as the whole read of a 4096 x 4096 W,
// so here every warp streams W from global memory straight into the operand
// registers of mma.sync (m16n8k32, 8-bit, fp32 sums): 16 rows of W by 8 tokens.
// The MMA's k positions may be dealt in any order as long as both operands agree:
// lane (g, i) = (lane / 4, lane % 4) reads 16 bytes of rows g and g + 8 at column
// 64 h + 16 i, and the same columns of token g, which are the operands of two MMAs
// with no shuffle. A K block (two such steps, four MMAs) starts from zero and is
// scaled as it is added to the sums. A CTA takes 16 rows, its 8 warps deal the
// K blocks among themselves and meet once in shared memory, in a fixed order. The
// loads of W run kRing blocks ahead, those of x and the scales (from L2) one. The
// code is kept short: a launch this small pays for every line that it fetches.
//
// Measured, one token: 4096 x 4096 4.6 us, 3.7 TB/s, of which about 2 us are the launch
// and the first round trip (the tiled kernel 7.2); 11008 x 4096 13.0 us (12.6); 1024 x
// 1024 2.4 us (5.0). Up to 8 tokens cost the same; 16 as two groups of 8 took 8.0 and
// 18.5 us against the tiled kernel's 7.7 and 13.2, so they go there.
#include "vnm_dense.h"
#include "vnm_fp8.cuh"

namespace vnm {
namespace {

constexpr int kRows = 16;                // rows of W of a CTA
constexpr int kWarps = 8;
constexpr int kMaxTokens = kMaxDecodeTokens;
constexpr int kRing = 4;

struct DecodeArgs {
    const uint8_t *x, *w;
    int64_t ld_x, ld_w;
    ScaleView xs, ws;
    int64_t T, R, K;
    const void* bias;
    int bias_type, act;
    void* y;
    int64_t ld_y;
    int y_type;
};

// 16 bytes of W: read once, not kept in L1.
__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// 16 bytes of a row from column k on, 0 from column K on (the last, shorter block).
// Rows are 16-byte aligned, so the 16 bytes lie within the row's pitch; the last
// row's pitch may not be all there, and its last bytes are read one by one.
__device__ __noinline__ uint4 load_edge(const uint8_t* row, int64_t k, int64_t K, bool last_row) {
    const int n = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(16), K - k)));  // bytes that exist
    uint32_t u[4] = {0u, 0u, 0u, 0u};
    if (n == 16 || (n > 0 && !last_row)) {
        const uint4 v = load_once(row + k);
        u[0] = v.x;
        u[1] = v.y;
        u[2] = v.z;
        u[3] = v.w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int left = n - 4 * j;
            u[j] = left >= 4 ? u[j] : left <= 0 ? 0u : u[j] & (0xFFFFFFFFu >> (8 * (4 - left)));
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const uint32_t byte = row[k + i];
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] |= j == i / 4 ? byte << (8 * (i & 3)) : 0u;
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// d += A (16 x 32, W) x B (32 x 8, X)
template <bool W5, bool X5>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
#define VNM_MMA(A, B)                                                                        \
    asm("mma.sync.aligned.m16n8k32.row.col.f32." A "." B ".f32 {%0, %1, %2, %3}, "           \
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"                                      \
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                     \
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
    if (W5 && X5)
        VNM_MMA("e5m2", "e5m2");
    else if (W5)
        VNM_MMA("e5m2", "e4m3");
    else if (X5)
        VNM_MMA("e4m3", "e5m2");
    else
        VNM_MMA("e4m3", "e4m3");
#undef VNM_MMA
}

// A lane's share of one K block.
struct Weights {
    uint4 v[2][2];  // [row g, g + 8][step]
};
struct Rest {
    uint4 x[2];          // token g
    float sw[2], sx[2];  // scales of rows g, g + 8; of tokens 2i, 2i + 1
};

template <bool W5, bool X5>
__global__ void __launch_bounds__(32 * kWarps, 2) fp8_decode_kernel(const DecodeArgs a) {
    __shared__ float part[kWarps][kMaxTokens][kRows + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, i = lane & 3;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows;
    // rows and tokens past the edges: the last ones again (their sums are not stored)
    const int64_t row0 = min(r0 + g, a.R - 1), row1 = min(r0 + g + 8, a.R - 1), last = a.T - 1;
    const int full = static_cast<int>(a.K / kGroup);
    const uint8_t *w0 = a.w + row0 * a.ld_w + 16 * i, *w1 = a.w + row1 * a.ld_w + 16 * i;
    const uint8_t* x0 = a.x + min(static_cast<int64_t>(g), last) * a.ld_x + 16 * i;
    const float *ws0 = a.ws.p + (row0 >> a.ws.shift) * a.ws.rs, *ws1 = a.ws.p + (row1 >> a.ws.shift) * a.ws.rs;
    const float* xs0 = a.xs.p + min(static_cast<int64_t>(2 * i), last) * a.xs.rs;
    const float* xs1 = a.xs.p + min(static_cast<int64_t>(2 * i + 1), last) * a.xs.rs;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};

    auto load_w = [&](Weights& w, int b) {
        const int64_t k = static_cast<int64_t>(b) * kGroup;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w.v[0][h] = load_once(w0 + k + 64 * h);
            w.v[1][h] = load_once(w1 + k + 64 * h);
        }
    };
    auto load_scales = [&](Rest& v, int b) {
        v.sw[0] = ws0[b * a.ws.cs];
        v.sw[1] = ws1[b * a.ws.cs];
        v.sx[0] = xs0[b * a.xs.cs];
        v.sx[1] = xs1[b * a.xs.cs];
    };
    auto load_rest = [&](Rest& v, int b) {
        const int64_t k = static_cast<int64_t>(b) * kGroup;
#pragma unroll
        for (int h = 0; h < 2; ++h) v.x[h] = __ldg(reinterpret_cast<const uint4*>(x0 + k + 64 * h));
        load_scales(v, b);
    };
    auto multiply = [&](const Weights& w, const Rest& v) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            mma<W5, X5>(d, w.v[0][h].x, w.v[1][h].x, w.v[0][h].y, w.v[1][h].y, v.x[h].x, v.x[h].y);
            mma<W5, X5>(d, w.v[0][h].z, w.v[1][h].z, w.v[0][h].w, w.v[1][h].w, v.x[h].z, v.x[h].w);
        }
        // d[0], d[1]: row g, tokens 2i and 2i + 1; d[2], d[3]: row g + 8
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = fmaf(d[e], v.sx[e & 1] * v.sw[e >> 1], sum[e]);
    };
    Weights ring[kRing];
    Rest cur, next;
#pragma unroll
    for (int u = 0; u < kRing; ++u)
        if (warp + u * kWarps < full) load_w(ring[u], warp + u * kWarps);
    if (warp < full) load_rest(next, warp);
#pragma unroll 1
    for (int b0 = warp; b0 < full; b0 += kRing * kWarps) {
#pragma unroll
        for (int u = 0; u < kRing; ++u) {
            const int b = b0 + u * kWarps;
            if (b >= full) break;  // the same for the whole warp
            cur = next;
            if (b + kWarps < full) load_rest(next, b + kWarps);
            multiply(ring[u], cur);
            if (b + kRing * kWarps < full) load_w(ring[u], b + kRing * kWarps);
        }
    }
    if (a.K % kGroup != 0 && full % kWarps == warp) {
        const int64_t k = static_cast<int64_t>(full) * kGroup + 16 * i;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ring[0].v[0][h] = load_edge(w0 - 16 * i, k + 64 * h, a.K, row0 == a.R - 1);
            ring[0].v[1][h] = load_edge(w1 - 16 * i, k + 64 * h, a.K, row1 == a.R - 1);
            cur.x[h] = load_edge(x0 - 16 * i, k + 64 * h, a.K, g >= last);
        }
        load_scales(cur, full);
        multiply(ring[0], cur);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) part[warp][2 * i + (e & 1)][g + 8 * (e >> 1)] = sum[e];
    __syncthreads();
    const int t = threadIdx.x / kRows, j = threadIdx.x % kRows;
    if (t >= kMaxTokens || t >= a.T || r0 + j >= a.R) return;
    float v = part[0][t][j];
#pragma unroll
    for (int k = 1; k < kWarps; ++k) v += part[k][t][j];
    if (a.bias) v += load_any(a.bias, a.bias_type, r0 + j);
    store_any(a.y, a.y_type, t * a.ld_y + r0 + j, activate(a.act, v));
}

template <bool W5, bool X5>
void launch(const DecodeArgs& a, cudaStream_t stream) {
    fp8_decode_kernel<W5, X5><<<static_cast<unsigned>((a.R + kRows - 1) / kRows), 32 * kWarps, 0, stream>>>(a);
}

}  // namespace

bool fp8_decode_serves(int64_t T) { return T <= kMaxTokens; }

cudaError_t launch_fp8_decode(const void* xq, int64_t ld_x, bool x_e5m2, const ScaleView& xs, const void* wq,
                              int64_t ld_w, bool w_e5m2, const ScaleView& ws, int64_t T, int64_t R, int64_t K,
                              const void* bias, vnm_dtype bias_type, int act, void* y, int64_t ld_y, vnm_dtype y_type,
                              cudaStream_t stream) {
    const DecodeArgs a{static_cast<const uint8_t*>(xq), static_cast<const uint8_t*>(wq), ld_x, ld_w, xs, ws, T, R, K,
                       bias, static_cast<int>(bias_type), act, y, ld_y, static_cast<int>(y_type)};
    if (w_e5m2)
        x_e5m2 ? launch<true, true>(a, stream) : launch<true, false>(a, stream);
    else
        x_e5m2 ? launch<false, true>(a, stream) : launch<false, false>(a, stream);
    return cudaGetLastError();
}

}  // namespace vnm

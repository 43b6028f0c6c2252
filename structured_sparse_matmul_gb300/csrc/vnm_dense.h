// Internal declarations of the dense neighbours of a pruned layer: RMS norm,
// block-scaled 8-bit quantiser, 8-bit Linear layer (kernels and their host side
// in dense_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/vnm.h"

namespace vnm {

constexpr int kGroup = 128;  // columns of a scale group, rows and columns of a scale block

struct RmsNormArgs {
    const void *x, *res, *w;
    void *h, *y, *q;
    float *rstd, *s;
    int64_t ld_x, ld_res, ld_h, ld_y, ld_q, s_rs, s_cs;
    int64_t T, D;
    float eps;
    bool e5m2;
};
cudaError_t launch_rmsnorm(const RmsNormArgs& a, vnm_dtype type, int sm_count, cudaStream_t stream);

struct RmsNormGradArgs {
    const void *dy, *h, *w, *dres;
    const float* rstd;
    void* dh;
    float* dw;
    float* partial;  // [rmsnorm_grad_parts(T, D)][D]
    int64_t ld_dy, ld_h, ld_dres, ld_dh;
    int64_t T, D;
};
// Rows of partial sums of dweight: a function of the sizes alone.
int64_t rmsnorm_grad_parts(int64_t T, int64_t D);
cudaError_t launch_rmsnorm_grad(const RmsNormGradArgs& a, vnm_dtype type, cudaStream_t stream);

struct QuantArgs {
    const void* x;
    uint8_t *q, *qt;
    float *s, *st;
    int64_t ld_x, ld_q, ld_qt, s_rs, s_cs, st_rs, st_cs;
    int64_t R, C;
    bool block;  // 128 x 128 blocks
    bool e5m2;
};
cudaError_t launch_fp8_quantize(const QuantArgs& a, vnm_dtype type, cudaStream_t stream);

// One operand's scales: element (i, b) for row i of the operand and group b.
struct ScaleView {
    const float* p;
    int64_t rs, cs;
    int shift;  // 7: one scale for 128 rows, 0: one for each row
};

// The product as the kernel sees it: P (128-row tiles, the MMA's M side) times
// Q (the MMA's N side). Y element (m, n) is at Y + m * y_ms + n * y_ns.
struct Fp8LinearArgs {
    const void *p, *q;
    int64_t ld_p, ld_q;
    bool p_e5m2, q_e5m2;
    ScaleView ps, qs;
    int64_t m, n, k;
    int64_t y_ms, y_ns;
    bool bias_on_m;
};
cudaError_t launch_fp8_linear(const void* xq, int64_t ld_x, bool x_e5m2, const ScaleView& xs, const void* wq,
                              int64_t ld_w, bool w_e5m2, const ScaleView& ws, int64_t T, int64_t R, int64_t K,
                              const void* bias, vnm_dtype bias_type, int act, void* y, int64_t ld_y, vnm_dtype y_type,
                              int* status, int skip_stage, int sm_count, cudaStream_t stream);

// Which kernel takes a product (K >= 1), by the rule that launch_fp8_linear goes by: tiles of 16, 32,
// 64 or 128 tokens with K over `splits` CTAs; pairs of CTAs (0); the few-token kernel (kMaxDecodeTokens).
constexpr int kMaxDecodeTokens = 8;
void fp8_linear_plan(int64_t T, int64_t R, int64_t K, bool one_scale, int sm_count, int* tile_tokens, int* splits);

// The first error that calls without status words recorded on the current device, and clears it.
cudaError_t take_fp8_linear_status(int* code, cudaStream_t stream);

// The same product for a few tokens (T >= 1, K >= 1).
bool fp8_decode_serves(int64_t T);
cudaError_t launch_fp8_decode(const void* xq, int64_t ld_x, bool x_e5m2, const ScaleView& xs, const void* wq,
                              int64_t ld_w, bool w_e5m2, const ScaleView& ws, int64_t T, int64_t R, int64_t K,
                              const void* bias, vnm_dtype bias_type, int act, void* y, int64_t ld_y, vnm_dtype y_type,
                              cudaStream_t stream);

}  // namespace vnm

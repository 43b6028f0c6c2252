// Host side of the dense 16-bit layers (include/vnm.h): argument checks, and the
// launches of the gated pair's backward pass. Every check runs before anything is enqueued.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "vnm_dense16.h"
#include "vnm_testing.h"

namespace {

constexpr int64_t kMaxSize = (int64_t(1) << 31) - 1024;  // TMA coordinates, of a tile past the edge too, are int32
constexpr int kMaxDevices = 64;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Element size of a vnm_dtype, 0 for anything else.
size_t size_of(vnm_dtype t) { return t == VNM_F32 ? 4 : t == VNM_F16 || t == VNM_BF16 ? 2 : 0; }

bool size_ok(int64_t n) { return n >= 0 && n <= kMaxSize; }
bool act_ok(vnm_activation a) { return a == VNM_ACT_NONE || a == VNM_ACT_RELU || a == VNM_ACT_GELU || a == VNM_ACT_SILU; }

bool matrix_ok(const void* p, int64_t ld, int64_t cols, size_t elem) {
    return p != nullptr && aligned(p, elem) && ld >= std::max<int64_t>(cols, 1);
}

// An operand's storage: `rows` rows of `cols` elements that start on 16 bytes. One row has no pitch.
bool operand_ok(vnm::Operand16* x, const void* p, int64_t ld, int64_t rows, int64_t cols, bool transposed) {
    if (rows == 1 && ld >= cols) ld = (cols + 7) / 8 * 8;
    *x = vnm::Operand16{p, ld, transposed};
    return matrix_ok(p, ld, cols, 16) && ld % 8 == 0;
}

// A checkpoint of T x F elements, at `k` as its kind says.
bool kept_ok(vnm::Kept* k, vnm_keep keep, const void* p, int64_t ld, const float* s, int64_t s_rs, int64_t s_cs, int64_t F) {
    *k = vnm::Kept{const_cast<void*>(p), ld, const_cast<float*>(s), s_rs, s_cs};
    if (keep == VNM_KEEP_NONE) return true;
    if (keep == VNM_KEEP_16) return matrix_ok(p, ld, F, 2);
    return matrix_ok(p, ld, F, 1) && s != nullptr && aligned(s, 4);
}

bool keep_ok(vnm_keep k) { return k == VNM_KEEP_NONE || k == VNM_KEEP_16 || k == VNM_KEEP_E4M3 || k == VNM_KEEP_E5M2; }

vnm::KeepKind kind_of(vnm_keep k) {
    return k == VNM_KEEP_NONE ? vnm::kKeepNone : k == VNM_KEEP_16 ? vnm::kKeep16 : vnm::kKeep8;
}

// SMs of the current device (0: no device), asked once for each.
int sm_count() {
    static std::atomic<int> known[kMaxDevices];
    int dev = -1, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
    if (dev < kMaxDevices && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < kMaxDevices) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

vnm_status launched(cudaError_t e) { return e == cudaSuccess ? VNM_OK : VNM_ERR_CUDA; }

vnm_status dense_linear(const void* X, int64_t ld_x, int32_t x_transposed, const void* W, int64_t ld_w,
                        int32_t w_transposed, vnm_dtype type, int64_t T, int64_t R, int64_t K, const void* bias,
                        vnm_dtype bias_type, vnm_activation act, const void* residual, int64_t ld_residual, void* Y,
                        int64_t ld_y, vnm_dtype y_type, int32_t* status, int skip_stage, vnm_stream_t stream) {
    if ((type != VNM_F16 && type != VNM_BF16) || (y_type != type && y_type != VNM_F32) || !act_ok(act) || !size_ok(T) ||
        !size_ok(R) || !size_ok(K) || (x_transposed != 0 && x_transposed != 1) || (w_transposed != 0 && w_transposed != 1))
        return VNM_ERR_INVALID_ARG;
    if (bias != nullptr && (size_of(bias_type) == 0 || !aligned(bias, size_of(bias_type)))) return VNM_ERR_INVALID_ARG;
    if (!aligned(status, 4)) return VNM_ERR_INVALID_ARG;
    if (T == 0 || R == 0) return VNM_OK;
    const size_t e = size_of(y_type);
    if (!matrix_ok(Y, ld_y, R, e) || (residual != nullptr && !matrix_ok(residual, ld_residual, R, e)) ||
        (residual == Y && ld_residual != ld_y && T > 1))
        return VNM_ERR_INVALID_ARG;
    vnm::ProductArgs p{};
    if (K > 0 && (!operand_ok(&p.x[0], X, ld_x, x_transposed ? K : T, x_transposed ? T : K, x_transposed != 0) ||
                  !operand_ok(&p.w[0], W, ld_w, w_transposed ? K : R, w_transposed ? R : K, w_transposed != 0)))
        return VNM_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms == 0) return VNM_ERR_CUDA;
    p.kind = vnm::kOneProduct;
    p.T = T;
    p.R = R;
    p.K = K;
    p.bf16 = type == VNM_BF16;
    p.y[0] = Y;
    p.ld_y = ld_y;
    p.y_type = y_type;
    p.bias = bias;
    p.bias_type = bias_type;
    p.act = act;
    p.residual[0] = residual;
    p.ld_residual = ld_residual;
    p.keep = vnm::kKeepNone;
    p.status = status;
    p.skip_stage = skip_stage;
    return launched(vnm::launch_product(p, vnm::plan_product(p, sms), sms, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t padded(int64_t F) { return (F + 7) / 8 * 8; }

vnm_status gated_linear(const void* X, int64_t ld_x, const void* Wg, int64_t ld_wg, const void* Wu, int64_t ld_wu,
                        vnm_dtype type, int64_t T, int64_t F, int64_t K, vnm_activation act, void* Y, int64_t ld_y,
                        vnm_keep keep, void* g, int64_t ld_g, float* g_scale, int64_t gs_rs, int64_t gs_cs, void* u,
                        int64_t ld_u, float* u_scale, int64_t us_rs, int64_t us_cs, int32_t* status,
                        int skip_stage, vnm_stream_t stream) {
    if ((type != VNM_F16 && type != VNM_BF16) || !act_ok(act) || !keep_ok(keep) || !size_ok(T) || !size_ok(F) || !size_ok(K) ||
        !aligned(status, 4))
        return VNM_ERR_INVALID_ARG;
    if (T == 0 || F == 0) return VNM_OK;
    vnm::ProductArgs p{};
    if (!matrix_ok(Y, ld_y, F, 2) || !kept_ok(&p.g, keep, g, ld_g, g_scale, gs_rs, gs_cs, F) ||
        !kept_ok(&p.u, keep, u, ld_u, u_scale, us_rs, us_cs, F))
        return VNM_ERR_INVALID_ARG;
    if (K > 0 && (!operand_ok(&p.x[0], X, ld_x, T, K, false) || !operand_ok(&p.w[0], Wg, ld_wg, F, K, false) ||
                  !operand_ok(&p.w[1], Wu, ld_wu, F, K, false)))
        return VNM_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms == 0) return VNM_ERR_CUDA;
    p.kind = vnm::kGatedPair;
    p.T = T;
    p.R = F;
    p.K = K;
    p.bf16 = type == VNM_BF16;
    p.y[0] = Y;
    p.ld_y = ld_y;
    p.y_type = type;
    p.act = act;
    p.keep = kind_of(keep);
    p.e5m2 = keep == VNM_KEEP_E5M2;
    p.status = status;
    p.skip_stage = skip_stage;
    return launched(vnm::launch_product(p, vnm::plan_product(p, sms), sms, reinterpret_cast<cudaStream_t>(stream)));
}

vnm_status gated_linear_backward(const void* dY, int64_t ld_dy, const void* X, int64_t ld_x, const void* Wg,
                                 int64_t ld_wg, const void* Wu, int64_t ld_wu, vnm_dtype type, int64_t T, int64_t F,
                                 int64_t K, vnm_activation act, vnm_keep keep, const void* g, int64_t ld_g,
                                 const float* g_scale, int64_t gs_rs, int64_t gs_cs, const void* u, int64_t ld_u,
                                 const float* u_scale, int64_t us_rs, int64_t us_cs, void* dX, int64_t ld_dx, void* dWg,
                                 void* dWu, int64_t ld_dw, vnm_dtype w_type, int32_t accumulate, void* H, int64_t ld_h,
                                 void* workspace, size_t workspace_bytes, int32_t* status, int skip_dx,
                                 int skip_dw, vnm_stream_t stream) {
    const bool weights = dWg != nullptr;
    if ((type != VNM_F16 && type != VNM_BF16) || !act_ok(act) || !keep_ok(keep) || keep == VNM_KEEP_NONE || !size_ok(T) ||
        !size_ok(F) || !size_ok(K) || !aligned(status, 4) || (accumulate != 0 && accumulate != 1) ||
        weights != (dWu != nullptr) || (weights && w_type != type && w_type != VNM_F32))
        return VNM_ERR_INVALID_ARG;
    vnm::ProductArgs in{}, gr{};  // of dX, of dWg and dWu
    vnm::GatedGradArgs e{};
    const bool any_dx = dX != nullptr && T > 0 && K > 0, any_dw = weights && F > 0 && K > 0, any_h = H != nullptr && T > 0 && F > 0;
    const bool products = (any_dx || any_dw) && T > 0 && F > 0;  // dG and dU are needed
    if (any_dx && !matrix_ok(dX, ld_dx, K, 2)) return VNM_ERR_INVALID_ARG;
    if (any_dw && (!matrix_ok(dWg, ld_dw, K, size_of(w_type)) || !matrix_ok(dWu, ld_dw, K, size_of(w_type)) || dWg == dWu))
        return VNM_ERR_INVALID_ARG;
    if (any_h && (!matrix_ok(H, ld_h, F, 2) || (H == dY && ld_h != ld_dy && T > 1))) return VNM_ERR_INVALID_ARG;
    if ((products || any_h) && (!kept_ok(&e.g, keep, g, ld_g, g_scale, gs_rs, gs_cs, F) ||
                                !kept_ok(&e.u, keep, u, ld_u, u_scale, us_rs, us_cs, F)))
        return VNM_ERR_INVALID_ARG;
    if (products) {
        size_t need = 0;
        if (!matrix_ok(dY, ld_dy, F, 2) || vnm_gated_linear_backward_workspace_size(T, F, &need) != VNM_OK || workspace == nullptr ||
            !aligned(workspace, 16) || workspace_bytes < need)
            return VNM_ERR_INVALID_ARG;
        if (any_dx && (!operand_ok(&in.w[0], Wg, ld_wg, F, K, true) || !operand_ok(&in.w[1], Wu, ld_wu, F, K, true)))
            return VNM_ERR_INVALID_ARG;
        if (any_dw && !operand_ok(&gr.w[0], X, ld_x, T, K, true)) return VNM_ERR_INVALID_ARG;
    }
    if (!any_dx && !any_dw && !any_h) return VNM_OK;
    const int sms = sm_count();
    if (sms == 0) return VNM_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t ld_d = 2 * padded(F);
    uint16_t *dg = static_cast<uint16_t*>(workspace), *du = dg == nullptr ? nullptr : dg + padded(F);
    cudaError_t err = cudaSuccess;
    if (products || any_h) {
        e.T = T;
        e.F = F;
        e.bf16 = type == VNM_BF16;
        e.act = act;
        e.keep = kind_of(keep);
        e.e5m2 = keep == VNM_KEEP_E5M2;
        if (products) {
            e.dy = dY;
            e.ld_dy = ld_dy;
            e.dg = dg;
            e.du = du;
            e.ld_d = ld_d;
        }
        e.h = H;
        e.ld_h = ld_h;
        err = vnm::launch_gated_grad(e, sms, s);
    }
    const bool dx = any_dx, dw = any_dw && !(T == 0 && accumulate);
    if (dx) {
        in.kind = vnm::kSumOfTwo;
        in.T = T;
        in.R = K;
        in.K = F;
        in.bf16 = type == VNM_BF16;
        in.x[0] = vnm::Operand16{dg, ld_d, false};
        in.x[1] = vnm::Operand16{du, ld_d, false};
        in.y[0] = dX;
        in.ld_y = ld_dx;
        in.y_type = type;
        in.act = VNM_ACT_NONE;
        in.status = status;
        in.skip_stage = skip_dx;
    }
    if (dw) {
        gr.kind = vnm::kTwoByRows;
        gr.T = F;
        gr.R = K;
        gr.K = T;
        gr.bf16 = type == VNM_BF16;
        gr.x[0] = vnm::Operand16{dg, ld_d, true};
        gr.x[1] = vnm::Operand16{du, ld_d, true};
        gr.y[0] = dWg;
        gr.y[1] = dWu;
        gr.ld_y = ld_dw;
        gr.y_type = w_type;
        gr.act = VNM_ACT_NONE;
        if (accumulate) {
            gr.residual[0] = dWg;
            gr.residual[1] = dWu;
            gr.ld_residual = ld_dw;
        }
        gr.status = status;
        gr.skip_stage = skip_dw;
    }
    // dX and the weights' gradients share dG and dU, and neither reads what the other writes: their grids run side by side.
    // The pass in us, one after the other and so (T x F over K): 42 x 1576 over 125 13.0 and 9.0, 333 x 1001 over 1023 22.8
    // and 20.5, 2042 x 654 over 684 34.9 and 25.6, 512 x 4096 over 1024 43.2 and 42.7; where both are pairs of CTAs, which take
    // whole SMs, the same within 1 %: 1176 x 6308 over 1314 120.9 and 119.4, 2048 x 5632 over 2048 136.9 and 137.5.
    in.next_beside = gr.beside = dx && dw && products;
    if (dx && err == cudaSuccess) err = vnm::launch_product(in, vnm::plan_product(in, sms), sms, s);
    if (dw && err == cudaSuccess) err = vnm::launch_product(gr, vnm::plan_product(gr, sms), sms, s);
    return launched(err);
}

}  // namespace

extern "C" {

vnm_status vnm_dense_linear(const void* X, int64_t ld_x, int32_t x_transposed, const void* W, int64_t ld_w,
                            int32_t w_transposed, vnm_dtype type, int64_t T, int64_t R, int64_t K, const void* bias,
                            vnm_dtype bias_type, vnm_activation act, const void* residual, int64_t ld_residual, void* Y,
                            int64_t ld_y, vnm_dtype y_type, int32_t* status, vnm_stream_t stream) {
    return dense_linear(X, ld_x, x_transposed, W, ld_w, w_transposed, type, T, R, K, bias, bias_type, act, residual,
                        ld_residual, Y, ld_y, y_type, status, -1, stream);
}

vnm_status vnm_testing_dense_linear_skip_stage(const void* X, int64_t ld_x, const void* W, int64_t ld_w, vnm_dtype type,
                                               int64_t T, int64_t R, int64_t K, void* Y, int64_t ld_y, vnm_dtype y_type,
                                               int32_t* status, int32_t skip_stage, vnm_stream_t stream) {
    if (skip_stage < 0) return VNM_ERR_INVALID_ARG;
    return dense_linear(X, ld_x, 0, W, ld_w, 0, type, T, R, K, nullptr, VNM_F32, VNM_ACT_NONE, nullptr, 0, Y, ld_y, y_type, status,
                        skip_stage, stream);
}

vnm_status vnm_testing_dense_plan(int32_t kind, int64_t T, int64_t R, int64_t K, int32_t x_transposed, int32_t w_transposed,
                                  vnm_keep keep, int32_t aligned, int32_t sm_count, int32_t* tile_tokens, int32_t* tile_rows,
                                  int32_t* splits) {
    if (kind < 0 || kind > vnm::kGatedPair || !size_ok(T) || !size_ok(R) || !size_ok(K) || T == 0 || R == 0 || K == 0 ||
        !keep_ok(keep) || (aligned != 0 && aligned != 1) || sm_count < 1 || tile_tokens == nullptr || tile_rows == nullptr || splits == nullptr)
        return VNM_ERR_INVALID_ARG;
    vnm::ProductArgs p{};
    p.kind = static_cast<vnm::ProductKind>(kind);
    p.T = T;
    p.R = R;
    p.K = K;
    p.x[0].transposed = x_transposed != 0;
    p.w[0].transposed = w_transposed != 0;
    p.keep = kind_of(keep);
    if (!aligned) p.y[0] = reinterpret_cast<void*>(2);  // (never followed)
    p.skip_stage = -1;
    const vnm::TilePlan plan = vnm::plan_product(p, sm_count);
    *tile_tokens = plan.bn;
    *tile_rows = plan.tile_n;
    *splits = plan.splits;
    return VNM_OK;
}

vnm_status vnm_gated_linear(const void* X, int64_t ld_x, const void* Wg, int64_t ld_wg, const void* Wu, int64_t ld_wu,
                            vnm_dtype type, int64_t T, int64_t F, int64_t K, vnm_activation act, void* Y, int64_t ld_y,
                            vnm_keep keep, void* g, int64_t ld_g, float* g_scale, int64_t gs_rs, int64_t gs_cs, void* u,
                            int64_t ld_u, float* u_scale, int64_t us_rs, int64_t us_cs, int32_t* status,
                            vnm_stream_t stream) {
    return gated_linear(X, ld_x, Wg, ld_wg, Wu, ld_wu, type, T, F, K, act, Y, ld_y, keep, g, ld_g, g_scale, gs_rs, gs_cs, u, ld_u,
                        u_scale, us_rs, us_cs, status, -1, stream);
}

vnm_status vnm_testing_gated_linear_skip_stage(const void* X, int64_t ld_x, const void* Wg, int64_t ld_wg, const void* Wu,
                                               int64_t ld_wu, vnm_dtype type, int64_t T, int64_t F, int64_t K,
                                               vnm_activation act, void* Y, int64_t ld_y, vnm_keep keep, void* g, int64_t ld_g,
                                               float* g_scale, int64_t gs_rs, int64_t gs_cs, void* u, int64_t ld_u,
                                               float* u_scale, int64_t us_rs, int64_t us_cs, int32_t* status,
                                               int32_t skip_stage, vnm_stream_t stream) {
    if (skip_stage < 0) return VNM_ERR_INVALID_ARG;
    return gated_linear(X, ld_x, Wg, ld_wg, Wu, ld_wu, type, T, F, K, act, Y, ld_y, keep, g, ld_g, g_scale, gs_rs, gs_cs, u, ld_u,
                        u_scale, us_rs, us_cs, status, skip_stage, stream);
}

vnm_status vnm_gated_linear_backward_workspace_size(int64_t T, int64_t F, size_t* bytes) {
    if (bytes == nullptr || !size_ok(T) || !size_ok(F)) return VNM_ERR_INVALID_ARG;
    *bytes = 4 * static_cast<size_t>(T) * static_cast<size_t>(padded(F));  // dG and dU side by side
    return VNM_OK;
}

vnm_status vnm_gated_linear_backward(const void* dY, int64_t ld_dy, const void* X, int64_t ld_x, const void* Wg,
                                     int64_t ld_wg, const void* Wu, int64_t ld_wu, vnm_dtype type, int64_t T, int64_t F,
                                     int64_t K, vnm_activation act, vnm_keep keep, const void* g, int64_t ld_g,
                                     const float* g_scale, int64_t gs_rs, int64_t gs_cs, const void* u, int64_t ld_u,
                                     const float* u_scale, int64_t us_rs, int64_t us_cs, void* dX, int64_t ld_dx, void* dWg,
                                     void* dWu, int64_t ld_dw, vnm_dtype w_type, int32_t accumulate, void* H, int64_t ld_h,
                                     void* workspace, size_t workspace_bytes, int32_t* status, vnm_stream_t stream) {
    return gated_linear_backward(dY, ld_dy, X, ld_x, Wg, ld_wg, Wu, ld_wu, type, T, F, K, act, keep, g, ld_g, g_scale, gs_rs, gs_cs, u,
                                 ld_u, u_scale, us_rs, us_cs, dX, ld_dx, dWg, dWu, ld_dw, w_type, accumulate, H, ld_h, workspace,
                                 workspace_bytes, status, -1, -1, stream);
}

vnm_status vnm_testing_gated_linear_backward_skip_stage(const void* dY, int64_t ld_dy, const void* X, int64_t ld_x, const void* Wg,
                                                        int64_t ld_wg, const void* Wu, int64_t ld_wu, vnm_dtype type, int64_t T, int64_t F,
                                                        int64_t K, vnm_activation act, vnm_keep keep, const void* g, int64_t ld_g,
                                                        const float* g_scale, int64_t gs_rs, int64_t gs_cs, const void* u, int64_t ld_u,
                                                        const float* u_scale, int64_t us_rs, int64_t us_cs, void* dX, int64_t ld_dx, void* dWg,
                                                        void* dWu, int64_t ld_dw, vnm_dtype w_type, int32_t accumulate, void* H, int64_t ld_h,
                                                        void* workspace, size_t workspace_bytes, int32_t* status,
                                                        int32_t skip_dx, int32_t skip_dw, vnm_stream_t stream) {
    if (skip_dx < -1 || skip_dw < -1) return VNM_ERR_INVALID_ARG;
    return gated_linear_backward(dY, ld_dy, X, ld_x, Wg, ld_wg, Wu, ld_wu, type, T, F, K, act, keep, g, ld_g, g_scale, gs_rs, gs_cs, u,
                                 ld_u, u_scale, us_rs, us_cs, dX, ld_dx, dWg, dWu, ld_dw, w_type, accumulate, H, ld_h, workspace,
                                 workspace_bytes, status, skip_dx,
                                 skip_dw, stream);
}

vnm_status vnm_dense_get_status(vnm_stream_t stream) {
    int code = 0;
    if (vnm::take_product_status(&code, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return VNM_ERR_CUDA;
    return static_cast<vnm_status>(code);
}

}  // extern "C"

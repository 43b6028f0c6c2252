// Host side of the dense neighbours of a pruned layer (include/vnm.h): argument
// checks of the RMS norm, its backward pass, the block-scaled 8-bit quantiser
// and the 8-bit Linear layer. Every check runs before anything is enqueued.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "vnm_dense.h"
#include "vnm_testing.h"

namespace {

constexpr int64_t kMaxSize = int64_t(1) << 31;  // TMA coordinates are int32
constexpr int kMaxDevices = 64;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Element size of a vnm_dtype, 0 for anything else.
size_t size_of(vnm_dtype t) { return t == VNM_F32 ? 4 : t == VNM_F16 || t == VNM_BF16 ? 2 : 0; }

bool fp8_ok(vnm_fp8 t) { return t == VNM_E4M3 || t == VNM_E5M2; }

// A matrix that may be absent: aligned to its elements, rows of `cols`.
bool optional_ok(const void* p, int64_t ld, int64_t cols, size_t elem) {
    return p == nullptr || (aligned(p, elem) && ld >= std::max<int64_t>(cols, 1));
}

bool matrix_ok(const void* p, int64_t ld, int64_t cols, size_t elem) {
    return p != nullptr && optional_ok(p, ld, cols, elem);
}

bool size_ok(int64_t n) { return n >= 0 && n <= kMaxSize; }

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

vnm_status fp8_linear(const void* xq, int64_t ld_x, vnm_fp8 x_type, const float* x_scale, int64_t xs_rs,
                      int64_t xs_cs, const void* wq, int64_t ld_w, vnm_fp8 w_type, const float* w_scale,
                      int64_t ws_rs, int64_t ws_cs, int32_t w_block_rows, int64_t T, int64_t R, int64_t K,
                      const void* bias, vnm_dtype bias_type, vnm_activation act, void* Y, int64_t ld_y,
                      vnm_dtype y_type, int32_t* status, int skip_stage, vnm_stream_t stream) {
    const size_t e = size_of(y_type);
    if (e == 0 || !size_ok(T) || !size_ok(R) || !size_ok(K) || !fp8_ok(x_type) || !fp8_ok(w_type) ||
        (w_block_rows != 1 && w_block_rows != vnm::kGroup))
        return VNM_ERR_INVALID_ARG;
    if (act != VNM_ACT_NONE && act != VNM_ACT_RELU && act != VNM_ACT_GELU) return VNM_ERR_INVALID_ARG;
    if (bias != nullptr && (size_of(bias_type) == 0 || !aligned(bias, size_of(bias_type)))) return VNM_ERR_INVALID_ARG;
    if (!aligned(status, 4)) return VNM_ERR_INVALID_ARG;
    if (T == 0 || R == 0) return VNM_OK;
    if (!matrix_ok(Y, ld_y, R, e)) return VNM_ERR_INVALID_ARG;
    // one row has no pitch
    if (T == 1 && ld_x >= K) ld_x = (K + 15) / 16 * 16;
    if (R == 1 && ld_w >= K) ld_w = (K + 15) / 16 * 16;
    if (K > 0 && (!matrix_ok(xq, ld_x, K, 16) || !matrix_ok(wq, ld_w, K, 16) || ld_x % 16 != 0 || ld_w % 16 != 0 ||
                  x_scale == nullptr || w_scale == nullptr || !aligned(x_scale, 4) || !aligned(w_scale, 4)))
        return VNM_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms == 0) return VNM_ERR_CUDA;
    const vnm::ScaleView xs{x_scale, xs_rs, xs_cs, 0};
    const vnm::ScaleView ws{w_scale, ws_rs, ws_cs, w_block_rows == 1 ? 0 : 7};
    return launched(vnm::launch_fp8_linear(xq, ld_x, x_type == VNM_E5M2, xs, wq, ld_w, w_type == VNM_E5M2, ws, T, R, K,
                                           bias, bias_type, static_cast<int>(act), Y, ld_y, y_type, status,
                                           skip_stage, sms,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

vnm_status vnm_rmsnorm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual, const void* weight,
                       float eps, int64_t T, int64_t D, vnm_dtype type, void* h, int64_t ld_h, void* y, int64_t ld_y,
                       float* rstd, void* q, int64_t ld_q, vnm_fp8 q_type, float* q_scale, int64_t s_rs, int64_t s_cs,
                       vnm_stream_t stream) {
    const size_t e = size_of(type);
    if (e == 0 || !size_ok(T) || !size_ok(D) || !(eps >= 0.f) || std::isinf(eps)) return VNM_ERR_INVALID_ARG;
    if (q != nullptr && !fp8_ok(q_type)) return VNM_ERR_INVALID_ARG;
    if (T == 0 || D == 0) return VNM_OK;
    if (!matrix_ok(x, ld_x, D, e) || !optional_ok(residual, ld_residual, D, e) || !optional_ok(h, ld_h, D, e) ||
        !optional_ok(y, ld_y, D, e) || !optional_ok(q, ld_q, D, 1) || !aligned(weight, e) || !aligned(rstd, 4) ||
        !aligned(q_scale, 4))
        return VNM_ERR_INVALID_ARG;
    if ((y == nullptr && q == nullptr) || (q == nullptr) != (q_scale == nullptr) ||
        (h != nullptr && residual == nullptr))
        return VNM_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms == 0) return VNM_ERR_CUDA;
    vnm::RmsNormArgs a{};
    a.x = x;
    a.res = residual;
    a.w = weight;
    a.h = h;
    a.y = y;
    a.q = q;
    a.rstd = rstd;
    a.s = q_scale;
    a.ld_x = ld_x;
    a.ld_res = ld_residual;
    a.ld_h = ld_h;
    a.ld_y = ld_y;
    a.ld_q = ld_q;
    a.s_rs = s_rs;
    a.s_cs = s_cs;
    a.T = T;
    a.D = D;
    a.eps = eps;
    a.e5m2 = q_type == VNM_E5M2;
    return launched(vnm::launch_rmsnorm(a, type, sms, reinterpret_cast<cudaStream_t>(stream)));
}

vnm_status vnm_rmsnorm_backward_workspace_size(int64_t T, int64_t D, size_t* bytes) {
    if (bytes == nullptr || !size_ok(T) || !size_ok(D)) return VNM_ERR_INVALID_ARG;
    *bytes = static_cast<size_t>(vnm::rmsnorm_grad_parts(T, D)) * static_cast<size_t>(D) * sizeof(float);
    return VNM_OK;
}

vnm_status vnm_rmsnorm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h, const void* weight,
                                const float* rstd, const void* dresidual, int64_t ld_dresidual, int64_t T, int64_t D,
                                vnm_dtype type, void* dh, int64_t ld_dh, float* dweight, void* workspace,
                                size_t workspace_bytes, vnm_stream_t stream) {
    const size_t e = size_of(type);
    if (e == 0 || !size_ok(T) || !size_ok(D)) return VNM_ERR_INVALID_ARG;
    if (D == 0) return VNM_OK;
    if (!aligned(dweight, 4) || !aligned(rstd, 4) || !aligned(weight, e)) return VNM_ERR_INVALID_ARG;
    if (T > 0) {
        if (!matrix_ok(dy, ld_dy, D, e) || !matrix_ok(h, ld_h, D, e) || rstd == nullptr ||
            !optional_ok(dresidual, ld_dresidual, D, e) || !optional_ok(dh, ld_dh, D, e) ||
            (dh == nullptr && dweight == nullptr))
            return VNM_ERR_INVALID_ARG;
        size_t need = 0;
        if (vnm_rmsnorm_backward_workspace_size(T, D, &need) != VNM_OK) return VNM_ERR_INVALID_ARG;
        if (dweight != nullptr && (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < need))
            return VNM_ERR_INVALID_ARG;
    }
    if (sm_count() == 0) return VNM_ERR_CUDA;
    vnm::RmsNormGradArgs a{};
    a.dy = dy;
    a.h = h;
    a.w = weight;
    a.dres = dresidual;
    a.rstd = rstd;
    a.dh = dh;
    a.dw = dweight;
    a.partial = static_cast<float*>(workspace);
    a.ld_dy = ld_dy;
    a.ld_h = ld_h;
    a.ld_dres = ld_dresidual;
    a.ld_dh = ld_dh;
    a.T = T;
    a.D = D;
    return launched(vnm::launch_rmsnorm_grad(a, type, reinterpret_cast<cudaStream_t>(stream)));
}

vnm_status vnm_fp8_quantize(const void* X, int64_t ld_x, int64_t R, int64_t C, vnm_dtype type, int32_t block_rows,
                            vnm_fp8 q_type, void* q, int64_t ld_q, float* s, int64_t s_rs, int64_t s_cs, void* qt,
                            int64_t ld_qt, float* st, int64_t st_rs, int64_t st_cs, vnm_stream_t stream) {
    const size_t e = size_of(type);
    if (e == 0 || !size_ok(R) || !size_ok(C) || !fp8_ok(q_type) || (block_rows != 1 && block_rows != vnm::kGroup))
        return VNM_ERR_INVALID_ARG;
    if (R == 0 || C == 0) return VNM_OK;
    if (!matrix_ok(X, ld_x, C, e) || !optional_ok(q, ld_q, C, 1) || !optional_ok(qt, ld_qt, R, 1) || !aligned(s, 4) ||
        !aligned(st, 4))
        return VNM_ERR_INVALID_ARG;
    if ((q == nullptr) != (s == nullptr) || (qt == nullptr) != (st == nullptr) || (q == nullptr && qt == nullptr))
        return VNM_ERR_INVALID_ARG;
    if (sm_count() == 0) return VNM_ERR_CUDA;
    vnm::QuantArgs a{};
    a.x = X;
    a.q = static_cast<uint8_t*>(q);
    a.qt = static_cast<uint8_t*>(qt);
    a.s = s;
    a.st = st;
    a.ld_x = ld_x;
    a.ld_q = ld_q;
    a.ld_qt = ld_qt;
    a.s_rs = s_rs;
    a.s_cs = s_cs;
    a.st_rs = st_rs;
    a.st_cs = st_cs;
    a.R = R;
    a.C = C;
    a.block = block_rows != 1;
    a.e5m2 = q_type == VNM_E5M2;
    return launched(vnm::launch_fp8_quantize(a, type, reinterpret_cast<cudaStream_t>(stream)));
}

vnm_status vnm_fp8_linear(const void* xq, int64_t ld_x, vnm_fp8 x_type, const float* x_scale, int64_t xs_rs,
                          int64_t xs_cs, const void* wq, int64_t ld_w, vnm_fp8 w_type, const float* w_scale,
                          int64_t ws_rs, int64_t ws_cs, int32_t w_block_rows, int64_t T, int64_t R, int64_t K,
                          const void* bias, vnm_dtype bias_type, vnm_activation act, void* Y, int64_t ld_y,
                          vnm_dtype y_type, int32_t* status, vnm_stream_t stream) {
    return fp8_linear(xq, ld_x, x_type, x_scale, xs_rs, xs_cs, wq, ld_w, w_type, w_scale, ws_rs, ws_cs, w_block_rows,
                      T, R, K, bias, bias_type, act, Y, ld_y, y_type, status, -1, stream);
}

vnm_status vnm_testing_fp8_linear_skip_stage(const void* xq, int64_t ld_x, vnm_fp8 x_type, const float* x_scale,
                                             int64_t xs_rs, int64_t xs_cs, const void* wq, int64_t ld_w,
                                             vnm_fp8 w_type, const float* w_scale, int64_t ws_rs, int64_t ws_cs,
                                             int32_t w_block_rows, int64_t T, int64_t R, int64_t K, const void* bias,
                                             vnm_dtype bias_type, vnm_activation act, void* Y, int64_t ld_y,
                                             vnm_dtype y_type, int32_t* status, int32_t skip_stage,
                                             vnm_stream_t stream) {
    if (skip_stage < 0 || status == nullptr) return VNM_ERR_INVALID_ARG;
    return fp8_linear(xq, ld_x, x_type, x_scale, xs_rs, xs_cs, wq, ld_w, w_type, w_scale, ws_rs, ws_cs, w_block_rows,
                      T, R, K, bias, bias_type, act, Y, ld_y, y_type, status, skip_stage, stream);
}

vnm_status vnm_testing_fp8_linear_skip_stage_no_status(const void* xq, int64_t ld_x, vnm_fp8 x_type,
                                                       const float* x_scale, int64_t xs_rs, int64_t xs_cs,
                                                       const void* wq, int64_t ld_w, vnm_fp8 w_type,
                                                       const float* w_scale, int64_t ws_rs, int64_t ws_cs,
                                                       int32_t w_block_rows, int64_t T, int64_t R, int64_t K, void* Y,
                                                       int64_t ld_y, vnm_dtype y_type, int32_t skip_stage,
                                                       vnm_stream_t stream) {
    if (skip_stage < 0) return VNM_ERR_INVALID_ARG;
    return fp8_linear(xq, ld_x, x_type, x_scale, xs_rs, xs_cs, wq, ld_w, w_type, w_scale, ws_rs, ws_cs, w_block_rows,
                      T, R, K, nullptr, VNM_F32, VNM_ACT_NONE, Y, ld_y, y_type, nullptr, skip_stage, stream);
}

vnm_status vnm_testing_fp8_linear_plan(int64_t T, int64_t R, int64_t K, int32_t w_block_rows, int32_t sm_count,
                                       int32_t* tile_tokens, int32_t* splits) {
    if (!size_ok(T) || !size_ok(R) || !size_ok(K) || T == 0 || R == 0 || K == 0 || sm_count < 1 ||
        (w_block_rows != 1 && w_block_rows != vnm::kGroup) || tile_tokens == nullptr || splits == nullptr)
        return VNM_ERR_INVALID_ARG;
    vnm::fp8_linear_plan(T, R, K, w_block_rows != 1, sm_count, tile_tokens, splits);
    return VNM_OK;
}

vnm_status vnm_fp8_linear_get_status(vnm_stream_t stream) {
    int code = 0;
    if (vnm::take_fp8_linear_status(&code, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return VNM_ERR_CUDA;
    return static_cast<vnm_status>(code);
}

}  // extern "C"

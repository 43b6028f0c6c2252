// Internal declarations of the dense 16-bit layers: the product with bias,
// activation and residual, the gated pair of projections and its backward pass
// (kernels in dense_linear.cu, dense_decode.cu and gated_grad.cu, argument checks in
// dense16_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/vnm.h"

namespace vnm {

// Launches that may start while the stream's previous grid drains (the kernels wait for its end by
// themselves before they touch global memory): it hides a launch's latency, about 2 us of a chain of small calls.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), int64_t blocks, int threads, size_t smem, int cluster, cudaStream_t stream,
                         const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A 16-bit operand of a product, rows x K: stored row-major (a row's K elements
// are neighbours), or transposed (an element of K is a row of the storage).
struct Operand16 {
    const void* p;
    int64_t ld;
    bool transposed;
};

// What the two halves of a product of two operands are.
enum ProductKind {
    kOneProduct,   // y[0] = x[0] . w[0]^T
    kSumOfTwo,     // y[0] = x[0] . w[0]^T + x[1] . w[1]^T
    kTwoByRows,    // y[i] = x[i] . w[0]^T
    kGatedPair     // y[0] = act(x[0] . w[0]^T) * (x[0] . w[1]^T)
};

// How a gated pair's two products are kept for the backward pass.
enum KeepKind { kKeepNone, kKeep16, kKeep8 };

struct Kept {
    void* p;        // T x R: the inputs' type, or fp8
    int64_t ld;
    float* s;       // kKeep8: a scale for each 128 columns of a row
    int64_t s_rs, s_cs;
};

struct ProductArgs {
    ProductKind kind;
    int64_t T, R, K;  // of one product
    bool bf16;
    Operand16 x[2], w[2];
    void* y[2];
    int64_t ld_y;
    vnm_dtype y_type;
    const void* bias;
    vnm_dtype bias_type;
    int act;
    const void* residual[2];
    int64_t ld_residual;
    KeepKind keep;
    bool e5m2;
    Kept g, u;
    // Two products that do not need each other, launched one after the other: the second starts its work when all CTAs of the
    // first run (and have seen the end of what came before it), and waits for the first's end at its own.
    bool beside, next_beside;  // this is the second; the first (both of K >= 1)
    int* status;
    int skip_stage;  // tests of the bounded waits only (-1: none)
};

// How a product (K >= 1) is tiled: pairs of CTAs (bn = 0), tile_n rows of W a tile (both of a gated pair's
// together), K over `splits` pairs of a cluster; tiles of bn = 16, 32, 64 or 128 tokens, K over `splits` CTAs of a cluster; or
// the few-token kernel.
struct TilePlan {
    int bn, splits, tile_n;
};
constexpr int kFewPlan = 8;     // bn of the few-token kernel
constexpr int kFewTokens = 16;  // the most that it takes
TilePlan plan_product(const ProductArgs& a, int sm_count);
cudaError_t launch_product(const ProductArgs& a, const TilePlan& plan, int sm_count, cudaStream_t stream);

// The first error that products without status words recorded on the current device, and clears it.
cudaError_t take_product_status(int* code, cudaStream_t stream);

// The same product for up to kFewTokens tokens: kOneProduct or kGatedPair without 8-bit
// checkpoints, both operands row-major.
cudaError_t launch_few_tokens(const ProductArgs& a, int sm_count, cudaStream_t stream);

// dg = dy * u * act'(g), du = dy * act(g), h = act(g) * u, element by element.
struct GatedGradArgs {
    int64_t T, F;
    bool bf16;
    int act;
    const void* dy;
    int64_t ld_dy;
    KeepKind keep;
    bool e5m2;
    Kept g, u;  // (read)
    void *dg, *du;
    int64_t ld_d;  // of both
    void* h;
    int64_t ld_h;
};
cudaError_t launch_gated_grad(const GatedGradArgs& a, int sm_count, cudaStream_t stream);

}  // namespace vnm

/*
 * Test support for libvnm: entry points that only tests call. The paper has
 * no counterpart; they exercise this library's own failure handling.
 */
#ifndef VNM_TESTING_H
#define VNM_TESTING_H

#include "vnm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * vnm_spmm on the tensor-core path, except that the first CTA never issues
 * the TMA loads of its pipeline stage number `skip_stage` (counted over the
 * tiles it takes). The waits on that stage are bounded (about 1 s): they run
 * out, every role of that CTA winds down, copies and MMAs already issued are
 * drained, TMEM is freed and VNM_ERR_TIMEOUT is recorded in the matrix's
 * status word (read it with vnm_get_status). C is then unspecified; the
 * device stays usable. Arguments as in vnm_spmm.
 * Errors: as vnm_spmm, plus VNM_ERR_UNSUPPORTED when the plan for this
 * product is not the tensor-core path or skip_stage < 0.
 */
vnm_status vnm_testing_spmm_skip_stage(vnm_matrix A, const void* B, int64_t ld_b, int64_t N, void* C,
                                       int64_t ld_c, vnm_dtype c_type, void* workspace, size_t workspace_bytes,
                                       int32_t skip_stage, vnm_stream_t stream);

/*
 * vnm_fp8_linear, except that the first CTA never issues the TMA loads of its
 * pipeline stage number `skip_stage` (counted over the tiles it takes): its
 * bounded waits run out after about 1 s, VNM_ERR_TIMEOUT goes to `status`
 * (needed here), and Y is unspecified; the device stays usable.
 * Errors: as vnm_fp8_linear, plus VNM_ERR_INVALID_ARG for skip_stage < 0 or no status.
 */
vnm_status vnm_testing_fp8_linear_skip_stage(const void* xq, int64_t ld_x, vnm_fp8 x_type, const float* x_scale,
                                             int64_t xs_rs, int64_t xs_cs, const void* wq, int64_t ld_w,
                                             vnm_fp8 w_type, const float* w_scale, int64_t ws_rs, int64_t ws_cs,
                                             int32_t w_block_rows, int64_t T, int64_t R, int64_t K, const void* bias,
                                             vnm_dtype bias_type, vnm_activation act, void* Y, int64_t ld_y,
                                             vnm_dtype y_type, int32_t* status, int32_t skip_stage,
                                             vnm_stream_t stream);

/* The same without status words, bias and activation (vnm_fp8_linear_get_status reads what it records). */
vnm_status vnm_testing_fp8_linear_skip_stage_no_status(const void* xq, int64_t ld_x, vnm_fp8 x_type,
                                                       const float* x_scale, int64_t xs_rs, int64_t xs_cs,
                                                       const void* wq, int64_t ld_w, vnm_fp8 w_type,
                                                       const float* w_scale, int64_t ws_rs, int64_t ws_cs,
                                                       int32_t w_block_rows, int64_t T, int64_t R, int64_t K, void* Y,
                                                       int64_t ld_y, vnm_dtype y_type, int32_t skip_stage,
                                                       vnm_stream_t stream);

/*
 * How vnm_fp8_linear takes a product on a GPU of sm_count SMs (host only): tiles of
 * *tile_tokens = 16, 32, 64 or 128 tokens with K over *splits CTAs of a cluster; 0: pairs of
 * CTAs, 256 x 256 outputs; 8: the few-token kernel.
 * Errors: VNM_ERR_INVALID_ARG (sizes below 1, w_block_rows, null pointers).
 */
vnm_status vnm_testing_fp8_linear_plan(int64_t T, int64_t R, int64_t K, int32_t w_block_rows, int32_t sm_count,
                                       int32_t* tile_tokens, int32_t* splits);

#ifdef __cplusplus
}
#endif

#endif /* VNM_TESTING_H */

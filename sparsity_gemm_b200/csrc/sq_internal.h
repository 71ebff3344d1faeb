// Host-side declarations shared by the library's translation units.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/sharq.h"

namespace sq {

struct LaunchCtx {
    cudaStream_t stream;
    unsigned *status;      // device status word
    uint64_t wait_ns;      // bound of every device-side wait
    int num_sms;
    int launches;          // kernels enqueued by the current entry point
};

// norm: 0 = LayerNorm, 1 = RMSNorm (beta must be NULL).
sharq_status launch_prepare(LaunchCtx &ctx, const sharq_prep &P, const void *x, const void *gamma,
                            const void *beta, float eps, int norm);
// The pair-wise 4:8 mode (P from prep_layout_sparse).
sharq_status launch_prepare_sparse(LaunchCtx &ctx, const sharq_prep &P, const void *x, const void *gamma,
                                   const void *beta, float eps, int norm);
// x_out = RN16(h + d), then the preparation of x_out (P from prep_layout).
sharq_status launch_prepare_add(LaunchCtx &ctx, const sharq_prep &P, const void *h, const void *d, void *x_out,
                                const void *gamma, const void *beta, float eps, int norm);
sharq_status launch_prepare_grouped(LaunchCtx &ctx, const sharq_prep &P, const void *x, int64_t rows,
                                    const int32_t *offsets, int32_t groups, const void *gamma, const void *beta,
                                    float eps, int norm);
sharq_status launch_quantize_weight(LaunchCtx &ctx, const sharq_wq &W, const void *w, int64_t groups,
                                   int64_t gstride);
sharq_status launch_quantize_weight_fused(LaunchCtx &ctx, const sharq_wq &W, const void *w, const int64_t *seg_rows,
                                         int n_segs);
// bias: fp16 [n_out] or NULL
sharq_status launch_linear(LaunchCtx &ctx, const sharq_prep &P, const sharq_wq &W, const void *bias, void *out);
sharq_status launch_linear_grouped(LaunchCtx &ctx, const sharq_prep &P, const sharq_wq &W, const int32_t *offsets,
                                   int32_t groups, int64_t rows, int64_t w_gstride, void *out);
sharq_status launch_gather(LaunchCtx &ctx, const sharq_prep &S, const int32_t *row_idx, const int32_t *offsets,
                           int32_t groups, int64_t rows, const sharq_prep &D);
sharq_status launch_wait_probe(LaunchCtx &ctx, uint64_t limit_ns);
// 2-D map of 16-bit elements [rows][cols] with a row stride in bytes; box =
// 64 elements x box_rows, 128-byte swizzle.
bool make_row_map(CUtensorMap *tm, const void *base, uint64_t cols, uint64_t rows, uint64_t ld_bytes, uint32_t box_rows);
// Records the kernel count that sharq_last_launch_count reports.
void note_launches(int n);
sharq_status launch_div_check(LaunchCtx &ctx, uint64_t count, uint64_t seed, uint64_t *mismatches, float *examples);

// Operators in 16 or 32 bits (norm.cu, route.cu, lora.cu). vec16: rows and
// buffers allow 16-byte accesses.
sharq_status launch_layer_norm(LaunchCtx &ctx, const void *x, int64_t rows, int64_t k, const void *w, const void *b,
                               float eps, int norm, int dtype, void *y, float *mean, float *rstd, bool vec16);
// Workspace of the backward pass in bytes; needed for weight gradients, and
// in any case where it takes more than one pass over a row.
int64_t norm_bwd_bytes(int64_t rows, int64_t k);
bool norm_bwd_one_pass(int64_t k);
sharq_status launch_layer_norm_backward(LaunchCtx &ctx, const void *dy, const void *x, int64_t rows, int64_t k,
                                        const void *w, const float *mean, const float *rstd, int norm, int dtype,
                                        void *dx, float *dw, float *db, void *ws, bool vec16);
sharq_status launch_route(LaunchCtx &ctx, const void *ids, int id_bytes, int64_t tokens, int64_t top_k, int64_t groups,
                          int32_t *offsets, int32_t *rows, int32_t *slots);
sharq_status launch_permute(LaunchCtx &ctx, const void *x, int64_t tokens, int64_t k, const int32_t *slots, int64_t top_k,
                            const int32_t *offsets, int64_t groups, int dtype, void *out, bool vec16);
sharq_status launch_combine(LaunchCtx &ctx, const void *y, int64_t n_rows, int64_t tokens, int64_t k,
                            const int32_t *slots, const float *weights, int64_t top_k, const void *residual, int dtype,
                            void *out, bool vec16);
sharq_status launch_combine_backward(LaunchCtx &ctx, const void *dout, const void *y, int64_t n_rows, int64_t tokens,
                                     int64_t k, const int32_t *slots, const float *weights, int64_t top_k,
                                     const int32_t *offsets, int64_t groups, int dtype, void *dy, float *dweights,
                                     bool vec16);
sharq_status launch_lora(LaunchCtx &ctx, const void *x, int64_t ldx, int64_t m, int64_t k, const void *a, const void *b,
                         int64_t n, int64_t rank, int64_t groups, const float *scales, const int32_t *offsets,
                         const int32_t *rows, const int32_t *slots, int dtype, const void *base, int64_t ldbase, void *out,
                         int64_t ldo, void *ws);
// Workspace of launch_lora in bytes (0: none).
int64_t lora_ws_bytes(int64_t m, int64_t rank, int64_t groups);

}  // namespace sq

#define SQ_CUDA_TRY(expr)                                         \
    do {                                                          \
        cudaError_t _e = (expr);                                  \
        if (_e != cudaSuccess) return SHARQ_ERR_CUDA;             \
    } while (0)

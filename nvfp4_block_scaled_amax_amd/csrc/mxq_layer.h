// mxq_layer.h -- internal launchers of the layer operators around the
// quantizers (routing, combine, few-token NVFP4 products, attention over an
// NVFP4 cache) behind the C ABI (mxq_api.cpp).  Arguments have been
// validated by the caller; each launcher enqueues on `stream` and returns the
// launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq.h"

namespace mxq {

// Routing keeps a token's experts in the registers of one wavefront.
constexpr int64_t MAX_EXPERTS = 1024;
constexpr int64_t MAX_TOP_K = 64;
// The router's maps hold 32-bit row numbers while they are formed.
constexpr int64_t MAX_COPIES = (int64_t)1 << 30;

int64_t moe_route_workspace(int64_t n_tokens, int64_t n_experts);

hipError_t launch_moe_route(bool bf16, const void *logits, const float *bias, int64_t n_tokens,
                            int64_t n_experts, const mxq_route_params &p, float *weights,
                            int64_t *experts, int64_t *token_rows, int64_t *row_tokens,
                            int64_t *seg_offsets, void *workspace, hipStream_t stream);

hipError_t launch_moe_route_backward(bool bf16, const float *d_weights, const void *logits,
                                     const int64_t *experts, int64_t n_tokens, int64_t n_experts,
                                     int64_t top_k, bool sigmoid, bool renorm, float scale,
                                     void *d_logits, hipStream_t stream);

hipError_t launch_moe_combine(bool bf16, const void *rows, int64_t total_rows,
                              const int64_t *token_rows, const float *weights, int64_t n_tokens,
                              int64_t top_k, int64_t cols, bool bf16_out, void *out,
                              hipStream_t stream);

hipError_t launch_moe_combine_backward(bool bf16, const void *d_out, const void *rows,
                                       int64_t total_rows, const int64_t *token_rows,
                                       const float *weights, const int64_t *seg_offsets,
                                       int64_t n_groups, int64_t n_tokens, int64_t top_k,
                                       int64_t cols, void *d_rows, float *d_weights,
                                       hipStream_t stream);

// An activation operand: fmt is an mxq_x_format; NVFP4 has block scales and
// one FP32 scale per row.
struct ActX {
    int fmt;
    const void *x;
    const uint8_t *bs;
    const float *s;
};
// One NVFP4 weight tensor [.][N][K]; scale of row n of expert e is
// s[(e * N + n) / rows_per_scale] (experts: one scale each, rows_per_scale N).
struct WeightB {
    const uint8_t *codes, *bs;
};

hipError_t launch_nvfp4_matvec(const ActX &x, const WeightB &b, const float *scales,
                               int64_t rows_per_scale, int64_t M, int64_t N, int64_t K,
                               bool bf16_out, void *c, hipStream_t stream);

// up.codes == nullptr: C[r] = scale (x[r] W_e^T) on expert-sorted rows.
// Otherwise x has n_tokens rows, row r of the layout is row row_tokens[r] of
// x, and C[r] = silu(scale x W_e^T) (scale x U_e^T).
hipError_t launch_nvfp4_expert_matvec(const ActX &x, int64_t n_tokens, const int64_t *row_tokens,
                                      const int64_t *seg_offsets, int64_t n_groups,
                                      int64_t total_rows, const WeightB &w, const WeightB &up,
                                      const float *scales, int64_t N, int64_t K, bool bf16_out,
                                      void *c, hipStream_t stream);

// The expert product's launch fits one grid.
bool expert_grid_ok(int64_t n_groups, int64_t total_rows, int64_t N);

struct AttnArgs {
    const uint16_t *q;
    const uint8_t *k, *kbs;
    const float *ks;
    const uint8_t *v, *vbs;
    const float *vs;
    const int64_t *block_table, *seq_lens;
    int64_t n_seqs, q_len, n_heads, n_kv_heads, head_dim, n_pages, page_size, max_pages;
    float scale;
    bool causal;
    int64_t window;
    uint16_t *out;
    float *lse;
};
int64_t nvfp4_attention_workspace(int64_t n_seqs, int64_t q_len, int64_t n_heads,
                                  int64_t n_kv_heads, int64_t head_dim, int64_t max_keys);
hipError_t launch_nvfp4_attention(const AttnArgs &a, void *workspace, hipStream_t stream);

}  // namespace mxq

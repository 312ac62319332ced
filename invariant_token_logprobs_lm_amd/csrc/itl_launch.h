// Host-side launchers of the library's kernels. Arguments are already
// validated by the C ABI layer (api.hip); these only size grids and launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace itl {

// Workspace layout of the forward: per-(slice, token) partial (max, sumexp)
// pairs, then the per-token sampled logit.
size_t lmhead_workspace_bytes(long long n_tok, long long vocab);

// logits (nullable): also write z[t, v] at logits[t * ld + v] for v < vocab.
hipError_t launch_lmhead_logprob(const void* H, const void* W, int dtype, int n_tok, int d, int vocab,
                                 const int32_t* tokens, float* logprob, float* lse, float* logits, long long ld,
                                 void* workspace, hipStream_t stream);

// Merge each token's n_parts (max, sumexp) partials (slice-major) into its
// logprob (z_y - lse) and lse (nullable).
hipError_t launch_lse_combine(const float2* part, const float* zy, int n_tok, int n_parts, float* logprob, float* lse,
                              hipStream_t stream);

hipError_t launch_group_advantage(const float* rewards, const int32_t* group_offsets, int n_groups,
                                  int n_resp, float* advantages, hipStream_t stream);

// Workspace of the loss: the fp64 per-response losses, the fp64 segment sums
// of responses longer than one segment, and the fp64 partial sums of the mean.
size_t loss_workspace_bytes(long long n_tok, long long n_resp);

hipError_t launch_reinforce_zero_loss(const float* logprob, const float* rollout_logprob,
                                      const float* advantages, const int64_t* resp_offsets, int n_resp,
                                      long long n_tok, float* resp_loss, float* loss, float* coef,
                                      void* workspace, hipStream_t stream);

size_t backward_workspace_bytes(long long n_tok, long long d, long long vocab, int dtype);

// Tokens per chunk of the backward (a multiple of the token block). dW's sum
// over tokens is carried across chunks in this order, so it is part of dW's
// bits; the build info reports it.
constexpr int kBwdChunkTokens = 16384;

// Largest vocabulary the backward handles (its padded rows must be
// addressable by 32-bit buffer offsets over 256-row tiles).
constexpr long long kBwdMaxVocab = (1LL << 31) / (256LL * 4) - 256;

// The backward's sampled term: dW[v] = sum over tokens t with y_t = v of
// coef[t] H[t] for every row v (zeros where no token samples v), in the
// fixed order of sampled_plan.h.
size_t sampled_dw_workspace_bytes(long long n_tok, long long d, long long vocab);
hipError_t launch_sampled_dw(const void* H, int dtype, int n_tok, int d, int vocab, const int32_t* tokens,
                             const float* coef, float* dW, void* workspace, hipStream_t stream);

// logits (nullable): the forward's z[t, v] at logits[t * ld + v]; the dlogits
// are then formed from them instead of recomputing the contraction (same bits).
hipError_t launch_reinforce_zero_backward(const void* H, const void* W, int dtype, int n_tok, int d, int vocab,
                                          const int32_t* tokens, const float* lse, const float* coef,
                                          const float* logits, long long ld, float* dH, float* dW, void* workspace,
                                          hipStream_t stream);

hipError_t launch_quantize_rows_fp8(const void* X, int dtype, long long n_rows, int d, uint8_t* Xq, float* scale,
                                    hipStream_t stream);

hipError_t launch_lmhead_logprob_fp8(const uint8_t* Hq, const float* h_scale, const uint8_t* Wq, const float* w_scale,
                                     int n_tok, int d, int vocab, const int32_t* tokens, float* logprob, float* lse,
                                     void* workspace, hipStream_t stream);

hipError_t launch_quantize_rows_mxfp4(const void* X, int dtype, long long n_rows, int d, uint8_t* Xq, uint8_t* sc,
                                      hipStream_t stream);

hipError_t launch_lmhead_logprob_mxfp4(const uint8_t* Hq, const float* h_scale, const uint8_t* Wq4,
                                       const uint8_t* w_sc, int n_tok, int d, int vocab, const int32_t* tokens,
                                       float* logprob, float* lse, void* workspace, hipStream_t stream);

size_t mismatch_stats_workspace_bytes(long long n_tok);

hipError_t launch_mismatch_stats(const float* lp, const float* lpr, const float* lps, long long n, double* stats,
                                 void* workspace, hipStream_t stream);

// Device-side validation; writes a nonzero value to *flag on a violation.
hipError_t launch_check_inputs(const int32_t* tokens, long long n_tok, int vocab, const int64_t* resp_offsets,
                               int n_resp, int* flag, hipStream_t stream);

// The norms around a block (norm.hip). codes (nullable): u as E4M3 codes with
// u_scale instead of u. gate_stride: 0 (one gate for all rows) or d.
hipError_t launch_residual_norm(const void* x, const void* y, const void* gate, long long gate_stride,
                                const void* w_post, const void* w_pre, int dtype, long long n_rows, int d, float scale,
                                float eps, void* h, void* u, uint8_t* codes, float* u_scale, float* rstd_pre,
                                float* rstd_post, hipStream_t stream);

size_t norm_backward_workspace_bytes(long long n_rows, long long d);

// dgate: fp32 [d] for one shared gate, else rows of the norm's type.
hipError_t launch_residual_norm_backward(const void* du, int grad_dtype, const void* dh, const void* h, const void* y,
                                         const void* gate, long long gate_stride, const void* w_post,
                                         const void* w_pre, const float* rstd_pre, const float* rstd_post, int dtype,
                                         long long n_rows, int d, float scale, void* dx, void* dy, void* dgate,
                                         float* dw_pre, float* dw_post, void* workspace, hipStream_t stream);

// The end of a norm's backward: the runs' column sums added (norm.hip). Null outputs are left out.
hipError_t launch_norm_backward_finish(const float* part, int runs, int d, float* dw_pre, float* dw_post, float* dgate,
                                       hipStream_t stream);

struct DropoutArgs;

// y = x with dropout (dropout.hip); y may be x.
hipError_t launch_dropout(const void* x, int dtype, long long n_rows, int d, const DropoutArgs& drop, void* y,
                          hipStream_t stream);

// The norms with dropout of y (norm_dropout.hip) and with u as block-scaled E4M3
// rows, u_scale [d / 128, n_rows] (norm_codes.hip; drop.seed null: no dropout).
hipError_t launch_residual_norm_dropout(const void* x, const void* y, const void* gate, long long gate_stride,
                                        const void* w_post, const void* w_pre, int dtype, long long n_rows, int d,
                                        float scale, float eps, const DropoutArgs& drop, void* h, void* u, float* rstd_pre,
                                        float* rstd_post, hipStream_t stream);
hipError_t launch_residual_norm_blocks(const void* x, const void* y, const void* gate, long long gate_stride,
                                       const void* w_post, const void* w_pre, int dtype, long long n_rows, int d,
                                       float scale, float eps, const DropoutArgs& drop, void* h, uint8_t* codes,
                                       float* u_scale, float* rstd_pre, float* rstd_post, hipStream_t stream);
hipError_t launch_residual_norm_dropout_backward(const void* du, int grad_dtype, const void* dh, const void* h, const void* y,
                                                 const void* gate, long long gate_stride, const void* w_post,
                                                 const void* w_pre, const float* rstd_pre, const float* rstd_post,
                                                 int dtype, long long n_rows, int d, float scale, const DropoutArgs& drop,
                                                 void* dx, void* dy, void* dgate, float* dw_pre, float* dw_post,
                                                 void* workspace, hipStream_t stream);

// E4M3 codes with a scale for each 128 values of a row (tiles false) or each 128 x 128
// tile (quantize_blocks.hip): Xq [n_rows, d rounded up to 128], scale [d / 128, n_rows]
// (tiles: [n_rows / 128, d / 128]), and of the transpose: Xtq [d, n_rows rounded up],
// t_scale [n_rows / 128, d] (tiles: [d / 128, n_rows / 128]). Either pair may be null.
hipError_t launch_quantize_blocks(const void* X, int dtype, long long n_rows, long long d, bool tiles, uint8_t* Xq,
                                  float* scale, uint8_t* Xtq, float* t_scale, hipStream_t stream);

// C [m, n] = A B^T of block-scaled E4M3 operands (matmul_fp8.hip).
struct MatmulFp8 {
  const uint8_t *A, *B;
  const float *a_scale, *b_scale;
  long long m, n, k;
  void* C;
  int out_dtype;
};
hipError_t launch_matmul_fp8_blocks(const MatmulFp8& c, hipStream_t stream);

// The vocabulary cross entropy (cross_entropy.hip), with the gradient where dH is given.
struct CeCall {
  const void *H, *W;
  int dtype;
  long long n_tok, d, vocab;
  const int32_t* targets;
  float smoothing, z_weight;
  int mean;  // the loss is the mean over the counted tokens (else their sum)
  float grad_scale;
  int grad_dtype;
  float *loss, *token_loss, *lse;  // lse nullable
  void *dH, *dW;
  void* workspace;
};
size_t cross_entropy_workspace_bytes(long long n_tok, long long d, long long vocab, int dtype, bool grad, int grad_dtype);
hipError_t launch_cross_entropy(const CeCall& c, hipStream_t stream);

// One AdamW step over a plan's pieces (adamw.hip).
size_t adamw_workspace_bytes();
hipError_t launch_adamw_step(const void* plan, long long n_pieces, int state_bits, void* m, void* v, float* m_scale,
                             float* v_scale, float* master, const float* lr, int64_t* step, double beta1, double beta2,
                             double eps, bool with_norm, float max_norm, float* norm, void* workspace,
                             hipStream_t stream);

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace itl

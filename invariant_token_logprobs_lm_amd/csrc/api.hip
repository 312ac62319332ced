// C ABI of the library (declared in include/itl.h): argument validation,
// workspace sizing, status codes. Every host-detectable error returns before
// anything is enqueued; nothing here allocates, frees or synchronises except
// itl_check_inputs.

#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>
#include <mutex>
#include <new>
#include <string>
#include <utility>
#include <vector>

#include "adamw_plan.h"
#include "itl.h"
#include "itl_config.h"
#include "itl_launch.h"
#include "sampled_plan.h"

namespace {

thread_local std::string g_last_error;

itl_status fail(itl_status s, const char* what) {
  g_last_error = what;
  return s;
}

itl_status hip_fail(hipError_t e, const char* where) {
  g_last_error = std::string(where) + ": " + hipGetErrorName(e) + " (" + hipGetErrorString(e) + ")";
  return ITL_ERR_HIP;
}

constexpr int64_t kMaxTok = (int64_t)INT32_MAX - itl::kBT;
constexpr int64_t kMaxVocab = (int64_t)INT32_MAX - itl::kBV;
constexpr int64_t kFp8DMultiple = 128;  // one 128-byte K step = 128 E4M3 values
// the loss's token pass has one workgroup per 2048-token window
constexpr int64_t kMaxLossTok = (int64_t)INT32_MAX * itl::kSegTokens;

int elem_size(itl_dtype dt) { return dt == ITL_BF16 ? 2 : 4; }

// Shared shape checks of the head entry points.
itl_status check_head(itl_dtype dtype, int64_t n_tok, int64_t d, int64_t vocab) {
  if (n_tok < 0 || d <= 0 || vocab <= 0) return fail(ITL_ERR_INVALID_ARG, "n_tok must be >= 0, d and vocab > 0");
  if (dtype != ITL_BF16 && dtype != ITL_F32) return fail(ITL_ERR_UNSUPPORTED, "dtype must be ITL_BF16 or ITL_F32");
  if (d % itl::kDMultiple != 0) return fail(ITL_ERR_UNSUPPORTED, "d must be a multiple of 64");
  if (n_tok > kMaxTok) return fail(ITL_ERR_UNSUPPORTED, "n_tok too large for one call");
  if (vocab > kMaxVocab) return fail(ITL_ERR_UNSUPPORTED, "vocab too large");
  // a 256-row operand block must be addressable with 32-bit buffer offsets
  if (d >= ((int64_t)1 << 31) / (elem_size(dtype) * (int64_t)itl::kBT)) return fail(ITL_ERR_UNSUPPORTED, "d too large");
  const int64_t grid = itl::ceil_div(n_tok, itl::kBT) * itl::n_slice_groups(n_tok, vocab);
  if (grid > INT32_MAX) return fail(ITL_ERR_UNSUPPORTED, "problem too large for one launch");
  return ITL_OK;
}

// A grid dimension holds less than 2^32 threads; a launch of more wraps without
// an error. The forwards have 16 threads per token to merge the slices and
// `threads` per token block and slice group.
constexpr int64_t kGridThreads = (int64_t)1 << 32;
itl_status check_forward_launch(int64_t n_tok, int64_t vocab, int threads) {
  const int64_t grid = itl::ceil_div(n_tok, itl::kBT) * itl::n_slice_groups(n_tok, vocab);
  if (16 * itl::ceil_div(n_tok, 64) * 64 >= kGridThreads || grid * threads >= kGridThreads)
    return fail(ITL_ERR_UNSUPPORTED, "n_tok too large for one launch");
  return ITL_OK;
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255) != 0; }

// The head kernels move H and W rows in 16-byte pieces per lane.
bool misaligned16(const void* a, const void* b) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 15) != 0;
}

// Scratch of itl_lmhead_logprob_noalloc: a file-scope device array, one
// copy per GPU, held until the process ends. Host code never uses its name
// as an address: the device address comes from hipGetSymbolAddress, once per
// device, with that device current.
constexpr size_t kNoAllocScratchBytes = (size_t)64 << 20;
constexpr int kMaxDevices = 64;

}  // namespace

__device__ __align__(256) unsigned char itl_noalloc_scratch[kNoAllocScratchBytes];

namespace {

std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

// The scratch's device address on the device `stream` belongs to (the
// current device for the null stream).
itl_status noalloc_scratch(hipStream_t stream, void** out) {
  int dev = -1;
  hipError_t e = stream ? hipStreamGetDevice(stream, &dev) : hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "itl_lmhead_logprob_noalloc: device of the stream");
  if (dev < 0 || dev >= kMaxDevices) return fail(ITL_ERR_UNSUPPORTED, "device index beyond the scratch table");
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    int cur = -1;
    e = hipGetDevice(&cur);
    if (e != hipSuccess) return hip_fail(e, "itl_lmhead_logprob_noalloc: current device");
    if (cur != dev && (e = hipSetDevice(dev)) != hipSuccess) return hip_fail(e, "itl_lmhead_logprob_noalloc: set device");
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(itl_noalloc_scratch));
    if (cur != dev) {
      const hipError_t e2 = hipSetDevice(cur);
      if (e == hipSuccess) e = e2;
    }
    if (e != hipSuccess || p == nullptr)
      return hip_fail(e != hipSuccess ? e : hipErrorInvalidSymbol, "itl_lmhead_logprob_noalloc: scratch address");
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return ITL_OK;
}

}  // namespace

extern "C" {

size_t itl_lmhead_logprob_workspace_bytes(int64_t n_tok, int64_t vocab) {
  if (n_tok < 0 || vocab <= 0 || n_tok > kMaxTok || vocab > kMaxVocab) return SIZE_MAX;
  return itl::lmhead_workspace_bytes(n_tok, vocab);
}

itl_status itl_lmhead_logprob(const void* H, const void* W, itl_dtype dtype, int64_t n_tok, int64_t d, int64_t vocab,
                              const int32_t* tokens, float* logprob, float* lse, void* workspace,
                              size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  itl_status st = check_head(dtype, n_tok, d, vocab);
  if (st == ITL_OK) st = check_forward_launch(n_tok, vocab, itl::kThreads8);
  if (st != ITL_OK) return st;
  if (n_tok == 0) return ITL_OK;
  if (!H || !W || !tokens || !logprob) return fail(ITL_ERR_INVALID_ARG, "null H, W, tokens or logprob");
  if (misaligned16(H, W)) return fail(ITL_ERR_INVALID_ARG, "H and W must be 16-byte aligned");
  if (!workspace || workspace_bytes < itl::lmhead_workspace_bytes(n_tok, vocab))
    return fail(ITL_ERR_WORKSPACE, "workspace missing or smaller than itl_lmhead_logprob_workspace_bytes()");
  if (misaligned(workspace)) return fail(ITL_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  hipError_t e = itl::launch_lmhead_logprob(H, W, (int)dtype, (int)n_tok, (int)d, (int)vocab, tokens, logprob, lse,
                                            nullptr, 0, workspace, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ITL_OK : hip_fail(e, "itl_lmhead_logprob");
}

itl_status itl_lmhead_logprob_noalloc(const void* H, const void* W, itl_dtype dtype, int64_t n_tok, int64_t d,
                                      int64_t vocab, const int32_t* tokens, float* logprob, float* lse, void* stream) {
  g_last_error.clear();
  itl_status st = check_head(dtype, n_tok, d, vocab);
  if (st != ITL_OK) return st;
  if (n_tok == 0) return ITL_OK;
  if (!H || !W || !tokens || !logprob) return fail(ITL_ERR_INVALID_ARG, "null H, W, tokens or logprob");
  if (misaligned16(H, W)) return fail(ITL_ERR_INVALID_ARG, "H and W must be 16-byte aligned");
  if (itl::lmhead_workspace_bytes(n_tok, vocab) > kNoAllocScratchBytes)
    return fail(ITL_ERR_UNSUPPORTED,
                "n_tok too large for itl_lmhead_logprob_noalloc's 64 MiB scratch (at most 16,368 tokens for "
                "vocab >= 65,281; use itl_lmhead_logprob with a workspace)");
  const hipStream_t s = static_cast<hipStream_t>(stream);
  void* scratch = nullptr;
  st = noalloc_scratch(s, &scratch);
  if (st != ITL_OK) return st;
  hipError_t e = itl::launch_lmhead_logprob(H, W, (int)dtype, (int)n_tok, (int)d, (int)vocab, tokens, logprob, lse,
                                            nullptr, 0, scratch, s);
  return e == hipSuccess ? ITL_OK : hip_fail(e, "itl_lmhead_logprob_noalloc");
}

namespace {

// The kept-logits buffer: [n_tok, ld] fp32, ld >= vocab and a multiple of 4,
// 16-byte aligned, every offset t * ld + v addressable.
itl_status check_logits(const float* logits, int64_t ld, int64_t n_tok, int64_t vocab) {
  if (!logits) return fail(ITL_ERR_INVALID_ARG, "null logits");
  if (ld < vocab || ld % 4 != 0) return fail(ITL_ERR_INVALID_ARG, "ld_logits must be >= vocab and a multiple of 4");
  // 128 token rows of the buffer must be addressable with 32-bit offsets
  if (ld > (int64_t)(UINT32_MAX / (4u * 128u))) return fail(ITL_ERR_UNSUPPORTED, "ld_logits too large");
  if ((reinterpret_cast<uintptr_t>(logits) & 15) != 0) return fail(ITL_ERR_INVALID_ARG, "logits must be 16-byte aligned");
  if (n_tok > 0 && ld > (INT64_MAX / 8) / n_tok) return fail(ITL_ERR_INVALID_ARG, "n_tok * ld_logits overflows");
  return ITL_OK;
}

}  // namespace

itl_status itl_lmhead_logprob_keep_logits(const void* H, const void* W, itl_dtype dtype, int64_t n_tok, int64_t d,
                                          int64_t vocab, const int32_t* tokens, float* logprob, float* lse,
                                          float* logits, int64_t ld_logits, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  g_last_error.clear();
  itl_status st = check_head(dtype, n_tok, d, vocab);
  if (st == ITL_OK) st = check_forward_launch(n_tok, vocab, itl::kThreads8);
  if (st != ITL_OK) return st;
  if (n_tok == 0) return ITL_OK;
  if (!H || !W || !tokens || !logprob) return fail(ITL_ERR_INVALID_ARG, "null H, W, tokens or logprob");
  if (misaligned16(H, W)) return fail(ITL_ERR_INVALID_ARG, "H and W must be 16-byte aligned");
  st = check_logits(logits, ld_logits, n_tok, vocab);
  if (st != ITL_OK) return st;
  if (!workspace || workspace_bytes < itl::lmhead_workspace_bytes(n_tok, vocab))
    return fail(ITL_ERR_WORKSPACE, "workspace missing or smaller than itl_lmhead_logprob_workspace_bytes()");
  if (misaligned(workspace)) return fail(ITL_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  hipError_t e = itl::launch_lmhead_logprob(H, W, (int)dtype, (int)n_tok, (int)d, (int)vocab, tokens, logprob, lse,
                                            logits, (long long)ld_logits, workspace, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ITL_OK : hip_fail(e, "itl_lmhead_logprob_keep_logits");
}

itl_status itl_group_advantage(const float* rewards, const int32_t* group_offsets, int32_t n_groups, int32_t n_resp,
                               float* advantages, void* stream) {
  g_last_error.clear();
  if (n_groups < 0 || n_resp < 0) return fail(ITL_ERR_INVALID_ARG, "n_groups and n_resp must be >= 0");
  if (n_groups == 0 || n_resp == 0) return ITL_OK;
  if (!rewards || !group_offsets || !advantages) return fail(ITL_ERR_INVALID_ARG, "null rewards, offsets or output");
  hipError_t e = itl::launch_group_advantage(rewards, group_offsets, n_groups, n_resp, advantages,
                                             static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ITL_OK : hip_fail(e, "itl_group_advantage");
}

size_t itl_reinforce_zero_loss_workspace_bytes(int64_t n_tok, int32_t n_resp) {
  if (n_tok < 0 || n_resp < 0 || n_tok > kMaxLossTok) return SIZE_MAX;
  return itl::loss_workspace_bytes(n_tok, n_resp);
}

itl_status itl_reinforce_zero_loss(const float* logprob, const float* rollout_logprob, const float* advantages,
                                   const int64_t* resp_offsets, int32_t n_resp, int64_t n_tok, float* resp_loss,
                                   float* loss, float* coef, void* workspace, size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  if (n_resp < 0 || n_tok < 0) return fail(ITL_ERR_INVALID_ARG, "n_resp and n_tok must be >= 0");
  if (n_tok > kMaxLossTok) return fail(ITL_ERR_UNSUPPORTED, "n_tok too large for one call");
  if (n_resp == 0) return ITL_OK;
  if (!resp_offsets || !advantages || !resp_loss || !loss)
    return fail(ITL_ERR_INVALID_ARG, "null offsets, advantages or outputs");
  if (n_tok > 0 && (!logprob || !rollout_logprob)) return fail(ITL_ERR_INVALID_ARG, "null logprob arrays");
  if (!workspace || workspace_bytes < itl::loss_workspace_bytes(n_tok, n_resp))
    return fail(ITL_ERR_WORKSPACE, "workspace missing or smaller than itl_reinforce_zero_loss_workspace_bytes()");
  if (misaligned(workspace)) return fail(ITL_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  hipError_t e = itl::launch_reinforce_zero_loss(logprob, rollout_logprob, advantages, resp_offsets, n_resp, n_tok,
                                                 resp_loss, loss, coef, workspace, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ITL_OK : hip_fail(e, "itl_reinforce_zero_loss");
}

size_t itl_reinforce_zero_backward_workspace_bytes(int64_t n_tok, int64_t d, int64_t vocab, itl_dtype dtype) {
  if (n_tok < 0 || d <= 0 || vocab <= 0 || n_tok > kMaxTok || vocab > kMaxVocab) return SIZE_MAX;
  if (dtype != ITL_BF16 && dtype != ITL_F32) return SIZE_MAX;
  // shapes the backward refuses get no size either (and no wrapped product)
  if (d % itl::kDMultiple != 0 || d >= ((int64_t)1 << 31) / (elem_size(dtype) * (int64_t)itl::kBT)) return SIZE_MAX;
  return itl::backward_workspace_bytes(n_tok, d, vocab, (int)dtype);
}

namespace {

itl_status backward(const void* H, const void* W, itl_dtype dtype, int64_t n_tok, int64_t d, int64_t vocab,
                    const int32_t* tokens, const float* lse, const float* coef, const float* logits, int64_t ld,
                    float* dH, float* dW, void* workspace, size_t workspace_bytes, void* stream, const char* name) {
  itl_status st = check_head(dtype, n_tok, d, vocab);
  if (st != ITL_OK) return st;
  if (!W || !dW) return fail(ITL_ERR_INVALID_ARG, "null W or dW");
  if (n_tok > 0 && (!H || !tokens || !lse || !coef || !dH))
    return fail(ITL_ERR_INVALID_ARG, "null H, tokens, lse, coef or dH");
  if (vocab > itl::kBwdMaxVocab) return fail(ITL_ERR_UNSUPPORTED, "vocab too large for the backward");
  if (((reinterpret_cast<uintptr_t>(H) | reinterpret_cast<uintptr_t>(W) | reinterpret_cast<uintptr_t>(dH) |
        reinterpret_cast<uintptr_t>(dW)) & 15) != 0)
    return fail(ITL_ERR_INVALID_ARG, "H, W, dH and dW must be 16-byte aligned");
  const size_t need = itl::backward_workspace_bytes(n_tok, d, vocab, (int)dtype);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(ITL_ERR_WORKSPACE, "workspace missing or smaller than itl_reinforce_zero_backward_workspace_bytes()");
  if (need > 0 && misaligned(workspace)) return fail(ITL_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  hipError_t e = itl::launch_reinforce_zero_backward(H, W, (int)dtype, (int)n_tok, (int)d, (int)vocab, tokens, lse,
                                                     coef, logits, (long long)ld, dH, dW, workspace,
                                                     static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ITL_OK : hip_fail(e, name);
}

}  // namespace

itl_status itl_reinforce_zero_backward_from_logits(const void* H, const void* W, itl_dtype dtype, int64_t n_tok,
                                                   int64_t d, int64_t vocab, const int32_t* tokens, const float* lse,
                                                   const float* coef, const float* logits, int64_t ld_logits,
                                                   float* dH, float* dW, void* workspace, size_t workspace_bytes,
                                                   void* stream) {
  g_last_error.clear();
  if (n_tok > 0) {
    itl_status st = check_logits(logits, ld_logits, n_tok, vocab);
    if (st != ITL_OK) return st;
  }
  return backward(H, W, dtype, n_tok, d, vocab, tokens, lse, coef, n_tok > 0 ? logits : nullptr, ld_logits, dH, dW,
                  workspace, workspace_bytes, stream, "itl_reinforce_zero_backward_from_logits");
}

itl_status itl_reinforce_zero_backward(const void* H, const void* W, itl_dtype dtype, int64_t n_tok, int64_t d,
                                       int64_t vocab, const int32_t* tokens, const float* lse, const float* coef,
                                       float* dH, float* dW, void* workspace, size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  return backward(H, W, dtype, n_tok, d, vocab, tokens, lse, coef, nullptr, 0, dH, dW, workspace, workspace_bytes,
                  stream, "itl_reinforce_zero_backward");
}

itl_status itl_quantize_rows_fp8(const void* X, itl_dtype dtype, int64_t n_rows, int64_t d, uint8_t* Xq, float* scale,
                                 void* stream) {
  g_last_error.clear();
  if (n_rows < 0 || d <= 0) return fail(ITL_ERR_INVALID_ARG, "n_rows must be >= 0 and d > 0");
  if (dtype != ITL_BF16 && dtype != ITL_F32) return fail(ITL_ERR_UNSUPPORTED, "dtype must be ITL_BF16 or ITL_F32");
  if (d % kFp8DMultiple != 0) return fail(ITL_ERR_UNSUPPORTED, "d must be a multiple of 128");
  if (n_rows > kGridThreads / 64 - 4 || d > INT32_MAX)  // (a wavefront per row, four a workgroup)
    return fail(ITL_ERR_UNSUPPORTED, "too many rows or columns");
  if (n_rows == 0) return ITL_OK;
  if (!X || !Xq || !scale) return fail(ITL_ERR_INVALID_ARG, "null X, Xq or scale");
  if ((reinterpret_cast<uintptr_t>(Xq) & 3) != 0) return fail(ITL_ERR_INVALID_ARG, "Xq must be 4-byte aligned");
  hipError_t e = itl::launch_quantize_rows_fp8(X, (int)dtype, n_rows, (int)d, Xq, scale,
                                               static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ITL_OK : hip_fail(e, "itl_quantize_rows_fp8");
}

itl_status itl_lmhead_logprob_fp8(const uint8_t* Hq, const float* h_scale, const uint8_t* Wq, const float* w_scale,
                                  int64_t n_tok, int64_t d, int64_t vocab, const int32_t* tokens, float* logprob,
                                  float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  if (n_tok < 0 || d <= 0 || vocab <= 0) return fail(ITL_ERR_INVALID_ARG, "n_tok must be >= 0, d and vocab > 0");
  if (d % kFp8DMultiple != 0) return fail(ITL_ERR_UNSUPPORTED, "d must be a multiple of 128");
  if (n_tok > kMaxTok) return fail(ITL_ERR_UNSUPPORTED, "n_tok too large for one call");
  if (vocab > kMaxVocab) return fail(ITL_ERR_UNSUPPORTED, "vocab too large");
  if (d >= ((int64_t)1 << 31) / (int64_t)itl::kBT) return fail(ITL_ERR_UNSUPPORTED, "d too large");
  if (vocab > (int64_t)(UINT32_MAX / 4)) return fail(ITL_ERR_UNSUPPORTED, "vocab too large");
  // the grid of the kernel that runs: narrow for few tokens
  const bool narrow = n_tok <= itl::kNarrowMaxTokens;
  const int64_t grid = narrow ? itl::ceil_div(n_tok, itl::kNarrowBRows) * itl::n_slices(vocab)
                              : itl::ceil_div(n_tok, itl::kBT) * itl::n_slice_groups(n_tok, vocab);
  if (grid > INT32_MAX) return fail(ITL_ERR_UNSUPPORTED, "problem too large for one launch");
  const itl_status fits = check_forward_launch(n_tok, vocab, itl::kThreads8);
  if (fits != ITL_OK) return fits;
  if (n_tok == 0) return ITL_OK;
  if (!Hq || !h_scale || !Wq || !w_scale || !tokens || !logprob)
    return fail(ITL_ERR_INVALID_ARG, "null Hq, h_scale, Wq, w_scale, tokens or logprob");
  if (((reinterpret_cast<uintptr_t>(Hq) | reinterpret_cast<uintptr_t>(Wq)) & 15) != 0)
    return fail(ITL_ERR_INVALID_ARG, "Hq and Wq must be 16-byte aligned");
  if (!workspace || workspace_bytes < itl::lmhead_workspace_bytes(n_tok, vocab))
    return fail(ITL_ERR_WORKSPACE, "workspace missing or smaller than itl_lmhead_logprob_workspace_bytes()");
  if (misaligned(workspace)) return fail(ITL_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  hipError_t e = itl::launch_lmhead_logprob_fp8(Hq, h_scale, Wq, w_scale, (int)n_tok, (int)d, (int)vocab, tokens,
                                                logprob, lse, workspace, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ITL_OK : hip_fail(e, "itl_lmhead_logprob_fp8");
}

itl_status itl_quantize_rows_mxfp4(const void* X, itl_dtype dtype, int64_t n_rows, int64_t d, uint8_t* Xq,
                                   uint8_t* scale_codes, void* stream) {
  g_last_error.clear();
  if (n_rows < 0 || d <= 0) return fail(ITL_ERR_INVALID_ARG, "n_rows must be >= 0 and d > 0");
  if (dtype != ITL_BF16 && dtype != ITL_F32) return fail(ITL_ERR_UNSUPPORTED, "dtype must be ITL_BF16 or ITL_F32");
  if (d % kFp8DMultiple != 0) return fail(ITL_ERR_UNSUPPORTED, "d must be a multiple of 128");
  if (d > INT32_MAX || n_rows > (kGridThreads - 256) / (d / 32)) return fail(ITL_ERR_UNSUPPORTED, "too many rows");
  if (n_rows == 0) return ITL_OK;
  if (!X || !Xq || !scale_codes) return fail(ITL_ERR_INVALID_ARG, "null X, Xq or scale_codes");
  if ((reinterpret_cast<uintptr_t>(Xq) & 15) != 0) return fail(ITL_ERR_INVALID_ARG, "Xq must be 16-byte aligned");
  hipError_t e = itl::launch_quantize_rows_mxfp4(X, (int)dtype, n_rows, (int)d, Xq, scale_codes,
                                                 static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ITL_OK : hip_fail(e, "itl_quantize_rows_mxfp4");
}

itl_status itl_lmhead_logprob_mxfp4(const uint8_t* Hq, const float* h_scale, const uint8_t* Wq4,
                                    const uint8_t* w_scale_codes, int64_t n_tok, int64_t d, int64_t vocab,
                                    const int32_t* tokens, float* logprob, float* lse, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  if (n_tok < 0 || d <= 0 || vocab <= 0) return fail(ITL_ERR_INVALID_ARG, "n_tok must be >= 0, d and vocab > 0");
  if (d % kFp8DMultiple != 0) return fail(ITL_ERR_UNSUPPORTED, "d must be a multiple of 128");
  if (n_tok > kMaxTok) return fail(ITL_ERR_UNSUPPORTED, "n_tok too large for one call");
  if (vocab > kMaxVocab) return fail(ITL_ERR_UNSUPPORTED, "vocab too large");
  if (d >= ((int64_t)1 << 31) / (int64_t)itl::kBT) return fail(ITL_ERR_UNSUPPORTED, "d too large");
  const int64_t grid = itl::ceil_div(n_tok, itl::kBT) * itl::n_slice_groups(n_tok, vocab);
  if (grid > INT32_MAX) return fail(ITL_ERR_UNSUPPORTED, "problem too large for one launch");
  const itl_status fits = check_forward_launch(n_tok, vocab, itl::kThreads);
  if (fits != ITL_OK) return fits;
  if (n_tok == 0) return ITL_OK;
  if (!Hq || !h_scale || !Wq4 || !w_scale_codes || !tokens || !logprob)
    return fail(ITL_ERR_INVALID_ARG, "null Hq, h_scale, Wq4, w_scale_codes, tokens or logprob");
  if (((reinterpret_cast<uintptr_t>(Hq) | reinterpret_cast<uintptr_t>(Wq4)) & 15) != 0)
    return fail(ITL_ERR_INVALID_ARG, "Hq and Wq4 must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(w_scale_codes) & 3) != 0)
    return fail(ITL_ERR_INVALID_ARG, "w_scale_codes must be 4-byte aligned");
  if (!workspace || workspace_bytes < itl::lmhead_workspace_bytes(n_tok, vocab))
    return fail(ITL_ERR_WORKSPACE, "workspace missing or smaller than itl_lmhead_logprob_workspace_bytes()");
  if (misaligned(workspace)) return fail(ITL_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  hipError_t e = itl::launch_lmhead_logprob_mxfp4(Hq, h_scale, Wq4, w_scale_codes, (int)n_tok, (int)d, (int)vocab,
                                                  tokens, logprob, lse, workspace, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ITL_OK : hip_fail(e, "itl_lmhead_logprob_mxfp4");
}

namespace {

constexpr int64_t kMaxNormWidth = 1 << 24;

bool known_dtype(itl_dtype dt) { return dt == ITL_BF16 || dt == ITL_F32; }

// Arrays of a call by their bytes; a null or empty one shares nothing.
struct Span {
  const void* p;
  int64_t bytes;
};

bool shares(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.bytes > 0 && b.bytes > 0 && x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// Whether an output shares memory with an input or another output: other
// workgroups may still read what one has written.
bool outputs_share(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (shares(*o, i)) return true;
    for (auto p = outs.begin(); p != o; ++p)
      if (shares(*o, *p)) return true;
  }
  return false;
}

// Rows the norms move in 16-byte pieces (widths of a multiple of 8) have to
// start at one; other widths are read value by value.
bool rows_misaligned(std::initializer_list<const void*> ps, int64_t d, itl_dtype dtype) {
  const uintptr_t mask = d % 8 == 0 ? 15 : (uintptr_t)elem_size(dtype) - 1;
  uintptr_t all = 0;
  for (const void* p : ps) all |= reinterpret_cast<uintptr_t>(p);
  return (all & mask) != 0;
}

itl_status check_norm(itl_dtype dtype, int64_t n_rows, int64_t d, int64_t gate_stride, const void* gate, const void* y,
                      const void* w_post, float scale, float eps) {
  if (n_rows < 0 || d <= 0) return fail(ITL_ERR_INVALID_ARG, "n_rows must be >= 0 and d > 0");
  if (!known_dtype(dtype)) return fail(ITL_ERR_UNSUPPORTED, "dtype must be ITL_BF16 or ITL_F32");
  if (n_rows > INT32_MAX || d > kMaxNormWidth) return fail(ITL_ERR_UNSUPPORTED, "too many rows or columns");
  if (!(eps > 0.0f) || !(eps < 1.0f)) return fail(ITL_ERR_INVALID_ARG, "eps must be in (0, 1)");
  if (!(scale - scale == 0.0f)) return fail(ITL_ERR_INVALID_ARG, "scale must be finite");
  if (gate && gate_stride != 0 && gate_stride != d) return fail(ITL_ERR_INVALID_ARG, "gate_stride must be 0 or d");
  if (n_rows > 0 && !y && (gate || w_post)) return fail(ITL_ERR_INVALID_ARG, "gate and w_post need y");
  return ITL_OK;
}

itl_status residual_norm(const void* x, const void* y, const void* gate, int64_t gate_stride, const void* w_post,
                         const void* w_pre, itl_dtype dtype, int64_t n_rows, int64_t d, float scale, float eps, void* h,
                         void* u, uint8_t* codes, float* u_scale, bool fp8, float* rstd_pre, float* rstd_post,
                         void* stream, const char* name) {
  itl_status st = check_norm(dtype, n_rows, d, gate_stride, gate, y, w_post, scale, eps);
  if (st != ITL_OK) return st;
  if (fp8 && d % kFp8DMultiple != 0) return fail(ITL_ERR_UNSUPPORTED, "d must be a multiple of 128");
  if (n_rows == 0) return ITL_OK;
  if (!x || !w_pre || (y && !h) || (fp8 ? !codes || !u_scale : !u))
    return fail(ITL_ERR_INVALID_ARG, "null x, w_pre, h (with y) or output");
  if (rows_misaligned({x, y, gate, w_post, w_pre, y ? h : nullptr, u}, d, dtype))
    return fail(ITL_ERR_INVALID_ARG, "arrays must be 16-byte aligned where d is a multiple of 8, else by element");
  if (fp8 && (reinterpret_cast<uintptr_t>(codes) & 7) != 0) return fail(ITL_ERR_INVALID_ARG, "Uq must be 8-byte aligned");
  const int64_t row_bytes = d * elem_size(dtype), all = n_rows * row_bytes, one = n_rows * 4;
  // (h may be x, row for row)
  if (outputs_share({{u, all}, {codes, n_rows * d}, {u_scale, one}, {rstd_pre, one}, {w_post ? rstd_post : nullptr, one},
                     {y ? h : nullptr, all}},
                    {{h == x ? nullptr : x, all}, {y, all}, {gate, gate_stride ? all : row_bytes}, {w_post, row_bytes},
                     {w_pre, row_bytes}}) ||
      (h == x && outputs_share({{u, all}, {codes, n_rows * d}, {u_scale, one}, {rstd_pre, one},
                                {w_post ? rstd_post : nullptr, one}}, {{x, all}})))
    return fail(ITL_ERR_INVALID_ARG, "outputs share memory with inputs or each other (only h may be x)");
  hipError_t e = itl::launch_residual_norm(x, y, gate, gate_stride, w_post, w_pre, (int)dtype, n_rows, (int)d, scale, eps,
                                           h, u, codes, u_scale, rstd_pre, rstd_post, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ITL_OK : hip_fail(e, name);
}

}  // namespace

itl_status itl_residual_norm(const void* x, const void* y, const void* gate, int64_t gate_stride, const void* w_post,
                             const void* w_pre, itl_dtype dtype, int64_t n_rows, int64_t d, float scale, float eps,
                             void* h, void* u, float* rstd_pre, float* rstd_post, void* stream) {
  g_last_error.clear();
  return residual_norm(x, y, gate, gate_stride, w_post, w_pre, dtype, n_rows, d, scale, eps, h, u, nullptr, nullptr, false,
                       rstd_pre, rstd_post, stream, "itl_residual_norm");
}

itl_status itl_residual_norm_fp8(const void* x, const void* y, const void* gate, int64_t gate_stride, const void* w_post,
                                 const void* w_pre, itl_dtype dtype, int64_t n_rows, int64_t d, float scale, float eps,
                                 void* h, uint8_t* Uq, float* u_scale, float* rstd_pre, float* rstd_post, void* stream) {
  g_last_error.clear();
  return residual_norm(x, y, gate, gate_stride, w_post, w_pre, dtype, n_rows, d, scale, eps, h, nullptr, Uq, u_scale, true,
                       rstd_pre, rstd_post, stream, "itl_residual_norm_fp8");
}

size_t itl_residual_norm_backward_workspace_bytes(int64_t n_rows, int64_t d) {
  if (n_rows < 0 || d <= 0 || n_rows > INT32_MAX || d > kMaxNormWidth) return SIZE_MAX;
  return itl::norm_backward_workspace_bytes(n_rows, d);
}

itl_status itl_residual_norm_backward(const void* du, itl_dtype du_dtype, const void* dh, const void* h, const void* y,
                                      const void* gate, int64_t gate_stride, const void* w_post, const void* w_pre,
                                      const float* rstd_pre, const float* rstd_post, itl_dtype dtype, int64_t n_rows,
                                      int64_t d, float scale, void* dx, void* dy, void* dgate, float* dw_pre,
                                      float* dw_post, void* workspace, size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  itl_status st = check_norm(dtype, n_rows, d, gate_stride, gate, y, w_post, scale, 0.5f);
  if (st != ITL_OK) return st;
  if (du_dtype != dtype && du_dtype != ITL_F32) return fail(ITL_ERR_UNSUPPORTED, "du_dtype must be dtype or ITL_F32");
  if (!w_pre || !dw_pre || (gate && !dgate) || (w_post && !dw_post))
    return fail(ITL_ERR_INVALID_ARG, "null w_pre, dw_pre, dgate (with gate) or dw_post (with w_post)");
  if (n_rows > 0 && (!du || !h || !dx || !rstd_pre || (y && !dy) || (w_post && !rstd_post)))
    return fail(ITL_ERR_INVALID_ARG, "null du, h, dx, rstd_pre, dy (with y) or rstd_post (with w_post)");
  if (n_rows > 0 && (rows_misaligned({dh, h, y, gate, w_post, w_pre, dx, y ? dy : nullptr,
                                      gate && gate_stride ? dgate : nullptr}, d, dtype) ||
                     rows_misaligned({du}, d, du_dtype)))
    return fail(ITL_ERR_INVALID_ARG, "arrays must be 16-byte aligned where d is a multiple of 8, else by element");
  if (!workspace || workspace_bytes < itl::norm_backward_workspace_bytes(n_rows, d))
    return fail(ITL_ERR_WORKSPACE, "workspace missing or smaller than itl_residual_norm_backward_workspace_bytes()");
  if (misaligned(workspace)) return fail(ITL_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  const int64_t row_bytes = d * elem_size(dtype), all = n_rows * row_bytes;
  // (dx may be dh, row for row)
  if (outputs_share({{dx, all}, {y ? dy : nullptr, all}, {gate ? dgate : nullptr, gate_stride ? all : d * 4},
                     {dw_pre, d * 4}, {w_post ? dw_post : nullptr, d * 4},
                     {workspace, (int64_t)itl::norm_backward_workspace_bytes(n_rows, d)}},
                    {{du, n_rows * d * elem_size(du_dtype)}, {dh == dx ? nullptr : dh, all}, {h, all}, {y, all},
                     {gate, gate_stride ? all : row_bytes}, {w_post, row_bytes}, {w_pre, row_bytes},
                     {rstd_pre, n_rows * 4}, {w_post ? rstd_post : nullptr, n_rows * 4}}))
    return fail(ITL_ERR_INVALID_ARG, "outputs share memory with inputs or each other (only dx may be dh)");
  hipError_t e = itl::launch_residual_norm_backward(du, (int)du_dtype, dh, h, y, gate, gate_stride, w_post, w_pre,
                                                    rstd_pre, rstd_post, (int)dtype, n_rows, (int)d, scale, dx, dy, dgate,
                                                    dw_pre, dw_post, workspace, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ITL_OK : hip_fail(e, "itl_residual_norm_backward");
}

namespace {

itl_status cross_entropy(const itl::CeCall& c, bool grad, size_t workspace_bytes, void* stream, const char* name) {
  itl_status st = check_head(c.dtype, c.n_tok, c.d, c.vocab);
  if (st != ITL_OK) return st;
  if (!(c.smoothing >= 0.0f && c.smoothing < 1.0f)) return fail(ITL_ERR_INVALID_ARG, "label_smoothing must be in [0, 1)");
  if (!(c.z_weight >= 0.0f && c.z_weight - c.z_weight == 0.0f))
    return fail(ITL_ERR_INVALID_ARG, "z_weight must be finite and >= 0");
  if (c.mean != 0 && c.mean != 1) return fail(ITL_ERR_INVALID_ARG, "reduction must be ITL_SUM or ITL_MEAN");
  if (grad && !(c.grad_scale - c.grad_scale == 0.0f)) return fail(ITL_ERR_INVALID_ARG, "grad_scale must be finite");
  if (grad && c.grad_dtype != c.dtype && c.grad_dtype != ITL_F32)
    return fail(ITL_ERR_UNSUPPORTED, "grad_dtype must be dtype or ITL_F32");
  if ((grad || c.dtype == ITL_F32) && c.vocab > itl::kBwdMaxVocab)
    return fail(ITL_ERR_UNSUPPORTED, "vocab too large for the gradient or an fp32 head");
  if (!c.W || !c.loss || (grad && !c.dW)) return fail(ITL_ERR_INVALID_ARG, "null W, loss or dW");
  if (c.n_tok > 0 && (!c.H || !c.targets || !c.token_loss || (grad && !c.dH)))
    return fail(ITL_ERR_INVALID_ARG, "null H, targets, token_loss or dH");
  if (misaligned16(c.H, c.W) || misaligned16(c.dH, c.dW))
    return fail(ITL_ERR_INVALID_ARG, "H, W, dH and dW must be 16-byte aligned");
  const size_t need = itl::cross_entropy_workspace_bytes(c.n_tok, c.d, c.vocab, c.dtype, grad, c.grad_dtype);
  if (need > 0 && (!c.workspace || workspace_bytes < need))
    return fail(ITL_ERR_WORKSPACE, "workspace missing or smaller than itl_cross_entropy_workspace_bytes()");
  if (need > 0 && misaligned(c.workspace)) return fail(ITL_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  const int64_t es = elem_size((itl_dtype)c.dtype), gs = elem_size((itl_dtype)c.grad_dtype);
  if (outputs_share({{c.loss, 4}, {c.token_loss, c.n_tok * 4}, {c.lse, c.n_tok * 4}, {c.dH, c.n_tok * c.d * gs},
                     {c.dW, c.vocab * c.d * gs}, {c.workspace, (int64_t)need}},
                    {{c.H, c.n_tok * c.d * es}, {c.W, c.vocab * c.d * es}, {c.targets, c.n_tok * 4}}))
    return fail(ITL_ERR_INVALID_ARG, "outputs share memory with inputs or each other");
  hipError_t e = itl::launch_cross_entropy(c, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ITL_OK : hip_fail(e, name);
}

}  // namespace

size_t itl_cross_entropy_workspace_bytes(int64_t n_tok, int64_t d, int64_t vocab, itl_dtype dtype, int32_t with_grad,
                                         itl_dtype grad_dtype) {
  if (n_tok < 0 || d <= 0 || vocab <= 0 || n_tok > kMaxTok || vocab > kMaxVocab || !known_dtype(dtype)) return SIZE_MAX;
  if (d % itl::kDMultiple != 0 || d >= ((int64_t)1 << 31) / (elem_size(dtype) * (int64_t)itl::kBT)) return SIZE_MAX;
  if ((with_grad || dtype == ITL_F32) && vocab > itl::kBwdMaxVocab) return SIZE_MAX;
  if (with_grad && grad_dtype != dtype && grad_dtype != ITL_F32) return SIZE_MAX;
  return itl::cross_entropy_workspace_bytes(n_tok, d, vocab, (int)dtype, with_grad != 0, (int)grad_dtype);
}

itl_status itl_cross_entropy(const void* H, const void* W, itl_dtype dtype, int64_t n_tok, int64_t d, int64_t vocab,
                             const int32_t* targets, float label_smoothing, float z_weight, int32_t reduction, float* loss,
                             float* token_loss, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  const itl::CeCall c{H, W, (int)dtype, n_tok, d, vocab, targets, label_smoothing, z_weight, reduction, 0.0f, (int)dtype,
                      loss, token_loss, lse, nullptr, nullptr, workspace};
  return cross_entropy(c, false, workspace_bytes, stream, "itl_cross_entropy");
}

itl_status itl_cross_entropy_grad(const void* H, const void* W, itl_dtype dtype, int64_t n_tok, int64_t d, int64_t vocab,
                                  const int32_t* targets, float label_smoothing, float z_weight, int32_t reduction,
                                  float grad_scale, itl_dtype grad_dtype, float* loss, float* token_loss, float* lse,
                                  void* dH, void* dW, void* workspace, size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  const itl::CeCall c{H, W, (int)dtype, n_tok, d, vocab, targets, label_smoothing, z_weight, reduction, grad_scale,
                      (int)grad_dtype, loss, token_loss, lse, dH, dW, workspace};
  return cross_entropy(c, true, workspace_bytes, stream, "itl_cross_entropy_grad");
}

namespace {

// Checks the tensors and counts the plan's pieces and the flat states' elements.
itl_status adamw_layout(const itl_adamw_tensor* tensors, int32_t n_tensors, int64_t* n_pieces, int64_t* n_state) {
  if (n_tensors < 0 || (n_tensors > 0 && !tensors)) return fail(ITL_ERR_INVALID_ARG, "null tensors or n_tensors < 0");
  int64_t pieces = 0, state = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    const itl_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n > ((int64_t)1 << 40)) return fail(ITL_ERR_INVALID_ARG, "a tensor's n must be in [0, 2^40]");
    if (!known_dtype(t.param_dtype) || !known_dtype(t.grad_dtype))
      return fail(ITL_ERR_UNSUPPORTED, "param_dtype and grad_dtype must be ITL_BF16 or ITL_F32");
    if (t.n > 0 && (!t.param || !t.grad)) return fail(ITL_ERR_INVALID_ARG, "null param or grad");
    if (!(t.weight_decay >= 0.0f && t.weight_decay - t.weight_decay == 0.0f))
      return fail(ITL_ERR_INVALID_ARG, "weight_decay must be finite and >= 0");
    if ((reinterpret_cast<uintptr_t>(t.param) & (elem_size(t.param_dtype) - 1)) != 0 ||
        (reinterpret_cast<uintptr_t>(t.grad) & (elem_size(t.grad_dtype) - 1)) != 0)
      return fail(ITL_ERR_INVALID_ARG, "param and grad must be aligned to their elements");
    pieces += itl::ceil_div(t.n, itl::kAdamPiece);
    state += itl::ceil_div(t.n, itl::kAdamBlock) * itl::kAdamBlock;
    if (pieces > itl::kAdamMaxPieces) return fail(ITL_ERR_UNSUPPORTED, "too many elements for one plan");
  }
  *n_pieces = pieces;
  *n_state = state;
  return ITL_OK;
}

}  // namespace

itl_status itl_adamw_plan_sizes(const itl_adamw_tensor* tensors, int32_t n_tensors, int64_t* plan_bytes,
                                int64_t* state_elements) {
  g_last_error.clear();
  if (!plan_bytes || !state_elements) return fail(ITL_ERR_INVALID_ARG, "null plan_bytes or state_elements");
  int64_t pieces = 0;
  itl_status st = adamw_layout(tensors, n_tensors, &pieces, state_elements);
  if (st == ITL_OK) *plan_bytes = pieces * (int64_t)sizeof(itl::AdamPiece);
  return st;
}

itl_status itl_adamw_plan(const itl_adamw_tensor* tensors, int32_t n_tensors, void* host_plan, size_t host_plan_bytes) {
  g_last_error.clear();
  int64_t pieces = 0, state = 0;
  itl_status st = adamw_layout(tensors, n_tensors, &pieces, &state);
  if (st != ITL_OK) return st;
  if (pieces == 0) return ITL_OK;
  if (!host_plan || host_plan_bytes < (size_t)pieces * sizeof(itl::AdamPiece))
    return fail(ITL_ERR_WORKSPACE, "host_plan missing or smaller than itl_adamw_plan_sizes() says");
  // two entries that share weights would be written by two workgroups at
  // once, and gradients among the weights read after they are written
  try {
    std::vector<std::pair<uintptr_t, uintptr_t>> spans;
    for (int32_t i = 0; i < n_tensors; ++i)
      if (tensors[i].n > 0) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(tensors[i].param);
        spans.emplace_back(at, at + (uintptr_t)tensors[i].n * elem_size(tensors[i].param_dtype));
      }
    std::sort(spans.begin(), spans.end());
    for (size_t i = 1; i < spans.size(); ++i)
      if (spans[i].first < spans[i - 1].second) return fail(ITL_ERR_INVALID_ARG, "two tensors share weights");
    for (int32_t i = 0; i < n_tensors; ++i) {
      if (tensors[i].n == 0) continue;
      const uintptr_t g = reinterpret_cast<uintptr_t>(tensors[i].grad);
      const uintptr_t end = g + (uintptr_t)tensors[i].n * elem_size(tensors[i].grad_dtype);
      // the last weights that begin before the gradient's end
      auto s = std::lower_bound(spans.begin(), spans.end(), std::make_pair(end, (uintptr_t)0));
      if (s != spans.begin() && (--s)->second > g)
        return fail(ITL_ERR_INVALID_ARG, "a gradient and weights share memory");
    }
  } catch (const std::bad_alloc&) {
    return fail(ITL_ERR_INVALID_ARG, "out of host memory");
  }
  char* out = static_cast<char*>(host_plan);
  int64_t at = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    const itl_adamw_tensor& t = tensors[i];
    const int ep = elem_size(t.param_dtype), eg = elem_size(t.grad_dtype);
    const bool vec = !misaligned16(t.param, t.grad);
    for (int64_t o = 0; o < t.n; o += itl::kAdamPiece) {
      itl::AdamPiece p{};
      p.param = static_cast<char*>(t.param) + o * ep;
      p.grad = static_cast<const char*>(t.grad) + o * eg;
      p.state = at + o;
      p.count = (int32_t)std::min<int64_t>(itl::kAdamPiece, t.n - o);
      p.flags = (t.param_dtype == ITL_F32 ? itl::kAdamParamF32 : 0) | (t.grad_dtype == ITL_F32 ? itl::kAdamGradF32 : 0) |
                (vec ? itl::kAdamVectors : 0);
      p.weight_decay = t.weight_decay;
      memcpy(out, &p, sizeof p);
      out += sizeof p;
    }
    at += itl::ceil_div(t.n, itl::kAdamBlock) * itl::kAdamBlock;
  }
  return ITL_OK;
}

size_t itl_adamw_step_workspace_bytes(void) { return itl::adamw_workspace_bytes(); }

itl_status itl_adamw_step(const void* plan, size_t plan_bytes, int32_t state_bits, void* exp_avg, void* exp_avg_sq,
                          float* exp_avg_scale, float* exp_avg_sq_scale, float* master, const float* lr, int64_t* step,
                          double beta1, double beta2, double eps, float max_norm, float* grad_norm, void* workspace,
                          size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  if (plan_bytes % sizeof(itl::AdamPiece) != 0) return fail(ITL_ERR_INVALID_ARG, "plan_bytes is not a plan's");
  if (state_bits != 8 && state_bits != 32) return fail(ITL_ERR_UNSUPPORTED, "state_bits must be 8 or 32");
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0))
    return fail(ITL_ERR_INVALID_ARG, "beta1 and beta2 must be in [0, 1)");
  if (!((float)eps > 0.0f && eps < 1.0)) return fail(ITL_ERR_INVALID_ARG, "eps must be in (0, 1) in fp32");
  if (!(max_norm > 0.0f)) return fail(ITL_ERR_INVALID_ARG, "max_norm must be > 0 (infinity: no clipping)");
  const int64_t pieces = (int64_t)(plan_bytes / sizeof(itl::AdamPiece));
  if (pieces > itl::kAdamMaxPieces) return fail(ITL_ERR_UNSUPPORTED, "too many elements for one plan");
  if (!lr || !step) return fail(ITL_ERR_INVALID_ARG, "null lr or step");
  if (pieces > 0 && (!plan || !exp_avg || !exp_avg_sq || (state_bits == 8 && (!exp_avg_scale || !exp_avg_sq_scale))))
    return fail(ITL_ERR_INVALID_ARG, "null plan or state");
  if (misaligned16(exp_avg, exp_avg_sq) || misaligned16(master, nullptr) || (reinterpret_cast<uintptr_t>(plan) & 7) != 0)
    return fail(ITL_ERR_INVALID_ARG, "states must be 16-byte aligned, the plan 8-byte aligned");
  if (!workspace || workspace_bytes < itl::adamw_workspace_bytes())
    return fail(ITL_ERR_WORKSPACE, "workspace missing or smaller than itl_adamw_step_workspace_bytes()");
  if (misaligned(workspace)) return fail(ITL_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  // (the states' sizes are in the plan, on the device: 256 elements a piece are there at least)
  const int64_t least = pieces * itl::kAdamBlock, code = state_bits == 8 ? 1 : 4;
  const bool scales = state_bits == 8;
  if (outputs_share({{exp_avg, least * code}, {exp_avg_sq, least * code}, {scales ? exp_avg_scale : nullptr, pieces * 4},
                     {scales ? exp_avg_sq_scale : nullptr, pieces * 4}, {master, least * 4}, {step, 8}, {grad_norm, 4},
                     {workspace, (int64_t)itl::adamw_workspace_bytes()}},
                    {{lr, 4}, {plan, (int64_t)plan_bytes}}))
    return fail(ITL_ERR_INVALID_ARG, "states, step, grad_norm or workspace share memory with each other, lr or the plan");
  const bool with_norm = grad_norm || max_norm < __builtin_inff();
  hipError_t e = itl::launch_adamw_step(plan, pieces, state_bits, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale,
                                        master, lr, step, beta1, beta2, eps, with_norm, max_norm, grad_norm, workspace,
                                        static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ITL_OK : hip_fail(e, "itl_adamw_step");
}

size_t itl_mismatch_stats_workspace_bytes(int64_t n_tok) {
  if (n_tok < 0 || n_tok > INT32_MAX) return SIZE_MAX;
  return n_tok == 0 ? 0 : itl::mismatch_stats_workspace_bytes(n_tok);
}

itl_status itl_mismatch_stats(const float* logprob, const float* rollout_logprob, const float* same_weights_logprob,
                              int64_t n_tok, double* stats, void* workspace, size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  if (n_tok < 0) return fail(ITL_ERR_INVALID_ARG, "n_tok must be >= 0");
  if (n_tok > INT32_MAX) return fail(ITL_ERR_UNSUPPORTED, "n_tok too large for one call");
  if (!stats) return fail(ITL_ERR_INVALID_ARG, "null stats");
  if (n_tok > 0 && (!logprob || !rollout_logprob)) return fail(ITL_ERR_INVALID_ARG, "null logprob arrays");
  const size_t need = n_tok == 0 ? 0 : itl::mismatch_stats_workspace_bytes(n_tok);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(ITL_ERR_WORKSPACE, "workspace missing or smaller than itl_mismatch_stats_workspace_bytes()");
  if (need > 0 && misaligned(workspace)) return fail(ITL_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  hipError_t e = itl::launch_mismatch_stats(logprob, rollout_logprob, same_weights_logprob, n_tok, stats, workspace,
                                            static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ITL_OK : hip_fail(e, "itl_mismatch_stats");
}

itl_status itl_check_inputs(const int32_t* tokens, int64_t n_tok, int64_t vocab, const int64_t* resp_offsets,
                            int32_t n_resp, void* stream) {
  g_last_error.clear();
  if (n_tok < 0 || n_resp < 0 || vocab <= 0 || vocab > kMaxVocab)
    return fail(ITL_ERR_INVALID_ARG, "bad sizes");
  hipStream_t s = static_cast<hipStream_t>(stream);
  int* flag = nullptr;
  hipError_t e = hipMalloc(&flag, sizeof(int));
  if (e != hipSuccess) return hip_fail(e, "itl_check_inputs");
  int host = 0;
  e = hipMemcpyAsync(flag, &host, sizeof(int), hipMemcpyHostToDevice, s);
  if (e == hipSuccess) e = itl::launch_check_inputs(tokens, n_tok, (int)vocab, resp_offsets, n_resp, flag, s);
  if (e == hipSuccess) e = hipMemcpyAsync(&host, flag, sizeof(int), hipMemcpyDeviceToHost, s);
  if (e == hipSuccess) e = hipStreamSynchronize(s);
  hipFree(flag);
  if (e != hipSuccess) return hip_fail(e, "itl_check_inputs");
  if (host == 1) return fail(ITL_ERR_BAD_INPUT, "a token id is outside [0, vocab)");
  if (host == 2) return fail(ITL_ERR_BAD_INPUT, "response offsets must start at 0, end at n_tok and increase");
  return ITL_OK;
}

const char* itl_status_string(itl_status status) {
  switch (status) {
    case ITL_OK: return "ITL_OK";
    case ITL_ERR_INVALID_ARG: return "ITL_ERR_INVALID_ARG: invalid argument";
    case ITL_ERR_UNSUPPORTED: return "ITL_ERR_UNSUPPORTED: shape or dtype not supported by this build";
    case ITL_ERR_WORKSPACE: return "ITL_ERR_WORKSPACE: workspace missing, too small or misaligned";
    case ITL_ERR_HIP: return "ITL_ERR_HIP: HIP runtime error";
    case ITL_ERR_BAD_INPUT: return "ITL_ERR_BAD_INPUT: invalid device-resident input";
  }
  return "unknown itl_status";
}

const char* itl_last_error(void) { return g_last_error.c_str(); }

const char* itl_build_info(void) {
  static const std::string info = [] {
    char buf[768];
    snprintf(buf, sizeof buf,
             "itl 0.3 arch=gfx950 threads=%d wide_threads=%d token_block=%d vocab_tile=%d k_step_bytes=%d w_slots=%d h_slots=%d "
             "swap_slots_over_k_steps=%d max_slices=%d slices=balanced narrow_max_tokens=%d narrow_token_block=%d narrow128_max_tokens=%d "
             "mfma_bf16=16x16x32 mfma_f32=16x16x4 fp8=e4m3_row_scaled mfma_fp8=16x16x128 mxfp4=e2m1_e8m0_32 mfma_mxfp4=32x32x64 "
             "bwd_chunk_tokens=%d loss_segment_tokens=%d loss_lane_segment=%d loss_wave_segment=%d loss_threads=%d "
             "loss_mean_chunk=%d loss_sums=f64 bwd_sampled_sort=stable_counting bwd_sampled_segment=%d "
             "bwd_sampled_group=%d",
             itl::kThreads, itl::kThreads8, itl::kBT, itl::kBV, itl::kStepBytes, itl::kWSlots, itl::kHSlots, itl::kNearBMaxSteps,
             itl::kMaxSlices, itl::kNarrowMaxTokens, itl::kNarrowBRows, itl::kNarrow128MaxTokens, itl::kBwdChunkTokens, itl::kSegTokens,
             itl::kLaneSeg, itl::kWaveSeg, itl::kLossThreads, itl::kFinishChunk, itl::kRunSeg, itl::kRunGroup);
    return std::string(buf);
  }();
  return info.c_str();
}

}  // extern "C"

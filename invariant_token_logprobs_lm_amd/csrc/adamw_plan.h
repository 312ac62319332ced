// Layout of an AdamW plan: the pieces of work of one step over many tensors,
// laid out once on the host and kept by the caller in device memory.
#pragma once

#include <stdint.h>

namespace itl {

// State of tensor i starts at a multiple of kAdamBlock elements behind the
// state of tensor i - 1; an 8-bit state has one scale per kAdamBlock.
constexpr int kAdamBlock = 256;
// Elements of a piece: one workgroup's work, within one tensor.
constexpr int kAdamPiece = 2048;
constexpr int kAdamThreads = 256;
constexpr int kAdamVec = 8;  // consecutive elements of a thread
// A workgroup per piece in one grid dimension, which holds less than 2^32 threads.
constexpr int64_t kAdamMaxPieces = (1LL << 32) / kAdamThreads - 1;
static_assert(kAdamPiece % (kAdamThreads * kAdamVec) == 0 && kAdamPiece % kAdamBlock == 0, "whole passes and blocks");

enum : uint32_t {
  kAdamParamF32 = 1,   // weights are fp32 (else bf16)
  kAdamGradF32 = 2,    // gradients are fp32 (else bf16)
  kAdamVectors = 4,    // weights and gradients are 16-byte aligned
};

struct AdamPiece {
  void* param;        // the piece's first weight
  const void* grad;   // its first gradient
  int64_t state;      // its first element in the flat states
  int32_t count;      // elements, 1 .. kAdamPiece
  uint32_t flags;
  float weight_decay;
  int32_t pad;
};
static_assert(sizeof(AdamPiece) == 40, "the plan's layout");

// Written by the step's first kernel, read by its second.
struct AdamScalars {
  float clip;   // factor on the gradients
  float rate;   // lr / (1 - beta1^t)
  float root;   // 1 / sqrt(1 - beta2^t)
  float lr;
  int32_t skip; // the gradients' norm is not finite: nothing is changed
};

// Workgroups of the gradients' square sum (fixed, so its order is).
constexpr int kAdamNormGroups = 2048;

}  // namespace itl

// Internal interface of the operators on packed weights with BF16 activations: the layer for few
// tokens, the choice of experts, and the experts' products.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/twq.h"

namespace twq {

constexpr int kA16MaxRows = 64;     // tokens of a call
constexpr int kMoeMaxChoices = 16;  // experts of a token
constexpr int kMoeMaxExperts = 1024;
constexpr int64_t kA16MaxDim = int64_t(1) << 20;

// The choice of k experts per row of `logits` (fp32, or BF16 where bf16 is set).
struct RouteCall {
  const void* logits;
  bool bf16;
  int64_t ld;
  int64_t b;
  int count, k;
  bool renormalize;
  int32_t* ids;
  float* weights;
};
cudaError_t launch_moe_route(const RouteCall& c, cudaStream_t st);

struct A16LinearCall {
  const uint16_t* x;
  int64_t ldx;
  int b;
  const twq_weights* w;
  uint16_t* h;  // b x r, or null with r == 0
  uint16_t* y;
};
cudaError_t launch_a16_linear(const A16LinearCall& c, cudaStream_t st);

struct MoeCall {
  const uint16_t* x;
  int64_t ldx;
  int b, k;
  const int32_t* ids;
  const float* weights;
  const twq_experts* e;
  const uint16_t* base;
  uint16_t* y;
  void* workspace;
};
cudaError_t launch_moe_experts(const MoeCall& c, cudaStream_t st);
size_t moe_workspace(int64_t pairs, const twq_experts* e);

// Self-test: while not 0, the calling thread's launches have a loading warp that stops early and
// this limit of their waits.
void set_a16_stall(int64_t wait_limit_ns);
cudaError_t read_and_clear_a16_status(int* code);

}  // namespace twq

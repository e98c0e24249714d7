// accept.cuh -- launch parameters of the check of drafted tokens.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>
#include "kernels.cuh"

namespace ddt {

constexpr int32_t kStatusBadToken = 256;
constexpr int32_t kStatusBadLogits = 512;

struct AcceptParams {
  const void* logits;          // bf16 or fp32, node (b, t) at logits + (b * T + t) * logit_stride
  int64_t logit_stride;
  const float* draft_prob;     // fp32, rows like the logits; or null
  int64_t draft_stride;
  const int32_t* tokens;       // [B, T]
  const int32_t* tree_parent;  // [B, T]
  const int32_t* tree_len;     // [B] or null
  const float* uniform;        // [B, T]
  const float* temperature;    // [B]
  int32_t batch, nodes, vocab;
  int32_t row_cluster, walk_cluster;  // CTAs of a node, of a request: 1, 2, 4 or 8
  // of each node: its row's maximum, where it is, what its refused children leave of the sum of its weights
  float* row_max;
  int32_t* row_arg;
  unsigned long long* left;
  // of each node as a child: accepted if its parent is; what its refusal takes, drawn tokens: S, else w (0: nothing)
  int32_t* accepted;
  unsigned long long* taken;
  int32_t* path;               // [B, T]
  int32_t* path_len;           // [B]
  int32_t* next_token;         // [B]
  int32_t* status;
};
cudaError_t launch_accept(const AcceptParams& p, bool bf16, cudaStream_t stream);

}  // namespace ddt

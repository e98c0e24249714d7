// accept.cuh -- launch parameters of the check of drafted tokens.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>
#include "kernels.cuh"

namespace ddt {

constexpr int32_t kStatusBadToken = 256;
constexpr int32_t kStatusBadLogits = 512;
constexpr int kAcceptVocab = 1 << 18;       // most tokens: a cluster of 16 CTAs holds a row of them in shared memory
constexpr int kAcceptBytes = 200 * 1024;    // of that, in one CTA
constexpr int kAcceptCluster = 16, kAcceptSizes = 5;  // most CTAs of a request; 1, 2, 4, 8, 16
// shared memory of a token: its logit, or with draft probabilities its weight and probability
constexpr int accept_value_bytes(bool drawn) { return drawn ? 12 : 4; }

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
  int32_t cluster;             // CTAs of a request: 1, 2, 4, 8 or 16
  int32_t share, warp_share;   // tokens of a CTA, and of each of its 16 warps
  int32_t* path;               // [B, T]
  int32_t* path_len;           // [B]
  int32_t* next_token;         // [B]
  int32_t* status;             // cleared before the launch
#ifdef DDT_TEST_HOOKS
  int32_t test_keep_back;      // reduction of which one warp's part is not sent (-1: none)
#endif
};
// How many clusters of 2^i CTAs one device runs at once; [1]: of at most half of kAcceptBytes, two CTAs to an SM
struct AcceptClusters {
  int count[kAcceptSizes][2] = {};
};
cudaError_t configure_accept(AcceptClusters* clusters);  // on the current device
cudaError_t launch_accept(const AcceptParams& p, bool bf16, cudaStream_t stream);

}  // namespace ddt

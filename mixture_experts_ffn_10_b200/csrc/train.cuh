// train.cuh -- arguments of the router's training kernels (train.cu).
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kBalanceMaxChunks = 444;  // blocks of tokens of the balance loss (three per SM: one wave)

struct RouterTrainArgs {
  const void* logits;        // [T, E]
  const void* router_bias;   // [E] or null
  const int32_t* idx;        // [T, k]
  const int32_t* seq;        // [B + 1] or null: {0, T}
  int T, E, k, B, bf16, score;
  float coef;
  int chunk;                 // tokens per block
  // balance loss
  int nchunks;               // blocks
  float* psum;               // [nchunks + B, E] shares summed per (block, sequence)
  int32_t* pcnt;             // [nchunks + B, E] slots likewise
  double* part;              // [B * E / 32] parts of the loss
  int32_t* ticket;           // finished blocks of the second kernel
  int32_t* counts;           // [B, E] out; backward: in, or null
  float* loss;               // [1]
  // backward
  int renorm;
  float scale;
  const float* dw;           // [T, k] or null
  const float* dloss;        // [1] or null
  void* dlogits;             // [T, E]
  int vec;                   // rows are read and written in 16-byte vectors
};

// The layer's checks of shape and options (api.cu).
int check_layer(const moe_shape* s, const moe_options* o);

cudaError_t launch_balance_loss(const RouterTrainArgs& a, cudaStream_t st);
cudaError_t launch_router_backward(const RouterTrainArgs& a, int num_sms, cudaStream_t st);

}  // namespace moe

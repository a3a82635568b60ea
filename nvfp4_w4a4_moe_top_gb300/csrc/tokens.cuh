// Arguments and launches of the operators at the token ends (embed.cu,
// sample.cu), behind their C ABI (tokens.cu).
#pragma once

#include "../../include/moe_tokens.h"
#include "learner.cuh"

namespace moe {

struct EmbedArgs {
  const int32_t* ids;
  const void* table;
  int dtype;
  int64_t ldt;
  int T, V, d;
  float scale;
  uint16_t* out;
  int64_t ldo;
  int* status;
};
struct EmbedBwdArgs {
  const uint16_t* dy;
  int64_t ldy;
  const int32_t* ids;
  int T, V, d;
  float scale;
  int accumulate;
  float* dtable;
  char* ws;
  int* status;
};
struct SampleArgs {
  const void* logits;
  int dtype;
  int64_t ld;
  int T, V;
  const float* inv_t;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* tokens;
  float* logprob;
  float* kept_logprob;
  int* status;
};

int launch_embed_tokens(const EmbedArgs& a, cudaStream_t s);
size_t embed_tokens_backward_ws(int T, int V, int d);
int launch_embed_tokens_backward(const EmbedBwdArgs& a, cudaStream_t s);
int launch_sample_tokens(const SampleArgs& a, cudaStream_t s);

}  // namespace moe

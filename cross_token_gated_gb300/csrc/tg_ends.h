// Internal launchers of the calls at the model's two ends: token lookup and its gradient, the
// norm and its gradient, distillation, sampling.
#pragma once
#include <cuda_runtime.h>

#include "tango.h"

namespace tg {

constexpr unsigned kKernDistill = 7u << 8;
constexpr unsigned kKernSample = 8u << 8;

// ---- embed.cu
struct EmbedCall {
  long long rows, pitch;
  int d, vocab, pad_id;
  bool padded;       // whether pad_id stands for no token
  float scale;
  tg_dtype dtype, grad_dtype;
  const int* ids;
  const void* E;     // lookup
  void* out;
  const void* dout;  // gradient
  const void* base;
  void* dE;
  void* ws;
  unsigned* err;
};
cudaError_t launch_embed_lookup(const EmbedCall& c, cudaStream_t s);
size_t embed_backward_ws_bytes(const EmbedCall& c);
cudaError_t launch_embed_backward(const EmbedCall& c, cudaStream_t s);

// ---- norm.cu
struct NormCall {
  long long rows, x_pitch;
  int d, norm;
  float eps;
  tg_dtype dtype;
  const void *x, *gamma, *beta;
  void* y;              // forward
  const void *dy, *dres;  // backward
  void* dx;
  float *dgamma, *dbeta;
  void* ws;
};
cudaError_t launch_norm(const NormCall& c, cudaStream_t s);
size_t norm_backward_ws_bytes(const NormCall& c);
cudaError_t launch_norm_backward(const NormCall& c, cudaStream_t s);

// ---- distill.cu
struct DistillCall {
  long long rows, pitch, grad_pitch;
  int vocab, k;
  float temperature;
  tg_dtype dtype;
  const void* logits;
  const float* t_logits;
  const int* t_ids;
  float* loss;
  float* stats_out;       // forward
  const float* stats;     // backward
  const float* dloss;
  void* dlogits;
  unsigned* err;
};
cudaError_t launch_distill(const DistillCall& c, cudaStream_t s);
cudaError_t launch_distill_backward(const DistillCall& c, cudaStream_t s);

// ---- sample.cu
struct SampleCall {
  tg_sample_params p;
  const void* logits;
  const float* uniform;
  int* token;
  float* logprob;
  unsigned* err;
};
cudaError_t launch_sample(const SampleCall& c, cudaStream_t s);

}  // namespace tg

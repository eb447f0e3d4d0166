// Internal launchers of the norm-and-rotate call, its gradient, and the paged cache calls.
#pragma once
#include <cuda_runtime.h>

#include "tango.h"
#include "tg_paged.cuh"

namespace tg {

// SMs of the current device (looked up once per device).
int serve_sm_count();

// ---- qk_rope.cu
struct QkCall {
  long long rows;
  int H, Hk, d_h, rotary, layout, norm, T;
  float eps;
  const int* positions;
  const double* freqs;
  const float *q_gain, *k_gain;
  long long q_pitch, k_pitch;
  const void *q, *k;
  void *q_out, *k_out;            // forward
  const void *dq_out, *dk_out;    // backward
  void *dq, *dk;
  float *dq_gain, *dk_gain, *part;
};
cudaError_t launch_qk_forward(tg_dtype dt, const QkCall& c, cudaStream_t s);
cudaError_t launch_qk_backward(tg_dtype dt, const QkCall& c, cudaStream_t s);
// Bytes of QkCall::part (the blocks' partial gain gradients).
size_t qk_backward_part_bytes(int d_h);

struct AppendCall {
  PagedBatch p;
  int H, d_h, m_h, m_pitch;
  int rotary, layout, norm;
  float eps;
  const double* freqs;
  int silu;
  long long q_pitch, k_pitch, g_pitch;
  const void *q, *k, *g;
  void *q_out, *k_pages, *g_pages;
};
cudaError_t launch_cache_append(tg_dtype dt, const AppendCall& c, cudaStream_t s);

// ---- aggregation over the cache: the weights of every (row, head) first, into scratch,
// then the gates they average.  Heads, and row tiles of one head, are taken in passes that keep
// the scratch bounded.
struct PagedCall {
  PagedBatch p;
  int H, d_h, m_h, m_pitch;
  float s;
  const float* tau;
  const float* null_bias;
  long long v_pitch;
  const void *q, *v;
  void* out;
  const void *k_pages, *g_pages;
  void* ws;
  int debug_timeout;
};
// Whether the grids fit: max_len up to 65,535 x 128.
bool paged_simt_takes(tg_dtype dt, const PagedCall& c);
size_t paged_simt_ws_bytes(tg_dtype dt, const PagedCall& c);
cudaError_t launch_paged_simt(tg_dtype dt, const PagedCall& c, cudaStream_t s);

// The same on the tensor cores (bf16).  Whether the shapes are ones it takes: head widths and
// pitches that TMA and tcgen05 read, pages of a multiple of 8 tokens.  q, out and the pools must
// also be 16-byte aligned (v need not be, and is read element-wise then).
bool paged_tc_takes(tg_dtype dt, const PagedCall& c);
size_t paged_tc_ws_bytes(const PagedCall& c);
cudaError_t launch_paged_tc(const PagedCall& c, cudaStream_t s);

}  // namespace tg

// RMS and layer norm of rows with their gradients ("TANGO: Token-Aggregated Nonlinear Gating
// Operators ...", sec. 2.1: the pre-norm of the residual stream; sec. 2.3: the final norm).
//
//   n = (x - mu) r,  y = gamma n + beta,  r = 1 / sqrt(mean (x - mu)^2 + eps)   (rms: mu = 0)
//   dn = gamma dy,  dx = r (dn - n <dn n> - <dn>) + dres,  dgamma = sum dy n,  dbeta = sum dy
//
// Means are over the row, <dn> only with mu.  All of it is bound by HBM bandwidth: each value is
// read and written once.
#include "tg_common.cuh"
#include "tg_ends.h"
#include "tg_serve.h"

namespace tg {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBwdPerSm = 4;  // blocks of the backward's persistent grid

// Sum over the block; every thread gets it.  `buf` holds kWarps floats and is free again after
// the next call's first barrier (two buffers are used in turn).
__device__ __forceinline__ float block_sum(float v, float* buf) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x / 32] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += buf[w];
  return s;
}

template <typename T>
struct NormArgs {
  long long rows, x_pitch;
  int d, layer;
  float eps;
  const T *x, *gamma, *beta, *dy, *dres;
  T *y, *dx;
  float* part;  // backward: [2][blocks][d] partial dgamma and dbeta
  int want_gamma, want_beta;
};

// Mean and 1 / sqrt(mean square + eps) of a row by the whole block.
template <typename T>
__device__ __forceinline__ float2 row_stats(const NormArgs<T>& a, const T* x, float (*buf)[kWarps]) {
  float mu = 0.f;
  if (a.layer) {
    float s = 0.f;
    for (int c = threadIdx.x; c < a.d; c += kThreads) s += io<T>::ld(x + c);
    mu = block_sum(s, buf[0]) / (float)a.d;
  }
  float ss = 0.f;
  for (int c = threadIdx.x; c < a.d; c += kThreads) {
    const float t = io<T>::ld(x + c) - mu;
    ss = fmaf(t, t, ss);
  }
  return make_float2(mu, 1.f / sqrtf(block_sum(ss, buf[1]) / (float)a.d + a.eps));
}

// One block per row, any width and alignment.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_any_kernel(const NormArgs<T> a) {
  __shared__ float buf[2][kWarps];
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = a.x + row * a.x_pitch;
    const float2 st = row_stats(a, x, buf);
    for (int c = threadIdx.x; c < a.d; c += kThreads) {
      const float n = (io<T>::ld(x + c) - st.x) * st.y;
      io<T>::st(a.y + row * a.d + c, fmaf(n, a.gamma ? io<T>::ld(a.gamma + c) : 1.f, a.beta ? io<T>::ld(a.beta + c) : 0.f));
    }
    __syncthreads();
  }
}

// The gradient, one block per row at a time; a thread adds up its columns' dgamma and dbeta in the
// block's partial sums.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_backward_any_kernel(const NormArgs<T> a) {
  __shared__ float buf[4][kWarps];
  float* pg = a.part + (size_t)blockIdx.x * a.d;
  float* pb = a.part + ((size_t)gridDim.x + blockIdx.x) * a.d;
  for (int c = threadIdx.x; c < a.d; c += kThreads) {
    if (a.want_gamma) pg[c] = 0.f;
    if (a.want_beta) pb[c] = 0.f;
  }
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T *x = a.x + row * a.x_pitch, *dy = a.dy + row * a.d;
    const float2 st = row_stats(a, x, buf);
    float s = 0.f, sn = 0.f;
    for (int c = threadIdx.x; c < a.d; c += kThreads) {
      const float n = (io<T>::ld(x + c) - st.x) * st.y, g = io<T>::ld(dy + c);
      const float dn = a.gamma ? g * io<T>::ld(a.gamma + c) : g;
      s += dn;
      sn = fmaf(dn, n, sn);
      if (a.want_gamma) pg[c] = fmaf(g, n, pg[c]);
      if (a.want_beta) pb[c] += g;
    }
    sn = block_sum(sn, buf[2]) / (float)a.d;
    s = a.layer ? block_sum(s, buf[3]) / (float)a.d : 0.f;
    for (int c = threadIdx.x; c < a.d; c += kThreads) {
      const float n = (io<T>::ld(x + c) - st.x) * st.y, g = io<T>::ld(dy + c);
      const float dn = a.gamma ? g * io<T>::ld(a.gamma + c) : g;
      const float dx = st.y * (dn - s - n * sn);
      io<T>::st(a.dx + row * a.d + c, a.dres ? dx + io<T>::ld(a.dres + row * a.d + c) : dx);
    }
    __syncthreads();
  }
}

// dgamma (blockIdx.y 0) and dbeta (1): a warp per column adds up the blocks' partial sums.
__global__ void __launch_bounds__(256) norm_weight_sum_kernel(const float* part, int blocks, int d, float* dgamma,
                                                              float* dbeta) {
  const int c = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x & 31;
  float* dst = blockIdx.y ? dbeta : dgamma;
  if (c >= d || !dst) return;
  const float* p = part + (size_t)blockIdx.y * blocks * d + c;
  float s = 0.f;
  for (int b = lane; b < blocks; b += 32) s += p[(size_t)b * d];
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) dst[c] = s;
}

template <typename T>
NormArgs<T> norm_args(const NormCall& c) {
  NormArgs<T> a;
  a.rows = c.rows; a.x_pitch = c.x_pitch; a.d = c.d; a.layer = c.norm == TG_NORM_LAYER; a.eps = c.eps;
  a.x = static_cast<const T*>(c.x); a.gamma = static_cast<const T*>(c.gamma); a.beta = static_cast<const T*>(c.beta);
  a.dy = static_cast<const T*>(c.dy); a.dres = static_cast<const T*>(c.dres);
  a.y = static_cast<T*>(c.y); a.dx = static_cast<T*>(c.dx);
  a.part = static_cast<float*>(c.ws);
  a.want_gamma = c.dgamma != nullptr; a.want_beta = c.dbeta != nullptr;
  return a;
}

int grid_of(long long rows, int per_sm) {
  const long long most = (long long)serve_sm_count() * per_sm;
  return (int)(rows < most ? rows : most);
}

template <typename T>
cudaError_t norm_t(const NormCall& c, cudaStream_t s) {
  norm_any_kernel<T><<<grid_of(c.rows, 8), kThreads, 0, s>>>(norm_args<T>(c));
  return cudaGetLastError();
}

template <typename T>
cudaError_t norm_backward_t(const NormCall& c, cudaStream_t s) {
  const NormArgs<T> a = norm_args<T>(c);
  const int grid = grid_of(c.rows, kBwdPerSm);
  norm_backward_any_kernel<T><<<grid, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !(c.dgamma || c.dbeta)) return e;
  norm_weight_sum_kernel<<<dim3(ceil_div(c.d, 8), 2), 256, 0, s>>>(a.part, grid, c.d, c.dgamma, c.dbeta);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(const NormCall& c, cudaStream_t s) {
  return c.dtype == TG_F32 ? norm_t<float>(c, s) : norm_t<__nv_bfloat16>(c, s);
}
size_t norm_backward_ws_bytes(const NormCall& c) {
  return (size_t)grid_of(c.rows, kBwdPerSm) * 2 * c.d * sizeof(float);
}
cudaError_t launch_norm_backward(const NormCall& c, cudaStream_t s) {
  return c.dtype == TG_F32 ? norm_backward_t<float>(c, s) : norm_backward_t<__nv_bfloat16>(c, s);
}

}  // namespace tg

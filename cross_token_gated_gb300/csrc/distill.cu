// Distillation from a teacher's top logits and its gradient, for training the tied logits
// ("TANGO: Token-Aggregated Nonlinear Gating Operators ...", sec. 2.3).
//
//   p = softmax(t / T) over a row's k entries, q = softmax(z / T) over the vocabulary,
//   loss = T^2 sum_e p_e (ln p_e - ln q_{i_e}),  dz_j = dloss T (q_j - sum_{i_e = j} p_e)
//
// Bound by HBM: the logits are read once and the gradient written once.
#include <math.h>

#include "tg_common.cuh"
#include "tg_ends.h"
#include "tg_serve.h"

namespace tg {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;

template <typename T>
struct DistillArgs {
  long long rows, pitch, grad_pitch;
  int vocab, k;
  float temp, c;  // T, log2(e) / T
  const T* z;
  const float* t;
  const int* ids;
  const float *dloss, *stats;
  float *loss, *stats_out;
  T* dz;
  unsigned* err;
};

struct Teacher {
  int id[TG_MAX_TEACHER];    // -1: absent
  float p[TG_MAX_TEACHER];   // the logit first, then e^{(t - max) / T}, then the probability
  float z[TG_MAX_TEACHER];   // the student's logit there
};

__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
// Over the block, for every thread; the barrier at the end frees buf again.
__device__ __forceinline__ float block_sum(float v, float* buf) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += buf[w];
  __syncthreads();
  return v;
}
__device__ __forceinline__ float block_max(float v, float* buf) {
  v = warp_max(v);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x / 32] = v;
  __syncthreads();
  v = buf[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) v = fmaxf(v, buf[w]);
  __syncthreads();
  return v;
}

// The row's entries and their probabilities; false for a row without entries.  ln p_e =
// (t_e - max) / T - lse is formed again where the loss wants it.
template <typename T>
__device__ bool teacher_row(const DistillArgs<T>& a, long long row, const T* z, Teacher& te, float* buf) {
  float mx = -INFINITY;
  bool any = false, nan = false;
  for (int e = threadIdx.x; e < a.k; e += kThreads) {
    int id = a.ids[row * a.k + e];
    const float t = a.t[row * a.k + e];
    if (id >= a.vocab) record_error(a.err, kErrValue | kKernDistill);
    if (id < 0 || id >= a.vocab || t == -INFINITY) id = -1;
    te.id[e] = id;
    te.p[e] = t;
    te.z[e] = id >= 0 ? io<T>::ld(z + id) : 0.f;
    any |= id >= 0;
    if (id >= 0) mx = fmaxf(mx, t);
    nan |= id >= 0 && t != t;
  }
  const int some = __syncthreads_or(any), bad = __syncthreads_or(nan);
  if (!some) return false;
  mx = block_max(mx, buf);
  if (bad) mx = NAN;
  float s = 0.f;
  for (int e = threadIdx.x; e < a.k; e += kThreads) {
    const float w = te.id[e] >= 0 ? exp2f((te.p[e] - mx) * a.c) : 0.f;
    te.p[e] = w;
    s += w;
  }
  const float inv = 1.f / block_sum(s, buf);
  for (int e = threadIdx.x; e < a.k; e += kThreads) te.p[e] *= inv;
  __syncthreads();
  return true;
}

// Largest logit (0 if there is none above -inf) and sum of e^{(z - largest) / T}.
template <typename T>
__device__ float2 student_row(const DistillArgs<T>& a, const T* z, float* buf) {
  float mx = -INFINITY;
  for (int j = threadIdx.x; j < a.vocab; j += kThreads) mx = fmaxf(mx, io<T>::ld(z + j));
  mx = block_max(mx, buf);
  if (mx == -INFINITY) mx = 0.f;
  float s = 0.f;
  for (int j = threadIdx.x; j < a.vocab; j += kThreads) s += exp2f((io<T>::ld(z + j) - mx) * a.c);
  return make_float2(mx, block_sum(s, buf));
}

// T^2 sum p (ln p - ln q), for every thread.
template <typename T>
__device__ float row_loss(const DistillArgs<T>& a, const Teacher& te, float2 st, float* buf) {
  const float lse = logf(st.y);
  float s = 0.f;
  for (int e = threadIdx.x; e < a.k; e += kThreads) {
    const float p = te.p[e], z = te.z[e];
    if (te.id[e] >= 0 && p != 0.f) s += p * (logf(p) - (z == -INFINITY ? z : (z - st.x) / a.temp - lse));
  }
  return a.temp * a.temp * block_sum(s, buf);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillArgs<T> a) {
  __shared__ Teacher te;
  __shared__ float buf[kWarps];
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* z = a.z + row * a.pitch;
    float2 st = make_float2(0.f, 0.f);
    float loss = 0.f;
    if (teacher_row(a, row, z, te, buf)) {
      st = student_row(a, z, buf);
      loss = row_loss(a, te, st, buf);
    }
    if (threadIdx.x == 0) {
      a.loss[row] = loss;
      if (a.stats_out) *reinterpret_cast<float2*>(a.stats_out + 2 * row) = st;
    }
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) distill_backward_kernel(const DistillArgs<T> a) {
  __shared__ Teacher te;
  __shared__ float buf[kWarps];
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* z = a.z + row * a.pitch;
    T* dz = a.dz + row * a.grad_pitch;
    if (!teacher_row(a, row, z, te, buf)) {
      for (int j = threadIdx.x; j < a.vocab; j += kThreads) dz[j] = T(0.f);
      if (threadIdx.x == 0 && a.loss) a.loss[row] = 0.f;
      continue;
    }
    const float2 st = a.stats ? *reinterpret_cast<const float2*>(a.stats + 2 * row) : student_row(a, z, buf);
    if (a.loss) {
      const float loss = row_loss(a, te, st, buf);
      if (threadIdx.x == 0) a.loss[row] = loss;
    }
    const float f = a.dloss[row] * a.temp, inv = st.y == 0.f ? 0.f : 1.f / st.y;
    for (int j = threadIdx.x; j < a.vocab; j += kThreads)
      io<T>::st(dz + j, f * (exp2f((io<T>::ld(z + j) - st.x) * a.c) * inv));
    __syncthreads();
    // the entries' tokens once more, each by its first entry
    for (int e = threadIdx.x; e < a.k; e += kThreads) {
      const int id = te.id[e];
      if (id < 0) continue;
      float p = 0.f;
      bool first = true;
      for (int i = 0; i < a.k; ++i)
        if (te.id[i] == id) {
          first &= i >= e;
          p += te.p[i];
        }
      if (first) io<T>::st(dz + id, f * (exp2f((te.z[e] - st.x) * a.c) * inv - p));
    }
    __syncthreads();
  }
}

template <typename T>
DistillArgs<T> distill_args(const DistillCall& c) {
  DistillArgs<T> a;
  a.rows = c.rows; a.pitch = c.pitch; a.grad_pitch = c.grad_pitch; a.vocab = c.vocab; a.k = c.k;
  a.temp = c.temperature; a.c = kLog2e / c.temperature;
  a.z = static_cast<const T*>(c.logits); a.t = c.t_logits; a.ids = c.t_ids;
  a.dloss = c.dloss; a.stats = c.stats; a.loss = c.loss; a.stats_out = c.stats_out;
  a.dz = static_cast<T*>(c.dlogits); a.err = c.err;
  return a;
}

int grid_of(long long rows) {
  const long long most = 4LL * serve_sm_count();
  return (int)(rows < most ? rows : most);
}

template <typename T>
cudaError_t forward_t(const DistillCall& c, cudaStream_t s) {
  distill_kernel<T><<<grid_of(c.rows), kThreads, 0, s>>>(distill_args<T>(c));
  return cudaGetLastError();
}
template <typename T>
cudaError_t backward_t(const DistillCall& c, cudaStream_t s) {
  distill_backward_kernel<T><<<grid_of(c.rows), kThreads, 0, s>>>(distill_args<T>(c));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_distill(const DistillCall& c, cudaStream_t s) {
  return c.dtype == TG_F32 ? forward_t<float>(c, s) : forward_t<__nv_bfloat16>(c, s);
}
cudaError_t launch_distill_backward(const DistillCall& c, cudaStream_t s) {
  return c.dtype == TG_F32 ? backward_t<float>(c, s) : backward_t<__nv_bfloat16>(c, s);
}

}  // namespace tg

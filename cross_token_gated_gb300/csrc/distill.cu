// Distillation from a teacher's top logits and its gradient, for training the tied logits
// ("TANGO: Token-Aggregated Nonlinear Gating Operators ...", sec. 2.3).
//
//   p = softmax(t / T) over a row's k entries, q = softmax(z / T) over the vocabulary,
//   loss = T^2 sum_e p_e (ln p_e - ln q_{i_e}),  dz_j = dloss T (q_j - sum_{i_e = j} p_e)
//
// Bound by HBM: the logits are read once and the gradient written once.  A block takes a row at a
// time and keeps it in registers, as the 16-byte vectors that were loaded, from its largest value
// and sum (formed at once, per thread, and joined over one barrier) to its gradient; rows that are
// longer are taken in batches and read again, mostly from L2.  One warp more than the row needs
// prepares the next row's teacher entries and forms the loss meanwhile.
#include <math.h>

#include "tg_common.cuh"
#include "tg_ends.h"
#include "tg_ptx.cuh"
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
// ------------------------------------------------------------------- rows in registers

enum Mode { kLoss, kGradFromStats, kGradAndLoss };

template <typename T> struct Wide;  // 16 bytes of T
template <> struct Wide<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ float largest(const uint4& u) {
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
  }
  static __device__ __forceinline__ void pairs(const uint4& u, uint64_t* p) {
    p[0] = ptx::f32x2_pack(__uint_as_float(u.x), __uint_as_float(u.y));
    p[1] = ptx::f32x2_pack(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <> struct Wide<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ __nv_bfloat162 two(unsigned x) { return *reinterpret_cast<__nv_bfloat162*>(&x); }
  static __device__ __forceinline__ float largest(const uint4& u) {
    const __nv_bfloat162 m = __hmax2(__hmax2(two(u.x), two(u.y)), __hmax2(two(u.z), two(u.w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ void pairs(const uint4& u, uint64_t* p) {
    p[0] = ptx::bf16x2_widen(u.x); p[1] = ptx::bf16x2_widen(u.y); p[2] = ptx::bf16x2_widen(u.z); p[3] = ptx::bf16x2_widen(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]), ptx::pack_bf16x2(f[4], f[5]),
                      ptx::pack_bf16x2(f[6], f[7]));
  }
};

// A row as 16-byte vectors with up to 15 bytes before the first and after the last: rows of any
// width start anywhere.
struct RowSpan {
  int lead, nvec, edge;  // elements before; vectors; elements before and after
};
template <typename T>
__device__ __forceinline__ RowSpan row_span(const T* row, int vocab) {
  constexpr int E = Wide<T>::E;
  RowSpan r;
  r.lead = (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T);
  if (r.lead > vocab) r.lead = vocab;
  r.nvec = (vocab - r.lead) / E;
  r.edge = vocab - r.nvec * E;
  return r;
}
// Column of edge element i.
template <typename T>
__device__ __forceinline__ int edge_col(const RowSpan& r, int i) { return i < r.lead ? i : i + r.nvec * Wide<T>::E; }

// Largest value so far and sum of e^{(z - largest) / T}; -inf and 0 at the start.
struct Running {
  float m, s;
};
__device__ __forceinline__ Running join(Running a, Running b, float c) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return Running{m, a.s + b.s};  // 0, or NaN
  return Running{m, a.s * ptx::ex2_approx((a.m - m) * c) + b.s * ptx::ex2_approx((b.m - m) * c)};
}

// The row's, from its warps'; the largest value as 0 where there is none above -inf.
template <int W>
__device__ __forceinline__ Running row_total(const Running (&part)[W], float c) {
  Running st = part[0];
#pragma unroll
  for (int w = 1; w < W; ++w) st = join(st, part[w], c);
  if (st.m == -INFINITY) st.m = 0.f;
  return st;
}
template <typename T>
__device__ __forceinline__ Running kept_stats(const DistillArgs<T>& a, long long row) {
  const float2 s = *reinterpret_cast<const float2*>(a.stats + 2 * row);
  return Running{s.x, s.y};
}
__device__ __forceinline__ float inverse(float s) { return s == 0.f ? 0.f : 1.f / s; }

// The gradient at the entries' tokens, where the teacher's share comes off: each token by its first
// entry, with the shares of all entries that name it.
template <typename T>
__device__ __forceinline__ void fix_entries(const DistillArgs<T>& a, const Teacher& t, long long row, Running st, int tid, int threads) {
  T* dz = a.dz + row * a.grad_pitch;
  const float f = a.dloss[row] * a.temp, inv = inverse(st.s);
  for (int e = tid; e < a.k; e += threads) {
    const int id = t.id[e];
    if (id < 0) continue;
    float p = 0.f;
    bool first = true;
    for (int i = 0; i < a.k; ++i)
      if (t.id[i] == id) {
        first &= i >= e;
        p += t.p[i];
      }
    if (first) io<T>::st(dz + id, f * (exp2f((t.z[e] - st.m) * a.c) * inv - p));
  }
}

// kRow threads hold the row, NV vectors each at a time; the last warp looks after the teacher.
template <typename T, int kRow, int NV, Mode kMode>
__global__ void __launch_bounds__(kRow + 32, 1088 / (kRow + 32)) distill_row_kernel(const DistillArgs<T> a) {
  constexpr int E = Wide<T>::E, W = kRow / 32;
  __shared__ Teacher te[2];
  __shared__ int any[2];
  __shared__ Running part[2][W];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const bool teacher = warp == W;

  // the entries of a row and their probabilities, by the last warp
  auto prepare = [&](long long row, int side) {
    Teacher& t = te[side];
    const T* z = a.z + row * a.pitch;
    float mx = -INFINITY;
    bool some = false, nan = false;
    for (int e = lane; e < a.k; e += 32) {
      int id = a.ids[row * a.k + e];
      const float v = a.t[row * a.k + e];
      if (id >= a.vocab) record_error(a.err, kErrValue | kKernDistill);
      if (id < 0 || id >= a.vocab || v == -INFINITY) id = -1;
      t.id[e] = id;
      t.p[e] = v;
      t.z[e] = id >= 0 ? io<T>::ld(z + id) : 0.f;
      some |= id >= 0;
      if (id >= 0) mx = fmaxf(mx, v);
      nan |= id >= 0 && v != v;
    }
    some = __any_sync(0xffffffffu, some);
    if (__any_sync(0xffffffffu, nan)) mx = NAN;
    else mx = warp_max(mx);
    float s = 0.f;
    for (int e = lane; e < a.k; e += 32) {
      const float w = t.id[e] >= 0 ? exp2f((t.p[e] - mx) * a.c) : 0.f;
      t.p[e] = w;
      s += w;
    }
    const float inv = 1.f / warp_sum(s);
    for (int e = lane; e < a.k; e += 32) t.p[e] *= inv;
    if (lane == 0) any[side] = some;
  };
  // T^2 sum p (ln p - ln q), by the last warp
  auto loss_of = [&](long long row, int side, Running st, bool some) {
    const Teacher& t = te[side];
    const float lse = logf(st.s);
    float s = 0.f;
    if (some)
      for (int e = lane; e < a.k; e += 32) {
        const float p = t.p[e], z = t.z[e];
        if (t.id[e] >= 0 && p != 0.f) s += p * (logf(p) - (z == -INFINITY ? z : (z - st.m) / a.temp - lse));
      }
    s = warp_sum(s);
    if (lane == 0) a.loss[row] = a.temp * a.temp * s;
  };

  // all threads meet here; the last warp and the others come from different places
  auto meet = [] { ptx::named_bar_sync(1, kRow + 32); };

  int side = 0;
  if (teacher) {
    if (blockIdx.x < a.rows) prepare(blockIdx.x, 0);
    meet();
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, side ^= 1) {
      const bool some = any[side], more = row + gridDim.x < a.rows;
      Running st{0.f, 0.f};
      if (kMode == kLoss && more) prepare(row + gridDim.x, side ^ 1);  // (no other warp reads entries)
      if (kMode == kGradAndLoss || (kMode == kLoss && some)) {
        meet();  // (also in padding: the row before is through with the other buffer)
        if (some) st = row_total(part[side], a.c);
      }
      if (lane == 0 && kMode == kLoss && a.stats_out) *reinterpret_cast<float2*>(a.stats_out + 2 * row) = make_float2(st.m, st.s);
      if (kMode != kGradFromStats && a.loss) loss_of(row, side, st, some);
      if (kMode != kLoss && more) prepare(row + gridDim.x, side ^ 1);
      if (kMode != kLoss || !some) meet();
      if (kMode != kLoss && some) fix_entries(a, te[side], row, kMode == kGradFromStats ? kept_stats(a, row) : st, tid, kRow + 32);
      if (kMode == kGradFromStats && some) meet();
    }
    return;
  }

  const uint64_t cc = ptx::f32x2_pack(a.c, a.c);
  meet();
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, side ^= 1) {
    const T* z = a.z + row * a.pitch;
    T* dz = a.dz + row * a.grad_pitch;
    if (!any[side]) {  // padding
      if (kMode == kGradAndLoss) meet();
      if (kMode != kLoss) {
        const RowSpan r = row_span(dz, a.vocab);
        uint4* v = reinterpret_cast<uint4*>(dz + r.lead);
        for (int i = tid; i < r.nvec; i += kRow) v[i] = make_uint4(0, 0, 0, 0);
        if (tid < r.edge) dz[edge_col<T>(r, tid)] = T(0.f);
      }
      meet();
      continue;
    }
    const RowSpan r = row_span(z, a.vocab);
    uint4 u[NV];
    const float edge = tid < r.edge ? io<T>::ld(z + edge_col<T>(r, tid)) : -INFINITY;
    auto load = [&](int i0) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int i = i0 + k * kRow + tid;
        // -inf elements where there is no vector: they add nothing
        constexpr unsigned none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
        u[k] = i < r.nvec ? reinterpret_cast<const uint4*>(z + r.lead)[i] : make_uint4(none, none, none, none);
      }
    };
    const int batches = (r.nvec + NV * kRow - 1) / (NV * kRow);
    Running st{edge, edge == -INFINITY ? 0.f : edge - edge + 1.f};  // (NaN stays NaN)
    if constexpr (kMode == kGradFromStats) {
      st = kept_stats(a, row);
    } else {
      for (int b = 0; b < batches; ++b) {
        load(b * NV * kRow);
        float m = Wide<T>::largest(u[0]);
#pragma unroll
        for (int k = 1; k < NV; ++k) m = fmaxf(m, Wide<T>::largest(u[k]));
        if (m > st.m) {
          st.s = st.m == -INFINITY ? st.s : st.s * ptx::ex2_approx((st.m - m) * a.c);
          st.m = m;
        }
        const float from = st.m == -INFINITY ? 0.f : st.m;
        const uint64_t neg = ptx::f32x2_pack(-from, -from);
        uint64_t sum = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          uint64_t p[E / 2];
          Wide<T>::pairs(u[k], p);
#pragma unroll
          for (int e = 0; e < E / 2; ++e) {
            float x, y;
            ptx::f32x2_unpack(ptx::mul_f32x2(ptx::add_f32x2(p[e], neg), cc), x, y);
            sum = ptx::add_f32x2(sum, ptx::f32x2_pack(ptx::ex2_approx(x), ptx::ex2_approx(y)));
          }
        }
        float x, y;
        ptx::f32x2_unpack(sum, x, y);
        st.s += x + y;
      }
      // over the warp: its largest value, then its threads' sums
      const float m = warp_max(st.m);
      st.s = warp_sum(st.m == -INFINITY ? st.s : st.s * ptx::ex2_approx((st.m - m) * a.c));
      if (lane == 0) part[side][warp] = Running{m, st.s};
      meet();
      if (kMode == kLoss) continue;
      st = row_total(part[side], a.c);
    }
    if constexpr (kMode != kLoss) {
      const float g = a.dloss[row] * a.temp * inverse(st.s);
      uint4* o = reinterpret_cast<uint4*>(dz + r.lead);
      const uint64_t neg = ptx::f32x2_pack(-st.m, -st.m), gg = ptx::f32x2_pack(g, g);
      // the batch that is still in registers first
      for (int b = batches - 1; b >= 0; --b) {
        if (kMode == kGradFromStats || b < batches - 1) load(b * NV * kRow);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int i = b * NV * kRow + k * kRow + tid;
          uint64_t p[E / 2];
          float q[E];
          Wide<T>::pairs(u[k], p);
#pragma unroll
          for (int e = 0; e < E / 2; ++e) {
            float x, y;
            ptx::f32x2_unpack(ptx::mul_f32x2(ptx::add_f32x2(p[e], neg), cc), x, y);
            ptx::f32x2_unpack(ptx::mul_f32x2(ptx::f32x2_pack(ptx::ex2_approx(x), ptx::ex2_approx(y)), gg), q[2 * e], q[2 * e + 1]);
          }
          if (i < r.nvec) o[i] = Wide<T>::pack(q);
        }
      }
      if (tid < r.edge) io<T>::st(dz + edge_col<T>(r, tid), ptx::ex2_approx((edge - st.m) * a.c) * g);
      meet();
      fix_entries(a, te[side], row, st, tid, kRow + 32);
      if (kMode == kGradFromStats) meet();  // before the entries' buffer is written again
    }
  }
}

// ------------------------------------------------------------------- element by element

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

// Rows of logits and dlogits that are aligned differently: element by element.
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
    const float g = a.dloss[row] * a.temp * inverse(st.y);
    for (int j = threadIdx.x; j < a.vocab; j += kThreads) io<T>::st(dz + j, exp2f((io<T>::ld(z + j) - st.x) * a.c) * g);
    __syncthreads();
    fix_entries(a, te, row, Running{st.x, st.y}, threadIdx.x, kThreads);
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

int grid_of(long long rows, int per_sm) {
  const long long most = (long long)per_sm * serve_sm_count();
  return (int)(rows < most ? rows : most);
}

// Whether a row of dlogits is aligned as its row of logits, so that both are taken in the same vectors.
template <typename T>
bool same_alignment(const DistillArgs<T>& a) {
  constexpr int E = Wide<T>::E;
  return !a.dz || ((reinterpret_cast<uintptr_t>(a.z) - reinterpret_cast<uintptr_t>(a.dz)) % 16 == 0 &&
                   (a.pitch - a.grad_pitch) % E == 0);
}

// Blocks of 512 threads and a warp, two per SM, or of 128 for rows of up to 1,024 vectors.
template <typename T, Mode kMode>
cudaError_t rows_t(const DistillArgs<T>& a, cudaStream_t s) {
  if (a.vocab <= 1024 * Wide<T>::E)
    distill_row_kernel<T, 128, 8, kMode><<<grid_of(a.rows, 6), 160, 0, s>>>(a);
  else
    distill_row_kernel<T, 512, 8, kMode><<<grid_of(a.rows, 2), 544, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t forward_t(const DistillCall& c, cudaStream_t s) { return rows_t<T, kLoss>(distill_args<T>(c), s); }
template <typename T>
cudaError_t backward_t(const DistillCall& c, cudaStream_t s) {
  const DistillArgs<T> a = distill_args<T>(c);
  if (!same_alignment(a)) {
    distill_backward_kernel<T><<<grid_of(c.rows, 4), kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  return c.stats ? rows_t<T, kGradFromStats>(a, s) : rows_t<T, kGradAndLoss>(a, s);
}

}  // namespace

cudaError_t launch_distill(const DistillCall& c, cudaStream_t s) {
  return c.dtype == TG_F32 ? forward_t<float>(c, s) : forward_t<__nv_bfloat16>(c, s);
}
cudaError_t launch_distill_backward(const DistillCall& c, cudaStream_t s) {
  return c.dtype == TG_F32 ? backward_t<float>(c, s) : backward_t<__nv_bfloat16>(c, s);
}

}  // namespace tg

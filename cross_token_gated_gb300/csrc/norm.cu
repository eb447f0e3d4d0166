// RMS and layer norm of rows with their gradients ("TANGO: Token-Aggregated Nonlinear Gating
// Operators ...", sec. 2.1: the pre-norm of the residual stream; sec. 2.3: the final norm).
//
//   n = (x - mu) r,  y = gamma n + beta,  r = 1 / sqrt(mean (x - mu)^2 + eps)   (rms: mu = 0)
//   dn = gamma dy,  dx = r (dn - n <dn n> - <dn>) + dres,  dgamma = sum dy n,  dbeta = sum dy
//
// Means are over the row, <dn> only with mu.  All of it is bound by HBM bandwidth: each value is
// read and written once.  A row stays in the registers of its group of threads (8 lanes to 512
// threads, by the row's length), as the 16-byte vectors that were loaded, and the next
// row is on its way meanwhile.  The gradient needs two joins a row: sum x, then sum (x - mu)^2,
// sum dn and sum dn (x - mu) at once (rms: one).  A thread keeps its columns' dgamma and dbeta in
// registers over all rows of its persistent block; a second kernel adds up the blocks' sums.
//
// Layer norm of 65,536 x 768 bf16: 35.5 us (5.7 TB/s; issue slots are 77 % full).  Gradients of 16,384 x
// 512 bf16 with a residual's: 14.6 us from L2 (4.6 TB/s), 23 us cold; of 5,003 x 768 fp32: 14.5 us, two
// launches.
#include "tg_common.cuh"
#include "tg_ends.h"
#include "tg_ptx.cuh"
#include "tg_serve.h"
#include "tg_vec.cuh"

#include <type_traits>

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

// ------------------------------------------------------------------- rows in registers

// A thread's share of a row comes in vectors: 16 bytes, or single values where rows are not aligned.
template <typename T>
struct Wide : Vec16<T> {
  using Value = T;
  using Raw = uint4;
  static __device__ __forceinline__ uint4 shared(uint32_t a) { return ptx::ld_shared_v4(a); }
};
template <typename T> struct Single;
template <> struct Single<float> {
  using Value = float;
  using Raw = uint32_t;
  static constexpr int E = 1;
  static __device__ __forceinline__ void unpack(uint32_t u, float* f) { f[0] = __uint_as_float(u); }
  static __device__ __forceinline__ uint32_t pack(const float* f) { return __float_as_uint(f[0]); }
  static __device__ __forceinline__ uint32_t shared(uint32_t a) {
    uint32_t u;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(u) : "r"(a));
    return u;
  }
};
template <> struct Single<__nv_bfloat16> {
  using Value = __nv_bfloat16;
  using Raw = uint16_t;
  static constexpr int E = 1;
  static __device__ __forceinline__ void unpack(uint16_t u, float* f) { f[0] = __uint_as_float((uint32_t)u << 16); }
  static __device__ __forceinline__ uint16_t pack(const float* f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f[0])); }
  static __device__ __forceinline__ uint16_t shared(uint32_t a) {
    uint16_t u;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(u) : "r"(a));
    return u;
  }
};
__device__ __forceinline__ float inv_sqrt(float v, float) { return 1.f / sqrtf(v); }
__device__ __forceinline__ float inv_sqrt(float v, __nv_bfloat16) { return rsqrtf(v); }  // 2 units: far below a bf16 rounding

template <int kGroup> constexpr int kBlock = kGroup > 256 ? kGroup : 256;

// Blocks of the persistent grids per SM.
template <int kGroup> constexpr int kForwardPerSm = kGroup > 256 ? 2 : 4;
// (gradients of 16,384 x 512 from L2: 2 blocks of 256 threads 14.6 us, 3 of them, or 2 of 384, 18.6 us)
template <int kGroup> constexpr int kBackwardPerSm = kGroup > 256 ? 1 : 2;

// Sums over the group of K values at a time; every thread gets them.  Groups of several warps join
// through shared memory, in two buffers taken in turn (all groups of a block make the same calls).
template <int kGroup, int K, int kWarpsOfBlock>
struct GroupSum {
  float (*buf)[K][kWarpsOfBlock];
  int side = 0;
  __device__ __forceinline__ void operator()(float (&v)[K]) {
    constexpr int W = kGroup / 32;
#pragma unroll
    for (int o = (kGroup < 32 ? kGroup : 32) / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < K; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (W > 1) {
      const int warp = threadIdx.x / 32;
      if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < K; ++i) buf[side][i][warp] = v[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < K; ++i) {
        v[i] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) v[i] += buf[side][i][warp / W * W + w];
      }
      side ^= 1;
    }
  }
};

// One row of the group's: NV vectors a thread, vector k * kGroup + lane.
template <int kGroup, int NV, typename Raw>
__device__ __forceinline__ void load_row(Raw (&u)[NV], const void* row, int lane, int nvec, bool live) {
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = k * kGroup + lane;
    u[k] = live && i < nvec ? reinterpret_cast<const Raw*>(row)[i] : Raw();
  }
}

// gamma and beta (or ones and zeros) as vectors in shared memory: kept in registers they would cost
// more warps an SM than their reading costs time.
template <typename V>
__device__ __forceinline__ void stage_vector(typename V::Raw* dst, const typename V::Value* src, float otherwise, int nvec) {
  float f[V::E];
#pragma unroll
  for (int e = 0; e < V::E; ++e) f[e] = otherwise;
  const typename V::Raw none = V::pack(f);
  for (int i = threadIdx.x; i < nvec; i += blockDim.x) dst[i] = src ? reinterpret_cast<const typename V::Raw*>(src)[i] : none;
}

template <typename V, int kGroup, int NV>
__global__ void __launch_bounds__(kBlock<kGroup>, kForwardPerSm<kGroup>) norm_kernel(const NormArgs<typename V::Value> a) {
  using Raw = typename V::Raw;
  constexpr int E = V::E, B = kBlock<kGroup>, kRows = B / kGroup;
  extern __shared__ __align__(16) uint4 weights[];  // [2][nvec]: gamma, beta
  __shared__ float buf[2][1][B / 32];
  GroupSum<kGroup, 1, B / 32> sum{buf};
  const int lane = threadIdx.x % kGroup, nvec = a.d / E;
  const float inv_d = 1.f / (float)a.d;
  Raw* const staged = reinterpret_cast<Raw*>(weights);
  stage_vector<V>(staged, a.gamma, 1.f, nvec);
  stage_vector<V>(staged + nvec, a.beta, 0.f, nvec);
  const uint32_t g = ptx::smem_u32(weights);
  Raw u[NV];
  const long long step = (long long)gridDim.x * kRows;
  long long row = (long long)blockIdx.x * kRows + threadIdx.x / kGroup, row0 = (long long)blockIdx.x * kRows;
  load_row<kGroup>(u, a.x + row * a.x_pitch, lane, nvec, row < a.rows);
  __syncthreads();
  for (; row0 < a.rows; row0 += step, row += step) {
    Raw next[NV];
    load_row<kGroup>(next, a.x + (row + step) * a.x_pitch, lane, nvec, row + step < a.rows);
    float mu = 0.f;
    if (a.layer) {
      float s[1] = {0.f};
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float f[E];
        V::unpack(u[k], f);
#pragma unroll
        for (int e = 0; e < E; ++e) s[0] += f[e];
      }
      sum(s);
      mu = s[0] * inv_d;
    }
    float ss[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (k * kGroup + lane >= nvec) continue;
      float f[E];
      V::unpack(u[k], f);
#pragma unroll
      for (int e = 0; e < E; ++e) ss[0] = fmaf(f[e] - mu, f[e] - mu, ss[0]);
    }
    sum(ss);
    const float r = inv_sqrt(fmaf(ss[0], inv_d, a.eps), typename V::Value());
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = k * kGroup + lane;
      if (row >= a.rows || i >= nvec) continue;
      float f[E], gf[E], bf[E];
      V::unpack(u[k], f);
      V::unpack(V::shared(g + i * (int)sizeof(Raw)), gf);
      V::unpack(V::shared(g + (nvec + i) * (int)sizeof(Raw)), bf);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = fmaf((f[e] - mu) * r, gf[e], bf[e]);
      reinterpret_cast<Raw*>(a.y + row * a.d)[i] = V::pack(f);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) u[k] = next[k];
  }
}

// The block's sums of dgamma or dbeta, of its groups in order, into its row of part.
template <int kGroup, int NV, int E>
__device__ __forceinline__ void block_columns(const float (&acc)[NV * E], float* sh, float* dst, int d) {
  constexpr int B = kBlock<kGroup>, kRows = B / kGroup;
  const int lane = threadIdx.x % kGroup, nvec = d / E;
  float* mine = kRows > 1 ? sh + (threadIdx.x / kGroup) * d : dst;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = k * kGroup + lane;
    if (i >= nvec) continue;
    if constexpr (E == 1) {
      mine[i] = acc[k];
    } else {
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<float4*>(mine + i * E + e) = make_float4(acc[k * E + e], acc[k * E + e + 1], acc[k * E + e + 2], acc[k * E + e + 3]);
    }
  }
  if constexpr (kRows > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += B) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kRows; ++w) s += sh[w * d + c];
      dst[c] = s;
    }
    __syncthreads();
  }
}

template <typename V, int kGroup, int NV, bool kBeta>
__global__ void __launch_bounds__(kBlock<kGroup>, kBackwardPerSm<kGroup>) norm_backward_kernel(const NormArgs<typename V::Value> a) {
  using Raw = typename V::Raw;
  constexpr int E = V::E, B = kBlock<kGroup>, kRows = B / kGroup;
  extern __shared__ __align__(16) uint4 weights[];  // gamma [nvec], then float [kRows][d], where kRows > 1
  __shared__ float buf1[2][1][B / 32], buf3[2][3][B / 32];
  GroupSum<kGroup, 1, B / 32> sum1{buf1};
  GroupSum<kGroup, 3, B / 32> sum3{buf3};
  const int lane = threadIdx.x % kGroup, nvec = a.d / E;
  const float inv_d = 1.f / (float)a.d;
  stage_vector<V>(reinterpret_cast<Raw*>(weights), a.gamma, 1.f, nvec);
  const uint32_t g = ptx::smem_u32(weights);
  float* columns = reinterpret_cast<float*>(weights + (nvec * (int)sizeof(Raw) + 15) / 16);
  Raw x[NV], y[NV];
  float dg[NV * E] = {}, db[kBeta ? NV * E : 1] = {};
  const long long step = (long long)gridDim.x * kRows;
  long long row = (long long)blockIdx.x * kRows + threadIdx.x / kGroup, row0 = (long long)blockIdx.x * kRows;
  load_row<kGroup>(x, a.x + row * a.x_pitch, lane, nvec, row < a.rows);
  load_row<kGroup>(y, a.dy + row * a.d, lane, nvec, row < a.rows);
  __syncthreads();
  for (; row0 < a.rows; row0 += step, row += step) {
    Raw res[NV], next_x[NV], next_y[NV];
    const bool live = row < a.rows, more = row + step < a.rows;
    load_row<kGroup>(res, a.dres + row * a.d, lane, nvec, live && a.dres);
    load_row<kGroup>(next_x, a.x + (row + step) * a.x_pitch, lane, nvec, more);
    load_row<kGroup>(next_y, a.dy + (row + step) * a.d, lane, nvec, more);
    float mu = 0.f;
    if (a.layer) {
      float s[1] = {0.f};
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float f[E];
        V::unpack(x[k], f);
#pragma unroll
        for (int e = 0; e < E; ++e) s[0] += f[e];
      }
      sum1(s);
      mu = s[0] * inv_d;
    }
    float s[3] = {0.f, 0.f, 0.f};  // (x - mu)^2, dn (x - mu), dn
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (k * kGroup + lane >= nvec) continue;
      float f[E], h[E], gf[E];
      V::unpack(x[k], f);
      V::unpack(y[k], h);
      V::unpack(V::shared(g + (k * kGroup + lane) * (int)sizeof(Raw)), gf);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float c = f[e] - mu, dn = h[e] * gf[e];
        s[0] = fmaf(c, c, s[0]);
        s[1] = fmaf(dn, c, s[1]);
        s[2] += dn;
      }
    }
    sum3(s);
    const float r = inv_sqrt(fmaf(s[0], inv_d, a.eps), typename V::Value());
    const float m1 = s[1] * inv_d * r, m0 = a.layer ? s[2] * inv_d : 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = k * kGroup + lane;
      if (!live || i >= nvec) continue;
      float f[E], h[E], gf[E], rf[E];
      V::unpack(x[k], f);
      V::unpack(y[k], h);
      V::unpack(V::shared(g + i * (int)sizeof(Raw)), gf);
      V::unpack(res[k], rf);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float n = (f[e] - mu) * r, dn = h[e] * gf[e];
        dg[k * E + e] = fmaf(h[e], n, dg[k * E + e]);
        if constexpr (kBeta) db[k * E + e] += h[e];
        f[e] = fmaf(r, dn - fmaf(n, m1, m0), rf[e]);
      }
      reinterpret_cast<Raw*>(a.dx + row * a.d)[i] = V::pack(f);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      x[k] = next_x[k];
      y[k] = next_y[k];
    }
  }
  let_next_start();
  if (a.want_gamma) block_columns<kGroup, NV, E>(dg, columns, a.part + (size_t)blockIdx.x * a.d, a.d);
  if constexpr (kBeta) block_columns<kGroup, NV, E>(db, columns, a.part + ((size_t)gridDim.x + blockIdx.x) * a.d, a.d);
}

// dgamma (blockIdx.y 0) and dbeta (1): 32 columns a block, each by 32 threads that take every 32nd
// of the blocks' partial sums.  Launched while the last blocks still run.
__global__ void __launch_bounds__(1024) norm_weight_sum_kernel(const float* part, int blocks, int d, float* dgamma,
                                                               float* dbeta) {
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  float* dst = blockIdx.y ? dbeta : dgamma;
  wait_for_previous();
  if (!dst) return;
  float s = 0.f;
  if (c < d) {
    const float* p = part + (size_t)blockIdx.y * blocks * d + c;
#pragma unroll 4
    for (int b = warp; b < blocks; b += 32) s += __ldcg(p + (size_t)b * d);
  }
  sh[warp][lane] = s;
  __syncthreads();
  s = sh[lane][warp];
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0 && blockIdx.x * 32 + warp < d) dst[blockIdx.x * 32 + warp] = s;
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

// Whether rows are taken 16 bytes at a time and fit the registers of at most 512 threads.
template <typename T>
bool in_registers(const NormArgs<T>& a) {
  constexpr int E = Wide<T>::E;
  const void* ptrs[] = {a.x, a.gamma, a.beta, a.dy, a.dres, a.y, a.dx};
  for (const void* p : ptrs)
    if (!aligned_16(p)) return false;
  return a.d % E == 0 && a.x_pitch % E == 0 && a.d / E <= 2048;
}

// Calls f with the group and the vectors of a thread for a row of nvec: as few threads as hold it in
// 2 or 3 vectors each, so that rows enough are under way (5,003 fp32 rows of 768: 64 threads with 3).
template <typename F>
auto by_length(int nvec, F f) {
  using std::integral_constant;
#define TG_CASE(G, N) f(integral_constant<int, G>(), integral_constant<int, N>())
  if (nvec <= 8) return TG_CASE(8, 1);
  if (nvec <= 16) return TG_CASE(8, 2);
  if (nvec <= 32) return TG_CASE(32, 1);
  if (nvec <= 64) return TG_CASE(32, 2);
  if (nvec <= 96) return TG_CASE(32, 3);
  if (nvec <= 128) return TG_CASE(64, 2);
  if (nvec <= 192) return TG_CASE(64, 3);
  if (nvec <= 256) return TG_CASE(128, 2);
  if (nvec <= 384) return TG_CASE(128, 3);
  if (nvec <= 512) return TG_CASE(256, 2);
  if (nvec <= 768) return TG_CASE(256, 3);
  if (nvec <= 1024) return TG_CASE(512, 2);
  if (nvec <= 1536) return TG_CASE(512, 3);
  return TG_CASE(512, 4);
#undef TG_CASE
}

// The same for rows of n single values, 4 or 8 of a thread (16 of the longest).
constexpr int kMostSingles = 8192;
template <typename F>
auto by_count(int n, F f) {
  using std::integral_constant;
#define TG_CASE(G, N) f(integral_constant<int, G>(), integral_constant<int, N>())
  if (n <= 32) return TG_CASE(8, 4);
  if (n <= 128) return TG_CASE(32, 4);
  if (n <= 256) return TG_CASE(32, 8);
  if (n <= 512) return TG_CASE(64, 8);
  if (n <= 1024) return TG_CASE(128, 8);
  if (n <= 2048) return TG_CASE(256, 8);
  if (n <= 4096) return TG_CASE(512, 8);
  return TG_CASE(512, 16);
#undef TG_CASE
}

// Dynamic shared memory that a kernel may have without asking: 48 KB with its static variables, which are
// less than 1 KB here.
constexpr int kDefaultSmem = 47 * 1024;

template <typename V, int G, int N>
cudaError_t forward_in(const NormArgs<typename V::Value>& a, cudaStream_t s) {
  constexpr int B = kBlock<G>, R = B / G;
  const int smem = 2 * a.d * (int)sizeof(typename V::Value);
  // the limit is the longest rows', whatever these are: another thread's lower one might come before the launch
  constexpr int kMost = 2 * G * N * (int)sizeof(typename V::Raw);
  if constexpr (kMost > kDefaultSmem) {
    const cudaError_t e = cudaFuncSetAttribute(norm_kernel<V, G, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
  }
  norm_kernel<V, G, N><<<grid_of((a.rows + R - 1) / R, kForwardPerSm<G>), B, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename V, int G, int N>
cudaError_t backward_in(const NormArgs<typename V::Value>& a, int* grid, cudaStream_t s) {
  constexpr int B = kBlock<G>, R = B / G;
  const auto kernel = a.want_beta ? norm_backward_kernel<V, G, N, true> : norm_backward_kernel<V, G, N, false>;
  const int smem = (a.d * (int)sizeof(typename V::Value) + 15) / 16 * 16 + (R > 1 ? R * a.d * 4 : 0);
  static_assert(G * N * (int)sizeof(typename V::Raw) + (R > 1 ? R * G * N * V::E * 4 : 0) <= kDefaultSmem);
  *grid = grid_of((a.rows + R - 1) / R, kBackwardPerSm<G>);
  kernel<<<*grid, B, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t norm_t(const NormCall& c, cudaStream_t s) {
  const NormArgs<T> a = norm_args<T>(c);
  if (in_registers(a))
    return by_length(c.d / Wide<T>::E, [&](auto group, auto n) {
      return forward_in<Wide<T>, decltype(group)::value, decltype(n)::value>(a, s);
    });
  if (c.d <= kMostSingles)
    return by_count(c.d, [&](auto group, auto n) {
      return forward_in<Single<T>, decltype(group)::value, decltype(n)::value>(a, s);
    });
  norm_any_kernel<T><<<grid_of(c.rows, 8), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t norm_backward_t(const NormCall& c, cudaStream_t s) {
  const NormArgs<T> a = norm_args<T>(c);
  int grid = grid_of(c.rows, kBwdPerSm);
  cudaError_t e;
  if (in_registers(a)) {
    e = by_length(c.d / Wide<T>::E, [&](auto group, auto n) {
      return backward_in<Wide<T>, decltype(group)::value, decltype(n)::value>(a, &grid, s);
    });
  } else if (c.d <= kMostSingles) {
    e = by_count(c.d, [&](auto group, auto n) {
      return backward_in<Single<T>, decltype(group)::value, decltype(n)::value>(a, &grid, s);
    });
  } else {
    norm_backward_any_kernel<T><<<grid, kThreads, 0, s>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || !(c.dgamma || c.dbeta)) return e;
  return launch_early(norm_weight_sum_kernel, dim3(ceil_div(c.d, 32), 2), 1024, s, (const float*)a.part, grid, c.d, c.dgamma, c.dbeta);
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

// Distillation from a teacher's top logits and its gradient, for training the tied logits
// ("TANGO: Token-Aggregated Nonlinear Gating Operators ...", sec. 2.3).
//
//   p = softmax(t / T) over a row's k entries, q = softmax(z / T) over the vocabulary,
//   loss = T^2 sum_e p_e (ln p_e - ln q_{i_e}),  dz_j = dloss T (q_j - sum_{i_e = j} p_e)
//
// Bound by HBM: the logits are read once and the gradient written once.  A block takes a row at a
// time and keeps it in registers, as the 16-byte vectors that were loaded, from its largest value
// and sum (formed at once, per thread, and joined over one barrier) to its gradient; rows that are
// longer are taken in batches and read again, mostly from L2.  The next vectors are on their way to
// shared memory meanwhile.  One or two warps more than the row needs prepare the next rows' teacher
// entries, in steps a row apart so that none waits for its loads, and form the loss.
//
// Loss of 8,192 rows of 32,768 bf16 logits: 90 us (6.0 TB/s of a measured copy's 6.8); without the
// fetch ahead and the steps 154 us.  Gradient of 16,384 rows: 338 us (6.4 TB/s), 547 us without.
#include <math.h>

#include "tg_common.cuh"
#include "tg_ends.h"
#include "tg_ptx.cuh"
#include "tg_serve.h"
#include "tg_vec.cuh"

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

template <typename T> struct Wide;
template <> struct Wide<float> : Vec16<float> {
  static __device__ __forceinline__ float largest(const uint4& u) {
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
  }
  static __device__ __forceinline__ void pairs(const uint4& u, uint64_t* p) {
    p[0] = ptx::f32x2_pack(__uint_as_float(u.x), __uint_as_float(u.y));
    p[1] = ptx::f32x2_pack(__uint_as_float(u.z), __uint_as_float(u.w));
  }
};
template <> struct Wide<__nv_bfloat16> : Vec16<__nv_bfloat16> {
  static __device__ __forceinline__ __nv_bfloat162 two(unsigned x) { return *reinterpret_cast<__nv_bfloat162*>(&x); }
  static __device__ __forceinline__ float largest(const uint4& u) {
    const __nv_bfloat162 m = __hmax2(__hmax2(two(u.x), two(u.y)), __hmax2(two(u.z), two(u.w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ void pairs(const uint4& u, uint64_t* p) {
    p[0] = ptx::bf16x2_widen(u.x); p[1] = ptx::bf16x2_widen(u.y); p[2] = ptx::bf16x2_widen(u.z); p[3] = ptx::bf16x2_widen(u.w);
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
  r.lead = row_lead(row, vocab);
  r.nvec = (vocab - r.lead) / E;
  r.edge = vocab - r.nvec * E;
  return r;
}
// Column of edge element i.
template <typename T>
__device__ __forceinline__ int edge_col(const RowSpan& r, int i) { return i < r.lead ? i : i + r.nvec * Wide<T>::E; }

// Largest value and sum of e^{(z - largest) / T} of a part of a row; -inf and 0 without elements.
struct Running {
  float m, s;
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait_but() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The row's, from its warps' by a whole warp; the largest value as 0 where there is none above -inf.
template <int W>
__device__ __forceinline__ Running row_total(const Running (&part)[W], float c) {
  static_assert(W <= 32 && (W & (W - 1)) == 0, "warps of a row");
  Running st = part[threadIdx.x & (W - 1)];
  float m = st.m;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (m == -INFINITY) m = 0.f;
  st.s = st.m == -INFINITY ? st.s : st.s * ptx::ex2_approx((st.m - m) * c);
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) st.s += __shfl_xor_sync(0xffffffffu, st.s, o);
  return Running{m, st.s};
}
template <typename T>
__device__ __forceinline__ Running kept_stats(const DistillArgs<T>& a, long long row) {
  const float2 s = *reinterpret_cast<const float2*>(a.stats + 2 * row);
  return Running{s.x, s.y};
}
__device__ __forceinline__ float inverse(float s) { return s == 0.f ? 0.f : 1.f / s; }

constexpr int kSlots = 8;  // rows whose entries are held

// A row's entries (dynamic shared memory, k of each).
struct Entries {
  int* id;      // -1: absent, or another entry stands for the token
  float* p;     // probability
  float* z;     // the student's logit
  float* share; // sum of p over the entries of this token
};
// What the loss needs of a row's entries: sums of p ln p and p (z - z0) / T, and z0, the largest z.
struct Target {
  float plogp, pz, z0;
};
constexpr int kSeenWords = 1024;  // one bit per token, modulo 32,768

// The gradient at the entries' tokens, where the teacher's share comes off.
template <typename T>
__device__ __forceinline__ void fix_entries(const DistillArgs<T>& a, const Entries& t, T* dz, float f, Running st, int tid,
                                            int threads) {
  const float inv = inverse(st.s);
  for (int e = tid; e < a.k; e += threads)
    if (t.id[e] >= 0) io<T>::st(dz + t.id[e], f * (exp2f((t.z[e] - st.m) * a.c) * inv - t.share[e]));
}

// The teacher's warp takes a row's entries in three steps, a row apart each, so that no step waits
// for its loads: ids and logits on their way to shared memory; the student's logits there; the
// probabilities.
template <typename T>
__device__ __forceinline__ void fetch_entries(const DistillArgs<T>& a, long long row, const Entries& t, int lane) {
  for (int e = lane; e < a.k; e += 32) {
    cp_async4(t.id + e, a.ids + row * a.k + e);
    cp_async4(t.p + e, a.t + row * a.k + e);
  }
}

constexpr int kGather = 8;  // student's logits of a lane that are under way at a time

// Ids to -1 where an entry is absent; whether any is left.  The first logits are left in z.
template <typename T>
__device__ __forceinline__ bool begin_gather(const DistillArgs<T>& a, long long row, const Entries& t, int lane, T (&z)[kGather]) {
  bool some = false;
  const T* src = a.z + row * a.pitch;
  for (int e0 = 0; e0 < a.k; e0 += 32 * kGather) {
    T x[kGather];  // (all of them asked for before the first is stored)
#pragma unroll
    for (int j = 0; j < kGather; ++j) {
      const int e = e0 + 32 * j + lane;
      int id = -1;
      if (e < a.k) {
        id = t.id[e];
        if (id >= a.vocab) record_error(a.err, kErrValue | kKernDistill);
        if (id < 0 || id >= a.vocab || t.p[e] == -INFINITY) t.id[e] = id = -1;
        some |= id >= 0;
      }
      x[j] = id >= 0 ? src[id] : T(0.f);
    }
#pragma unroll
    for (int j = 0; j < kGather; ++j) {
      if (e0 == 0) z[j] = x[j];
      else if (e0 + 32 * j + lane < a.k) t.z[e0 + 32 * j + lane] = (float)x[j];
    }
  }
  return __any_sync(0xffffffffu, some);
}
template <typename T>
__device__ __forceinline__ void end_gather(const DistillArgs<T>& a, const Entries& t, int lane, const T (&z)[kGather]) {
#pragma unroll
  for (int j = 0; j < kGather; ++j)
    if (32 * j + lane < a.k) t.z[32 * j + lane] = (float)z[j];
}

// Largest of a warp's floats (none NaN), by one reduction of integers in the same order.
__device__ __forceinline__ float warp_largest(float v) {
  const unsigned b = __float_as_uint(v), m = __reduce_max_sync(0xffffffffu, b & 0x80000000u ? ~b : b | 0x80000000u);
  return __uint_as_float(m & 0x80000000u ? m & 0x7fffffffu : ~m);
}

// The probabilities; `seen` holds zeros before and after.
template <typename T>
__device__ __forceinline__ Target finish_entries(const DistillArgs<T>& a, const Entries& t, unsigned* seen, int lane, bool shares) {
  float mx = -INFINITY;
  Target g{0.f, 0.f, -INFINITY};
  bool nan = false;
#pragma unroll 4
  for (int e = lane; e < a.k; e += 32) {
    const float v = t.p[e], z = t.z[e];
    const bool live = t.id[e] >= 0;
    mx = fmaxf(mx, live ? v : -INFINITY);
    g.z0 = fmaxf(g.z0, live ? z : -INFINITY);
    nan |= live && v != v;
  }
  mx = warp_largest(mx);
  g.z0 = warp_largest(g.z0);
  if (__any_sync(0xffffffffu, nan)) mx = NAN;
  if (g.z0 == -INFINITY) g.z0 = 0.f;
  float s = 0.f;
#pragma unroll 4
  for (int e = lane; e < a.k; e += 32) {
    const float y = t.id[e] >= 0 ? (t.p[e] - mx) * a.c : -INFINITY, w = exp2f(y);
    t.p[e] = w;
    s += w;
    if (w != 0.f) {  // (also NaN)
      g.plogp = fmaf(w, y, g.plogp);
      g.pz = fmaf(w, t.z[e] - g.z0, g.pz);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    g.plogp += __shfl_xor_sync(0xffffffffu, g.plogp, o);
    g.pz += __shfl_xor_sync(0xffffffffu, g.pz, o);
  }
  const float inv = 1.f / s;
  g.plogp = fmaf(g.plogp * inv, 0.69314718f, -logf(s));
  g.pz = g.pz * inv / a.temp;
#pragma unroll 4
  for (int e = lane; e < a.k; e += 32) t.share[e] = t.p[e] * inv;
  if (!shares) return g;
  // Entries that may name a token a second time (or one that differs by a multiple of 32,768), by
  // lane and number; the token's entries are taken together under the first of them.
  unsigned late = 0;
#pragma unroll 4
  for (int e = lane; e < a.k; e += 32) {
    const int id = t.id[e];
    const unsigned bit = 1u << (id & 31);
    if (id >= 0 && (atomicOr(seen + (id >> 5 & (kSeenWords - 1)), bit) & bit)) late |= 1u << (e >> 5);
  }
  __syncwarp();
#pragma unroll 4
  for (int e = lane; e < a.k; e += 32)
    if (t.id[e] >= 0) seen[t.id[e] >> 5 & (kSeenWords - 1)] = 0;
  __syncwarp();
  if (!__any_sync(0xffffffffu, late != 0)) return g;
  for (int c = 0; 32 * c < a.k; ++c) {
    for (unsigned todo = __ballot_sync(0xffffffffu, late >> c & 1); todo; todo &= todo - 1) {
      const int token = t.id[32 * c + __ffs(todo) - 1];
      if (token < 0) continue;  // already taken together
      int first = -1;
      float sum = 0.f;
      for (int i0 = 0; i0 < a.k; i0 += 32) {
        const bool same = i0 + lane < a.k && t.id[i0 + lane] == token;
        const unsigned who = __ballot_sync(0xffffffffu, same);
        if (first < 0 && who) first = i0 + __ffs(who) - 1;
        for (unsigned w = who; w; w &= w - 1) sum += t.share[i0 + __ffs(w) - 1];
        if (same && i0 + lane != first) t.id[i0 + lane] = -1;
      }
      __syncwarp();
      if (lane == 0) t.share[first] = sum;
      __syncwarp();
    }
  }
  return g;
}

// Warps that look after the teacher: one, or, where the row's own time is short beside theirs, one
// that gathers the entries and one that forms probabilities and loss.
template <Mode kMode, int kRow> constexpr int kTeachers = kMode == kGradAndLoss && kRow == 512 ? 2 : 1;

// kRow threads hold the row, NV vectors each at a time; the next ones are on their way to shared
// memory meanwhile, each to a slot of the thread that will read it.  The last warps look after the
// teacher.
template <typename T, int kRow, int NV, Mode kMode>
__global__ void __launch_bounds__(kRow + 32 * kTeachers<kMode, kRow>, kRow == 512 ? 2 : kRow == 256 ? 4 : kRow == 128 ? 6 : 16)
    distill_row_kernel(const DistillArgs<T> a) {
  constexpr int E = Wide<T>::E, W = kRow / 32, kAll = kRow + 32 * kTeachers<kMode, kRow>;
  extern __shared__ __align__(16) uint4 ahead[];  // [NV][kRow], then the entries of kSlots rows
  __shared__ int any[kSlots];                     // whether a row has entries: of this row and the next ones
  __shared__ unsigned seen[kSeenWords];
  __shared__ Running part[2][W];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  float* const words = reinterpret_cast<float*>(ahead + NV * kRow);
  auto entries = [&](int n) {
    float* w = words + (n & (kSlots - 1)) * 4 * a.k;
    return Entries{reinterpret_cast<int*>(w), w + a.k, w + 2 * a.k, w + 3 * a.k};
  };
  auto has_entries = [&](int n) { return any[n & (kSlots - 1)] != 0; };
  // all threads meet here; the last warps and the others come from different places
  auto meet = [] { ptx::named_bar_sync(1, kAll); };
  const long long step = gridDim.x;
  int n = 0;  // rows so far

  if (warp >= W) {
    // of row n: the loss; of n + 1: the probabilities; of n + 2: logits arrive; of n + 3: they are
    // asked for; of n + 5: ids and the teacher's logits are asked for
    const bool finishes = warp == W, gathers = warp == W + kTeachers<kMode, kRow> - 1;
    const long long row0 = blockIdx.x;
    const int rows = (int)((a.rows - row0 + step - 1) / step);  // of this block
    T z[kGather];
    bool arriving = false;  // row n + 2 has logits under way
    Target now{0.f, 0.f, 0.f}, ahead_of{0.f, 0.f, 0.f};  // of rows n and n + 1
    if (gathers) {
      for (int i = lane; i < kSeenWords; i += 32) seen[i] = 0;
      for (int i = 0; i < 5 && i < rows; ++i) fetch_entries(a, row0 + i * step, entries(i), lane);
      cp_async_wait();
      __syncwarp();
#pragma unroll 1
      for (int i = 0; i < 3; ++i) {
        const bool live = i < rows && begin_gather(a, row0 + i * step, entries(i), lane, z);
        if (live) end_gather(a, entries(i), lane, z);
        if (lane == 0) any[i] = live;
      }
    }
    if (kTeachers<kMode, kRow> > 1) ptx::named_bar_sync(2, 64);
    else __syncwarp();
    if (finishes && has_entries(0)) now = finish_entries(a, entries(0), seen, lane, kMode != kLoss);
    meet();
    for (; n < rows; ++n) {
      const long long row = row0 + n * step;
      const bool live = has_entries(n);
      auto look_ahead = [&] {
        if (gathers) {
          cp_async_wait_but<1>();
          __syncwarp();
          if (arriving) end_gather(a, entries(n + 2), lane, z);
          arriving = n + 3 < rows && begin_gather(a, row + 3 * step, entries(n + 3), lane, z);
          if (lane == 0) any[(n + 3) & (kSlots - 1)] = arriving;
          if (n + 5 < rows) fetch_entries(a, row + 5 * step, entries(n + 5), lane);
          cp_async_commit();
        }
        if (finishes && n + 1 < rows && has_entries(n + 1))
          ahead_of = finish_entries(a, entries(n + 1), seen, lane, kMode != kLoss);
      };
      if (kMode == kGradAndLoss) look_ahead();
      Running st{0.f, 0.f};
      if (kMode == kGradAndLoss || (kMode == kLoss && live)) {
        meet();  // (also in padding: one step for all)
        if (live) st = row_total(part[n & 1], a.c);
      }
      if (finishes && lane == 0 && kMode == kLoss && a.stats_out)
        *reinterpret_cast<float2*>(a.stats_out + 2 * row) = make_float2(st.m, st.s);
      // sum p (ln p - ln q), ln q_e = (z_e - z0) / T + (z0 - m) / T - ln sum; inf where an entry has z = -inf
      if (finishes && kMode != kGradFromStats && a.loss && lane == 0) {
        float loss = now.plogp - now.pz - (now.z0 - st.m) / a.temp + logf(st.s);
        if (now.pz == -INFINITY) loss = INFINITY + 0.f * st.s;  // (NaN if the row has one)
        a.loss[row] = live ? a.temp * a.temp * loss : 0.f;
      }
      if (kMode != kGradAndLoss) look_ahead();
      if (kMode != kLoss || !live) meet();
      now = ahead_of;
    }
    return;
  }

  const uint64_t cc = ptx::f32x2_pack(a.c, a.c);
  uint4* const slot = ahead + tid;
  auto fetch = [&](const T* z, int batch) {
    const RowSpan r = row_span(z, a.vocab);
    const uint4* v = reinterpret_cast<const uint4*>(z + r.lead);
    if ((batch + 1) * NV * kRow <= r.nvec) {
      v += batch * NV * kRow + tid;
#pragma unroll
      for (int k = 0; k < NV; ++k) cp_async16(slot + k * kRow, v + k * kRow);
      return;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (batch * NV + k) * kRow + tid;
      constexpr unsigned none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
      // -inf elements where there is no vector: they add nothing
      if (i < r.nvec) cp_async16(slot + k * kRow, v + i);
      else slot[k * kRow] = make_uint4(none, none, none, none);
    }
  };
  meet();
  if (has_entries(0)) fetch(a.z + blockIdx.x * a.pitch, 0);
  for (long long row = blockIdx.x; row < a.rows; row += step, ++n) {
    const T* z = a.z + row * a.pitch;
    T* dz = a.dz + row * a.grad_pitch;
    const bool next = row + step < a.rows && has_entries(n + 1);
    if (!has_entries(n)) {  // padding
      if (next) fetch(z + step * a.pitch, 0);
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
    const float edge = tid < r.edge ? io<T>::ld(z + edge_col<T>(r, tid)) : -INFINITY;
    // batches in order, then back (the last one is still in registers) for the gradient
    const int batches = max(1, (r.nvec + NV * kRow - 1) / (NV * kRow));
    const int tiles = kMode == kGradAndLoss ? 2 * batches - 1 : batches;
    uint4 u[NV];
    auto take = [&](int tile) {  // this batch into registers, and the next one on its way
      cp_async_wait();
#pragma unroll
      for (int k = 0; k < NV; ++k) u[k] = slot[k * kRow];
      if (tile + 1 < tiles) fetch(z, tile + 1 < batches ? tile + 1 : 2 * batches - 2 - (tile + 1));
      else if (next) fetch(z + step * a.pitch, 0);
    };
    Running st{edge, edge == -INFINITY ? 0.f : edge - edge + 1.f};  // (NaN stays NaN)
    if constexpr (kMode == kGradFromStats) {
      st = kept_stats(a, row);
    } else {
      for (int b = 0; b < batches; ++b) {
        take(b);
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
      if (lane == 0) part[n & 1][warp] = Running{m, st.s};
      meet();
      if (kMode == kLoss) continue;
      st = row_total(part[n & 1], a.c);
    }
    if constexpr (kMode != kLoss) {
      const float f = a.dloss[row] * a.temp, g = f * inverse(st.s);
      uint4* o = reinterpret_cast<uint4*>(dz + r.lead);
      const uint64_t neg = ptx::f32x2_pack(-st.m, -st.m), gg = ptx::f32x2_pack(g, g);
      for (int tile = kMode == kGradAndLoss ? batches - 1 : 0; tile < tiles; ++tile) {
        if (kMode == kGradFromStats || tile >= batches) take(tile);
        const int b = tile < batches ? tile : 2 * batches - 2 - tile;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int i = (b * NV + k) * kRow + tid;
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
      fix_entries(a, entries(n), dz, f, st, tid, kRow);
    }
  }
}

// ------------------------------------------------------------------- element by element

struct Teacher {
  int id[TG_MAX_TEACHER];    // -1: absent
  float p[TG_MAX_TEACHER];   // the logit first, then e^{(t - max) / T}, then the probability
  float z[TG_MAX_TEACHER];   // the student's logit there
};

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
    const float f = a.dloss[row] * a.temp, inv = inverse(st.y);
    for (int e = threadIdx.x; e < a.k; e += kThreads) {
      const int id = te.id[e];
      if (id < 0) continue;
      float p = 0.f;
      bool first = true;  // each token by its first entry
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

template <typename T, int kRow, Mode kMode>
cudaError_t rows_of(const DistillArgs<T>& a, int per_sm, cudaStream_t s) {
  const auto kernel = distill_row_kernel<T, kRow, 8, kMode>;
  const int smem = 8 * kRow * 16 + kSlots * 4 * a.k * 4;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             8 * kRow * 16 + kSlots * 4 * TG_MAX_TEACHER * 4);
  if (e != cudaSuccess) return e;
  kernel<<<grid_of(a.rows, per_sm), kRow + 32 * kTeachers<kMode, kRow>, smem, s>>>(a);
  return cudaGetLastError();
}

// Threads of a row: 512 where it stays in registers for its gradient (4,096 vectors), else 256 with
// twice the blocks; 128 or 32 for short ones (up to 1,024 or 256 vectors), whose time is the
// latency of a row's steps.
template <typename T, Mode kMode>
cudaError_t rows_t(const DistillArgs<T>& a, cudaStream_t s) {
  if (a.vocab <= 256 * Wide<T>::E) return rows_of<T, 32, kMode>(a, 16, s);
  if (a.vocab <= 1024 * Wide<T>::E) return rows_of<T, 128, kMode>(a, 6, s);
  return kMode != kGradAndLoss ? rows_of<T, 256, kMode>(a, 4, s) : rows_of<T, 512, kMode>(a, 2, s);
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

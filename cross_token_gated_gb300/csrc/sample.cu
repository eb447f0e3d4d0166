// Drawing tokens from logits with temperature, top-k, top-p and min-p and given uniform numbers
// (generation with the model of "TANGO: Token-Aggregated Nonlinear Gating Operators ...", sec. 2.3).
//
//   w_i = e^{(x_i - max) / T};  kept: the k largest, of these the shortest run with a share top_p of
//   the mass, of these w >= min_p;  token: first i with sum_{kept j <= i} w_j > u sum_{kept} w_j
//
// A token is a whole number, so the sums have to decide as those of the real numbers: weights are
// formed to a relative 2^-33 and summed as integers (units of 2^-44).  What is kept is a
// run of the order (logit descending, index ascending): all logits above a cut, and the first
// few that equal it.
//
// Bound by instructions and barriers, not by the 64 KB of a row: a pass for the range, one for a
// histogram and one with exact weights (about 76 instructions a logit, from the issue rate and the
// cycles of 61 fp32 rows).  One row of 32,768 bf16 logits
// with top-p takes 16.6 us on 8 blocks; 256 rows with settings of their own 36 us, with top-k 50 and top-p
// 26 us, greedily 12 us.  A border deep in the tail (top-p 0.9999) takes one row 50 us, 256 rows 103 us.
#include <float.h>
#include <math.h>

#include "tg_common.cuh"
#include "tg_ends.h"
#include "tg_exp2_table.cuh"
#include "tg_ptx.cuh"
#include "tg_serve.h"
#include "tg_vec.cuh"

namespace tg {
namespace {

// Threads of one of the C blocks that share a row.  A row by itself wants all the warps an SM takes at
// 64 registers (256 rows of 32,768: 36 us, with 512 threads 43 us); shares of rows are passed
// more quickly through the barriers of half as many (one row by 8 blocks: 16.6 us, 20.7 us).
template <int C> constexpr int kThreads = C == 1 ? 1024 : 512;
template <int C> constexpr int kWarps = kThreads<C> / 32;
constexpr int kUnit = 44;                      // a weight of 1 is 2^44
constexpr unsigned kFull = 0xffffffffu;

// ------------------------------------------------------------------- weights in fixed point

// 2^(i/256), i < 256: in units of 2^-46, and as a float in units of 2^-38.
struct Exp2Table {
  uint64_t t[256];
  float f[256];
};
// A thread's share of the table, asked for early and stored later.
struct Exp2Share {
  uint64_t t;
  __device__ __forceinline__ Exp2Share() : t(kExp2Table[threadIdx.x & 255]) {}
  __device__ __forceinline__ void store(Exp2Table& tab) const {
    if (threadIdx.x >= 256) return;
    tab.t[threadIdx.x] = t;
    tab.f[threadIdx.x] = (float)t * 0.00390625f;  // 2^-8
  }
};

// log2(e) / T as a sum of two floats; both are finite for T from FLT_MIN to FLT_MAX.
struct Scale {
  float hi, lo;
};
__device__ __forceinline__ Scale scale_of(float temp) {
  constexpr float lh = 1.44269502162933349609375f, ll = 1.925963033500011e-08f;  // log2(e)
  const float hi = lh / temp;
  return Scale{hi, (fmaf(-hi, temp, lh) + ll) / temp};
}

// e^{(x - max) / T} in units of 2^-44, 0 where it is less than 2^-40 (and for NaN); max is finite.
// y = (x - max) log2(e) / T is carried as a sum of two floats, 2^y = 2^k 2^(i/256) 2^r with |r| < 1/500.
// 2^r - 1 is below 2^-8.5, so that its roundings in fp32 leave a relative error of 2^-33; the sum
// with the table's 47 bits and the shift by k are integers.  Sums and products are rounded one by
// one (none may be fused).
__device__ __forceinline__ uint64_t weight(float x, float mx, Scale c, const Exp2Table& tab) {
  const float d = __fsub_rn(x, mx), back = __fsub_rn(d, x);
  const float dl = __fsub_rn(__fsub_rn(x, __fsub_rn(d, back)), __fadd_rn(mx, back));
  const float yh = __fmul_rn(d, c.hi);
  const float yl = __fadd_rn(__fmaf_rn(d, c.hi, -yh), __fmaf_rn(d, c.lo, __fmul_rn(dl, c.hi)));
  const float m = __fmaf_rn(yh, 256.f, 12582912.f);  // 1.5 2^23: the sum's low bits are the nearest integer
  const int n = __float_as_int(m) - 0x4b400000;
  const float r = __fadd_rn(__fmaf_rn(__fsub_rn(m, 12582912.f), -0.00390625f, yh), yl);
  // ln 2, ln^2 2 / 2, ln^3 2 / 6
  const float e = __fmul_rn(r, __fmaf_rn(r, __fmaf_rn(r, 0.055504109f, 0.24022651f), 0.69314718f));
  const int part = __float2int_rn(__fmul_rn(e, tab.f[n & 255]));
  const uint64_t w = tab.t[n & 255] + (int64_t)part * 256;
  // one less than the shift, 1 .. 41, or what shifts all out
  const int s = __fadd_rn(yh, yl) >= -40.f ? 46 - kUnit - 1 - (n >> 8) : 63;
  return ((w >> s) + 1) >> 1;
}

// Order of the logits as unsigned integers.
__device__ __forceinline__ unsigned key_of(float x) {
  const unsigned b = __float_as_uint(__fadd_rn(x, 0.f));  // (-0 as 0)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// --------------------------------------------------------------------------- reductions

constexpr int kMostBins = 4096;
template <int C> constexpr int kList = kThreads<C>;
template <int C> constexpr int kSpans = kThreads<C>;
constexpr int kShort = 256;  // a list that is gone through twice per entry

template <int C>
struct Shared {
  Exp2Table tab;
  uint64_t mass[kSpans<C>];     // kept mass of the row's spans
  unsigned bins[kMostBins];
  uint64_t order[kList<C>];     // the logits of the bins that hold a border: a number that falls along
                             // the row's order, (key, ~index)
  uint64_t w[kList<C>];
  int listed;
  uint64_t buf[kWarps<C>], buf2[kWarps<C>], buf3[kWarps<C>];
  unsigned ubuf[2][kWarps<C>];
  float fbuf[kWarps<C>];
  int first, last, found;
  uint64_t rest;
  uint64_t given[2][3];      // what the cluster's blocks tell each other, in turn
  uint64_t answer;           // the first block's, to all
};

// By 32-bit reductions of 22 bits at a time.
__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
  const unsigned lo = __reduce_add_sync(kFull, (unsigned)v & 0x3fffffu), mid = __reduce_add_sync(kFull, (unsigned)(v >> 22) & 0x3fffffu);
  return lo + ((uint64_t)mid << 22) + ((uint64_t)__reduce_add_sync(kFull, (unsigned)(v >> 44)) << 44);
}
// Over the block, for every thread; the barrier at the end frees the buffer again.
template <int C>
__device__ __forceinline__ uint64_t block_sum64(uint64_t v, Shared<C>& sh) {
  v = warp_sum64(v);
  if ((threadIdx.x & 31) == 0) sh.buf[threadIdx.x / 32] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  v = warp_sum64(lane < kWarps<C> ? sh.buf[lane] : 0);
  __syncthreads();
  return v;
}
// Three at once.
template <int C>
__device__ __forceinline__ void block_sum64(uint64_t& a, uint64_t& b, uint64_t& c, Shared<C>& sh) {
  a = warp_sum64(a);
  b = warp_sum64(b);
  c = warp_sum64(c);
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  if (lane == 0) sh.buf[warp] = a, sh.buf2[warp] = b, sh.buf3[warp] = c;
  __syncthreads();
  a = warp_sum64(lane < kWarps<C> ? sh.buf[lane] : 0);
  b = warp_sum64(lane < kWarps<C> ? sh.buf2[lane] : 0);
  c = warp_sum64(lane < kWarps<C> ? sh.buf3[lane] : 0);
  __syncthreads();
}
template <int C>
__device__ __forceinline__ unsigned block_max(unsigned v, Shared<C>& sh) {
  v = __reduce_max_sync(kFull, v);
  if ((threadIdx.x & 31) == 0) sh.ubuf[0][threadIdx.x / 32] = v;
  __syncthreads();
  v = __reduce_max_sync(kFull, sh.ubuf[0][threadIdx.x & (kWarps<C> - 1)]);
  __syncthreads();
  return v;
}
// Sum over the threads before this one, and over all.
template <int C, typename N>
__device__ __forceinline__ N block_before(N v, N* buf, N* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  auto scan = [lane](N x) {
    for (int o = 1; o < 32; o <<= 1) {
      const N up = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += up;
    }
    return x;
  };
  const N incl = scan(v);
  if (lane == 31) buf[warp] = incl;
  __syncthreads();
  const N warps = scan(buf[lane & (kWarps<C> - 1)]);  // (lanes past the warps are not looked at)
  const N before = __shfl_sync(kFull, warps, (warp + 31) & 31);
  *total = __shfl_sync(kFull, warps, kWarps<C> - 1);
  __syncthreads();
  return (warp ? before : N(0)) + incl - v;
}

// C blocks that share a row (a cluster; block number `rank`).  The results of these calls are the
// same in all threads of all blocks.
template <int C>
struct Group {
  Shared<C>& sh;
  unsigned rank;
  int turn = 0;
  __device__ __forceinline__ explicit Group(Shared<C>& s) : sh(s), rank(0) {
    if constexpr (C > 1) asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  }
  __device__ __forceinline__ void sync() const {
    if constexpr (C > 1)
      asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    else __syncthreads();
  }
  // before a block ends: no other block reads its memory any more
  __device__ __forceinline__ void leave() const {
    if constexpr (C > 1) sync();
  }
  // the same variable of block q
  template <typename N>
  __device__ __forceinline__ N* of(N* p, unsigned q) const {
    if constexpr (C == 1) return p;
    uint64_t a;
    asm("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"((uint64_t)p), "r"(q));
    return reinterpret_cast<N*>(a);
  }
  // lane q of each warp gets what thread 0 of block q gives (others zero)
  __device__ __forceinline__ void exchange(uint64_t& a, uint64_t& b, uint64_t& c) {
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) sh.given[turn][0] = a, sh.given[turn][1] = b, sh.given[turn][2] = c;
    sync();
    const uint64_t* p = of(sh.given[turn], lane < C ? lane : 0);
    a = lane < C ? p[0] : 0;
    b = lane < C ? p[1] : 0;
    c = lane < C ? p[2] : 0;
    turn ^= 1;
  }
  __device__ __forceinline__ uint64_t sum(uint64_t v) {
    v = block_sum64(v, sh);
    if constexpr (C > 1) {
      uint64_t none = 0, more = 0;
      exchange(v, none, more);
      v = warp_sum64(v);
    }
    return v;
  }
  __device__ __forceinline__ unsigned largest(unsigned v) {
    v = block_max(v, sh);
    if constexpr (C > 1) {
      uint64_t x = v, none = 0, more = 0;
      exchange(x, none, more);
      v = __reduce_max_sync(kFull, (unsigned)x);
    }
    return v;
  }
};

// --------------------------------------------------------------------------------- row

// What is kept of the row's order: larger keys, and of the equal ones those up to an index.
struct Cut {
  unsigned key, last;
  __device__ __forceinline__ bool keeps(unsigned k, unsigned i) const { return k > key || (k == key && i <= last); }
};

template <typename T> struct Wide;
template <> struct Wide<float> : Vec16<float> {
  // largest and lowest of all so far, NaN left out
  static __device__ __forceinline__ void range(const uint4& u, float& top, float& low) {
    float f[4];
    unpack(u, f);
    top = fmaxf(fmaxf(top, fmaxf(f[0], f[1])), fmaxf(f[2], f[3]));
    low = fminf(fminf(low, fminf(f[0], f[1])), fminf(f[2], f[3]));
  }
};
template <> struct Wide<__nv_bfloat16> : Vec16<__nv_bfloat16> {
  static __device__ __forceinline__ __nv_bfloat162 two(unsigned x) { return *reinterpret_cast<__nv_bfloat162*>(&x); }
  static __device__ __forceinline__ void range(const uint4& u, float& top, float& low) {
    const __nv_bfloat162 a = two(u.x), b = two(u.y), c = two(u.z), d = two(u.w);
    const __nv_bfloat162 m = __hmax2(__hmax2(a, b), __hmax2(c, d)), n = __hmin2(__hmin2(a, b), __hmin2(c, d));
    top = fmaxf(top, fmaxf(__low2float(m), __high2float(m)));
    low = fminf(low, fminf(__low2float(n), __high2float(n)));
  }
};

// A block's part of the row as 16-byte vectors, with the elements before the first and after the
// last one of the row by themselves; it is read again in every pass, from L1 or L2.  32 vectors
// that a warp reads at once are a span; `wide` doublings of that keep their number within kSpans<C>.
template <typename T, int C>
struct Row {
  static constexpr int E = Wide<T>::E;
  const T* x;
  int V, lead, all, per;   // of the row: elements before the vectors, vectors, vectors of a block
  int rank, v0, nvec;      // of this block: first vector, vectors
  int head, edge, wide;    // single elements before the vectors, single elements in all
  __device__ __forceinline__ Row(const T* row, int vocab, int block) : x(row), V(vocab), rank(block) {
    lead = row_lead(row, vocab);
    all = (vocab - lead) / E;
    per = C == 1 ? all : ((all + 31) / 32 + C - 1) / C * 32;
    v0 = min(rank * per, all);
    nvec = min(per, all - v0);
    head = rank == 0 ? lead : 0;
    edge = head + (rank == C - 1 ? vocab - lead - all * E : 0);
    wide = 0;
    while ((per >> 5 >> wide) >= kSpans<C>) ++wide;
  }
  __device__ __forceinline__ float at(int i) const { return io<T>::ld(x + i); }
  __device__ __forceinline__ int edge_index(int t) const { return t < head ? t : lead + all * E + t - head; }
  __device__ __forceinline__ int index(int v) const { return lead + (v0 + v) * E; }
  // the block and span of an element
  __device__ __forceinline__ int owner(int i) const {
    return C == 1 || i < lead ? 0 : (i - lead) / E >= all ? C - 1 : (i - lead) / E / per;
  }
  __device__ __forceinline__ int span_of(int i) const {
    if (i < lead) return 0;
    const int q = owner(i), first = min(q * per, all), n = min(per, all - first);
    return n > 0 ? min(n - 1, (i - lead) / E - first) >> 5 >> wide : 0;
  }
  // elements of a span of this block
  __device__ __forceinline__ int2 span(int s) const {
    const int step = (32 << wide) * E, n = nvec > 0 ? ((nvec - 1) >> 5 >> wide) + 1 : 1;
    return make_int2(s == 0 && rank == 0 ? 0 : index(0) + s * step,
                     s < n - 1 ? index(0) + (s + 1) * step : rank == C - 1 ? V : index(nvec));
  }
  // largest and lowest logit of the thread's, NaN left out
  __device__ __forceinline__ float2 range() const {
    float top = -INFINITY, low = INFINITY;
    if ((int)threadIdx.x < edge) {
      const float v = at(edge_index(threadIdx.x));
      top = fmaxf(top, v);
      low = fminf(low, v);
    }
    const uint4* v = reinterpret_cast<const uint4*>(x + lead) + v0;
#pragma unroll 4
    for (int i = threadIdx.x; i < nvec; i += kThreads<C>) Wide<T>::range(__ldg(v + i), top, low);
    return make_float2(top, low);
  }
  // f(value, index) for the thread's elements
  template <int U, typename F>
  __device__ __forceinline__ void each(F f) const {
    const int tid = threadIdx.x;
    if (tid < edge) {  // (fewer than 16)
      const int i = edge_index(tid);
      f(at(i), i);
    }
    const uint4* v = reinterpret_cast<const uint4*>(x + lead) + v0;
#pragma unroll 1
    for (int b = tid; b < nvec; b += U * kThreads<C>) {
      uint4 u[U];
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (b + k * kThreads<C> < nvec) u[k] = __ldg(v + b + k * kThreads<C>);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (b + k * kThreads<C> >= nvec) break;
        float e[E];
        Wide<T>::unpack(u[k], e);
#pragma unroll
        for (int j = 0; j < E; ++j) f(e[j], index(b + k * kThreads<C>) + j);
      }
    }
  }
  // Adds f(value, index) up in mass[span], which holds zeros; returns the thread's own sum.
  template <typename F>
  __device__ __forceinline__ uint64_t sum_spans(uint64_t* mass, F f) const {
    using u64 = unsigned long long;
    const int tid = threadIdx.x;
    uint64_t all = 0;
    if (tid < edge) {
      const int i = edge_index(tid);
      const uint64_t w = f(at(i), i);
      all += w;
      if (w) atomicAdd((u64*)mass + span_of(i), (u64)w);
    }
    const uint4* v = reinterpret_cast<const uint4*>(x + lead) + v0;
#pragma unroll 1
    for (int b = tid & ~31; b < nvec; b += kThreads<C>) {
      const int i = b + (tid & 31);
      uint64_t w = 0;
      if (i < nvec) {
        float e[E];
        Wide<T>::unpack(__ldg(v + i), e);
#pragma unroll
        for (int j = 0; j < E; ++j) w += f(e[j], index(i) + j);
      }
      if (!__any_sync(kFull, w != 0)) continue;
      all += w;
      w = warp_sum64(w);
      if ((tid & 31) == 0) atomicAdd((u64*)mass + (b >> 5 >> wide), (u64)w);
    }
    return all;
  }
};

struct Settings {
  float temp, top_p, min_p, u;
  int top_k;
};

__device__ __forceinline__ Settings settings_of(const SampleCall& c, int row) {
  const tg_sample_params& p = c.p;
  return Settings{p.temperatures ? p.temperatures[row] : p.temperature, p.top_ps ? p.top_ps[row] : p.top_p,
                  p.min_ps ? p.min_ps[row] : p.min_p, c.uniform[row], p.top_ks ? p.top_ks[row] : p.top_k};
}
__device__ __forceinline__ Settings checked(Settings s, const SampleCall& c) {
  bool bad = false;
  if (!(s.temp >= 0.f)) { bad = true; s.temp = s.temp < 0.f ? 0.f : 1.f; }
  if (s.temp > FLT_MAX) { bad = true; s.temp = FLT_MAX; }
  // log2(e) / T overflows from a T of 4e-39 down; the weights differ for logits less than 3.3e-37 apart only
  if (s.temp > 0.f) s.temp = fmaxf(s.temp, FLT_MIN);
  if (s.top_p != s.top_p) { bad = true; s.top_p = 1.f; }
  if (!(s.min_p <= 1.f)) { bad = true; s.min_p = s.min_p > 1.f ? 1.f : 0.f; }
  if (!(s.u >= 0.f && s.u < 1.f)) { bad = true; s.u = s.u >= 1.f ? 0.99999994f : 0.f; }
  if (bad && threadIdx.x == 0) record_error(c.err, kErrValue | kKernSample);
  return s;
}

// u in [0, 1) as a fraction of 2^64.
__device__ __forceinline__ uint64_t fraction(float u) { return (uint64_t)(u * 18446744073709551616.f); }

// Bins of a row: equal steps of the logits from the largest one down to 2^-40 of its weight, or to
// the lowest logit.  2 of each thread, or 8 for the largest vocabularies, whose bins would hold more
// than the list.
template <int C>
struct Bins {
  int each, count;
  float mx, per_unit, log2_step;
  __device__ __forceinline__ Bins(float mx_, float low, float temp, Scale sc, int vocab) : mx(mx_) {
    each = vocab > 1 << 17 && C > 1 ? kMostBins / kThreads<C> : 2;
    count = each * kThreads<C>;
    // 27.8 > 40 ln 2; logits that differ by less than 1e-30 may share a bin; both may overflow (masked
    // logits at a T above 1.2e37)
    const float reach = fmaxf(fminf(fminf(27.8f * temp, __fsub_rn(mx, low)), FLT_MAX), 1e-30f);
    per_unit = __fdiv_rn((float)(count - 1), reach);
    log2_step = sc.hi / per_unit;
  }
  // distance from the largest in bins; outside where it is not below count - 0.5 (NaN too)
  __device__ __forceinline__ float place(float x) const { return __fmul_rn(__fsub_rn(mx, x), per_unit); }
  __device__ __forceinline__ bool inside(float y) const { return y < (float)count - 0.5f; }
  // the nearest bin as 1.5 2^23 + bin: its low bits are the number
  static __device__ __forceinline__ float bin(float y) { return __fadd_rn(y, 12582912.f); }
  static __device__ __forceinline__ int number(float b) { return __float_as_int(b) - 0x4b400000; }
  // the keys that bins first .. last and their neighbours may hold, but for roundings
  __device__ __forceinline__ unsigned lowest_key(int last) const { return key_of(mx - (float)(last + 1) / per_unit); }
  __device__ __forceinline__ unsigned highest_key(int first) const { return key_of(mx - (float)(first - 1) / per_unit); }
};

// The index of the m-th logit (from 1) that equals a key, or of the last one where there are
// fewer.  Overwrites sh.mass.
template <typename T, int C>
__device__ __noinline__ unsigned nth_equal(const Row<T, C>& row, unsigned key, uint64_t m, Group<C>& g) {
  Shared<C>& sh = g.sh;
  sh.mass[threadIdx.x] = 0;
  if (threadIdx.x == 0) sh.found = 0;
  __syncthreads();
  row.sum_spans(sh.mass, [&](float x, int) { return (uint64_t)(key_of(x) == key); });
  __syncthreads();
  uint64_t total;
  const uint64_t mine = sh.mass[threadIdx.x];
  uint64_t before = block_before<C>(mine, sh.buf, &total);
  if constexpr (C > 1) {
    uint64_t each = total, none = 0, more = 0;
    g.exchange(each, none, more);
    before += warp_sum64((threadIdx.x & 31) < g.rank ? each : 0);
    total = warp_sum64(each);
  }
  if (m > total) m = total;
  if (before < m && m <= before + mine) {  // walk through the span
    const int2 at = row.span(threadIdx.x);
    uint64_t n = before;
    for (int i = at.x; i < at.y && n < m; ++i) {
      n += key_of(row.at(i)) == key;
      sh.found = i;
    }
  }
  __syncthreads();
  return g.largest(sh.found);
}

// Exact borders by bisection between two keys, for rows whose listed bins hold too many logits (few
// distinct ones, as a rule).  bf16 logits need the keys' upper half only.  The border is first
// looked for in [lo, hi], and in all of [low, top] if it is not there.
template <typename T> constexpr int kKeyShift = sizeof(T) == 2 ? 16 : 0;
template <typename T>
__device__ __forceinline__ unsigned short_key(float x) { return key_of(x) >> kKeyShift<T>; }
template <typename T>
__device__ __forceinline__ unsigned whole_key(unsigned k) {
  return kKeyShift<T> == 0 ? k : k << 16 | (k & 0x8000u ? 0u : 0xffffu);
}
struct Between {
  unsigned lo, hi, low, top;
  template <typename T>
  __device__ __forceinline__ Between shortened() const {
    const Between b{max(lo, low) >> kKeyShift<T>, min(hi, top) >> kKeyShift<T>, low >> kKeyShift<T>, top >> kKeyShift<T>};
    return b.lo <= b.hi ? b : Between{b.low, b.top, b.low, b.top};
  }
};

template <typename T, int C>
__device__ __noinline__ Cut bisect_count(const Row<T, C>& row, Between keys, uint64_t k, Group<C>& g) {
  auto count = [&](unsigned key) {  // logits of at least this key
    uint64_t n = 0;
    row.template each<1>([&](float x, int) { n += x == x && short_key<T>(x) >= key; });
    return g.sum(n);
  };
  Between b = keys.shortened<T>();
  if (b.lo > b.low && count(b.lo) < k) b.lo = b.low;
  if (b.hi < b.top && count(b.hi + 1) >= k) b.hi = b.top;
  while (b.lo < b.hi) {  // the largest key that at least k logits reach
    const unsigned mid = b.lo + (b.hi - b.lo + 1) / 2;
    if (count(mid) >= k) b.lo = mid;
    else b.hi = mid - 1;
  }
  const uint64_t above = b.lo < b.top ? count(b.lo + 1) : 0;
  const unsigned key = whole_key<T>(b.lo);
  return Cut{key, nth_equal(row, key, k - above, g)};
}
template <typename T, int C>
__device__ __noinline__ Cut bisect_mass(const Row<T, C>& row, Between keys, Cut within, uint64_t need, float mx, Scale sc,
                                        Group<C>& g) {
  auto above = [&](unsigned key) {  // mass of the larger keys
    uint64_t n = 0;
    row.template each<1>([&](float x, int i) {
      if (short_key<T>(x) > key && within.keeps(key_of(x), i)) n += weight(x, mx, sc, g.sh.tab);
    });
    return g.sum(n);
  };
  Between b = keys.shortened<T>();
  if (b.hi < b.top && above(b.hi) >= need) b.hi = b.top;
  if (b.lo > b.low && above(b.lo - 1) < need) b.lo = b.low;
  while (b.lo < b.hi) {  // the smallest key above which there is less than what is needed
    const unsigned mid = b.lo + (b.hi - b.lo) / 2;
    if (above(mid) < need) b.hi = mid;
    else b.lo = mid + 1;
  }
  const unsigned key = whole_key<T>(b.lo);
  const uint64_t w = weight(value_of(key), mx, sc, g.sh.tab);
  if (w == 0) return Cut{key, kFull};  // all of the mass is needed
  const Cut cut{key, nth_equal(row, key, (need - above(b.lo) + w - 1) / w, g)};
  return key == within.key && within.last < cut.last ? within : cut;
}

// The list's kept entries join their spans, the last of them is the cut; `sure` is the mass before
// the list.  No cut (all ones) where the list is too long or does not hold the border.  All blocks
// have to be through with the list.
template <typename T, int C>
__device__ __forceinline__ uint64_t join_list(const Row<T, C>& row, uint64_t sure, uint64_t need, uint64_t least, Group<C>& g) {
  Shared<C>& sh = g.sh;
  const int n = sh.listed;
  if (g.rank == 0 && n <= kList<C> && (int)threadIdx.x < n && sure < need) {
    const uint64_t mine = sh.order[threadIdx.x], w = sh.w[threadIdx.x];
    uint64_t before = sure;
    for (int j = 0; j < n; ++j) before += sh.order[j] > mine ? sh.w[j] : 0;
    if (before < need) {
      const int i = kFull - (unsigned)mine;
      if (w >= least) atomicAdd((unsigned long long*)g.of(sh.mass, row.owner(i)) + row.span_of(i), (unsigned long long)w);
      if (before + w >= need) sh.answer = mine;
    }
  }
  g.sync();
  return g.of(&sh, 0)->answer;
}

// The border of the mass where bins first .. last hold too many logits for the list, which is so
// from a top_p of some 0.9995 on: their exact masses in kSteps finer steps of equal width, and a list
// of the one step that holds the border.  Two passes in place of a bisection's many (256 rows of 32,768
// with top_p 0.9999: 103 us, 281 us bisected).
template <typename T, int C>
__device__ __noinline__ uint64_t finer_border(const Row<T, C>& row, const Bins<C>& bins, int first, int last, Cut within,
                                              uint64_t sure, uint64_t need, uint64_t least, float mx, Scale sc, Group<C>& g) {
  using u64 = unsigned long long;
  constexpr int kSteps = kMostBins / 2, kEach = kSteps / kThreads<C>;
  Shared<C>& sh = g.sh;
  Shared<C>* const home = g.of(&sh, 0);
  const int tid = threadIdx.x;
  u64* const steps = reinterpret_cast<u64*>(sh.bins);
  g.sync();  // all have read that there is no answer yet
  for (int j = 0; j < kEach; ++j) steps[tid + j * kThreads<C>] = 0;
  sh.mass[tid] = 0;
  if (tid == 0) sh.listed = 0, sh.answer = ~0ull, sh.first = -1;
  g.sync();
  const float first_bin = 12582912.f + first, last_bin = 12582912.f + last;
  const float start = (float)first - 0.5f, per_bin = __fdiv_rn((float)kSteps, (float)(last - first + 1));
  // falls with x, as each of its roundings keeps the order
  auto step = [&](float y) { return max(0, min(kSteps - 1, (int)__fmul_rn(__fsub_rn(y, start), per_bin))); };
  row.template each<1>([&](float x, int i) {
    const float y = bins.place(x), b = bins.bin(y);
    if (!(b >= first_bin && b <= last_bin) || !within.keeps(key_of(x), i)) return;
    const uint64_t w = weight(x, mx, sc, sh.tab);
    if (w) atomicAdd(steps + step(y), (u64)w);
  });
  g.sync();
  uint64_t m[kEach], own = 0, total;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    m[j] = 0;
#pragma unroll
    for (int q = 0; q < C; ++q) m[j] += g.of(steps, q)[tid * kEach + j];
    own += m[j];
  }
  uint64_t before = sure + block_before<C>(own, sh.buf, &total);
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    if (before < need && need <= before + m[j]) sh.first = tid * kEach + j, sh.rest = before;
    before += m[j];
  }
  __syncthreads();
  const int at = sh.first;
  if (at >= 0) {  // (the same in all blocks)
    sure = sh.rest;
    row.sum_spans(sh.mass, [&](float x, int i) -> uint64_t {
      const float y = bins.place(x), b = bins.bin(y);
      if (!(b <= last_bin) || !within.keeps(key_of(x), i)) return 0;
      const int n = b < first_bin ? -1 : step(y);
      if (n > at) return 0;
      const uint64_t w = weight(x, mx, sc, sh.tab);
      if (n < at) return w >= least ? w : 0;
      if (w == 0) return 0;
      const int e = atomicAdd(&home->listed, 1);
      if (e < kList<C>) {
        home->order[e] = (uint64_t)key_of(x) << 32 | (kFull - (unsigned)i);
        home->w[e] = w;
      }
      return 0;
    });
  }
  g.sync();
  return at >= 0 ? join_list(row, sure, need, least, g) : ~0ull;
}

// The token of a row from its list, which holds all of the top_k logits.
template <int C>
__device__ __forceinline__ void draw_listed(const SampleCall& c, const Settings& s, long long r, uint64_t least, Shared<C>& sh) {
  const int tid = threadIdx.x, n = sh.listed;
  uint64_t mine = 0, w = 0, before = 0;
  unsigned rank = 0;
  if (tid < n) {
    mine = sh.order[tid];
    w = sh.w[tid];
    for (int j = 0; j < n; ++j)
      if (sh.order[j] > mine) {
        ++rank;
        before += sh.w[j];
      }
  }
  bool kept = tid < n && rank < (unsigned)s.top_k && w > 0;
  if (s.top_p < 1.f) {
    const uint64_t mass = block_sum64(kept ? w : 0, sh), p = fraction(s.top_p > 0.f ? s.top_p : 0.f);
    const uint64_t need = __umul64hi(p, mass) + (p * mass != 0);
    kept = kept && (before < need || before == 0);
  }
  w = kept && w >= least ? w : 0;
  if (tid < n) sh.mass[tid] = w;
  const uint64_t total = block_sum64(w, sh), target = __umul64hi(fraction(s.u), total);
  if (w == 0) return;
  const unsigned index = kFull - (unsigned)mine;
  uint64_t sum = 0;
  for (int j = 0; j < n; ++j)
    if (kFull - (unsigned)sh.order[j] < index) sum += sh.mass[j];
  if (sum <= target && target < sum + w) {
    c.token[r] = (int)index;
    if (c.logprob) c.logprob[r] = w == total ? 0.f : logf((float)w / (float)total);
  }
}

// C blocks per row.  A border (of the k-th logit, or of the share of the mass) is found with a
// histogram of counts, or of masses good to about 1e-5; only the logits of the bins that may hold it
// are listed and compared one by one, in exact sums.  Should there be too many of them, a border of
// the mass is looked for in finer steps; what is too many then (many equal logits), and a border of
// the counts, is bisected.  The histogram of masses is a hint only: more than 16,383 logits of a block
// in one bin overflow it.  Where its bins do not hold the border then, the exact sums show it, and the
// border is bisected over the whole row.
template <typename T, int C>
__global__ void __launch_bounds__(kThreads<C>, 1024 / kThreads<C>) sample_kernel(const SampleCall c) {
  using u64 = unsigned long long;
  __shared__ Shared<C> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const long long r = blockIdx.x / C;
  Group<C> g(sh);
  Shared<C>* const home = g.of(&sh, 0);  // the first block's, which keeps the list
  const Row<T, C> row(static_cast<const T*>(c.logits) + r * c.p.pitch, c.p.vocab, g.rank);
  const Exp2Share share_of_table;
  const Settings given = settings_of(c, (int)r);
  const float2 own = row.range();
  const Settings s = checked(given, c);
  share_of_table.store(sh.tab);
  sh.mass[tid] = 0;
  unsigned top = __reduce_max_sync(kFull, key_of(own.x)), low = __reduce_min_sync(kFull, key_of(own.y));
  if (lane == 0) sh.ubuf[0][warp] = top, sh.ubuf[1][warp] = low;
  __syncthreads();
  top = __reduce_max_sync(kFull, sh.ubuf[0][lane & (kWarps<C> - 1)]);
  low = __reduce_min_sync(kFull, sh.ubuf[1][lane & (kWarps<C> - 1)]);
  __syncthreads();
  if constexpr (C > 1) {
    uint64_t each = top, each_low = low, none = 0;
    g.exchange(each, each_low, none);
    top = __reduce_max_sync(kFull, lane < C ? (unsigned)each : 0);
    low = __reduce_min_sync(kFull, lane < C ? (unsigned)each_low : kFull);
  }
  const float mx = value_of(top);
  if (mx == -INFINITY || s.temp == 0.f) {
    unsigned first = 0;
    row.template each<2>([&](float x, int i) {
      if (x == mx) first = max(first, kFull - (unsigned)i);
    });
    first = kFull - g.largest(first);
    if (tid == 0 && g.rank == 0) {
      c.token[r] = mx == -INFINITY ? -1 : (int)first;
      if (c.logprob) c.logprob[r] = mx == -INFINITY ? mx : 0.f;
    }
    g.leave();
    return;
  }
  if (mx == INFINITY) {  // all weights are 1, of these logits alone
    uint64_t n = 0;
    row.template each<1>([&](float x, int) { n += x == mx; });
    n = g.sum(n);
    if (s.top_k > 0 && (uint64_t)s.top_k < n) n = s.top_k;
    if (s.top_p < 1.f) {
      const uint64_t f = fraction(s.top_p > 0.f ? s.top_p : 0.f);
      n = __umul64hi(f, n) + (f * n != 0);
      if (n == 0) n = 1;
    }
    const unsigned at = nth_equal(row, top, __umul64hi(fraction(s.u), n) + 1, g);
    if (tid == 0 && g.rank == 0) {
      c.token[r] = (int)at;
      if (c.logprob) c.logprob[r] = -logf((float)n);
    }
    g.leave();
    return;
  }
  const Scale sc = scale_of(s.temp);
  const Bins<C> bins(mx, value_of(low), s.temp, sc, c.p.vocab);
  const uint64_t least = s.min_p > 0.f ? (uint64_t)ceilf(s.min_p * 17592186044416.f) : 0;  // 2^44
  const bool some_least = least > 0;
  auto clear_bins = [&] {
    for (int i = tid; i < bins.count; i += kThreads<C>) sh.bins[i] = 0;
    if (tid == 0) sh.listed = 0, sh.answer = ~0ull;
    __syncthreads();
  };
  auto list = [&](unsigned key, int i, uint64_t w) {
    const int n = atomicAdd(&home->listed, 1);
    if (n < kList<C>) {
      home->order[n] = (uint64_t)key << 32 | (kFull - (unsigned)i);
      home->w[n] = w;
    }
  };
  // the row's order, by key, falling, then by index, as one number that falls
  auto cut_at = [&](uint64_t order) { return Cut{(unsigned)(order >> 32), kFull - (unsigned)order}; };

  Cut cut{0, kFull};
  bool some_cut = false;
  if (s.top_k > 0 && s.top_k < row.V) {
    const unsigned k = s.top_k;
    clear_bins();
    row.template each<2>([&](float x, int) {
      const float y = bins.place(x);
      if (bins.inside(y)) atomicAdd(sh.bins + bins.number(bins.bin(y)), 1u);
    });
    g.sync();
    // the thread's bins of all blocks, those before them, and the one that holds the k-th
    unsigned own = 0, total;
    for (int j = 0; j < bins.each; j += 2)
#pragma unroll
      for (int q = 0; q < C; ++q) {
        const uint2 n = *reinterpret_cast<const uint2*>(g.of(sh.bins, q) + tid * bins.each + j);
        own += n.x + n.y;
      }
    unsigned before = block_before<C>(own, sh.ubuf[0], &total);
    if (total > k) {  // (else the k-th has less than 2^-40)
      if (before < k && k <= before + own) {
        for (int j = 0; j < bins.each; ++j) {
          unsigned n = 0;
#pragma unroll
          for (int q = 0; q < C; ++q) n += g.of(sh.bins, q)[tid * bins.each + j];
          if (before < k && k <= before + n) sh.first = tid * bins.each + j, sh.last = before, sh.found = n;
          before += n;
        }
      }
      __syncthreads();
      const int bin = sh.first;
      some_cut = true;
      const unsigned above = sh.last, in_bin = sh.found;
      const float wanted = 12582912.f + bin;
      if (above + in_bin <= kShort) {  // all that may be kept fits a short list
        row.template each<2>([&](float x, int i) {
          if (bins.bin(bins.place(x)) <= wanted) list(key_of(x), i, weight(x, mx, sc, sh.tab));
        });
        g.sync();
        if (g.rank == 0) draw_listed(c, s, r, least, sh);
        return;
      }
      if (in_bin <= kList<C>) {
        row.template each<2>([&](float x, int i) {
          if (bins.bin(bins.place(x)) == wanted) list(key_of(x), i, 0);
        });
        g.sync();
        if (g.rank == 0 && tid < sh.listed) {
          const int n = sh.listed;
          const uint64_t mine = sh.order[tid];
          unsigned rank = above + 1;
          for (int j = 0; j < n; ++j) rank += sh.order[j] > mine;
          if (rank == k) sh.answer = mine;
        }
        g.sync();
        cut = cut_at(home->answer);
      } else {
        cut = bisect_count(row, Between{bins.lowest_key(bin), bins.highest_key(bin), low, top}, k, g);
        sh.mass[tid] = 0;
      }
    }
    g.sync();  // all are through with the bins and the list
  }

  if (s.top_p < 1.f) {
    clear_bins();
    // a bin's masses in units of 2^-18 of the weight at its middle, modulo 2^32
    row.template each<2>([&](float x, int i) {
      const float y = bins.place(x);
      if (!bins.inside(y) || (some_cut && !cut.keeps(key_of(x), i))) return;
      const float b = bins.bin(y), q = ptx::ex2_approx(fmaf(__fsub_rn(b, 12582912.f) - y, bins.log2_step, 18.f));
      atomicAdd(sh.bins + bins.number(b), (unsigned)(__float_as_int(q + 8388608.f) - 0x4b000000));
    });
    g.sync();
    // the first bins that reach the share less and more the error
    float m[kMostBins / kThreads<8>], own = 0.f, all;
#pragma unroll
    for (int j = 0; j < kMostBins / kThreads<8>; j += 2) {
      m[j] = m[j + 1] = 0.f;
      if (j >= bins.each) continue;
      const int b = tid * bins.each + j;
#pragma unroll
      for (int q = 0; q < C; ++q) {
        const uint2 n = *reinterpret_cast<const uint2*>(g.of(sh.bins, q) + b);
        m[j] += (float)n.x;
        m[j + 1] += (float)n.y;
      }
      own += m[j] *= ptx::ex2_approx((float)-b * bins.log2_step);
      own += m[j + 1] *= ptx::ex2_approx((float)(-b - 1) * bins.log2_step);
    }
    float reached = block_before<C>(own, sh.fbuf, &all);
    const float share = s.top_p > 0.f ? s.top_p : 0.f, from = share * all * (1.f - 3e-5f), to = share * all * (1.f + 3e-5f);
    unsigned f = bins.count - 1, t = f;
#pragma unroll
    for (int j = 0; j < kMostBins / kThreads<8>; ++j) {
      if (j >= bins.each) continue;
      reached += m[j];
      const unsigned b = tid * bins.each + j;
      if (reached >= from) f = min(f, b);
      if (reached >= to) t = min(t, b);
    }
    f = __reduce_min_sync(kFull, f);
    t = __reduce_min_sync(kFull, t);
    if (lane == 0) sh.ubuf[0][warp] = f, sh.ubuf[1][warp] = t;
    __syncthreads();
    const int first = __reduce_min_sync(kFull, sh.ubuf[0][lane & (kWarps<C> - 1)]);
    const int last = __reduce_min_sync(kFull, sh.ubuf[1][lane & (kWarps<C> - 1)]);
    // exact sums of everything and of the bins before; the bins between are listed
    uint64_t rest = 0, small = 0;  // mass from the first listed bin on, and of what min_p drops before it
    const float first_bin = 12582912.f + first, last_bin = 12582912.f + last;
    uint64_t sure = row.sum_spans(sh.mass, [&](float x, int i) -> uint64_t {
      const float b = bins.bin(bins.place(x));
      if (some_cut && !cut.keeps(key_of(x), i)) return 0;
      const uint64_t w = weight(x, mx, sc, sh.tab);
      if (b < first_bin) {
        if (!some_least || w >= least) return w;
        small += w;
        return 0;
      }
      rest += w;
      if (b <= last_bin && w) list(key_of(x), i, w);
      return 0;
    });
    sure += small;
    uint64_t unused = 0;
    __syncthreads();
    block_sum64(rest, sure, unused, sh);
    if constexpr (C > 1) {
      g.exchange(rest, sure, unused);
      rest = warp_sum64(rest);
      sure = warp_sum64(sure);
    }
    const uint64_t mass = sure + rest;
    const uint64_t p = fraction(share);
    uint64_t need = __umul64hi(p, mass) + (p * mass != 0);
    if (need == 0) need = 1;
    uint64_t order = join_list(row, sure, need, least, g);
    if (order == ~0ull) order = finer_border(row, bins, first, last, cut, sure, need, least, mx, sc, g);
    if (order != ~0ull) {
      cut = cut_at(order);
    } else {
      const Between keys{bins.lowest_key(last), bins.highest_key(first), max(low, cut.key), top};
      cut = bisect_mass(row, keys, cut, need, mx, sc, g);
      sh.mass[tid] = 0;
      __syncthreads();
      row.sum_spans(sh.mass, [&](float x, int i) {
        const uint64_t w = cut.keeps(key_of(x), i) ? weight(x, mx, sc, sh.tab) : 0;
        return some_least && w < least ? 0 : w;
      });
    }
  } else {
    row.sum_spans(sh.mass, [&](float x, int i) {
      const uint64_t w = !some_cut || cut.keeps(key_of(x), i) ? weight(x, mx, sc, sh.tab) : 0;
      return some_least && w < least ? 0 : w;
    });
  }
  __syncthreads();

  // the span that holds the token, then the token
  uint64_t total;
  const uint64_t mine = sh.mass[tid];
  uint64_t before = block_before<C>(mine, sh.buf, &total);
  if (tid == 0) sh.first = -1;
  if constexpr (C > 1) {
    uint64_t each = total, none = 0, more = 0;
    g.exchange(each, none, more);
    before += warp_sum64(lane < (int)g.rank ? each : 0);
    total = warp_sum64(each);
  }
  __syncthreads();
  const uint64_t target = __umul64hi(fraction(s.u), total);  // the token is the first to pass it
  if (before <= target && target < before + mine) {
    sh.first = tid;
    sh.rest = target - before;
  }
  __syncthreads();
  g.leave();
  if (warp != 0 || sh.first < 0) return;
  const uint64_t rest = sh.rest;
  const int2 span = row.span(sh.first);
  const int per = (span.y - span.x + 31) / 32, from = span.x + lane * per, to = min(span.y, from + per);
  auto kept_weight = [&](int i) -> uint64_t {
    if (i >= to) return 0;
    const float x = row.at(i);
    const uint64_t w = cut.keeps(key_of(x), i) ? weight(x, mx, sc, sh.tab) : 0;
    return w < least ? 0 : w;
  };
  // (a span of 32 vectors and edges: at most 9 of a lane)
  constexpr int kHeld = Wide<T>::E + 1;
  uint64_t held[kHeld], own_mass = 0;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) own_mass += held[k] = kept_weight(from + k);
  for (int i = from + kHeld; i < to; ++i) own_mass += kept_weight(i);
  uint64_t incl = own_mass;
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t up = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += up;
  }
  const unsigned hit = __ballot_sync(kFull, incl > rest);
  if (lane != __ffs(hit) - 1) return;
  uint64_t sum = incl - own_mass, drawn = 0;
  int token = -1;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    sum += held[k];
    if (token < 0 && sum > rest) token = from + k, drawn = held[k];
  }
  for (int i = from + kHeld; token < 0 && i < to; ++i) {
    const uint64_t w = kept_weight(i);
    sum += w;
    if (sum > rest) token = i, drawn = w;
  }
  c.token[r] = token;
  if (c.logprob) c.logprob[r] = drawn == total ? 0.f : logf((float)drawn / (float)total);
}

template <typename T, int C>
cudaError_t sample_in(const SampleCall& c, cudaStream_t s) {
  if (c.p.rows > (int)((1u << 31) - 1) / C) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)c.p.rows * C);
  cfg.blockDim = dim3(kThreads<C>);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T, C>, c);
}

// Blocks of a row: as many as the SMs hold two of at once, while each still has a vector a thread.
template <typename T>
cudaError_t sample_t(const SampleCall& c, cudaStream_t s) {
  const int sms = serve_sm_count(), vectors = c.p.vocab / Wide<T>::E;
  int blocks = 1;
  while (blocks < 8 && c.p.rows <= sms / blocks && vectors >= 2 * blocks * kThreads<8>) blocks *= 2;
  return blocks == 8 ? sample_in<T, 8>(c, s) : blocks == 4 ? sample_in<T, 4>(c, s)
       : blocks == 2 ? sample_in<T, 2>(c, s) : sample_in<T, 1>(c, s);
}

}  // namespace

cudaError_t launch_sample(const SampleCall& c, cudaStream_t s) {
  return c.p.dtype == TG_F32 ? sample_t<float>(c, s) : sample_t<__nv_bfloat16>(c, s);
}

}  // namespace tg

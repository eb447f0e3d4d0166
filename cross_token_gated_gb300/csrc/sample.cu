// Drawing tokens from logits with temperature, top-k, top-p and min-p and given uniform numbers
// (generation with the model of "TANGO: Token-Aggregated Nonlinear Gating Operators ...", sec. 2.3).
//
//   w_i = e^{(x_i - max) / T};  kept: the k largest, of these the shortest run with a share top_p of
//   the mass, of these w >= min_p;  token: first i with sum_{kept j <= i} w_j > u sum_{kept} w_j
//
// A token is a whole number, so the sums have to decide as those of the real numbers: weights are
// formed to about 2^-42 of the largest and summed as integers (units of 2^-44).  What is kept is a
// run of the order (logit descending, index ascending): all logits above a cut, and the first
// few that equal it.
#include <math.h>

#include "tg_common.cuh"
#include "tg_ends.h"
#include "tg_exp2_table.cuh"
#include "tg_serve.h"

namespace tg {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kUnit = 44;                      // a weight of 1 is 2^44
constexpr unsigned kFull = 0xffffffffu;

// ------------------------------------------------------------------- weights in fixed point

struct Exp2Entry {
  uint64_t t;    // 2^(i/256) 2^46
  float hi, lo;  // the same as a sum of two floats
};
__device__ __forceinline__ void load_exp2(Exp2Entry* tab) {
  for (int i = threadIdx.x; i < 256; i += kThreads) {
    const uint64_t t = kExp2Table[i];
    // 47 bits: the upper 24 and the lower 23 are exact floats
    const float hi = (float)(t >> 23) * 1.1920928955078125e-7f;                            // 2^-23
    tab[i] = Exp2Entry{t, hi, (float)(t & 0x7fffff) * 1.4210854715202004e-14f};            // 2^-46
  }
}

// log2(e) / T as a sum of two floats.
struct Scale {
  float hi, lo;
};
__device__ __forceinline__ Scale scale_of(float temp) {
  constexpr float lh = 1.44269502162933349609375f, ll = 1.925963033500011e-08f;  // log2(e)
  const float hi = lh / temp;
  return Scale{hi, (fmaf(-hi, temp, lh) + ll) / temp};
}

// e^{(x - max) / T} in units of 2^-44, 0 where it is less than 2^-40.  y = (x - max) log2(e) / T
// is carried as a sum of two floats; 2^y = 2^k 2^(i/256) (1 + t + t^2/2 + ...), |t| < 2^-9.5, whose
// terms up to t^4 reach 2^-44.  Sums and products are rounded one by one (none may be fused).
__device__ __forceinline__ uint64_t weight(float x, float mx, Scale c, const Exp2Entry* tab) {
  if (x == mx) return 1ull << kUnit;
  const float d = __fsub_rn(x, mx), back = __fsub_rn(d, x);
  const float dl = __fsub_rn(__fsub_rn(x, __fsub_rn(d, back)), __fadd_rn(mx, back));
  float yh = __fmul_rn(d, c.hi);
  if (!(yh > -41.f)) return 0;  // -inf and NaN too
  float yl = __fadd_rn(__fmaf_rn(d, c.hi, -yh), __fmaf_rn(d, c.lo, __fmul_rn(dl, c.hi)));
  const float y = __fadd_rn(yh, yl);
  yl = __fsub_rn(yl, __fsub_rn(y, yh));
  yh = y;
  if (yh < -40.f || (yh == -40.f && yl < 0.f)) return 0;
  const float m = __fmaf_rn(yh, 256.f, 12582912.f);  // 1.5 2^23: the sum's low bits are the nearest integer
  const int n = __float_as_int(m) - 0x4b400000;
  const float r0 = __fmaf_rn(__fsub_rn(m, 12582912.f), -0.00390625f, yh), r = __fadd_rn(r0, yl);
  yl = __fsub_rn(yl, __fsub_rn(r, r0));
  constexpr float l2h = 0.693147182464599609375f, l2l = -1.9046542121259336e-09f;  // ln 2
  const float th = __fmul_rn(r, l2h);
  const float tl = __fadd_rn(__fmaf_rn(r, l2h, -th), __fmaf_rn(r, l2l, __fmul_rn(yl, l2h)));
  const float q = __fmul_rn(__fmul_rn(th, th), __fmaf_rn(th, __fmaf_rn(th, 1.f / 24, 1.f / 6), 0.5f));
  const Exp2Entry e = tab[n & 255];
  const float p = __fmul_rn(e.hi, th);
  const float pe = __fmaf_rn(e.hi, th, -p);
  const float low = __fadd_rn(pe, __fmaf_rn(e.lo, th, __fmul_rn(e.hi, __fadd_rn(tl, q))));
  // the two parts as integers, by sums whose last bit is 2^-30 and 2^-41
  constexpr float c1 = 0.01171875f, c2 = 5.7220458984375e-06f;  // 1.5 2^-7, 1.5 2^-18
  const float s1 = __fadd_rn(p, c1);
  const int i1 = __float_as_int(s1) - __float_as_int(c1);
  const float rest = __fadd_rn(__fsub_rn(p, __fsub_rn(s1, c1)), low);
  const int i2 = __float_as_int(__fadd_rn(rest, c2)) - __float_as_int(c2);
  const uint64_t w = e.t + (int64_t)i1 * 65536 + (int64_t)i2 * 32;
  const int s = 46 - kUnit - (n >> 8);  // 2..42
  return (w + (1ull << (s - 1))) >> s;
}

// Order of the logits as unsigned integers.
__device__ __forceinline__ unsigned key_of(float x) {
  const unsigned b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// --------------------------------------------------------------------------- reductions

struct Shared {
  Exp2Entry tab[256];
  uint64_t mass[kThreads];
  int ties[kThreads];
  uint64_t buf[kWarps];
  unsigned ubuf[kWarps];
  int seg, tie_before;
  uint64_t rest;
};

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ uint64_t block_sum64(uint64_t v, Shared& sh) {
  v = warp_sum64(v);
  if ((threadIdx.x & 31) == 0) sh.buf[threadIdx.x / 32] = v;
  __syncthreads();
  v = warp_sum64(sh.buf[threadIdx.x & 31]);
  __syncthreads();
  return v;
}
__device__ __forceinline__ unsigned block_max(unsigned v, Shared& sh) {
  v = __reduce_max_sync(kFull, v);
  if ((threadIdx.x & 31) == 0) sh.ubuf[threadIdx.x / 32] = v;
  __syncthreads();
  v = __reduce_max_sync(kFull, sh.ubuf[threadIdx.x & 31]);
  __syncthreads();
  return v;
}
// Sum over the threads before this one.
__device__ __forceinline__ uint64_t block_before(uint64_t v, Shared& sh, uint64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  uint64_t incl = v;
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t up = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) sh.buf[warp] = incl;
  __syncthreads();
  uint64_t before = 0, all = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh.buf[w];
    all += sh.buf[w];
  }
  __syncthreads();
  *total = all;
  return before + incl - v;
}

// ------------------------------------------------------------------------------- kernel

struct Settings {
  float temp, top_p, min_p, u;
  int top_k;
};

__device__ Settings settings_of(const SampleCall& c, int row) {
  const tg_sample_params& p = c.p;
  Settings s{p.temperatures ? p.temperatures[row] : p.temperature, p.top_ps ? p.top_ps[row] : p.top_p,
             p.min_ps ? p.min_ps[row] : p.min_p, c.uniform[row], p.top_ks ? p.top_ks[row] : p.top_k};
  bool bad = false;
  if (!(s.temp >= 0.f)) { bad = true; s.temp = s.temp < 0.f ? 0.f : 1.f; }
  if (s.top_p != s.top_p) { bad = true; s.top_p = 1.f; }
  if (!(s.min_p <= 1.f)) { bad = true; s.min_p = s.min_p > 1.f ? 1.f : 0.f; }
  if (!(s.u >= 0.f && s.u < 1.f)) { bad = true; s.u = s.u >= 1.f ? 0.99999994f : 0.f; }
  if (bad && threadIdx.x == 0) record_error(c.err, kErrValue | kKernSample);
  return s;
}

// u in [0, 1) as a fraction of 2^64.
__device__ __forceinline__ uint64_t fraction(float u) { return (uint64_t)(u * 18446744073709551616.f); }

// One block per row.
template <typename T>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const SampleCall c) {
  __shared__ Shared sh;
  const int row = blockIdx.x, V = c.p.vocab, tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const T* x = static_cast<const T*>(c.logits) + (long long)row * c.p.pitch;
  // NaN as -inf, -0 as 0
  auto at = [&](int i) {
    const float v = io<T>::ld(x + i);
    return v == v ? v + 0.f : -INFINITY;
  };
  const Settings s = settings_of(c, row);
  load_exp2(sh.tab);
  unsigned top = 0;
  for (int i = tid; i < V; i += kThreads) top = max(top, key_of(at(i)));
  top = block_max(top, sh);
  const float mx = value_of(top);
  if (mx == -INFINITY || s.temp == 0.f) {
    unsigned first = 0;
    for (int i = tid; i < V; i += kThreads)
      if (at(i) == mx) first = max(first, kFull - (unsigned)i);
    first = kFull - block_max(first, sh);
    if (tid == 0) {
      c.token[row] = mx == -INFINITY ? -1 : (int)first;
      if (c.logprob) c.logprob[row] = mx == -INFINITY ? mx : 0.f;
    }
    return;
  }
  const Scale sc = scale_of(s.temp);

  // the cut: logits with a larger key are kept, and the first `ties` of those that equal it
  unsigned cut = 0;
  uint64_t ties = ~0ull;
  if (s.top_k > 0 && s.top_k < V) {  // the largest key that at least top_k logits reach
    unsigned lo = 0, hi = top;
    while (lo < hi) {
      const unsigned mid = lo + (hi - lo + 1) / 2;
      unsigned n = 0;
      for (int i = tid; i < V; i += kThreads) n += key_of(at(i)) >= mid;
      if (block_sum64(n, sh) >= (uint64_t)s.top_k) lo = mid;
      else hi = mid - 1;
    }
    cut = lo;
    unsigned n = 0;
    for (int i = tid; i < V; i += kThreads) n += key_of(at(i)) > cut;
    ties = s.top_k - block_sum64(n, sh);
  }
  auto above = [&](unsigned key) {  // mass of the logits above a key
    uint64_t g = 0;
    for (int i = tid; i < V; i += kThreads) {
      const float v = at(i);
      if (key_of(v) > key) g += weight(v, mx, sc, sh.tab);
    }
    return block_sum64(g, sh);
  };
  if (s.top_p < 1.f) {  // the smallest key above which there is less than the share
    const uint64_t w_cut = cut ? weight(value_of(cut), mx, sc, sh.tab) : 0;
    const uint64_t mass = above(cut) + (w_cut ? ties * w_cut : 0);
    const uint64_t f = fraction(s.top_p > 0.f ? s.top_p : 0.f), hi_part = __umul64hi(f, mass);
    uint64_t need = hi_part + (f * mass != 0);
    need = need ? need : 1;
    unsigned lo = cut, hi = top;
    while (lo < hi) {
      const unsigned mid = lo + (hi - lo) / 2;
      if (above(mid) < need) hi = mid;
      else lo = mid + 1;
    }
    const uint64_t w = lo ? weight(value_of(lo), mx, sc, sh.tab) : 0, g = above(lo);
    if (w) {
      const uint64_t n = (need - g + w - 1) / w;
      ties = lo > cut || n < ties ? n : ties;
    }
    cut = lo;
  }
  const uint64_t least = s.min_p > 0.f ? (uint64_t)ceilf(s.min_p * 17592186044416.f) : 0;  // 2^44
  const uint64_t w_cut = cut ? weight(value_of(cut), mx, sc, sh.tab) : 0;
  const bool cut_lives = w_cut && w_cut >= least;

  // mass and ties of up to kThreads equal spans of the row, then of the span that holds the token
  int span = 256;
  while ((V + span - 1) / span > kThreads) span *= 2;
  const int spans = (V + span - 1) / span;
  for (int g = warp; g < kThreads; g += kWarps) {
    uint64_t m = 0;
    unsigned n = 0;
    const int i1 = g < spans ? min(V, (g + 1) * span) : 0;
    for (int i = g * span + lane; i < i1; i += 32) {
      const float v = at(i);
      const unsigned key = key_of(v);
      if (key > cut) {
        const uint64_t w = weight(v, mx, sc, sh.tab);
        if (w >= least) m += w;
      }
      n += key == cut;
    }
    m = warp_sum64(m);
    n = __reduce_add_sync(kFull, n);
    if (lane == 0) {
      sh.mass[g] = m;
      sh.ties[g] = n;
    }
  }
  __syncthreads();
  uint64_t total;
  const uint64_t tie_before = block_before(sh.ties[tid], sh, &total);
  const uint64_t tie_left = tie_before < ties ? ties - tie_before : 0;
  const uint64_t n = tie_left < (uint64_t)sh.ties[tid] ? tie_left : sh.ties[tid];
  const uint64_t mine = sh.mass[tid] + (cut_lives ? n * w_cut : 0);
  const uint64_t before = block_before(mine, sh, &total);
  const uint64_t target = __umul64hi(fraction(s.u), total);  // the token is the first to pass it
  if (before <= target && target < before + mine) {
    sh.seg = tid;
    sh.rest = target - before;
    sh.tie_before = (int)(tie_before < ties ? tie_before : ties);
  }
  __syncthreads();
  if (warp != 0) return;
  uint64_t rest = sh.rest;
  uint64_t tb = sh.tie_before;
  const int i1 = min(V, (sh.seg + 1) * span);
  for (int i0 = sh.seg * span; i0 < i1; i0 += 32) {
    const float v = i0 + lane < i1 ? at(i0 + lane) : -INFINITY;
    const unsigned key = key_of(v);
    const bool tie = key == cut && i0 + lane < i1;
    const unsigned tie_mask = __ballot_sync(kFull, tie);
    uint64_t w = key > cut || (tie && tb + __popc(tie_mask & ((1u << lane) - 1)) < ties) ? weight(v, mx, sc, sh.tab) : 0;
    if (w < least) w = 0;
    tb += __popc(tie_mask);
    uint64_t incl = w;
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t up = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned hit = __ballot_sync(kFull, incl > rest);
    if (hit) {
      if (lane == __ffs(hit) - 1) {
        c.token[row] = i0 + lane;
        if (c.logprob) c.logprob[row] = w == total ? 0.f : logf((float)w / (float)total);
      }
      return;
    }
    rest -= __shfl_sync(kFull, incl, 31);
  }
}

}  // namespace

cudaError_t launch_sample(const SampleCall& c, cudaStream_t s) {
  if (c.p.dtype == TG_F32) sample_kernel<float><<<c.p.rows, kThreads, 0, s>>>(c);
  else sample_kernel<__nv_bfloat16><<<c.p.rows, kThreads, 0, s>>>(c);
  return cudaGetLastError();
}

}  // namespace tg

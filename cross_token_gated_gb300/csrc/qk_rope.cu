// Per-head norm of queries and keys with the rotary position in the same pass, its
// gradient, and the append of new keys and gates to a paged cache ("TANGO: Token-Aggregated
// Nonlinear Gating Operators ...", sec. 2.1: RoPE and the unit norm of q and k; eq. 2: the
// SiLU gate).
//
//   n = x r,  z = gain n,  out = R(pos) z;   r = 1/max(|x|, 1e-12) or 1/sqrt(mean x^2 + eps) or 1
//   backward: dz = R^T dout, dgain = sum dz n, dn = gain dz, dx = r (dn - n <n, dn>)
//
// Angles: a pair's frequency becomes turns per position as a 64-bit fraction F = frac(f / 2 pi)
// 2^64, and pos * F wraps at whole turns by itself; its high 32 bits are the angle in units
// of 2^-31 half turns, exact at any position, for sincospi.
//
// All of it is bound by HBM bandwidth (each value is read and written once), closely followed
// by issue slots, and for few rows by launch latency.  A block takes a few rows at a time: one
// thread per (row, pair) forms the angles' cos and sin in shared memory once for all heads of
// the row (a sincospi per element pair and head would cost more issue slots than the copy
// leaves).  A thread keeps one place of a row, 32 bytes of one head in two 16-byte vectors,
// and walks the rows, loaded ahead of the angles; the norm's sums are shuffles between the
// d_h / E lanes of a head, the arithmetic is packed two f32 at a time.  65,536 rows of 32
// heads of 32 in bf16 take 49.5 us (5.4 TB/s); gradients of 16,384 rows of 12 heads of 64 with
// gains 35.5 us, bound by latency at 16 warps an SM (124 registers a thread).  An append of
// 9,192 tokens of 9,504 gates takes 61.7 us (5.8 TB/s): a block per row, the row's slot looked
// up once while its gates are on their way.
#include <math.h>

#include <atomic>

#include "tg_common.cuh"
#include "tg_kernels.h"
#include "tg_paged.cuh"
#include "tg_ptx.cuh"
#include "tg_serve.h"

namespace tg {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 64;  // rotary_dim <= 128
constexpr int kMaxRowsBlk = 32;
constexpr int kAngles = 512;   // (row, pair) angles of a step

struct QkShared {
  uint64_t turns[kMaxPairs];
  // [row][pair]: the step's angles, and the one before's
  __align__(16) float cos[2][kAngles];
  __align__(16) float sin[2][kAngles];
};
// One row's angles.
struct RowAngles {
  const float *c, *s;
};
__device__ __forceinline__ RowAngles angles_of(const QkShared& sh, int side, int at) {
  return RowAngles{sh.cos[side] + at, sh.sin[side] + at};
}

// Turns per position of frequency f (radians per position, >= 0), as a fraction of 2^64.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  double t = f * 0.15915494309189535;  // 1 / (2 pi)
  t -= floor(t);
  return t >= 0.0 && t < 1.0 ? (uint64_t)(t * 18446744073709551616.0) : 0;  // NaN, inf: no rotation
}
// Cosine and sine of pos * turns.  A float holds up to a half turn to pi 2^-25, far below a bf16
// rounding; for fp32 outputs it holds the distance from the next quarter turn, to pi 2^-27 (gradients
// of 5,003 rows: error 8.0e-8 -> 7.0e-8; in bf16 the selections took 65,536 rows from 49.3 to 51.4 us).
template <typename T> __device__ __forceinline__ float2 turn_cos_sin(uint64_t turns, int pos);
template <> __device__ __forceinline__ float2 turn_cos_sin<__nv_bfloat16>(uint64_t turns, int pos) {
  const int half_turns = (int)((turns * (uint64_t)(int64_t)pos) >> 32);
  float s, c;
  sincospif((float)half_turns * 4.656612873077393e-10f, &s, &c);  // 2^-31
  return make_float2(c, s);
}
template <> __device__ __forceinline__ float2 turn_cos_sin<float>(uint64_t turns, int pos) {
  const unsigned angle = (unsigned)((turns * (uint64_t)(int64_t)pos) >> 32);
  const unsigned quarter = (angle + (1u << 29)) >> 30;
  float s, c;
  sincospif((float)(int)(angle - (quarter << 30)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
  const float x = quarter & 1 ? -s : c, y = quarter & 1 ? c : s;
  return quarter & 2 ? make_float2(-x, -y) : make_float2(x, y);
}

// A head's values as the threads of its group hold them: E values in two 16-byte vectors,
// V = E / 2 pairs that turn together, X the pairs' first values and Y their second ones, two
// per register pair (packed f32 arithmetic takes half the instructions, and these kernels
// are nearly bound by them).
template <typename T> struct Vec;
template <> struct Vec<float> {
  static constexpr int E = 8;  // values of a thread
  static __device__ __forceinline__ void unpack(const uint4& u, float* f) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y); f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int E = 16;
  static __device__ __forceinline__ void unpack(const uint4& u, float* f) {
    f[0] = ptx::bf16lo(u.x); f[1] = ptx::bf16hi(u.x); f[2] = ptx::bf16lo(u.y); f[3] = ptx::bf16hi(u.y);
    f[4] = ptx::bf16lo(u.z); f[5] = ptx::bf16hi(u.z); f[6] = ptx::bf16lo(u.w); f[7] = ptx::bf16hi(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]), ptx::pack_bf16x2(f[4], f[5]),
                      ptx::pack_bf16x2(f[6], f[7]));
  }
};

// Where lane l of a head's group finds its two vectors, and whether it rotates.
struct LaneMap {
  int off0, off1, pair0;
  bool rot;
};
template <typename T>
__device__ __forceinline__ LaneMap lane_map(int l, int rotary, int layout) {
  constexpr int E = Vec<T>::E, V = E / 2;
  LaneMap m;
  m.rot = l < rotary / E;
  const bool split = m.rot && layout == TG_ROPE_HALF;
  m.off0 = split ? l * V : l * E;
  m.off1 = split ? rotary / 2 + l * V : l * E + V;
  m.pair0 = l * V;
  return m;
}

template <typename T, bool kHalf>
struct Pairs {
  static constexpr int V = Vec<T>::E / 2, W = V / 2;
  uint64_t X[W], Y[W];
  // half layout: X is the first vector and Y the second; interleaved: neighbours of both
  __device__ __forceinline__ void load(const uint4& u0, const uint4& u1) {
    float f[2 * V];
    Vec<T>::unpack(u0, f);
    Vec<T>::unpack(u1, f + V);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      X[i] = kHalf ? ptx::f32x2_pack(f[2 * i], f[2 * i + 1]) : ptx::f32x2_pack(f[4 * i], f[4 * i + 2]);
      Y[i] = kHalf ? ptx::f32x2_pack(f[V + 2 * i], f[V + 2 * i + 1]) : ptx::f32x2_pack(f[4 * i + 1], f[4 * i + 3]);
    }
  }
  __device__ __forceinline__ void store(uint4& u0, uint4& u1) const {
    float f[2 * V];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (kHalf) {
        ptx::f32x2_unpack(X[i], f[2 * i], f[2 * i + 1]);
        ptx::f32x2_unpack(Y[i], f[V + 2 * i], f[V + 2 * i + 1]);
      } else {
        ptx::f32x2_unpack(X[i], f[4 * i], f[4 * i + 2]);
        ptx::f32x2_unpack(Y[i], f[4 * i + 1], f[4 * i + 3]);
      }
    }
    u0 = Vec<T>::pack(f);
    u1 = Vec<T>::pack(f + V);
  }
  // column of the pair's first (second) value
  static __device__ __forceinline__ int col_x(const LaneMap& m, int i) { return kHalf ? m.off0 + i : m.off0 + 2 * i; }
  static __device__ __forceinline__ int col_y(const LaneMap& m, int i) { return kHalf ? m.off1 + i : m.off0 + 2 * i + 1; }
  __device__ __forceinline__ void scale(float r) {
    const uint64_t rr = ptx::f32x2_pack(r, r);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      X[i] = ptx::mul_f32x2(X[i], rr);
      Y[i] = ptx::mul_f32x2(Y[i], rr);
    }
  }
  __device__ __forceinline__ void times(const float* gain, const LaneMap& m) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      X[i] = ptx::mul_f32x2(X[i], ptx::f32x2_pack(gain[col_x(m, 2 * i)], gain[col_x(m, 2 * i + 1)]));
      Y[i] = ptx::mul_f32x2(Y[i], ptx::f32x2_pack(gain[col_y(m, 2 * i)], gain[col_y(m, 2 * i + 1)]));
    }
  }
  // turned by the row's angles, or back
  __device__ __forceinline__ void turn(const RowAngles& e, const LaneMap& m, bool back) {
    if (!m.rot) return;
#pragma unroll
    for (int i = 0; i < W; i += 2) {
      const float4 c = *reinterpret_cast<const float4*>(e.c + m.pair0 + 2 * i);
      const float4 s = *reinterpret_cast<const float4*>(e.s + m.pair0 + 2 * i);
      const uint64_t C[2] = {ptx::f32x2_pack(c.x, c.y), ptx::f32x2_pack(c.z, c.w)};
      const uint64_t S[2] = {ptx::f32x2_pack(s.x, s.y), ptx::f32x2_pack(s.z, s.w)};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint64_t x = X[i + k], y = Y[i + k], n = ptx::neg_f32x2(S[k]);
        X[i + k] = ptx::fma_f32x2(y, back ? S[k] : n, ptx::mul_f32x2(x, C[k]));
        Y[i + k] = ptx::fma_f32x2(x, back ? n : S[k], ptx::mul_f32x2(y, C[k]));
      }
    }
  }
  __device__ __forceinline__ float dot(const Pairs& o) const {
    uint64_t s = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      s = ptx::fma_f32x2(X[i], o.X[i], s);
      s = ptx::fma_f32x2(Y[i], o.Y[i], s);
    }
    float lo, hi;
    ptx::f32x2_unpack(s, lo, hi);
    return lo + hi;
  }
};

// Sum over the lh lanes of a head's group (lh a power of two, lanes aligned to it).
__device__ __forceinline__ float group_sum(float v, int lh) {
  for (int o = lh >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Quotient, and 1 / sqrt: each step rounded once in fp32; the fast forms' errors (2 units of
// the last place) are far below a bf16 rounding.
template <typename T> __device__ __forceinline__ float quotient(float x, float y);
template <> __device__ __forceinline__ float quotient<float>(float x, float y) { return x / y; }
template <> __device__ __forceinline__ float quotient<__nv_bfloat16>(float x, float y) { return __fdividef(x, y); }
template <typename T> __device__ __forceinline__ float inv_sqrt(float x);
template <> __device__ __forceinline__ float inv_sqrt<float>(float x) { return 1.f / sqrtf(x); }
template <> __device__ __forceinline__ float inv_sqrt<__nv_bfloat16>(float x) { return rsqrtf(x); }

// r of the norm from the sum of squares.  A NaN stays one (a maximum would replace it by the
// floor, and leave a head with one NaN 1e12 times its other values).
template <typename T>
__device__ __forceinline__ float inv_norm(float ss, int d_h, int norm, float eps) {
  if (norm == TG_NORM_UNIT) return inv_sqrt<T>(ss < 1e-24f ? 1e-24f : ss);  // 1 / max(|x|, 1e-12)
  if (norm == TG_NORM_RMS) return inv_sqrt<T>(quotient<T>(ss, (float)d_h) + eps);
  return 1.f;
}

// What a forward pass over rows needs, shared by the norm call and the cache append.
struct FwdRows {
  int d_h, rotary, layout, norm;
  float eps;
};

// One head by its group of lanes, from the two vectors each has loaded: norm, gain, rotate,
// store.
template <typename T, bool kHalf>
__device__ __forceinline__ void head_forward(const uint4& u0, const uint4& u1, T* dst, bool live, const FwdRows& f,
                                             const LaneMap& m, int lh, const float* gain, const RowAngles& e) {
  Pairs<T, kHalf> z;
  z.load(u0, u1);
  if (f.norm != TG_NORM_NONE) z.scale(inv_norm<T>(group_sum(z.dot(z), lh), f.d_h, f.norm, f.eps));
  if (gain) z.times(gain, m);
  z.turn(e, m, false);
  uint4 w0, w1;
  z.store(w0, w1);
  if (live) {
    *reinterpret_cast<uint4*>(dst + m.off0) = w0;
    *reinterpret_cast<uint4*>(dst + m.off1) = w1;
  }
}

// A head by a whole warp, any width, pairing and alignment: values go through `buf`
// (2 x 128 floats per warp).
template <typename T>
__device__ __forceinline__ void head_forward_any(const T* src, T* dst, const FwdRows& f, const float* gain,
                                                 const RowAngles& e, float* buf) {
  const int lane = threadIdx.x & 31;
  float ss = 0.f;
  for (int c = lane; c < f.d_h; c += 32) {
    const float x = io<T>::ld(src + c);
    buf[c] = x;
    ss += x * x;
  }
  const float r = f.norm == TG_NORM_NONE ? 1.f : inv_norm<T>(group_sum(ss, 32), f.d_h, f.norm, f.eps);
  __syncwarp();
  const int hp = f.rotary / 2;
  for (int c = lane; c < f.d_h; c += 32) {
    float z = buf[c] * r * (gain ? gain[c] : 1.f);
    if (c < f.rotary) {
      const bool first = f.layout == TG_ROPE_HALF ? c < hp : !(c & 1);
      const int pair = f.layout == TG_ROPE_HALF ? (first ? c : c - hp) : c >> 1;
      const int mate = f.layout == TG_ROPE_HALF ? (first ? c + hp : c - hp) : c ^ 1;
      const float w = buf[mate] * r * (gain ? gain[mate] : 1.f);
      z = first ? z * e.c[pair] - w * e.s[pair] : z * e.c[pair] + w * e.s[pair];
    }
    io<T>::st(dst + c, z);
  }
  __syncwarp();
}

__device__ __forceinline__ void load_turns(QkShared& sh, const double* freqs, int pairs) {
  for (int c = threadIdx.x; c < pairs; c += kThreads) sh.turns[c] = turn_fraction(freqs[c]);
  __syncthreads();
}

template <typename T>
struct QkArgs {
  long long rows;
  int H, Hk, T_len;
  FwdRows f;
  const int* positions;
  const double* freqs;
  const float *q_gain, *k_gain;
  long long q_pitch, k_pitch;
  const T *q, *k;
  T *q_out, *k_out;
  const T *dq_out, *dk_out;  // backward
  T *dq, *dk;
  float* part;               // backward: [blocks][2][d_h] gain gradients
  int want_gain;
  int rb;                    // rows of a block's step (<= kMaxRowsBlk)
};

__device__ __forceinline__ int row_pos(const int* positions, int T_len, long long row) {
  return positions ? positions[row] : (int)(row % T_len);
}

// The rows' angles: one thread per (row, pair).
template <typename T>
__device__ __forceinline__ void row_angles(QkShared& sh, int buf, const QkArgs<T>& a, long long row0, int nr) {
  const int pairs = a.f.rotary / 2;
  for (int i = threadIdx.x; i < nr * pairs; i += kThreads) {
    const int r = i / pairs, c = i - r * pairs;
    const float2 e = turn_cos_sin<T>(sh.turns[c], row_pos(a.positions, a.T_len, row0 + r));
    sh.cos[buf][i] = e.x;
    sh.sin[buf][i] = e.y;
  }
}

constexpr int kAheadRows = 2;  // rows of a thread that are loaded before the angles are formed

// Where head number h of a step's rows lies: q's heads of a row, then k's.
struct HeadRef {
  int r, hh;
  bool live, is_q;
};
__device__ __forceinline__ HeadRef head_ref(int h, int heads, int H, int HT) {
  HeadRef x;
  x.live = h < heads;
  x.r = x.live ? h / HT : 0;
  x.hh = x.live ? h - x.r * HT : 0;
  x.is_q = x.hh < H;
  return x;
}

// A thread's fixed place in a row: one head (q's, then k's) and its lane there, `cols` places
// in all; rows are spread over the block's other threads (no division is left in the loop).
// Rows of more places than threads are walked in rounds of kThreads.
struct Place {
  int cols, row_step, row, first;  // row >= row_step: no work
  __device__ __forceinline__ Place(int cols_) : cols(cols_) {
    row_step = cols < kThreads ? kThreads / cols : 1;
    row = cols < kThreads ? (int)threadIdx.x / cols : 0;
    first = cols < kThreads ? (int)threadIdx.x - row * cols : (int)threadIdx.x;
  }
};

template <typename T, bool kVec, bool kHalf>
__global__ void __launch_bounds__(kThreads, 4) qk_forward_kernel(const QkArgs<T> a) {
  __shared__ QkShared sh;
  __shared__ float buf[kVec ? 1 : kThreads / 32][kVec ? 1 : 128];
  load_turns(sh, a.freqs, a.f.rotary / 2);
  const int HT = a.H + a.Hk, lh = kVec ? a.f.d_h / Vec<T>::E : 32, pairs = a.f.rotary / 2;
  const LaneMap m = lane_map<T>(threadIdx.x % lh, a.f.rotary, a.f.layout);
  const Place pl(HT * lh);
  int side = 0;
  for (long long row0 = (long long)blockIdx.x * a.rb; row0 < a.rows; row0 += (long long)gridDim.x * a.rb, side ^= 1) {
    const int nr = (int)min((long long)a.rb, a.rows - row0);
    if (kVec) {
      for (int c0 = 0; c0 < pl.cols; c0 += kThreads) {  // (one round but for very wide rows)
        const int hh = (c0 + pl.first) / lh;
        const bool is_q = hh < a.H, mine = pl.row < pl.row_step && hh < HT;
        const T* src = is_q ? a.q + hh * a.f.d_h : a.k + (hh - a.H) * a.f.d_h;
        T* dst = is_q ? a.q_out + hh * a.f.d_h : a.k_out + (hh - a.H) * a.f.d_h;
        const long long sp = is_q ? a.q_pitch : a.k_pitch, dp = (long long)(is_q ? a.H : a.Hk) * a.f.d_h;
        // the first rows are on their way while the angles are formed
        uint4 u[kAheadRows][2];
        auto load = [&](int k, int r) {
          const bool live = mine && r < nr;
          const T* x = src + (row0 + r) * sp;
          u[k][0] = live ? *reinterpret_cast<const uint4*>(x + m.off0) : make_uint4(0, 0, 0, 0);
          u[k][1] = live ? *reinterpret_cast<const uint4*>(x + m.off1) : make_uint4(0, 0, 0, 0);
        };
#pragma unroll
        for (int k = 0; k < kAheadRows; ++k) load(k, pl.row + k * pl.row_step);
        if (c0 == 0) {
          row_angles(sh, side, a, row0, nr);
          __syncthreads();
        }
        for (int r0 = 0; r0 < nr; r0 += kAheadRows * pl.row_step) {
#pragma unroll
          for (int k = 0; k < kAheadRows; ++k) {
            const int r = r0 + k * pl.row_step + pl.row;
            if (r0 > 0) load(k, r);
            const bool live = mine && r < nr;
            head_forward<T, kHalf>(u[k][0], u[k][1], dst + (row0 + r) * dp, live, a.f, m, lh, is_q ? a.q_gain : a.k_gain,
                            angles_of(sh, side, (live ? r : 0) * pairs));
          }
        }
      }
    } else {
      row_angles(sh, side, a, row0, nr);
      __syncthreads();
      for (int h = threadIdx.x / 32; h < nr * HT; h += kThreads / 32) {
        const HeadRef x = head_ref(h, nr * HT, a.H, HT);
        const long long row = row0 + x.r;
        const T* src = x.is_q ? a.q + row * a.q_pitch + (long long)x.hh * a.f.d_h
                              : a.k + row * a.k_pitch + (long long)(x.hh - a.H) * a.f.d_h;
        T* dst = x.is_q ? a.q_out + (row * a.H + x.hh) * a.f.d_h : a.k_out + (row * a.Hk + x.hh - a.H) * a.f.d_h;
        head_forward_any<T>(src, dst, a.f, x.is_q ? a.q_gain : a.k_gain, angles_of(sh, side, x.r * pairs),
                            buf[kVec ? 0 : threadIdx.x / 32]);
      }
    }
    // (no barrier here: the next step's angles go to the other buffer)
  }
}

// ------------------------------------------------------------------------ backward

// One head's gradient by its group of lanes, from the vectors of x and dout that each has
// loaded.  n * dz is added to the lane's sums for the gain's gradient.
template <typename T, bool kHalf, bool kGain>
__device__ __forceinline__ void head_backward(const uint4 (&u)[4], T* dst, bool live, const FwdRows& f, const LaneMap& m,
                                              int lh, const float* gain, const RowAngles& e, Pairs<T, kHalf>& sum) {
  Pairs<T, kHalf> n, d;
  n.load(u[0], u[1]);
  d.load(u[2], u[3]);
  d.turn(e, m, true);  // dz
  float rn = 1.f;
  bool floor_hit = false;
  if (f.norm != TG_NORM_NONE) {
    const float ss = group_sum(n.dot(n), lh);
    rn = inv_norm<T>(ss, f.d_h, f.norm, f.eps);
    floor_hit = f.norm == TG_NORM_UNIT && ss < 1e-24f;
    n.scale(rn);
  }
  if (gain) {
    if (kGain) {  // (lanes without a row hold zeros)
#pragma unroll
      for (int i = 0; i < Pairs<T, kHalf>::W; ++i) {
        sum.X[i] = ptx::fma_f32x2(d.X[i], n.X[i], sum.X[i]);
        sum.Y[i] = ptx::fma_f32x2(d.Y[i], n.Y[i], sum.Y[i]);
      }
    }
    d.times(gain, m);  // dn
  }
  if (f.norm != TG_NORM_NONE) {
    float along = group_sum(n.dot(d), lh);
    if (f.norm == TG_NORM_RMS) along = quotient<T>(along, (float)f.d_h);
    if (floor_hit) along = 0.f;
    const uint64_t rr = ptx::f32x2_pack(rn, rn), aa = ptx::f32x2_pack(-along * rn, -along * rn);
#pragma unroll
    for (int i = 0; i < Pairs<T, kHalf>::W; ++i) {
      d.X[i] = ptx::fma_f32x2(n.X[i], aa, ptx::mul_f32x2(d.X[i], rr));
      d.Y[i] = ptx::fma_f32x2(n.Y[i], aa, ptx::mul_f32x2(d.Y[i], rr));
    }
  }
  uint4 w0, w1;
  d.store(w0, w1);
  if (live) {
    *reinterpret_cast<uint4*>(dst + m.off0) = w0;
    *reinterpret_cast<uint4*>(dst + m.off1) = w1;
  }
}

// The same by whole warps for any width and alignment; gain gradients go to acc[d_h],
// one float per column of this warp.
template <typename T>
__device__ __forceinline__ void rows_backward_any(const QkArgs<T>& a, QkShared& sh, int side, long long row0, int nr, int H,
                                                  const T* x, long long pitch, const T* dout, T* dx,
                                                  const float* gain, float* buf, float* acc) {
  const int lane = threadIdx.x & 31, hp = a.f.rotary / 2;
  for (int h = threadIdx.x / 32; h < nr * H; h += kThreads / 32) {
    const int r = h / H, hh = h - r * H;
    const long long row = row0 + r, at = (row * H + hh) * a.f.d_h;
    const T* src = x + row * pitch + (long long)hh * a.f.d_h;
    float ss = 0.f;
    for (int c = lane; c < a.f.d_h; c += 32) {
      const float v = io<T>::ld(src + c);
      ss += v * v;
      buf[c] = io<T>::ld(dout + at + c);
    }
    float rn = 1.f;
    bool floor_hit = false;
    if (a.f.norm != TG_NORM_NONE) {
      ss = group_sum(ss, 32);
      rn = inv_norm<T>(ss, a.f.d_h, a.f.norm, a.f.eps);
      floor_hit = a.f.norm == TG_NORM_UNIT && ss < 1e-24f;
    }
    __syncwarp();
    float n[4], dn[4], dot = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = lane + 32 * i;
      if (c >= a.f.d_h) break;
      float dz = buf[c];
      if (c < a.f.rotary) {
        const bool first = a.f.layout == TG_ROPE_HALF ? c < hp : !(c & 1);
        const int pair = a.f.layout == TG_ROPE_HALF ? (first ? c : c - hp) : c >> 1;
        const int mate = a.f.layout == TG_ROPE_HALF ? (first ? c + hp : c - hp) : c ^ 1;
        const float c0 = sh.cos[side][r * hp + pair], s0 = sh.sin[side][r * hp + pair];
        dz = first ? dz * c0 + buf[mate] * s0 : dz * c0 - buf[mate] * s0;
      }
      n[i] = io<T>::ld(src + c) * rn;
      if (gain && acc) acc[c] = fmaf(dz, n[i], acc[c]);
      dn[i] = gain ? dz * gain[c] : dz;
      dot += n[i] * dn[i];
    }
    if (a.f.norm != TG_NORM_NONE) {
      dot = group_sum(dot, 32);
      if (a.f.norm == TG_NORM_RMS) dot /= (float)a.f.d_h;
    }
    if (floor_hit || a.f.norm == TG_NORM_NONE) dot = 0.f;
    __syncwarp();  // every lane has read buf, and dout where dx overwrites it
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = lane + 32 * i;
      if (c >= a.f.d_h) break;
      io<T>::st(dx + at + c, rn * (dn[i] - n[i] * dot));
    }
    __syncwarp();
  }
}

template <typename T, bool kVec, bool kHalf, bool kGain>
__global__ void __launch_bounds__(kThreads, kVec ? 2 : 1) qk_backward_kernel(const QkArgs<T> a) {
  constexpr int V = Vec<T>::E / 2;
  __shared__ QkShared sh;
  __shared__ float buf[kVec ? 1 : kThreads / 32][kVec ? 1 : 128];
  __shared__ float acc[2][kThreads / 32][kGain ? 128 : 1];  // gain gradients, one copy per warp
  if (kGain) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  load_turns(sh, a.freqs, a.f.rotary / 2);
  const int HT = a.H + a.Hk, lh = kVec ? a.f.d_h / Vec<T>::E : 32, w = threadIdx.x / 32, pairs = a.f.rotary / 2;
  const LaneMap m = lane_map<T>(threadIdx.x % lh, a.f.rotary, a.f.layout);
  const Place pl(HT * lh);
  if (kGain) {
    for (int i = threadIdx.x; i < 2 * (kThreads / 32) * 128; i += kThreads) (&acc[0][0][0])[i] = 0.f;
    __syncthreads();
  }
  int side = 0;
  // the places of a round are walked over all the block's rows, so that a thread's head, and
  // with it the gain it sums for, stays the same
  for (int c0 = 0; c0 < (kVec ? pl.cols : 1); c0 += kThreads) {
    const int hh = (c0 + pl.first) / lh;
    const bool is_q = hh < a.H, mine = pl.row < pl.row_step && hh < HT;
    const T* src = is_q ? a.q + hh * a.f.d_h : a.k + (hh - a.H) * a.f.d_h;
    const T* dy = is_q ? a.dq_out + hh * a.f.d_h : a.dk_out + (hh - a.H) * a.f.d_h;
    T* dst = is_q ? a.dq + hh * a.f.d_h : a.dk + (hh - a.H) * a.f.d_h;
    const float* gain = is_q ? a.q_gain : a.k_gain;
    const long long sp = is_q ? a.q_pitch : a.k_pitch, dp = (long long)(is_q ? a.H : a.Hk) * a.f.d_h;
    Pairs<T, kHalf> sum = {};  // the gain's gradient, this lane's columns
    for (long long row0 = (long long)blockIdx.x * a.rb; row0 < a.rows; row0 += (long long)gridDim.x * a.rb, side ^= 1) {
      const int nr = (int)min((long long)a.rb, a.rows - row0);
      if (kVec) {
        uint4 u[kAheadRows][4];
        auto load = [&](int k, int r) {
          const bool live = mine && r < nr;
          const T *x = src + (row0 + r) * sp, *y = dy + (row0 + r) * dp;
          const uint4 z = make_uint4(0, 0, 0, 0);
          u[k][0] = live ? *reinterpret_cast<const uint4*>(x + m.off0) : z;
          u[k][1] = live ? *reinterpret_cast<const uint4*>(x + m.off1) : z;
          u[k][2] = live ? *reinterpret_cast<const uint4*>(y + m.off0) : z;
          u[k][3] = live ? *reinterpret_cast<const uint4*>(y + m.off1) : z;
        };
#pragma unroll
        for (int k = 0; k < kAheadRows; ++k) load(k, pl.row + k * pl.row_step);
        row_angles(sh, side, a, row0, nr);
        __syncthreads();
        for (int r0 = 0; r0 < nr; r0 += kAheadRows * pl.row_step) {
#pragma unroll
          for (int k = 0; k < kAheadRows; ++k) {
            const int r = r0 + k * pl.row_step + pl.row;
            if (r0 > 0) load(k, r);
            const bool live = mine && r < nr;
            head_backward<T, kHalf, kGain>(u[k], dst + (row0 + r) * dp, live, a.f, m, lh, gain,
                                           angles_of(sh, side, (live ? r : 0) * pairs), sum);
          }
        }
      } else {
        row_angles(sh, side, a, row0, nr);
        __syncthreads();
        rows_backward_any<T>(a, sh, side, row0, nr, a.H, a.q, a.q_pitch, a.dq_out, a.dq, a.q_gain, buf[kVec ? 0 : w],
                             kGain ? acc[0][w] : nullptr);
        rows_backward_any<T>(a, sh, side, row0, nr, a.Hk, a.k, a.k_pitch, a.dk_out, a.dk, a.k_gain, buf[kVec ? 0 : w],
                             kGain ? acc[1][w] : nullptr);
      }
    }
    if (kVec && kGain) {
      // over the warp's lanes of the same columns, q's and k's heads apart
      float sx[V], sy[V];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        ptx::f32x2_unpack(sum.X[i], sx[2 * i], sx[2 * i + 1]);
        ptx::f32x2_unpack(sum.Y[i], sy[2 * i], sy[2 * i + 1]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float qx = mine && is_q ? sx[i] : 0.f, qy = mine && is_q ? sy[i] : 0.f;
        float kx = mine && !is_q ? sx[i] : 0.f, ky = mine && !is_q ? sy[i] : 0.f;
        for (int o = 16; o >= lh; o >>= 1) {
          qx += __shfl_xor_sync(0xffffffffu, qx, o);
          qy += __shfl_xor_sync(0xffffffffu, qy, o);
          kx += __shfl_xor_sync(0xffffffffu, kx, o);
          ky += __shfl_xor_sync(0xffffffffu, ky, o);
        }
        if ((threadIdx.x & 31) < lh) {
          const int cx = Pairs<T, kHalf>::col_x(m, i), cy = Pairs<T, kHalf>::col_y(m, i);
          acc[0][w][kGain ? cx : 0] += qx;
          acc[0][w][kGain ? cy : 0] += qy;
          acc[1][w][kGain ? cx : 0] += kx;
          acc[1][w][kGain ? cy : 0] += ky;
        }
      }
    }
  }
  if (!kGain) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.f.d_h; i += kThreads) {
    const int side = i / a.f.d_h, c = i - side * a.f.d_h;  // q's gain, k's gain
    float s = 0.f;
    for (int k = 0; k < kThreads / 32; ++k) s += acc[side][k][kGain ? c : 0];
    a.part[((size_t)blockIdx.x * 2 + side) * a.f.d_h + c] = s;
  }
}

// dgain[c] = sum of the blocks' partial sums, in a fixed order: grid (d_h / 8, 2), a warp per
// column.
__global__ void __launch_bounds__(256) qk_gain_sum_kernel(const float* part, int blocks, int d_h, float* dqg, float* dkg) {
  const int c = blockIdx.x * 8 + threadIdx.x / 32, side = blockIdx.y, lane = threadIdx.x & 31;
  float* dst = side ? dkg : dqg;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c >= d_h || !dst) return;
  float s = 0.f;
  for (int b = lane; b < blocks; b += 32) s += __ldcg(part + ((size_t)b * 2 + side) * d_h + c);
  s = group_sum(s, 32);
  if (lane == 0) dst[c] = s;
}

// --------------------------------------------------------------------------- append

template <typename T>
struct AppendArgs {
  PagedBatch p;
  int H, m_h, m_pitch;
  FwdRows f;
  const double* freqs;
  int silu;
  long long q_pitch, k_pitch, g_pitch;
  const T *q, *k, *g;
  T *q_out, *k_pages, *g_pages;
  int qk_blocks, rb;   // the first qk_blocks blocks take rb rows of q and k at a time
  int chunks;          // gate chunks of a row
};

struct Slot {
  int pos;        // position, negative: none
  long long tok;  // page * page_size + offset, or -1
};
// Where new token `row` goes; a whole warp asks for one row.
__device__ __forceinline__ Slot find_slot(const PagedBatch& p, int row) {
  const int b = paged_find(p, row);
  const PagedSeq s = paged_seq(p, b, true);
  Slot r{-1, -1};
  if (row < s.r0 || row >= s.r0 + s.n) {
    return r;  // a row of no sequence
  }
  r.pos = s.len - s.n + (row - s.r0);
  if (r.pos < 0) return r;
  const int pi = r.pos / p.page_size, pg = paged_page(p, b, pi);
  if (pg >= 0) r.tok = (long long)pg * p.page_size + (r.pos - pi * p.page_size);
  return r;
}

// x sigmoid(x); the fast exponential's error (a few 2^-22) is far below a bf16 rounding
template <typename T> __device__ __forceinline__ float silu_of(float x);
template <> __device__ __forceinline__ float silu_of<float>(float x) { return x / (1.f + expf(-x)); }
template <> __device__ __forceinline__ float silu_of<__nv_bfloat16>(float x) { return __fdividef(x, 1.f + __expf(-x)); }

constexpr int kGateVecs = 4;  // 16-byte vectors of a thread that are on their way at a time

template <typename T, bool kVec, bool kHalf>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const AppendArgs<T> a) {
  __shared__ QkShared sh;
  __shared__ Slot slot[kMaxRowsBlk];
  __shared__ float buf[kVec ? 1 : kThreads / 32][kVec ? 1 : 128];
  const int w = threadIdx.x / 32;
  if ((int)blockIdx.x >= a.qk_blocks) {
    // ---- gates: one chunk of one row
    const int gb = blockIdx.x - a.qk_blocks, row = gb / a.chunks, chunk = gb - row * a.chunks;
    const T* src = a.g + (long long)row * a.g_pitch;
    if (kVec) {
      constexpr int EV = 16 / sizeof(T);
      const int nv = a.H * a.m_pitch / EV, per = (nv + a.chunks - 1) / a.chunks;
      const int end = min(nv, (chunk + 1) * per);
      uint4 u[kGateVecs];
      int v0 = chunk * per + threadIdx.x;
      auto load = [&]() {
#pragma unroll
        for (int i = 0; i < kGateVecs; ++i)
          if (v0 + i * kThreads < end) u[i] = ptx::ld_global_v4(src + (long long)(v0 + i * kThreads) * EV);
      };
      load();  // on its way before the slot is known
      const Slot s = find_slot(a.p, row);
      if (s.tok < 0) return;
      T* dst = a.g_pages + s.tok * ((long long)a.H * a.m_pitch);
      for (; v0 < end; v0 += kGateVecs * kThreads, load()) {
#pragma unroll
        for (int i = 0; i < kGateVecs; ++i) {
          if (v0 + i * kThreads >= end) break;
          if (a.silu) {
            float x[EV];
            Vec<T>::unpack(u[i], x);
#pragma unroll
            for (int e = 0; e < EV; ++e) x[e] = silu_of<T>(x[e]);
            u[i] = Vec<T>::pack(x);
          }
          *reinterpret_cast<uint4*>(dst + (long long)(v0 + i * kThreads) * EV) = u[i];
        }
      }
    } else {
      const Slot s = find_slot(a.p, row);
      if (s.tok < 0) return;
      T* dst = a.g_pages + s.tok * ((long long)a.H * a.m_pitch);
      const int m = a.H * a.m_h, per = (m + a.chunks - 1) / a.chunks;
      for (int i = chunk * per + threadIdx.x; i < min(m, (chunk + 1) * per); i += kThreads) {
        const int h = i / a.m_h, at = h * a.m_pitch + (i - h * a.m_h);
        const float x = io<T>::ld(src + at);
        io<T>::st(dst + at, a.silu ? silu_of<T>(x) : x);
      }
    }
    return;
  }
  // ---- keys, and queries where asked
  load_turns(sh, a.freqs, a.f.rotary / 2);
  const int HT = a.q ? 2 * a.H : a.H, lh = kVec ? a.f.d_h / Vec<T>::E : 32;
  const LaneMap m = lane_map<T>(threadIdx.x % lh, a.f.rotary, a.f.layout);
  const int pairs = a.f.rotary / 2;
  int side = 0;
  for (int row0 = blockIdx.x * a.rb; row0 < a.p.N; row0 += a.qk_blocks * a.rb, side ^= 1) {
    const int nr = min(a.rb, a.p.N - row0);
    __syncthreads();  // the step before has read its slots
    for (int r = w; r < nr; r += kThreads / 32) {
      const Slot s = find_slot(a.p, row0 + r);
      if ((threadIdx.x & 31) == 0) slot[r] = s;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nr * pairs; i += kThreads) {
      const int r = i / pairs, c = i - r * pairs;
      const float2 e = turn_cos_sin<T>(sh.turns[c], slot[r].pos);
      sh.cos[side][i] = e.x;
      sh.sin[side][i] = e.y;
    }
    __syncthreads();
    const int heads = nr * HT;
    for (int h0 = 0; h0 < heads; h0 += kThreads / lh) {
      const HeadRef x = head_ref(h0 + threadIdx.x / lh, heads, a.H, HT);
      const bool is_k = x.is_q;  // keys come first here
      const int hd = is_k ? x.hh : x.hh - a.H;
      const long long row = row0 + x.r;
      const bool live = x.live && (!is_k || slot[x.r].tok >= 0);
      const T* src = is_k ? a.k + row * a.k_pitch + (long long)hd * a.f.d_h : a.q + row * a.q_pitch + (long long)hd * a.f.d_h;
      T* dst = is_k ? a.k_pages + (max(slot[x.r].tok, 0ll) * a.H + hd) * a.f.d_h : a.q_out + (row * a.H + hd) * a.f.d_h;
      if (kVec) {
        const uint4 z = make_uint4(0, 0, 0, 0);
        const uint4 u0 = live ? *reinterpret_cast<const uint4*>(src + m.off0) : z;
        const uint4 u1 = live ? *reinterpret_cast<const uint4*>(src + m.off1) : z;
        head_forward<T, kHalf>(u0, u1, dst, live, a.f, m, lh, nullptr, angles_of(sh, side, x.r * pairs));
      } else if (live) {
        head_forward_any<T>(src, dst, a.f, nullptr, angles_of(sh, side, x.r * pairs), buf[kVec ? 0 : w]);
      }
    }
  }
}

// --------------------------------------------------------------------------- launch

bool pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether heads split into two 16-byte vectors per lane: whole lanes rotate or pass, a
// head's lanes are a power of two, and every row starts on 16 bytes.
bool vec_heads(int d_h, int rotary, int es, std::initializer_list<const void*> ptrs,
               std::initializer_list<long long> pitches) {
  const int E = 32 / es;
  if (d_h % E != 0 || rotary % E != 0 || !pow2(d_h / E)) return false;
  for (const void* p : ptrs)
    if (!al16(p)) return false;
  for (long long x : pitches)
    if (x * es % 16 != 0) return false;
  return true;
}

// Rows of a block's step: as many as its threads load ahead (`places` threads a row), fewer
// while that leaves SMs idle.
int rows_per_block(long long rows, int places, int pairs) {
  const int want = 2 * serve_sm_count();
  int rb = kAheadRows * (places < kThreads ? kThreads / places : 1);
  if (rb > kMaxRowsBlk) rb = kMaxRowsBlk;
  if (pairs > 0 && rb > kAngles / pairs) rb = kAngles / pairs;
  while (rb > 1 && rows / rb < want) rb = (rb + 1) / 2;
  return rb;
}

template <typename T>
QkArgs<T> qk_args(const QkCall& c) {
  QkArgs<T> a;
  a.rows = c.rows; a.H = c.H; a.Hk = c.Hk; a.T_len = c.T;
  a.f = FwdRows{c.d_h, c.rotary, c.layout, c.norm, c.eps};
  a.positions = c.positions; a.freqs = c.freqs; a.q_gain = c.q_gain; a.k_gain = c.k_gain;
  a.q_pitch = c.q_pitch; a.k_pitch = c.k_pitch;
  a.q = static_cast<const T*>(c.q); a.k = static_cast<const T*>(c.k);
  a.q_out = static_cast<T*>(c.q_out); a.k_out = static_cast<T*>(c.k_out);
  a.dq_out = static_cast<const T*>(c.dq_out); a.dk_out = static_cast<const T*>(c.dk_out);
  a.dq = static_cast<T*>(c.dq); a.dk = static_cast<T*>(c.dk);
  a.part = c.part;
  a.want_gain = c.dq_gain || c.dk_gain;
  a.rb = rows_per_block(c.rows, (c.H + c.Hk) * ((c.d_h * (int)sizeof(T) + 31) / 32), c.rotary / 2);
  return a;
}

int qk_grid(long long rows, int rb, int per_sm) {
  const long long blocks = (rows + rb - 1) / rb, most = (long long)serve_sm_count() * per_sm;
  return (int)(blocks < most ? blocks : most);
}

template <typename T>
cudaError_t forward_t(const QkCall& c, cudaStream_t s) {
  const QkArgs<T> a = qk_args<T>(c);
  const int grid = qk_grid(c.rows, a.rb, 4);
  if (vec_heads(c.d_h, c.rotary, sizeof(T), {c.q, c.k, c.q_out, c.k_out}, {c.q_pitch, c.k_pitch}))
    c.layout == TG_ROPE_HALF ? qk_forward_kernel<T, true, true><<<grid, kThreads, 0, s>>>(a)
                             : qk_forward_kernel<T, true, false><<<grid, kThreads, 0, s>>>(a);
  else
    qk_forward_kernel<T, false, true><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

constexpr int kBwdPerSm = 2;  // the blocks that fit: the grid is persistent

template <typename T, bool kVec, bool kHalf>
void backward_vt(const QkArgs<T>& a, int grid, cudaStream_t s) {
  if (a.want_gain) qk_backward_kernel<T, kVec, kHalf, true><<<grid, kThreads, 0, s>>>(a);
  else qk_backward_kernel<T, kVec, kHalf, false><<<grid, kThreads, 0, s>>>(a);
}

template <typename T>
cudaError_t backward_t(const QkCall& c, cudaStream_t s) {
  const QkArgs<T> a = qk_args<T>(c);
  const int grid = qk_grid(c.rows, a.rb, kBwdPerSm);
  if (vec_heads(c.d_h, c.rotary, sizeof(T), {c.q, c.k, c.dq_out, c.dk_out, c.dq, c.dk}, {c.q_pitch, c.k_pitch}))
    c.layout == TG_ROPE_HALF ? backward_vt<T, true, true>(a, grid, s) : backward_vt<T, true, false>(a, grid, s);
  else
    backward_vt<T, false, true>(a, grid, s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.want_gain) return e;
  // launched while the last blocks still run; it waits for their sums itself
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ceil_div(c.d_h, 8), 2);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_gain_sum_kernel, (const float*)c.part, grid, c.d_h, c.dq_gain, c.dk_gain);
}

template <typename T>
cudaError_t append_t(const AppendCall& c, cudaStream_t s) {
  AppendArgs<T> a;
  a.p = c.p; a.H = c.H; a.m_h = c.m_h; a.m_pitch = c.m_pitch;
  a.f = FwdRows{c.d_h, c.rotary, c.layout, c.norm, c.eps};
  a.freqs = c.freqs; a.silu = c.silu;
  a.q_pitch = c.q_pitch; a.k_pitch = c.k_pitch; a.g_pitch = c.g_pitch;
  a.q = static_cast<const T*>(c.q); a.k = static_cast<const T*>(c.k); a.g = static_cast<const T*>(c.g);
  a.q_out = static_cast<T*>(c.q_out);
  a.k_pages = static_cast<T*>(c.k_pages); a.g_pages = static_cast<T*>(c.g_pages);
  a.rb = rows_per_block(c.p.N, (c.q ? 2 : 1) * c.H * ((c.d_h * (int)sizeof(T) + 31) / 32), c.rotary / 2);
  a.qk_blocks = qk_grid(c.p.N, a.rb, 2);
  const bool vec = vec_heads(c.d_h, c.rotary, sizeof(T), {c.q, c.k, c.g, c.q_out, c.k_pages, c.g_pages},
                             {c.q_pitch, c.k_pitch, c.g_pitch, (long long)c.H * c.m_pitch});
  // a block takes a whole row (its slot is looked up once), or, for few rows, as large a part
  // of one as keeps the SMs busy
  constexpr int EV = 16 / sizeof(T);
  const int most = ceil_div((long long)c.H * (vec ? c.m_pitch / EV : c.m_h), kThreads);
  const int want = ceil_div(8LL * serve_sm_count(), c.p.N);
  a.chunks = want < most ? want : most;
  const long long blocks = a.qk_blocks + (long long)c.p.N * a.chunks;
  if (blocks > (1ll << 31) - 1) return cudaErrorInvalidConfiguration;
  if (vec)
    c.layout == TG_ROPE_HALF ? cache_append_kernel<T, true, true><<<(unsigned)blocks, kThreads, 0, s>>>(a)
                             : cache_append_kernel<T, true, false><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  else
    cache_append_kernel<T, false, true><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

int serve_sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  const bool kept = dev >= 0 && dev < 64;
  int n = kept ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
  if (kept) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

size_t qk_backward_part_bytes(int d_h) { return (size_t)serve_sm_count() * kBwdPerSm * 2 * d_h * sizeof(float); }

cudaError_t launch_qk_forward(tg_dtype dt, const QkCall& c, cudaStream_t s) {
  return dt == TG_F32 ? forward_t<float>(c, s) : forward_t<__nv_bfloat16>(c, s);
}
cudaError_t launch_qk_backward(tg_dtype dt, const QkCall& c, cudaStream_t s) {
  return dt == TG_F32 ? backward_t<float>(c, s) : backward_t<__nv_bfloat16>(c, s);
}
cudaError_t launch_cache_append(tg_dtype dt, const AppendCall& c, cudaStream_t s) {
  return dt == TG_F32 ? append_t<float>(c, s) : append_t<__nv_bfloat16>(c, s);
}

}  // namespace tg

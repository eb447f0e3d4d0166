// TANGO aggregation of new tokens over a paged cache, CUDA-core kernels ("TANGO:
// Token-Aggregated Nonlinear Gating Operators ...", sec. 2.1 eq. 5 with sec. 2.2 eq. 6):
//   out_i = v_i [ sum_{j<=i} w_ij g_j ] / [ sum_{j<=i} w_ij + (i+1) e^{b - tau} ],
//   w_ij = e^{tau (q_i . k_j - 1)}.
// The shift by tau cancels; with unit vectors and tau <= 20 every weight lies in
// [e^-40, 1] and the sums of key ranges simply add, so no running maximum is kept.  A row whose
// weights say that its vectors are not unit ones is flagged (not_unit).
//
// Rows are taken in tiles of R (1, 2, 4 or 8) new tokens of one sequence.
//   paged_scores_kernel  one thread per cached key: its R dot products (q in shared memory),
//       weights in f32 to scratch [tile][head][key][R], and the key span's weight sums.
//   paged_gates_kernel   per (tile, head, up to 512 or 1024 columns, span of keys): the weighted
//       sum over the span's gate rows.  Bound by HBM for few rows: each gate is read once per
//       tile; tiles of one chunk stand next to each other in the grid and share the gates in
//       L2.  4 keys of a thread are multiplied while the next 4 are on their way, rows in pairs
//       through f32x2 arithmetic.  The spans of one output are joined, 16 neighbours first, by
//       the block of them that finishes last, in the spans' order (no order-dependent sums).
// 71 new tokens of 4 sequences over 2,297 cached ones, fp32, 2 x 4,747 gates in rows that are not
// 16-byte aligned: 47 us, bound by the latency of 4-byte loads and of two kernels in a row (the
// bytes alone would take 14 us).  Whole chunks are bound by the latency of L2 and of a block's start:
// 201 rows over 870 keys, 16 x 1,780 gates: 320 us, 28 TFLOP/s (660 us without the second
// batch of loads and with single f32 arithmetic).  Tiles of 16 rows halve the reads but leave
// 12 to 16 warps on an SM: 352 to 412 us there.  A ring of asynchronous copies in shared memory
// instead of registers: 351 us there, 2 to 3 % faster for few aligned rows, 117 -> 156 us for
// unaligned single rows.
// Keys past a row's own position are selected away, not multiplied by zero, so gates of
// later tokens and of unused slots may be NaN.
#include <type_traits>

#include "tg_common.cuh"
#include "tg_kernels.h"
#include "tg_paged.cuh"
#include "tg_ptx.cuh"
#include "tg_serve.h"

namespace tg {
namespace {

constexpr int kKeysBlk = 128;   // keys of a scores block
constexpr int kVT = 128;        // column vectors of a gates block, half of them for narrow heads

template <typename T>
struct SimtArgs {
  PagedBatch p;
  int H, d_h, m_h, m_pitch;
  int h0, tile0;                 // the pass: heads from h0, tiles from tile0 (the grid says how many)
  int key_pitch;                 // keys of a (tile, head) in the weights scratch
  int spans;                     // score spans: ceil(max_len / kKeysBlk)
  int span_keys, gspans;         // keys of a gates block's span; spans of the longest sequence
  int chunks;                    // column chunks of a head
  int counts;                    // counters of a chunk's spans: the groups', then each group's
  float s;
  const float* tau;
  const float* null_bias;
  long long v_pitch;
  const T *q, *v;
  T* out;
  const T *k_pages, *g_pages;
  // scratch, by the tile and head of the pass
  float* w;     // [tile][head][key][R]
  float* den;   // [tile][head][span][R]
  float* part;  // [tile][head][chunk][gspan][R][VT EV]
  int* count;   // [tile][head][chunk][counts]: spans or groups that are done
};

// grid (tiles, heads, spans), 128 threads.
template <typename T, int R, bool kVec>
__global__ void __launch_bounds__(kKeysBlk) paged_scores_kernel(const SimtArgs<T> a) {
  __shared__ __align__(16) float qs[R][128];
  __shared__ float red[kKeysBlk / 32][R];
  const int tile = a.tile0 + blockIdx.x, hl = blockIdx.y, head = a.h0 + hl, t = threadIdx.x;
  const size_t th = (size_t)blockIdx.x * gridDim.y + hl;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.z == 0)
    for (int c = t; c < a.chunks * a.counts; c += kKeysBlk) a.count[th * a.chunks * a.counts + c] = 0;
  const TileRef tr = find_tile<R>(a.p, tile, hl == 0 && blockIdx.z == 0);
  const int vis = tr.pos0 + tr.n;  // keys that the last row sees
  if (tr.n == 0 || (int)blockIdx.z * kKeysBlk >= vis) return;
  for (int i = t; i < tr.n * a.d_h; i += kKeysBlk) {
    const int r = i / a.d_h, c = i - r * a.d_h;
    qs[r][c] = io<T>::ld(a.q + ((size_t)(tr.row0 + r) * a.H + head) * a.d_h + c);
  }
  __syncthreads();
  const int key = blockIdx.z * kKeysBlk + t;
  const float tau = head_tau(a.tau, a.s, head, a.p.err, kKernPaged);
  float x[R] = {};
  if (key < vis) {
    const int pi = key / a.p.page_size, pg = paged_page(a.p, tr.b, pi);
    if (pg >= 0) {
      const T* kp = a.k_pages + (((size_t)pg * a.p.page_size + (key - pi * a.p.page_size)) * a.H + head) * a.d_h;
      if (kVec) {
        constexpr int EV = 16 / sizeof(T);
#pragma unroll 4
        for (int c = 0; c < a.d_h; c += EV) {
          const uint4 u = *reinterpret_cast<const uint4*>(kp + c);
          const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
              if (sizeof(T) == 2) {
                x[r] = fmaf(ptx::bf16lo(uu[e]), qs[r][c + 2 * e], x[r]);
                x[r] = fmaf(ptx::bf16hi(uu[e]), qs[r][c + 2 * e + 1], x[r]);
              } else {
                x[r] = fmaf(__uint_as_float(uu[e]), qs[r][c + e], x[r]);
              }
            }
          }
        }
      } else {
        for (int c = 0; c < a.d_h; ++c) {
          const float kv = io<T>::ld(kp + c);
#pragma unroll
          for (int r = 0; r < R; ++r) x[r] = fmaf(kv, qs[r][c], x[r]);
        }
      }
    }
  }
  float* dst = a.w + (th * a.key_pitch + key) * R;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float w = r < tr.n && key <= tr.pos0 + r ? exp2f(tau * kLog2e * (x[r] - 1.f)) : 0.f;
    if (key < vis) dst[r] = w;
    float s = w;
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((t & 31) == 0) red[t / 32][r] = s;
  }
  __syncthreads();
  if (t < R) {
    float s = 0.f;
    for (int i = 0; i < kKeysBlk / 32; ++i) s += red[i][t];
    a.den[(th * a.spans + blockIdx.z) * R + t] = s;
    const int k0 = blockIdx.z * kKeysBlk;
    if (t < tr.n && not_unit(s, min(k0 + kKeysBlk, tr.pos0 + t + 1) - k0)) record_error(a.p.err, kErrValue | kKernPaged);
  }
}

template <typename T> struct Cols;
template <> struct Cols<float> {
  static constexpr int EV = 4;
  static __device__ __forceinline__ void get(const uint4& u, float* f) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y); f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
};
template <> struct Cols<__nv_bfloat16> {
  static constexpr int EV = 8;
  static __device__ __forceinline__ void get(const uint4& u, float* f) {
    f[0] = ptx::bf16lo(u.x); f[1] = ptx::bf16hi(u.x); f[2] = ptx::bf16lo(u.y); f[3] = ptx::bf16hi(u.y);
    f[4] = ptx::bf16lo(u.z); f[5] = ptx::bf16hi(u.z); f[6] = ptx::bf16lo(u.w); f[7] = ptx::bf16hi(u.w);
  }
};

constexpr int kSpanMax = 512;
// Spans whose sums are joined first.  20 rows over 8,000 keys (125 spans, 4 x 256 gates) take
// 56 us, against 103 where one block adds all spans up row by row.
constexpr int kJoin = 16;

// grid (tiles, chunks * heads, gspans), VT threads; a thread owns EV columns of R rows: EV
// neighbours (one 16-byte load) where the gates' rows are 16-byte aligned, else every VT-th
// (so that a warp's loads are neighbours).
// At least 5 blocks on an SM (3 for bf16, whose threads hold twice the columns): with the 110
// registers that the compiler would take there are 4, and 201 rows over 870 keys take 466 us
// instead of 339 (6 blocks, with spills: 354).
template <typename T, int R, bool kVec, int VT>
__global__ void __launch_bounds__(VT, (sizeof(T) == 4 ? 5 : 3) * (128 / VT)) paged_gates_kernel(const SimtArgs<T> a) {
  constexpr int EV = Cols<T>::EV;
  constexpr int U = R == 1 ? 8 : 4;  // keys of a batch of loads
  __shared__ __align__(16) int tok[kSpanMax + 3 * U];
  __shared__ __align__(16) float ws[(kSpanMax + U) * R];
  __shared__ float dinv[R];
  __shared__ int last;
  const int tile = a.tile0 + blockIdx.x, hl = blockIdx.y / a.chunks, chunk = blockIdx.y - hl * a.chunks;
  const int head = a.h0 + hl;
  const int heads = gridDim.y / a.chunks, t = threadIdx.x;
  // launched while the scores kernel still runs: what follows up to the wait is not its work
  const TileRef tr = find_tile<R>(a.p, tile, false);
  const int vis = max(0, tr.pos0 + tr.n), k0 = blockIdx.z * a.span_keys;
  const int nsp = max(1, (vis + a.span_keys - 1) / a.span_keys);
  const bool mine = tr.n > 0 && (int)blockIdx.z < nsp;
  const int nk = mine ? min(a.span_keys, vis - k0) : 0;
  const size_t th = (size_t)blockIdx.x * heads + hl;
  // the span's tokens, and some more for the loads that run ahead (any token of the pool does)
  bool bad = false;
  for (int i = t; i < nk + 3 * U; i += VT) {
    const int key = k0 + i, pi = key / a.p.page_size, pg = i < nk ? paged_page(a.p, tr.b, pi) : 0;
    bad |= pg < 0;
    tok[i] = i >= nk ? 0 : pg < 0 ? -1 : pg * a.p.page_size + (key - pi * a.p.page_size);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!mine) return;
  const float* w = a.w + (th * a.key_pitch + k0) * R;
  // weights are not negative; -1 stands for a key to be skipped
  for (int i = t; i < (nk + U) * R; i += VT) ws[i] = i < nk * R ? __ldcg(w + i) : -1.f;
  bad = __syncthreads_or(bad);
  if (bad) {  // pages outside the pool: their gates count as zeros
    for (int i = t; i < nk; i += VT)
      if (tok[i] < 0) {
        tok[i] = 0;
        for (int r = 0; r < R; ++r) ws[i * R + r] = -1.f;
      }
    __syncthreads();
  }
  const int c0 = chunk * VT * EV + (kVec ? t * EV : t);  // first column of the head
  constexpr int cs = kVec ? 1 : VT;                      // and the step to the next
  const bool live = c0 < a.m_h;
  constexpr int P = R > 1 ? 2 : 1;  // rows of an accumulator: pairs go through f32x2 arithmetic
  uint64_t acc2[R / P][EV];
  float acc[R][EV];
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int e = 0; e < EV; ++e) acc[r][e] = 0.f, acc2[r / P][e] = 0;
  }
  const size_t row_elems = (size_t)a.H * a.m_pitch;
  const T* gcol = a.g_pages + (size_t)head * a.m_pitch + c0;
  // gates of U keys as loaded: one vector each, or EV single values
  using Raw = typename std::conditional<kVec, uint4, T[EV]>::type;
  auto load = [&](int i, Raw (&g)[U]) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const T* src = gcol + (size_t)(unsigned)tok[i + j] * row_elems;
      if constexpr (kVec) {
        g[j] = ptx::ld_global_v4(src);
      } else {
#pragma unroll
        for (int e = 0; e < EV; ++e) g[j][e] = e == 0 || c0 + e * cs < a.m_h ? src[e * cs] : T(0.f);
      }
    }
  };
  auto widen = [&](const Raw& g, float (&f)[EV]) {
    if constexpr (kVec) {
      Cols<T>::get(g, f);
    } else {
#pragma unroll
      for (int e = 0; e < EV; ++e) f[e] = io<T>::ld(&g[e]);
    }
  };
  // keys up to `all` are seen by every row of the tile, the last ones by some
  const int all = bad ? 0 : min(nk, max(0, tr.pos0 + 1 - k0));
  auto add = [&](int i, const Raw (&g)[U]) {
    if (i + U <= all) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float f[EV];
        widen(g[j], f);
        if constexpr (R == 1) {
          const float wr = ws[i + j];
#pragma unroll
          for (int e = 0; e < EV; ++e) acc[0][e] = fmaf(wr, f[e], acc[0][e]);
        } else {
          uint64_t ff[EV];
#pragma unroll
          for (int e = 0; e < EV; ++e) ff[e] = ptx::f32x2_pack(f[e], f[e]);
#pragma unroll
          for (int r = 0; r < R / 2; ++r) {
            const uint64_t wr = *reinterpret_cast<const uint64_t*>(&ws[(i + j) * R + 2 * r]);
#pragma unroll
            for (int e = 0; e < EV; ++e) acc2[r][e] = ptx::fma_f32x2(wr, ff[e], acc2[r][e]);
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float f[EV];
        widen(g[j], f);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float wr = ws[(i + j) * R + r];
          if (!(wr < 0.f) && k0 + i + j <= tr.pos0 + r) {
#pragma unroll
            for (int e = 0; e < EV; ++e) {
              if constexpr (R == 1) {
                acc[0][e] = fmaf(wr, f[e], acc[0][e]);
              } else {
                float x[2];
                ptx::f32x2_unpack(acc2[r / 2][e], x[0], x[1]);
                x[r % 2] = fmaf(wr, f[e], x[r % 2]);
                acc2[r / 2][e] = ptx::f32x2_pack(x[0], x[1]);
              }
            }
          }
        }
      }
    }
  };
  if (live && nk > 0) {
    Raw ga[U], gb[U];
    load(0, ga);
#pragma unroll 1
    for (int i = 0; i < nk; i += 2 * U) {
      load(i + U, gb);
      add(i, ga);
      load(i + 2 * U, ga);
      if (i + U < nk) add(i + U, gb);
    }
  }
  if constexpr (R > 1) {
#pragma unroll
    for (int r = 0; r < R; r += 2) {
#pragma unroll
      for (int e = 0; e < EV; ++e) ptx::f32x2_unpack(acc2[r / 2][e], acc[r][e], acc[r + 1][e]);
    }
  }
  if (nsp > 1) {
    // This span's sums go to scratch; the block that finishes last of kJoin neighbouring spans
    // adds theirs up in order, and the last of those blocks the groups' sums.
    constexpr size_t kSums = (size_t)R * VT * EV;
    float* base = a.part + (th * a.chunks + chunk) * a.gspans * kSums + t;
    int* count = a.count + (th * a.chunks + chunk) * a.counts;
    auto put = [&](int z) {
      if (live) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (r >= tr.n) break;
#pragma unroll
          for (int e = 0; e < EV; ++e) __stcg(base + z * kSums + (r * EV + e) * VT, acc[r][e]);
        }
      }
    };
    auto last_of = [&](int* c, int n) {
      __threadfence();
      __syncthreads();
      if (t == 0) last = atomicAdd(c, 1) == n - 1;
      __syncthreads();
      if (last) __threadfence();
      return last != 0;
    };
    auto add_up = [&](int z, int end, int step) {
      if (!live) return;
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int e = 0; e < EV; ++e) acc[r][e] = 0.f;
      }
      if (tr.n == R) {  // full tiles: 32 to 64 loads of a thread in flight
#pragma unroll(R >= 4 ? 2 : 8 / R)
        for (int i = z; i < end; i += step) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int e = 0; e < EV; ++e) acc[r][e] += __ldcg(base + i * kSums + (r * EV + e) * VT);
          }
        }
        return;
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= tr.n) break;
#pragma unroll 8
        for (int i = z; i < end; i += step) {
#pragma unroll
          for (int e = 0; e < EV; ++e) acc[r][e] += __ldcg(base + i * kSums + (r * EV + e) * VT);
        }
      }
    };
    const int z = blockIdx.z, z0 = z / kJoin * kJoin, z1 = min(nsp, z0 + kJoin);
    put(z);
    if (!last_of(count + 1 + z / kJoin, z1 - z0)) return;
    add_up(z0, z1, 1);
    if (nsp > kJoin) {
      put(z0);
      if (!last_of(count, (nsp + kJoin - 1) / kJoin)) return;
      add_up(0, nsp, kJoin);
    }
  }
  // denominators of the tile's rows: the spans' sums, and the null gate
  if (t < R) {
    const int pos = tr.pos0 + t, ns = (vis + kKeysBlk - 1) / kKeysBlk;
    float d = 0.f;
    for (int z = 0; z < ns; ++z) d += __ldcg(a.den + (th * a.spans + z) * R + t);
    if (a.null_bias && pos >= 0) {
      const float tau = head_tau(a.tau, a.s, head, a.p.err, kKernPaged);
      d += (float)(pos + 1) * expf(a.null_bias[head] - tau);
    }
    dinv[t] = t < tr.n && pos >= 0 ? 1.f / d : 0.f;
  }
  __syncthreads();
  if (!live) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r >= tr.n) break;
    const size_t row = tr.row0 + r, col = (size_t)head * a.m_pitch + c0;
#pragma unroll
    for (int e = 0; e < EV; ++e) {
      if (c0 + e * cs >= a.m_h) break;
      float y = tr.pos0 + r >= 0 ? acc[r][e] * dinv[r] : 0.f;
      if (a.v && tr.pos0 + r >= 0) y *= io<T>::ld(a.v + row * a.v_pitch + col + e * cs);
      io<T>::st(a.out + row * row_elems + col + e * cs, y);
    }
  }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr size_t kScratch = size_t(1) << 30;  // of a pass
// Where the call would run on the tensor cores but for a pointer that is not 16-byte aligned:
// no more than the tensor cores' own scratch, or 256 MB, so that aligned calls, whose scratch has
// to hold either path's, need not bring more.
constexpr size_t kScratchTwin = size_t(256) << 20;

struct SimtPlan {
  int VT, R, tiles, spans, span_keys, gspans, chunks, counts, key_pitch;
  int heads, pass_tiles;  // of a pass
  size_t w, den, part, count, total;
};

SimtPlan simt_plan(tg_dtype dt, const PagedCall& c) {
  SimtPlan l;
  const int EV = dt == TG_F32 ? 4 : 8;
  l.R = c.p.max_new >= 5 ? 8 : c.p.max_new >= 3 ? 4 : c.p.max_new;
  l.tiles = c.p.N / l.R + c.p.B;
  l.spans = ceil_div(c.p.max_len, kKeysBlk);
  l.key_pitch = l.spans * kKeysBlk;
  // heads of up to 64 vectors: a wider block's other threads would idle (1,500 rows over 3,000
  // keys, 4 x 256 gates, fp32: 370 -> 294 us)
  l.VT = c.m_h <= kVT / 2 * EV ? kVT / 2 : kVT;
  l.chunks = ceil_div(c.m_h, l.VT * EV);
  // spans of 512 keys, shorter where the grid would hold fewer than 20 blocks per SM (a block
  // starts with some 4 us of dependent look-ups and its sums are written and read again: over
  // batches of 1 to 276 new rows, fp32, 147 us on average against 153 with 32; with 16 the
  // 71-row batch takes 56 us instead of 46)
  l.span_keys = kSpanMax;
  while (l.span_keys > 64 &&
         (long long)l.tiles * c.H * l.chunks * ceil_div(c.p.max_len, l.span_keys) < 20LL * serve_sm_count())
    l.span_keys /= 2;
  l.gspans = ceil_div(c.p.max_len, l.span_keys);
  l.counts = 1 + ceil_div(l.gspans, kJoin);
  // A pass takes as many heads as fit its scratch, or, where one does not, as many tiles of one
  // head; never less than one tile of one head (4 R bytes a key for the weights, 4 R / span_keys
  // bytes a key and gate for the sums: 1.6 % of an fp32 cache's own bytes in spans of 512).
  const size_t per = (size_t)l.key_pitch * l.R * 4 + (size_t)l.spans * l.R * 4 +
                     (size_t)l.chunks * l.gspans * l.R * l.VT * EV * 4 + (size_t)l.chunks * l.counts * 4;
  size_t most = kScratch;
  if (paged_tc_takes(dt, c)) {
    const size_t tc = paged_tc_ws_bytes(c);
    most = tc < kScratchTwin ? kScratchTwin : tc < kScratch ? tc : kScratch;
  }
  const size_t fit = most / per;  // (tile, head) pairs
  l.heads = (int)(fit / l.tiles < 1 ? 1 : fit / l.tiles > (size_t)c.H ? (size_t)c.H : fit / l.tiles);
  l.pass_tiles = (int)(fit < 1 ? 1 : fit > (size_t)l.tiles ? (size_t)l.tiles : fit);
  const size_t th = (size_t)l.pass_tiles * l.heads;
  l.w = 0;
  l.den = l.w + align256(th * l.key_pitch * l.R * 4);
  l.part = l.den + align256(th * l.spans * l.R * 4);
  l.count = l.part + align256(th * l.chunks * l.gspans * l.R * l.VT * EV * 4);
  l.total = l.count + align256(th * l.chunks * l.counts * 4);
  return l;
}

template <typename T, int R>
cudaError_t run(const PagedCall& c, const SimtPlan& l, cudaStream_t s) {
  SimtArgs<T> a;
  a.p = c.p; a.H = c.H; a.d_h = c.d_h; a.m_h = c.m_h; a.m_pitch = c.m_pitch;
  a.key_pitch = l.key_pitch; a.spans = l.spans; a.span_keys = l.span_keys; a.gspans = l.gspans;
  a.chunks = l.chunks; a.counts = l.counts;
  a.s = c.s; a.tau = c.tau; a.null_bias = c.null_bias; a.v_pitch = c.v_pitch;
  a.q = static_cast<const T*>(c.q); a.v = static_cast<const T*>(c.v); a.out = static_cast<T*>(c.out);
  a.k_pages = static_cast<const T*>(c.k_pages); a.g_pages = static_cast<const T*>(c.g_pages);
  char* base = static_cast<char*>(c.ws);
  a.w = reinterpret_cast<float*>(base + l.w);
  a.den = reinterpret_cast<float*>(base + l.den);
  a.part = reinterpret_cast<float*>(base + l.part);
  a.count = reinterpret_cast<int*>(base + l.count);
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  const bool kvec = al(c.k_pages) && c.d_h * sizeof(T) % 16 == 0;
  // whole 16-byte vectors of a head: its last one may run into the pitch's padding, never
  // into the next head
  const bool gvec = al(c.g_pages) && c.m_pitch * sizeof(T) % 16 == 0;
  for (a.h0 = 0; a.h0 < c.H; a.h0 += l.heads) {
    for (a.tile0 = 0; a.tile0 < l.tiles; a.tile0 += l.pass_tiles) {
      const int heads = c.H - a.h0 < l.heads ? c.H - a.h0 : l.heads;
      const int tiles = l.tiles - a.tile0 < l.pass_tiles ? l.tiles - a.tile0 : l.pass_tiles;
      const dim3 gs(tiles, heads, l.spans), gg(tiles, heads * l.chunks, l.gspans);
      if (kvec) paged_scores_kernel<T, R, true><<<gs, kKeysBlk, 0, s>>>(a);
      else paged_scores_kernel<T, R, false><<<gs, kKeysBlk, 0, s>>>(a);
      cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = gg;
      cfg.blockDim = dim3(l.VT);
      cfg.stream = s;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (l.VT == kVT)
        e = gvec ? cudaLaunchKernelEx(&cfg, paged_gates_kernel<T, R, true, kVT>, a)
                 : cudaLaunchKernelEx(&cfg, paged_gates_kernel<T, R, false, kVT>, a);
      else
        e = gvec ? cudaLaunchKernelEx(&cfg, paged_gates_kernel<T, R, true, kVT / 2>, a)
                 : cudaLaunchKernelEx(&cfg, paged_gates_kernel<T, R, false, kVT / 2>, a);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

template <typename T>
cudaError_t run_t(const PagedCall& c, const SimtPlan& l, cudaStream_t s) {
  switch (l.R) {
    case 1: return run<T, 1>(c, l, s);
    case 2: return run<T, 2>(c, l, s);
    case 4: return run<T, 4>(c, l, s);
    default: return run<T, 8>(c, l, s);
  }
}

}  // namespace

bool paged_simt_takes(tg_dtype dt, const PagedCall& c) {
  const SimtPlan l = simt_plan(dt, c);  // (spans of gates are no more than spans of scores)
  return l.spans <= 65535 && (long long)c.H * l.chunks <= 65535;
}

size_t paged_simt_ws_bytes(tg_dtype dt, const PagedCall& c) { return simt_plan(dt, c).total; }

cudaError_t launch_paged_simt(tg_dtype dt, const PagedCall& c, cudaStream_t s) {
  const SimtPlan l = simt_plan(dt, c);
  return dt == TG_F32 ? run_t<float>(c, l, s) : run_t<__nv_bfloat16>(c, l, s);
}

}  // namespace tg

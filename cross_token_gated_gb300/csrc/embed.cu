// Token lookup with scaling, and the embedding's gradient by sorted tokens ("TANGO:
// Token-Aggregated Nonlinear Gating Operators ...", sec. 2.3: the tied token embedding).
//
//   out[n] = s E[id_n];   dE[v] = base[v] + s sum_{n: id_n = v} dout[n]
//
// Both are bound by HBM bandwidth: rows are read and written once.  The gradient sorts the tokens
// by id (a stable counting sort, so that the order of every sum is fixed), writes the rows of ids
// without tokens on the way, and sums the sorted rows of dout in fp32 in equal chunks, so that a
// frequent token loads no warp more than a rare one; sums that cross chunks are joined in order.
#include "tg_common.cuh"
#include "tg_ends.h"
#include "tg_ptx.cuh"
#include "tg_serve.h"

namespace tg {
namespace {

// A kernel's launch that may start while the one before it still runs; it waits itself.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------------------- lookup

// E values of 16 bytes times s, each rounded once.
__device__ __forceinline__ uint4 scaled(uint4 u, float s, float) {
  return make_uint4(__float_as_uint(__uint_as_float(u.x) * s), __float_as_uint(__uint_as_float(u.y) * s),
                    __float_as_uint(__uint_as_float(u.z) * s), __float_as_uint(__uint_as_float(u.w) * s));
}
__device__ __forceinline__ uint4 scaled(uint4 u, float s, __nv_bfloat16) {
  return make_uint4(ptx::pack_bf16x2(ptx::bf16lo(u.x) * s, ptx::bf16hi(u.x) * s),
                    ptx::pack_bf16x2(ptx::bf16lo(u.y) * s, ptx::bf16hi(u.y) * s),
                    ptx::pack_bf16x2(ptx::bf16lo(u.z) * s, ptx::bf16hi(u.z) * s),
                    ptx::pack_bf16x2(ptx::bf16lo(u.w) * s, ptx::bf16hi(u.w) * s));
}

// One warp per row, 16 bytes a lane (kVec) or single values.  A scale of 1 copies the bits.
template <typename T, bool kVec>
__global__ void __launch_bounds__(256) embed_lookup_kernel(const int* ids, const T* E, T* out, long long rows, int d,
                                                           int vocab, long long pitch, float scale, int pad,
                                                           unsigned* err) {
  constexpr int N = kVec ? 16 / (int)sizeof(T) : 1;
  const long long r = (long long)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (r >= rows) return;
  const int id = ids[r];
  const bool known = id >= 0 && id < vocab;
  if (!known && id != pad && lane == 0) record_error(err, kErrValue | kKernModel);
  const bool live = known && id != pad;
  const T* src = E + (long long)(live ? id : 0) * d;
  T* dst = out + r * pitch;
#pragma unroll 4
  for (int c = lane * N; c < d; c += 32 * N) {
    if constexpr (kVec) {
      const uint4 u = live ? *reinterpret_cast<const uint4*>(src + c) : make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(dst + c) = scale == 1.f ? u : scaled(u, scale, T());
    } else {
      if (!live) dst[c] = T(0.f);
      else if (scale == 1.f) dst[c] = src[c];
      else io<T>::st(dst + c, io<T>::ld(src + c) * scale);
    }
  }
}

// ------------------------------------------------------------------------------ sort

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kMaxSortRows = 1536;  // ids of a block: kSortWarps counters each in shared memory
constexpr int kAhead = 8;           // ids of a lane that are loaded at a time

struct SortArgs {
  const int* ids;
  int N, vocab, pad;
  int R;        // ids of a block
  int* order;   // [N] tokens by id, then by position
  int* sorted;  // [N] their ids
  int* start;   // [vocab] first entry of each id in order
  int* count;   // [vocab]
  // rows of ids without tokens: zeros, or base's
  const char* base;
  char* dE;
  long long row_bytes;
  int step;     // bytes of an access: 16 where rows are aligned, else an element
  unsigned* err;
};

// A row of dE for an id without tokens, by one warp.
__device__ __forceinline__ void empty_row(const SortArgs& a, int v, int lane) {
  const long long o = (long long)v * a.row_bytes;
  char* dst = a.dE + o;
  const char* src = a.base ? a.base + o : nullptr;
  if (a.step == 16) {
    for (long long b = lane * 16; b < a.row_bytes; b += 512)
      *reinterpret_cast<uint4*>(dst + b) = src ? *reinterpret_cast<const uint4*>(src + b) : make_uint4(0, 0, 0, 0);
  } else if (a.step == 4) {
    for (long long b = lane * 4; b < a.row_bytes; b += 128)
      *reinterpret_cast<unsigned*>(dst + b) = src ? *reinterpret_cast<const unsigned*>(src + b) : 0u;
  } else {
    for (long long b = lane * 2; b < a.row_bytes; b += 64)
      *reinterpret_cast<unsigned short*>(dst + b) = src ? *reinterpret_cast<const unsigned short*>(src + b) : 0;
  }
}

// Block b sorts the ids of [b R, (b + 1) R): every block reads all ids, so that it also knows how
// many lie below its own, and no block waits for another (the ids are a small part of dout, and
// stay in L2).  Warp w counts, and then places, the w-th share of the positions; a counter per
// (warp, id) keeps the order of positions.
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const SortArgs a) {
  extern __shared__ int cnt[];  // [kSortWarps][R]
  __shared__ int below_w[kSortWarps], scan_w[kSortWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int v0 = blockIdx.x * a.R, nr = min(a.R, a.vocab - v0);
  const int share = ((a.N + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int n0 = (int)min((long long)warp * share, (long long)a.N), n1 = (int)min((long long)n0 + share, (long long)a.N);
  int* mine = cnt + warp * a.R;
  let_next_start();
  for (int i = threadIdx.x; i < kSortWarps * a.R; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  int below = 0;
  bool bad = false;
  for (int n = n0; n < n1; n += 32 * kAhead) {
    int id[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) id[j] = n + 32 * j + lane < n1 ? a.ids[n + 32 * j + lane] : a.pad;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const bool live = id[j] != a.pad && id[j] >= 0 && id[j] < a.vocab;
      bad |= !live && id[j] != a.pad;
      below += live && id[j] < v0;
      const bool in = live && id[j] >= v0 && id[j] < v0 + nr;
      if (__ballot_sync(0xffffffffu, in) == 0) continue;
      const unsigned same = __match_any_sync(0xffffffffu, in ? id[j] - v0 : -1);
      if (in && (same & ((1u << lane) - 1)) == 0) mine[id[j] - v0] += __popc(same);
      __syncwarp();
    }
  }
  if (blockIdx.x == 0 && bad) record_error(a.err, kErrValue | kKernModel);
  below = __reduce_add_sync(0xffffffffu, below);
  if (lane == 0) below_w[warp] = below;
  __syncthreads();
  // counters become places: ids in order, of one id the warps in order
  int run = 0;
  for (int w = 0; w < kSortWarps; ++w) run += below_w[w];
  for (int r0 = 0; r0 < nr; r0 += kSortThreads) {
    const int r = r0 + threadIdx.x;
    int sum = 0;
    if (r < nr)
      for (int w = 0; w < kSortWarps; ++w) sum += cnt[w * a.R + r];
    int incl = sum;
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) scan_w[warp] = incl;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) before += scan_w[w];
      total += scan_w[w];
    }
    if (r < nr) {
      int at = run + before + incl - sum;
      a.start[v0 + r] = at;
      a.count[v0 + r] = sum;
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = cnt[w * a.R + r];
        cnt[w * a.R + r] = at;
        at += c;
      }
    }
    run += total;
    __syncthreads();
  }
  // rows without tokens: the last warp's place is the row's end, the first one's its start
  if (a.base != a.dE)
    for (int r = warp; r < nr; r += kSortWarps)
      if (a.count[v0 + r] == 0) empty_row(a, v0 + r, lane);
  for (int n = n0; n < n1; n += 32 * kAhead) {
    int id[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) id[j] = n + 32 * j + lane < n1 ? a.ids[n + 32 * j + lane] : a.pad;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const bool in = id[j] != a.pad && id[j] >= v0 && id[j] < v0 + nr;
      if (__ballot_sync(0xffffffffu, in) == 0) continue;
      const unsigned same = __match_any_sync(0xffffffffu, in ? id[j] - v0 : -1);
      const unsigned earlier = same & ((1u << lane) - 1);
      const int at = in ? mine[id[j] - v0] : 0;
      if (in) {
        a.order[at + __popc(earlier)] = n + 32 * j + lane;
        a.sorted[at + __popc(earlier)] = id[j];
      }
      __syncwarp();
      if (in && earlier == 0) mine[id[j] - v0] = at + __popc(same);
      __syncwarp();
    }
  }
}

// ------------------------------------------------------------------------------- sums

constexpr int kChunk = 32;  // sorted tokens of a warp

template <typename T> struct Wide;  // 16 bytes of T
template <> struct Wide<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void add(const uint4& u, float* f) {
    f[0] += __uint_as_float(u.x); f[1] += __uint_as_float(u.y); f[2] += __uint_as_float(u.z); f[3] += __uint_as_float(u.w);
  }
};
template <> struct Wide<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void add(const uint4& u, float* f) {
    f[0] += ptx::bf16lo(u.x); f[1] += ptx::bf16hi(u.x); f[2] += ptx::bf16lo(u.y); f[3] += ptx::bf16hi(u.y);
    f[4] += ptx::bf16lo(u.z); f[5] += ptx::bf16hi(u.z); f[6] += ptx::bf16lo(u.w); f[7] += ptx::bf16hi(u.w);
  }
};

template <typename T, typename G>
struct SumArgs {
  const int *order, *sorted, *start, *count;
  const T* dout;
  const G* base;
  G* dE;
  float* part;      // [2 chunks][part_pitch]: sums of a chunk's first and last id that other chunks go on with
  int d, vocab, part_pitch;
  long long pitch;
  float scale;
};

// dst = base + scale f, E values at a multiple of E.
template <int E>
__device__ __forceinline__ void finish_vec(float* dst, const float* f, float scale, const float* base) {
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    const float4 b = base ? *reinterpret_cast<const float4*>(base + e) : make_float4(0, 0, 0, 0);
    *reinterpret_cast<float4*>(dst + e) = make_float4(fmaf(f[e], scale, b.x), fmaf(f[e + 1], scale, b.y),
                                                      fmaf(f[e + 2], scale, b.z), fmaf(f[e + 3], scale, b.w));
  }
}
template <int E>
__device__ __forceinline__ void finish_vec(__nv_bfloat16* dst, const float* f, float scale, const __nv_bfloat16* base) {
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    const uint2 b = base ? *reinterpret_cast<const uint2*>(base + e) : make_uint2(0, 0);
    *reinterpret_cast<uint2*>(dst + e) =
        make_uint2(ptx::pack_bf16x2(fmaf(f[e], scale, ptx::bf16lo(b.x)), fmaf(f[e + 1], scale, ptx::bf16hi(b.x))),
                   ptx::pack_bf16x2(fmaf(f[e + 2], scale, ptx::bf16lo(b.y)), fmaf(f[e + 3], scale, ptx::bf16hi(b.y))));
  }
}

// A warp sums the tokens of one chunk over a tile of columns: lane l holds 2 vectors (kVec), or 4
// single columns.  An id that begins and ends in the chunk is finished here; of one that goes past
// an end the sum is kept in part.
template <typename T, typename G, bool kVec>
__global__ void __launch_bounds__(256) embed_sum_kernel(const SumArgs<T, G> a) {
  constexpr int E = kVec ? Wide<T>::E : 1, NV = kVec ? 2 : 4, kRows = 8;
  const int lane = threadIdx.x & 31, q = blockIdx.x * 8 + threadIdx.x / 32, p0 = q * kChunk;
  wait_for_previous();
  let_next_start();
  const int M = a.start[a.vocab - 1] + a.count[a.vocab - 1];
  if (p0 >= M) return;
  const int n = min(kChunk, M - p0);
  const int token = lane < n ? a.order[p0 + lane] : 0, id = lane < n ? a.sorted[p0 + lane] : -1;
  const int before = p0 > 0 ? a.sorted[p0 - 1] : -1, after = p0 + kChunk < M ? a.sorted[p0 + kChunk] : -1;
  for (int c0 = blockIdx.y * 32 * NV * E; c0 < a.d; c0 += gridDim.y * 32 * NV * E) {
    float acc[NV * E] = {};
    for (int i0 = 0; i0 < n; i0 += kRows) {
      uint4 u[kVec ? kRows : 1][NV];
      float f[kVec ? 1 : kRows][NV];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const T* src = a.dout + __shfl_sync(0xffffffffu, token, i0 + i) * a.pitch;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int c = c0 + (k * 32 + lane) * E;
          const bool live = i0 + i < n && c < a.d;
          if constexpr (kVec) u[i][k] = live ? *reinterpret_cast<const uint4*>(src + c) : make_uint4(0, 0, 0, 0);
          else f[i][k] = live ? io<T>::ld(src + c) : 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (i0 + i >= n) break;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          if constexpr (kVec) Wide<T>::add(u[i][k], acc + k * E);
          else acc[k] += f[i][k];
        }
        const int v = __shfl_sync(0xffffffffu, id, i0 + i);
        const bool last = i0 + i == n - 1;
        if (!last && v == __shfl_sync(0xffffffffu, id, (i0 + i + 1) & 31)) continue;
        const bool goes_on = last && v == after, came_in = v == before;
        // (a chunk of one id that does both counts as its first)
        float* kept = goes_on || came_in ? a.part + (size_t)(2 * q + (came_in ? 0 : 1)) * a.part_pitch : nullptr;
        const long long o = (long long)v * a.d;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int c = c0 + (k * 32 + lane) * E;
          float* f = acc + k * E;
          if (c < a.d) {
            if constexpr (kVec) {
              if (kept) {
#pragma unroll
                for (int e = 0; e < E; e += 4)
                  *reinterpret_cast<float4*>(kept + c + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
              } else {
                finish_vec<E>(a.dE + o + c, f, a.scale, a.base ? a.base + o + c : nullptr);
              }
            } else {
              if (kept) kept[c] = *f;
              else io<G>::st(a.dE + o + c, fmaf(*f, a.scale, a.base ? io<G>::ld(a.base + o + c) : 0.f));
            }
          }
#pragma unroll
          for (int e = 0; e < E; ++e) f[e] = 0.f;
        }
      }
    }
  }
}

// Joins the sums of an id that goes past the end of chunk q - 1, if it began there: the last sum of
// that chunk and the first ones of those that follow.  8 warps take consecutive shares of them
// over 128 columns.
template <typename T, typename G>
__global__ void __launch_bounds__(256) embed_join_kernel(const SumArgs<T, G> a) {
  __shared__ float4 sums[8][32];
  const int q = blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  wait_for_previous();
  const int M = a.start[a.vocab - 1] + a.count[a.vocab - 1];
  if (q * kChunk >= M) return;
  const int v = a.sorted[q * kChunk];
  if (a.sorted[q * kChunk - 1] != v) return;
  const int s = a.start[v], last = (s + a.count[v] - 1) / kChunk;
  if (s / kChunk != q - 1) return;
  const int parts = last - q + 2, share = (parts + 7) / 8, i1 = min(parts, (warp + 1) * share);
  const int c = (blockIdx.y * 32 + lane) * 4;
  float4 t = make_float4(0, 0, 0, 0);
  if (c < a.d) {
#pragma unroll 8
    for (int i = warp * share; i < i1; ++i) {
      const size_t row = i == 0 ? 2 * (q - 1) + 1 : 2 * (size_t)(q - 1 + i);
      const float4 x = __ldcg(reinterpret_cast<const float4*>(a.part + row * a.part_pitch + c));
      t.x += x.x; t.y += x.y; t.z += x.z; t.w += x.w;
    }
  }
  sums[warp][lane] = t;
  __syncthreads();
  if (warp != 0) return;
  for (int w = 1; w < 8; ++w) {
    const float4 x = sums[w][lane];
    t.x += x.x; t.y += x.y; t.z += x.z; t.w += x.w;
  }
  const float f[4] = {t.x, t.y, t.z, t.w};
  const long long o = (long long)v * a.d;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c + e < a.d) io<G>::st(a.dE + o + c + e, fmaf(f[e], a.scale, a.base ? io<G>::ld(a.base + o + c + e) : 0.f));
}

// Ids of a sorting block: one block per SM, as far as the counters fit.
int sort_rows(int vocab) {
  const int r = ceil_div(vocab, serve_sm_count());
  return r < kMaxSortRows ? r : kMaxSortRows;
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

struct EmbedWs {
  size_t order, sorted, start, count, part, total;
  int part_pitch;
};
EmbedWs embed_ws(const EmbedCall& c) {
  EmbedWs w;
  const size_t tokens = up256((size_t)c.rows * 4), ids = up256((size_t)c.vocab * 4);
  w.part_pitch = (c.d + 3) / 4 * 4;
  w.order = 0;
  w.sorted = tokens;
  w.start = 2 * tokens;
  w.count = w.start + ids;
  w.part = w.count + ids;
  w.total = w.part + up256((size_t)ceil_div(c.rows, kChunk) * 2 * w.part_pitch * 4);
  return w;
}

template <typename T, typename G>
cudaError_t sums(const EmbedCall& c, const SortArgs& t, const EmbedWs& w, cudaStream_t s) {
  SumArgs<T, G> a;
  a.order = t.order; a.sorted = t.sorted; a.start = t.start; a.count = t.count;
  a.dout = static_cast<const T*>(c.dout); a.base = static_cast<const G*>(c.base); a.dE = static_cast<G*>(c.dE);
  a.part = reinterpret_cast<float*>(static_cast<char*>(c.ws) + w.part);
  a.d = c.d; a.vocab = c.vocab; a.part_pitch = w.part_pitch; a.pitch = c.pitch; a.scale = c.scale;
  const int chunks = ceil_div(c.rows, kChunk);
  const bool vec = c.d % Wide<T>::E == 0 && c.pitch % Wide<T>::E == 0 && aligned16(c.dout) && aligned16(c.base) &&
                   aligned16(c.dE);
  const int tile = vec ? 64 * Wide<T>::E : 128, tiles = ceil_div(c.d, tile);
  const dim3 grid(ceil_div(chunks, 8), tiles < 65535 ? tiles : 65535);
  cudaError_t e = vec ? launch_early(embed_sum_kernel<T, G, true>, grid, 256, s, a)
                      : launch_early(embed_sum_kernel<T, G, false>, grid, 256, s, a);
  if (e != cudaSuccess || chunks < 2) return e;
  return launch_early(embed_join_kernel<T, G>, dim3(chunks - 1, ceil_div(c.d, 128)), 256, s, a);
}

template <typename T>
cudaError_t lookup(const EmbedCall& c, cudaStream_t s) {
  const T* E = static_cast<const T*>(c.E);
  T* out = static_cast<T*>(c.out);
  constexpr int N = 16 / sizeof(T);
  const unsigned blocks = (unsigned)((c.rows + 7) / 8);
  const auto kernel = c.d % N == 0 && c.pitch % N == 0 && aligned16(c.E) && aligned16(c.out) ? embed_lookup_kernel<T, true>
                                                                                         : embed_lookup_kernel<T, false>;
  kernel<<<blocks, 256, 0, s>>>(c.ids, E, out, c.rows, c.d, c.vocab, c.pitch, c.scale, c.pad_id, c.err);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_embed_lookup(const EmbedCall& c, cudaStream_t s) {
  return c.dtype == TG_F32 ? lookup<float>(c, s) : lookup<__nv_bfloat16>(c, s);
}

size_t embed_backward_ws_bytes(const EmbedCall& c) { return embed_ws(c).total; }

cudaError_t launch_embed_backward(const EmbedCall& c, cudaStream_t s) {
  const EmbedWs w = embed_ws(c);
  char* ws = static_cast<char*>(c.ws);
  const int gs = c.grad_dtype == TG_F32 ? 4 : 2;
  SortArgs a;
  a.ids = c.ids; a.N = (int)c.rows; a.vocab = c.vocab; a.pad = c.pad_id;
  a.R = sort_rows(c.vocab);
  a.order = reinterpret_cast<int*>(ws + w.order);
  a.sorted = reinterpret_cast<int*>(ws + w.sorted);
  a.start = reinterpret_cast<int*>(ws + w.start);
  a.count = reinterpret_cast<int*>(ws + w.count);
  a.base = static_cast<const char*>(c.base); a.dE = static_cast<char*>(c.dE);
  a.row_bytes = (long long)c.d * gs;
  a.step = a.row_bytes % 16 == 0 && aligned16(c.base) && aligned16(c.dE) ? 16 : gs;
  a.err = c.err;
  const size_t smem = (size_t)kSortWarps * a.R * 4;
  cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSortWarps * kMaxSortRows * 4);
  if (e != cudaSuccess) return e;
  embed_sort_kernel<<<ceil_div(c.vocab, a.R), kSortThreads, smem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || c.rows == 0) return e;
  using bf16 = __nv_bfloat16;
  if (c.dtype == TG_F32)
    return c.grad_dtype == TG_F32 ? sums<float, float>(c, a, w, s) : sums<float, bf16>(c, a, w, s);
  return c.grad_dtype == TG_F32 ? sums<bf16, float>(c, a, w, s) : sums<bf16, bf16>(c, a, w, s);
}

}  // namespace tg

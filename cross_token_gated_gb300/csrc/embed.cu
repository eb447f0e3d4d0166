// Token lookup with scaling, and the embedding's gradient by sorted tokens ("TANGO:
// Token-Aggregated Nonlinear Gating Operators ...", sec. 2.3: the tied token embedding).
//
//   out[n] = s E[id_n];   dE[v] = base[v] + s sum_{n: id_n = v} dout[n]
//
// Both are bound by HBM bandwidth: rows are read and written once.  The gradient sorts the tokens
// by id (a stable counting sort, so that the order of every sum is fixed) and sums the sorted rows of
// dout in fp32 in equal chunks, so that a frequent token loads no warp more than a rare one; sums
// that cross chunks are joined in order by the warp that comes last.  Where a token's chunks begin
// follows from the other ids, from the number of SMs (the sort's order) and from the alignment (the
// chunks' size), and so do the last bits of its sum.  The rows of ids without tokens are written by the
// same launch.
//
// 16,384 tokens of 512 bf16 values into 32,768 fp32 rows: 25 us (floor 12.4), most of it the sums,
// whose first loads wait for order, row and neighbour in a row.  5,003 fp32 tokens of 768 onto a
// base: 51 us (floor 32), most of it the copy of the base.
#include "tg_common.cuh"
#include "tg_ends.h"
#include "tg_ptx.cuh"
#include "tg_serve.h"
#include "tg_vec.cuh"

namespace tg {
namespace {

// ---------------------------------------------------------------------------- lookup

// A vector's values times s, each rounded once.
template <typename T>
__device__ __forceinline__ uint4 scaled(const uint4& u, float s) {
  float f[Vec16<T>::E];
  Vec16<T>::unpack(u, f);
#pragma unroll
  for (int e = 0; e < Vec16<T>::E; ++e) f[e] *= s;
  return Vec16<T>::pack(f);
}

// One warp per row, 16 bytes a lane (kVec) or single values.  A scale of 1 copies the bits.
template <typename T, bool kVec>
__global__ void __launch_bounds__(256) embed_lookup_kernel(const int* ids, const T* E, T* out, long long rows, int d,
                                                           int vocab, long long pitch, float scale, int pad,
                                                           bool padded, unsigned* err) {
  constexpr int N = kVec ? 16 / (int)sizeof(T) : 1;
  const long long r = (long long)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (r >= rows) return;
  const int id = ids[r];
  const bool known = id >= 0 && id < vocab, none = padded && id == pad;
  if (!known && !none && lane == 0) record_error(err, kErrValue | kKernModel);
  const bool live = known && !none;
  const T* src = E + (long long)(live ? id : 0) * d;
  T* dst = out + r * pitch;
#pragma unroll 4
  for (int c = lane * N; c < d; c += 32 * N) {
    if constexpr (kVec) {
      const uint4 u = live ? *reinterpret_cast<const uint4*>(src + c) : make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(dst + c) = scale == 1.f || !live ? u : scaled<T>(u, scale);
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
constexpr int kAhead = 16;          // ids of a lane that are loaded at a time
constexpr int kOffsetBits = 21;     // of a queue entry: the position; the id's number takes 11
constexpr int kSortSmem = 224 * 1024;

struct SortArgs {
  const int* ids;
  int N, vocab, pad;
  int R;        // ids of a block: b, b + gridDim.x, b + 2 gridDim.x, ...
  int queue;    // entries of a warp's queue
  unsigned magic;  // 2^shift / gridDim.x, rounded up
  int shift;
  int* order;   // [N] tokens by id, then by position
  int* sorted;  // [N] their ids
  int* start;   // [vocab] first entry of each id in order
  int* count;   // [vocab]
  int* total;   // tokens in order
  int* arrived; // the sums' counters, to be zeroed
  long long n_arrived;
  unsigned* err;
};

// Block b sorts the ids that leave the remainder b (frequent tokens often have neighbouring ids,
// which would fall to few blocks otherwise); the order is by remainder, then by id.  Every block
// reads all ids, so that it also knows how many come before its own, and no block waits for another
// (the ids are a small part of dout, and stay in L2).  Warp w counts, and then places, the w-th
// share of the positions; a counter per (warp, id) keeps the order of positions.  What a warp finds
// in the first pass it queues in shared memory for the second (which goes through the ids again
// where a very frequent token fills the queue).
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const SortArgs a) {
  extern __shared__ int cnt[];  // [kSortWarps][R], then the queues [kSortWarps][queue]
  __shared__ int below_w[kSortWarps], scan_w[kSortWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int mod = gridDim.x, nr = (a.vocab - (int)blockIdx.x + mod - 1) / mod;
  auto quotient = [&](int id) { return (int)((uint64_t)(unsigned)id * a.magic >> a.shift); };
  const int share = ((a.N + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int n0 = (int)min((long long)warp * share, (long long)a.N), n1 = (int)min((long long)n0 + share, (long long)a.N);
  int* mine = cnt + warp * a.R;
  unsigned* queue = reinterpret_cast<unsigned*>(cnt + kSortWarps * a.R) + warp * a.queue;
  int queued = 0;
  let_next_start();
  for (int i = threadIdx.x; i < kSortWarps * a.R; i += kSortThreads) cnt[i] = 0;
  for (long long i = (long long)blockIdx.x * kSortThreads + threadIdx.x; i < a.n_arrived; i += (long long)gridDim.x * kSortThreads)
    a.arrived[i] = 0;
  __syncthreads();
  int below = 0;
  bool bad = false;
  int id[kAhead];
  auto load = [&](int n) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) id[j] = n + 32 * j + lane < n1 ? a.ids[n + 32 * j + lane] : a.pad;
  };
  for (int n = n0; n < n1; n += 32 * kAhead) {
    load(n);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (n + 32 * j >= n1) break;
      const bool known = (unsigned)id[j] < (unsigned)a.vocab, live = known && id[j] != a.pad;
      bad |= !known && id[j] != a.pad;
      const int at = quotient(id[j]), rest = id[j] - at * mod;
      below += live && rest < (int)blockIdx.x;
      const bool in = live && rest == (int)blockIdx.x;
      const unsigned who = __ballot_sync(0xffffffffu, in);
      if (who == 0) continue;
      const unsigned same = __match_any_sync(0xffffffffu, in ? at : -1);
      if (in && (same & ((1u << lane) - 1)) == 0) mine[at] += __popc(same);
      const int k = queued + __popc(who & ((1u << lane) - 1));
      if (in && k < a.queue) queue[k] = (unsigned)at << kOffsetBits | (unsigned)(n - n0 + 32 * j + lane);
      queued += __popc(who);
      __syncwarp();
    }
  }
  if (blockIdx.x == 0 && bad) record_error(a.err, kErrValue | kKernModel);
  below = __reduce_add_sync(0xffffffffu, below);
  if (lane == 0) below_w[warp] = below;
  __syncthreads();
  // counters become places: ids in order, of one id the warps in order
  int run = __reduce_add_sync(0xffffffffu, below_w[lane]);
  // (4 threads an id, 8 warps' counters each)
  constexpr int kShare = 4, kEach = kSortWarps / kShare;
  for (int r0 = 0; r0 < nr; r0 += kSortThreads / kShare) {
    const int r = r0 + threadIdx.x / kShare, part = threadIdx.x % kShare;
    int c[kEach], sum = 0;
#pragma unroll
    for (int w = 0; w < kEach; ++w) {
      c[w] = r < nr ? cnt[(part * kEach + w) * a.R + r] : 0;
      sum += c[w];
    }
    int incl = sum;
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) scan_w[warp] = incl;
    __syncthreads();
    int warps = scan_w[lane];
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, warps, o);
      if (lane >= o) warps += up;
    }
    const int before = __shfl_sync(0xffffffffu, warps, (warp + 31) & 31);
    int at = run + (warp ? before : 0) + incl - sum;
    run += __shfl_sync(0xffffffffu, warps, 31);
    const int first = __shfl_sync(0xffffffffu, at, lane & ~(kShare - 1));
    const int next = __shfl_sync(0xffffffffu, at + sum, lane | (kShare - 1));
    if (r < nr) {
      if (part == 0) {
        a.start[r * mod + blockIdx.x] = first;
        a.count[r * mod + blockIdx.x] = next - first;
      }
#pragma unroll
      for (int w = 0; w < kEach; ++w) {
        cnt[(part * kEach + w) * a.R + r] = at;
        at += c[w];
      }
    }
    __syncthreads();
  }
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) *a.total = run;
  auto place = [&](bool in, int q, int position) {
    const unsigned same = __match_any_sync(0xffffffffu, in ? q : -1);
    const unsigned earlier = same & ((1u << lane) - 1);
    const int at = in ? mine[q] : 0;
    if (in) {
      a.order[at + __popc(earlier)] = position;
      a.sorted[at + __popc(earlier)] = q * mod + blockIdx.x;
    }
    __syncwarp();
    if (in && earlier == 0) mine[q] = at + __popc(same);
    __syncwarp();
  };
  if (queued <= a.queue && share <= 1 << kOffsetBits) {
    for (int k = 0; k < queued; k += 32) {
      const unsigned e = k + lane < queued ? queue[k + lane] : 0;
      place(k + lane < queued, e >> kOffsetBits, n0 + (int)(e & ((1u << kOffsetBits) - 1)));
    }
    return;
  }
  for (int n = n0; n < n1; n += 32 * kAhead) {
    load(n);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (n + 32 * j >= n1) break;
      const int q = quotient(id[j]);
      const bool in = (unsigned)id[j] < (unsigned)a.vocab && id[j] != a.pad && id[j] - q * mod == (int)blockIdx.x;
      if (__any_sync(0xffffffffu, in)) place(in, q, n + 32 * j + lane);
    }
  }
}

// ------------------------------------------------------------------------------- sums

constexpr int kRows = 8;      // rows of dout that a warp has under way
constexpr int kFill = 4;      // ids of a warp that writes rows without tokens
constexpr int kGroup = 32;    // parts of an id's sum that are joined first

template <typename T, typename G>
struct SumArgs {
  const int *order, *sorted, *start, *count, *total;
  const T* dout;
  const G* base;
  G* dE;
  float* part;      // [2 sum_blocks][part_pitch]: a block's sums for an id that came in, and for one that goes on
  int* arrived;     // [tiles][3 sum_blocks]: parts of a group (by its first part's row), groups of an id (by its first block)
  int N, d, vocab, part_pitch;
  int chunk, sum_blocks, tiles;  // tokens of a warp (<= 32); blocks that sum, of 8 chunks each; column tiles
  long long pitch;
  float scale;
};

// Rows of ids without tokens: zeros, or base's.  A warp takes kFill ids.
template <typename T, typename G, bool kVec>
__device__ __forceinline__ void empty_rows(const SumArgs<T, G>& a, int v0, int lane) {
  const int n = lane < kFill && v0 + lane < a.vocab ? a.count[v0 + lane] : 1;
  for (unsigned todo = __ballot_sync(0xffffffffu, n == 0); todo; todo &= todo - 1) {
    const long long o = (long long)(v0 + __ffs(todo) - 1) * a.d;
    if constexpr (kVec) {
      constexpr int E = 16 / sizeof(G);
      if (a.d % E == 0) {
        // two rows at a time, so that more loads are under way
        const unsigned rest = todo & (todo - 1);
        const long long o2 = rest ? (long long)(v0 + __ffs(rest) - 1) * a.d : o;
#pragma unroll 4
        for (int c = lane * E; c < a.d; c += 32 * E) {
          const uint4 x = a.base ? *reinterpret_cast<const uint4*>(a.base + o + c) : make_uint4(0, 0, 0, 0);
          const uint4 y = a.base ? *reinterpret_cast<const uint4*>(a.base + o2 + c) : make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(a.dE + o + c) = x;
          if (rest) *reinterpret_cast<uint4*>(a.dE + o2 + c) = y;
        }
        if (rest) todo = rest;
        continue;
      }
    }
    for (int c = lane; c < a.d; c += 32) a.dE[o + c] = a.base ? a.base[o + c] : G(0.f);
  }
}

// E values of base at a multiple of E, as they are stored.
template <int E> struct BaseOf {
  float4 f[E / 4];
  uint2 h[E / 4];
  __device__ __forceinline__ void load(const float* base) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) f[i] = base ? reinterpret_cast<const float4*>(base)[i] : make_float4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* base) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) h[i] = base ? reinterpret_cast<const uint2*>(base)[i] : make_uint2(0, 0);
  }
};
// dst = base + scale f.
template <int E>
__device__ __forceinline__ void finish_vec(float* dst, const float* f, float scale, const BaseOf<E>& base) {
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    const float4 b = base.f[e / 4];
    *reinterpret_cast<float4*>(dst + e) = make_float4(fmaf(f[e], scale, b.x), fmaf(f[e + 1], scale, b.y),
                                                      fmaf(f[e + 2], scale, b.z), fmaf(f[e + 3], scale, b.w));
  }
}
template <int E>
__device__ __forceinline__ void finish_vec(__nv_bfloat16* dst, const float* f, float scale, const BaseOf<E>& base) {
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    const uint2 b = base.h[e / 4];
    *reinterpret_cast<uint2*>(dst + e) =
        make_uint2(ptx::pack_bf16x2(fmaf(f[e], scale, ptx::bf16lo(b.x)), fmaf(f[e + 1], scale, ptx::bf16hi(b.x))),
                   ptx::pack_bf16x2(fmaf(f[e + 2], scale, ptx::bf16lo(b.y)), fmaf(f[e + 3], scale, ptx::bf16hi(b.y))));
  }
}

// A warp's columns of a tile: lane l holds a vector (kVec), or 4 single columns.
template <typename T, bool kVec>
struct Columns {
  static constexpr int E = kVec ? Vec16<T>::E : 1, NV = kVec ? 1 : 4, N = NV * E, kTile = 32 * N;
  float f[N];
  int c0;  // first column of the tile
  __device__ __forceinline__ int col(int k) const { return c0 + (k * 32 + (int)(threadIdx.x & 31)) * E; }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = 0.f;
  }
  // a row of the tile in shared memory, [lane][N]
  __device__ __forceinline__ void put(float* row) const {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(row + (threadIdx.x & 31) * N + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  }
  __device__ __forceinline__ void take(const float* row) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(row + (threadIdx.x & 31) * N + i);
      f[i] += x.x; f[i + 1] += x.y; f[i + 2] += x.z; f[i + 3] += x.w;
    }
  }
  __device__ __forceinline__ void store(float* row, int d) const {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = col(k);
      if (c >= d) continue;
      if constexpr (kVec) {
#pragma unroll
        for (int e = 0; e < E; e += 4)
          *reinterpret_cast<float4*>(row + c + e) = make_float4(f[k * E + e], f[k * E + e + 1], f[k * E + e + 2], f[k * E + e + 3]);
      } else {
        row[c] = f[k];
      }
    }
  }
  // adds a stored row that another SM may have written
  __device__ __forceinline__ void add(const float* row, int d) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = col(k);
      if (c >= d) continue;
      if constexpr (kVec) {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(row + c + e));
          f[k * E + e] += x.x; f[k * E + e + 1] += x.y; f[k * E + e + 2] += x.z; f[k * E + e + 3] += x.w;
        }
      } else {
        f[k] += __ldcg(row + c);
      }
    }
  }
  template <typename G>
  __device__ __forceinline__ void finish(const SumArgs<T, G>& a, int v) const {
    const long long o = (long long)v * a.d;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = col(k);
      if (c >= a.d) continue;
      if constexpr (kVec) {
        BaseOf<E> b;
        b.load(a.base ? a.base + o + c : nullptr);
        finish_vec<E>(a.dE + o + c, f + k * E, a.scale, b);
      } else io<G>::st(a.dE + o + c, fmaf(f[k], a.scale, a.base ? io<G>::ld(a.base + o + c) : 0.f));
    }
  }
};

// Counts the warp in; true for the last of `all`, which then sees (past L1) what the others stored.
__device__ __forceinline__ bool last_of(int* counter, int all) {
  __syncwarp();
  int n = 0;
  if ((threadIdx.x & 31) == 0)
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(n) : "l"(counter) : "memory");
  n = __shfl_sync(0xffffffffu, n, 0);
  __syncwarp();
  return n == all - 1;
}

// Block q has summed a part of id v.  The last warp of a group of parts joins them, the last one
// of the groups writes the row; both in order.
template <typename T, typename G, bool kVec>
__device__ __forceinline__ void add_part(const SumArgs<T, G>& a, Columns<T, kVec>& sum, int v, int2 run, int q, bool came) {
  sum.store(a.part + (2 * (size_t)q + (came ? 0 : 1)) * a.part_pitch, a.d);
  const int unit = 8 * a.chunk, first = run.x / unit, parts = (run.x + run.y - 1) / unit - first + 1;
  const int g = (q - first) / kGroup, n = min(kGroup, parts - g * kGroup), groups = (parts + kGroup - 1) / kGroup;
  int* arrived = a.arrived + (size_t)(sum.c0 / Columns<T, kVec>::kTile) * 3 * a.sum_blocks;
  auto row_of = [&](int part) { return part == 0 ? 2 * (size_t)first + 1 : 2 * (size_t)(first + part); };
  if (!last_of(arrived + row_of(g * kGroup), n)) return;
  sum.clear();
#pragma unroll 8
  for (int k = 0; k < n; ++k) sum.add(a.part + row_of(g * kGroup + k) * a.part_pitch, a.d);
  if (groups > 1) {
    sum.store(a.part + row_of(g * kGroup) * a.part_pitch, a.d);
    if (!last_of(arrived + 2 * (size_t)a.sum_blocks + first, groups)) return;
    sum.clear();
#pragma unroll 8
    for (int k = 0; k < groups; ++k) sum.add(a.part + row_of(k * kGroup) * a.part_pitch, a.d);
  }
  sum.finish(a, v);
}

// A warp sums the tokens of one chunk over a tile of columns.  An id that begins and ends in the
// chunk is finished at once; one that goes past an end is joined with the neighbouring chunks of
// the block in shared memory, and past the block's ends in part.
// With kBase (and kVec) the rows of base are asked for together with those of dout: where base is dE
// and no rows of other ids are to be copied, which wants more warps instead of more registers.
template <typename T, typename G, bool kVec, bool kBase>
__global__ void __launch_bounds__(256, kVec && !kBase ? 3 : 2) embed_sum_kernel(const SumArgs<T, G> a) {
  using Cols = Columns<T, kVec>;
  // of each chunk: the sum for an id that came in, and for one that goes on (a chunk of one id that
  // does both has the first only, and is through)
  __shared__ __align__(16) float came_sum[8][Cols::kTile], goes_sum[8][Cols::kTile];
  __shared__ int through[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  wait_for_previous();
  if ((int)blockIdx.x >= a.sum_blocks * a.tiles) {
    empty_rows<T, G, kVec>(a, (((int)blockIdx.x - a.sum_blocks * a.tiles) * 8 + warp) * kFill, lane);
    return;
  }
  const int q = blockIdx.x / a.tiles, p0 = (q * 8 + warp) * a.chunk;
  const bool mine = lane < a.chunk && p0 + lane < a.N;
  const int token = mine ? a.order[p0 + lane] : 0, sorted = mine ? a.sorted[p0 + lane] : -1;
  const int left = p0 > 0 && p0 < a.N ? a.sorted[p0 - 1] : -1, right = p0 + a.chunk < a.N ? a.sorted[p0 + a.chunk] : -1;
  const int M = *a.total;  // (padding is not in order)
  if (q * 8 * a.chunk >= M) return;
  // (of the entries from M on, only their memory is there)
  const int n = min(a.chunk, M - p0), id = lane < n ? sorted : -1, before = n > 0 ? left : -1;
  const int after = p0 + a.chunk < M ? right : -1;
  // first token and count of the ids at the chunk's ends, in case they go past them
  const int v0 = __shfl_sync(0xffffffffu, id, 0), v1 = __shfl_sync(0xffffffffu, id, n > 0 ? n - 1 : 0);
  const int2 run0 = n > 0 && v0 == before ? make_int2(a.start[v0], a.count[v0]) : make_int2(0, 0);
  const int2 run1 = n > 0 && v1 == after ? make_int2(a.start[v1], a.count[v1]) : make_int2(0, 0);
  Cols acc;
  acc.c0 = ((int)blockIdx.x - q * a.tiles) * Cols::kTile;
  acc.clear();
  int came = -1, goes = -1;
  bool thru = false;
  for (int i0 = 0; i0 < n; i0 += kRows) {
    uint4 u[kVec ? kRows : 1][Cols::NV];
    float f[kVec ? 1 : kRows][Cols::NV];
    BaseOf<kVec ? Cols::E : 4> base[kBase ? kRows : 1];  // of the rows that end here
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if constexpr (kBase) {
        const int v = __shfl_sync(0xffffffffu, id, i0 + i), w = __shfl_sync(0xffffffffu, id, (i0 + i + 1) & 31);
        const bool ends = i0 + i < n && (i0 + i == n - 1 || v != w);
        base[i].load(ends && acc.col(0) < a.d ? a.base + (long long)v * a.d + acc.col(0) : nullptr);
      }
      const T* src = a.dout + __shfl_sync(0xffffffffu, token, i0 + i) * a.pitch;
#pragma unroll
      for (int k = 0; k < Cols::NV; ++k) {
        const int c = acc.col(k);
        const bool live = i0 + i < n && c < a.d;
        if constexpr (kVec) u[i][k] = live ? *reinterpret_cast<const uint4*>(src + c) : make_uint4(0, 0, 0, 0);
        else f[i][k] = live ? io<T>::ld(src + c) : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (i0 + i >= n) break;
#pragma unroll
      for (int k = 0; k < Cols::NV; ++k) {
        if constexpr (kVec) {
          float x[Cols::E];
          Vec16<T>::unpack(u[i][k], x);
#pragma unroll
          for (int e = 0; e < Cols::E; ++e) acc.f[k * Cols::E + e] += x[e];
        } else {
          acc.f[k] += f[i][k];
        }
      }
      const int v = __shfl_sync(0xffffffffu, id, i0 + i);
      const bool last = i0 + i == n - 1;
      if (!last && v == __shfl_sync(0xffffffffu, id, (i0 + i + 1) & 31)) continue;
      if (v == before) {
        acc.put(came_sum[warp]);
        came = v;
        thru = last && v == after;
      } else if (last && v == after) {
        acc.put(goes_sum[warp]);
        goes = v;
      } else if constexpr (kBase) {
        if (acc.col(0) < a.d) finish_vec<Cols::E>(a.dE + (long long)v * a.d + acc.col(0), acc.f, a.scale, base[i]);
      } else {
        acc.finish(a, v);
      }
      acc.clear();
    }
  }
  if (lane == 0) through[warp] = thru;
  __syncthreads();
  if (warp == 0 && came >= 0) {  // from the block before
    acc.take(came_sum[0]);
    for (int w = 1; w < 8 && through[w - 1]; ++w) acc.take(came_sum[w]);
    add_part<T, G, kVec>(a, acc, came, run0, q, true);
    acc.clear();
  }
  if (goes >= 0) {
    acc.take(goes_sum[warp]);
    bool open = true;
    for (int w = warp + 1; w < 8 && open; ++w) {
      acc.take(came_sum[w]);
      open = through[w];
    }
    if (open) add_part<T, G, kVec>(a, acc, goes, run1, q, false);
    else acc.finish(a, goes);
  }
}

// Ids of a sorting block: one block per SM, as far as the counters fit.
int sort_rows(int vocab) {
  const int r = ceil_div(vocab, serve_sm_count());
  return r < kMaxSortRows ? r : kMaxSortRows;
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// How the sums are taken, from the sizes alone (the workspace's size depends on it).
struct EmbedPlan {
  int chunk, blocks, tile, tiles, part_pitch;
  size_t order, sorted, start, count, tokens, arrived, part, total;  // offsets in the workspace
};
EmbedPlan embed_plan(const EmbedCall& c, bool vec) {
  EmbedPlan w;
  w.tile = vec ? 32 * (c.dtype == TG_F32 ? 4 : 8) : 128;
  w.tiles = ceil_div(c.d, w.tile);
  // chunks of 32 tokens, or of 16 or 8 where that makes fewer warps than 12 an SM
  w.chunk = 32;
  while (w.chunk > kRows && (long long)ceil_div(c.rows, w.chunk) * w.tiles < 1800) w.chunk /= 2;
  w.blocks = ceil_div(c.rows, 8 * w.chunk);
  w.part_pitch = (c.d + 3) / 4 * 4;
  const size_t tokens = up256((size_t)c.rows * 4), ids = up256((size_t)c.vocab * 4);
  w.order = 0;
  w.sorted = tokens;
  w.start = 2 * tokens;
  w.count = w.start + ids;
  w.tokens = w.count + ids;
  w.arrived = w.tokens + 256;
  w.part = w.arrived + up256((size_t)w.tiles * 3 * w.blocks * 4);
  w.total = w.part + up256((size_t)w.blocks * 2 * w.part_pitch * 4);
  return w;
}

// Whether rows of dout, base and dE are read and written 16 bytes at a time.
bool vector_rows(const EmbedCall& c) {
  const int E = c.dtype == TG_F32 ? 4 : 8;
  return c.d % E == 0 && c.pitch % E == 0 && aligned_16(c.dout) && aligned_16(c.base) && aligned_16(c.dE);
}

template <typename T, typename G>
cudaError_t sums(const EmbedCall& c, const SortArgs& t, const EmbedPlan& w, bool vec, cudaStream_t s) {
  SumArgs<T, G> a;
  a.order = t.order; a.sorted = t.sorted; a.start = t.start; a.count = t.count; a.total = t.total; a.arrived = t.arrived;
  a.dout = static_cast<const T*>(c.dout); a.base = static_cast<const G*>(c.base); a.dE = static_cast<G*>(c.dE);
  a.part = reinterpret_cast<float*>(static_cast<char*>(c.ws) + w.part);
  a.N = (int)c.rows; a.d = c.d; a.vocab = c.vocab; a.part_pitch = w.part_pitch; a.pitch = c.pitch; a.scale = c.scale;
  a.chunk = w.chunk; a.sum_blocks = w.blocks; a.tiles = w.tiles;
  const long long blocks = (long long)w.blocks * w.tiles + (c.base == c.dE ? 0 : ceil_div(c.vocab, 8 * kFill));
  if (blocks == 0) return cudaSuccess;
  if (blocks > (1ll << 31) - 1) return cudaErrorInvalidConfiguration;
  const auto kernel = !vec ? embed_sum_kernel<T, G, false, false>
                           : c.base == c.dE ? embed_sum_kernel<T, G, true, true> : embed_sum_kernel<T, G, true, false>;
  return launch_early(kernel, dim3((unsigned)blocks), 256, s, a);
}

template <typename T>
cudaError_t lookup(const EmbedCall& c, cudaStream_t s) {
  const T* E = static_cast<const T*>(c.E);
  T* out = static_cast<T*>(c.out);
  constexpr int N = 16 / sizeof(T);
  const unsigned blocks = (unsigned)((c.rows + 7) / 8);
  const auto kernel = c.d % N == 0 && c.pitch % N == 0 && aligned_16(c.E) && aligned_16(c.out) ? embed_lookup_kernel<T, true>
                                                                                         : embed_lookup_kernel<T, false>;
  kernel<<<blocks, 256, 0, s>>>(c.ids, E, out, c.rows, c.d, c.vocab, c.pitch, c.scale, c.pad_id, c.padded, c.err);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_embed_lookup(const EmbedCall& c, cudaStream_t s) {
  return c.dtype == TG_F32 ? lookup<float>(c, s) : lookup<__nv_bfloat16>(c, s);
}

size_t embed_backward_ws_bytes(const EmbedCall& c) {
  // (the size query knows no addresses: it covers both ways of reading rows)
  const size_t one = embed_plan(c, true).total, other = embed_plan(c, false).total;
  return one > other ? one : other;
}

cudaError_t launch_embed_backward(const EmbedCall& c, cudaStream_t s) {
  const bool vec = vector_rows(c);
  const EmbedPlan w = embed_plan(c, vec);
  char* ws = static_cast<char*>(c.ws);
  SortArgs a;
  a.ids = c.ids; a.N = (int)c.rows; a.vocab = c.vocab; a.pad = c.pad_id;
  a.R = sort_rows(c.vocab);
  a.order = reinterpret_cast<int*>(ws + w.order);
  a.sorted = reinterpret_cast<int*>(ws + w.sorted);
  a.start = reinterpret_cast<int*>(ws + w.start);
  a.count = reinterpret_cast<int*>(ws + w.count);
  a.total = reinterpret_cast<int*>(ws + w.tokens);
  a.arrived = reinterpret_cast<int*>(ws + w.arrived);
  a.n_arrived = (long long)w.tiles * 3 * w.blocks;
  a.err = c.err;
  const int counters = kSortWarps * a.R * 4, left = (kSortSmem - counters) / (kSortWarps * 4);
  // a token that a quarter of the positions name still fits (more shared memory than that delays the
  // kernel behind: 16,384 tokens 25 us with 512 entries, 26 with 2,048; 262,144 tokens 201 and 154 us)
  a.queue = a.N / kSortWarps / 4 > 512 ? a.N / kSortWarps / 4 : 512;
  if (a.queue > left) a.queue = left;
  const int smem = counters + kSortWarps * a.queue * 4;
  cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSortSmem);
  if (e != cudaSuccess) return e;
  const unsigned blocks = ceil_div(c.vocab, a.R);
  a.shift = 31;
  while ((1u << (a.shift - 31)) < blocks) ++a.shift;  // quotients of ids below 2^31 are exact
  a.magic = (unsigned)(((1ull << a.shift) + blocks - 1) / blocks);
  embed_sort_kernel<<<blocks, kSortThreads, smem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  using bf16 = __nv_bfloat16;
  if (c.dtype == TG_F32)
    return c.grad_dtype == TG_F32 ? sums<float, float>(c, a, w, vec, s) : sums<float, bf16>(c, a, w, vec, s);
  return c.grad_dtype == TG_F32 ? sums<bf16, float>(c, a, w, vec, s) : sums<bf16, bf16>(c, a, w, vec, s);
}

}  // namespace tg

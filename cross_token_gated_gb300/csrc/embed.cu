// Token lookup with scaling, and the embedding's gradient by sorted tokens ("TANGO:
// Token-Aggregated Nonlinear Gating Operators ...", sec. 2.3: the tied token embedding).
//
//   out[n] = s E[id_n];   dE[v] = base[v] + s sum_{n: id_n = v} dout[n]
//
// The gradient sorts the tokens by id (a stable counting sort, so that the order of every sum is
// fixed), then sums each id's rows of dout in fp32.
#include "tg_common.cuh"
#include "tg_ends.h"
#include "tg_serve.h"

namespace tg {
namespace {

// ---------------------------------------------------------------------------- lookup

// One warp per row.
template <typename T>
__global__ void __launch_bounds__(256) embed_lookup_kernel(const int* ids, const T* E, T* out, long long rows, int d,
                                                           int vocab, long long pitch, float scale, int pad,
                                                           unsigned* err) {
  const long long r = (long long)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (r >= rows) return;
  const int id = ids[r];
  const bool known = id >= 0 && id < vocab;
  if (!known && id != pad && lane == 0) record_error(err, kErrValue | kKernModel);
  const bool live = known && id != pad;
  const T* src = E + (long long)(live ? id : 0) * d;
  T* dst = out + r * pitch;
  for (int c = lane; c < d; c += 32) {
    if (!live) dst[c] = T(0.f);
    else if (scale == 1.f) dst[c] = src[c];
    else io<T>::st(dst + c, io<T>::ld(src + c) * scale);
  }
}

// ------------------------------------------------------------------------------ sort

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kMaxSortRows = 1536;  // ids of a block: kSortWarps counters each in shared memory

struct SortArgs {
  const int* ids;
  int N, vocab, pad;
  int R;        // ids of a block
  int* order;   // [N] tokens by id, then by position
  int* start;   // [vocab] first entry of each id in order
  int* count;   // [vocab]
  unsigned* err;
};

// Block b sorts the ids of [b R, (b + 1) R): every block reads all ids, so that it also knows how
// many lie below its own, and no block waits for another.  Warp w counts, and then places, the
// w-th share of the positions; a counter per (warp, id) keeps the order of positions.
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const SortArgs a) {
  extern __shared__ int cnt[];  // [kSortWarps][R]
  __shared__ int below_w[kSortWarps], scan_w[kSortWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int v0 = blockIdx.x * a.R, nr = min(a.R, a.vocab - v0);
  const int share = ((a.N + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const long long p0 = (long long)warp * share;
  const int n0 = (int)min(p0, (long long)a.N), n1 = (int)min(p0 + share, (long long)a.N);
  int* mine = cnt + warp * a.R;
  for (int i = threadIdx.x; i < kSortWarps * a.R; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  int below = 0;
  bool bad = false;
  for (int n = n0; n < n1; n += 32) {
    const int id = n + lane < n1 ? a.ids[n + lane] : a.pad;
    const bool live = id != a.pad && id >= 0 && id < a.vocab;
    bad |= !live && id != a.pad;
    below += live && id < v0;
    const bool in = live && id >= v0 && id < v0 + nr;
    const unsigned who = __ballot_sync(0xffffffffu, in);
    if (who == 0) continue;
    const unsigned same = __match_any_sync(0xffffffffu, in ? id - v0 : -1);
    if (in && (same & ((1u << lane) - 1)) == 0) mine[id - v0] += __popc(same);
    __syncwarp();
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
  for (int n = n0; n < n1; n += 32) {
    const int id = n + lane < n1 ? a.ids[n + lane] : a.pad;
    const bool in = id != a.pad && id >= v0 && id < v0 + nr;
    const unsigned who = __ballot_sync(0xffffffffu, in);
    if (who == 0) continue;
    const unsigned same = __match_any_sync(0xffffffffu, in ? id - v0 : -1);
    const unsigned earlier = same & ((1u << lane) - 1);
    const int at = in ? mine[id - v0] : 0;
    if (in) a.order[at + __popc(earlier)] = n + lane;
    __syncwarp();
    if (in && earlier == 0) mine[id - v0] = at + __popc(same);
    __syncwarp();
  }
}

// ------------------------------------------------------------------------------- sums

template <typename T, typename G>
struct SumArgs {
  const int *order, *start, *count;
  const T* dout;
  const G* base;
  G* dE;
  int d, vocab;
  long long pitch;
  float scale;
};

// One warp per id.
template <typename T, typename G>
__global__ void __launch_bounds__(256) embed_sum_kernel(const SumArgs<T, G> a) {
  const int v = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x & 31;
  if (v >= a.vocab) return;
  const int at = a.start[v], n = a.count[v];
  for (int c = lane; c < a.d; c += 32) {
    float s = 0.f;
    for (int i = 0; i < n; ++i) s += io<T>::ld(a.dout + (long long)a.order[at + i] * a.pitch + c);
    const long long o = (long long)v * a.d + c;
    io<G>::st(a.dE + o, fmaf(s, a.scale, a.base ? io<G>::ld(a.base + o) : 0.f));
  }
}

// Ids of a sorting block: one block per SM, as far as the counters fit.
int sort_rows(int vocab) {
  const int r = ceil_div(vocab, serve_sm_count());
  return r < kMaxSortRows ? r : kMaxSortRows;
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

template <typename T, typename G>
cudaError_t sums(const EmbedCall& c, const int* order, const int* start, const int* count, cudaStream_t s) {
  SumArgs<T, G> a{order, start, count, static_cast<const T*>(c.dout), static_cast<const G*>(c.base),
                  static_cast<G*>(c.dE), c.d, c.vocab, c.pitch, c.scale};
  embed_sum_kernel<T, G><<<ceil_div(c.vocab, 8), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_embed_lookup(const EmbedCall& c, cudaStream_t s) {
  const unsigned blocks = (unsigned)((c.rows + 7) / 8);
  if (c.dtype == TG_F32)
    embed_lookup_kernel<float><<<blocks, 256, 0, s>>>(c.ids, static_cast<const float*>(c.E), static_cast<float*>(c.out),
                                                      c.rows, c.d, c.vocab, c.pitch, c.scale, c.pad_id, c.err);
  else
    embed_lookup_kernel<__nv_bfloat16><<<blocks, 256, 0, s>>>(
        c.ids, static_cast<const __nv_bfloat16*>(c.E), static_cast<__nv_bfloat16*>(c.out), c.rows, c.d, c.vocab,
        c.pitch, c.scale, c.pad_id, c.err);
  return cudaGetLastError();
}

size_t embed_backward_ws_bytes(const EmbedCall& c) {
  return up256((size_t)c.rows * 4) + 2 * up256((size_t)c.vocab * 4);
}

cudaError_t launch_embed_backward(const EmbedCall& c, cudaStream_t s) {
  SortArgs a;
  a.ids = c.ids; a.N = (int)c.rows; a.vocab = c.vocab; a.pad = c.pad_id;
  a.R = sort_rows(c.vocab);
  char* ws = static_cast<char*>(c.ws);
  a.order = reinterpret_cast<int*>(ws);
  a.start = reinterpret_cast<int*>(ws + up256((size_t)c.rows * 4));
  a.count = reinterpret_cast<int*>(ws + up256((size_t)c.rows * 4) + up256((size_t)c.vocab * 4));
  a.err = c.err;
  const size_t smem = (size_t)kSortWarps * a.R * 4;
  cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSortWarps * kMaxSortRows * 4);
  if (e != cudaSuccess) return e;
  embed_sort_kernel<<<ceil_div(c.vocab, a.R), kSortThreads, smem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  using bf16 = __nv_bfloat16;
  if (c.dtype == TG_F32)
    return c.grad_dtype == TG_F32 ? sums<float, float>(c, a.order, a.start, a.count, s)
                                  : sums<float, bf16>(c, a.order, a.start, a.count, s);
  return c.grad_dtype == TG_F32 ? sums<bf16, float>(c, a.order, a.start, a.count, s)
                                : sums<bf16, bf16>(c, a.order, a.start, a.count, s);
}

}  // namespace tg

// Ragged batches over a paged cache: how a kernel finds a row's sequence, position and
// page, with every device value checked against its range before it is used.
#pragma once
#include "tg_common.cuh"

namespace tg {

constexpr unsigned kKernPaged = 6u << 8;

struct PagedBatch {
  int B, N, max_new, max_len;
  int page_size, n_pages, table_pitch;
  const int* cu_new;
  const int* lens;
  const int* page_table;
  unsigned* err;
};

// Sequence b's rows [r0, r0 + n) and its cached length, each forced into its range.
struct PagedSeq {
  int r0, n, len;
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedBatch& p, int b, bool flag) {
  const int c0 = p.cu_new[b], c1 = p.cu_new[b + 1], l = p.lens[b];
  PagedSeq s;
  s.r0 = min(max(c0, 0), p.N);
  s.n = min(min(max(c1, s.r0), p.N) - s.r0, p.max_new);
  s.len = min(max(l, 0), p.max_len);
  if (flag && (s.r0 != c0 || s.r0 + s.n != c1 || s.len != l)) record_error(p.err, kErrValue | kKernPaged);
  return s;
}

// Page of token `pos` (0 <= pos < max_len <= table_pitch * page_size); -1, flagged, if the
// table's entry is not a page of the pool.
__device__ __forceinline__ int paged_page(const PagedBatch& p, int b, int page_index) {
  const int pg = p.page_table[(size_t)b * p.table_pitch + page_index];
  if (pg >= 0 && pg < p.n_pages) return pg;
  record_error(p.err, kErrValue | kKernPaged);
  return -1;
}

// Whether a row's weights e^{tau (q.k - 1)}, of which n keys' sum up to `sum`, lie outside what
// unit vectors give.  Rounded to bf16 they are at most 1 + 2^-8 long, so that with tau <= 20 a
// weight lies within e^{20 (2^-7 + 2^-16)} = 1.17 and e^{-20 (2 + 2^-7 + 2^-16)} = 2^-57.9, and its
// own rounding moves it by 2^-8.  Longer vectors can leave the range of fp32, which a sum without
// a running maximum does not survive.  (NaN is no reason: it shows in the result.)
__device__ __forceinline__ bool not_unit(float sum, int n) {
  return n > 0 && (sum > 1.25f * (float)n || sum < 0x1p-59f * (float)n);
}

// The last sequence whose first row is <= row, by a 32-way search; a whole warp calls it
// with one row.  With rising cu_new this is the row's sequence (empty ones are skipped).
__device__ __forceinline__ int paged_find(const PagedBatch& p, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = p.B;
  while (n > 1) {
    const int step = (n + 31) / 32, i = lo + lane * step;
    const bool le = lane * step < n && p.cu_new[i] <= row;
    const int cnt = max(1, __popc(__ballot_sync(0xffffffffu, le)));
    const int adv = (cnt - 1) * step;
    lo += adv;
    n = min(step, n - adv);
  }
  return lo;
}

// Tiles of R rows are numbered so that no scan is needed: sequence b's first tile is
// cu_new[b] / R + b (the numbers in between are skipped).
struct TileRef {
  int b, row0, n, pos0;  // first row, rows (0: no such tile), first row's position
};
template <int R>
__device__ __forceinline__ TileRef find_tile(const PagedBatch& p, int tile, bool flag) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = p.B;
  while (n > 1) {
    const int step = (n + 31) / 32, i = lo + lane * step;
    const bool le = lane * step < n && min(max(p.cu_new[i], 0), p.N) / R + i <= tile;
    const int cnt = max(1, __popc(__ballot_sync(0xffffffffu, le)));
    const int adv = (cnt - 1) * step;
    lo += adv;
    n = min(step, n - adv);
  }
  const PagedSeq s = paged_seq(p, lo, flag);
  const int k = tile - (s.r0 / R + lo);
  TileRef t{lo, s.r0 + k * R, 0, 0};
  if (k < 0 || k * R >= s.n) return t;
  t.n = min(R, s.n - k * R);
  t.pos0 = s.len - s.n + k * R;
  return t;
}

}  // namespace tg

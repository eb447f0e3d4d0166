// TANGO aggregation of chunks of new tokens over a paged cache on the tensor cores (tcgen05),
// "TANGO: Token-Aggregated Nonlinear Gating Operators ...", sec. 2.1 eq. 5 with sec. 2.2
// eq. 6.  Two kernels per pass over heads:
//
// paged_weights_kernel  S = Q K^T (128 rows x 128 keys, tcgen05), P = e^{tau (S - 1)} rounded
//     to bf16 (half a step of 2^-8 per weight; the rounded weights are also what the
//     denominators sum, so a row's weights still add up to one), masked weights selected to
//     zero.  P goes to scratch in the layout of the next kernel's shared-memory operand
//     ([64-key block][row][64], 128-byte swizzle), so that it is copied in as it lies.
//     Weights are formed once per (row, head, key), not once per gate strip: at 14,240
//     gates a head a strip-wise recomputation would spend as many exp2 as the product has
//     tensor cycles.
// paged_weights_few_kernel  the same P for up to 8 new tokens of a sequence on the CUDA
//     cores, a thread per key: a 128-row product would be nearly all padding.
// paged_gates_kernel    U = P G: tiles of 128 rows x 256 gate columns, 64 keys a step.
//     warps 0, 3 TMA producers (4 stages of P 16 KB + G 32 KB), a step each in turn; 32 pages
//                looked up at a time, one lane per page issues its copies; the first job's G
//                is asked for while the weights kernel still runs
//     warp 1     MMA issuer (128 x 256 x 16), two accumulators in TMEM.  Tiles of a few rows
//                run the same product on unused rows: it is shorter than the step's G takes
//                from memory (D^T = G^T P^T with 16 columns, which does an eighth of the work,
//                measured slower: 8 products a step of about 100 cycles each)
//     warp 2     scheduler: takes jobs from a counter, works out what they are
//     warps 4-11 epilogue: times 1 / den and v, bf16 out; or f32 partial sums of a key range.
//                Rows are turned into columns through shared memory, so that v and out move
//                in whole 64-byte pieces of a row
//     warps 12-15 scrub: only in steps with keys that some row of the tile does not see:
//                slots past the sequence's length become zeros, and non-finite gates of the
//                chunk's own tokens are taken out of the product (0 * NaN would reach rows
//                that do not see them); the epilogue adds them back to the rows that do
//
// The weights of a pass stay within 2 GB: a pass takes some of the heads, or the tiles of one head
// that start within a range of scratch rows.
//
// A job is a (sequence, key range, head, strip, row tile) with the row tile fastest, so the
// CTAs that work side by side share their G out of L2.  Key ranges are cut when the tiles
// alone would not fill the SMs; the job that finishes a tile last adds the ranges' partial
// sums in their order.  Every wait is bounded; on expiry the kernel records a timeout in
// the error word.
//
// Decode steps are bound by HBM: 8 sequences of one new token over 1,025 to 8,192 cached ones
// (2 x 14,240 gates) take 361 to 367 us, 6.36 TB/s.  512 new tokens over 8,192 take 208 us, 1,118
// TFLOP/s; what bounds whole tiles is not known.  A step brings 48 KB into the SM, 768 cycles at 64
// bytes a clock against 512 of products, but CTA pairs, which bring 32 KB, gained nothing.  Any
// other load of the SM waits some 5,000 cycles behind the copies, hence eight epilogue warps and v
// asked for before the products end (prompts of 2,048 tokens and decode steps in one batch: 832 ->
// 733 us).
#include <atomic>

#include "tg_common.cuh"
#include "tg_paged.cuh"
#include "tg_ptx.cuh"
#include "tg_serve.h"
#include "tg_tma.h"

namespace tg {
namespace {

using namespace ptx;

constexpr int kM = 128;           // rows of a tile
constexpr int kN = 256;           // gate columns of a strip
constexpr int kK = 64;            // keys of a step
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kJobsPerSm = 4;     // at most; see TcArgs::jobs_per_sm
constexpr int kFewRows = 16;      // tiles of at most this many rows finish a thread per column

__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Untiled copies (16-byte aligned on both sides, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
// 16 bytes global -> shared; zeros instead where !valid (nothing is read then).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

__host__ __device__ constexpr int up8(int x) { return (x + 7) & ~7; }

struct TcArgs {
  PagedBatch p;
  int H, d_h, m_h, m_pitch;
  int h0, heads;             // heads of this pass
  int row0, rows;            // tiles of this pass: scratch rows from row0 on, in a span of `rows`
  int rows_tot;              // scratch rows of a head: those, and one tile's more unless it is all
  int key_blocks;            // ceil(max_len / 64)
  int span_keys, spans;      // of the weights kernel; spans: ceil(max_len / span_keys), up to 4s
  int strips;                // ceil(m_h / 256)
  int tiles;                 // tile numbers: N / 128 + B
  int r8cap;                 // rows of a partial: min(128, up8(max_new))
  int min_steps;             // a key range is at least this many steps
  int jobs_per_sm;           // key ranges are cut for about this many jobs per SM
  int nc_cap;                // key ranges of a tile, at most
  int n_slots;
  int box_rows;              // rows of a G box
  float s;
  const float* tau;
  const float* null_bias;
  long long v_pitch;
  int v_vec;                 // v rows are 16-byte aligned
  const __nv_bfloat16 *q, *v;
  __nv_bfloat16* out;
  const __nv_bfloat16 *k_pages, *g_pages;
  uint8_t* P;                // [head][row][key block][128 bytes], see p_block()
  float* den;                // [head][row][span]
  float* part;               // [slot]: [32][r8cap][4], or [row][128] for tiles of few rows
  int* slot;                 // [head][strip][tile][half][nc_cap]
  int* done;                 // [head][strip][tile][half]: ranges that are done
  int* next;                 // [0] next job, [1] next partial slot
  uint64_t timeout_ns;
  int debug_timeout;         // test hook: both kernels first wait on a barrier nothing signals
};

// Scratch row of a sequence's first row: sequences start at multiples of 8.  Less than 0, or
// from a.rows on, a tile belongs to another pass.
__device__ __forceinline__ int scratch_row(const TcArgs& a, int r0, int b) { return up8(r0) + 8 * b - a.row0; }
// P of key block kb of a tile with r8 scratch rows.
__device__ __forceinline__ uint8_t* p_block(const TcArgs& a, int hl, int prow, int r8, int kb) {
  return a.P + (((size_t)hl * a.rows_tot + prow) * a.key_blocks + (size_t)kb * r8) * 128;
}

// The gates kernel's counters, cleared by all CTAs of a weights kernel together.
__device__ __forceinline__ void clear_counters(const TcArgs& a, int tile, int hl, int span) {
  const size_t n = (size_t)a.heads * a.strips * a.tiles * 2;
  const size_t cta = ((size_t)span * gridDim.y + hl) * gridDim.x + tile, ctas = (size_t)gridDim.x * gridDim.y * gridDim.z;
  for (size_t i = cta * blockDim.x + threadIdx.x; i < n; i += ctas * blockDim.x) a.done[i] = 0;
  if (cta == 0 && threadIdx.x < 2) a.next[threadIdx.x] = 0;
}

// ============================================================================ weights

constexpr int kWThreads = 256;
constexpr uint32_t kWQ = kM * 128;  // 16 KB at d_h = 64
constexpr size_t kWSmem = 1024 + 3 * kWQ + 2 * (kM * 128) + 64;

// grid (tiles, heads, spans)
__global__ void __launch_bounds__(kWThreads) paged_weights_kernel(const TcArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sQ = base, *sK = base + kWQ, *sP = base + 3 * kWQ;
  uint64_t *bar = reinterpret_cast<uint64_t*>(sP + 2 * kM * 128), *never = bar + 1;
  uint32_t* tm = reinterpret_cast<uint32_t*>(bar + 2);
  __shared__ float half_sum[kM];
  const int t = threadIdx.x, warp = t / 32, lane = t & 31;
  const int tile = blockIdx.x, hl = blockIdx.y, span = blockIdx.z, head = a.h0 + hl;

  griddep_launch();
  clear_counters(a, tile, hl, span);
  const TileRef tr = find_tile<kM>(a.p, tile, hl == 0 && span == 0);
  const int vis = tr.pos0 + tr.n;
  const int key0 = span * a.span_keys, key1 = min(key0 + a.span_keys, (vis + 63) & ~63);
  if (tr.n == 0 || vis <= 0 || key0 >= vis) return;
  const PagedSeq sq = paged_seq(a.p, tr.b, false);
  const int prow = scratch_row(a, sq.r0, tr.b) + (tr.row0 - sq.r0), r8 = up8(tr.n);
  if (prow < 0 || prow >= a.rows) return;

  if (t == 0) {
    mbar_init(bar, 1);
    mbar_init(never, 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tm, 128);
    tmem_relinquish();
  }
  const int cpr = a.d_h / 8;                    // 16-byte chunks of a row: 8, 4 or 2
  const int sh = cpr == 8 ? 0 : cpr == 4 ? 1 : 2;  // swizzle: chunk ^= (row >> sh) & (cpr - 1)
  const uint32_t q_s = smem_u32(sQ), k_s = smem_u32(sK);
  auto place = [&](int row, int c) -> uint32_t {
    return (uint32_t)row * (cpr * 16) + (uint32_t)((c ^ ((row >> sh) & (cpr - 1))) << 4);
  };
  auto load_keys = [&](int k0, int buf) {
    for (int i = t; i < kM * cpr; i += kWThreads) {
      const int row = i / cpr, c = i - row * cpr, key = k0 + row;
      const __nv_bfloat16* src = a.k_pages;
      bool ok = key < vis;
      if (ok) {
        const int pi = key / a.p.page_size, pg = paged_page(a.p, tr.b, pi);
        ok = pg >= 0;
        if (ok) src = a.k_pages + (((size_t)pg * a.p.page_size + (key - pi * a.p.page_size)) * a.H + head) * a.d_h + c * 8;
      }
      cp_async16(k_s + buf * kWQ + place(row, c), src, ok);
    }
    cp_async_commit();
  };
  for (int i = t; i < kM * cpr; i += kWThreads) {
    const int row = i / cpr, c = i - row * cpr;
    const bool ok = row < tr.n;
    cp_async16(q_s + place(row, c), ok ? a.q + ((size_t)(tr.row0 + row) * a.H + head) * a.d_h + c * 8 : a.q, ok);
  }
  load_keys(key0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tm;
  const uint32_t layout = a.d_h == 64 ? kSwizzle128B : a.d_h == 32 ? kSwizzle64B : kSwizzle32B;
  const uint32_t idesc = idesc_bf16_f32(kM, 128, false, false);
  const float c2 = head_tau(a.tau, a.s, head, a.p.err, kKernPaged) * kLog2e;
  const int wg = warp / 4, quarter = warp & 3, row = quarter * 32 + lane;
  const bool mine = quarter * 32 < r8;  // this warp holds rows that are kept
  uint8_t* stage = sP + wg * (kM * 128);
  const uint32_t st = smem_u32(stage) + row * 128;
  const int last = tr.pos0 + row;       // the row sees keys <= last
  float sum = 0.f;
  bool ok = true;
  int n = 0;
  for (int k0 = key0; k0 < key1; k0 += 128, ++n) {
    const int buf = n & 1;
    cp_async_wait_all();
    fence_proxy_async_smem();
    __syncthreads();
    if (t == 0) {
      tc_fence_after();
      for (int kk = 0; kk < a.d_h / 16; ++kk)
        mma_bf16_ss(tmem, smem_desc(q_s + kk * 32, 16, 8 * a.d_h * 2, layout),
                    smem_desc(k_s + buf * kWQ + kk * 32, 16, 8 * a.d_h * 2, layout), idesc, kk != 0);
      mma_commit(bar);
    }
    if (k0 + 128 < key1) load_keys(k0 + 128, buf ^ 1);
    // a bounded wait, after which every warp leaves together below
    ok = mbar_wait(a.debug_timeout ? never : bar, n & 1, a.timeout_ns);
    if (!__syncthreads_and(ok)) {
      if (t == 0) record_error(a.p.err, kErrTimeout | kKernPaged);
      break;
    }
    tc_fence_after();
    const int kb0 = k0 + wg * 64;         // this warpgroup's 64 keys
    const bool keep = kb0 < key1;
    if (t % 128 == 0) bulk_wait_group_read0();  // the stage's previous store has read it
    named_bar_sync(1 + wg, 128);
    if (keep && mine) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r[32];
        tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + wg * 64 + h * 32, r);
        tmem_ld_wait();
        const int first = kb0 + h * 32;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = u * 8 + e * 2;
            float w0 = ex2_approx(fmaf(__uint_as_float(r[i]), c2, -c2));
            float w1 = ex2_approx(fmaf(__uint_as_float(r[i + 1]), c2, -c2));
            w0 = first + i <= last ? w0 : 0.f;
            w1 = first + i + 1 <= last ? w1 : 0.f;
            pk[e] = pack_bf16x2(w0, w1);
            sum += bf16lo(pk[e]) + bf16hi(pk[e]);
          }
          st_shared_v4(st + (uint32_t)(((h * 4 + u) ^ (row & 7)) << 4), make_uint4(pk[0], pk[1], pk[2], pk[3]));
        }
      }
    }
    tc_fence_before();
    fence_proxy_async_smem();
    named_bar_sync(1 + wg, 128);
    if (t % 128 == 0 && keep) {
      bulk_store(p_block(a, hl, prow, r8, kb0 / 64), stage, (uint32_t)r8 * 128);
      bulk_commit_group();
    }
  }
  if (t % 128 == 0) bulk_wait_group0();
  // both warpgroups' halves of a row's sum
  __syncthreads();
  if (wg == 1) half_sum[row] = sum;
  __syncthreads();
  if (wg == 0 && row < tr.n) {
    sum += half_sum[row];
    a.den[((size_t)hl * a.rows_tot + prow + row) * a.spans + span] = sum;
    if (ok && not_unit(sum, min(key0 + a.span_keys, last + 1) - key0)) record_error(a.p.err, kErrValue | kKernPaged);
  }
  cp_async_wait_all();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    // after a wait that ran out the product may still be on its way
    if (!ok) mbar_wait(bar, n & 1, a.timeout_ns);
    tmem_dealloc(tmem, 128);
  }
}

// grid (tiles, heads, spans), 256 threads, one key each per round.
template <int R, int DH>
__global__ void __launch_bounds__(kWThreads, 4) paged_weights_few_kernel(const TcArgs a) {
  __shared__ __align__(16) float qs[R][DH];
  __shared__ float red[kWThreads / 32][R];
  const int t = threadIdx.x, lane = t & 31;
  const int tile = blockIdx.x, hl = blockIdx.y, span = blockIdx.z, head = a.h0 + hl;
  griddep_launch();
  clear_counters(a, tile, hl, span);
  const TileRef tr = find_tile<kM>(a.p, tile, hl == 0 && span == 0);
  const int vis = tr.pos0 + tr.n;
  const int key0 = span * a.span_keys, key1 = min(key0 + a.span_keys, (vis + 63) & ~63);
  if (tr.n == 0 || vis <= 0 || key0 >= vis) return;
  const int rows = min(tr.n, R);  // R >= max_new
  const PagedSeq sq = paged_seq(a.p, tr.b, false);
  const int prow = scratch_row(a, sq.r0, tr.b), r8 = up8(tr.n);
  if (prow < 0 || prow >= a.rows) return;
  constexpr int C = DH / 8;
  uint4 u[C];
  auto load = [&](int key) {
    const __nv_bfloat16* kp = nullptr;
    if (key < vis) {
      const int pi = key / a.p.page_size, pg = paged_page(a.p, tr.b, pi);
      if (pg >= 0) kp = a.k_pages + (((size_t)pg * a.p.page_size + (key - pi * a.p.page_size)) * a.H + head) * DH;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) u[c] = kp ? ld_global_v4(kp + c * 8) : make_uint4(0, 0, 0, 0);
  };
  load(key0 + t);
  for (int i = t; i < R * DH; i += kWThreads) {
    const int r = i / DH, c = i - r * DH;
    qs[r][c] = r < rows ? __bfloat162float(a.q[((size_t)(tr.row0 + r) * a.H + head) * DH + c]) : 0.f;
  }
  const float c2 = head_tau(a.tau, a.s, head, a.p.err, kKernPaged) * kLog2e;
  float sum[R] = {};
  __syncthreads();
  for (int key = key0 + t; key < key1; key += kWThreads) {
    float x[R] = {};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t uu[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 q0 = *reinterpret_cast<const float4*>(&qs[r][c * 8]);
        const float4 q1 = *reinterpret_cast<const float4*>(&qs[r][c * 8 + 4]);
        x[r] = fmaf(bf16lo(uu[0]), q0.x, x[r]);
        x[r] = fmaf(bf16hi(uu[0]), q0.y, x[r]);
        x[r] = fmaf(bf16lo(uu[1]), q0.z, x[r]);
        x[r] = fmaf(bf16hi(uu[1]), q0.w, x[r]);
        x[r] = fmaf(bf16lo(uu[2]), q1.x, x[r]);
        x[r] = fmaf(bf16hi(uu[2]), q1.y, x[r]);
        x[r] = fmaf(bf16lo(uu[3]), q1.z, x[r]);
        x[r] = fmaf(bf16hi(uu[3]), q1.w, x[r]);
      }
    }
    if (key + kWThreads < key1) load(key + kWThreads);
    const int kc = key & 63;
    uint8_t* pb = p_block(a, hl, prow, r8, key / kK) + (kc & 7) * 2;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float w = key <= tr.pos0 + r ? ex2_approx(fmaf(x[r], c2, -c2)) : 0.f;
      const __nv_bfloat16 wb = __float2bfloat16_rn(w);
      sum[r] += __bfloat162float(wb);
      if (r < rows) *reinterpret_cast<__nv_bfloat16*>(pb + r * 128 + (((kc >> 3) ^ (r & 7)) << 4)) = wb;
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float s = sum[r];
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) red[t / 32][r] = s;
  }
  __syncthreads();
  if (t < rows) {
    float s = 0.f;
    for (int i = 0; i < kWThreads / 32; ++i) s += red[i][t];
    a.den[((size_t)hl * a.rows_tot + prow + t) * a.spans + span] = s;
    if (not_unit(s, min(key0 + a.span_keys, tr.pos0 + t + 1) - key0)) record_error(a.p.err, kErrValue | kKernPaged);
  }
}

// ============================================================================== gates

constexpr int kStages = 4;
constexpr uint32_t kABytes = kM * 128;       // 16 KB of P
constexpr uint32_t kBBytes = kK * kN * 2;    // 32 KB of G
constexpr uint32_t kTurnBytes = 8 * 4096;    // epilogue: 32 rows x 32 columns in f32 per warp
constexpr int kGThreads = 512;
constexpr int kJobSlots = 4;
constexpr int kNearEnd = 12;  // steps of a job that are left when the next one is taken
constexpr int kSched = 2, kProducers = 2, kEpi0 = 4, kScrub0 = 12;  // warps (producers: 0 and 3)

struct Job {
  int b, row0, rows, pos0, hl, strip, it0, it1, nc, c, tile, prow;  // b < 0: no more jobs
};

struct __align__(8) GBars {
  uint64_t full[kStages], empty[kStages];
  uint64_t dirty_full[kStages], clean[kStages];  // of the dirty steps' G, a ring of their own
  uint64_t acc_full[2], acc_empty[2];
  uint64_t job_full[kJobSlots], job_empty[kJobSlots];
  uint64_t near_end;  // the producers are in a job's last steps: time to take the next one
  uint64_t drain, never;
  uint32_t tmem_base;
  int abort;
  int last[2];
  Job job[kJobSlots];
  int page[kJobSlots][32];  // pages of a job's first 32 boxes
  // Whether the scrub warps took something out of job n's products, at n % 8, for each half of
  // the epilogue, which clears its entry.  Job n + 8 is not copied before both are through
  // with job n (two accumulators and at most 4 steps lie between).
  int poison[2][8];
};
// With the weights kernel's shared memory this exceeds an SM's, so a CTA of this kernel that
// is launched early never sits beside one of that kernel's (which may still have to
// allocate its tensor memory).
constexpr size_t kGSmem = 1024 + kStages * (size_t)(kABytes + kBBytes) + kTurnBytes + sizeof(GBars);
static_assert(kGSmem <= 232448, "shared memory budget");
static_assert(kGSmem + kWSmem > 233472, "the two kernels never share an SM");

// A bounded wait.  The wall clock is read only every 64 tries: a read takes longer than
// the hand-over between two roles does.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, GBars& b, const TcArgs& a) {
  uint64_t t0 = 0;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*(volatile int*)&b.abort) return false;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    else if (now - t0 > a.timeout_ns) break;
  }
  *(volatile int*)&b.abort = 1;
  record_error(a.p.err, kErrTimeout | kKernPaged);
  return false;
}

// The same for a whole warp: one lane polls, every lane returns its answer.  What the barrier
// guards (jobs, pages, copied gates) is read by all lanes: __syncwarp hands the polling lane's
// view of memory to the others, which the shuffle does not.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, GBars& b, const TcArgs& a) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = wait_bar(bar, parity, b, a);
  __syncwarp();
  return __shfl_sync(0xffffffffu, ok, 0);
}

// 64-key steps of a tile that sees keys [0, vis): at least one, so that rows without keys
// are written too.
__device__ __forceinline__ int steps_of(int vis) { return max(1, (vis + kK - 1) / kK); }

// A sequence's row tiles of this pass, [t0, t1).
struct SeqTiles {
  int t0, t1;
};
__device__ __forceinline__ SeqTiles seq_tiles(const TcArgs& a, const PagedSeq& s, int b) {
  const int at = scratch_row(a, s.r0, b), mt = (s.n + kM - 1) / kM;
  SeqTiles t;
  t.t0 = min(mt, (max(0, -at) + kM - 1) / kM);
  t.t1 = max(t.t0, min(mt, (max(0, a.rows - at) + kM - 1) / kM));
  return t;
}
// Keys that a sequence's tiles up to t1 see.
__device__ __forceinline__ int seq_vis(const PagedSeq& s, int t1) { return s.len - s.n + min(s.n, t1 * kM); }
// Steps of one (head, strip) of a sequence's tiles [t0, t1): whole tiles, each two steps more
// than the one before, and the last one.
__device__ __forceinline__ long long seq_steps(const PagedSeq& s, const SeqTiles& t) {
  if (t.t0 >= t.t1) return 0;
  const long long before = max(0, s.len - s.n + kK - 1) / kK, x = t.t0, y = t.t1 - 1;
  return (y - x) * before + y * (y + 1) - x * (x + 1) + steps_of(seq_vis(s, t.t1));
}

// Key ranges of a tile of u steps: as many as of `range` steps come nearest.
__device__ __forceinline__ int ranges_of(int u, int range) { return max(1, (u + range / 2) / range); }

struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++stage == n) { stage = 0; phase ^= 1; }
  }
};

// A tile's steps from this one on are dirty: they hold keys that some of its rows do not
// see (and slots past the sequence's length).
__device__ __forceinline__ int first_dirty(int pos0) { return pos0 < 0 ? 0 : (pos0 + 1) / kK; }

__device__ __forceinline__ int job_cols(const TcArgs& a, const Job& j) { return min(kN, a.m_h - j.strip * kN); }

// Of a pair of bf16: bits 15 and 31 set for a half whose exponent is all ones (an infinity or
// NaN), and the pair with such halves zeroed.
__device__ __forceinline__ uint32_t non_finite(uint32_t x) { return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
__device__ __forceinline__ uint32_t drop(uint32_t x) { return x & ~((non_finite(x) >> 15) * 0xffffu); }

// Page of box x (br keys) of a sequence; n_pages, which TMA reads as zeros, for a box past
// box1 and for an entry that is not a page.
__device__ __forceinline__ int box_page(const TcArgs& a, int b, int box, int box1) {
  if (box >= box1) return a.p.n_pages;
  const int pg = paged_page(a.p, b, box * a.box_rows / a.p.page_size);
  return pg < 0 ? a.p.n_pages : pg;
}
// Boxes of a sequence up to the end of a job's keys.
__device__ __forceinline__ int job_boxes(const TcArgs& a, const Job& j) {
  const int vis = j.pos0 + j.rows;
  return vis <= 0 ? 0 : (min(j.it1 * kK, vis) + a.box_rows - 1) / a.box_rows;
}

// Warp kSched: takes jobs from the counter, works out what they are and hands them to the
// other roles.
__device__ __forceinline__ void schedule(const TcArgs& a, GBars& b, int lane) {
  // steps of the whole launch, and from them the steps of a key range
  const int HS = a.heads * a.strips;
  long long total = 0;
  for (int i = lane; i < a.p.B; i += 32) {
    const PagedSeq s = paged_seq(a.p, i, false);
    total += seq_steps(s, seq_tiles(a, s, i));
  }
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  total *= HS;
  const long long want = a.jobs_per_sm * (long long)gridDim.x;
  const int range = (int)max((long long)a.min_steps, (total + want - 1) / want);

  // a window of 32 sequences, one per lane: rows, length, jobs (inclusive prefix)
  int w0 = -32;
  long long jbase = 0, jend = 0, pre = 0;
  PagedSeq ws{0, 0, 0};
  SeqTiles wt{0, 0};
  Ring jr;
  bool first = true;
  uint32_t taken = 0;        // jobs handed out and nearly copied
  long long j = blockIdx.x;  // then from the counter, gridDim.x on
  while (true) {
    while (j >= jend && w0 + 32 < a.p.B) {
      w0 += 32;
      jbase = jend;
      long long jobs = 0;
      if (w0 + lane < a.p.B) {
        ws = paged_seq(a.p, w0 + lane, false);
        wt = seq_tiles(a, ws, w0 + lane);
        jobs = (long long)(wt.t1 - wt.t0) * ranges_of(steps_of(seq_vis(ws, wt.t1)), range) * HS;
      }
      pre = jobs;
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += x;
      }
      jend = jbase + __shfl_sync(0xffffffffu, pre, 31);
    }
    Job job;
    job.b = -1;
    bool skip = false;
    if (j < jend) {
      const long long rel = j - jbase;
      const int owner = __popc(__ballot_sync(0xffffffffu, pre <= rel));
      const long long before = __shfl_sync(0xffffffffu, pre, owner > 0 ? owner - 1 : 0);
      const int idx = (int)(rel - (owner > 0 ? before : 0));
      const int r0 = __shfl_sync(0xffffffffu, ws.r0, owner), n = __shfl_sync(0xffffffffu, ws.n, owner);
      const int len = __shfl_sync(0xffffffffu, ws.len, owner), t1 = __shfl_sync(0xffffffffu, wt.t1, owner);
      const int mt = t1 - __shfl_sync(0xffffffffu, wt.t0, owner);
      // row tiles of a strip side by side (they share G in L2), then the strips of the same
      // keys (they share DRAM pages), then the key ranges; later row tiles, the longer ones,
      // come first
      const int ti = t1 - 1 - idx % mt, hs = idx / mt % HS;
      job.c = idx / mt / HS;
      job.b = w0 + owner;
      job.row0 = r0 + ti * kM;
      job.rows = min(kM, n - ti * kM);
      job.pos0 = len - n + ti * kM;
      job.hl = hs / a.strips;
      job.strip = hs - job.hl * a.strips;
      const int u = steps_of(job.pos0 + job.rows);
      job.nc = min(ranges_of(u, range), a.nc_cap);
      job.it0 = (int)((long long)u * job.c / job.nc);  // never empty: u >= nc
      job.it1 = (int)((long long)u * (job.c + 1) / job.nc);
      job.tile = r0 / kM + job.b + ti;
      job.prow = scratch_row(a, r0, job.b) + ti * kM;
      skip = job.c >= job.nc;  // a tile of the sequence that sees fewer keys
    }
    if (!skip) {
      const int box = job.it0 * (kK / a.box_rows) + lane;
      const int page = job.b < 0 ? 0 : box_page(a, job.b, box, job_boxes(a, job));
      if (!warp_wait(&b.job_empty[jr.stage], jr.phase ^ 1, b, a)) break;
      b.page[jr.stage][lane] = page;
      if (lane == 0) b.job[jr.stage] = job;
      __syncwarp();
      if (lane == 0) mbar_arrive(&b.job_full[jr.stage]);
      jr.next(kJobSlots);
      if (job.b < 0) break;
    }
    if (first) griddep_wait();  // the counters are the weights kernel's
    first = false;
    // no earlier: a CTA that held jobs in advance would leave others without
    if (!skip) {
      if (!warp_wait(&b.near_end, taken & 1, b, a)) break;
      ++taken;
    }
    int nxt = 0;
    if (lane == 0) nxt = atomicAdd(a.next, 1);
    j = (long long)gridDim.x + __shfl_sync(0xffffffffu, nxt, 0);
  }
  if (first) griddep_wait();
}

// Warps 0 and 3: copy each step's P and G, in turn.
__device__ __forceinline__ void produce(const TcArgs& a, GBars& b, uint8_t* sA, uint8_t* sB, const CUtensorMap* tmG,
                                        const CUtensorMap* tmG4, int part, int lane) {
  Ring st, jr, dr;
  uint32_t issued_mask = 0, issued_phase = 0;  // bits 0..: full, 8..: dirty_full
  bool ok = true, waited = false;
  int turn = 0;                              // whose step it is
  const int br = a.box_rows, spp = kK / br;  // boxes of a step
  const int win = 32 / spp;                  // steps of a window of 32 boxes
  const int lane_step = lane / spp, lane_dst = (lane - lane_step * spp) * (4 * br * 128);
  while (ok) {
    if (!(ok = warp_wait(&b.job_full[jr.stage], jr.phase, b, a))) break;
    const Job job = b.job[jr.stage];
    int page = b.page[jr.stage][lane], page2 = a.p.n_pages;  // this window's, and the next one's
    if (job.b < 0) break;
    const int nbc = (job_cols(a, job) + 63) / 64, head = a.h0 + job.hl, x0 = job.strip * kN;
    const bool whole = x0 + kN <= a.m_h;  // the strip's four 64-column boxes in one copy
    const int box1 = job_boxes(a, job), r8 = up8(job.rows);
    const uint32_t pbytes = job.pos0 + job.rows > 0 ? (uint32_t)r8 * 128 : 0u;
    const uint32_t box_bytes = (uint32_t)(whole ? 4 : nbc) * br * 128;
    const uint8_t* psrc = p_block(a, job.hl, job.prow, r8, job.it0);
    const int dirty = first_dirty(job.pos0), nsteps = job.it1 - job.it0;
    bool told = false;  // that the job nears its end
    for (int w = 0; w < nsteps && ok; w += win) {
      const int box = (job.it0 + w) * spp + lane, prw = box * br % a.p.page_size;
      if (w + win < nsteps) page2 = box_page(a, job.b, box + 32, box1);
      const bool there = box < box1;
      const int wn = min(win, nsteps - w);
      for (int i = 0; i < wn; ++i) {
        const bool is_dirty = job.it0 + w + i >= dirty;
        if (turn == part) {
          if (w + i >= nsteps - kNearEnd && !told) {
            told = true;
            if (lane == 0) mbar_arrive(&b.near_end);
          }
          if (waited && !__all_sync(0xffffffffu, mbar_try_wait(&b.empty[st.stage], st.phase ^ 1))) {
            ok = warp_wait(&b.empty[st.stage], st.phase ^ 1, b, a);
            if (!ok) break;
          }
          uint64_t* gbar = is_dirty ? &b.dirty_full[dr.stage] : &b.full[st.stage];
          const bool issue = there && lane_step == i;
          const uint32_t gbytes = __popc(__ballot_sync(0xffffffffu, issue)) * box_bytes;
          if (lane == 0) {
            mbar_arrive_expect_tx(&b.full[st.stage], pbytes + (is_dirty ? 0u : gbytes));
            if (is_dirty) mbar_arrive_expect_tx(gbar, gbytes);
            if (pbytes && waited) bulk_load(sA + st.stage * kABytes, psrc, pbytes, &b.full[st.stage]);
          }
          __syncwarp();
          if (issue) {
            uint8_t* dst = sB + st.stage * kBBytes + lane_dst;
            if (whole) {
              tma_load_5d(dst, tmG4, gbar, 0, prw, x0 / 64, head, page);
            } else {
              for (int c = 0; c < nbc; ++c) tma_load_4d(dst + c * br * 128, tmG, gbar, x0 + c * 64, head, prw, page);
            }
          }
        }
        // (each producer keeps count of all steps: which fill of a stage is the last one)
        issued_mask |= 1u << st.stage;
        issued_phase = (issued_phase & ~(1u << st.stage)) | (st.phase << st.stage);
        if (is_dirty) {
          issued_mask |= 256u << dr.stage;
          issued_phase = (issued_phase & ~(256u << dr.stage)) | (dr.phase << (dr.stage + 8));
          dr.next(kStages);
        }
        st.next(kStages);
        if (++turn == kProducers) turn = 0;
        psrc += (size_t)r8 * 128;
        if (!waited && w + i + 1 == min(nsteps, kStages)) {
          // the first stages' G is on its way; their P once the weights are there
          griddep_wait();
          waited = true;
          if (lane == 0 && pbytes)
            for (int x = part; x <= w + i; x += kProducers)
              bulk_load(sA + x * kABytes, p_block(a, job.hl, job.prow, r8, job.it0 + x), pbytes, &b.full[x]);
        }
      }
      page = page2;
    }
    if (!told && lane == 0) mbar_arrive(&b.near_end);  // (none of the last steps was this warp's)
    __syncwarp();
    if (lane == 0) mbar_arrive(&b.job_empty[jr.stage]);
    jr.next(kJobSlots);
  }
  if (!waited) griddep_wait();
  // copies still in flight must land before the CTA exits
  for (int s = 0; s < kStages; ++s) {
    if (issued_mask >> s & 1) mbar_wait(&b.full[s], issued_phase >> s & 1, a.timeout_ns);
    if (issued_mask >> (s + 8) & 1) mbar_wait(&b.dirty_full[s], issued_phase >> (s + 8) & 1, a.timeout_ns);
  }
}

// Warp 1, one thread: issues the products.
__device__ __forceinline__ void multiply(const TcArgs& a, GBars& b, const uint8_t* sA, const uint8_t* sB, uint32_t tmem) {
  // Descriptors stay in registers: stages and k-steps differ in the start address alone,
  // whose field (bytes / 16, shared memory < 256 KB) never carries.  G lies as [box of br
  // keys][64-column chunk][key][128 bytes]: 64-column chunks are br * 128 bytes apart, 8-key
  // groups 1024 (or, in boxes of 8 keys, a whole box).
  const int br = a.box_rows;
  const uint64_t pd0 = smem_desc(smem_u32(sA), 16, 1024, kSwizzle128B);
  const uint64_t gd0 = smem_desc(smem_u32(sB), br * 128, br == 8 ? 4096u : 1024u, kSwizzle128B);
  uint32_t koff[4];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    const int key = kk * 16, box = key / br;
    koff[kk] = (uint32_t)(box * (4 * br * 128) + (key - box * br) * 128) >> 4;
  }
  Ring st, jr, acc, dr;
  bool ok = !a.debug_timeout || wait_bar(&b.never, 0, b, a);  // nothing ever arrives there
  while (ok) {
    if (!(ok = wait_bar(&b.job_full[jr.stage], jr.phase, b, a))) break;
    const Job job = b.job[jr.stage];
    if (job.b < 0) break;
    const int vis = job.pos0 + job.rows;
    const uint32_t idesc = idesc_bf16_f32(kM, (job_cols(a, job) + 15) & ~15, false, true);
    const uint32_t d = tmem + acc.stage * kN;
    if (!(ok = wait_bar(&b.acc_empty[acc.stage], acc.phase ^ 1, b, a))) break;
    tc_fence_after_nc();
    uint32_t accum = 0;  // of a step's first k-step
    int it = job.it0;
    for (const int e = min(first_dirty(job.pos0), job.it1); it < e; ++it) {
      if (!(ok = wait_bar(&b.full[st.stage], st.phase, b, a))) break;
      tc_fence_after_nc();
      const uint64_t pd = pd0 + (uint64_t)(st.stage * (kABytes >> 4)), gd = gd0 + (uint64_t)(st.stage * (kBBytes >> 4));
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) mma_bf16_ss_nc(d, pd + kk * 2, gd + koff[kk], idesc, accum | (uint32_t)(kk > 0));
      accum = 1;
      mma_commit_nc(&b.empty[st.stage]);
      st.next(kStages);
    }
    for (; ok && it < job.it1; ++it) {
      if (!(ok = wait_bar(&b.full[st.stage], st.phase, b, a))) break;
      if (!(ok = wait_bar(&b.clean[dr.stage], dr.phase, b, a))) break;
      dr.next(kStages);
      tc_fence_after_nc();
      const uint64_t pd = pd0 + (uint64_t)(st.stage * (kABytes >> 4)), gd = gd0 + (uint64_t)(st.stage * (kBBytes >> 4));
      const int keys = vis - it * kK;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        if (kk * 16 < keys) mma_bf16_ss_nc(d, pd + kk * 2, gd + koff[kk], idesc, accum | (uint32_t)(kk > 0));
      accum = 1;
      mma_commit_nc(&b.empty[st.stage]);
      st.next(kStages);
    }
    if (!ok) break;
    mma_commit(&b.acc_full[acc.stage]);
    mbar_arrive(&b.job_empty[jr.stage]);
    acc.next(2);
    jr.next(kJobSlots);
  }
  mma_commit(&b.drain);
  mbar_wait(&b.drain, 0, a.timeout_ns);
}

// Warps 12-15: dirty steps.
__device__ __forceinline__ void scrub(const TcArgs& a, GBars& b, uint8_t* sB, int t, int lane) {
  const int br = a.box_rows;
  Ring jr, dr;
  int step = 0;  // steps before the job, modulo the stages
  int n = 0;     // jobs before
  bool ok = true;
  while (ok) {
    if (!(ok = warp_wait(&b.job_full[jr.stage], jr.phase, b, a))) break;
    const Job job = b.job[jr.stage];
    if (job.b < 0) break;
    const int nbc = (job_cols(a, job) + 63) / 64;
    for (int it = max(job.it0, first_dirty(job.pos0)); it < job.it1; ++it) {
      if (!(ok = warp_wait(&b.dirty_full[dr.stage], dr.phase, b, a))) break;
      const int keys = min(kK, max(0, job.pos0 + job.rows - it * kK)), rows = (keys + 15) & ~15;
      const int lo = max(0, job.pos0 + 1 - it * kK);  // rows before are seen by all
      const uint32_t s0 = smem_u32(sB + ((step + it - job.it0) % kStages) * kBBytes);
      // rows t / 8 + 16 k: their 16-byte pieces are on their way before the first is looked
      // at (this stands between a step's copy and its product)
      bool found = false;
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2) {
        uint4 x[2][4];
        uint32_t at[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = t / 8 + 16 * (2 * k2 + k), box = r / br;
          at[k] = s0 + box * (4 * br * 128) + (r - box * br) * 128 + (t & 7) * 16;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            x[k][c] = c < nbc && r >= lo && r < keys ? ld_shared_v4(at[k] + c * br * 128) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = t / 8 + 16 * (2 * k2 + k);
          uint32_t any = 0;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            any |= non_finite(x[k][c].x) | non_finite(x[k][c].y) | non_finite(x[k][c].z) | non_finite(x[k][c].w);
          if (r >= keys && r < rows) {
#pragma unroll
            for (int c = 0; c < 4; ++c) st_shared_v4(at[k] + c * br * 128, make_uint4(0, 0, 0, 0));
          } else if (any) {
            found = true;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              st_shared_v4(at[k] + c * br * 128, make_uint4(drop(x[k][c].x), drop(x[k][c].y), drop(x[k][c].z), drop(x[k][c].w)));
          }
        }
      }
      if (found) {
        *(volatile int*)&b.poison[0][n & 7] = 1;
        *(volatile int*)&b.poison[1][n & 7] = 1;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b.clean[dr.stage]);
      dr.next(kStages);
    }
    if (!ok) break;
    step = (step + job.it1 - job.it0) % kStages;
    ++n;
    __syncwarp();
    if (lane == 0) mbar_arrive(&b.job_empty[jr.stage]);
    jr.next(kJobSlots);
  }
}

// Warps 4-11: accumulators to outputs, or to partial sums.  Two halves of four warps take 128
// columns each and know nothing of each other: a load waits for thousands of cycles behind
// the copies, and twice the warps have twice the loads on their way.
__device__ __forceinline__ void finish_tiles(const TcArgs& a, GBars& b, uint8_t* sTurn, uint32_t tmem, int warp, int lane) {
  const int g = (warp - kEpi0) / 4, bar = 1 + g;
  const int quarter = warp & 3, r = quarter * 32 + lane;  // TMEM lane, the tile's row
  const bool lead = quarter == 0 && lane == 0;
  constexpr int kHalfN = kN / 2;
  const size_t width = (size_t)a.H * a.m_pitch;
  Ring jr, acc;
  for (int n = 0;; ++n) {
    bool ok = warp_wait(&b.job_full[jr.stage], jr.phase, b, a);
    const Job job = b.job[jr.stage];
    const bool is_job = ok && job.b >= 0;
    const int cols = is_job ? min(kHalfN, max(0, job_cols(a, job) - g * kHalfN)) : 0;
    // v's rows of the tile come into L2 while the products run
    if (a.v && cols > 0 && r < job.rows) {
      const char* vp = reinterpret_cast<const char*>(a.v + (size_t)(job.row0 + r) * a.v_pitch +
                                                     (size_t)(a.h0 + job.hl) * a.m_pitch + job.strip * kN + g * kHalfN);
      for (int x = 0; x < cols * 2; x += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(vp + x));
    }
    // In row order this lane takes 4 columns of rows quarter * 32 + lane / 8 + 4 k.  v of the
    // first 64 columns is on its way before the products are done, that of the others while
    // the first are finished.
    const int lr = quarter * 32 + lane / 8, lc = (lane & 7) * 4;
    const bool turned = is_job && job.rows > kFewRows && quarter * 32 < job.rows && cols > 0;
    uint2 vr[2][8];
    // v of such a row's columns c .. c + 3; rows and columns that are not there read ones that
    // are (no branch, so that the loads go out together)
    auto load_v = [&](int k, int c) -> uint2 {
      const int rr = min(lr + 4 * k, job.rows - 1), cc = min(c, (cols - 1) & ~3);
      const __nv_bfloat16* vp = a.v + (size_t)(job.row0 + rr) * a.v_pitch + (size_t)(a.h0 + job.hl) * a.m_pitch +
                                job.strip * kN + g * kHalfN + cc;
      if (a.v_vec) return *reinterpret_cast<const uint2*>(vp);
      uint32_t w[2];
#pragma unroll
      for (int q = 0; q < 2; ++q)
        w[q] = pack_bf16x2(__bfloat162float(vp[2 * q]), cc + 2 * q + 1 < cols ? __bfloat162float(vp[2 * q + 1]) : 0.f);
      return make_uint2(w[0], w[1]);
    };
    auto load_v64 = [&](int c0) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 8; ++k) vr[h][k] = load_v(k, c0 + h * 32 + lc);
    };
    if (a.v && turned) load_v64(0);
    if (is_job) ok = warp_wait(&b.acc_full[acc.stage], acc.phase, b, a);
    if (!named_bar_and(bar, 128, ok)) break;
    if (job.b < 0) break;
    tc_fence_after();
    const bool poison = *(volatile int*)&b.poison[g][n & 7] != 0;
    const int vis = job.pos0 + job.rows, head = a.h0 + job.hl, pos = job.pos0 + r, r8 = up8(job.rows);
    const uint32_t trow = tmem + acc.stage * kN + g * kHalfN + ((uint32_t)(quarter * 32) << 16);
    const bool warp_rows = quarter * 32 < job.rows;  // else this warp's rows are not there
    const bool live = r < job.rows;
    const size_t tkey = (((size_t)job.hl * a.strips + job.strip) * a.tiles + job.tile) * 2 + g;
    const size_t col0 = (size_t)head * a.m_pitch + job.strip * kN + g * kHalfN;
    const float* den = a.den + ((size_t)job.hl * a.rows_tot + job.prow) * a.spans;
    const int ns = vis <= 0 ? 0 : (vis + a.span_keys - 1) / a.span_keys;
    const float null_w = a.null_bias ? expf(a.null_bias[head] - head_tau(a.tau, a.s, head, a.p.err, kKernPaged)) : 0.f;

    // The keys whose non-finite gates the scrub warps took out of this job's product.
    const int bad0 = max(job.pos0 + 1, job.it0 * kK), bad1 = min(vis, job.it1 * kK);
    // The accumulator's 32 columns from c0 on of row r, with what was taken out put back
    // where the row sees it.
    auto fetch = [&](int c0, float (&y)[32]) {
      uint32_t x[32];
      __syncwarp();
      tmem_ld32(trow + c0, x);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 32; ++c) y[c] = __uint_as_float(x[c]);
      if (poison && live) {
        for (int key = bad0; key < min(bad1, pos + 1); ++key) {
          const int pi = key / a.p.page_size, pg = paged_page(a.p, job.b, pi);
          if (pg < 0) continue;
          const __nv_bfloat16* g = a.g_pages + ((size_t)pg * a.p.page_size + (key - pi * a.p.page_size)) * width + col0 + c0;
          const int kc = key % kK;
          const float w = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(
              p_block(a, job.hl, job.prow, r8, key / kK) + r * 128 + ((((kc >> 3) ^ (r & 7)) << 4) | ((kc & 7) * 2))));
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float gv = c0 + c < cols ? __bfloat162float(g[c]) : 0.f;
            if (!isfinite(gv)) y[c] += w * gv;
          }
        }
      }
    };
    // A key range's slot for its partial sums, and, once they are written, whether this is
    // the tile's last range to finish, which joins them all.
    auto take_slot = [&]() -> int {
      if (lead) {
        const int sl = atomicAdd(a.next + 1, 1);
        // (never by the plan's count; a sum that is not kept must not pass unseen)
        if ((unsigned)sl >= (unsigned)a.n_slots) record_error(a.p.err, kErrValue | kKernPaged);
        a.slot[tkey * a.nc_cap + job.c] = sl;
        b.last[g] = sl;
      }
      named_bar_sync(bar, 128);
      return b.last[g];
    };
    auto is_last = [&]() -> bool {
      __threadfence();
      named_bar_sync(bar, 128);
      if (lead) {
        b.last[g] = atomicAdd(a.done + tkey, 1) == job.nc - 1;
        __threadfence();
      }
      named_bar_sync(bar, 128);
      return b.last[g] != 0;
    };
    // slots of kSlotRegs ranges, looked up side by side
    constexpr int kSlotRegs = 4;
    int sl_reg[kSlotRegs];
    auto slots = [&](int k0) {
#pragma unroll
      for (int k = 0; k < kSlotRegs; ++k) sl_reg[k] = k0 + k < job.nc ? __ldcg(a.slot + tkey * a.nc_cap + k0 + k) : -1;
    };

    if (job.rows <= kFewRows) {
      // ---- few rows: the accumulator's rows go to shared memory, then this thread takes
      // column t of each
      const int t = (threadIdx.x - kEpi0 * 32) & 127, c = t;
      float* turn = reinterpret_cast<float*>(sTurn + g * (kTurnBytes / 2));  // this half's own part
      static_assert(kFewRows * kHalfN * 4 <= kTurnBytes / 2, "a half's few rows fit its part");
      auto at = [](int row, int col) { return row * kHalfN + ((((col >> 2) ^ (row & 7)) << 2) | (col & 3)); };
      // v and the denominators' parts arrive meanwhile
      float vv[kFewRows], dn[kFewRows];
      auto ask = [&]() {
#pragma unroll
        for (int i = 0; i < kFewRows; ++i) {
          dn[i] = 0.f;
          vv[i] = 1.f;
          if (i < job.rows && job.pos0 + i >= 0) {
            for (int k = lane; k < ns; k += 32) dn[i] += __ldcg(den + (size_t)i * a.spans + k);
            if (a.v && c < cols) vv[i] = __bfloat162float(a.v[(size_t)(job.row0 + i) * a.v_pitch + col0 + c]);
          }
        }
      };
      if (job.nc == 1) ask();
      if (quarter == 0) {
        for (int c0 = 0; c0 < cols; c0 += 32) {
          float y[32];
          fetch(c0, y);
          if (live) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
              *reinterpret_cast<float4*>(turn + at(r, c0 + 4 * u)) =
                  make_float4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
          }
        }
      }
      named_bar_sync(bar, 128);
      bool finish = true;
      if (job.nc > 1) {
        const int sl = take_slot();
        float* dst = a.part + (size_t)sl * (kHalfN * a.r8cap);
        if ((unsigned)sl < (unsigned)a.n_slots) {
          for (int i = 0; i < job.rows; ++i) __stcg(dst + i * kHalfN + c, turn[at(i, c)]);
        }
        finish = is_last();
        if (finish) ask();
      }
      if (finish) {
        float y[kFewRows];
#pragma unroll
        for (int i = 0; i < kFewRows; ++i) y[i] = job.nc == 1 && i < job.rows ? turn[at(i, c)] : 0.f;
        for (int k0 = 0; job.nc > 1 && k0 < job.nc; k0 += kSlotRegs) {
          slots(k0);
#pragma unroll
          for (int k = 0; k < kSlotRegs; ++k) {
            if ((unsigned)sl_reg[k] >= (unsigned)a.n_slots) continue;
            const float* src = a.part + (size_t)sl_reg[k] * (kHalfN * a.r8cap) + c;
#pragma unroll
            for (int i = 0; i < kFewRows; ++i) {
              if (i >= job.rows) break;
              y[i] += __ldcg(src + i * kHalfN);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kFewRows; ++i) {
          if (i >= job.rows) break;
          float d = dn[i];
          for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
          const int ps = job.pos0 + i;
          const float inv = 1.f / (d + (float)(ps + 1) * null_w);
          if (c < cols)
            a.out[(size_t)(job.row0 + i) * width + col0 + c] = __float2bfloat16_rn(ps >= 0 ? y[i] * inv * vv[i] : 0.f);
        }
      }
    } else {
      bool finish = true;
      if (job.nc > 1) {
        const int sl = take_slot();
        float* dst = a.part + (size_t)sl * (kHalfN * a.r8cap);
        if (warp_rows && (unsigned)sl < (unsigned)a.n_slots) {
          for (int c0 = 0; c0 < cols; c0 += 32) {
            float y[32];
            fetch(c0, y);
            if (r < r8) {
#pragma unroll
              for (int u = 0; u < 8; ++u)
                __stcg(reinterpret_cast<float4*>(dst) + (size_t)(c0 / 4 + u) * a.r8cap + r,
                       make_float4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]));
            }
          }
        }
        finish = is_last();
      }
      if (finish && warp_rows) {
        uint8_t* turn = sTurn + (warp - kEpi0) * 4096;
        const uint32_t t_s = smem_u32(turn);
        float inv = 0.f;
        if (live && pos >= 0) {
          float d = 0.f;
#pragma unroll 4
          for (int i = 0; i < ns; i += 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(den + (size_t)r * a.spans + i));
            d += x.x + (i + 1 < ns ? x.y : 0.f) + (i + 2 < ns ? x.z : 0.f) + (i + 3 < ns ? x.w : 0.f);
          }
          inv = 1.f / (d + (float)(pos + 1) * null_w);
        }
        for (int c64 = 0; c64 < cols; c64 += 64) {
          if (a.v && c64 > 0) load_v64(c64);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c0 = c64 + h * 32, c = c0 + lc;
            if (c0 >= cols) break;
            float y[32];
            if (job.nc == 1) {
              fetch(c0, y);
            } else {
#pragma unroll
              for (int q = 0; q < 32; ++q) y[q] = 0.f;
              for (int k0 = 0; k0 < job.nc; k0 += kSlotRegs) {
                if (c0 == 0 || job.nc > kSlotRegs) slots(k0);
#pragma unroll
                for (int k = 0; k < kSlotRegs; ++k) {
                  if (!live || (unsigned)sl_reg[k] >= (unsigned)a.n_slots) continue;
                  const float4* src = reinterpret_cast<const float4*>(a.part + (size_t)sl_reg[k] * (kHalfN * a.r8cap));
#pragma unroll
                  for (int u = 0; u < 8; ++u) {
                    const float4 x = __ldcg(src + (size_t)(c0 / 4 + u) * a.r8cap + r);
                    y[4 * u] += x.x; y[4 * u + 1] += x.y; y[4 * u + 2] += x.z; y[4 * u + 3] += x.w;
                  }
                }
              }
            }
            // a row without keys gives zeros, whatever its accumulator holds
            const bool seen = live && pos >= 0;
            __syncwarp();  // the previous columns have been read
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              uint32_t e[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) e[q] = seen ? __float_as_uint(y[4 * u + q] * inv) : 0u;
              st_shared_v4(t_s + lane * 128 + ((u ^ (lane & 7)) << 4), make_uint4(e[0], e[1], e[2], e[3]));
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int rw = lane / 8 + 4 * k, rr = quarter * 32 + rw;
              const uint4 x = ld_shared_v4(t_s + rw * 128 + (((lane & 7) ^ (rw & 7)) << 4));
              float z[4] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w)};
              if (a.v && job.pos0 + rr >= 0) {
                z[0] *= bf16lo(vr[h][k].x); z[1] *= bf16hi(vr[h][k].x);
                z[2] *= bf16lo(vr[h][k].y); z[3] *= bf16hi(vr[h][k].y);
              }
              // four columns: the last ones may run into the pitch's padding
              if (rr < job.rows && c < cols)
                *reinterpret_cast<uint2*>(a.out + (size_t)(job.row0 + rr) * width + col0 + c) =
                    make_uint2(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]));
            }
          }
        }
      }
    }
    if (poison) {  // (the same for the half's four warps, which have all read it)
      named_bar_sync(bar, 128);
      if (lead) b.poison[g][n & 7] = 0;
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&b.acc_empty[acc.stage]);
      mbar_arrive(&b.job_empty[jr.stage]);
    }
    acc.next(2);
    jr.next(kJobSlots);
  }
}

__global__ void __launch_bounds__(kGThreads, 1)
    paged_gates_kernel(const __grid_constant__ CUtensorMap tmG, const __grid_constant__ CUtensorMap tmG4, const TcArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = base;
  uint8_t* sB = base + kStages * kABytes;
  uint8_t* sTurn = sB + kStages * kBBytes;
  GBars& b = *reinterpret_cast<GBars*>(sTurn + kTurnBytes);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&b.full[s], 1);
      mbar_init(&b.empty[s], 1);
      mbar_init(&b.dirty_full[s], 1);
      mbar_init(&b.clean[s], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.acc_full[i], 1);
      mbar_init(&b.acc_empty[i], 8);
    }
    for (int i = 0; i < kJobSlots; ++i) {
      mbar_init(&b.job_full[i], 1);
      mbar_init(&b.job_empty[i], kProducers + 1 + 8 + 4);  // producers, MMA issuer, epilogue and scrub warps
    }
    mbar_init(&b.near_end, kProducers);
    mbar_init(&b.drain, 1);
    mbar_init(&b.never, 1);
    b.abort = 0;
    for (int i = 0; i < 16; ++i) (&b.poison[0][0])[i] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&b.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = b.tmem_base;

  // the epilogue's two warpgroups take registers that the other two do not need (2 x 128 x 80 +
  // 2 x 128 x 176 = the 65,536 that the block has)
  if (warp < kEpi0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 1) {
      if (lane == 0) multiply(a, b, sA, sB, tmem);
    } else if (warp == kSched) {
      schedule(a, b, lane);
    } else {
      produce(a, b, sA, sB, &tmG, &tmG4, warp == 0 ? 0 : 1, lane);
    }
  } else if (warp < kScrub0) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    finish_tiles(a, b, sTurn, tmem, warp, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    scrub(a, b, sB, threadIdx.x - kScrub0 * 32, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ============================================================================= launch

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Rows of a G box: the largest power of two that divides a page, at most a step.
int box_rows(int page_size) {
  int r = page_size & -page_size;
  return r > kK ? kK : r;
}

constexpr size_t kScratch = size_t(2) << 30;  // P of a pass

struct TcPlan {
  int rows_all, rows, rows_tot;  // scratch rows of a head: of all tiles; of a pass's starts; in a pass
  int key_blocks, span_keys, spans, strips, tiles, r8cap, min_steps, jobs_per_sm, nc_cap, n_slots, heads, grid;
  size_t P, den, part, slot, done, next, total;
};

TcPlan tc_plan(const PagedCall& c) {
  TcPlan l;
  const int sms = serve_sm_count();
  l.rows_all = up8(c.p.N) + 8 * c.p.B;
  l.key_blocks = ceil_div(c.p.max_len, kK);
  // at most 32 spans of whole 128-key blocks (their sums are added once per strip)
  l.span_keys = ceil_div(ceil_div(c.p.max_len, 32), 128) * 128;
  if (l.span_keys < 256) l.span_keys = 256;
  l.spans = (ceil_div(c.p.max_len, l.span_keys) + 3) & ~3;
  l.strips = ceil_div(c.m_h, kN);
  l.tiles = c.p.N / kM + c.p.B;
  l.r8cap = c.p.max_new < kM ? up8(c.p.max_new) : kM;
  // joining key ranges is cheap for few rows; for many it moves as much as their products
  // take, so tiles are left whole when they are about two per SM
  l.min_steps = 8;
  l.jobs_per_sm = l.r8cap <= kFewRows ? kJobsPerSm : 2;
  l.grid = sms;
  // A tile that is cut has at least 3/2 ranges' worth of steps and at most 4/3 as many ranges as
  // whole ones fit in it: together at most 4/3 of the jobs wanted.  Two halves each: 8/3 of them,
  // for 4.
  l.n_slots = 2 * 2 * kJobsPerSm * sms;
  // A pass takes as many heads as keep P within kScratch, or, where one does not, the tiles of
  // one head that start within so many rows (whole tiles' worth of starts: a tile's rows may
  // reach one tile further); never less than 128 starts, 256 rows.
  const size_t per_row = (size_t)l.key_blocks * 128, fit = kScratch / per_row;
  l.rows = l.rows_tot = l.rows_all;
  l.heads = 1;
  if (fit < (size_t)l.rows_all) {
    l.rows = fit < 3 * kM ? kM : (int)((fit - kM) / kM * kM);
    l.rows_tot = l.rows + kM;
  } else {
    l.heads = (int)(fit / l.rows_all > (size_t)c.H ? (size_t)c.H : fit / l.rows_all);
  }
  // A tile's steps are at most the launch's in one of its heads and strips, so that it has no
  // more ranges than the launch has jobs for each of these.
  const int least = (c.H % l.heads ? c.H % l.heads : l.heads) * l.strips;
  l.nc_cap = ceil_div(l.key_blocks, l.min_steps);
  if (l.nc_cap > l.jobs_per_sm * l.grid / least + 1) l.nc_cap = l.jobs_per_sm * l.grid / least + 1;
  const size_t tk = (size_t)l.heads * l.strips * l.tiles * 2;
  l.P = 0;
  l.den = l.P + align256((size_t)l.heads * l.rows_tot * per_row);
  l.part = l.den + align256((size_t)l.heads * l.rows_tot * l.spans * 4);
  l.slot = l.part + align256((size_t)l.n_slots * (kN / 2) * l.r8cap * 4);
  l.done = l.slot + align256(tk * l.nc_cap * 4);
  l.next = l.done + align256(tk * 4);
  l.total = l.next + 256;
  return l;
}

template <int DH>
void launch_weights_few_dh(const TcArgs& a, int rows, dim3 g, cudaStream_t s) {
  if (rows == 1) paged_weights_few_kernel<1, DH><<<g, kWThreads, 0, s>>>(a);
  else if (rows == 2) paged_weights_few_kernel<2, DH><<<g, kWThreads, 0, s>>>(a);
  else if (rows <= 4) paged_weights_few_kernel<4, DH><<<g, kWThreads, 0, s>>>(a);
  else paged_weights_few_kernel<8, DH><<<g, kWThreads, 0, s>>>(a);
}
void launch_weights_few(const TcArgs& a, int rows, dim3 g, cudaStream_t s) {
  if (a.d_h == 64) launch_weights_few_dh<64>(a, rows, g, s);
  else if (a.d_h == 32) launch_weights_few_dh<32>(a, rows, g, s);
  else launch_weights_few_dh<16>(a, rows, g, s);
}

// Both kernels' dynamic shared memory, allowed once per device.
cudaError_t allow_shared_memory() {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool kept = dev >= 0 && dev < 64;
  if (kept && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(paged_weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kWSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(paged_gates_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGSmem);
  if (e == cudaSuccess && kept) done[dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace

bool paged_tc_takes(tg_dtype dt, const PagedCall& c) {
  // the shape alone decides, so that the workspace can be sized without the pointers
  return dt == TG_BF16 && (c.d_h == 16 || c.d_h == 32 || c.d_h == 64) && c.m_pitch % 8 == 0 &&
         box_rows(c.p.page_size) >= 8;
}

size_t paged_tc_ws_bytes(const PagedCall& c) { return tc_plan(c).total; }

cudaError_t launch_paged_tc(const PagedCall& c, cudaStream_t s) {
  const TcPlan l = tc_plan(c);
  TcArgs a = {};
  a.p = c.p; a.H = c.H; a.d_h = c.d_h; a.m_h = c.m_h; a.m_pitch = c.m_pitch;
  a.rows = l.rows; a.rows_tot = l.rows_tot; a.key_blocks = l.key_blocks; a.span_keys = l.span_keys; a.spans = l.spans;
  a.strips = l.strips; a.tiles = l.tiles; a.r8cap = l.r8cap; a.min_steps = l.min_steps;
  a.jobs_per_sm = l.jobs_per_sm; a.nc_cap = l.nc_cap; a.n_slots = l.n_slots;
  a.box_rows = box_rows(c.p.page_size);
  a.s = c.s; a.tau = c.tau; a.null_bias = c.null_bias; a.v_pitch = c.v_pitch;
  a.v_vec = c.v && (reinterpret_cast<uintptr_t>(c.v) & 15u) == 0 && c.v_pitch % 8 == 0;
  a.q = static_cast<const __nv_bfloat16*>(c.q); a.v = static_cast<const __nv_bfloat16*>(c.v);
  a.out = static_cast<__nv_bfloat16*>(c.out);
  a.k_pages = static_cast<const __nv_bfloat16*>(c.k_pages); a.g_pages = static_cast<const __nv_bfloat16*>(c.g_pages);
  char* base = static_cast<char*>(c.ws);
  a.P = reinterpret_cast<uint8_t*>(base + l.P);
  a.den = reinterpret_cast<float*>(base + l.den);
  a.part = reinterpret_cast<float*>(base + l.part);
  a.slot = reinterpret_cast<int*>(base + l.slot);
  a.done = reinterpret_cast<int*>(base + l.done);
  a.next = reinterpret_cast<int*>(base + l.next);
  a.debug_timeout = c.debug_timeout;
  a.timeout_ns = c.debug_timeout ? 1000000ull : kTimeoutNs;

  CUtensorMap mG, mG4;
  cudaError_t e = make_tmap_4d_heads(&mG, c.g_pages, c.p.n_pages, c.p.page_size, c.H, c.m_h, c.m_pitch, a.box_rows, 64);
  mG4 = mG;  // used only where a head holds a whole strip
  if (e == cudaSuccess && c.m_h >= kN)
    e = make_tmap_5d_chunks(&mG4, c.g_pages, c.p.n_pages, c.p.page_size, c.H, c.m_h, c.m_pitch, a.box_rows, 4);
  if (e == cudaSuccess) e = allow_shared_memory();
  if (e != cudaSuccess) return e;
  for (a.h0 = 0; a.h0 < c.H; a.h0 += l.heads) {
    for (a.row0 = 0; a.row0 < l.rows_all; a.row0 += l.rows) {
      a.heads = c.H - a.h0 < l.heads ? c.H - a.h0 : l.heads;
      const dim3 gw(l.tiles, a.heads, ceil_div(c.p.max_len, l.span_keys));
      if (c.p.max_new > 8) paged_weights_kernel<<<gw, kWThreads, kWSmem, s>>>(a);
      else launch_weights_few(a, c.p.max_new, gw, s);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(l.grid);
      cfg.blockDim = dim3(kGThreads);
      cfg.dynamicSmemBytes = kGSmem;
      cfg.stream = s;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaLaunchKernelEx(&cfg, paged_gates_kernel, mG, mG4, a);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace tg

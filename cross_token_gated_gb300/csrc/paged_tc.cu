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
// paged_gates_kernel    U = P G: tiles of 128 rows x 256 gate columns, 64 keys a step.
//     warp 0     scheduler and TMA producer (4 stages of P 16 KB + G 32 KB): takes jobs from a
//                counter, looks up pages 32 at a time, one lane per page issues its boxes
//     warp 1     MMA issuer (128 x 256 x 16), two accumulators in TMEM
//     warps 2-5  epilogue: times 1 / den and v, bf16 out; or f32 partial sums of a key range
//     warps 6-9  scrub: only in steps with keys that some row of the tile does not see:
//                slots past the sequence's length become zeros, and non-finite gates of the
//                chunk's own tokens are taken out of the product (0 * NaN would reach rows
//                that do not see them); the epilogue adds them back to the rows that do
//
// A job is a (sequence, head, strip, key range, row tile) with the row tile fastest, so the
// CTAs that work side by side share their G out of L2.  Key ranges are cut so that there are
// about kJobsPerSm jobs per SM when the tiles alone would not fill the SMs; the job that
// finishes a tile last adds the ranges' partial sums in their order.
// Every wait is bounded; on expiry the kernel records a timeout in the error word.
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
constexpr int kJobsPerSm = 4;
constexpr int kMinSteps = 8;      // a key range is at least this many steps

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
  int rows_tot;              // scratch rows of a head: up8(N) + 8 B
  int key_blocks;            // ceil(max_len / 64)
  int span_keys, spans;      // of the weights kernel; spans: ceil(max_len / span_keys)
  int strips;                // ceil(m_h / 256)
  int tiles;                 // tile numbers: N / 128 + B
  int r8cap;                 // rows of a partial: min(128, up8(max_new))
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
  float* part;               // [slot][64][r8cap][4]
  int* slot;                 // [head][strip][tile][nc_cap]
  int* done;                 // [head][strip][tile]: ranges that are done
  int* next;                 // [0] next job, [1] next partial slot
  uint64_t timeout_ns;
};

// Scratch row of a sequence's first row: sequences start at multiples of 8.
__device__ __forceinline__ int scratch_row(int r0, int b) { return up8(r0) + 8 * b; }
// P of key block kb of a tile with r8 scratch rows.
__device__ __forceinline__ uint8_t* p_block(const TcArgs& a, int hl, int prow, int r8, int kb) {
  return a.P + (((size_t)hl * a.rows_tot + prow) * a.key_blocks + (size_t)kb * r8) * 128;
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
  uint64_t* bar = reinterpret_cast<uint64_t*>(sP + 2 * kM * 128);
  uint32_t* tm = reinterpret_cast<uint32_t*>(bar + 1);
  __shared__ float half_sum[kM];
  const int t = threadIdx.x, warp = t / 32, lane = t & 31;
  const int tile = blockIdx.x, hl = blockIdx.y, span = blockIdx.z, head = a.h0 + hl;

  griddep_launch();
  // the gates kernel's counters
  const size_t nd = (size_t)a.heads * a.strips * a.tiles;
  const size_t cta = ((size_t)span * gridDim.y + hl) * gridDim.x + tile, ctas = (size_t)gridDim.x * gridDim.y * gridDim.z;
  for (size_t i = cta * kWThreads + t; i < nd; i += ctas * kWThreads) a.done[i] = 0;
  if (cta == 0 && t < 2) a.next[t] = 0;

  const TileRef tr = find_tile<kM>(a.p, tile, hl == 0 && span == 0);
  const int vis = tr.pos0 + tr.n;
  const int key0 = span * a.span_keys, key1 = min(key0 + a.span_keys, (vis + 63) & ~63);
  if (tr.n == 0 || vis <= 0 || key0 >= vis) return;
  const PagedSeq sq = paged_seq(a.p, tr.b, false);
  const int prow = scratch_row(sq.r0, tr.b) + (tr.row0 - sq.r0), r8 = up8(tr.n);

  if (t == 0) {
    mbar_init(bar, 1);
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
    // one wait per warp; a bounded one, after which every warp leaves together below
    ok = mbar_wait(bar, n & 1, a.timeout_ns);
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
  if (wg == 0 && row < tr.n) a.den[((size_t)hl * a.rows_tot + prow + row) * a.spans + span] = sum + half_sum[row];
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

// ============================================================================== gates

constexpr int kStages = 4;
constexpr uint32_t kABytes = kM * 128;       // 16 KB of P
constexpr uint32_t kGBox = kK * 128;         // 8 KB: 64 keys x 64 columns
constexpr uint32_t kBBytes = 4 * kGBox;      // 32 KB
constexpr int kGThreads = 320;
constexpr int kJobSlots = 4;
constexpr int kEpi0 = 2, kScrub0 = 6;

struct Job {
  int b, row0, rows, pos0, hl, strip, it0, it1, nc, c, tile, prow;  // b < 0: no more jobs
  int poison;
};

struct __align__(8) GBars {
  uint64_t full[kStages], empty[kStages], clean[kStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t job_full[kJobSlots], job_empty[kJobSlots];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int last;
  Job job[kJobSlots];
};
// With the weights kernel's shared memory this exceeds an SM's, so a CTA of this kernel that
// is launched early never sits beside one of that kernel's (which may still have to
// allocate its tensor memory).
constexpr size_t kGSmem = 1024 + kStages * (size_t)(kABytes + kBBytes) + sizeof(GBars);
static_assert(kGSmem <= 232448, "shared memory budget");
static_assert(kGSmem + kWSmem > 233472, "the two kernels never share an SM");

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, GBars& b, const TcArgs& a) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*(volatile int*)&b.abort) return false;
  if (mbar_wait(bar, parity, a.timeout_ns)) return true;
  *(volatile int*)&b.abort = 1;
  record_error(a.p.err, kErrTimeout | kKernPaged);
  return false;
}

// The same for a whole warp: every lane returns the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, GBars& b, const TcArgs& a) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, b, a));
}

// 64-key steps of a tile that sees keys [0, vis): at least one, so that rows without keys
// are written too.
__device__ __forceinline__ int steps_of(int vis) { return max(1, (vis + kK - 1) / kK); }

// Steps of one (head, strip) of a sequence, all its tiles.
__device__ __forceinline__ long long seq_steps(const PagedSeq& s) {
  if (s.n == 0) return 0;
  const long long mt = (s.n + kM - 1) / kM, before = max(0, s.len - s.n + kK - 1) / kK;
  return (mt - 1) * before + mt * (mt - 1) + steps_of(s.len);
}

struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++stage == n) { stage = 0; phase ^= 1; }
  }
};

// The keys of a step that are there, and whether some row of the tile misses one of them.
__device__ __forceinline__ int step_keys(const Job& j, int it) { return min(kK, j.pos0 + j.rows - it * kK); }
__device__ __forceinline__ bool step_dirty(const Job& j, int it) { return it * kK + kK - 1 > j.pos0; }

__device__ __forceinline__ int job_cols(const TcArgs& a, const Job& j) { return min(kN, a.m_h - j.strip * kN); }

__device__ __forceinline__ bool bad_bits(uint32_t x, uint32_t m) { return (x & m) == m; }

__global__ void __launch_bounds__(kGThreads, 1)
    paged_gates_kernel(const __grid_constant__ CUtensorMap tmG, const TcArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = base;
  uint8_t* sB = base + kStages * kABytes;
  GBars& b = *reinterpret_cast<GBars*>(sB + kStages * kBBytes);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&b.full[s], 1);
      mbar_init(&b.empty[s], 5);  // the products' commit and the 4 scrub warps
      mbar_init(&b.clean[s], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.acc_full[i], 1);
      mbar_init(&b.acc_empty[i], 4);
    }
    for (int i = 0; i < kJobSlots; ++i) {
      mbar_init(&b.job_full[i], 1);
      mbar_init(&b.job_empty[i], 9);  // MMA issuer, 4 epilogue warps, 4 scrub warps
    }
    mbar_init(&b.drain, 1);
    b.abort = 0;
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

  if (warp == 0) {
    // ------------------------------------------------------------ scheduler, TMA producer
    // steps of the whole launch, and from them the steps of a key range
    const int HS = a.heads * a.strips;
    long long total = 0;
    for (int i = lane; i < a.p.B; i += 32) total += seq_steps(paged_seq(a.p, i, false));
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    total *= HS;
    const int range = (int)max((long long)kMinSteps, (total + kJobsPerSm * gridDim.x - 1) / (kJobsPerSm * (long long)gridDim.x));
    griddep_wait();  // P, den and the counters are the weights kernel's

    // a window of 32 sequences, one per lane: rows, length, jobs (inclusive prefix)
    int w0 = -32;
    long long jbase = 0, jend = 0, pre = 0;
    PagedSeq ws{0, 0, 0};
    int wmt = 0, wnc = 0;
    Ring st, jr;
    uint32_t issued_mask = 0, issued_phase = 0;
    bool ok = true;
    int nxt = 0;
    if (lane == 0) nxt = atomicAdd(a.next, 1);
    while (ok) {
      long long j = __shfl_sync(0xffffffffu, nxt, 0);
      if (lane == 0) nxt = atomicAdd(a.next, 1);  // the next job's number, while this one runs
      while (j >= jend && w0 + 32 < a.p.B) {
        w0 += 32;
        jbase = jend;
        long long jobs = 0;
        if (w0 + lane < a.p.B) {
          ws = paged_seq(a.p, w0 + lane, false);
          wmt = (ws.n + kM - 1) / kM;
          wnc = (steps_of(ws.len) + range - 1) / range;
          jobs = (long long)wmt * wnc * HS;
        }
        pre = jobs;
        for (int o = 1; o < 32; o <<= 1) {
          const long long x = __shfl_up_sync(0xffffffffu, pre, o);
          if (lane >= o) pre += x;
        }
        jend = jbase + __shfl_sync(0xffffffffu, pre, 31);
      }
      const bool none = j >= jend;
      Job job;
      job.b = -1;
      int r8 = 0;
      if (!none) {
        const long long rel = j - jbase;
        const int owner = __popc(__ballot_sync(0xffffffffu, pre <= rel));
        const long long before = __shfl_sync(0xffffffffu, pre, owner > 0 ? owner - 1 : 0);
        const int idx = (int)(rel - (owner > 0 ? before : 0));
        const int r0 = __shfl_sync(0xffffffffu, ws.r0, owner), n = __shfl_sync(0xffffffffu, ws.n, owner);
        const int len = __shfl_sync(0xffffffffu, ws.len, owner);
        const int mt = __shfl_sync(0xffffffffu, wmt, owner), nc = __shfl_sync(0xffffffffu, wnc, owner);
        const int i = idx % mt, hs = idx / mt / nc;
        job.c = idx / mt % nc;
        job.b = w0 + owner;
        job.row0 = r0 + i * kM;
        job.rows = min(kM, n - i * kM);
        job.pos0 = len - n + i * kM;
        job.hl = hs / a.strips;
        job.strip = hs - job.hl * a.strips;
        const int u = steps_of(job.pos0 + job.rows);
        job.nc = (u + range - 1) / range;
        job.it0 = job.c * range;
        job.it1 = min(u, job.it0 + range);
        job.tile = r0 / kM + job.b + i;
        job.prow = scratch_row(r0, job.b) + i * kM;
        job.poison = 0;
        if (job.c >= job.nc) continue;  // an earlier tile of the sequence sees fewer keys
        r8 = up8(job.rows);
      }
      ok = warp_wait(&b.job_empty[jr.stage], jr.phase ^ 1, b, a);
      if (!ok) break;
      if (lane == 0) {
        b.job[jr.stage] = job;
        mbar_arrive(&b.job_full[jr.stage]);
      }
      jr.next(kJobSlots);
      if (none) break;

      const int vis = job.pos0 + job.rows, cols = job_cols(a, job);
      const int nbc = (cols + 63) / 64, head = a.h0 + job.hl;
      const int br = a.box_rows, spp = kK / br;  // boxes of a step
      const int box1 = vis <= 0 ? 0 : (min(job.it1 * kK, vis) + br - 1) / br;
      int first = job.it0 * spp;  // box of lane 0
      auto lookup = [&](int box) -> int {
        if (box >= box1) return -1;
        const int key = box * br, pi = key / a.p.page_size;
        return paged_page(a.p, job.b, pi);
      };
      int page = lookup(first + lane);
      for (int it = job.it0; ok && it < job.it1; ++it) {
        if (it * spp >= first + 32) {
          first += 32;
          page = lookup(first + lane);
        }
        ok = warp_wait(&b.empty[st.stage], st.phase ^ 1, b, a);
        if (!ok) break;
        const int box0 = it * spp, nb = max(0, min(spp, box1 - box0));
        uint8_t* dB = sB + st.stage * kBBytes;
        // boxes whose page is not one of the pool are loaded as zeros (out of range)
        const uint32_t bytes = (uint32_t)(vis > 0 ? r8 * 128 : 0) + (uint32_t)(nb * nbc * br * 128);
        if (lane == 0) {
          mbar_arrive_expect_tx(&b.full[st.stage], bytes);
          if (vis > 0) bulk_load(sA + st.stage * kABytes, p_block(a, job.hl, job.prow, r8, it), r8 * 128, &b.full[st.stage]);
        }
        __syncwarp();
        const int mybox = first + lane;
        if (mybox >= box0 && mybox < box0 + nb) {
          const int key = mybox * br, r = key % a.p.page_size;
          const int pg = page < 0 ? a.p.n_pages : page;
          for (int c = 0; c < nbc; ++c)
            tma_load_4d(dB + c * kGBox + (mybox - box0) * br * 128, &tmG, &b.full[st.stage], job.strip * kN + c * 64,
                        head, r, pg);
        }
        issued_mask |= 1u << st.stage;
        issued_phase = (issued_phase & ~(1u << st.stage)) | (st.phase << st.stage);
        st.next(kStages);
      }
    }
    // copies still in flight must land before the CTA exits
    for (int s = 0; s < kStages; ++s)
      if (issued_mask >> s & 1) mbar_wait(&b.full[s], issued_phase >> s & 1, a.timeout_ns);
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      Ring st, jr, acc;
      uint32_t clean_phase = 0;
      bool ok = true;
      while (ok) {
        if (!(ok = wait_bar(&b.job_full[jr.stage], jr.phase, b, a))) break;
        const Job job = b.job[jr.stage];
        if (job.b < 0) break;
        const uint32_t idesc = idesc_bf16_f32(kM, (job_cols(a, job) + 15) & ~15, false, true);
        const uint32_t d = tmem + acc.stage * kN;
        if (!(ok = wait_bar(&b.acc_empty[acc.stage], acc.phase ^ 1, b, a))) break;
        for (int it = job.it0; it < job.it1; ++it) {
          if (!(ok = wait_bar(&b.full[st.stage], st.phase, b, a))) break;
          if (step_dirty(job, it)) {
            if (!(ok = wait_bar(&b.clean[st.stage], clean_phase >> st.stage & 1, b, a))) break;
            clean_phase ^= 1u << st.stage;
          }
          tc_fence_after();
          const uint32_t aa = smem_u32(sA + st.stage * kABytes), bb = smem_u32(sB + st.stage * kBBytes);
          const int ks = (step_keys(job, it) + 15) / 16;
          for (int kk = 0; kk < ks; ++kk)
            mma_bf16_ss(d, smem_desc(aa + kk * 32, 16, 1024, kSwizzle128B),
                        smem_desc(bb + kk * 2048, kGBox, 1024, kSwizzle128B), idesc, it != job.it0 || kk != 0);
          mma_commit(&b.empty[st.stage]);
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
  } else if (warp < kScrub0) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const bool lead = warp == kEpi0 && lane == 0;
    Ring jr, acc;
    while (true) {
      bool ok = wait_bar(&b.job_full[jr.stage], jr.phase, b, a);
      const Job job = b.job[jr.stage];
      if (ok && job.b >= 0) ok = wait_bar(&b.acc_full[acc.stage], acc.phase, b, a);
      if (!named_bar_and(1, 128, ok)) break;
      if (job.b < 0) break;
      tc_fence_after();
      const bool poison = *(volatile int*)&b.job[jr.stage].poison != 0;
      const int vis = job.pos0 + job.rows, cols = job_cols(a, job), head = a.h0 + job.hl, pos = job.pos0 + r;
      const int r8 = up8(job.rows);
      const uint32_t trow = tmem + acc.stage * kN + ((uint32_t)(quarter * 32) << 16);
      const bool warp_rows = quarter * 32 < job.rows;  // else this warp's rows are not there
      const bool live = r < job.rows;
      const size_t tkey = ((size_t)job.hl * a.strips + job.strip) * a.tiles + job.tile;
      const size_t width = (size_t)a.H * a.m_pitch;

      // the accumulator's 32 columns from c0 on of this thread's row, with the non-finite
      // gates that the scrub warps took out put back where the row sees them
      auto fetch = [&](int c0, float (&y)[32]) {
        uint32_t x[32];
        __syncwarp();
        tmem_ld32(trow + c0, x);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 32; ++c) y[c] = __uint_as_float(x[c]);
        if (poison && live) {
          const int k1 = min(min(pos, vis - 1), job.it1 * kK - 1);
          for (int key = max(job.pos0 + 1, job.it0 * kK); key <= k1; ++key) {
            const int pi = key / a.p.page_size, pg = paged_page(a.p, job.b, pi);
            if (pg < 0) continue;
            const uint8_t* pb = p_block(a, job.hl, job.prow, r8, key / kK) + r * 128;
            const int kc = key % kK;
            const float w = __bfloat162float(
                *reinterpret_cast<const __nv_bfloat16*>(pb + ((((kc >> 3) ^ (r & 7)) << 4) | ((kc & 7) * 2))));
            const __nv_bfloat16* g = a.g_pages + ((size_t)pg * a.p.page_size + (key - pi * a.p.page_size)) * width +
                                     (size_t)head * a.m_pitch + job.strip * kN + c0;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const float gv = c0 + c < cols ? __bfloat162float(g[c]) : 0.f;
              if (!isfinite(gv)) y[c] += w * gv;
            }
          }
        }
      };

      bool finish = true;
      if (job.nc > 1) {
        // a key range's partial sums; the last range of the tile to finish joins them
        if (lead) {
          const int sl = atomicAdd(a.next + 1, 1);
          a.slot[tkey * a.nc_cap + job.c] = sl;
          b.last = sl;
        }
        named_bar_sync(1, 128);
        const int sl = b.last;
        float* dst = a.part + (size_t)sl * (kN * a.r8cap);
        if (warp_rows && sl < a.n_slots) {
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
        __threadfence();
        named_bar_sync(1, 128);
        if (lead) {
          b.last = atomicAdd(a.done + tkey, 1) == job.nc - 1;
          __threadfence();
        }
        named_bar_sync(1, 128);
        finish = b.last != 0;
      }
      if (finish && warp_rows) {
        float inv = 0.f;
        if (live && pos >= 0) {
          const float* dp = a.den + ((size_t)job.hl * a.rows_tot + job.prow + r) * a.spans;
          const int ns = (vis + a.span_keys - 1) / a.span_keys;
          float d = 0.f;
          for (int i = 0; i < ns; ++i) d += __ldcg(dp + i);
          if (a.null_bias) {
            const float tau = head_tau(a.tau, a.s, head, a.p.err, kKernPaged);
            d += (float)(pos + 1) * expf(a.null_bias[head] - tau);
          }
          inv = 1.f / d;
        }
        const size_t row = job.row0 + r, col = (size_t)head * a.m_pitch + job.strip * kN;
        for (int c0 = 0; c0 < cols; c0 += 32) {
          float y[32];
          if (job.nc == 1) {
            fetch(c0, y);
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) y[c] = 0.f;
            if (live) {
              for (int k = 0; k < job.nc; ++k) {
                const int sl = __ldcg(a.slot + tkey * a.nc_cap + k);
                if ((unsigned)sl >= (unsigned)a.n_slots) continue;
                const float4* src = reinterpret_cast<const float4*>(a.part + (size_t)sl * (kN * a.r8cap));
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                  const float4 x = __ldcg(src + (size_t)(c0 / 4 + u) * a.r8cap + r);
                  y[4 * u] += x.x; y[4 * u + 1] += x.y; y[4 * u + 2] += x.z; y[4 * u + 3] += x.w;
                }
              }
            }
          }
          if (!live) continue;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int cc = c0 + 8 * u;
            if (cc >= cols) break;
            float z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = pos >= 0 ? y[8 * u + e] * inv : 0.f;
            if (a.v && pos >= 0) {
              const __nv_bfloat16* vp = a.v + row * a.v_pitch + col + cc;
              if (a.v_vec) {
                const uint4 x = *reinterpret_cast<const uint4*>(vp);
                z[0] *= bf16lo(x.x); z[1] *= bf16hi(x.x); z[2] *= bf16lo(x.y); z[3] *= bf16hi(x.y);
                z[4] *= bf16lo(x.z); z[5] *= bf16hi(x.z); z[6] *= bf16lo(x.w); z[7] *= bf16hi(x.w);
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] *= cc + e < cols ? __bfloat162float(vp[e]) : 0.f;
              }
            }
            // whole vectors: the last one may run into the pitch's padding
            st_global_v4(a.out + row * width + col + cc, pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]),
                         pack_bf16x2(z[4], z[5]), pack_bf16x2(z[6], z[7]));
          }
        }
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
  } else {
    // ------------------------------------------------------------ scrub
    const int t = threadIdx.x - kScrub0 * 32;
    Ring st, jr;
    bool ok = true;
    while (ok) {
      if (!(ok = warp_wait(&b.job_full[jr.stage], jr.phase, b, a))) break;
      const Job job = b.job[jr.stage];
      if (job.b < 0) break;
      const int nbc = (job_cols(a, job) + 63) / 64;
      // every step is waited for, and its stage is free only once this warp has seen it too:
      // a parity wait that ran more than one fill ahead or behind would see the wrong fill
      for (int it = job.it0; it < job.it1; ++it) {
        if (!(ok = warp_wait(&b.full[st.stage], st.phase, b, a))) break;
        if (step_dirty(job, it)) {
          const int keys = max(0, step_keys(job, it)), rows = (keys + 15) & ~15;
          const int seen = job.pos0 - it * kK;  // rows <= seen are seen by all
          const uint32_t s0 = smem_u32(sB + st.stage * kBBytes);
          bool found = false;
          for (int r = max(0, seen + 1) + t / 8; r < rows; r += 16) {
            for (int c = 0; c < nbc; ++c) {
              const uint32_t at = s0 + c * kGBox + r * 128 + (t & 7) * 16;
              if (r >= keys) {
                st_shared_v4(at, make_uint4(0, 0, 0, 0));
                continue;
              }
              uint4 x = ld_shared_v4(at);
              uint32_t y[4] = {x.x, x.y, x.z, x.w};
              bool hit = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (bad_bits(y[e], 0x7f80u)) { y[e] &= 0xffff0000u; hit = true; }
                if (bad_bits(y[e], 0x7f800000u)) { y[e] &= 0xffffu; hit = true; }
              }
              if (hit) {
                st_shared_v4(at, make_uint4(y[0], y[1], y[2], y[3]));
                found = true;
              }
            }
          }
          if (found) *(volatile int*)&b.job[jr.stage].poison = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b.clean[st.stage]);
        }
        if (lane == 0) mbar_arrive(&b.empty[st.stage]);
        st.next(kStages);
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&b.job_empty[jr.stage]);
      jr.next(kJobSlots);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ============================================================================= launch

int num_sms() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 1;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Rows of a G box: the largest power of two that divides a page, at most a step.
int box_rows(int page_size) {
  int r = page_size & -page_size;
  return r > kK ? kK : r;
}

struct TcPlan {
  int rows_tot, key_blocks, span_keys, spans, strips, tiles, r8cap, nc_cap, n_slots, heads, grid;
  size_t P, den, part, slot, done, next, total;
};

TcPlan tc_plan(const PagedCall& c) {
  TcPlan l;
  const int sms = num_sms();
  l.rows_tot = up8(c.p.N) + 8 * c.p.B;
  l.key_blocks = ceil_div(c.p.max_len, kK);
  // at most 32 spans of whole 128-key blocks (their sums are added once per strip)
  l.span_keys = ceil_div(ceil_div(c.p.max_len, 32), 128) * 128;
  if (l.span_keys < 256) l.span_keys = 256;
  l.spans = ceil_div(c.p.max_len, l.span_keys);
  l.strips = ceil_div(c.m_h, kN);
  l.tiles = c.p.N / kM + c.p.B;
  l.r8cap = c.p.max_new < kM ? up8(c.p.max_new) : kM;
  l.nc_cap = ceil_div(l.key_blocks, kMinSteps);
  l.grid = sms;
  // a tile that is cut has at most twice as many ranges as whole ranges fit in it
  l.n_slots = 2 * kJobsPerSm * sms;
  // heads of a pass: as many as keep P within 2 GB
  const size_t per_head = (size_t)l.rows_tot * l.key_blocks * 128;
  const size_t fit = (size_t(2) << 30) / per_head;
  l.heads = (int)(fit < 1 ? 1 : fit > (size_t)c.H ? (size_t)c.H : fit);
  const size_t tk = (size_t)l.heads * l.strips * l.tiles;
  l.P = 0;
  l.den = l.P + align256(per_head * l.heads);
  l.part = l.den + align256((size_t)l.heads * l.rows_tot * l.spans * 4);
  l.slot = l.part + align256((size_t)l.n_slots * kN * l.r8cap * 4);
  l.done = l.slot + align256(tk * l.nc_cap * 4);
  l.next = l.done + align256(tk * 4);
  l.total = l.next + 256;
  return l;
}

}  // namespace

bool paged_tc_takes(tg_dtype dt, const PagedCall& c) {
  // the shape alone decides, so that the workspace can be sized without the pointers
  return dt == TG_BF16 && c.p.max_new > 8 && (c.d_h == 16 || c.d_h == 32 || c.d_h == 64) && c.m_pitch % 8 == 0 &&
         box_rows(c.p.page_size) >= 8;
}

size_t paged_tc_ws_bytes(const PagedCall& c) { return tc_plan(c).total; }

cudaError_t launch_paged_tc(const PagedCall& c, cudaStream_t s) {
  const TcPlan l = tc_plan(c);
  TcArgs a = {};
  a.p = c.p; a.H = c.H; a.d_h = c.d_h; a.m_h = c.m_h; a.m_pitch = c.m_pitch;
  a.rows_tot = l.rows_tot; a.key_blocks = l.key_blocks; a.span_keys = l.span_keys; a.spans = l.spans;
  a.strips = l.strips; a.tiles = l.tiles; a.r8cap = l.r8cap; a.nc_cap = l.nc_cap; a.n_slots = l.n_slots;
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
  a.timeout_ns = kTimeoutNs;

  CUtensorMap mG;
  cudaError_t e = make_tmap_4d_heads(&mG, c.g_pages, c.p.n_pages, c.p.page_size, c.H, c.m_h, c.m_pitch, a.box_rows, 64);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(paged_weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kWSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(paged_gates_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGSmem);
  if (e != cudaSuccess) return e;
  for (a.h0 = 0; a.h0 < c.H; a.h0 += l.heads) {
    a.heads = c.H - a.h0 < l.heads ? c.H - a.h0 : l.heads;
    paged_weights_kernel<<<dim3(l.tiles, a.heads, l.spans), kWThreads, kWSmem, s>>>(a);
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
    e = cudaLaunchKernelEx(&cfg, paged_gates_kernel, mG, a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace tg

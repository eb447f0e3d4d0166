/*
 * tango.h -- C ABI of the GB300 (sm_103a) cross-token gate aggregation library.
 *
 * Operations defined by "TANGO: Token-Aggregated Nonlinear Gating Operators for
 * Natural and Formal Language Modeling" (arXiv 2608.22117):
 *   - tango_aggregate      sec. 2.1 eq. 5 with the full-prefix weights of sec. 2.2 eq. 6
 *   - wango_aggregate      sec. 2.1 eq. 5 with the windowed weights of sec. 2.2 eqs. 7-10
 *   - tango_block_forward  one block application, sec. 2.1 eqs. 2-3 around either of the above
 *   - wango_decode_step    one autoregressive token of the windowed aggregation (eqs. 7-10)
 *                          from a constant-size state
 *   - tango_model_forward  the language model of sec. 2.3: token embedding, the shared block
 *                          applied n times (eq. 11), final RMSNorm and tied logits; with
 *                          one weight set, or with the revision's gated-projection sets
 *   - tango_aggregate_backward, wango_aggregate_backward
 *                          gradients of the two aggregations (eq. 5 differentiated with
 *                          respect to q, k, g and v), for training (sec. 3); the
 *                          tango_aggregate_save / wango_aggregate_save forwards keep what
 *                          they need
 *   - tango_qk_norm_rope (and _backward), tango_cache_append, tango_paged_aggregate
 *                          norm and rotation of q and k, and serving from a paged cache
 *   - tango_embed, tango_norm, tango_distill (each with _backward), tango_sample
 *                          the model's two ends (sec. 2.3) for training and generation: token
 *                          lookup, RMS or layer norm, the loss against a teacher's top
 *                          logits, and drawing tokens
 *
 * Conventions shared by every call:
 *   - Every pointer argument named as "device" is a CUDA device pointer owned by the
 *     caller.  The library never allocates, frees or synchronises; scratch memory is
 *     passed in as a workspace whose size tg_workspace_size() reports.
 *   - Tensors are row-major and contiguous.  q, k: [B, T, d_qk]; g, v, out: [B, T, m];
 *     h: [B, T, d]; weights are [out_features, in_features].  Head a owns columns
 *     [a*d_qk/H, (a+1)*d_qk/H) of q/k and [a*m/H, (a+1)*m/H) of g/v/out.
 *   - All tensors of one call share one storage type (tg_dtype).  Accumulation is
 *     always fp32.  TG_BF16 runs on the tensor cores (tcgen05); TG_F32 runs on the
 *     CUDA cores in full fp32 (no TF32).
 *   - Arguments are validated on the host before anything is launched; a bad
 *     argument returns an error status and launches nothing.  A failed launch
 *     returns TG_ERR_CUDA.  Errors found on the device (a bounded wait that ran out,
 *     a temperature outside [0, 20]) are recorded in a per-device error word that
 *     tg_check_device_error() reads and clears.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default stream).
 *   - Calls are thread-safe with respect to each other; concurrent calls that share
 *     a workspace race.
 *   - The library runs in each device's primary context (the CUDA runtime's); the
 *     device address of the error word is looked up once per device and kept, so
 *     cudaDeviceReset, or a non-primary context made current through the driver API,
 *     is not supported.
 */
#ifndef TANGO_GB300_H
#define TANGO_GB300_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *tg_stream_t; /* identical to cudaStream_t */

typedef enum {
    TG_OK = 0,
    TG_ERR_INVALID_ARG = 1, /* null pointer, non-positive size, inconsistent shape */
    TG_ERR_UNSUPPORTED = 2, /* valid but not implemented (e.g. bf16 head width not in {16,32,64}) */
    TG_ERR_WORKSPACE = 3,   /* workspace missing, misaligned or smaller than required */
    TG_ERR_CUDA = 4,        /* a CUDA runtime or driver call failed */
    TG_ERR_TIMEOUT = 5,     /* (device) a bounded wait inside a kernel ran out */
    TG_ERR_DEVICE = 6       /* (device) an out-of-range value was seen in device memory */
} tg_status;

typedef enum { TG_F32 = 0, TG_BF16 = 1 } tg_dtype;

/* tg_agg_params.flags */
#define TG_FLAG_QK_NORMALIZED 0x1u  /* q and k are already unit vectors per head */
#define TG_FLAG_DEBUG_TIMEOUT 0x100u /* test hook: a bf16 kernel waits on a barrier that is
                                        never signalled, with a ~1 ms limit, and returns
                                        TG_ERR_TIMEOUT through tg_check_device_error().
                                        tango_aggregate: the TANGO kernel; wango_aggregate:
                                        the gate-strip kernel; tango_block_forward: the
                                        projection GEMM; tango/wango_aggregate_backward:
                                        the pair-gradient, dq/dk and running-sum scan
                                        kernels; tango_paged_aggregate: the weights and
                                        gates kernels of the tensor-core path (the outputs
                                        are then undefined) */
#define TG_FLAG_FUSED_V 0x200u       /* tango_block_forward, WANGO mode, bf16: v = W_v x is
                                        formed inside the aggregation kernel instead of by
                                        the projection GEMM (v is then never stored); see
                                        tango_block_forward */
#define TG_FLAG_BWD_FAR_SCAN 0x400u  /* wango_aggregate_backward: the older pairs beyond the
                                        window's band of 128-row blocks always go through
                                        running-sum scans (linear in T) */
#define TG_FLAG_BWD_FAR_PAIRS 0x800u /* wango_aggregate_backward: every older pair is formed
                                        pair by pair (T^2 m).  With neither flag the call
                                        picks by an estimate of the two costs (scans from
                                        about T = 4,096 at B = 8, m = 28,480); both flags:
                                        TG_ERR_INVALID_ARG */

/* tango_block_forward mode */
#define TG_MODE_TANGO 0
#define TG_MODE_WANGO 1

/* tg_workspace_size() selector */
#define TG_WS_TANGO 0 /* params: const tg_agg_params*   */
#define TG_WS_WANGO 1 /* params: const tg_agg_params*   */
#define TG_WS_BLOCK 2 /* params: const tg_block_params* */
#define TG_WS_MODEL 3 /* params: const tg_model_params* */
#define TG_WS_DECODE 4 /* params: const tg_agg_params*: bytes of the wango_decode_step state */
#define TG_WS_TANGO_BWD 5 /* params: const tg_agg_params*: tango_aggregate_backward */
#define TG_WS_WANGO_BWD 6 /* params: const tg_agg_params*: wango_aggregate_backward */

#define TG_WS_QK_BWD 16 /* params: const tg_qk_params*: tango_qk_norm_rope_backward */
#define TG_WS_PAGED 17  /* params: const tg_paged_params*: tango_paged_aggregate */
#define TG_WS_EMBED_BWD 18 /* params: const tg_embed_params*: tango_embed_backward */
#define TG_WS_NORM_BWD 19  /* params: const tg_norm_params*: tango_norm_backward */

#define TG_MAX_HEADS 64

/* tg_qk_params.layout, tg_append_params.layout: which columns of a head form a pair that
 * turns together, for rotary width r: c and c + r/2, or 2c and 2c + 1 */
#define TG_ROPE_HALF 0
#define TG_ROPE_INTERLEAVED 1
/* tg_qk_params.norm, tg_append_params.norm */
#define TG_NORM_NONE 0 /* n = x                          */
#define TG_NORM_UNIT 1 /* n = x / max(|x|, 1e-12)        */
#define TG_NORM_RMS 2  /* n = x / sqrt(mean(x^2) + eps)  */
/* tg_norm_params.norm: TG_NORM_RMS, or */
#define TG_NORM_LAYER 3 /* n = (x - mean(x)) / sqrt(mean((x - mean(x))^2) + eps) */

/* most teacher entries of a row (tg_distill_params.k) */
#define TG_MAX_TEACHER 1024

/*
 * Parameters of one aggregation (eq. 5).
 *   B, T       batch and sequence length (>= 1)
 *   H          heads (1..TG_MAX_HEADS); d_qk % H == 0 and m % H == 0
 *   d_qk       total query/key width (d_h = d_qk / H per head)
 *   m          total gate width F (m_h = m / H per head)
 *   s          temperature tau used for every head when tau == NULL; 0 <= s <= 20
 *              (eq. 4 caps tau at 20)
 *   tau        device float[H] of per-head temperatures, or NULL.  Values outside
 *              [0, 20] are clamped and flagged as TG_ERR_DEVICE.
 *   null_bias  device float[H] of null-gate biases b_a, or NULL for no null gate
 *              (eq. 5: weight n_i exp(b_a), n_i = i + 1, in the denominator only)
 *   window     WANGO window W >= 1, counting the destination itself (eq. 7);
 *              ignored by tango_aggregate
 *   phi_mode   WANGO feature map: 0 = eq. 8 (max(ELU(u)+1+1e-4, 1e-4)/sqrt(d_h)),
 *              1 = plain ELU(u) + 1
 *   flags      TG_FLAG_*
 *   dtype      storage type of q, k, g, v, out
 *   m_pitch    gate columns per head in memory: 0 means m_h = m / H (dense).  Otherwise
 *              >= m_h, and the gate-indexed tensors (g, v, out, and the backward's dout,
 *              dg, dv) are [B, T, H * m_pitch] with head a's m_h gates in columns
 *              [a*m_pitch, a*m_pitch + m_h); the other columns are not read, and in
 *              the outputs their contents are unspecified.  This lets a head width that is not a multiple of 8 (e.g. the
 *              revision's three-set width m = 9,494, m_h = 4,747) run in bf16 at a padded
 *              pitch.  wango_decode_step takes dense tensors only (0 or m_h), and a
 *              block's agg.m_pitch must be 0 (the block pads its own gates).
 * bf16 requirements: d_h in {16, 32, 64}, the per-head pitch (m_pitch, else m_h) a
 * multiple of 8, all tensor base addresses 16-byte aligned (else TG_ERR_UNSUPPORTED).
 */
typedef struct {
    int B, T, H, d_qk, m;
    float s;
    const float *tau;
    const float *null_bias;
    int window;
    int phi_mode;
    unsigned flags;
    tg_dtype dtype;
    int m_pitch;
} tg_agg_params;

/*
 * Full-prefix aggregation (sec. 2.2 eq. 6 in sec. 2.1 eq. 5):
 *   out[b,i,a-cols] = gbar_ia * v[b,i,a-cols],
 *   gbar_ia = sum_{j<=i} e^{l_ija} g_ja / (sum_{j<=i} e^{l_ija} + (i+1) e^{b_a}),
 *   l_ija = tau_a qhat_ia . khat_ja (unit-normalised unless TG_FLAG_QK_NORMALIZED).
 * q, k, g: device, read only.  v: device, or NULL (then out = gbar).  out: device,
 * written; may alias v, must not overlap q, k or g.  ws: device scratch of at least
 * tg_workspace_size(TG_WS_TANGO, p) bytes (256-byte aligned; may be NULL if 0).
 */
tg_status tango_aggregate(const tg_agg_params *p, const void *q, const void *k, const void *g,
                          const void *v, void *out, void *ws, size_t ws_bytes,
                          tg_stream_t stream);

/*
 * Windowed aggregation (sec. 2.2 eqs. 7-10): sources i-W < j <= i get e^{l_ija};
 * older sources j <= i-W get phi(sqrt(tau_a) qhat_ia) . phi(sqrt(tau_a) khat_ja),
 * evaluated through the running sums S = sum phi(k~) g^T, z = sum phi(k~); one joint
 * numerator and denominator (with the null term) per destination.  Arguments as for
 * tango_aggregate; the workspace is sized by tg_workspace_size(TG_WS_WANGO, p).
 */
tg_status wango_aggregate(const tg_agg_params *p, const void *q, const void *k, const void *g,
                          const void *v, void *out, void *ws, size_t ws_bytes,
                          tg_stream_t stream);

/*
 * tango_aggregate / wango_aggregate that also keep what their backward needs, as a
 * training forward does (bf16 only; TG_F32 returns TG_ERR_UNSUPPORTED):
 *   gbar  device, laid out as out: gbar = out / v (the aggregated gate before the
 *         product with v), in the storage type; written
 *   den   device float [B, H, T]: every row's denominator as the kernels form it
 *         (sum of the weights e^{tau (qhat.khat - 1)} as applied, plus the null term,
 *         all shifted by e^-tau); written.  An opaque statistic for the backward.
 * Passing both to the backward skips its recomputation of the forward.  Other arguments
 * as for tango_aggregate / wango_aggregate.
 */
tg_status tango_aggregate_save(const tg_agg_params *p, const void *q, const void *k, const void *g,
                               const void *v, void *out, void *gbar, float *den, void *ws,
                               size_t ws_bytes, tg_stream_t stream);
tg_status wango_aggregate_save(const tg_agg_params *p, const void *q, const void *k, const void *g,
                               const void *v, void *out, void *gbar, float *den, void *ws,
                               size_t ws_bytes, tg_stream_t stream);

/*
 * Backward of tango_aggregate (sec. 2.1 eq. 5 with the weights of sec. 2.2 eq. 6):
 * given dout = dL/d(out) for the output out = gbar * v (out = gbar when v == NULL),
 * writes the gradients of L with respect to the call's inputs:
 *   dv_i = dout_i * gbar_i,   dg_j = sum_{i>=j} alpha_ij (dout_i * v_i),
 *   dq, dk through the weights alpha_ij = w_ij / den_i: with
 *   dL/dw_ij = (dout_i * v_i) . (g_j - gbar_i) / den_i, the score gradient
 *   tau w_ij dL/dw_ij goes to qhat_i (times khat_j) and khat_j (times qhat_i), and from
 *   there through the unit normalisation qhat = q / max(|q|, 1e-12) of sec. 2.1 (with
 *   TG_FLAG_QK_NORMALIZED the gradients are those of the given unit vectors).
 * The null gate, if any, enters through the denominator; tau and null_bias receive no
 * gradient.
 *   p, q, k, g, v   as for the forward call (bf16 only: TG_F32 returns TG_ERR_UNSUPPORTED;
 *                   flags may hold TG_FLAG_QK_NORMALIZED only)
 *   dout            device [B, T, m], read only
 *   gbar, den       the forward's gbar and den from tango_aggregate_save with the same
 *                   arguments, or both NULL: the backward then recomputes them
 *   dq, dk          device [B, T, d_qk], written
 *   dg              device [B, T, m], written
 *   dv              device [B, T, m], written, or NULL (must be NULL when v is NULL)
 *   ws              device scratch of tg_workspace_size(TG_WS_TANGO_BWD, p) bytes,
 *                   256-byte aligned.  It holds the recomputed forward (gbar and the
 *                   denominators), E = dout * v / den, and the pair-weight gradients of
 *                   every causal pair in bf16, B * H * T_pad^2 * 2 bytes with
 *                   T_pad = T rounded up to a multiple of 128.
 * Outputs must not overlap inputs or each other.  Arithmetic: bf16 operands and fp32
 * accumulation on the tensor cores for the two T^2 m contractions; fp32 on the CUDA
 * cores elsewhere.
 */
tg_status tango_aggregate_backward(const tg_agg_params *p, const void *q, const void *k, const void *g,
                                   const void *v, const void *dout, const void *gbar, const float *den,
                                   void *dq, void *dk, void *dg, void *dv, void *ws, size_t ws_bytes,
                                   tg_stream_t stream);

/*
 * Backward of wango_aggregate (sec. 2.2 eqs. 7-10 in sec. 2.1 eq. 5).  Arguments,
 * outputs and requirements as for tango_aggregate_backward; the workspace is sized by
 * tg_workspace_size(TG_WS_WANGO_BWD, p); gbar and den come from wango_aggregate_save.
 * Window pairs contribute as in TANGO; an older
 * pair's weight phi(sqrt(tau) qhat_i) . phi(sqrt(tau) khat_j) passes its gradient
 * through phi' (ELU's derivative, over sqrt(d_h) for eq. 8) and sqrt(tau).  dg is the
 * forward numerator of the time-reversed sequence (linear in T).  The older pairs next
 * to the window (128-row blocks within ceil((W-1)/128) of the destination's) are formed
 * pair by pair; the rest either pair by pair too (T^2 m) or through running sums of
 * phi(k~_j) g_j^T and of phi(q~_i) E_i^T, eq. 10 taken backwards (linear in T): flags may
 * add TG_FLAG_BWD_FAR_SCAN or TG_FLAG_BWD_FAR_PAIRS to force one, else the call picks
 * by a cost estimate that depends on the current device's SM count (query the workspace
 * with the same device current).  The scans add 2 * ceil(m_h / n_s) * B * T * d_qk * 4
 * bytes of workspace (strips of n_s = 256, 384 or 512 gate columns, also picked by the SM
 * count).
 */
tg_status wango_aggregate_backward(const tg_agg_params *p, const void *q, const void *k, const void *g,
                                   const void *v, const void *dout, const void *gbar, const float *den,
                                   void *dq, void *dk, void *dg, void *dv, void *ws, size_t ws_bytes,
                                   tg_stream_t stream);

/*
 * One autoregressive step of the windowed aggregation (sec. 2.2 eqs. 7-10) for B
 * sequences that are all at position pos.  For destination i = pos the output equals row
 * i of wango_aggregate over the sequence so far: window sources i-W < j <= i get
 * e^{l_ij}, older sources enter through the running sums S = sum phi(k~_j) g_j^T and
 * z = sum phi(k~_j) (eq. 10).
 *   p         as for wango_aggregate; T is ignored; flags may hold TG_FLAG_QK_NORMALIZED
 *   q, k      device [B, d_qk]: this token's query and key (unit-normalised per head
 *             unless TG_FLAG_QK_NORMALIZED)
 *   g, v      device [B, m]: this token's gate and feature; v may be NULL (out = gbar)
 *   out       device [B, m], written
 *   state     device buffer of tg_workspace_size(TG_WS_DECODE, p) bytes, 256-byte aligned,
 *             owned by the caller and kept between steps: S and z in f32, a ring of the
 *             last W + 8 tokens' unit k and g (storage type), and per-step scratch.  The
 *             call with pos == 0 clears it; steps must then come in order pos = 0, 1, 2, ...
 * Sources enter S and z in groups of 8: one that has left the window waits in the ring,
 * weighted by e^-tau phi(q~_i) . phi(k~_j) directly, until the step that completes its
 * group adds the group to S and z (the same sums, formed later).
 * Requirements: d_h <= 128, W <= 2^30.  Arithmetic is fp32 for either storage type; the
 * weights are not rounded to bf16.  The step reads the ring (W + 8 g vectors) and S, and
 * rewrites S on one step in 8: it is bound by HBM bandwidth and, for one sequence, by
 * latency.
 */
tg_status wango_decode_step(const tg_agg_params *p, long long pos, const void *q, const void *k,
                            const void *g, const void *v, void *out, void *state,
                            size_t state_bytes, tg_stream_t stream);

/* Weights of one block, all of the block's dtype, row-major [out, in]. */
typedef struct {
    const void *rms_gamma; /* [d]      RMSNorm gain                           */
    const void *Wq;        /* [d_qk, d]                                        */
    const void *Wk;        /* [d_qk, d]                                        */
    const void *Wg;        /* [m, d]   gate projection (SiLU applied, eq. 2)   */
    const void *Wv;        /* [m, d]   feature projection (eq. 2)              */
    const void *Wo;        /* [d, m]   output projection (eq. 3)               */
} tg_block_weights;

/*
 * Block parameters: agg gives B, T, H, d_qk, m, s/tau, null_bias, window, phi_mode,
 * dtype (agg.flags: 0, TG_FLAG_DEBUG_TIMEOUT and/or TG_FLAG_FUSED_V).  d: residual width.  mode: TG_MODE_TANGO or
 * TG_MODE_WANGO.  rms_eps: RMSNorm epsilon (> 0).  rope_base: RoPE base (0 = no
 * RoPE); rotate-half pairing (c, c + d_h/2), positions 0..T-1 per sequence.
 */
typedef struct {
    tg_agg_params agg;
    int d;
    int mode;
    float rms_eps;
    float rope_base;
} tg_block_params;

/*
 * One block application (sec. 2.1 eqs. 2-3):
 *   x = RMSNorm(h); q, k = RoPE(W_q x), RoPE(W_k x), unit-normalised per head;
 *   g = SiLU(W_g x); v = W_v x; gbar by TANGO or WANGO; h_out = h + W_o (gbar * v).
 * h: device [B, T, d], read.  h_out: device [B, T, d], written; may alias h.
 * ws: device scratch of at least tg_workspace_size(TG_WS_BLOCK, p) bytes, 256-byte
 * aligned.  On return it holds, in this order, each region starting on a 256-byte
 * boundary: x [B*T, d], unit q [B*T, d_qk], unit k [B*T, d_qk], g [B*T, m'] and
 * u = gbar * v [B*T, m'] (v is overwritten in place).  With TG_FLAG_FUSED_V (bf16 WANGO
 * mode), v = W_v x is formed tile by tile inside the aggregation kernel (a 128-row x
 * 128-column tile on the tensor cores, rounded to bf16 as a stored v would be) and never
 * written to memory; the region then holds u only.  Both forms give the same v.  The
 * fused form saves the v write and read in HBM (2 m 2 bytes per token) but streams x and
 * a 128-row strip of W_v (256 KB at d = 512) through shared memory for every 128 x 128
 * output tile; on GB300 it is the slower of the two (2.31 against 1.72 ms per WANGO block
 * at B=8, T=2048, d=512, m=28,480), so it is not the default.
 * Gate width: the aggregate calls need m_h % 8 == 0 in bf16; the block does not.  In
 * bf16 it keeps each head's gates at a pitch of m_hp = m_h rounded up to a multiple
 * of 8, m' = H * m_hp: it copies W_g, W_v (rows) and W_o (columns) into the end of ws
 * at that pitch with zeros in the added entries, so g, v and u are zero there and
 * h_out is the unpadded block's.  Otherwise (fp32, or m_h % 8 == 0) m' = m and no copy
 * is made.
 */
tg_status tango_block_forward(const tg_block_params *p, const tg_block_weights *w,
                              const void *h, void *h_out, void *ws, size_t ws_bytes,
                              tg_stream_t stream);

/*
 * A language model built from one shared block (sec. 2.3): token embedding with the
 * tied matrix E, n_apps block applications h^(r+1) = Block(h^(r)) (eq. 11), a final
 * RMSNorm and logits = RMSNorm(h) E^T.  No application embedding is added and the
 * token embeddings are not re-added between applications.
 */
typedef struct {
    const void *embedding;          /* device [vocab, d]: input lookup and output matrix */
    const void *final_gamma;        /* device [d]: gain of the final RMSNorm              */
    const tg_block_weights *sets;   /* HOST array [n_sets] of weight sets (device
                                       pointers); the sets may share rms_gamma, Wq and Wk */
} tg_model_weights;

/*
 * block          every application's parameters (B, T, H, d_qk, m, s/tau, null_bias,
 *                window, phi_mode, dtype, d, mode, rms_eps, rope_base); m is the gate
 *                width of every set
 * vocab          rows of the embedding (>= 1; bf16 needs vocab % 8 == 0)
 * n_apps         block applications (1..64)
 * n_sets         weight sets (1..16)
 * set_of_app     HOST int[n_apps]: the set of each application, or NULL for the
 *                default: set 0 everywhere (n_sets == 1), or set 0 for the first
 *                application, set 2 for the last and set 1 for the others (n_sets ==
 *                3, the revision's first / middle / last assignment); NULL with any
 *                other n_sets is TG_ERR_INVALID_ARG
 * final_rms_eps  epsilon of the final RMSNorm (> 0)
 */
typedef struct {
    tg_block_params block;
    int vocab;
    int n_apps;
    int n_sets;
    const int *set_of_app;
    float final_rms_eps;
} tg_model_params;

/*
 * ids: device int32 [B, T] token ids; an id outside [0, vocab) gives a zero embedding
 * row and TG_ERR_DEVICE (kernel code 4) through tg_check_device_error().  logits:
 * device [B, T, vocab], written.  ws: device scratch of at least
 * tg_workspace_size(TG_WS_MODEL, p) bytes, 256-byte aligned: the residual stream
 * [B*T, d], the final normalised x [B*T, d], then one block's workspace.  Each
 * application is a tango_block_forward call and returns its errors.
 */
tg_status tango_model_forward(const tg_model_params *p, const tg_model_weights *w, const int *ids,
                              void *logits, void *ws, size_t ws_bytes, tg_stream_t stream);

/*
 * tango_aggregate for callers that cannot allocate device memory: runtimes that
 * forbid cudaMalloc once they are running, code confined to a memory pool it does not
 * own, or drivers that must not meet an out-of-memory failure mid-work.  The paper has
 * no counterpart; this is a deployment variant of tango_aggregate with no workspace
 * argument.
 *   - Scratch: one fixed array of TG_NOALLOC_SCRATCH_BYTES in device memory, declared
 *     by the library; every GPU that loads the library holds it until the process
 *     exits.  The call itself allocates nothing (no cudaMalloc, cudaFree or allocating
 *     library routine).
 *   - Limit: the call needs tg_workspace_size(TG_WS_TANGO, p) bytes of that array
 *     (two 256-byte-aligned copies of B*T*d_qk elements; none with
 *     TG_FLAG_QK_NORMALIZED).  Larger problems return TG_ERR_WORKSPACE and launch
 *     nothing; for bf16 that is B*T*d_qk > 4,194,304.
 *   - The first call on each device looks up the array's device address with that
 *     device current (cudaGetSymbolAddress); make that first call before any stream
 *     capture.  The address is kept for the life of the process and belongs to the
 *     device's primary context (the one the CUDA runtime uses): cudaDeviceReset, or a
 *     non-primary context made current through the driver API, is not supported.
 *   - Every call on a device shares the one array and keeps the last call's contents;
 *     each call overwrites the part it reads before reading it, so nothing has to be
 *     cleared between calls.  Calls whose kernels overlap on the GPU (different
 *     streams, or concurrent host threads) race on the array.
 * Other arguments, results and errors are those of tango_aggregate.
 */
#define TG_NOALLOC_SCRATCH_BYTES (16u << 20)
tg_status tango_aggregate_noalloc(const tg_agg_params *p, const void *q, const void *k,
                                  const void *g, const void *v, void *out, tg_stream_t stream);

/*
 * Norm and rotary position of every query and key head in one pass (sec. 2.1 takes RoPE
 * and the unit norm; the two commute), for callers that make q and k outside
 * tango_block_forward.  Per row and head, with x the head's d_h values:
 *   n = x r (r by `norm`),  z = gain * n,  out = R(position) z,
 * R turning the pairs of the first rotary_dim columns by position * freqs[c]; the other
 * columns pass.  The aggregations want unit vectors (TG_NORM_UNIT without a gain).
 *   rows         rows (tokens) of q and k (0 launches nothing)
 *   H, H_k       query and key heads (1..1024; H_k may be 0: no k)
 *   d_h          head width (1..128)
 *   rotary_dim   even, 0..d_h; 0 = no rotation
 *   layout, norm TG_ROPE_*, TG_NORM_*
 *   eps          TG_NORM_RMS only (> 0)
 *   T            positions == NULL: row r stands at position r % T (T >= 1)
 *   positions    device int[rows], any sign, or NULL
 *   freqs        device double[rotary_dim / 2]: radians per position, >= 0 (a long
 *                context's scaling is the caller's choice of these; tg_rope_freqs makes
 *                the usual ones).  Angles are reduced exactly (64-bit turns), so a
 *                position of a million is as accurate as position 1.
 *   q_gain, k_gain  device float[d_h], shared by all heads, or NULL (gain 1)
 *   q_pitch, k_pitch  elements between rows of q, k (0: H * d_h, H_k * d_h): q and k may
 *                be slices of one fused projection
 *   dtype        of q, k and the outputs; arithmetic is fp32, outputs are rounded once
 */
typedef struct {
    long long rows;
    int H, H_k, d_h, rotary_dim, layout, norm;
    float eps;
    int T;
    const int *positions;
    const double *freqs;
    const float *q_gain, *k_gain;
    long long q_pitch, k_pitch;
    tg_dtype dtype;
} tg_qk_params;

/* q_out [rows, H * d_h], k_out [rows, H_k * d_h]: device, dense, written; q_out may be q
 * and k_out may be k when those are dense.  k and k_out are NULL when H_k == 0. */
tg_status tango_qk_norm_rope(const tg_qk_params *p, const void *q, const void *k, void *q_out, void *k_out,
                             tg_stream_t stream);

/*
 * Gradients of tango_qk_norm_rope: given dq_out, dk_out = dL/d(q_out), dL/d(k_out) (dense),
 *   dz = R^T dout,  dgain = sum over rows and heads of dz * n,  dn = gain * dz,
 *   dx = r (dn - n <n, dn>) (unit; rms: the mean instead of the sum; none: dx = dn).
 * A unit-norm head with |x| < 1e-12 takes dx = r dn.  q, k as for the forward call.
 * dq [rows, H * d_h], dk: dense, written; may be dq_out, dk_out.  dq_gain, dk_gain: device
 * float[d_h], written (summed in a fixed order), or NULL; they need the gain.  ws: device
 * scratch of tg_workspace_size(TG_WS_QK_BWD, p) bytes (0 without gains).
 */
tg_status tango_qk_norm_rope_backward(const tg_qk_params *p, const void *q, const void *k, const void *dq_out,
                                      const void *dk_out, void *dq, void *dk, float *dq_gain, float *dk_gain,
                                      void *ws, size_t ws_bytes, tg_stream_t stream);

/*
 * Fills freqs (HOST double[rotary_dim / 2]) with f_c = base^(-2c / rotary_dim), scaled for
 * contexts `factor` times longer than the orig_len positions a model was trained on:
 *   orig_len == 0: every f_c / factor (interpolated positions);
 *   orig_len > 0: with n_c = orig_len f_c / (2 pi) the turns that pair c makes over the
 *     trained length and w = clamp((n_c - turns_lo) / (turns_hi - turns_lo), 0, 1),
 *     f_c (w + (1 - w) / factor): fast pairs are kept, slow ones interpolated.
 * Needs rotary_dim even and >= 0, base > 0, factor >= 1, orig_len >= 0, and turns_hi >
 * turns_lo >= 0 when orig_len > 0.
 */
tg_status tg_rope_freqs(int rotary_dim, double base, double factor, long long orig_len, double turns_lo,
                        double turns_hi, double *freqs);

/*
 * A ragged batch of B sequences over a paged cache of keys and gates.
 *   B            sequences (>= 1)
 *   H, d_h, m    heads, head width (1..128), total gate width (m % H == 0; m_h = m / H)
 *   m_pitch      gate columns per head in memory (0: m_h; else >= m_h), as in
 *                tg_agg_params, for the cache's gates and for g, v and out
 *   N            rows of the new-token tensors, all sequences' new tokens in order (0
 *                launches nothing)
 *   max_new      upper bound of the new tokens of one sequence (>= 1)
 *   max_len      upper bound of lens (>= 1); <= table_pitch * page_size
 *   page_size    tokens of a page (1..65536); n_pages: pages of the pool (>= 1)
 *   table_pitch  entries of page_table per sequence (>= 1)
 *   cu_new       device int[B + 1]: sequence b owns rows [cu_new[b], cu_new[b+1])
 *   lens         device int[B]: cached tokens of sequence b, its new ones included; the
 *                new tokens stand at positions lens[b] - n_b .. lens[b] - 1.  A token
 *                whose position is negative is not appended, and its outputs are 0
 *   page_table   device int[B, table_pitch]: page of tokens [p * page_size, (p+1) *
 *                page_size) of a sequence; entries past its last token are not used
 *   s, tau, null_bias   as in tg_agg_params (aggregation only)
 *   v_pitch      elements between rows of v (0: H * m_pitch)
 *   dtype        of the cache and of every tensor
 *   flags        0 or TG_FLAG_DEBUG_TIMEOUT (aggregation only)
 * Device values outside their range (cu_new not rising within [0, N], more new tokens
 * than max_new, lens outside [0, max_len], a page outside [0, n_pages)) are clamped or
 * skipped, never followed, and flagged TG_ERR_DEVICE; the sequence's results are then
 * unspecified.
 * The cache is two pools owned by the caller: k_pages [n_pages, page_size, H * d_h]
 * (normed, rotated keys) and g_pages [n_pages, page_size, H * m_pitch].  Slots past a
 * sequence's length may hold anything (NaN included): they are never used.  The columns
 * between m_h and m_pitch of a head may be read and are written with unspecified values;
 * they reach no result.
 * Rows of no sequence (before cu_new[0], from cu_new[B] on) are left as they are.
 * TG_BF16 runs the aggregation on the tensor cores when d_h is 16, 32 or 64, m_pitch and
 * page_size are multiples of 8, and q, out and the pools are 16-byte aligned; anything else, and
 * TG_F32, runs on the CUDA cores, which take max_len up to 8,388,480 (65,535 * 128).
 * On the tensor cores the weights e^{l_j - tau_a} are rounded to bf16 before they are summed (as
 * in tango_aggregate), and the denominators sum the rounded ones; sums, and everything on the
 * CUDA cores, are fp32.
 * max_new and max_len size grids, spans and scratch: results do not depend on them, times and
 * scratch do.  Bounds near the batch's own are the fastest.
 */
typedef struct {
    int B, H, d_h, m, m_pitch, N, max_new, max_len, page_size, n_pages, table_pitch;
    const int *cu_new, *lens, *page_table;
    float s;
    const float *tau;
    const float *null_bias;
    long long v_pitch;
    tg_dtype dtype;
    unsigned flags;
} tg_paged_params;

/*
 * What tango_cache_append does to the new tokens on their way into the cache.
 *   rotary_dim, layout, norm, eps, freqs   as in tg_qk_params, positions from lens; the
 *                aggregation wants norm TG_NORM_UNIT (or TG_NORM_NONE of unit vectors).  A model
 *                trained with another norm or with gains (tango_qk_norm_rope, then
 *                tango_aggregate, which makes unit vectors of them) runs tango_qk_norm_rope at
 *                the tokens' positions first and appends its outputs with TG_NORM_UNIT and
 *                rotary_dim 0
 *   silu         1: g holds the gate projection W_g x, and SiLU(g) is cached (eq. 2);
 *                0: g is cached as it is
 *   q_pitch, k_pitch, g_pitch   elements between rows of q, k, g (0: dense)
 */
typedef struct {
    int rotary_dim, layout, norm;
    float eps;
    const double *freqs;
    int silu;
    long long q_pitch, k_pitch, g_pitch;
} tg_append_params;

/*
 * Appends the new tokens' keys and gates to the cache: k [N, H * d_h] normed and rotated
 * at its token's position, g [N, H * m_pitch] through SiLU if asked, both written to the
 * token's slot.  q [N, H * d_h], if not NULL, is normed and rotated in the same launch into
 * q_out [N, H * d_h] (dense; may be a dense q) for the aggregation that follows; a row of no
 * sequence leaves an unspecified row there.  A token's slot must not be shared with another
 * sequence's new token.
 */
tg_status tango_cache_append(const tg_paged_params *p, const tg_append_params *a, const void *q, const void *k,
                             const void *g, void *q_out, void *k_pages, void *g_pages, tg_stream_t stream);

/*
 * TANGO aggregation of the new tokens over the cache: for the token at position i of its
 * sequence (already appended),
 *   out = v * sum_{j<=i} e^{l_j} g_j / (sum_{j<=i} e^{l_j} + (i+1) e^{b_a}),  l_j = tau_a q . k_j,
 * as tango_aggregate gives for the row of the whole sequence.  q [N, H * d_h] and the cached
 * keys are unit vectors per head (TG_NORM_UNIT, or already so): tango_aggregate normalises, this
 * call does not.  Where they are not and a row's mean weight e^{l_j - tau_a} leaves [2^-59, 1.25],
 * outside of what unit vectors in bf16 reach, the row is unspecified and flagged TG_ERR_DEVICE.  v [N, H * m_pitch] or NULL (out = gbar); out [N, H *
 * m_pitch], written (columns past m_h of a head: unspecified); may alias a dense v.
 * ws: device scratch of tg_workspace_size(TG_WS_PAGED, p) bytes, 256-byte aligned.  Large batches
 * run in passes over it: at most 1 GB on the CUDA cores, or what 8 rows of one head take there if
 * that is more (32 bytes a key of max_len, and 1/16 byte a key and gate); on the tensor cores at
 * most 2 GB of weights, or what 256 rows of one head take (512 bytes a key), and, for up to 65,536
 * sequences, half a GB of sums and counters.
 */
tg_status tango_paged_aggregate(const tg_paged_params *p, const void *q, const void *v, void *out,
                                const void *k_pages, const void *g_pages, void *ws, size_t ws_bytes,
                                tg_stream_t stream);

/*
 * Token lookup and its gradient, as tango_model_forward's embedding is trained.
 *   rows        tokens (0: the lookup launches nothing; the gradient is base or zeros);
 *               <= 2^30
 *   d, vocab    width (<= 2^20) and rows (<= 2^28) of the embedding
 *   scale       factor on every looked-up row
 *   pad_id      an id that stands for no token: its output rows are zeros and it gives no
 *               gradient (any value; -1 for ids that are padded with -1)
 *   pitch       elements between rows of out / dout (0: d)
 *   dtype       of the embedding, out and dout
 *   grad_dtype  of dembedding and base
 * ids: device int[rows].  An id that is neither pad_id nor in [0, vocab) gives a zero row,
 * no gradient and TG_ERR_DEVICE (kernel code 4).
 */
typedef struct {
    long long rows;
    int d, vocab;
    float scale;
    int pad_id;
    long long pitch;
    tg_dtype dtype, grad_dtype;
} tg_embed_params;

/* out[n] = scale * embedding[ids[n]], formed in fp32 and rounded once (scale 1: the row itself).
 * embedding: device [vocab, d]; out: device [rows, d] at `pitch`, written. */
tg_status tango_embed(const tg_embed_params *p, const int *ids, const void *embedding, void *out,
                      tg_stream_t stream);

/*
 * dembedding[v] = base[v] + scale * sum over the tokens n with ids[n] = v of dout[n].
 * base: device [vocab, d] or NULL (zeros); may be dembedding itself, so that the gradient of the
 * tied output matrix is added to.  dembedding: device [vocab, d], dense, every row written.  The
 * tokens are sorted by id first and summed in fp32 in an order that the sizes, the ids, whether dout,
 * base and dembedding are 16-byte aligned, and the device's number of SMs fix (no atomics on sums:
 * the same call on the same memory gives the same bits).  ws: device scratch of
 * tg_workspace_size(TG_WS_EMBED_BWD, p) bytes, 256-byte aligned.
 */
tg_status tango_embed_backward(const tg_embed_params *p, const int *ids, const void *dout, const void *base,
                               void *dembedding, void *ws, size_t ws_bytes, tg_stream_t stream);

/*
 * RMS or layer norm of rows of d values, y = gamma * n + beta.
 *   rows     rows (0 launches nothing but for the gradients' zeros)
 *   d        width (1..2^24)
 *   norm     TG_NORM_RMS or TG_NORM_LAYER
 *   eps      > 0
 *   x_pitch  elements between rows of x (0: d)
 *   dtype    of x, gamma, beta, y and their gradients dy, dres, dx; arithmetic is fp32, outputs
 *            are rounded once
 */
typedef struct {
    long long rows;
    int d, norm;
    float eps;
    long long x_pitch;
    tg_dtype dtype;
} tg_norm_params;

/* gamma, beta: device [d], or NULL (1, 0).  y: device [rows, d], dense, written; may be a dense x. */
tg_status tango_norm(const tg_norm_params *p, const void *x, const void *gamma, const void *beta, void *y,
                     tg_stream_t stream);

/*
 * Gradients of tango_norm: with r = 1 / sqrt(mean square + eps) and dn = gamma * dy,
 *   dx = r (dn - n mean(dn * n) - mean(dn)) + dres     (rms: without mean(dn)),
 *   dgamma = sum over rows of dy * n,  dbeta = sum over rows of dy.
 * The row statistics are formed from x again.  dres: device [rows, d] or NULL: the gradient that
 * reaches x past the norm (a residual stream's).  dx: device [rows, d], written; may be dy, dres or
 * a dense x.  dgamma, dbeta: device float[d], written (summed in a fixed order), or NULL; dgamma
 * needs gamma.  ws: device scratch of tg_workspace_size(TG_WS_NORM_BWD, p) bytes, 256-byte aligned
 * (not used, and may be NULL, without dgamma and dbeta).  The size follows the current device's
 * number of SMs: ask for it with the device current that the call runs on.
 */
tg_status tango_norm_backward(const tg_norm_params *p, const void *x, const void *gamma, const void *dy,
                              const void *dres, void *dx, float *dgamma, float *dbeta, void *ws, size_t ws_bytes,
                              tg_stream_t stream);

/*
 * Distillation from a teacher's top logits.  Per row, with the student's logits z over the
 * vocabulary and the teacher's k logits t at the tokens i_1 .. i_k:
 *   p = softmax(t / T) over the row's entries,  q = softmax(z / T) over the vocabulary,
 *   loss = T^2 sum_e p_e (ln p_e - ln q_{i_e}).
 * One entry a row (k = 1) at T = 1 is the cross entropy with that token.
 *   rows         rows (0 launches nothing)
 *   vocab, k     1 <= vocab, 1 <= k <= TG_MAX_TEACHER
 *   temperature  T in [0.001, 1000]
 *   pitch        elements between rows of logits (0: vocab)
 *   grad_pitch   elements between rows of dlogits (0: vocab)
 *   dtype        of logits and dlogits; arithmetic is fp32.  From T = 1 on the loss is good to
 *                2^-22 T^2 ln vocab: where the entries are the whole vocabulary, so that the loss
 *                does not grow with T, T = 30 leaves it three digits and T = 1000 none
 * t_logits: device float[rows, k].  t_ids: device int[rows, k]: an entry with a negative id, or
 * with t = -inf, is absent; an id >= vocab is absent too and flagged TG_ERR_DEVICE (kernel code
 * 7).  A token may stand in several entries.  A row without entries (padding) has loss 0 and
 * gradient 0.  Student logits of -inf have q = 0 (an entry there gives loss inf; its gradient is
 * finite); a row with NaN gives NaN, as does a student's +inf; a teacher's +inf gives loss NaN and
 * NaN in its entries' columns.
 */
typedef struct {
    long long rows;
    int vocab, k;
    float temperature;
    long long pitch, grad_pitch;
    tg_dtype dtype;
} tg_distill_params;

/* loss: device float[rows], written.  stats: device float[rows, 2] or NULL: every row's largest
 * logit and sum of e^{(z - largest) / T}, for the backward; written. */
tg_status tango_distill(const tg_distill_params *p, const void *logits, const float *t_logits, const int *t_ids,
                        float *loss, float *stats, tg_stream_t stream);

/*
 * Gradient of sum over rows of dloss * loss:
 *   dz_j = dloss T (q_j - sum over the entries e with i_e = j of p_e).
 * dloss: device float[rows].  dlogits: device [rows, vocab] at grad_pitch, written; may be logits
 * (at the same pitch).  stats: as tango_distill left them for the same arguments, or NULL: they are
 * formed here from the one reading of the logits, so that with `loss` (device float[rows] or NULL;
 * NULL with stats) one call gives a training step's loss and gradient.
 */
tg_status tango_distill_backward(const tg_distill_params *p, const void *logits, const float *t_logits,
                                 const int *t_ids, const float *dloss, const float *stats, void *dlogits, float *loss,
                                 tg_stream_t stream);

/*
 * Draws one token a row from given uniform numbers.  Per row, with logits x:
 *   w_i = e^{(x_i - max x) / T}; a token with w_i < 2^-40 (-inf, NaN) is never drawn;
 *   of these the k largest (top_k); of these the shortest run from the largest down with at least
 *   the share top_p of their mass; of these the ones with w_i >= min_p (the largest stays always);
 *   the token is the first one i in ascending order with
 *   sum over kept j <= i of w_j  >  u * sum over kept j of w_j.
 * Equal logits are ranked by ascending index.  T = 0 takes the largest logit (lowest index).  +inf
 * logits share the row evenly.  A row with no token to draw (all -inf or NaN) gives -1.  The sums
 * are formed in 64-bit fixed point from weights good to about 2^-33, so that the token is that of
 * the real numbers but where u or top_p lie within about 1e-10 of a border.  (From T = 2^112 on the
 * weights are good to |x - max x| 2^-150; a logit more than 3.4e38 below the largest weighs nothing.)
 *   rows, vocab     rows >= 0 (0 launches nothing); 1 <= vocab <= 2^19
 *   pitch           elements between rows of logits (0: vocab)
 *   dtype           of logits
 *   temperature, top_k, top_p, min_p   settings of every row, unless the array of that setting is
 *                   given: T >= 0 and finite (0 < T < 2^-126 counts as 2^-126); top_k <= 0: off;
 *                   top_p >= 1: off, <= 0: the largest only; min_p <= 0: off
 *   temperatures, top_ks, top_ps, min_ps  device [rows], or NULL.  Values outside their range (T < 0,
 *                   T = inf, NaN, min_p > 1) are clamped into it (NaN: the setting is off, T = 1)
 *                   and flagged TG_ERR_DEVICE (kernel code 8)
 */
typedef struct {
    int rows, vocab;
    long long pitch;
    tg_dtype dtype;
    float temperature;
    int top_k;
    float top_p, min_p;
    const float *temperatures;
    const int *top_ks;
    const float *top_ps, *min_ps;
} tg_sample_params;

/* uniform: device float[rows], in [0, 1); other values are clamped into it and flagged TG_ERR_DEVICE (kernel
 * code 8).  token: device int[rows], written.  logprob: device float[rows] or NULL: ln of the
 * probability the token was drawn with, w / sum over kept (T = 0: 0; no token: -inf); written. */
tg_status tango_sample(const tg_sample_params *p, const void *logits, const float *uniform, int *token,
                       float *logprob, tg_stream_t stream);

/* Workspace bytes needed by the call `which` (TG_WS_*) with `params`; 0 for invalid
 * parameters (validate with the call itself to get the reason). */
size_t tg_workspace_size(int which, const void *params);

/* Static, NUL-terminated description of a status. */
const char *tg_status_string(tg_status s);

/*
 * Synchronises `stream`, then reads and clears the current device's error word.
 * Returns TG_OK, TG_ERR_TIMEOUT or TG_ERR_DEVICE (the first kind recorded), or
 * TG_ERR_CUDA if the synchronisation itself failed.  If `detail` is not NULL it
 * receives the raw word (bit 0: timeout, bit 1: value out of range; bits 8..15:
 * the kernel that recorded it, 1 = TANGO, 2 = WANGO, 3 = GEMM, 4 = embedding lookup,
 * 5 = the aggregation backward, 6 = the paged cache calls, 7 = distillation, 8 = sampling).
 */
tg_status tg_check_device_error(tg_stream_t stream, unsigned *detail);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int tg_version(void);

#ifdef __cplusplus
}
#endif

#endif /* TANGO_GB300_H */

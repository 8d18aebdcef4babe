/*
 * gdr.h -- C ABI of the MI355X (gfx950) chunked gated-delta-rule library.
 *
 * The library computes the chunked prefill of the gated delta rule, the
 * linear-attention recurrence of Gated DeltaNet (GDN):
 *
 *     S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T
 *     o_t = scale * S_t^T q_t
 *
 * with an fp32 [K, V] state per value head, in the chunked (WY) form whose
 * forward and backward passes the FlashQLA pages fuse and accelerate
 * (FlashQLA curated summary, sections "核心亮點" and
 * "GDN Chunked Prefill的效率問題").  The argument lists follow that page's
 * low-level forward/backward listing (section "使用方式與需求"):
 *   forward:  q, k, v, g, beta, scale, initial_state, cu_seqlens
 *             -> g (processed), A, o, final_state
 *   backward: q, k, v, g, beta, A, do, dht, scale, initial_state, cu_seqlens
 *             -> dq, dk, dv, dbeta, dg, dh0
 * Variable-length packing and state continuation follow the Tongyi page
 * "FlashQLA - Tongyi Labsがオープンソース化した高性能線形アテンション演算子ライブラリ",
 * sections "FlashQLAの主な機能" and "FlashQLAの使い方".
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Pointers: every tensor pointer is a DEVICE pointer, except arguments whose
 *   name ends in _host (host memory).  Device pointers must be 16-byte
 *   aligned.  The library never allocates or frees device memory, never
 *   synchronises the device and never writes its inputs; it enqueues kernels
 *   on `stream` (a hipStream_t; NULL = the null stream) and returns.
 * Layouts (row-major, dense):
 *   q, k, dq, dk      [B, T, Hq, K]   dtype of the call
 *   v, o, do, dv      [B, T, Hv, V]   dtype of the call
 *   g, beta, dg, dbeta, g_cum        [B, T, Hv]  fp32
 *   A                 [B, T, Hv, 64]  fp32: row of the chunk's A for each token
 *   initial_state, final_state, dht, dh0   [N, Hv, K, V]  fp32
 *   cu_seqlens        [N + 1] int32 token offsets (packed mode, B must be 1)
 *   N = B without cu_seqlens, N = shape->num_seqs with it.
 * Heads: value head h reads query/key head h / (Hv / Hq) (contiguous groups).
 * Gate: g is the per-token log-gate (decay exp(g)); g <= 0 is expected.  A
 *   head with any g > 0 is still computed exactly, but never from a warmup
 *   (see the context-parallel options below).
 * Chunks: 64 tokens, restarting at every sequence start; the last chunk of a
 *   sequence may be short.
 * Supported: K, V in {32, 64, 128} with K == V; Hv a multiple of Hq;
 *   dtype bf16 (q, k, v, o, do, dq, dk, dv in bfloat16) or fp32; fp32 needs
 *   K <= 64 in the forward and K == 32 in the backward.
 * Errors: arguments are validated on the host before anything is enqueued; a
 *   negative status is returned and gdr_last_error() describes it.  Launch
 *   failures map to GDR_ERR_HIP.  Faults inside kernels surface at the
 *   caller's next synchronisation, as usual for HIP.
 * Threads: calls are thread-safe; gdr_last_error() is per thread.
 */
#ifndef GDR_H_
#define GDR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GDR_OK = 0,
  GDR_ERR_INVALID_ARG = -1,   /* null/misaligned pointer, bad shape, bad cu_seqlens_host */
  GDR_ERR_UNSUPPORTED = -2,   /* shape or dtype outside the supported set */
  GDR_ERR_WORKSPACE = -3,     /* workspace too small (see *_workspace_size) */
  GDR_ERR_HIP = -4            /* a HIP launch/runtime call failed */
} gdr_status;

typedef enum { GDR_BF16 = 0, GDR_F32 = 1 } gdr_dtype;

typedef struct {
  int32_t B, T;      /* batch, tokens per batch row (packed: B = 1, T = total) */
  int32_t Hq, Hv;    /* query/key heads, value heads (Hv % Hq == 0) */
  int32_t K, V;      /* key and value head dimensions */
  int32_t num_seqs;  /* N in packed mode (cu_seqlens given); ignored otherwise */
  gdr_dtype dtype;   /* element type of q, k, v, o, do, dq, dk, dv */
} gdr_shape;

/* Intra-card context parallelism (the pages' automatic single-card CP:
 * FlashQLA curated summary, section "平衡解決方案：雙核心融合與自動CP";
 * Tongyi page, section "FlashQLAの技術原則").  When (sequence, head) units are
 * too few to fill the GPU, each sequence is cut into segments of
 * `cp_segment_chunks` chunks; a segment's start state is rebuilt from zero over
 * the `cp_warmup_chunks` chunks before it, which is exact up to a factor
 * exp(sum of g over those chunks) as long as every token transition is a
 * contraction (g <= 0 and 0 <= beta |k|^2 <= 2).  A head is certified, and
 * uses the segments, when every token of the sequence meets those two
 * conditions and every warmup window has sum(g) <= cp_log_eps; each segment
 * of it then warms up over the fewest of those chunks
 * (counted back from its start) whose sum(g) already reaches cp_log_eps, which
 * keeps the same bound.  Any other head (for example one with g = 0) gets its segment
 * start states exactly instead: the map from a segment's start state to its
 * end state is affine, h_out = M h_in + b (the correction matrix the Tongyi
 * page describes for CP), so every segment's (M, b) is computed in parallel,
 * the start states follow from a short scan, and the segments then run from
 * them; with cp_serial_fallback = 1 such heads run serially instead.  Results
 * never depend on an uncertified warmup.  The bf16 backward uses the same
 * segments for both of its serial passes: the recomputed chunk states as
 * above, and the reverse pass over the state gradient, whose segments start
 * at their ends after up to cp_warmup_chunks chunks of warmup, again the
 * fewest that reach cp_log_eps (the reverse map is the transposed M plus an
 * offset); its certificate also covers the windows after every segment end.  The fp32 backward runs each head whole.
 * Pass NULL for the defaults; a zero-initialised struct also gives the
 * defaults. */
typedef enum { GDR_CP_AUTO = 0, GDR_CP_OFF = 1, GDR_CP_FORCE = 2 } gdr_cp_mode;

typedef struct {
  gdr_cp_mode cp_mode;       /* default GDR_CP_AUTO */
  int32_t cp_segment_chunks; /* GDR_CP_FORCE: chunks per segment (>= 1) */
  int32_t cp_warmup_chunks;  /* most warmup chunks before each segment; default 8 */
  float cp_log_eps;          /* certificate threshold on sum(g); default ln(1e-6) */
  int32_t cp_serial_fallback;/* 1: uncertified heads run serially; 0 (default): exact segment states */
  int32_t precise_vnew;      /* 1: the bf16 forward's output pass takes Vnew = A''(V - Gamma K h) as two
                              * bf16 terms (hi + lo) in its two products, P Vnew and the state update
                              * K^T (d * Vnew), instead of one bf16 rounding: for strongly coupled keys
                              * (nearly parallel keys without decay, where the chunk system I + L is
                              * badly conditioned), at the cost of one more MFMA per product; see the
                              * notes on precision.  0 (default): one bf16 operand.  Ignored in fp32
                              * and by the backward's recomputation. */
} gdr_options;

/* What the planner chose for a forward call (for tests and reporting). */
typedef struct {
  int32_t num_seqs;          /* N */
  int32_t total_chunks;      /* sum over sequences of ceil(len / 64) */
  int32_t max_chunks;        /* longest sequence, in chunks */
  int32_t v_blocks;          /* state column blocks per workgroup of the state pass */
  int32_t segment_chunks;    /* chunks per CP segment (>= max_chunks: no CP) */
  int32_t warmup_chunks;     /* most warmup chunks per segment (0 without CP) */
  int32_t total_segments;    /* sum over sequences of ceil(chunks / segment_chunks) */
  int32_t state_workgroups;  /* workgroups of the state pass */
} gdr_plan_info;

/* Bytes of device workspace gdr_chunk_fwd needs for this problem.
 * cu_seqlens_host is required in packed mode (num_seqs + 1 int32 values).
 * Returns 0 and sets gdr_last_error() on invalid arguments. */
size_t gdr_chunk_fwd_workspace_size(const gdr_shape* shape, const gdr_options* opts,
                                    const int32_t* cu_seqlens_host);

/* Forward chunked prefill.
 *   q, k, v, g, beta, scale   inputs as laid out above; scale > 0 finite.
 *   initial_state             nullable: zero initial state.
 *   cu_seqlens                nullable: B rows of T tokens; else packed mode,
 *                             with cu_seqlens_host its host copy (must match).
 *   o                         output [B, T, Hv, V] (call dtype).
 *   final_state               nullable: not written.
 *   g_cum_out                 nullable: chunk-local inclusive cumsum of g.
 *   A_out                     nullable: per-chunk A = (I + L)^-1 rows, where
 *                             L_ij = beta_i exp(gcum_i - gcum_j) k_i.k_j, i > j.
 *   workspace                 >= gdr_chunk_fwd_workspace_size() bytes, owned by
 *                             the caller, contents ignored and clobbered.
 */
gdr_status gdr_chunk_fwd(const gdr_shape* shape, const gdr_options* opts,
                         const void* q, const void* k, const void* v,
                         const float* g, const float* beta, float scale,
                         const float* initial_state,
                         const int32_t* cu_seqlens, const int32_t* cu_seqlens_host,
                         void* o, float* final_state, float* g_cum_out, float* A_out,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of the library-owned scratch that gdr_chunk_fwd_noalloc uses as its
 * workspace (128 MiB, held on every device that loads the library until the
 * process ends). */
#define GDR_NOALLOC_SCRATCH_BYTES (128u << 20)

/* gdr_chunk_fwd without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc): the workspace is the library's own
 * scratch on the current device, and the call allocates nothing (no
 * hipMalloc, hipFree or allocating library routine).  Arguments, layouts and
 * results are those of gdr_chunk_fwd; `stream` must belong to the current
 * device.  Problems whose gdr_chunk_fwd_workspace_size() exceeds
 * GDR_NOALLOC_SCRATCH_BYTES are rejected with GDR_ERR_WORKSPACE (for example
 * the long-context shape B=1, T=65536, Hv=8, K=V=128 needs 114 MiB and fits).
 * Every call on one device shares that device's scratch: calls that overlap
 * in time on one device (concurrent streams or host threads) race and must
 * be serialised by the caller; calls in stream order are safe.  The first
 * call on a device looks up the scratch's device address there. */
gdr_status gdr_chunk_fwd_noalloc(const gdr_shape* shape, const gdr_options* opts,
                                 const void* q, const void* k, const void* v,
                                 const float* g, const float* beta, float scale,
                                 const float* initial_state,
                                 const int32_t* cu_seqlens, const int32_t* cu_seqlens_host,
                                 void* o, float* final_state, float* g_cum_out, float* A_out,
                                 void* stream);

/* Planner decision for the forward (host only, nothing is enqueued). */
gdr_status gdr_chunk_fwd_plan(const gdr_shape* shape, const gdr_options* opts,
                              const int32_t* cu_seqlens_host, gdr_plan_info* out);

/* Bytes of device workspace gdr_chunk_bwd needs. */
size_t gdr_chunk_bwd_workspace_size(const gdr_shape* shape, const gdr_options* opts,
                                    const int32_t* cu_seqlens_host);

/* Backward of gdr_chunk_fwd for the loss <o, d_o> + <final_state, dht>.
 *   g                         the RAW log-gate (not g_cum).
 *   A                         nullable: the forward's A_out; recomputed if NULL.
 *   d_o                       [B, T, Hv, V] (call dtype).
 *   dht                       nullable: zero.
 *   initial_state             nullable: zero.
 *   dq, dk, dv                outputs (call dtype); dq, dk sum over each group.
 *   dbeta, dg                 outputs fp32 [B, T, Hv]; dg is w.r.t. raw g.
 *   dh0                       nullable output [N, Hv, K, V] (gradient at the
 *                             initial state, zero state if none was given).
 */
gdr_status gdr_chunk_bwd(const gdr_shape* shape, const gdr_options* opts,
                         const void* q, const void* k, const void* v,
                         const float* g, const float* beta, const float* A,
                         const void* d_o, const float* dht, float scale,
                         const float* initial_state,
                         const int32_t* cu_seqlens, const int32_t* cu_seqlens_host,
                         void* dq, void* dk, void* dv, float* dbeta, float* dg, float* dh0,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Message for the last non-OK status returned on this thread ("" if none). */
const char* gdr_last_error(void);

/* ==== the operators around the rule in a linear-attention layer ============
 * The short causal convolution in front of the mixer, the rule's form for one
 * new token, the selective state space scan (the mixer's sibling without the
 * delta term, for layers of that kind in one model), and the root-mean-square
 * norm before and after the mixer.
 *
 * They share the conventions above, with these differences:
 * Strides: an operand marked "strided" may be a slice of a wider row: its
 *   token stride is given in elements (0: dense).  Tokens of a batch are
 *   numbered b * T + t through one stride.
 * Alignment: tensors need the alignment of their elements only, except where
 *   16-byte rows are asked for (the scan and the steps).
 * Overlap: outputs must not overlap inputs, or each other, except where an
 *   entry point says so (states of the steps, residual_out).
 * Sequences: cu_seqlens is read on the device only; no host copy is needed
 *   and a captured graph may be replayed with other offsets.  It must be
 *   non-decreasing; offsets are clamped to [0, T], so that no value of it can
 *   make a kernel leave its buffers.  Tokens before cu_seqlens[0] or from
 *   cu_seqlens[N] on belong to no sequence: their output rows (and input
 *   gradients) are zero.  Empty sequences are allowed; their final state is
 *   their initial state.
 * State pools (the steps): state holds num_slots states; row r works on slot
 *   slots[r] (slots NULL: slot r, rows <= num_slots), in place.  A row whose
 *   slot is outside [0, num_slots), or was named by an earlier row of the same
 *   call, is padding: its output row is zero and no state changes.
 *   Each row looks at the slots of all rows before it: 2 % of a call at 256
 *   rows, 10 % at 1024, as much again at 4096 (convolution; the rule's and the
 *   scan's larger states hide it).  Without slots nothing is looked at.
 * Non-finite inputs reach what the formulas let them reach and nothing else:
 *   no earlier token, no other sequence, no other row.  In the scan an
 *   infinity may come out as a NaN. */

typedef enum { GDR_ACT_NONE = 0, GDR_ACT_SILU = 1 } gdr_activation;

/* ---- short causal convolution ----------------------------------------------
 *   z_t = bias + sum_{j < W} weight[:, j] * x_{t - W + 1 + j},  y_t = act(z_t)
 * per channel; inputs before a sequence's first token are the rows of its
 * initial state (zeros without one).  Sums are fp32. */
typedef struct {
  int32_t B, T;               /* as in gdr_shape */
  int32_t D, W;               /* channels, at most 2^30; taps, 2 to 4 */
  int32_t num_seqs;           /* N in packed mode; ignored otherwise */
  gdr_dtype dtype;            /* of x, weight, bias, states, y and the gradients */
  gdr_activation activation;
  int64_t x_stride;           /* elements between tokens of x (0: D) */
} gdr_conv_shape;

/*   x              [B, T, D], strided;  weight [D, W];  bias [D], nullable
 *   initial_state  [N, W - 1, D], nullable: the W - 1 inputs before each sequence, oldest first
 *   y              [B, T, D] dense
 *   final_state    [N, W - 1, D], nullable: the last W - 1 inputs (reaching into the initial state) */
gdr_status gdr_causal_conv_fwd(const gdr_conv_shape* shape, const void* x, const void* weight, const void* bias,
                               const void* initial_state, const int32_t* cu_seqlens, void* y, void* final_state,
                               void* stream);

/* Bytes of device workspace gdr_causal_conv_bwd needs (0 on invalid arguments). */
size_t gdr_causal_conv_bwd_workspace_size(const gdr_conv_shape* shape);

/* Gradients of <y, dy> + <final_state, dht>.  dy dense; dht nullable.  dx is
 * [B, T, D] dense; dw [D, W], db [D] (nullable) and dh0 [N, W - 1, D]
 * (nullable) have the call's dtype, each rounded once from an fp32 sum that is
 * added in a fixed order. */
gdr_status gdr_causal_conv_bwd(const gdr_conv_shape* shape, const void* x, const void* weight, const void* bias,
                               const void* initial_state, const int32_t* cu_seqlens, const void* dy,
                               const void* dht, void* dx, void* dw, void* db, void* dh0, void* workspace,
                               size_t workspace_bytes, void* stream);

/* One new token per row: x [rows, D] strided, y [rows, D]; state
 * [num_slots, W - 1, D] moves on by one input.  shape: B = rows, T = 1. */
gdr_status gdr_causal_conv_step(const gdr_conv_shape* shape, const void* x, const void* weight, const void* bias,
                                void* state, int32_t num_slots, const int32_t* slots, void* y, void* stream);

/* ---- gated delta rule, one new token per row -------------------------------
 *   S = exp(g) S;  S += k (beta (v - S^T k))^T;  o = scale S^T q
 * shape: B = rows, T = 1; q, k [rows, Hq, K], v, o [rows, Hv, V], g, beta
 * [rows, Hv] fp32; state [num_slots, Hv, K, V] fp32, in place.  bf16 and fp32,
 * K = V in {32, 64, 128} for both.  q_stride, k_stride, v_stride: elements
 * between rows (0: dense); rows and state must be 16-byte aligned. */
gdr_status gdr_step(const gdr_shape* shape, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                    const void* v, int64_t v_stride, const float* g, const float* beta, float scale, float* state,
                    int32_t num_slots, const int32_t* slots, void* o, void* stream);

/* ---- selective state space scan (inference) --------------------------------
 *   d_t = dt_t + dt_bias, through softplus if dt_softplus
 *   S_t = exp(d_t A) S_{t-1} + d_t B_t x_t^T,   y_t = S_t^T C_t + D x_t
 * per head, with an fp32 [N, P] state; head h reads group h / (H / G) of B and
 * C.  States, gates, sums and D x are fp32.  With bf16, y's products over a
 * chunk of tokens take two operands rounded to bf16: the decayed scores
 * d_j (C_i . B_j) e^(sum of d A), and the chunk's entry state (the state itself is not
 * rounded).  No gradient is offered. */
typedef struct {
  int32_t B, T;               /* as in gdr_shape */
  int32_t H, G;               /* heads; groups of B and C (H % G == 0) */
  int32_t P, N;               /* head dimension and state size: 32, 64 or 128 each */
  int32_t num_seqs;           /* sequences in packed mode; ignored otherwise */
  gdr_dtype dtype;            /* of x, dt, B, C and y */
  int32_t dt_softplus;        /* 0 or 1 */
  int64_t x_stride, dt_stride, b_stride, c_stride;  /* elements between tokens (0: dense) */
} gdr_ssm_shape;

/* Bytes of device workspace gdr_ssm_scan_fwd needs (0 on invalid arguments). */
size_t gdr_ssm_scan_fwd_workspace_size(const gdr_ssm_shape* shape);

/*   x [B, T, H, P], dt [B, T, H], B, C [B, T, G, N]: strided; the rows of x, B and C 16-byte aligned
 *   A [H] fp32;  D, dt_bias [H] fp32, nullable
 *   initial_state, final_state   [num_seqs or B, H, N, P] fp32, nullable
 *   y [B, T, H, P] dense */
gdr_status gdr_ssm_scan_fwd(const gdr_ssm_shape* shape, const void* x, const void* dt, const float* A,
                            const void* B, const void* C, const float* D, const float* dt_bias,
                            const float* initial_state, const int32_t* cu_seqlens, void* y, float* final_state,
                            void* workspace, size_t workspace_bytes, void* stream);

/* One new token per row (shape: B = rows, T = 1); state [num_slots, H, N, P]
 * fp32, in place. */
gdr_status gdr_ssm_step(const gdr_ssm_shape* shape, const void* x, const void* dt, const float* A, const void* B,
                        const void* C, const float* D, const float* dt_bias, float* state, int32_t num_slots,
                        const int32_t* slots, void* y, void* stream);

/* ---- root-mean-square norm --------------------------------------------------
 *   h = x (+ residual),  y = h / sqrt(mean(h^2) + eps) * weight (* gate sigmoid(gate))
 * over rows of dim values (dim <= 16384), statistics in fp32.  Row r of a
 * strided operand starts (r / inner) * outer_stride + (r % inner) * inner_stride
 * elements behind its pointer (both strides 0: dense), so that [tokens, heads,
 * dim] slices of a wider row can be given as they are. */
typedef struct { int64_t outer, inner; } gdr_row_stride;
typedef struct {
  int64_t rows;
  int32_t inner;              /* rows per outer step (heads), >= 1; rows % inner == 0 */
  int32_t dim;
  gdr_dtype dtype;            /* of x, residual, gate, weight, 16- or 32-bit outputs and gradients */
  float eps;                  /* >= 0 (rows whose squares fp32 holds with few bits, from 1e-19 on down, are as exact as those) */
  int32_t quant;              /* 1: y in 8 bits (e4m3) with an fp32 scale for each 128 values of a row */
  gdr_row_stride x_stride, residual_stride, gate_stride;
} gdr_norm_shape;

/*   y             [rows, dim] of the call's dtype, or with quant one byte per value:
 *                 y = e4m3 value * scale, scale = max(max |y| of the group, 2^-100) / 448;
 *                 the value is y / scale (of 64 bits) rounded to fp32 and from there to e4m3;
 *                 the last group of a row may be short.  A group with a NaN is NaN.
 *   scales        [rows, ceil(dim / 128)] fp32 (quant only)
 *   residual_out  [rows, dim] dense: h rounded to the call's dtype; nullable without residual.
 *                 It may be the residual or x itself where that is dense. */
gdr_status gdr_rms_norm_fwd(const gdr_norm_shape* shape, const void* x, const void* residual, const void* gate,
                            const void* weight, void* y, float* scales, void* residual_out, void* stream);

/* Bytes of device workspace gdr_rms_norm_bwd needs (0 on invalid arguments). */
size_t gdr_rms_norm_bwd_workspace_size(const gdr_norm_shape* shape);

/* Gradients of <y, dy> + <h, d_res> at h (x_stride is its stride): dh [rows,
 * dim] dense (the gradient of x and of residual), dw [dim] and dgate [rows,
 * dim] dense (with a gate), in the call's dtype.  d_res nullable; dy and d_res
 * dense; shape->quant and residual_stride are ignored.  dw is added in a fixed order. */
gdr_status gdr_rms_norm_bwd(const gdr_norm_shape* shape, const void* h, const void* gate, const void* weight,
                            const void* dy, const void* d_res, void* dh, void* dw, void* dgate, void* workspace,
                            size_t workspace_bytes, void* stream);

/* ---- gated linear recurrence -------------------------------------------------
 *   e = sigmoid(r_t),  a = exp(A e),  b = sqrt(1 - a^2) sigmoid(i_t) x_t
 *   h_t = a h_{t-1} + b,  y_t = h_t
 * per channel; A <= 0 (a positive one gives NaN where a > 1).  States and sums
 * are fp32; y is h rounded once.  An infinite state stays infinite until its
 * sequence ends (NaN behind a decay that is zero in fp32, e^-87 and less). */
typedef struct {
  int32_t B, T;               /* as in gdr_shape */
  int32_t D;                  /* channels, at most 2^25 */
  int32_t num_seqs;           /* sequences in packed mode; ignored otherwise */
  gdr_dtype dtype;            /* of x, r, i, y and their gradients */
  int64_t x_stride, r_stride, i_stride;  /* elements between tokens (0: D) */
} gdr_linear_scan_shape;

/* Bytes of device workspace the forward needs (0 on invalid arguments).  Calls
 * that overlap in time need workspaces of their own, as everywhere: tiles of one
 * prompt tell each other through it how far they are.  Calls that share one all
 * the same end (the waits between tiles are bounded) and report nothing: their
 * values mean nothing, NaN among them. */
size_t gdr_linear_scan_fwd_workspace_size(const gdr_linear_scan_shape* shape);

/*   x, r, i                      [B, T, D], strided;  A [D] fp32
 *   initial_state, final_state   [num_seqs or B, D] fp32, nullable
 *   y                            [B, T, D] dense */
gdr_status gdr_linear_scan_fwd(const gdr_linear_scan_shape* shape, const void* x, const void* r, const void* i,
                               const float* A, const float* initial_state, const int32_t* cu_seqlens, void* y,
                               float* final_state, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace the backward needs (0 on invalid arguments). */
size_t gdr_linear_scan_bwd_workspace_size(const gdr_linear_scan_shape* shape);

/* Gradients of <y, dy> + <final_state, dht>.  dy dense; dht nullable.  dx, dr,
 * di [B, T, D] dense, in the call's dtype; dA [D] and dh0 [num_seqs or B, D]
 * (nullable) fp32.  sqrt(1 - a^2) has no derivative where it is zero: that
 * token adds nothing through it.  dA is added in a fixed order. */
gdr_status gdr_linear_scan_bwd(const gdr_linear_scan_shape* shape, const void* x, const void* r, const void* i,
                               const float* A, const float* initial_state, const int32_t* cu_seqlens, const void* dy,
                               const float* dht, void* dx, void* dr, void* di, float* dA, float* dh0, void* workspace,
                               size_t workspace_bytes, void* stream);

/* One new token per row (shape: B = rows, T = 1); state [num_slots, D] fp32, in
 * place. */
gdr_status gdr_linear_scan_step(const gdr_linear_scan_shape* shape, const void* x, const void* r, const void* i,
                                const float* A, float* state, int32_t num_slots, const int32_t* slots, void* y,
                                void* stream);

/* ---- norms around a block ----------------------------------------------------
 *   p = x / rms(x) * post_weight (* gate sigmoid(gate)),  rms(v) = sqrt(mean(v^2) + eps)
 *   h = residual + (scale *) p,  y = h / rms(h) * pre_weight
 * over rows of dim values (dim <= 16384): the norm behind a block with its gate
 * and scale, the residual's addition, and the norm before the next block.
 * Statistics are fp32; y is made from the unrounded h. */
typedef struct {
  int64_t rows;
  int32_t dim;
  gdr_dtype dtype;            /* of all tensors and gradients */
  float eps;                  /* >= 0 (rows whose squares fp32 holds with few bits, from 1e-19 on down, are as exact as those) */
  int64_t x_stride, residual_stride, gate_stride;  /* elements between rows (0: dim) */
} gdr_block_norm_shape;

/*   x, residual, gate           [rows, dim], strided; gate nullable
 *   post_weight, pre_weight, scale  [dim]; scale nullable
 *   y, h                        [rows, dim] dense; h may be residual itself where that is dense */
gdr_status gdr_block_norm_fwd(const gdr_block_norm_shape* shape, const void* x, const void* residual, const void* gate,
                              const void* post_weight, const void* pre_weight, const void* scale, void* y, void* h,
                              void* stream);

/* Bytes of device workspace gdr_block_norm_bwd needs (0 on invalid arguments). */
size_t gdr_block_norm_bwd_workspace_size(const gdr_block_norm_shape* shape);

/* Gradients of <y, dy> + <h, d_res> at x and h (the forward's h;
 * residual_stride is its stride).  dy and d_res (nullable) dense; dx, dh (the
 * gradient of residual) and dgate (with a gate) [rows, dim] dense; dpost, dpre
 * and dscale (with a scale) [dim], added in a fixed order. */
gdr_status gdr_block_norm_bwd(const gdr_block_norm_shape* shape, const void* x, const void* h, const void* gate,
                              const void* post_weight, const void* pre_weight, const void* scale, const void* dy,
                              const void* d_res, void* dx, void* dh, void* dgate, void* dpost, void* dpre,
                              void* dscale, void* workspace, size_t workspace_bytes, void* stream);

/* ---- products in 8-bit integers (inference) ----------------------------------
 * Rows quantised with one scale each:
 *   scale = max(max |x|, 2^-100) / 127,  q = the fp32 quotient x / scale rounded to an integer, ties to even
 * A row with an infinity or a NaN gets the scale NaN and zeros. */
typedef struct {
  int64_t rows;
  int32_t dim;                /* at most 32768 */
  gdr_dtype dtype;            /* of x */
  int64_t x_stride;           /* elements between rows (0: dim) */
  int64_t q_stride;           /* bytes between rows of q, a multiple of 16 (0: dim rounded up to one) */
} gdr_quantize_shape;

/* x [rows, dim] strided; q [rows, dim] int8, 16-byte aligned; the bytes from
 * dim up to the next multiple of 16 are set to zero.  scales [rows] fp32. */
gdr_status gdr_quantize_rows(const gdr_quantize_shape* shape, const void* x, int8_t* q, float* scales, void* stream);

/* y[m, n] = (sum over k of x[m, k] weight[n, k]) x_scales[m] weight_scales[n] + bias[n]
 * x [M, K] and weight [N, K] int8, the sum exact; scales and bias (nullable)
 * fp32; y [M, N] dense, in dtype, rounded once from fp32. */
typedef struct {
  int32_t M, N;
  int32_t K;                  /* at most 2^17 - 1 */
  gdr_dtype dtype;            /* of y */
  int64_t x_stride, w_stride; /* bytes between rows, multiples of 16 (0: K rounded up to one), at most 2^22.  The rows'
                               * starts are 16-byte aligned, and the last row's last 16-byte piece is readable whole
                               * (what lies behind K in it does not matter). */
} gdr_matmul_i8_shape;
gdr_status gdr_matmul_i8(const gdr_matmul_i8_shape* shape, const int8_t* x, const float* x_scales, const int8_t* weight,
                         const float* weight_scales, const float* bias, void* y, void* stream);

/* ---- kernel timing (diagnostics) ------------------------------------------
 * When enabled, every kernel the library enqueues is bracketed by a pair of
 * HIP events recorded on the launch stream.  gdr_timing_collect() waits for
 * the recorded events, folds their durations into per-kernel totals and
 * returns the number of distinct kernels seen; gdr_timing_entry() reads them.
 * Timing adds two event records per launch; it is off by default. */
void gdr_timing_enable(int enable);
int gdr_timing_collect(void);
int gdr_timing_entry(int i, const char** name, double* total_ms, int32_t* launches);
void gdr_timing_reset(void);

#ifdef __cplusplus
}
#endif

#endif /* GDR_H_ */

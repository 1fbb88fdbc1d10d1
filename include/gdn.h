/*
 * gdn.h -- C ABI of the MI355X (gfx950) chunked Gated DeltaNet prefill library.
 *
 * Operation.  The pages this library follows ("Qwen's FlashQLA targets the
 * expensive bit of long-context AI", section "What happened"; "FlashQLA
 * resource", section 2 "What It Actually Is") describe the forward and backward
 * pass of Gated DeltaNet (GDN) chunked prefill.  They print no formula; the
 * computation is the published gated delta rule, per sequence and head:
 *
 *     S_t = exp(g_t) S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,    S_0 = h0^T
 *     o_t = scale * S_t q_t,                                               hT = S_T^T
 *
 * with S a Dv x Dk matrix, evaluated chunk by chunk (64 tokens) in the exact
 * WY/UT form ("FlashQLA resource", section 3: an algebraic reformulation that
 * keeps full precision).  Long sequences with few heads are split into
 * segments that run side by side on one GPU; the exponential decay of the
 * gates bounds how far a segment boundary's state must be propagated
 * ("FlashQLA resource", section 3, gate-driven intra-card context parallelism;
 * section 5 for the backward pass).  The split changes the result by at most
 * 2^-24 of the norm of the state (or state gradient) at a segment boundary
 * carried across it, so a split and an unsplit run differ at fp32 round-off
 * level (the tests hold them to 1e-5 relative, elementwise).
 *
 * Layouts (row-major, last dimension contiguous, all pointers device memory
 * unless stated otherwise; every tensor pointer 16-byte aligned):
 *   q, k                [B, T, H, Dk]   dtype
 *   v, o                [B, T, H, Dv]   dtype
 *   beta                [B, T, H]       dtype
 *   g                   [B, T, H]       fp32, natural-log decay (<= 0 in the tested domain)
 *   h0, hT, dhT, dh0    [N, H, Dk, Dv]  fp32, h = S^T
 *   do, dq, dk, dv, dbeta   like o, q, k, v, beta; dg like g (fp32)
 * Variable-length batches: B == 1, sequences packed along T, described by
 * cu_seqlens (int32 [N+1], cu[0] = 0, non-decreasing, cu[N] = T).  The
 * recurrence restarts at every sequence start.  Without cu_seqlens, N = B.
 *
 * Supported: dtype GDN_BF16 with Dk, Dv in {64, 128}; GDN_F32 with Dk = Dv = 64.
 *
 * Ownership.  The caller owns every buffer, including the workspace, whose size
 * the *_workspace_size functions report for the same arguments.  The library
 * allocates no device memory and keeps no state besides a per-device cache of
 * the compute-unit count and a thread-local error string.
 *
 * Asynchrony.  Calls enqueue kernels on the caller's HIP stream and return
 * without synchronising.  Buffers must stay valid until the stream has passed
 * the call.  Two calls that share a workspace must be ordered on one stream.
 *
 * Errors.  All argument checks run before anything is enqueued: a call that
 * returns GDN_E_INVALID / GDN_E_UNSUPPORTED / GDN_E_WORKSPACE has written
 * nothing.  GDN_E_HIP reports a failed launch (the message carries HIP's
 * error string).  gdn_last_error() returns a description of the last non-OK
 * status on the calling thread.  Nothing throws or aborts across this ABI.
 * Non-finite inputs propagate; they are not detected.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ABI_VERSION 11

typedef enum {
  GDN_OK = 0,
  GDN_E_INVALID = 1,     /* null pointer, bad size, misalignment, bad cu_seqlens, ... */
  GDN_E_UNSUPPORTED = 2, /* dtype / head-size combination not built */
  GDN_E_WORKSPACE = 3,   /* workspace missing or smaller than *_workspace_size */
  GDN_E_HIP = 4          /* a HIP launch or query failed */
} gdn_status;

typedef enum { GDN_F32 = 0, GDN_BF16 = 1 } gdn_dtype;

/* Arguments shared by forward and backward. */
typedef struct {
  int32_t dtype;               /* gdn_dtype of q, k, v, beta (and o, do, dq, dk, dv, dbeta) */
  int32_t B, T, H, Dk, Dv;     /* with cu_seqlens: B == 1 and T = total packed tokens */
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const void* beta;
  const float* h0;             /* nullable: zero initial state */
  float scale;                 /* output scale; the usual choice is Dk^-0.5 */
  const int32_t* cu_seqlens;   /* nullable device pointer [N+1] */
  const int32_t* cu_seqlens_host; /* host copy of the same [N+1]; required with cu_seqlens.  The
                                  host copy sizes the work and the workspace; the kernels read
                                  the device copy.  If the device copy starts at a nonzero
                                  value, ends at a value other than T, has a negative length or
                                  gives other chunk or segment totals than the host copy, the
                                  call writes no output (o, hT and the gradients are left as
                                  they were) and reads nothing past its buffers; the status is
                                  still GDN_OK, since nothing is checked on the host side. */
  int32_t num_seqs;            /* N: len(cu_seqlens) - 1, or B when cu_seqlens is NULL */
  int32_t cp_mode;             /* intra-card sequence splitting: 0 = automatic,
                                  -1 = off (one segment per sequence and head),
                                  k > 0 = segments of k chunks (64 tokens each) */
  void* workspace;             /* device scratch of at least workspace_bytes */
  size_t workspace_bytes;
  /* Optional input pre-processing inside the kernels (0 = off):
   *   qk_norm:  q and k are raw; each (token, head) vector is divided by
   *             sqrt(|x|^2 + 1e-6) before use;
   *   gate_act: g and beta hold logits a, b; the kernels use
   *             g = -gate_scale[h] * softplus(a) and beta = sigmoid(b).
   * The backward then returns dq, dk, dg, dbeta with respect to these raw
   * inputs.  Outputs o, hT and the states are unchanged in meaning. */
  int32_t qk_norm;
  int32_t gate_act;
  const float* gate_scale;     /* nullable [H] fp32 (1 when NULL); only with gate_act */
} gdn_common_args;

typedef struct {
  gdn_common_args a;
  void* o;                     /* [B,T,H,Dv] dtype, written */
  float* hT;                   /* nullable [N,H,Dk,Dv] fp32, written */
  void* h_save;                /* nullable, 16-byte aligned, gdn_chunk_states_bytes(&a) bytes: the
                                  state at the start of every 64-token chunk, written for a later
                                  gdn_chunk_bwd (layout below) */
  float* t_save;               /* nullable, 16-byte aligned, gdn_chunk_t_bytes(&a) bytes: every
                                  chunk's matrix T (below), written for a later gdn_chunk_bwd */
} gdn_fwd_args;

typedef struct {
  gdn_common_args a;           /* the forward's inputs; the backward recomputes what it needs */
  const void* h_saved;         /* nullable: h_save of a gdn_chunk_fwd call on the same inputs;
                                  given, the backward reads the chunk states instead of
                                  recomputing them (no forward replay) */
  const float* t_saved;        /* nullable: t_save of a gdn_chunk_fwd call on the same inputs;
                                  given, the backward reads every chunk's T instead of solving
                                  for it once itself */
  const void* do_;             /* [B,T,H,Dv] dtype: gradient of o */
  const float* dhT;            /* nullable [N,H,Dk,Dv]: gradient of hT (NULL = zero) */
  void* dq;                    /* [B,T,H,Dk] dtype, written */
  void* dk;                    /* [B,T,H,Dk] dtype, written */
  void* dv;                    /* [B,T,H,Dv] dtype, written */
  void* dbeta;                 /* [B,T,H] dtype, written */
  float* dg;                   /* [B,T,H] fp32, written */
  float* dh0;                  /* nullable [N,H,Dk,Dv] fp32, written */
} gdn_bwd_args;

/* Bytes of device workspace gdn_chunk_fwd / gdn_chunk_bwd need for these
 * arguments (pointers other than cu_seqlens_host are not read, except that the
 * forward needs less when t_save is non-NULL and the backward less when
 * h_saved or t_saved is).  Returns 0 and sets the error string when the
 * arguments are invalid. */
size_t gdn_chunk_fwd_workspace_size(const gdn_fwd_args* args);
size_t gdn_chunk_bwd_workspace_size(const gdn_bwd_args* args);

/* Bytes of the saved chunk states (h_save / h_saved) for these arguments:
 * C * H * (Dk * Dv + 64 * Dv) elements of the input dtype (bf16: C * H *
 * (Dk * Dv + 2 * 64 * Dv)), C = sum over sequences of ceil(len / 64).  The
 * first C * H * Dk * Dv elements are the
 * states: state (c, h) is h (= S^T, Dk x Dv) at the start of chunk c (chunks
 * numbered sequence after sequence), rounded to the dtype, stored at element
 * offset (c * H + h) * Dk * Dv in 4 x 16 blocks: h[i][j] (key i, value j) sits at
 *     ((i / 4) * (Dv / 16) + j / 16) * 64 + (i % 4) * 16 + j % 16
 * (each block row-major and contiguous, blocks in row-major order), so that
 * the state can be read both along and across its rows in whole cache lines.
 * Then, at element offset C * H * Dk * Dv + (c * H + h) * 64 * Dv, each
 * chunk's value residual U = T (diag(beta) V - diag(beta Gam) K h), 64 x Dv
 * (h the chunk-start state, Gam_r = exp(G_r), T and G as for
 * gdn_chunk_t_bytes; rows past a sequence's end are zero), stored as Dv / 16
 * column blocks of 64 x 16, each row-major and contiguous: U[r][j] sits at
 *     (j / 16) * 1024 + r * 16 + j % 16.
 * For bf16 a third part follows, at element offset C * H * (Dk * Dv + 64 * Dv),
 * laid out like U: bf16(U - bf16(U)), the residual of U's rounding (the
 * backward's decay gradient takes U to about 16 bits).
 * Returns 0 and sets the error string for invalid arguments (and returns 0
 * without error when there are no tokens). */
size_t gdn_chunk_states_bytes(const gdn_common_args* a);

/* Bytes of the saved chunk matrices (t_save / t_saved): C * H * (64 * 64 + 324)
 * fp32 values, C as above.  Entry (c, h), 16 KiB at element offset
 * (c * H + h) * 4096, holds the 64 x 64 row-major lower-triangular matrix
 *     T = (I + diag(beta) strict_lower((K K^T) * D))^-1,   D[r][i] = exp(G_r - G_i),
 * of chunk c and head h (K: the chunk's 64 keys as rows, after the optional
 * normalisation; beta after the optional activation; G_r the running sum of
 * g over the chunk up to row r), the inverse of the chunk's unit lower-
 * triangular system in the WY/UT form ("FlashQLA resource", section 3).  Rows
 * past a sequence's end have beta = 0 (rows of the identity).  For fp32 inputs
 * the entry is T in fp32; for bf16 inputs it is two 64 x 64 row-major bf16
 * planes, T rounded to bf16 and then the residual T - that value rounded to
 * bf16 (their sum carries T to about 16 significant bits; the forward and
 * reverse state chains read the first plane only).  After the
 * C * H matrices, at element offset C * H * 4096 + (c * H + h) * 324, the
 * chunk's scalar record (g, beta after the optional activation; rows past a
 * sequence end have g = beta = 0): G_r (64 values), exp(G_r), exp(G_63 - G_r),
 * beta_r, beta_r exp(G_r), then Lambda = sum_r [g_r + log max(1, |1 - beta_r
 * |k_r|^2|)] (the log-bound on the chunk's state transition), exp(G_63), 0, 0.
 * Returns 0 and sets the error string for invalid arguments (and returns 0
 * without error when there are no tokens). */
size_t gdn_chunk_t_bytes(const gdn_common_args* a);

/* Forward: o and (optionally) hT, the chunk states and the chunk matrices T
 * -- the chunked prefill forward pass ("FlashQLA resource", section 2 "What It
 * Actually Is", and section 3 for the reformulated chunk form and the
 * intra-card splitting; "Qwen's FlashQLA targets the expensive bit of
 * long-context AI", section "What happened").  stream is a hipStream_t (NULL =
 * default stream). */
gdn_status gdn_chunk_fwd(const gdn_fwd_args* args, void* stream);

/* Bytes of the scratch array gdn_chunk_fwd_noalloc uses in place of a workspace. */
#define GDN_NOALLOC_SCRATCH_BYTES (64u << 20)

/* gdn_chunk_fwd without a workspace, for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that
 * forbid allocation.  Same arguments and results as gdn_chunk_fwd, except that
 * a.workspace / a.workspace_bytes are ignored: the work tables (and, when
 * t_save is NULL, every chunk's T and scalar record) go to a scratch array
 * of GDN_NOALLOC_SCRATCH_BYTES (64 MiB) that the library holds on each device
 * it runs on, from its load until the process ends.  Arguments whose
 * gdn_chunk_fwd_workspace_size exceeds that size are rejected with
 * GDN_E_WORKSPACE before anything is enqueued (without t_save that is about
 * 3,700 chunk-heads, e.g. 16 heads of 15,000 tokens; with t_save the tables
 * alone, a few bytes per chunk).  The call allocates nothing: no hipMalloc,
 * hipFree or allocating library routine, and no timing events
 * (gdn_profile_enable does not apply to it).  Every call on one device shares
 * that device's scratch, which keeps the last call's contents (the forward
 * reads nothing it has not written in the same call): calls that overlap on
 * one device -- on different streams, or from several threads without
 * ordering -- race and give undefined results; order them on one stream.
 * The first call on a device looks the scratch address up (not under graph
 * capture on that device, which forbids that query in some runtimes: make one
 * call outside capture first). */
gdn_status gdn_chunk_fwd_noalloc(const gdn_fwd_args* args, void* stream);

/* Backward: gradients of <do, o> + <dhT, hT> with respect to q, k, v, beta, g
 * and (optionally) h0 -- the matching backward pass ("FlashQLA resource",
 * section 2, and section 5 for its intra-card splitting; "Qwen's FlashQLA
 * targets the expensive bit of long-context AI", section "What happened").  It
 * recomputes the forward states from the inputs unless h_saved provides them,
 * and solves for each chunk's T once unless t_saved provides them.  stream as
 * for gdn_chunk_fwd. */
gdn_status gdn_chunk_bwd(const gdn_bwd_args* args, void* stream);

/* One recurrent decode step: every listed sequence takes one new token and
 * advances its state in place.  The pages present the kernels as serving
 * training and inference ("Qwen's FlashQLA targets the expensive bit of
 * long-context AI", section "What happened"; "FlashQLA resource", section 4);
 * after a prefill (gdn_chunk_fwd with hT) the state continues token by token
 * with the same recurrence, per sequence n and head:
 *     S <- exp(g) S (I - beta k k^T) + beta v k^T,      o = scale * S q
 * with the state stored as h = S^T (fp32 [Dk, Dv], as hT of the forward).
 *
 * Layouts (row-major, last dimension contiguous, device memory, every pointer
 * 16-byte aligned except g and beta):
 *   q, k [N, H, Dk], v, o [N, H, Dv] dtype;  g [N, H] fp32;  beta [N, H] dtype;
 *   state [num_slots, H, Dk, Dv] fp32, read and written in place.
 * state_idx (nullable int32 [N], device): sequence n uses slot state_idx[n];
 * an index outside [0, num_slots) marks a padding entry, which is skipped
 * (its o is not written).  NULL means slot n (num_slots >= N).  Two
 * sequences of one call must not share a slot.
 * Supported: bf16 and fp32 with Dk, Dv in {64, 128}.  Errors as for the chunk
 * calls (checked before anything is enqueued); asynchronous on `stream`. */
typedef struct {
  int32_t dtype;               /* gdn_dtype of q, k, v, beta, o */
  int32_t N, H, Dk, Dv;
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const void* beta;
  float scale;
  float* state;
  const int32_t* state_idx;
  int32_t num_slots;
  void* o;
  int32_t qk_norm;             /* as in gdn_common_args */
  int32_t gate_act;
  const float* gate_scale;
} gdn_decode_args;

gdn_status gdn_decode_step(const gdn_decode_args* args, void* stream);

/* ---------------------------------------------------------------------------
 * Operators around the recurrence: what a layer built on it runs beside it --
 * a short causal convolution of its inputs, a selective state space scan in
 * the recurrence's place, a gated group norm of its outputs.  dtype, alignment,
 * ownership, streams and errors follow the rules above; bf16 and fp32 inputs
 * throughout, sums and states in fp32.  These functions were added beside the
 * chunk calls without changing any struct of theirs.
 *
 * Token strides (*_stride, in elements) let an input be a slice of a wider row:
 * token t of the flattened [B * T] tokens starts at pointer + t * stride, its
 * own entries contiguous.  A stride below the row's own width is invalid.
 * 16-byte accesses are used where pointers, widths and strides allow them, and
 * element accesses elsewhere; only the scan requires them (below). */

/* Short causal depthwise convolution over [B, T, D], channels last:
 *     u_t = bias + sum_{k < W} w_k x_{t-W+1+k},    y_t = u_t, or u_t sigmoid(u_t) with silu
 * per channel, W in 2..4.  The W-1 inputs before a sequence's start are its
 * initial state (rows oldest first; zero when NULL); its final state is its
 * last W-1 inputs, initial state included when it is shorter.  cu_seqlens
 * (device, int32 [num_seqs + 1], B == 1) packs sequences; tokens at or past
 * cu_seqlens[N] belong to none: their y and dx are left as they were.
 * B * T stays below 2^31 - 1024 tokens. */
typedef struct {
  int32_t dtype;
  int32_t B, T, D, W;
  const void* x;               /* [B, T, D] */
  int64_t x_stride;
  const void* w;               /* [D, W] */
  const void* bias;            /* nullable [D] */
  const void* init;            /* nullable [N, W-1, D] */
  const int32_t* cu_seqlens;   /* nullable */
  int32_t num_seqs;            /* N; B when cu_seqlens is NULL */
  int32_t silu;                /* 0 or 1 */
} gdn_conv_args;

typedef struct {
  gdn_conv_args a;
  void* y;                     /* [B, T, D], written */
  void* final_state;           /* nullable [N, W-1, D], written */
} gdn_conv_fwd_args;

typedef struct {
  gdn_conv_args a;
  const void* dy;              /* [B, T, D] */
  const void* dfinal;          /* nullable [N, W-1, D]: gradient of the final state */
  void* dx;                    /* [B, T, D], written */
  void* dw;                    /* [D, W], written */
  void* dbias;                 /* nullable [D], written */
  void* dinit;                 /* nullable [N, W-1, D], written */
  void* workspace;             /* gdn_conv_bwd_workspace_size bytes, 16-byte aligned */
  size_t workspace_bytes;
} gdn_conv_bwd_args;

typedef struct {               /* one token for each of N sequences */
  int32_t dtype;
  int32_t N, D, W;
  const void* x;               /* [N, D] */
  int64_t x_stride;
  void* state;                 /* [num_slots, W-1, D], advanced in place */
  const int32_t* state_idx;    /* nullable [N]; out of range: padding, skipped (as gdn_decode_step) */
  int32_t num_slots;
  const void* w;
  const void* bias;            /* nullable */
  int32_t silu;
  void* y;                     /* [N, D], written */
} gdn_conv_step_args;

gdn_status gdn_conv_fwd(const gdn_conv_fwd_args* args, void* stream);
size_t gdn_conv_bwd_workspace_size(const gdn_conv_bwd_args* args);
gdn_status gdn_conv_bwd(const gdn_conv_bwd_args* args, void* stream);
gdn_status gdn_conv_step(const gdn_conv_step_args* args, void* stream);

/* Selective state space scan, per sequence and head h of group g = h / (H / G):
 *     d_t = dt_t, or softplus(dt_t + dt_bias[h]) with dt_softplus  (dt_bias is added either way)
 *     h_t = exp(d_t A[h]) h_{t-1} + d_t B_t x_t^T      (Dk x Dv),   h_0 = h0
 *     y_t = h_t^T C_t + D[h] x_t,                                  hT = the last h_t
 * A <= 0 and d_t >= 0 in the intended domain (the decay never exceeds 1); a
 * token with d_t = 0 leaves the state as it is.  Dk in {64, 128}; Dv a
 * multiple of 64 up to 256; H a multiple of G.  x, B and C need 16-byte
 * aligned pointers and token strides of whole 16 bytes, below 2^22 elements; at
 * most 65535 sequences.  A value that is not finite makes its sequence not finite
 * from the start of its chunk of 64 tokens on, and no other sequence.
 * cu_seqlens / cu_seqlens_host as for the chunk calls.  seg_mode: sequences
 * are cut into segments that run side by side and are joined exactly
 * (0 = automatic, -1 = off, k > 0 = segments of k chunks of 64 tokens).
 * Precision: fp32 results carry fp32's, and dB, dC and ddt are rounded once.  Inside
 * a bf16 y and dx the 64 x 64 matrix of a chunk and the state entering it are
 * rounded to bf16 as well (rms error 1.8e-3 to 2.1e-3 of the values, of which the
 * output's rounding is 1.65e-3), unless round_once is 1: then y and dx too are the
 * fp32 result rounded once (2 to 10 % more time).  The
 * gradient's workspace holds a state for every chunk: 4 Dk Dv H bytes for every
 * 64 tokens. */
typedef struct {
  int32_t dtype;               /* of x, B, C (and y, dy, dx, dB, dC) */
  int32_t dt_dtype;            /* of dt (and ddt): GDN_F32, or GDN_BF16 */
  int32_t B, T, H, G, Dk, Dv;
  const void* x;               /* [B, T, H, Dv] */
  const void* dt;              /* [B, T, H] */
  const void* b;               /* [B, T, G, Dk] */
  const void* c;               /* [B, T, G, Dk] */
  int64_t x_stride, dt_stride, b_stride, c_stride;
  const float* A;              /* [H] */
  const float* D;              /* nullable [H] */
  const float* dt_bias;        /* nullable [H] */
  int32_t dt_softplus;
  int32_t round_once;          /* 0 or 1 (see above) */
  const float* h0;             /* nullable [N, H, Dk, Dv] */
  const int32_t* cu_seqlens;
  const int32_t* cu_seqlens_host;
  int32_t num_seqs;
  int32_t seg_mode;
  void* workspace;
  size_t workspace_bytes;
} gdn_scan_args;

typedef struct {
  gdn_scan_args a;
  void* y;                     /* [B, T, H, Dv], written */
  float* hT;                   /* nullable [N, H, Dk, Dv], written */
  float* h_save;               /* nullable, gdn_scan_states_bytes(&a) bytes: the state entering every
                                  segment, for gdn_scan_bwd */
} gdn_scan_fwd_args;

typedef struct {
  gdn_scan_args a;
  const float* h_saved;        /* nullable: h_save of the forward on the same inputs (else recomputed) */
  const void* dy;              /* [B, T, H, Dv], 16-byte aligned */
  const float* dhT;            /* nullable [N, H, Dk, Dv] */
  void* dx;                    /* [B, T, H, Dv], written */
  void* ddt;                   /* [B, T, H], written */
  void* db;                    /* [B, T, G, Dk], written */
  void* dc;                    /* [B, T, G, Dk], written */
  float* dA;                   /* [H], written */
  float* dD;                   /* nullable [H], written */
  float* ddt_bias;             /* nullable [H], written */
  float* dh0;                  /* nullable [N, H, Dk, Dv], written */
} gdn_scan_bwd_args;

typedef struct {               /* one token for each of N sequences */
  int32_t dtype, dt_dtype;
  int32_t N, H, G, Dk, Dv;     /* as for the scan */
  const void* x;               /* [N, H, Dv] */
  const void* dt;              /* [N, H] */
  const void* b;               /* [N, G, Dk] */
  const void* c;
  int64_t x_stride, dt_stride, b_stride, c_stride;
  const float* A;
  const float* D;
  const float* dt_bias;
  int32_t dt_softplus;
  float* state;                /* [num_slots, H, Dk, Dv], advanced in place */
  const int32_t* state_idx;    /* nullable [N], as gdn_decode_step */
  int32_t num_slots;
  void* y;                     /* [N, H, Dv], written */
} gdn_scan_step_args;

size_t gdn_scan_fwd_workspace_size(const gdn_scan_fwd_args* args);
size_t gdn_scan_bwd_workspace_size(const gdn_scan_bwd_args* args);
size_t gdn_scan_states_bytes(const gdn_scan_args* a);  /* 0 when no sequence is cut */
gdn_status gdn_scan_fwd(const gdn_scan_fwd_args* args, void* stream);
gdn_status gdn_scan_bwd(const gdn_scan_bwd_args* args, void* stream);
gdn_status gdn_scan_step(const gdn_scan_step_args* args, void* stream);

/* Gated group norm over [R, G, D], channels last: every token's groups of D
 * channels are normalised on their own.
 *     v = x silu(z) with z and gate_first, else x
 *     n = (v - m) / sqrt(mean((v - m)^2) + eps),   m = mean(v) with center, else 0
 *     y = n w + bias,  times silu(z) with z and not gate_first
 * w and bias are [G, D], or [D] for all groups with shared.  R * G stays below
 * 2^31, G below 2^16. */
typedef struct {
  int32_t dtype;
  int64_t R;
  int32_t G, D;
  const void* x;               /* [R, G, D] */
  int64_t x_stride;
  const void* z;               /* nullable [R, G, D] */
  int64_t z_stride;
  const void* w;
  const void* bias;            /* nullable */
  int32_t shared, center, gate_first;
  float eps;                   /* > 0 */
} gdn_norm_args;

typedef struct {
  gdn_norm_args a;
  void* y;                     /* [R, G, D], written */
} gdn_norm_fwd_args;

typedef struct {
  gdn_norm_args a;
  const void* dy;              /* [R, G, D] */
  void* dx;                    /* [R, G, D], written */
  void* dz;                    /* [R, G, D], written; needed with z */
  void* dw;                    /* like w, written */
  void* dbias;                 /* like bias, written; needed with bias */
  void* workspace;
  size_t workspace_bytes;
} gdn_norm_bwd_args;

gdn_status gdn_norm_fwd(const gdn_norm_fwd_args* args, void* stream);
size_t gdn_norm_bwd_workspace_size(const gdn_norm_bwd_args* args);
gdn_status gdn_norm_bwd(const gdn_norm_bwd_args* args, void* stream);

/* Per-kernel timing, for benchmarks (off by default).  While enabled, every
 * kernel the library launches is bracketed by a pair of HIP events recorded on
 * the call's stream.  gdn_profile_read waits for the recorded events, adds
 * their elapsed times to per-kernel totals and writes up to `max` entries:
 * the kernel's name (static storage), total milliseconds and launch count.
 * It returns the number of distinct kernels seen since the last reset (or -1
 * on a HIP error).  gdn_profile_reset clears the totals.  Not thread-safe with
 * respect to concurrent calls on other threads. */
int gdn_profile_enable(int on);
int gdn_profile_read(int max, const char** names, double* ms, int* launches);
void gdn_profile_reset(void);

/* Thread-local description of the last non-OK status ("" if none). */
const char* gdn_last_error(void);

/* GDN_ABI_VERSION of the library. */
int gdn_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* GDN_H */

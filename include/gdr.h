/*
 * gdr.h -- C ABI of the chunked gated delta-rule backward for AMD MI355X (gfx950).
 *
 * The op.  Per sequence n and head h, with Dv x Dk state S and tokens t:
 *   qn = q / sqrt(|q|^2 + 1e-6), kn likewise, beta = sigmoid(b),
 *   lambda_t = g_t                                   (GDR_GATE_SCALAR, GDN)
 *   lambda_t = -exp(A_log[h]) * softplus(g_t + dt_bias[h])  (GDR_GATE_CHANNEL, KDA)
 *   lambda_t = gate_scale * sigmoid(exp(A_log[h]) * (g_t + dt_bias[h]))
 *                                        (GDR_GATE_CHANNEL_SIGMOID, the bounded KDA
 *                                         gate of the FlashKDA K1 page, section 5.2)
 *   S_t = S_{t-1} Diag(exp(lambda_t)) (I - beta_t kn_t kn_t^T) + beta_t v_t kn_t^T,
 *   o_t = scale * S_t qn_t,  S_0 = h0 (or 0).
 * The backward returns the gradients of L = sum_t <dO_t, o_t> + <dht, S_T> with
 * respect to q, k, v, g, the beta logit, h0, A_log and dt_bias.
 *
 * Citations (the pages describing the method):
 *  - FlashQLA GDN backward overview (lqnn.cn/news/272630), section 1: entry
 *    conventions -- dh0 returned in fp32 while dq/dk/dv are stored in bf16,
 *    dht optional (absent = zero); section 2: the state gradient recursion runs
 *    strictly from the last chunk to the first; section 3: the recursion
 *    dh <- g_last*dh + R^T dO + X^T Y with X = A_beta K.
 *  - FlashKDA backward "K1" page (yuyanqi.com), listing and sections 1-6: the
 *    prepare stage (L2-norm backward, reverse cumsum of the gate gradient plus
 *    the chunk-total term, gate backward, per-head parameter sums by atomics,
 *    beta-logit backward, tail-row masking).
 *
 * Memory and streams.  Every pointer is caller-owned.  Token tensors are
 * row-major [B, T, H, D] (dense) or [1, T_total, H, D] (varlen, B == 1 and
 * T == T_total); per-token scalars are [B, T, H]; states are [N, H, Dv, Dk]
 * fp32.  Device pointers must be 16-byte aligned.  The library never allocates,
 * frees or synchronises, and reads no host memory after a call returns: all
 * work is enqueued on `stream` (a hipStream_t; NULL = the null stream) as kernel
 * launches -- the chunk and sequence tables are written into the workspace by a
 * kernel that receives the sequence lengths as launch arguments -- so a call
 * can be recorded into a HIP graph.  The workspace carries state from
 * gdr_fwd_recompute to gdr_bwd; its layout is internal (gdr_workspace_region
 * exposes it for tests).  Outputs are overwritten, never accumulated.
 *
 * Errors.  All argument checks run before anything is enqueued; a non-OK status
 * means nothing was launched, except GDR_EHIP (a HIP call failed while
 * enqueueing).  gdr_last_error() returns a thread-local message for the last
 * non-OK status of the calling thread.
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
  GDR_EINVAL = 1,        /* bad argument: null/misaligned pointer, bad cu_seqlens, gate/param mismatch */
  GDR_EUNSUPPORTED = 2,  /* Dk != Dv, D not in {64, 128}, or a size beyond the int32 index range */
  GDR_EWORKSPACE = 3,    /* workspace smaller than gdr_workspace_bytes() */
  GDR_EHIP = 4           /* a HIP runtime call failed while enqueueing */
} gdr_status;

typedef enum { GDR_GATE_SCALAR = 0, GDR_GATE_CHANNEL = 1, GDR_GATE_CHANNEL_SIGMOID = 2 } gdr_gate;
typedef enum { GDR_BF16 = 0, GDR_F32 = 1 } gdr_dtype;

typedef struct {
  int32_t B, T, H, Dk, Dv;          /* dense: [B,T,H,D]; varlen: B == 1, T == total tokens */
  int32_t N;                        /* sequences: == B when dense, == len(cu_seqlens) - 1 when varlen */
  const int64_t* cu_seqlens_host;   /* host array [N+1], non-decreasing, [0] == 0, [N] == T; NULL = dense.
                                       Read during the call only. */
  int32_t gate;                     /* gdr_gate */
  int32_t dtype;                    /* gdr_dtype of q, k, v, g, b, dO and of dq, dk, dv, dg, dbeta */
  float scale;                      /* readout scale (usually 1/sqrt(Dk)) */
  float gate_scale;                 /* GDR_GATE_CHANNEL_SIGMOID: the bound of the per-token log decay,
                                       finite and <= 0 (natural log: the pages' log2-unit bound times
                                       ln 2); ignored otherwise */
  int32_t Hk;                       /* heads of q and k (grouped heads): 0 means H; else H % Hk == 0 and
                                       value head h reads key head h / (H / Hk), and dq, dk sum over the
                                       H / Hk value heads of each key head (FlashQLA GDN overview,
                                       section 4: hk and hv head counts, GQA tests).  Hk < H needs
                                       workspace for the per-value-head dq, dk before that sum. */
  int32_t seq_split;                /* segments per sequence for the two chunk recursions: 0 = chosen
                                       by the library (a split pays only when few (sequence, head)
                                       pairs leave compute units idle), 1 = never split, n >= 2 = split
                                       every sequence of two or more chunks into min(n, 16, its chunks)
                                       runs of whole chunks.  The split is exact (the chunk recursions
                                       are affine in the carried state; the FlashQLA overview's section
                                       3 splits them across devices with a warm-up approximation
                                       instead): each segment runs from a zero state with its transfer
                                       product, the true boundary states are composed in order, and
                                       every segment then runs again from its true state.  Results
                                       agree with the unsplit recursion up to rounding. */
} gdr_shape;

/* Below, CHANNEL stands for either per-channel gate (GDR_GATE_CHANNEL or
 * GDR_GATE_CHANNEL_SIGMOID): both take the raw gate g, A_log and dt_bias and return
 * dg, dA_log and ddt_bias in the same shapes. */
typedef struct {                    /* device pointers; the token tensors (q, k, v, g, beta_logit) may be
                                       NULL when B * T == 0 */
  const void *q, *k;                /* [B,T,Hk,Dk] dtype (Hk = H unless grouped) */
  const void *v;                    /* [B,T,H,Dv] dtype */
  const void *g;                    /* SCALAR: [B,T,H] log decay; CHANNEL: [B,T,H,Dk] raw gate; dtype */
  const void *beta_logit;           /* [B,T,H] dtype (pre-sigmoid) */
  const float *A_log;               /* CHANNEL: [H]; SCALAR: must be NULL */
  const float *dt_bias;             /* CHANNEL: [H,Dk]; SCALAR: must be NULL */
  const float *h0;                  /* [N,H,Dv,Dk] or NULL (zero initial state) */
} gdr_inputs;

typedef struct {                    /* device pointers, all overwritten; the token gradients (dq, dk, dv,
                                       dg, dbeta) may be NULL when B * T == 0 */
  void *dq, *dk;                    /* [B,T,Hk,Dk] dtype (Hk = H unless grouped) */
  void *dv;                         /* [B,T,H,Dv] dtype */
  void *dg;                         /* SCALAR: [B,T,H]; CHANNEL: [B,T,H,Dk] (w.r.t. the raw gate); dtype */
  void *dbeta;                      /* [B,T,H] dtype, w.r.t. the logit */
  float *dh0;                       /* [N,H,Dv,Dk] or NULL (not returned) */
  float *dA_log, *ddt_bias;         /* CHANNEL: [H], [H,Dk] required; SCALAR: must be NULL */
} gdr_grads;

/* Bytes of workspace the compute calls need for this shape (host only; no
 * device work).  The workspace holds the per-chunk intermediates of the chunked
 * form: the states at chunk starts and the state gradients at chunk ends (the
 * quantities the FlashQLA overview's sections 2-3 carry between its forward
 * and backward passes), the in-chunk UT/WY inverse, the gate cumsum and the
 * chunk/sequence tables.  Returns GDR_EINVAL / GDR_EUNSUPPORTED for a bad shape. */
gdr_status gdr_workspace_bytes(const gdr_shape* shape, size_t* bytes);

/* Forward recompute: the preprocessing that precedes the backward's main
 * kernels (FlashQLA GDN backward overview, section 1: a backward call is a
 * preprocessing stage plus two main kernels, fed the in-chunk cumsum of the
 * gate; section 3: the UT/WY product X = A_beta K).  Per chunk: normalisation,
 * beta, the in-chunk gate cumsum, the UT/WY inverse
 * A = (I + StrictLower(diag(beta) (K K^T o decay)))^-1, U' = A diag(beta) V and
 * W = A diag(beta) K e^Gamma; then the serial state pass storing the state at
 * the start of every chunk and v_new = U' - W S^T.
 * Arguments: shape and inputs as above; ws / ws_bytes a device workspace of at
 * least gdr_workspace_bytes(shape) bytes, 256-byte aligned; o the forward output
 * [B,T,H,Dv] in the input dtype (o_t = scale S_t qn_t, formed chunk-parallel as
 * Qbar S_n^T + P U) or NULL to skip it; ht the final state per sequence
 * [N,H,Dv,Dk] fp32 or NULL.  Leaves what gdr_bwd needs in `ws`; every stage
 * only reads inputs and what earlier stages wrote, so the call may be repeated.
 * Errors: GDR_EINVAL (null required / misaligned pointer, bad shape, gate and
 * parameter mismatch), GDR_EUNSUPPORTED, GDR_EWORKSPACE; nothing is enqueued
 * then.  GDR_EHIP if a launch fails. */
gdr_status gdr_fwd_recompute(const gdr_shape* shape, const gdr_inputs* in, void* ws, size_t ws_bytes, void* o,
                             float* ht, void* stream);

/* The forward pass for training use: gdr_fwd_recompute with the output o
 * required (GDR_EINVAL if NULL while there are tokens).  o = scale S_t qn_t per
 * token, formed per chunk as Qbar S_n^T + P U (Qbar = scale qn e^Gamma,
 * P = scale (Qn Kn^T o decay) on and below the diagonal, U = v_new): the chunked
 * form of the read-out (FlashQLA GDN overview, section 3).  Leaves the same
 * workspace, so gdr_bwd may follow. */
gdr_status gdr_fwd(const gdr_shape* shape, const gdr_inputs* in, void* ws, size_t ws_bytes, void* o, float* ht,
                   void* stream);

/* Backward, after gdr_fwd_recompute on the same shape, inputs and workspace:
 *  - the reverse-chunk state-gradient recursion, run strictly from the last
 *    chunk to the first (FlashQLA overview, section 2; its section 3 gives the
 *    recursion dh <- g_last dh + R^T dO + X^T Y with X = A_beta K), starting
 *    from dht (NULL = zero, section 1) and returning dh0 in fp32 (section 1);
 *  - the chunk-parallel gradients of q, k, v, beta and the gate (section 2: the
 *    compute-bound main backward);
 *  - the prepare-backward of the FlashKDA K1 page: L2-norm backward (section
 *    3.3), reverse cumsum of the gate gradient plus the chunk-total term
 *    (section 5), gate-function backward and the per-head sums dA_log, ddt_bias
 *    (section 5.2), beta-logit backward (section 6), tail rows masked (section 8).
 * dO: [B,T,H,Dv] dtype, required unless there are no tokens; dht: [N,H,Dv,Dk]
 * fp32 or NULL; grads: every token gradient required (dq, dk [B,T,Hk,Dk], dv,
 * dg, dbeta in the input dtype), dh0 optional, dA_log / ddt_bias required for
 * the per-channel gates and NULL for the scalar gate.  Errors as for
 * gdr_fwd_recompute. */
gdr_status gdr_bwd(const gdr_shape* shape, const gdr_inputs* in, const void* dO, const float* dht,
                   void* ws, size_t ws_bytes, gdr_grads* grads, void* stream);

/* The whole backward in one call: the same kernels as gdr_fwd_recompute
 * followed by gdr_bwd, except that the forward state pass and the reverse
 * state-gradient recursion (which do not depend on each other) run side by
 * side in one launch.  Same results, bit for bit; ht may be NULL.  Arguments
 * and errors as gdr_fwd_recompute and gdr_bwd together. */
gdr_status gdr_fwd_bwd(const gdr_shape* shape, const gdr_inputs* in, const void* dO, const float* dht,
                       void* ws, size_t ws_bytes, gdr_grads* grads, float* ht, void* stream);

/* Workspace regions, for tests that inspect intermediates.  Layouts (NC =
 * total chunks of 64 tokens over all sequences, chunk c of sequence n numbered
 * after all chunks of sequences < n; rows past a sequence's end are padding):
 *   GDR_WS_STATE   bf16 [H][NC][Dv][Dk]  state at the start of each chunk
 *   GDR_WS_DSTATE  bf16 [H][NC][Dv][Dk]  gradient w.r.t. the state at the end of each chunk
 *   GDR_WS_U       bf16 [H][NC][Dv][64]  v_new = U' - W S^T, transposed (column v of the chunk is contiguous)
 *   GDR_WS_A       bf16 [H][NC][64][64]  the UT/WY inverse
 *   GDR_WS_GAMMA   fp32 [H][NC][64] (SCALAR) or [H][NC][64][Dk] (CHANNEL): in-chunk gate cumsum
 */
enum { GDR_WS_STATE = 0, GDR_WS_DSTATE = 1, GDR_WS_U = 2, GDR_WS_A = 3, GDR_WS_GAMMA = 4 };
gdr_status gdr_workspace_region(const gdr_shape* shape, int32_t which, size_t* offset, size_t* bytes);

/* One stage of gdr_fwd_bwd enqueued alone, for benchmarks and kernel profiles
 * (same arguments as gdr_fwd_bwd; the workspace must already hold what the
 * earlier stages leave there, e.g. after one gdr_fwd_bwd call).  Stages:
 *   GDR_STAGE_PREP        per-chunk prologue and UT/WY inverse (one launch)
 *   GDR_STAGE_CHAIN_FWD   forward state pass alone
 *   GDR_STAGE_CHAIN_BWD   reverse state-gradient recursion alone
 *   GDR_STAGE_CHAIN_BOTH  both recursions in one launch, as gdr_fwd_bwd runs them
 *   GDR_STAGE_GRADS       chunk-parallel gradients and the prepare-backward (norm,
 *                         sigmoid, gate backward); writes every per-token gradient
 *   GDR_STAGE_FINISH      the per-head reduction of dA_log, ddt_bias (CHANNEL) and the
 *                         dq, dk group sums (grouped heads); enqueues nothing for
 *                         GDR_GATE_SCALAR with Hk = H */
enum { GDR_STAGE_PREP = 0, GDR_STAGE_CHAIN_FWD = 1, GDR_STAGE_CHAIN_BWD = 2, GDR_STAGE_CHAIN_BOTH = 3,
       GDR_STAGE_GRADS = 4, GDR_STAGE_FINISH = 5 };
gdr_status gdr_run_stage(const gdr_shape* shape, const gdr_inputs* in, const void* dO, const float* dht,
                         void* ws, size_t ws_bytes, gdr_grads* grads, float* ht, int32_t stage, void* stream);

/* gdr_fwd_bwd without a caller-supplied workspace, for callers that cannot
 * allocate device memory (code being captured into a HIP graph, tight serving
 * loops, harnesses that forbid allocation).  The workspace is a device array of
 * 128 MiB (134217728 bytes) that the library holds on every GPU it runs on until
 * the process ends; the call itself allocates and
 * frees nothing.  Shapes whose gdr_workspace_bytes() exceed it are rejected with
 * GDR_EWORKSPACE before anything is enqueued.  Every call on one GPU uses that
 * GPU's single array, so calls that overlap in time on one GPU (different
 * streams, threads or processes sharing the array) race; calls in order on one
 * stream are safe.  Inputs, outputs and errors as gdr_fwd_bwd.  The first call
 * on a device looks up that device's copy of the array (hipGetSymbolAddress). */
gdr_status gdr_fwd_bwd_noalloc(const gdr_shape* shape, const gdr_inputs* in, const void* dO, const float* dht,
                               gdr_grads* grads, float* ht, void* stream);

/* ------------------------------------------------------------------------
 * Single-token step of the gated delta rule (serving).
 *
 * One token for each of N rows: shape is a dense gdr_shape with T == 1 and
 * B == N rows (seq_split is ignored), `in` as above with h0 NULL.  `state` holds
 * P states [P,H,Dv,Dk] fp32, as gdr_fwd's ht leaves them, updated in place; row
 * n works on state slots[n] (slots: device int32 [N]; NULL: slot n, which needs
 * P >= N).  Row n's token:
 *   S <- S Diag(exp(lambda)) (I - beta kn kn^T) + beta v kn^T,  o = scale S qn.
 * A row whose slot is outside [0, P) is padding: no state is touched and its row
 * of o is left as it was.  Rows with the same slot are successive tokens of one
 * sequence, taken in the order of n.  o: [N,1,H,Dv] dtype.  No workspace.
 * No output may overlap an input.  Each row reads all of `slots` (N^2 reads in
 * all).  Errors as gdr_fwd_recompute, and GDR_EINVAL for T != 1, a varlen shape, an
 * h0, a NULL state, P < 0 or P < N without slots, and GDR_EUNSUPPORTED from N H Dk /
 * 32 = 2^24 on. */
gdr_status gdr_step(const gdr_shape* shape, const gdr_inputs* in, float* state, int32_t P, const int32_t* slots,
                    void* o, void* stream);

/* ------------------------------------------------------------------------
 * Gated linear recurrence: the channel-wise member of the same family, for
 * layers whose state is one number per channel.  Per sequence, head and channel:
 *   a_t = exp(lambda_t), lambda_t by the gate as in the delta rule above,
 *   s_t = a_t s_{t-1} + m_t x_t,   m_t = 1, or 1 - a_t with `convex`,
 *   y_t = s_t,  s_0 = h0 (or 0).
 * GDR_GATE_SCALAR takes one log decay per token and head, shared by the head's D
 * channels (D == 1: one per channel); the per-channel gates take g, A_log and
 * dt_bias as the delta rule does.  The log decay is meant to be <= 0; -inf is a
 * reset (a = 0), and so is one below -87.3 (exp(lambda) < 2^-126).  A positive one is
 * taken as it stands as long as the product of exp(lambda) over any run of tokens
 * stays in the fp32 range.  Infinities and NaN in x, h0, dy and dht go where the
 * formulas take them token by token, and no further (0 times infinity is NaN: an
 * infinite state does not pass a reset unharmed).
 * The backward returns the gradients of L = sum_t <dy_t, y_t> + <dht, s_T>.
 * x, y: [B,T,H,D] (or packed [1,T,H,D]), 1 <= D <= 256 with D == 1 or a multiple
 * of 8; B, T, N, cu_seqlens_host, dtype and alignment as in gdr_shape.  States,
 * products and sums are fp32; y, dx and dg are rounded once to dtype.
 * GDR_EUNSUPPORTED above 2^21 channels H D, from 2^31 tokens B T or 2^40 elements on,
 * and where a launch would take 2^32 threads: not with fewer than 2^24 tiles times
 * ceil(H D / 64), counting a tile for every 64 tokens of a sequence (at least one). */
typedef struct {
  int32_t B, T, H, D;               /* dense: [B,T,H,D]; varlen: B == 1, T == total tokens */
  int32_t N;                        /* sequences, as in gdr_shape */
  const int64_t* cu_seqlens_host;   /* as in gdr_shape (read during the call only) */
  int32_t gate;                     /* gdr_gate */
  int32_t dtype;                    /* gdr_dtype of x, g, y, dy, dx, dg */
  float gate_scale;                 /* GDR_GATE_CHANNEL_SIGMOID only, as in gdr_shape */
  int32_t convex;                   /* 0: s = a s + x; 1: s = a s + (1 - a) x */
} gdr_scan_shape;

typedef struct {                    /* device pointers; x and g may be NULL when B * T == 0 */
  const void* x;                    /* [B,T,H,D] dtype */
  const void* g;                    /* SCALAR: [B,T,H] log decay; CHANNEL: [B,T,H,D] raw gate; dtype */
  const float *A_log, *dt_bias;     /* CHANNEL: [H], [H,D]; SCALAR: must be NULL */
  const float* h0;                  /* [N,H,D] or NULL (zero initial state) */
} gdr_scan_inputs;

typedef struct {                    /* device pointers, all overwritten; dx and dg may be NULL when B * T == 0 */
  void *dx, *dg;                    /* as x and g */
  float* dh0;                       /* [N,H,D] or NULL (not returned) */
  float *dA_log, *ddt_bias;         /* CHANNEL: [H], [H,D] required; SCALAR: must be NULL */
} gdr_scan_grads;

gdr_status gdr_scan_workspace_bytes(const gdr_scan_shape* shape, size_t* bytes);

/* Forward: y (required unless there are no tokens) and optionally the final
 * states ht [N,H,D] fp32 (a sequence without tokens returns its h0).  `ws` needs
 * gdr_scan_workspace_bytes(), 256-byte aligned, with any content; afterwards it
 * holds the states that gdr_scan_bwd on the same shape and inputs starts from.
 * Calls that overlap in time need a workspace each.  Outputs must not overlap
 * inputs.  Errors as gdr_fwd_recompute. */
gdr_status gdr_scan_fwd(const gdr_scan_shape* shape, const gdr_scan_inputs* in, void* ws, size_t ws_bytes, void* y,
                        float* ht, void* stream);

/* Backward, after gdr_scan_fwd on the same shape, inputs and workspace (which it
 * leaves fit for another gdr_scan_bwd).  dy as y, required unless there are no
 * tokens; dht [N,H,D] fp32 or NULL (zero).  Outputs must not overlap inputs. */
gdr_status gdr_scan_bwd(const gdr_scan_shape* shape, const gdr_scan_inputs* in, const void* dy, const float* dht,
                        void* ws, size_t ws_bytes, const gdr_scan_grads* grads, void* stream);

/* One token for each of N rows on a pool of states [P,H,D] fp32, updated in
 * place: shape dense with T == 1, in->h0 NULL; state, P, slots, padding rows and
 * rows that share a slot as in gdr_step.  y: [N,1,H,D] dtype. */
gdr_status gdr_scan_step(const gdr_scan_shape* shape, const gdr_scan_inputs* in, float* state, int32_t P,
                         const int32_t* slots, void* y, void* stream);

/* ------------------------------------------------------------------------
 * Root-mean-square norm of rows with the residual's addition: what stands
 * between the recurrences and the projections (over one head's channels of an
 * output o, or over the whole model width).
 *   r = x + res (res NULL: r = x),  n = r / sqrt(mean(r^2) + eps),  y = n * w.
 * x, res, y, res_out: [rows,width] dtype; w: [width] fp32 or NULL (ones).  r is
 * kept in fp32 for y; res_out (required with res, NULL without) is r rounded to
 * dtype and may be res or x itself; y may be x or res itself unless that is
 * res_out.  1 <= width <= 32768; fewer than 2^31 rows, and so many that a launch
 * stays under 2^32 threads (fewer than 2^22 rows of any width do, fewer than 2^24
 * of up to 16 KiB), else GDR_EUNSUPPORTED.  Squares are summed in fp32: a row whose
 * sum of squares leaves that range gives zeros or NaN; with eps 0 a row of zeros
 * gives NaN. */
typedef struct {
  int64_t rows;
  int32_t width;
  int32_t dtype;                    /* gdr_dtype of x, res, res_out, y, r, dy, dres, dx */
  float eps;                        /* finite, >= 0 */
  int32_t group;                    /* gdr_norm_quant: channels per scale, 0 (the whole row) or 128; else ignored */
} gdr_norm_shape;

gdr_status gdr_norm_fwd(const gdr_norm_shape* shape, const void* x, const void* res, const float* w, void* y,
                        void* res_out, void* stream);

/* The same with an 8-bit output: per row and group of channels
 *   scale = max(max|y| / 448, 2^-126),  q = e4m3(y / scale)
 * (OCP e4m3, the fp32 quotient to nearest even), so that q * scale stands for y.  q:
 * [rows,width] bytes; scales: [rows,ceil(width / group)] fp32 (group 0: [rows,1];
 * the last group of a width that is no multiple of it is shorter).  A group that
 * holds a NaN gets a NaN scale and NaN bytes. */
gdr_status gdr_norm_quant(const gdr_norm_shape* shape, const void* x, const void* res, const float* w, void* q,
                          float* scales, void* res_out, void* stream);

/* Backward from r (res_out of the forward, or x without a residual; the row's
 * statistics are taken again from it):
 *   dr = (w dy - n mean(n w dy)) / sqrt(mean(r^2) + eps) + dres,  dw = sum_rows dy n
 * dr is the gradient of x and of res alike.  dres: the gradient that reaches
 * res_out from elsewhere, or NULL.  dx: [rows,width], may be dy or dres itself;
 * dw: [width] fp32 or NULL (not returned; then ws may be NULL).  ws:
 * gdr_norm_workspace_bytes(), 256-byte aligned, any content; calls that overlap
 * in time need one each.  Sums run in a fixed order. */
gdr_status gdr_norm_workspace_bytes(const gdr_norm_shape* shape, size_t* bytes);
gdr_status gdr_norm_bwd(const gdr_norm_shape* shape, const void* r, const float* w, const void* dy, const void* dres,
                        void* ws, size_t ws_bytes, void* dx, float* dw, void* stream);

/* ------------------------------------------------------------------------
 * Linear attention with a decay for each head: the delta rule's family without
 * its correction term, and with a decay that is a constant of the head.  Per
 * sequence and head:
 *   S_t = e^lambda S_{t-1} + v_t k_t^T,  o_t = scale S_t q_t,  S_0 = h0 (or 0).
 * The backward returns the gradients of L = sum_t <dO_t, o_t> + <dht, S_T> with
 * respect to q, k, v and h0 (the decay is a constant).  q and k are taken as they
 * are, without the delta rule's normalisation.
 * B, T, H, N, cu_seqlens_host, dtype, scale, Hk, the tensors' layouts and the
 * states [N,H,D,D] (row v, column k) as in gdr_shape; D is 64 or 128.  log_decay:
 * [H] fp32 on the device, meant to be <= 0; -inf keeps nothing of the state.  A
 * positive one is taken as it stands as long as e^(lambda n) and scale e^(lambda n)
 * stay in the fp32 range for every n up to the longest sequence.
 * States, products and sums are fp32.  With bf16 tensors the products of pairs of
 * tokens and the states are rounded to bf16 once where they are multiplied with
 * bf16 tensors; the states themselves are not: what a block adds to one keeps 16 bits
 * of significand, or 24 where the state is returned or starts another run of tokens, so
 * that asking for ht (dh0) may change the last bit of some o (dv).  An infinity or NaN
 * at a token reaches no token before it (after it, in the gradients of k and v) and no
 * other sequence; from there on, what the formulas make infinite or NaN is infinite or
 * NaN, not always the same of the two.  GDR_EUNSUPPORTED above 2^16 heads, and from
 * 2^20 blocks of 64 tokens times heads on (B T / 64 + N blocks). */
typedef struct {
  int32_t B, T, H, D;               /* dense: [B,T,H,D]; varlen: B == 1, T == total tokens */
  int32_t N;                        /* sequences, as in gdr_shape */
  const int64_t* cu_seqlens_host;   /* as in gdr_shape (read during the call only) */
  int32_t dtype;                    /* gdr_dtype of q, k, v, o, dO, dq, dk, dv */
  float scale;                      /* readout scale, finite */
  int32_t Hk;                       /* heads of q and k, as in gdr_shape; 0 means H */
} gdr_lin_shape;

typedef struct {                    /* device pointers; q, k, v may be NULL when B * T == 0 */
  const void *q, *k;                /* [B,T,Hk,D] dtype */
  const void *v;                    /* [B,T,H,D] dtype */
  const float *log_decay;           /* [H] */
  const float *h0;                  /* [N,H,D,D] or NULL (zero initial state) */
} gdr_lin_inputs;

typedef struct {                    /* device pointers, all overwritten; dq, dk, dv may be NULL when B * T == 0 */
  void *dq, *dk, *dv;               /* as q, k, v */
  float *dh0;                       /* [N,H,D,D] or NULL (not returned) */
} gdr_lin_grads;

/* Workspace of gdr_lin_fwd alone (backward 0), or of a gdr_lin_fwd that a
 * gdr_lin_bwd follows (backward 1; with Hk < H it includes dq or dk per value head
 * in fp32). */
gdr_status gdr_lin_workspace_bytes(const gdr_lin_shape* shape, int32_t backward, size_t* bytes);

/* Forward: o (required unless there are no tokens) and optionally the final states
 * ht [N,H,D,D] fp32 (a sequence without tokens returns its h0).  `ws` needs
 * gdr_lin_workspace_bytes(), 256-byte aligned, with any content; afterwards it
 * holds the states that gdr_lin_bwd on the same shape and inputs starts from.
 * Calls that overlap in time need a workspace each.  Outputs must not overlap
 * inputs.  Errors as gdr_fwd_recompute. */
gdr_status gdr_lin_fwd(const gdr_lin_shape* shape, const gdr_lin_inputs* in, void* ws, size_t ws_bytes, void* o,
                       float* ht, void* stream);

/* Backward, after gdr_lin_fwd on the same shape, inputs and workspace (which it
 * leaves fit for another gdr_lin_bwd).  dO as o, required unless there are no
 * tokens; dht [N,H,D,D] fp32 or NULL (zero).  Outputs must not overlap inputs. */
gdr_status gdr_lin_bwd(const gdr_lin_shape* shape, const gdr_lin_inputs* in, const void* dO, const float* dht,
                       void* ws, size_t ws_bytes, const gdr_lin_grads* grads, void* stream);

/* One token for each of N rows on a pool of states [P,H,D,D] fp32, updated in
 * place: shape dense with T == 1, in->h0 NULL; state, P, slots, padding rows and
 * rows that share a slot as in gdr_step.  o: [N,1,H,D] dtype. */
gdr_status gdr_lin_step(const gdr_lin_shape* shape, const gdr_lin_inputs* in, float* state, int32_t P,
                        const int32_t* slots, void* o, void* stream);

/* ------------------------------------------------------------------------
 * 8-bit projections: the product of e4m3 matrices with a scale for each 128
 * elements of the contraction, and the quantisation that makes such matrices
 * (gdr_norm_quant with group 128 makes them too).
 *
 * gdr_quant: y = x, or x^T with `transpose`, as bytes and scales.  y has R rows and
 * C columns ([rows,cols], or [cols,rows] transposed); a scale belongs to `block`
 * rows (1 or 128) and 128 columns of y, fewer at its end:
 *   scale = max(max|y| / 448, 2^-126),  q = e4m3(y / scale)
 * as in gdr_norm_quant, NaN and infinities included.  x: [rows,cols] dtype; q: [R,C]
 * bytes; scales: [ceil(R / block),ceil(C / 128)] fp32.  q and scales must not
 * overlap x.  GDR_EUNSUPPORTED from 2^31 rows or columns or 2^24 tiles of 128 x 128 on. */
typedef struct {
  int64_t rows, cols;               /* of x */
  int32_t dtype;                    /* gdr_dtype of x */
  int32_t block;                    /* rows of y per scale: 1 or 128 */
  int32_t transpose;                /* 0 or 1 */
} gdr_quant_shape;

gdr_status gdr_quant(const gdr_quant_shape* shape, const void* x, void* q, float* scales, void* stream);

/* c[m][n] = sum over groups g of 128 elements k of the contraction (the last may be
 * shorter) of a_scales[m][g] b_scales[n / block][g] sum_{k in g} a[m][k] b[n][k].
 * a: [M,K] e4m3 bytes with a_scales [M,G], G = ceil(K / 128); b: [N,K] bytes with
 * b_scales [ceil(N / block),G], block 1 or 128; c: [M,N] dtype.  With an fp32 c products
 * are exact and sums fp32.  With a bf16 c the matrix instructions take the bytes as
 * they are: within a group they sum the products of up to 8 neighbouring k with the bits
 * below 2^-13 of the largest of them dropped (2^-10 of the sum of their magnitudes at
 * most), the rest is fp32 and c is rounded once.  The two scales of a group are multiplied
 * first, in fp32: where their product is infinite c is infinite or NaN, whatever the sum,
 * and where it is subnormal (below 2^-126) or zero it has as few bits.  A linear layer
 * y = x w^T takes a = x and b = w (block 128); its backward takes the same product with
 * a = dy and b = w^T, and with a = dy^T and b = x^T (block 1), each quantised along the
 * contraction.  K >= 1; M and N may be zero.  ws: gdr_gemm_workspace_bytes() (zero
 * for most shapes; then ws may be NULL), 256-byte aligned, any content; calls that
 * overlap in time need one each.  c must not overlap the inputs.  Sums run in an
 * order that depends on the shape alone.  GDR_EUNSUPPORTED above 2^30 rows or columns
 * of a matrix and from 2^19 tiles of 128 x 128 of c on. */
typedef struct {
  int32_t M, N, K;
  int32_t dtype;                    /* gdr_dtype of c */
  int32_t block;                    /* rows of b per scale: 1 or 128 */
} gdr_gemm_shape;

gdr_status gdr_gemm_workspace_bytes(const gdr_gemm_shape* shape, size_t* bytes);
gdr_status gdr_gemm(const gdr_gemm_shape* shape, const void* a, const float* a_scales, const void* b,
                    const float* b_scales, void* ws, size_t ws_bytes, void* c, void* stream);

/* Thread-local text for the last non-OK status returned to this thread. */
const char* gdr_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* GDR_H_ */

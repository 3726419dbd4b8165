/*
 * gdn.h -- C ABI of libgdn.so: the Gated DeltaNet chunked forward pass on one
 * GB300 (sm_103a).
 *
 * Operator (MegaGDN-PTO walkthrough, section 1.1, the seven-stage chunk
 * pipeline; TileLang x xLLM page, Step 1, chunk_gated_delta_rule_fwd_h):
 *
 *   S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T     (S is [K][V])
 *   o_t = scale * S_t^T q_t
 *
 * evaluated chunk-wise (cumsum -> scaled_dot_kkt -> solve_tril -> wy_fast ->
 * chunk_h -> chunk_o).  Inputs with GQA: value head h reads q/k head
 * h / (Hv / Hqk) (MegaGDN-PTO walkthrough, section 5.2).  Packed variable-length
 * batches use cu_seqlens (section 5.3).
 *
 * Conventions shared by every entry point:
 *  - All tensor pointers are DEVICE pointers to contiguous row-major arrays,
 *    owned by the caller; the library allocates nothing.
 *  - q, k, v and o must be 16-byte aligned (they are read/written by TMA).
 *  - Every call is asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *    default stream).  Host-side argument checks run before any launch; a
 *    failed check returns an error and launches nothing.  Errors found on the
 *    device (malformed cu_seqlens, a bounded wait that timed out) are written
 *    to a status word inside the workspace; read it with
 *    gdn_get_device_status().
 *  - No exception or C++ type crosses this boundary.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GDN_OK = 0,
  GDN_ERR_INVALID_ARG = 1,   /* bad pointer, size, alignment or workspace too small */
  GDN_ERR_UNSUPPORTED = 2,   /* valid request that this build does not implement */
  GDN_ERR_CUDA = 3,          /* a CUDA runtime call failed (launch, attribute, ...) */
  GDN_ERR_DEVICE = 4,        /* the device reported an error through the status word */
  GDN_ERR_SCRATCH_LIMIT = 5  /* gdn_chunk_fwd_noalloc: problem larger than its static scratch */
} gdn_status;

typedef enum { GDN_F32 = 0, GDN_BF16 = 1 } gdn_dtype;

/* Device status word values (read by gdn_get_device_status). */
#define GDN_DEV_OK 0
#define GDN_DEV_BAD_CU_SEQLENS 1   /* cu[0] != 0, decreasing, or cu[N] != T */
#define GDN_DEV_WAIT_TIMEOUT 2     /* a bounded spin-wait inside a kernel gave up */

/* Execution path. */
typedef enum {
  GDN_PATH_AUTO = 0,    /* cp or fused when supported, else staged */
  GDN_PATH_STAGED = 1,  /* one kernel per stage, intermediates in the workspace */
  GDN_PATH_FUSED = 2,   /* single persistent tcgen05 kernel: two CTAs per SM for bf16 K = V = 128
                           (the throughput form), the one-CTA-per-SM kernel for bf16 K = V = 256 */
  GDN_PATH_CP = 3,      /* chunk-parallel: each sequence cut into segments run on separate SMs
                           (bf16, K = V = 128); AUTO takes it for sequences of >= 2048 tokens
                           when the (sequence, value head) chains number at most half the SMs */
  GDN_PATH_FUSED1 = 4   /* single tcgen05 kernel with one CTA per SM and the value dimension in
                           slices of 128 columns (bf16, K in {128, 256}, V in {128, 256}); AUTO
                           takes it for K = 256, and for K = V = 128 when the (sequence, value
                           head) chains number at most the SMs or a packed batch is small enough
                           (ceil(T / 64) + N chunks a value head, times Hv, at most 256 x SMs)
                           that its longest sequence bounds the step */
} gdn_path;

/*
 * Problem description.
 *   B, T      : fixed-length batch [B, T] (cu_seqlens == NULL, N = B), or the
 *               packed batch [1, T] of N sequences (cu_seqlens != NULL, B = 1,
 *               T = total tokens, may be 0).
 *   Hqk, Hv   : q/k heads and value heads; Hv % Hqk == 0.
 *   K, V      : key and value head dims, each in {64, 128, 256}.
 *   C         : chunk length, 64 or 128.
 *   dt        : dtype of q, k, v and o (fp32 or bf16); g, beta, h0, ht are fp32.
 */
typedef struct {
  int B, T, N, Hqk, Hv, K, V, C;
  gdn_dtype dt;
  int varlen;   /* 1 when cu_seqlens is given */
} gdn_problem;

/*
 * Bytes of workspace that gdn_chunk_fwd needs for `path` (AUTO resolves as in
 * gdn_chunk_fwd).  Returns 0 for an invalid problem.  The varlen bound assumes
 * at most ceil(T / C) + N chunks, so cu_seqlens need not be read on the host.
 * The fused path over equal-length sequences spreads the (sequence, head)
 * chains' chunks evenly over the CTAs the current device holds at once (two
 * per SM), cutting a chain in two where a share ends; its workspace then holds
 * one K x V fp32 hand-over state per CTA (about 20 MB on 152 SMs), so query
 * the size with the device that will run the call current.  On packed
 * sequences (2 to 16384 of them) the fused paths also keep a table of N int32
 * there: a launch before the pass ranks the sequences by length so that the
 * longest chains start first.
 */
size_t gdn_chunk_fwd_workspace_size(const gdn_problem* p, gdn_path path);

/*
 * The chunked forward pass.
 *   q, k    : [B, T, Hqk, K]  dtype p->dt
 *   v       : [B, T, Hv, V]   dtype p->dt
 *   g       : [B, T, Hv] fp32, log-decay (used as given; no activation)
 *   beta    : [B, T, Hv] fp32
 *   scale   : multiplies o only (never the state); callers usually pass K^-0.5
 *   h0      : [N, Hv, K, V] fp32 initial state, or NULL for zeros
 *   cu_seqlens : [N + 1] int32 device array of token offsets, or NULL
 *   o       : out [B, T, Hv, V] dtype p->dt (round-to-nearest-even for bf16)
 *   ht      : out [N, Hv, K, V] fp32 final state, or NULL to skip it
 *   workspace / workspace_bytes : device scratch of at least
 *             gdn_chunk_fwd_workspace_size(p, path) bytes, 256-byte aligned
 * Returns GDN_OK once everything is enqueued on `stream`.
 */
gdn_status gdn_chunk_fwd(const gdn_problem* p, gdn_path path,
                         const void* q, const void* k, const void* v,
                         const float* g, const float* beta, float scale,
                         const float* h0, const int32_t* cu_seqlens,
                         void* o, float* ht,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * Staged path with a stop point (the pages' staged mode and MEGA_STOP_AFTER_*
 * hooks, MegaGDN-PTO walkthrough, section 7.4).  Runs stages 0..stop_after:
 *   0 prepare (chunk tables), 1 cumsum, 2 scaled_dot_kkt, 3 solve_tril,
 *   4 wy_fast, 5 chunk_h, 6 chunk_o (6 = full forward; o/ht written only by
 *   stages 6 and 5 respectively).
 * Intermediates stay in the workspace at the offsets of gdn_staged_layout.
 */
gdn_status gdn_chunk_fwd_staged(const gdn_problem* p, int stop_after,
                                 const void* q, const void* k, const void* v,
                                 const float* g, const float* beta, float scale,
                                 const float* h0, const int32_t* cu_seqlens,
                                 void* o, float* ht,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * Byte offsets of the staged path's intermediates inside its workspace.
 * nc_max = B * ceil(T / C) (fixed length) or ceil(T / C) + N (varlen).
 *   tables : int32 seq_chunk0[N + 1] | chunk_seq[nc_max] | chunk_tok0[nc_max] |
 *            chunk_len[nc_max] | nc[1]   (chunk c of the packed token stream
 *            covers tokens chunk_tok0[c] .. + chunk_len[c] of sequence chunk_seq[c])
 *   status : int32 device status word
 *   gamma  : f32 [nc_max][Hv][C]      in-chunk cumsum of g
 *   A      : f32 [nc_max][Hv][C][C]   strictly lower, beta_i exp(g_i - g_j) k_i.k_j
 *   Tinv   : f32 [nc_max][Hv][C][C]   (I + A)^{-1}
 *   W, U   : f32 [nc_max][Hv][C][K] and [nc_max][Hv][C][V]
 *   S0     : f32 [nc_max][Hv][K][V]   state at each chunk's start
 *   Vn     : f32 [nc_max][Hv][C][V]   v_new = U - W S0
 * Rows past a chunk's length hold zeros, except Tinv, which holds the
 * identity there (the inverse of I + A with A zero-padded).
 */
typedef struct {
  size_t tables, status, gamma, A, Tinv, W, U, S0, Vn, total;
  int nc_max;
} gdn_staged_layout_t;

gdn_status gdn_staged_layout(const gdn_problem* p, gdn_staged_layout_t* out);

/*
 * Waits for `stream`, then reads the device status word that the last call
 * using `workspace` left (GDN_DEV_*) into *dev_status and clears it.
 * `path` must be the path that call ran with (it locates the status word).
 * Returns GDN_ERR_CUDA if the synchronisation or the copy fails.
 */
gdn_status gdn_get_device_status(const gdn_problem* p, gdn_path path, void* workspace,
                                 void* stream, int* dev_status);

/*
 * The forward pass on HOST tensors (no counterpart on the pages: the
 * streaming form of gdn_chunk_fwd for callers whose q, k, v, g, beta, h0 and
 * outputs live in host memory).  Same shapes and meaning as gdn_chunk_fwd,
 * but q, k, v, g, beta, h0, cu_seqlens, o and ht are HOST pointers; page-locked
 * memory (cudaHostAlloc) is needed for the copies to overlap the compute
 * (pageable memory is copied synchronously by the driver, still correctly).
 * The batch is cut into at most `nsplit` sub-batches of whole sequences (about
 * equal token counts); sub-batch i's inputs are copied to the device while
 * sub-batch i - 1 runs gdn_chunk_fwd(path) and sub-batch i - 2's o and ht are
 * copied back, on three streams that the library creates once per device and
 * orders after `stream`; `stream` resumes once every output is in host memory.
 * Calls from several host threads are enqueued one at a time.
 *   workspace : DEVICE memory of gdn_chunk_fwd_host_workspace_size(p,
 *               cu_seqlens, nsplit, path) bytes, 256-byte aligned: two sets
 *               of device buffers for the largest sub-batch and the inner
 *               forward's workspace.
 * Host-side checks: the ones of gdn_chunk_fwd and, for packed sequences,
 * cu_seqlens[0] == 0, cu_seqlens[N] == T and non-decreasing offsets
 * (GDN_ERR_INVALID_ARG otherwise, nothing enqueued).  Device-side errors of
 * any sub-batch (the first one kept) are read with
 * gdn_chunk_fwd_host_get_device_status.  The host buffers must stay valid and
 * unmodified until `stream` has passed the call.
 */
size_t gdn_chunk_fwd_host_workspace_size(const gdn_problem* p, const int32_t* cu_seqlens, int nsplit,
                                         gdn_path path);
gdn_status gdn_chunk_fwd_host(const gdn_problem* p, gdn_path path, int nsplit,
                              const void* q, const void* k, const void* v,
                              const float* g, const float* beta, float scale,
                              const float* h0, const int32_t* cu_seqlens,
                              void* o, float* ht,
                              void* workspace, size_t workspace_bytes, void* stream);
/* Waits for `stream`, reads and clears the status word of a
 * gdn_chunk_fwd_host workspace (GDN_DEV_*). */
gdn_status gdn_chunk_fwd_host_get_device_status(void* workspace, void* stream, int* dev_status);

/*
 * Self-test of the tensor-core operand layouts used by the fused kernel (no
 * counterpart on the pages; a test hook).  Computes D = A B (or -A B) with one
 * CTA through tcgen05.mma over 128-byte-swizzled shared-memory tiles.
 *   A : bf16 [128][Kd] row-major, B : bf16 [Kd][N] row-major, D : fp32 [128][N]
 *   variant bits: 1 = A staged MN-major (else K-major), 2 = B staged MN-major,
 *                 4 = N 128 (else 64), 8 = Kd 128 (else 64), 16 = negate A,
 *                 32 = stage A with a TMA tiled load (needs bit 1 clear,
 *                 A 16-byte aligned)
 *   workspace : >= 4 bytes of device memory for the status word
 */
gdn_status gdn_selftest_umma(int variant, const void* A, const void* B, float* D, void* workspace,
                             void* stream);

/*
 * Test hook of the fused paths' bounded waits (no counterpart on the pages).
 * Runs gdn_chunk_fwd(p, path, ...) (path GDN_PATH_FUSED or GDN_PATH_FUSED1)
 * on an equal-length batch whose chains the fused kernel deals out as windows
 * that hand a cut chain's state over from one CTA to another, except that
 * window `drop_window` never raises its hand-over flag and every window waits
 * at most `wait_ns` nanoseconds for the flag it needs.  The window that would
 * continue that chain (drop_window - 1 for GDN_PATH_FUSED; for
 * GDN_PATH_FUSED1, whose windows come in groups of G x V / 128, the window one
 * group below) therefore gives up: it records GDN_DEV_WAIT_TIMEOUT in the
 * workspace's status word (read it with gdn_get_device_status with the same
 * path) and stops, leaving the o rows and the final state of the chain it was
 * waiting for unwritten; every other window completes and the launch ends.
 * The failure is made on purpose in a wait that has a limit: nothing faults
 * and nothing hangs.
 *   Arguments as gdn_chunk_fwd (no cu_seqlens).  Returns GDN_ERR_UNSUPPORTED
 *   when the fused pass over p hands no chain over at the start of window
 *   drop_window (then nothing is launched).
 */
gdn_status gdn_selftest_handover_timeout(const gdn_problem* p, gdn_path path,
                                         const void* q, const void* k, const void* v,
                                         const float* g, const float* beta, float scale,
                                         const float* h0, void* o, float* ht,
                                         void* workspace, size_t workspace_bytes,
                                         int drop_window, long long wait_ns, void* stream);

/*
 * Forward pass for callers that cannot allocate device memory (no counterpart
 * on the pages).  Some callers cannot call cudaMalloc in their call path: an
 * op inside a host framework that owns every device buffer and passes the op
 * only its inputs and outputs, or a caller that cannot accept the implicit
 * device-wide synchronisation of cudaMalloc/cudaFree.  This entry point
 * allocates nothing and takes no workspace: it runs the forward pass with its
 * workspace in a file-scope device array of 32 MiB that every GPU which
 * loads libgdn.so holds until the process exits.  Path: AUTO's choice, with
 * GDN_PATH_FUSED in place of GDN_PATH_CP, when that path's workspace
 * (gdn_chunk_fwd_workspace_size) fits 32 MiB - 256 bytes (the array's first
 * 256 bytes hold the status word) -- the fused kernels need at most about 20
 * MB -- else GDN_PATH_STAGED when its workspace fits.
 *   Arguments as gdn_chunk_fwd (the caller still passes inputs and outputs).
 *   Returns GDN_ERR_SCRATCH_LIMIT, launching nothing, when neither fits (the
 *   staged path for problems no fused kernel takes, such as fp32 inputs).
 *   The first call on a device (and the first after a device reset replaced
 *   its context) looks up the array's device address with
 *   cudaGetSymbolAddress, with that device current; make that first call
 *   before any stream capture.
 *   All calls share the one array: calls whose executions overlap on the GPU
 *   (other streams, other host threads) race on it and must be serialised by
 *   the caller.
 *   Errors found on the device (malformed cu_seqlens) leave o and ht
 *   incomplete and are recorded in the array's status word, which
 *   gdn_chunk_fwd_noalloc_get_device_status reads: it waits for `stream`,
 *   then returns the status (GDN_DEV_*) of the last gdn_chunk_fwd_noalloc call
 *   on the current device in *dev_status and clears it.  It allocates
 *   nothing either.
 */
gdn_status gdn_chunk_fwd_noalloc(const gdn_problem* p,
                                 const void* q, const void* k, const void* v,
                                 const float* g, const float* beta, float scale,
                                 const float* h0, const int32_t* cu_seqlens,
                                 void* o, float* ht, void* stream);
gdn_status gdn_chunk_fwd_noalloc_get_device_status(void* stream, int* dev_status);

/*
 * Fused recurrent (decode) step with sigmoid gating (TileLang x xLLM page,
 * fused_sigmoid_gating_delta_rule: the decode-phase operator that fuses the
 * sigmoid activation, the gate computation from the decay rate A_log and the
 * delta-rule update of the fp32 state, with per-sequence state offsets).
 * For every token t of every sequence, value head h:
 *     g_t    = -exp(A_log[h]) * softplus(a_t + dt_bias[h])
 *     beta_t = sigmoid(b_t)
 *     S <- e^{g_t} (I - beta_t k_t k_t^T) S + beta_t k_t v_t^T,   o_t = scale * S^T q_t
 * Tokens of a sequence are processed in order (one token per sequence is the
 * decode case; several run the plain recurrence).
 *   p           : as for gdn_chunk_fwd (C is ignored; V a multiple of 64)
 *   q, k        : [B, T, Hqk, K];  v : [B, T, Hv, V];  o : out [B, T, Hv, V]  (dtype p->dt)
 *   a, b        : [B, T, Hv] fp32 gate and beta pre-activations
 *   A_log       : [Hv] fp32;  dt_bias : [Hv] fp32 or NULL (= 0)
 *   state       : [state_slots, Hv, K, V] fp32 pool, read and updated in place
 *   state_indices : [N] int32 slot of each sequence, or NULL (slot n); a
 *                 sequence whose slot is negative or >= state_slots gets zero
 *                 outputs and no state update
 *   cu_seqlens  : [N + 1] int32 or NULL, as for gdn_chunk_fwd; sequences whose
 *                 offsets fall outside [0, T] are skipped
 * No workspace; asynchronous on `stream`.
 */
gdn_status gdn_recurrent_fwd(const gdn_problem* p, const void* q, const void* k, const void* v,
                             const float* a, const float* b, const float* A_log, const float* dt_bias,
                             float scale, float* state, const int32_t* state_indices, int state_slots,
                             const int32_t* cu_seqlens, void* o, void* stream);

/*
 * Backward pass of gdn_chunk_fwd (the FlashQLA notes list a backward of the
 * chunk kernel among its variants, section 4.3): for upstream gradients
 * dout = dL/do and dht = dL/dht, the gradients of L with respect to q, k, v,
 * g, beta and h0, by reverse mode of the token recurrence
 *     G <- G + scale q_t dout_t^T;  dq_t = scale S_t dout_t
 *     u = S_{t-1}^T k_t, w = G^T k_t;  dv_t = beta_t w
 *     dg_t = e^{g_t} (<G, S_{t-1}> - beta_t w.u);  dbeta_t = -e^{g_t} w.u + w.v_t
 *     dk_t = -e^{g_t} beta_t (G u + S_{t-1} w) + beta_t G v_t
 *     G <- e^{g_t} (G - beta_t k_t w^T)
 * from G = dht down to dh0 = G (S_t the state after token t, S_0 = h0).
 * With K = V = 128 (and q, k, v, dout 16-byte aligned) the chunked form of
 * the same reverse mode runs (64-token chunks: batched products for
 * everything but the chunk-to-chunk state and adjoint recurrences, on the
 * tensor cores as tf32 in three terms, about 2^-19 of each product; about
 * 0.8 MB of workspace per (chunk, value head)): equal-length batches in
 * sequence groups within 16 GiB; packed sequences in one group sized for
 * ceil(T / 64) + N chunks a value head, with the chunk tables built on the
 * device from cu_seqlens (packed batches whose bound exceeds 32 GiB take the
 * token recurrence).  Other problems recompute the states in fp32 from
 * checkpoints at every 64th token.  Both keep fp32 accuracy.
 *   p, q, k, v, g, beta, scale, h0, cu_seqlens : as for gdn_chunk_fwd (K in
 *                 {64, 128}, V a multiple of 16; any C)
 *   dout        : [B, T, Hv, V], dtype p->dt;  dht : [N, Hv, K, V] fp32 or NULL (= 0)
 *   dq, dk      : out [B, T, Hqk, K] fp32 (summed over the value heads of each
 *                 q/k head);  dv : out [B, T, Hv, V] fp32
 *   dg, dbeta   : out [B, T, Hv] fp32;  dh0 : out [N, Hv, K, V] fp32 or NULL
 *   workspace   : gdn_chunk_bwd_workspace_size(p) bytes, 256-byte aligned
 *                 (the device status word and the per-chunk intermediates;
 *                 the size covers either form, since the choice also depends
 *                 on the alignment of q, k, v and dout)
 * dq and dk (and, for packed sequences or K = 64, dg and dbeta) are sums of
 * fp32 atomic additions across value heads or column slices (their rounding
 * may differ between runs).  Malformed cu_seqlens set the status word (read it
 * with gdn_chunk_bwd_get_device_status) and leave the gradients incomplete.
 * Asynchronous on `stream`.
 */
size_t gdn_chunk_bwd_workspace_size(const gdn_problem* p);
gdn_status gdn_chunk_bwd(const gdn_problem* p, const void* q, const void* k, const void* v,
                         const float* g, const float* beta, float scale, const float* h0,
                         const int32_t* cu_seqlens, const void* dout, const float* dht,
                         float* dq, float* dk, float* dv, float* dg, float* dbeta, float* dh0,
                         void* workspace, size_t workspace_bytes, void* stream);
/* Status word of a gdn_chunk_bwd workspace (synchronises `stream`, then
 * clears the word).  GDN_DEV_OK or GDN_DEV_BAD_CU_SEQLENS. */
gdn_status gdn_chunk_bwd_get_device_status(void* workspace, void* stream, int* dev_status);

/* Activation applied after the convolution of gdn_causal_conv1d_fwd. */
typedef enum { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1 } gdn_activation;

/*
 * Causal depthwise convolution with a carried state (TileLang x xLLM page,
 * causal_conv1d: each output token depends on the current and earlier inputs
 * of its own sequence only; the convolution state keeps the last W-1 inputs of
 * every sequence for incremental decode, in the state-pool slot that
 * cache_indices gives it).  For a sequence with inputs x_0..x_{L-1}, let
 * ext = [the W-1 initial inputs ; x_0 .. x_{L-1}]; then for every channel d
 *     y_p[d]    = act(bias[d] + sum_{w<W} weight[d*W + w] * ext_{p+w}[d])
 *     new state = ext_L .. ext_{L+W-2}
 * so weight[d*W + W-1] multiplies the current token.  act is the identity or
 * SiLU, u * sigmoid(u).  The initial inputs are the slot's state, or zeros
 * when the sequence has no slot or has_initial_state[n] == 0.
 *   x, y        : [B, T, D] of dtype dt, 16-byte aligned, D % 8 == 0; with
 *                 cu_seqlens, B == 1 and T is the packed total.  y must not
 *                 overlap x or conv_state.
 *   weight      : [D, W] fp32, 1 <= W <= 4;  bias : [D] fp32 or NULL (= 0)
 *   conv_state  : [state_slots, W-1, D] of dtype dt (16-byte aligned), or NULL
 *                 (zero initial inputs, nothing kept).  Read by the
 *                 convolution, then rewritten in place with the new state.
 *                 Ignored when W == 1.
 *   cache_indices : [N] int32 slot per sequence, or NULL (slot n; then
 *                 state_slots >= N).  A slot outside [0, state_slots) means
 *                 "no state": zero initial inputs, nothing written.  Distinct
 *                 sequences must use distinct slots.
 *   has_initial_state : [N] int32 or NULL (all 1); 0 starts the sequence from
 *                 zeros but still writes its slot.
 *   cu_seqlens  : [N + 1] int32 or NULL (then N == B and sequence n is row n
 *                 of x).  A sequence whose offsets fall outside [0, T] or
 *                 decrease is skipped (outputs and state); tokens that no
 *                 well-formed sequence covers are not written.
 * States are exact copies of inputs.  Two launches (convolution, then state
 * update), asynchronous on `stream`; no workspace.  Returns
 * GDN_ERR_INVALID_ARG for a failed host-side check (nothing launched).
 */
gdn_status gdn_causal_conv1d_fwd(const void* x, const float* weight, const float* bias, int W,
                                 void* conv_state, int state_slots, const int32_t* cache_indices,
                                 const int32_t* has_initial_state, const int32_t* cu_seqlens, int N,
                                 int B, int T, int D, gdn_dtype dt, gdn_activation act, void* y,
                                 void* stream);

/*
 * Backward of gdn_causal_conv1d_fwd, with the initial inputs given per sequence
 * (the forward call overwrites its state pool): for upstream gradients dout =
 * dL/dy and dfinal_state = dL/d(new state), the gradients of L with respect to
 * x, weight, bias and the initial inputs.
 *   x, dout, dx : [B, T, D] of dtype dt, 16-byte aligned, D % 8 == 0
 *   weight, bias, W, act, cu_seqlens, N, B, T : as for gdn_causal_conv1d_fwd
 *   initial_state : [N, W-1, D] of dtype dt or NULL (= 0);  dfinal_state : the
 *                 same shape or NULL (= 0).  16-byte aligned; ignored when W == 1.
 *   dweight     : out [D, W] fp32;  dbias : out [D] fp32 or NULL
 *   dinitial_state : out [N, W-1, D] of dtype dt or NULL
 *   workspace   : gdn_causal_conv1d_bwd_workspace_size(B, T, D, W) bytes (0:
 *                 invalid; query it with the device current that will run the
 *                 call), 256-byte aligned (partial sums of dweight and dbias)
 * A sequence with malformed offsets is skipped as in the forward (no gradient of
 * it is written or added).  Sums are added in a fixed order: results do not
 * depend on the run.  Asynchronous on `stream`.
 */
size_t gdn_causal_conv1d_bwd_workspace_size(int B, int T, int D, int W);
gdn_status gdn_causal_conv1d_bwd(const void* x, const float* weight, const float* bias, int W,
                                 const void* initial_state, const int32_t* cu_seqlens, int N, int B, int T, int D,
                                 gdn_dtype dt, gdn_activation act, const void* dout, const void* dfinal_state,
                                 void* dx, float* dweight, float* dbias, void* dinitial_state, void* workspace,
                                 size_t workspace_bytes, void* stream);

/*
 * A few rows times a matrix of 4-bit weights with group scales (the projections
 * of a decode step; any number of rows is computed, 32 of bf16 or 10 of fp32 a
 * pass over the weights):
 *     y[m][n] = sum_k x[m][k] (code[n][k] - zero[n][k / group]) scale[n][k / group] + bias[n]
 *   x           : [M, K] of dtype dt, rows ld_x elements apart (0: K)
 *   qweight     : [N, K / 2] bytes, 16-byte aligned; byte j of a row holds code 2j
 *                 in its low four bits and code 2j + 1 in its high four
 *   scales      : [N, K / group] of dtype sdt
 *   zeros       : [N, K / group] bytes, 0 .. 127, or NULL (8 everywhere)
 *   bias        : [N] fp32 or NULL
 *   K           : a multiple of group, at most 2^20;  group : a multiple of 32
 *   y           : out [M, N] of dtype dt, contiguous
 * No weight and, in fp32, no x is rounded; products with codes less zero points are
 * exact in fp32 and their sums, over a group and over the groups, round as fp32 sums do
 * (by about 2e-6 of sum |x w| at most for K = 8192).  y is rounded once to dt.  No
 * workspace; asynchronous on `stream`.
 */
gdn_status gdn_q4_matvec(const void* x, int64_t ld_x, const uint8_t* qweight, const void* scales, gdn_dtype sdt,
                         const uint8_t* zeros, const float* bias, int M, int N, int K, int group, gdn_dtype dt,
                         void* y, void* stream);

/*
 * Selective state space scan (a diagonal linear recurrence whose steps, input
 * and output maps depend on the token): the mixer that hybrid stacks put next
 * to the gated delta rule, behind the same short causal convolution.  For
 * channel d of group g = d / (D / G) and state n < S,
 *     dt_t   = softplus(delta_t[d] + dt_bias[d])      (without softplus: the sum itself)
 *     h_t[n] = e^{dt_t A[d][n]} h_{t-1}[n] + dt_t x_t[d] B_t[g][n]
 *     y_t[d] = (sum_n C_t[g][n] h_t[n] + Dskip[d] x_t[d]) * silu(z_t[d])
 * States, steps and sums are fp32; y is rounded once to p->dt.
 *
 * Problem description.
 *   B, T, N, varlen : as for gdn_problem (N = B for equal lengths)
 *   D, S, G  : channels (at most 65536), states a channel (at most 64) and
 *              groups of channels that share B and C; D % G == 0
 *   dt       : dtype of x, delta, z, B, C, y and of their gradients
 *   softplus : 0 or 1, as above
 *   ld_*     : elements from one token's row to the next (0: rows are
 *              contiguous), at least a row; a sequence's rows and the
 *              sequences of a batch follow one another at this stride, so a
 *              column slice of a wider matrix can be passed as it is.  ld_x,
 *              ld_delta, ld_z: rows of D elements; ld_b, ld_c: rows of G * S.
 * y, gradients and everything else are contiguous.  Outputs must not overlap
 * inputs or one another, but ht may be h0 and dh0 may be h0 or dht (the same
 * pointer: states updated in place).  Pointers need the alignment of their
 * elements only, except A, h0, ht, state, dA, dht and dh0: 16 bytes when
 * S % 4 == 0.
 */
typedef struct {
  int B, T, N, D, S, G;
  gdn_dtype dt;
  int varlen;
  int softplus;
  int64_t ld_x, ld_delta, ld_z, ld_b, ld_c;
} gdn_scan_problem;

/*
 * The scan over prompts or training sequences.
 *   x, delta    : [B, T, D];  A : [D, S] fp32;  Bm, Cm : [B, T, G, S]
 *   Dskip       : [D] fp32 or NULL (= 0);  z : [B, T, D] or NULL (no gate)
 *   dt_bias     : [D] fp32 or NULL (= 0)
 *   h0          : [N, D, S] fp32 or NULL (= 0);  cu_seqlens as for gdn_chunk_fwd
 *   y           : out [B, T, D];  ht : out [N, D, S] fp32 or NULL
 *   workspace   : gdn_selective_scan_fwd_workspace_size(p) bytes (0: invalid
 *                 problem), 256-byte aligned.  Sequences are cut into segments
 *                 that run side by side when the channels of all sequences do
 *                 not fill the device: query the size with the device current
 *                 that will run the call.
 * Malformed cu_seqlens set the status word (GDN_DEV_BAD_CU_SEQLENS, read with
 * gdn_selective_scan_get_device_status) and leave y and ht unwritten.
 * Asynchronous on `stream`; results do not depend on the run.
 */
size_t gdn_selective_scan_fwd_workspace_size(const gdn_scan_problem* p);
gdn_status gdn_selective_scan_fwd(const gdn_scan_problem* p, const void* x, const void* delta, const float* A,
                                  const void* Bm, const void* Cm, const float* Dskip, const void* z,
                                  const float* dt_bias, const float* h0, const int32_t* cu_seqlens, void* y,
                                  float* ht, void* workspace, size_t workspace_bytes, void* stream);
/*
 * The same, with the final states written to rows of a pool, as
 * gdn_selective_scan_step finds them: prompts of new sequences.
 *   state       : [state_slots, D, S] fp32 pool;  state_indices : [N] int32, row
 *                 of each sequence.  A sequence whose row is outside
 *                 [0, state_slots) keeps no state (its outputs are computed);
 *                 distinct sequences must use distinct rows.  The pool must not
 *                 overlap h0.  Malformed cu_seqlens leave it as it is.
 */
gdn_status gdn_selective_scan_fwd_pool(const gdn_scan_problem* p, const void* x, const void* delta, const float* A,
                                       const void* Bm, const void* Cm, const float* Dskip, const void* z,
                                       const float* dt_bias, const float* h0, const int32_t* cu_seqlens, void* y,
                                       float* state, const int32_t* state_indices, int state_slots, void* workspace,
                                       size_t workspace_bytes, void* stream);
/* Status word that the last scan call on `workspace` left (forward or
 * backward; synchronises `stream`, then clears the word).  Equal-length calls
 * write none: GDN_DEV_OK. */
gdn_status gdn_selective_scan_get_device_status(const gdn_scan_problem* p, void* workspace, void* stream,
                                                int* dev_status);

/*
 * Backward of gdn_selective_scan_fwd: for upstream gradients dout = dL/dy and
 * dht = dL/dht, the gradients of L with respect to every input, by the adjoint
 * recurrence q_t = C_t dout_t silu(z_t) + e^{dt_{t+1} A} q_{t+1}.
 *   inputs      : as for gdn_selective_scan_fwd (G at most 32768)
 *   dout        : [B, T, D] dtype p->dt, contiguous;  dht : [N, D, S] fp32 or NULL (= 0)
 *   dx, ddelta  : out [B, T, D] dtype p->dt;  dB, dC : out [B, T, G, S] dtype p->dt
 *                 (fp32 sums over the channels of a group, rounded once)
 *   dz          : out [B, T, D] dtype p->dt, required with z, else NULL
 *   dA          : out [D, S] fp32;  dD, ddt_bias : out [D] fp32 or NULL to skip them
 *                 (sums over all tokens of the batch; given whether or not
 *                 Dskip and dt_bias are)
 *   dh0         : out [N, D, S] fp32 or NULL
 *   workspace   : gdn_selective_scan_bwd_workspace_size(p) bytes, 256-byte
 *                 aligned (states before the tiles of tokens, and partial sums)
 * Sums are added in a fixed order (no atomics): results do not depend on the
 * run.  Malformed cu_seqlens set the status word and leave the gradients
 * unwritten.  Asynchronous on `stream`.
 */
size_t gdn_selective_scan_bwd_workspace_size(const gdn_scan_problem* p);
gdn_status gdn_selective_scan_bwd(const gdn_scan_problem* p, const void* x, const void* delta, const float* A,
                                  const void* Bm, const void* Cm, const float* Dskip, const void* z,
                                  const float* dt_bias, const float* h0, const int32_t* cu_seqlens,
                                  const void* dout, const float* dht, void* dx, void* ddelta, float* dA, void* dB,
                                  void* dC, float* dD, void* dz, float* ddt_bias, float* dh0, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * The scan on a pool of states, for single tokens (decode); several tokens of
 * a sequence run one after the other.
 *   state       : [state_slots, D, S] fp32 pool, read and updated in place
 *   state_indices : [N] int32 slot of each sequence, or NULL (slot n; then
 *                 state_slots >= N).  A sequence whose slot is outside
 *                 [0, state_slots) gets zero outputs and no state update;
 *                 distinct sequences must use distinct slots.
 *   cu_seqlens  : as for gdn_chunk_fwd; a sequence whose offsets fall outside
 *                 [0, T] or decrease is skipped
 *   other arguments as for gdn_selective_scan_fwd
 * One launch, no workspace; asynchronous on `stream`.
 */
gdn_status gdn_selective_scan_step(const gdn_scan_problem* p, const void* x, const void* delta, const float* A,
                                   const void* Bm, const void* Cm, const float* Dskip, const void* z,
                                   const float* dt_bias, float* state, const int32_t* state_indices,
                                   int state_slots, const int32_t* cu_seqlens, void* y, void* stream);

/*
 * Test hook (no counterpart on the pages): y[i] = e^{x[i]} computed the way
 * the fused kernel computes its decay factors (2^{x log2 e} on the MUFU ex2
 * unit), so tests can bound its error against CUDA's expf.  x, y device
 * arrays of n floats.
 */
gdn_status gdn_selftest_exp(const float* x, float* y, int n, void* stream);

/* Path that GDN_PATH_AUTO selects for this problem (STAGED, FUSED or CP). */
gdn_path gdn_resolve_path(const gdn_problem* p);

/* Human-readable name of a status code (static string). */
const char* gdn_status_string(gdn_status s);

/* Library version string, e.g. "gdn 0.1 sm_103a". */
const char* gdn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */

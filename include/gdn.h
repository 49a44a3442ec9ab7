/*
 * gdn.h -- C ABI of the MI355X (gfx950) chunked Gated DeltaNet prefill.
 *
 * The operation.  For every sequence i (tokens cu[i] .. cu[i+1]-1 of a packed
 * batch) and every value head h (reading key head h / (Hv/Hk)), starting from
 * the d_k x d_v state H = init_state[i, h] (or zeros):
 *
 *     q^ = q_t / sqrt(|q_t|^2 + eps),  k^ = k_t / sqrt(|k_t|^2 + eps)
 *     H  = exp(g_t) (I - beta_t k^ k^T) H + beta_t k^ v_t^T
 *     out[t, h] = scale * H^T q^
 *
 * and final_state[i, h] = H after the sequence's last token: the gated
 * delta rule, with the state stored as d_k x d_v.  The serving pages name
 * the operation as the chunked Gated DeltaNet prefill of their native
 * Qwen3.5 backend ("Cua-S1 4B 0.2 native text worker"; "Open-Jev-27B-v1.1
 * native text worker", section "Validation and optimization scope") and
 * test it against float64 references, as this library's tests do; they
 * print no formula, so the recurrence above is the definition this library
 * takes.
 *
 * The library evaluates it chunk by chunk (chunk C in {16, 32, 64}, default
 * 64) on the caller's HIP stream with three kernels: a chunk table, a fused
 * L2-norm / gate-prep / intra-chunk WY kernel, and a fused inter-chunk
 * state-scan / output kernel (two with GDN_SCAN_TWO_LEVEL).
 *
 * Conventions taken from the pages:
 *   - a versioned ABI that callers are rebuilt against ("Cua-S1 4B 0.2
 *     native text worker"; "Open-Jev-27B-v1.1 native text worker", section
 *     "Build and serve");
 *   - invalid or oversize inputs are rejected before any work starts
 *     (same page, section "Prepare the checkpoint");
 *   - vector memory paths only where width, stride and pointers permit
 *     (same page, section "Validation and optimization scope"); here
 *     layouts that do not permit them are rejected with GDN_ERR_LAYOUT.
 *
 * Error behaviour (all entry points): arguments are validated on the host
 * before any HIP call; a failed validation returns a negative status and
 * enqueues nothing.  No exception crosses the ABI.  gdn_last_error() gives a
 * message for the calling thread's last failure.  The contents of
 * cu_seqlens are a precondition (cu[0] = 0, non-decreasing, cu[N] <= T);
 * by default the library does not read device memory on the host, so it
 * does not check them, but the kernels clamp them so that a bad table
 * cannot make them access memory outside the tensors.  gdn_check_cu_seqlens
 * checks a host copy.  With the environment variable GDN_DEBUG_CHECK=1, a
 * packed prefill first checks the device table in a one-workgroup kernel,
 * waits for it (a stream synchronisation) and, if the table is malformed,
 * returns GDN_ERR_INPUT with nothing else enqueued (the pages reject bad
 * input before any work starts: "Open-Jev-27B-v1.1 native text worker",
 * section "Prepare the checkpoint").  The check is skipped while the stream
 * is being captured into a graph (a capture cannot wait).  Faults of
 * enqueued work surface at the caller's next synchronisation of the
 * stream.  Apart from GDN_DEBUG_CHECK, no call synchronises the device.
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ABI_VERSION 11

/* Status codes. */
#define GDN_OK 0
#define GDN_ERR_NULL_ARG (-1)    /* a required tensor or pointer is NULL      */
#define GDN_ERR_DTYPE (-2)       /* unsupported or mismatched element types   */
#define GDN_ERR_SHAPE (-3)       /* inconsistent or out-of-range sizes        */
#define GDN_ERR_LAYOUT (-4)      /* strides / alignment the kernels cannot use */
#define GDN_ERR_UNSUPPORTED (-5) /* valid but not built: head size, chunk ... */
#define GDN_ERR_WORKSPACE (-6)   /* workspace missing, too small or misaligned */
#define GDN_ERR_HIP (-7)         /* a HIP call or kernel launch failed        */
#define GDN_ERR_INPUT (-8)       /* malformed input values (cu_seqlens)       */

/* Element types. */
#define GDN_DTYPE_BF16 1
#define GDN_DTYPE_F32 2
#define GDN_DTYPE_I32 3
#define GDN_DTYPE_I64 4
/* 8-bit float, 4 exponent and 3 mantissa bits, no infinities, largest value
 * 448: an output type of gdn_add_rms_norm only.                            */
#define GDN_E4M3 5

/* A strided view of caller-owned memory (device memory for every tensor
 * argument).  shape/stride have ndim valid entries, outermost first; strides
 * are in elements.  The library never frees, retains or reallocates it. */
typedef struct gdn_tensor {
  void* data;
  int32_t dtype;
  int32_t ndim;
  int64_t shape[4];
  int64_t stride[4];
} gdn_tensor;

/* Stage mask bits for gdn_options.stages.  A full call runs all of them; a
 * caller-owned workspace keeps the intermediates between partial calls so a
 * caller may run (and time) the stages one at a time, in order. */
#define GDN_STAGE_TABLE 1u /* chunk table from cu_seqlens                   */
#define GDN_STAGE_WY 2u    /* L2 norms, gate cumsum, (I+A)^-1, W, U~, Q', O_loc */
#define GDN_STAGE_SCAN 4u  /* sequential state scan fused with the output   */
#define GDN_STAGE_ALL 7u

typedef struct gdn_options {
  int32_t chunk;      /* 16, 32 or 64 (default 64)                          */
  float scale;        /* output multiplier (default 1.0)                     */
  float l2_eps;       /* epsilon inside the L2 norm's square root (1e-6)     */
  uint32_t stages;    /* GDN_STAGE_* mask (default GDN_STAGE_ALL)            */
  int32_t scan_split; /* GDN_SCAN_* (default GDN_SCAN_AUTO)                  */
  uint32_t flags;     /* GDN_FLAG_* (default 0)                              */
  /* GDN_FLAG_DECAY_PROJ: per value head f32 [Hv] device arrays A and bias
   * (NULL reads as zeros; default NULL)                                     */
  const float* decay_a_log;
  const float* decay_bias;
  /* GDN_FLAG_OUTPUT_GATE: the gate projection z, device memory laid out
   * exactly as `out` (same shape, dtype and strides); the weight, f32 [dv]
   * device array (NULL reads as ones); the epsilon inside the root (1e-6) */
  const void* gate_z;
  const float* norm_weight;
  float norm_eps;
  /* Segments (uniform sequences, all stages, one-pass scan; ignored
   * otherwise): the sequences run as consecutive segments of whole chunks,
   * each the WY transform and then the scan from the previous segment's
   * state (carried in f32 in the workspace), so that a segment's
   * intermediates stay in the GPU's 256 MiB memory-side cache between the
   * two launches.  The results are bit-identical to one pass.  0 (default):
   * automatic, when the intermediates of the whole call (W, Q', U~ and
   * O_loc over all sequences and value heads) exceed 128 MiB: segments
   * within 128 MiB each, at least 8 chunks long, the longest whose WY work
   * items (sequences x key heads x chunks) fill whole rounds of the 512
   * WY workgroups an MI355X holds at once, else the fewest of equal
   * length; -1: never; n > 0: segments of n chunks.                      */
  int32_t segment_chunks;
  /* GDN_FLAG_QKV_CONV: the short convolution's taps, an f32 device array
   * [D][conv_width] (channel-major, the last tap multiplies the current
   * token) over D = 2 Hk dk + Hv dv channels in the order q | k | v, each
   * part in its tensor's [H][d] order, 16-byte aligned; its width, 1 .. 4
   * (default 4); the raw rows before each sequence, a contiguous device
   * array [N][conv_width - 1][D] of the input dtype, 16-byte aligned, or
   * NULL for zeros (fresh sequences); and where the last conv_width - 1 raw
   * rows of each sequence go, the same layout, or NULL (not written).
   * conv_state_out may be conv_state_in.  Sizes are not checked: the arrays
   * must hold what these shapes name.                                     */
  const float* conv_weight;
  int32_t conv_width;
  const void* conv_state_in;
  void* conv_state_out;
} gdn_options;

/*
 * GDN_FLAG_BETA_LOGITS: `beta` holds the write gate's raw projection b, and
 * the kernels use beta = sigmoid(b) = 1 / (1 + e^-b), computed in fp32 as the
 * gate is loaded (beta in (0, 1) is a sigmoid of a projection), so
 * no separate activation pass over [T, Hv] runs before the prefill or the
 * decode step.  b = +-inf give beta = 1 / 0.
 */
#define GDN_FLAG_BETA_LOGITS 1u

/*
 * The gates on either side of the prefill.  The serving pages run "fused
 * norm, activation" operations around the chunked Gated DeltaNet and keep
 * the bf16 rounding points of the unfused sequence when they fuse a gate
 * into an epilogue ("Open-Jev-27B-v1.1 native text worker", section
 * "Validation and optimization scope"); they print no formula for either,
 * so the two below are this library's reading.
 *
 * GDN_FLAG_DECAY_PROJ: `g` holds the decay gate's raw projection a, and the
 * kernels take
 *     g = -exp(A[h]) * softplus(a + bias[h]),   softplus(x) = log(1 + e^x)
 * in fp32 as they load it (A = decay_a_log, bias = decay_bias, per value
 * head), so every g is <= 0 for any a and no activation pass over [T, Hv]
 * runs first.  (A = bias = 0 with -a in place of a gives log sigmoid(a).)
 *
 * GDN_FLAG_OUTPUT_GATE: after the outputs are stored (rounded to the output
 * type, as an unfused norm would read them), each (token, value head) row o
 * of d_v outputs is replaced, in one pass, by
 *     y = o / sqrt(mean(o^2) + norm_eps) * w * silu(z),  silu(z) = z / (1 + e^-z)
 * computed in fp32 from the stored o and rounded once.  The norm spans the
 * whole row, which the state scan writes in 16-column slices from separate
 * workgroups, so it runs as its own bandwidth-bound kernel at the end of the
 * call (the same kernel as gdn_output_gate).  z is read with out's strides.
 */
#define GDN_FLAG_DECAY_PROJ 2u
#define GDN_FLAG_OUTPUT_GATE 4u

/*
 * GDN_FLAG_QKV_SILU: q, k and v hold the values before the activation that
 * precedes the layer, and the kernels (prefill and decode) take
 *     silu(x) = x / (1 + e^-x)
 * elementwise in fp32 as they load them, each result rounded to the input
 * dtype as a separate activation pass would store it (so the L2 norms of q
 * and k are taken of the activated rows).  The same reading as the gates
 * above: the pages run "fused norm, activation" operations around the
 * chunked Gated DeltaNet and name SiLU as the activation they check
 * ("Open-Jev-27B-v1.1 native text worker", section "Validation and
 * optimization scope").  Alone it applies no convolution (see
 * GDN_FLAG_QKV_CONV).  In the prefill the WY kernel writes the activated key rows to the workspace
 * (the `k_act` region, laid out as a contiguous [T][Hk][dk] tensor of the
 * input dtype) for the scan.
 */
#define GDN_FLAG_QKV_SILU 8u

/*
 * GDN_FLAG_QKV_CONV: before the activation, every channel c of q, k and v
 * passes through a causal depthwise convolution of width W = conv_width
 * along the tokens of its own sequence:
 *     y[t, c] = sum_{j=0}^{W-1} conv_weight[c][j] * e[t + j, c],
 * e being the sequence's W - 1 history rows (conv_state_in, or zeros)
 * followed by its raw rows.  y then goes through silu when
 * GDN_FLAG_QKV_SILU is also set, and is rounded once to the input dtype;
 * the L2 norms of q and k are taken of the result.  Computed in fp32 as the
 * rows are loaded: the WY kernel reads W - 1 rows before each chunk (from
 * the inputs, or from conv_state_in at a sequence's first chunk) and writes
 * the chunk's key rows as used to the `k_act` workspace region for the
 * scan.  With conv_state_out the last W - 1 raw rows of each sequence (the
 * history a later call continues from; fewer rows than that shift in the
 * tail of conv_state_in) are written after the WY stage.  The decode step
 * does the same per token and shifts its row into conv_state_out.
 * Reading: the pages name "fused norm, activation" operations around the
 * chunked Gated DeltaNet ("Open-Jev-27B-v1.1 native text worker", section
 * "Validation and optimization scope") and name no convolution; this is the
 * short convolution a Gated DeltaNet layer runs on its q, k, v projections
 * before the SiLU, for callers that fuse it here.
 */
#define GDN_FLAG_QKV_CONV 16u

/*
 * The state scan's schedule.  Each chunk maps its incoming state affinely
 * (the recurrence above summed over a chunk): H' = M H + B with
 * M = e^{gamma_last} I - K~^T W and B = K~^T U~.
 * GDN_SCAN_TWO_LEVEL splits every sequence (at about 17/32 of its chunks) and scans
 * both halves at once: the second from zero, beside the product of its M
 * (d_k more state columns), then adds M-product x (state at the split) to
 * its outputs and final state.  The chain of dependent chunk steps shortens
 * to about 17/32 of the chunks; the arithmetic differs from the one-pass scan only
 * in rounding.  Offered
 * for bf16 inputs without cu_seqlens (uniform sequences), d_k and d_v
 * multiples of 32 and chunks of 32 or 64; GDN_SCAN_TWO_LEVEL elsewhere is
 * GDN_ERR_UNSUPPORTED.  GDN_SCAN_AUTO is the one-pass scan (on MI355X the
 * two-level scan's two launches take longer at the sizes measured).
 */
#define GDN_SCAN_AUTO 0
#define GDN_SCAN_ONE_PASS 1
#define GDN_SCAN_TWO_LEVEL 2

/* Returns GDN_ABI_VERSION of the built library. */
int gdn_abi_version(void);

/* Fills *opts with the defaults listed in gdn_options. */
void gdn_default_options(gdn_options* opts);

/*
 * gdn_prefill -- the whole prefill on `stream` (a hipStream_t; NULL = the
 * null stream), with default options and a workspace the library allocates
 * and frees stream-ordered (hipMallocAsync / hipFreeAsync on `stream`).
 *
 *   q, k        [T, Hk, dk] or [B, T/B, Hk, dk]; bf16 or f32
 *   v, out      [T, Hv, dv] (or 4-D like q); same dtype as q
 *   g, beta     [T, Hv] (or [B, T/B, Hv]) f32: g is the log-decay (<= 0,
 *               alpha = exp(g)), beta the write strength in [0, 1] (already
 *               passed through the sigmoid).  These ranges are
 *               preconditions, not checked (see GDN_FLAG_DECAY_PROJ and
 *               GDN_FLAG_BETA_LOGITS for raw projections).
 *   cu_seqlens  int32 or int64 [N+1] device array of sequence starts
 *               (entries below 2^31), or NULL: one
 *               sequence of T tokens (3-D inputs) or B sequences of T/B
 *               tokens each (4-D inputs).  With cu_seqlens, 4-D inputs need
 *               B == 1, and the bounds are read from it also for N = 1:
 *               rows at or after cu[N] are not written.
 *   init_state  f32 [N, Hv, dk, dv] contiguous, or NULL for zeros
 *   final_state f32 [N, Hv, dk, dv] contiguous, or NULL (not written); it
 *               may be the same memory as init_state.
 * Sizes: dk, dv in {16, 32, 64, 128}; Hv a multiple of Hk; N, T < 2^31.
 * Layout: unit stride in the last dimension; other strides multiples of 8
 * elements (bf16) or 4 (f32); 16-byte aligned data pointers; for 4-D
 * tensors stride[0] == shape[1] * stride[1].  Otherwise GDN_ERR_LAYOUT.
 * All tensors are caller-owned device memory that must stay valid until
 * the stream reaches the end of the enqueued work.  Returns a GDN_* status.
 */
int gdn_prefill(const gdn_tensor* q, const gdn_tensor* k, const gdn_tensor* v,
                const gdn_tensor* g, const gdn_tensor* beta,
                const gdn_tensor* cu_seqlens, const gdn_tensor* init_state,
                gdn_tensor* out, gdn_tensor* final_state, void* stream);

/*
 * gdn_prefill_ex -- as gdn_prefill, with options (NULL = defaults) and a
 * caller-owned device workspace of at least gdn_workspace_size() bytes,
 * 256-byte aligned.  It allocates nothing.  The workspace must not be used
 * by another call that overlaps on the device.
 */
int gdn_prefill_ex(const gdn_tensor* q, const gdn_tensor* k,
                   const gdn_tensor* v, const gdn_tensor* g,
                   const gdn_tensor* beta, const gdn_tensor* cu_seqlens,
                   const gdn_tensor* init_state, gdn_tensor* out,
                   gdn_tensor* final_state, const gdn_options* opts,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * gdn_prefill_noalloc -- gdn_prefill_ex without a workspace argument and
 * without any allocation, for callers that cannot allocate device memory:
 * code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  Its workspace is a static device array of
 * GDN_NOALLOC_SCRATCH_BYTES held by the library on every GPU it runs on
 * until the process ends (looked up on the first call on each device).  The
 * caller still passes every input and output; `opts` may be NULL.  Sizes
 * whose workspace (gdn_workspace_size) exceeds the scratch are rejected with
 * GDN_ERR_WORKSPACE before anything is enqueued (96 MiB covers, e.g., 4096
 * tokens x 16 heads at d = 128 in bf16, which needs 64 MiB).  No part of the
 * scratch has to start at zero: each call writes everything it reads.  All
 * calls on one GPU share its scratch, which keeps the last call's contents:
 * calls that overlap on one GPU (different streams or threads) race, and
 * must be serialised by the caller.
 */
#define GDN_NOALLOC_SCRATCH_BYTES ((size_t)96 << 20)
int gdn_prefill_noalloc(const gdn_tensor* q, const gdn_tensor* k,
                        const gdn_tensor* v, const gdn_tensor* g,
                        const gdn_tensor* beta, const gdn_tensor* cu_seqlens,
                        const gdn_tensor* init_state, gdn_tensor* out,
                        gdn_tensor* final_state, const gdn_options* opts,
                        void* stream);

/* Byte offsets of the intermediates inside the workspace (for inspection and
 * tests).  Per (chunk c, value head h) block, all in the input dtype:
 *   w     diag(s) W,  W = T diag(beta e^gamma) K^     C x dk, k-tile order
 *   qp    Q' = scale diag(e^gamma) Q^ - P W             C x dk, k-tile order
 *   ut    diag(s) U~, U~ = T diag(beta) V              C x dv, accumulator tiles
 *   oloc  O_loc = P U~                                  C x dv, transposed tiles
 * with the row scale s_r = e^(gamma_last - gamma_r) / sqrt(|k_r|^2 + eps)
 * (k_r the key row as passed), and f32 decay[c][h] = e^(gamma_last).  With
 * U' = diag(s) U~ - diag(s) W H the state update is H' = e^(gamma_last) H +
 * K^T U' with K the chunk's key rows as passed, equal to K~^T U for
 * K~_r = e^(gamma_last - gamma_r) k^_r.  A block starts at
 * offset + (c * Hv + h) * (its element count) * element_size.
 * "k-tile order": 16-row tiles one after another; inside a tile, for the
 * 16-wide k-tile t of the second index, lane l = m + 16 ((k % 16) / 4)
 * holds the 4 elements k % 4 = 0..3.  bf16 pairs k-tiles 2u and 2u+1 into
 * one unit of 8 elements per lane (4 of k-tile 2u, then 4 of 2u+1; a
 * trailing single k-tile has 4); f32 has one k-tile (4 elements) per unit.
 * Units follow each other, lanes in order inside a unit.
 * "Accumulator tiles": 16 x 16 tiles, column-tile major (tile (ct, rt) at
 * ct * C/16 + rt), of 64 lanes x 4, lane l holding rows 4 (l / 16) .. +3 of
 * column l % 16; "transposed tiles" hold the same tiles with lane l holding
 * columns 4 (l / 16) .. +3 of row l % 16.  Rows past the end of a short
 * chunk are zero.  chunk_table is int32 [max_chunks][4] = (sequence, first
 * token, length, 0) in packed mode. */
typedef struct gdn_workspace_layout {
  size_t total_bytes;
  int64_t max_chunks;
  size_t chunk_table, chunk_offsets, seq_starts, decay, w, qp, ut, oloc;
  /* two-level scan (split_chunks > 0: chunks in the first segment), else 0:
   *   split_y      bf16 [chunk][Hv][C][dk]  Q' x M-product, second segment
   *   split_hmid   f32 [N][Hv][dk][dv]      state at the split
   *   split_hmid_t bf16 [N][Hv][dv][dk]     its transpose
   *   split_psi    f32 [N][Hv][dk][dv]      second segment's end from zero
   *   split_phi    f32 [N][Hv][dk][dk]      second segment's M-product   */
  int32_t split_chunks;
  size_t split_y, split_hmid, split_hmid_t, split_psi, split_phi;
  /* segments (gdn_options.segment_chunks): chunks per segment, 0 for one
   * pass, and the state carried between segments, f32 [N][Hv][dk][dv]    */
  int32_t segment_chunks;
  size_t segment_state;
  /* GDN_FLAG_QKV_SILU or GDN_FLAG_QKV_CONV: the key rows as the
   * recurrence uses them (activated, convolved), a contiguous [T][Hk][dk]
   * tensor of the input dtype (0 without either flag)                    */
  size_t k_act;
} gdn_workspace_layout;

/* Computes the workspace size / layout for the given tensors and options
 * (host only; data pointers are not read). */
int gdn_workspace_size(const gdn_tensor* q, const gdn_tensor* k,
                       const gdn_tensor* v, const gdn_tensor* cu_seqlens,
                       const gdn_options* opts, size_t* bytes);
int gdn_get_workspace_layout(const gdn_tensor* q, const gdn_tensor* k,
                             const gdn_tensor* v, const gdn_tensor* cu_seqlens,
                             const gdn_options* opts,
                             gdn_workspace_layout* layout);

/*
 * gdn_decode -- one recurrent step per sequence: the single-token form of
 * the same gated delta rule, as a
 * generator runs it after the prefill, on the state the prefill returned.
 * For every sequence i and value head h (key head h / (Hv/Hk)):
 *     H = state[i, h];  H <- exp(g) (I - beta k^ k^T) H + beta k^ v^T;
 *     out[i, h] = scale * H^T q^;  state[i, h] = H (in place)
 * with q^, k^ L2-normalised as in gdn_prefill.  Computed in fp32.
 *   q, k     [N, Hk, dk]; v, out [N, Hv, dv]; one dtype, bf16 or f32; unit
 *            stride in the last dimension
 *   g, beta  [N, Hv] f32 (same preconditions as gdn_prefill)
 *   state    f32 [N, Hv, dk, dv] contiguous and 16-byte aligned, read and
 *            written in place; v and out rows start on 4-element
 *            boundaries (address and strides)
 *   opts     NULL or options; scale, l2_eps, flags and the gate fields are
 *            used (with GDN_FLAG_OUTPUT_GATE, gate_z is laid out as out;
 *            with GDN_FLAG_QKV_CONV the convolution fields, N sequences of
 *            one token each: the history is read from conv_state_in and
 *            the step's raw row shifted into conv_state_out, which may be
 *            conv_state_in)
 * dk, dv in {16, 32, 64, 128}.  N = 0 enqueues nothing.  Allocates nothing.
 * Returns a GDN_* status; validation errors enqueue nothing.
 */
int gdn_decode(const gdn_tensor* q, const gdn_tensor* k, const gdn_tensor* v,
               const gdn_tensor* g, const gdn_tensor* beta, gdn_tensor* state,
               gdn_tensor* out, const gdn_options* opts, void* stream);

/*
 * Captured replays.  gdn_prefill_graph behaves as gdn_prefill_ex, but keeps
 * a HIP graph of the launches in `cache`.  A graph is found by every
 * argument the launches depend on: device, tensor descriptors (which
 * optional tensors and options pointers are NULL, dtypes, shapes, strides),
 * option values and workspace size (the shape key), and the data, options
 * and workspace pointers (the pointer key).  A hit (both keys stored) only
 * launches the stored graph, which removes the per-kernel launch cost.
 * Otherwise the launches are recorded on a private stream (stream capture):
 * while fewer than 4 graphs of the same shape key are stored, the recording
 * is instantiated as a new graph (a miss); from then on the least recently
 * used graph of that shape key is updated in place to the new pointers
 * (hipGraphExecUpdate: an update, no instantiation; launches of it already
 * enqueued keep their arguments), or replaced by a new instantiation if the
 * update is refused.  If capture or instantiation fails the call runs the
 * launches eagerly (and counts a fallback).  The sequence lengths are read from cu_seqlens on the device by
 * the kernels themselves, so one capture stays valid for any lengths with
 * the same shapes and buffers (the serving pages key their captures by the
 * length tuple: "Cua-S1 4B 0.2 native text worker"; "Open-Jev-27B-v1.1
 * native text worker", section "Build and serve").  The cache holds at most
 * `capacity` graphs and drops the least recently used.  Buffers named by a
 * stored graph must stay allocated while it may be replayed: call
 * gdn_graph_cache_clear after freeing or growing any of them.  A cache may be
 * shared by threads (calls are serialised); entries of one cache must not be
 * replayed on overlapping streams with the same workspace.
 */
typedef struct gdn_graph_cache gdn_graph_cache;

int gdn_graph_cache_create(int capacity, gdn_graph_cache** cache);
void gdn_graph_cache_destroy(gdn_graph_cache* cache);
void gdn_graph_cache_clear(gdn_graph_cache* cache);
int gdn_graph_cache_stats(gdn_graph_cache* cache, int* entries, int64_t* hits,
                          int64_t* misses, int64_t* updates, int64_t* fallbacks);
int gdn_prefill_graph(gdn_graph_cache* cache, const gdn_tensor* q,
                      const gdn_tensor* k, const gdn_tensor* v,
                      const gdn_tensor* g, const gdn_tensor* beta,
                      const gdn_tensor* cu_seqlens, const gdn_tensor* init_state,
                      gdn_tensor* out, gdn_tensor* final_state,
                      const gdn_options* opts, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * gdn_output_gate -- the gated output norm of GDN_FLAG_OUTPUT_GATE on its
 * own, for outputs already in memory:
 *     out[r] = x[r] / sqrt(mean(x[r]^2) + eps) * w * silu(z[r])
 * for every row r of d_v elements, computed in fp32, rounded once.
 *   x, z, out  [R, dv] or [T, H, dv]; one dtype, bf16 or f32; unit stride
 *              in the last dimension; other strides multiples of 8 (bf16)
 *              or 4 (f32) elements; 16-byte aligned data.  out may be x
 *              (in place).
 *   weight     f32 [dv] device array (4-byte aligned), or NULL for ones
 *   eps        >= 0
 * dv in {16, 32, 64, 128}.  No rows enqueues nothing.  Allocates nothing.
 * The reading and its citation are at GDN_FLAG_OUTPUT_GATE.  Returns a
 * GDN_* status; validation errors enqueue nothing.
 */
int gdn_output_gate(const gdn_tensor* x, const gdn_tensor* z, const float* weight,
                    float eps, gdn_tensor* out, void* stream);

/*
 * gdn_check_cu_seqlens -- checks a host copy of a cu_seqlens table of
 * n_seq + 1 entries for t_total tokens against the preconditions above
 * (cu[0] = 0, non-decreasing, cu[n_seq] <= t_total) with the predicate the
 * GDN_DEBUG_CHECK device check uses.  cu_host is host memory.  Returns
 * GDN_OK, GDN_ERR_INPUT (the message names the first bad entry), or
 * GDN_ERR_NULL_ARG / GDN_ERR_SHAPE for a NULL table or n_seq < 1.
 */
int gdn_check_cu_seqlens(const int32_t* cu_host, int64_t n_seq, int64_t t_total);

/* ------------------------------------------------------------------------
 * The operators around a recurrent layer's projections.  They share the
 * conventions above: tensors as descriptors, packed batches by cu_seqlens
 * (int32 or int64, clamped on the device, checked with GDN_DEBUG_CHECK=1),
 * validation on the host before any HIP call, work enqueued on the caller's
 * stream, nothing allocated, no synchronisation.  An output may share memory
 * with an input only where its description says so; other overlaps are
 * GDN_ERR_LAYOUT, and so are output rows that overlap each other (a token or
 * head stride of zero).  All sums, norms and states are fp32, and each output
 * is rounded once.  Tokens, sequences and channels: at most 2^31 - 2^21.
 * A dimension of one may have any stride >= 0: it is never taken.
 */

/*
 * gdn_short_conv -- the causal depthwise convolution along the tokens of
 * each sequence that a recurrent layer runs on its projections (the one
 * GDN_FLAG_QKV_CONV fuses into the delta-rule prefill), on its own and over
 * any channels:
 *     y[t, c] = bias[c] + sum_{j=0}^{W-1} weight[c][j] * e[t + j, c],
 * e being the sequence's W - 1 history rows (state_in, or zeros) followed by
 * its rows; then silu(y) = y / (1 + e^-y) with GDN_CONV_SILU.
 *   x, out     [T, D] (one sequence, or packed by cu_seqlens) or [B, L, D]
 *              (B sequences of L tokens; L = 1 is one step for each of B
 *              running sequences); bf16 or f32; unit stride in the last
 *              dimension, token stride any; [B, L, D] with stride[0] ==
 *              L * stride[1].  16-byte vector accesses are used where D,
 *              the strides and the addresses allow, else element accesses.
 *   weight     f32 [D][W] contiguous device array, W = 1 .. 4, the last tap
 *              on the current token; bias f32 [D] or NULL
 *   cu_seqlens [N + 1] device array or NULL, as gdn_prefill; rows at or
 *              after cu[N] are not written
 *   state_in   [N, W - 1, D] of x's dtype, contiguous, or NULL for zeros
 *   state_out  the last W - 1 rows of e for each sequence, the same layout,
 *              or NULL (not written); it may be state_in
 * Returns a GDN_* status; validation errors enqueue nothing.
 */
#define GDN_CONV_SILU 1u
int gdn_short_conv(const gdn_tensor* x, const gdn_tensor* weight, const float* bias,
                   const gdn_tensor* cu_seqlens, const gdn_tensor* state_in,
                   gdn_tensor* state_out, gdn_tensor* out, uint32_t flags, void* stream);

/*
 * The selective state space scan.  For every sequence i and head h (reading
 * group h / (H/G) of b and c), from the N x P state S = init_state[i, h] (or
 * zeros):
 *     d_t = softplus(dt[t, h] + dt_bias[h])      (GDN_SSM_SOFTPLUS; else
 *                                                 d_t = dt[t, h] + dt_bias[h])
 *     S   = exp(-exp(a_log[h]) d_t) S + d_t b_t x_t^T
 *     out[t, h] = S^T c_t + d_skip[h] x_t
 * and final_state[i, h] = S after the last token.  The state is laid out as
 * the delta rule's (d_k x d_v, here N x P), so both mixers' states can share
 * one pool.  d_t >= 0 is a precondition without GDN_SSM_SOFTPLUS.  Inputs
 * are expected to be finite: a NaN or infinity reaches the later tokens of
 * its own sequence and may reach up to 31 earlier ones (its block of the
 * matrix products); one in x or dt stays in its head, one in b or c in its
 * group's heads, and none reaches another sequence.
 */
#define GDN_SSM_SOFTPLUS 1u
typedef struct gdn_ssm_options {
  const float* a_log;    /* f32 [H] device array, or NULL for zeros (rate 1)  */
  const float* dt_bias;  /* f32 [H] device array, or NULL for zeros           */
  const float* d_skip;   /* f32 [H] device array, or NULL (no skip)           */
  uint32_t flags;        /* GDN_SSM_* (default GDN_SSM_SOFTPLUS)              */
  /* Segments: a sequence's transition is one number per token and head, so
   * it can be cut into segments whose end states are formed at once (each
   * from zero), joined in order, and then scanned at once.  0 (default):
   * automatic; -1: one pass over each sequence; n > 0: segments of n blocks
   * of 64 tokens.  The results differ in rounding, and the automatic choice
   * follows the whole batch (its tokens and sequences, the heads and types);
   * with -1 or n, a sequence's results do not depend on the others.  None
   * depends on whether final_state is given.                                */
  int32_t segment_blocks;
} gdn_ssm_options;

/* Fills *opts with the defaults listed in gdn_ssm_options. */
void gdn_ssm_default_options(gdn_ssm_options* opts);

/*
 * gdn_ssm_prefill -- the scan over prompts.
 *   x, out      [T, H, P] or [B, T/B, H, P]; bf16 or f32
 *   dt          [T, H] (or [B, T/B, H]) f32
 *   b, c        [T, G, N] (or 4-D); x's dtype; H a multiple of G
 *   cu_seqlens, init_state, final_state ([Nseq, H, N, P] f32)  as
 *               gdn_prefill; final_state may be init_state
 *   opts        NULL for the defaults
 *   workspace   gdn_ssm_workspace_size() bytes of device memory, 256-byte
 *               aligned (NULL if that is 0); not to be used by another call
 *               that overlaps on the device
 * Sizes: N, P in {16, 32, 64, 128}; at most 65535 heads; (segments + 7) x
 * heads x 4 P < 2^32, and sequences x heads < 2^24 where sequences are cut
 * (GDN_ERR_SHAPE).  Layout of x, b, c and out as gdn_prefill's (16-byte
 * vector accesses), token strides at most 2^24 elements, else GDN_ERR_LAYOUT;
 * dt's strides are any (token stride at most 2^24).
 */
int gdn_ssm_prefill(const gdn_tensor* x, const gdn_tensor* dt, const gdn_tensor* b,
                    const gdn_tensor* c, const gdn_tensor* cu_seqlens,
                    const gdn_tensor* init_state, gdn_tensor* out, gdn_tensor* final_state,
                    const gdn_ssm_options* opts, void* workspace, size_t workspace_bytes,
                    void* stream);

/* Workspace bytes of gdn_ssm_prefill for these shapes (host only; the data
 * pointers are not read). */
int gdn_ssm_workspace_size(const gdn_tensor* x, const gdn_tensor* b,
                           const gdn_tensor* cu_seqlens, const gdn_ssm_options* opts,
                           size_t* bytes);

/*
 * gdn_ssm_decode -- the scan of one token for each of Nseq running
 * sequences, on their states in place.
 *   x, out  [Nseq, H, P]; dt [Nseq, H] f32; b, c [Nseq, G, N]; one dtype,
 *           bf16 or f32, for x, b, c and out
 *   state   f32 [Nseq, H, N, P] contiguous, 16-byte aligned, read and written
 *   opts    NULL for the defaults (segment_blocks is ignored)
 * x and out rows start on 4-element boundaries (address and strides); N, P
 * in {16, 32, 64, 128}.  Nseq = 0 enqueues nothing.
 */
int gdn_ssm_decode(const gdn_tensor* x, const gdn_tensor* dt, const gdn_tensor* b,
                   const gdn_tensor* c, gdn_tensor* state, gdn_tensor* out,
                   const gdn_ssm_options* opts, void* stream);

/*
 * gdn_add_rms_norm -- the residual's addition and the root-mean-square norm
 * before a layer's projections, with its output in the input's type, in 8
 * bits with scales, or both:
 *     r = x + residual (residual NULL: r = x),  residual_out = r,
 *     y = r / sqrt(mean(r^2) + eps) * weight,   out = y,
 *     scales = max(max|y|, 2^-100) / 448,       out_q = y / scales
 * over rows of D elements.  r is kept in fp32 for the norm (residual_out is
 * its rounding); the maximum is taken over each row, or over each 128
 * columns (the last group may be shorter).  out_q rounds to nearest even;
 * dequantised values are out_q * scales.  A NaN anywhere in a row makes the
 * row's y and scales NaN.
 *   x, residual, residual_out, out  [R, D]; one dtype, bf16 or f32
 *   out_q   [R, D] GDN_E4M3;  scales  f32 contiguous, [R] (rows) or
 *           [R, ceil(D / 128)] (groups); both or neither
 *   weight  f32 [D] device array, or NULL for ones;  eps >= 0
 * residual, residual_out, out, out_q with scales, each may be NULL, but not
 * all outputs.  Unit stride in the last dimension, row stride any; 16-byte
 * accesses are used where D, strides and addresses allow.  residual_out may
 * be x or residual, and out may be x or residual (same memory and strides).
 * D <= 65536.
 */
int gdn_add_rms_norm(const gdn_tensor* x, const gdn_tensor* residual, const float* weight,
                     float eps, gdn_tensor* residual_out, gdn_tensor* out, gdn_tensor* out_q,
                     gdn_tensor* scales, void* stream);

/* ------------------------------------------------------------------------
 * The attention layers that a hybrid model has between its recurrent ones,
 * over a paged key-value cache.  The conventions are those of the operators
 * above.  A cache is two arrays [pages, page_size, Hk, d] (any strides that
 * 16-byte accesses fit, so that page-major, head-major and interleaved pools
 * all do); slot s is place s % page_size of page s / page_size.  Row i of a
 * block table [N, M] int32 names the pages that hold request i's tokens in
 * order: its token p lies in page block_table[i][p / page_size].  Entries
 * behind the pages that a request's length needs are not read.  A page
 * outside the cache, inside that length, holds no token that is seen; lengths
 * below 0 or past M * page_size count as those.  page_size is 1 or more,
 * M * page_size and the tokens at most 2^31 - 2^21, requests at most 2^20.
 */

/*
 * gdn_cache_plan -- block tables and slot maps on the device, from the
 * requests' lengths.  Request i has ctx_lens[i] tokens in the cache and the
 * new ones of cu_seqlens (one each without it).  It holds the first
 * ceil(ctx / page_size) pages of its row of the table, and takes what
 * ceil((ctx + new) / page_size) needs more off the top of the stack
 * free_pages[0 .. n_free), from the highest index down, request by request:
 * all of its pages or, if the stack or its row of the table has not that
 * many, none (so does then every later request that needs any from the
 * stack).
 *   block_table  [N, M] int32, in place: only entries of taken pages are
 *                written
 *   seq_lens     [N] int32: ctx + new, or ctx where a request got no pages
 *                (may be ctx_lens)
 *   slots        [T] int64: each new token's slot; -1 for those of a request
 *                that got no pages and those in no sequence.  Nothing of such a
 *                token is stored; its rows of the attention that follows mean
 *                nothing (they are taken for the last tokens of the length that
 *                stayed) and are left out by their slots, until a later plan
 *                serves the request
 *   n_free_out   [1] int32: what is left on the stack (may be n_free)
 * ctx_lens [N], free_pages [F], n_free [1] are int32; all contiguous, the
 * table's row stride any.  A count n_free outside 0 .. F counts as those.
 */
int gdn_cache_plan(const gdn_tensor* ctx_lens, const gdn_tensor* cu_seqlens,
                   gdn_tensor* block_table, const gdn_tensor* free_pages,
                   const gdn_tensor* n_free, int32_t page_size, gdn_tensor* seq_lens,
                   gdn_tensor* slots, gdn_tensor* n_free_out, void* stream);

/*
 * gdn_cache_release -- the pages of the requests with done[i] != 0 back onto
 * the stack, in the order of the requests and of their pages; their lengths
 * become 0 and their entries -1.  Entries below 0 name no page (one given up
 * behind a window, say) and are passed over; any other is taken for a page of
 * the cache.  Pages past the end of free_pages [F] are dropped.  A page belongs
 * to one request.  done, seq_lens [N], block_table
 * [N, M], free_pages [F], n_free [1]: int32, the last four in place.
 */
int gdn_cache_release(const gdn_tensor* done, gdn_tensor* seq_lens, gdn_tensor* block_table,
                      gdn_tensor* free_pages, gdn_tensor* n_free, int32_t page_size,
                      void* stream);

/*
 * gdn_cache_store -- rows of new keys and values into their slots.
 *   k, v              [T, Hk, d]; bf16 or f32, unit stride in d, other strides
 *                     multiples of 16 bytes
 *   slots             [T] int64, as gdn_cache_plan gives them; those below 0
 *                     or past the cache are not stored.  No slot twice (of two
 *                     rows either one's elements may stay)
 *   k_cache, v_cache  [pages, page_size, Hk, d] of the same dtype; they may
 *                     interleave in one allocation
 * d in {64, 128, 256}.
 */
int gdn_cache_store(const gdn_tensor* k, const gdn_tensor* v, const gdn_tensor* slots,
                    gdn_tensor* k_cache, gdn_tensor* v_cache, void* stream);

/*
 * Attention.  The query at place p of its sequence sees the keys j <= p, with
 * a window w > 0 only those of j > p - w or j < sinks:
 *     out[t, h] = sum_j softmax_j(scale q[t, h].k_j) v_j
 * over the keys it sees, query head h reading key head h / (H/Hk); a row that
 * sees none is 0.  Scores, the softmax's maximum and sum and the output are
 * held in fp32, and the output is rounded once; with bf16 inputs the weights
 * enter the product with v in bf16 (prompts: one term; single tokens: two).
 * Scores may be of any size that fp32 holds (times log2 e).
 * Inputs of what is seen are expected to be finite: a NaN or infinity in a key
 * reaches the rows that see it and no others; one in a value these, and it may
 * reach the other rows of their tiles of 128 queries (counted from a sequence's
 * first query of the call), earlier ones and, with a window, later ones that no
 * longer see it.  None reaches another sequence, and what lies in the cache
 * behind a sequence's length is never read.
 */
typedef struct gdn_attn_options {
  float scale;     /* multiplies the scores, within +-2^64; 0 (default):
                      1 / sqrt(d)                                             */
  int32_t window;  /* keys that a query sees, its own among them; 0: all      */
  int32_t sinks;   /* first tokens that every query sees beside its window    */
} gdn_attn_options;

/* Fills *opts with the defaults listed in gdn_attn_options. */
void gdn_attn_default_options(gdn_attn_options* opts);

/*
 * gdn_attn_prefill -- attention of prompts.
 *   q, out      [T, H, d] or [B, T/B, H, d]; bf16 or f32
 *   cu_seqlens  as gdn_prefill; rows at or after cu[N] are not written
 *   k, v        without a block table [T, Hk, d] (or 4-D as q): the queries'
 *               own tokens are the whole sequences.  With one, the caches: the
 *               queries are the last tokens of the first seq_lens[i] that the
 *               cache holds of sequence i (the new ones stored already), so
 *               that a prompt can come in chunks or continue what is cached; a
 *               query before a sequence's first token sees none.  Rows of a
 *               request that gdn_cache_plan did not serve mean nothing
 *   block_table, seq_lens  [N, M], [N] int32, or both NULL
 *   opts        NULL for the defaults
 * d in {64, 128, 256}; unit stride in d, other strides multiples of 16 bytes;
 * tokens of k and v at most 2^24 elements apart; at most 65535 query heads, and
 * fewer than 2^23 (tile, head) pairs: tiles of 128 queries (f32: 64), T / 128
 * and one for each sequence of a packed batch, those that a sequence fills
 * without cu_seqlens (so 2^20 requests of a few tokens with 7 heads, or 2^17
 * with 60; a larger batch in several calls).  The last bits of a result
 * depend on whether the call is large or small (keys are shared out between
 * more waves where tiles are few).
 */
int gdn_attn_prefill(const gdn_tensor* q, const gdn_tensor* k, const gdn_tensor* v,
                     const gdn_tensor* cu_seqlens, const gdn_tensor* block_table,
                     const gdn_tensor* seq_lens, gdn_tensor* out, const gdn_attn_options* opts,
                     void* stream);

/*
 * gdn_attn_decode -- attention of one new token for each of N sequences, the
 * last of the seq_lens[i] that the cache holds (the new one stored already;
 * the row of a request that gdn_cache_plan did not serve means nothing).
 *   q, out     [N, H, d]; bf16 or f32; d in {64, 128, 256}, strides as
 *              gdn_attn_prefill, at most 65535 query heads
 *   workspace  gdn_attn_workspace_size() bytes of device memory, 256-byte
 *              aligned; not to be used by another call that overlaps on the
 *              device.  It follows q's dtype and d alone
 * The work is shared out in equal parts over the device, whatever the
 * lengths, and parts of one sequence are joined by a second launch: the last
 * bits of a result depend on the whole batch's lengths.
 */
int gdn_attn_decode(const gdn_tensor* q, const gdn_tensor* k_cache, const gdn_tensor* v_cache,
                    const gdn_tensor* block_table, const gdn_tensor* seq_lens, gdn_tensor* out,
                    const gdn_attn_options* opts, void* workspace, size_t workspace_bytes,
                    void* stream);

/* Workspace bytes of gdn_attn_decode for a q of this dtype and d (host only). */
int gdn_attn_workspace_size(const gdn_tensor* q, size_t* bytes);

/* Short description of a status code (static storage). */
const char* gdn_status_string(int status);

/* Message of the calling thread's last failed call ("" if none). */
const char* gdn_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */

/*
 * kda.h -- C ABI of the MI355X (gfx950) Kimi Delta Attention library.
 *
 * KDA is the gated delta rule with a channel-wise forget gate and one
 * fixed-size state matrix S (d_k x d_v, fp32) per (sequence, head):
 *
 *     S_t = (I - beta_t k_t k_t^T) diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *     o_t = S_t^T q_t,           alpha_t = exp(max(g_t, g_floor))
 *
 * Sources (page title, section):
 *   - delta-rule update (erase along k, then write), output read from the
 *     updated state, state of size [d, d_v]: "Kimi K3 深度拆解" (chenxutan.com),
 *     4.2 "线性注意力与 Delta Rule";
 *   - one forget rate per key channel rather than per head: "Kimi K3 技術報告：
 *     三個架構改動一次看懂" (akiraxclaw.com), "長度：KDA 為什麼還要搭配 Gated MLA？";
 *   - fixed-size recurrent state, chunk-parallel computation: "3 分钟看懂
 *     Kimi K3" (landx.limxdynamics.com), "第一条主线";
 *   - lower bound on the log-decay so that every causal chunk, the diagonal
 *     block included, is a dense matrix product: same page, Figure 3; and
 *     "Kimi K3 发布 47 页技术报告" (163.com), section 01;
 *   - decode cost and state size independent of context length: "Kimi K3：
 *     预训练规模与推理算力，必须一起扩展" (studioglobal.ai), "KDA 与 Gated MLA".
 * The pages leave the position of the gate relative to the erase open; this
 * library decays first, as in the formula above.
 *
 * Gate variants (kda_gate_t).  KDA's channel-wise gate extends Gated
 * DeltaNet, where one forget rate per head and token serves every key
 * channel (akiraxclaw.com page above, same section); with no gate at all the
 * recurrence is the plain delta rule (chenxutan.com page above, 4.2).  Both
 * are KDA with alpha_t the same for every channel, or 1:
 *   KDA_GATE_CHANNEL  g is [.., H, d_k]: one log-decay per key channel (KDA);
 *   KDA_GATE_HEAD     g is [.., H]: one log-decay per (token, head), applied
 *                     to every key channel (Gated DeltaNet);
 *   KDA_GATE_NONE     alpha = 1, g is not read and may be NULL (DeltaNet).
 *
 * Conventions for every entry point
 *   - Tensor pointers are DEVICE pointers to contiguous row-major arrays,
 *     16-byte aligned.  The caller owns every buffer; the library allocates
 *     nothing, never synchronises and is reentrant.  Its one piece of global
 *     state is the fixed device scratch of kda_chunk_forward_noalloc.
 *   - Arguments are validated on the host before any launch, so argument
 *     errors come back as status codes even on a machine without a GPU.  The
 *     only HIP calls before the launches are one device-attribute query
 *     (the current device's compute units, which the chunked forward's cut
 *     into segments depends on; 256 when no device answers) and, in
 *     kda_chunk_forward_noalloc, the device address of its scratch.
 *   - Work is enqueued on `stream` (a hipStream_t; NULL = the default stream)
 *     and is asynchronous: results are valid once the caller synchronises.
 *   - A failed launch returns KDA_ERR_HIP: each launch's own status is
 *     checked (an error that earlier, unrelated HIP calls left on the calling
 *     thread is neither reported nor cleared).  No C++ exception crosses the
 *     ABI.
 *   - Log-decays g must be <= 0 (alpha in (0, 1]); the library applies
 *     max(g, g_floor) itself, which is a no-op on inputs already floored.
 *   - NaN or Inf inputs propagate into the outputs; they never fault or hang.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_VERSION 20100 /* 2.1.0 */

typedef enum {
  KDA_OK = 0,
  KDA_ERR_INVALID_ARGUMENT = 1, /* NULL pointer, bad size, misalignment, overlap */
  KDA_ERR_UNSUPPORTED = 2,      /* valid but not implemented (e.g. d_k = 96)   */
  KDA_ERR_WORKSPACE_TOO_SMALL = 3,
  KDA_ERR_HIP = 4               /* the HIP runtime reported an error          */
} kda_status_t;

typedef enum { KDA_DTYPE_F32 = 0, KDA_DTYPE_BF16 = 1 } kda_dtype_t;

typedef enum { KDA_GATE_CHANNEL = 0, KDA_GATE_HEAD = 1, KDA_GATE_NONE = 2 } kda_gate_t;

/* Shape of one chunked forward call (the KDA gate: g per key channel). */
typedef struct {
  int B;            /* batch; must be 1 when n_seqs > 0                      */
  int T;            /* tokens per batch row (packed total when n_seqs > 0)   */
  int H;            /* heads                                                 */
  int d_k;          /* key/query channels: 64 or 128 (fp32 chunked: 64)     */
  int d_v;          /* value channels: must equal d_k                        */
  int chunk;        /* tokens per chunk: 64                                  */
  int n_seqs;       /* 0: B sequences of T tokens; > 0: packed sequences     */
  kda_dtype_t dtype;/* dtype of q, k, v, g and o                             */
  float g_floor;    /* per-step log-decay floor, in [-1, 0), |chunk*floor|<=16 */
} kda_chunk_desc_t;

/* The shape and the layout of g, for the entry points that take every gate
 * variant (kda_chunk_forward_gated and the measurement, prefix-cache, MXFP8
 * and backward entry points).  gate = KDA_GATE_CHANNEL is kda_chunk_forward's
 * case exactly. */
typedef struct {
  kda_chunk_desc_t shape;
  kda_gate_t gate;
} kda_chunk_desc_ex_t;

/* Static, human-readable name of a status code; never NULL. */
const char* kda_status_string(int status);

/* KDA_VERSION of the built library. */
int kda_version(void);

/*
 * Bytes of device workspace that kda_chunk_forward (and every forward entry
 * point with the same shape) needs for `d`, on the current device.  No
 * launch; see the conventions above.  Returns KDA_OK or KDA_ERR_* for an
 * invalid or unsupported descriptor.  The workspace holds three d_k x d_v
 * fp32 matrices per (segment, head) when sequences are cut into segments
 * (192 KiB at d = 128; the cut aims at about one workgroup per compute unit
 * over all (segment, head) pairs, so 48 MiB at H = 16 for T = 4,096 as for
 * T = 1,048,576), and 16 bytes per packed sequence.
 */
int kda_chunk_forward_workspace_size(const kda_chunk_desc_t* d, size_t* bytes);

/*
 * Chunked forward ("prefill") over whole sequences.
 *
 * Computes, for every sequence and head, the recurrence above over the
 * sequence's tokens, starting from h0 (or zeros), writing o for every token
 * and the final state to ht.  Internally the sequence is cut into chunks of
 * `chunk` tokens (restarting at every sequence start; the last chunk may be
 * short): the chunk-local work is dense bf16/fp32 matrix products and a
 * triangular solve, then the state is carried from chunk to chunk.  The
 * result equals the token-by-token recurrence up to rounding.
 *
 *   q, k    : [B, T, H, d_k]  dtype
 *   g       : [B, T, H, d_k]  dtype, log-decays (natural log) per key channel
 *   v       : [B, T, H, d_v]  dtype
 *   beta    : [B, T, H]       fp32, write strengths in [0, 1]
 *   h0      : [S, H, d_k, d_v] fp32 or NULL (= zero state); S = n_seqs or B
 *   cu_seqlens: device int32 [n_seqs + 1], cu[0] = 0, non-decreasing,
 *             cu[n_seqs] = T; NULL when n_seqs == 0.  Contents are trusted
 *             (they live on the device); callers validate them beforehand.
 *   o       : [B, T, H, d_v]  dtype, written
 *   ht      : [S, H, d_k, d_v] fp32, written, or NULL; may alias h0 exactly
 *   workspace: device buffer of at least kda_chunk_forward_workspace_size()
 *             bytes, 256-byte aligned; its contents are scratch.
 * o must not overlap any input; ht must not overlap q, k, v, g, beta or o.
 */
int kda_chunk_forward(const kda_chunk_desc_t* d,
                      const void* q, const void* k, const void* v, const void* g,
                      const float* beta, const float* h0,
                      const int32_t* cu_seqlens,
                      void* o, float* ht,
                      void* workspace, size_t workspace_bytes,
                      void* stream);

/*
 * kda_chunk_forward for every gate variant: d->gate selects the layout of g,
 *   g : [B, T, H, d_k] (KDA_GATE_CHANNEL), [B, T, H] (KDA_GATE_HEAD) dtype,
 *       or NULL (KDA_GATE_NONE: not read).
 * Workspace: kda_chunk_forward_workspace_size(&d->shape).  Everything else
 * as kda_chunk_forward; with KDA_GATE_CHANNEL the two calls are identical.
 */
int kda_chunk_forward_gated(const kda_chunk_desc_ex_t* d,
                            const void* q, const void* k, const void* v, const void* g,
                            const float* beta, const float* h0,
                            const int32_t* cu_seqlens,
                            void* o, float* ht,
                            void* workspace, size_t workspace_bytes,
                            void* stream);

/*
 * kda_chunk_forward for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same call with no workspace argument.  Its workspace is a
 * fixed scratch array of KDA_NOALLOC_SCRATCH_BYTES (64 MiB) in the library's
 * device code, one per device, held from the library's load on that device
 * until the process ends; the call itself allocates nothing.  The cut into
 * segments keeps to that size (at H = 16 the best cut needs 48 MiB, and
 * shapes whose best cut needs more take the best one that fits); a call
 * whose smallest cut does not fit (more than about 4 million packed
 * sequences) returns KDA_ERR_WORKSPACE_TOO_SMALL before any launch.  Calls
 * on one device share its scratch: two calls in flight at once on one
 * device (on different streams, or from different threads without ordering)
 * race and give undefined results; calls ordered on one stream are safe.
 * Nothing in the scratch needs clearing between calls.  Everything else as
 * kda_chunk_forward; on the same plan the results are bit-identical to it.
 */
#define KDA_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
int kda_chunk_forward_noalloc(const kda_chunk_desc_t* d,
                              const void* q, const void* k, const void* v, const void* g,
                              const float* beta, const float* h0,
                              const int32_t* cu_seqlens,
                              void* o, float* ht,
                              void* stream);

/*
 * Measurement twin of kda_chunk_forward_gated: the same call, and in
 * addition hipEventRecord(events[i], stream) before each of the call's
 * launches and events[3] after the last one.  The launches, in stream order:
 *   0: map sweep       (each segment's affine state map, from the inputs)
 *   1: segment scan    (every segment's incoming state)
 *   2: output sweep    (o, the final state, prefix-cache states)
 * so hipEventElapsedTime(events[i], events[i + 1]) is launch i's time.  A
 * launch with nothing to do (no tokens, or one segment per sequence: no maps
 * to build or chain) is skipped, its events still recorded.  events: 4
 * hipEvent_t handles created by the caller (any entry may be NULL: not
 * recorded); the array itself must not be NULL.  No synchronisation.
 * Returns what kda_chunk_forward_gated returns, or KDA_ERR_HIP if recording
 * an event fails.
 */
int kda_chunk_forward_timed(const kda_chunk_desc_ex_t* d,
                            const void* q, const void* k, const void* v, const void* g,
                            const float* beta, const float* h0,
                            const int32_t* cu_seqlens,
                            void* o, float* ht,
                            void* workspace, size_t workspace_bytes,
                            void* stream, void* const* events);

/*
 * kda_chunk_forward_gated with q, k and v in MXFP8 (OCP microscaling): each
 * element is one e4m3 byte (finite-only encoding), and every block of 32
 * consecutive channels of one (token, head) shares a scale byte s meaning
 * 2^(s - 127) (e8m0; 255 is not allowed).  Element value = e4m3(byte) *
 * 2^(s - 127).  The decoded values are exact in bf16, and from there the call
 * is the bf16 path: d->shape.dtype must be KDA_DTYPE_BF16, which is the dtype
 * of g and o.  (K3 trains with MXFP8 activations: "Kimi K3 技術報告：三個架構改動
 * 一次看懂" (akiraxclaw.com), "MoonViT-V2 與低位元訓練也不能省略"; here MXFP8
 * halves the bytes of q, k and v.)
 *   q, k, v             : [B, T, H, d] e4m3 bytes, 16-byte aligned
 *   q/k/v_scale         : [B, T, H, d / 32] scale bytes
 * Everything else as kda_chunk_forward_gated (same workspace size); the scale
 * tensors count as inputs in the overlap rules.
 */
int kda_chunk_forward_mx(const kda_chunk_desc_ex_t* d,
                         const void* q, const uint8_t* q_scale,
                         const void* k, const uint8_t* k_scale,
                         const void* v, const uint8_t* v_scale,
                         const void* g, const float* beta, const float* h0,
                         const int32_t* cu_seqlens,
                         void* o, float* ht,
                         void* workspace, size_t workspace_bytes,
                         void* stream);

/*
 * States at chunk boundaries, for prefix caching (the system side of a
 * long-context KDA model keeps KDA states and a prefix cache: "3 分钟看懂
 * Kimi K3" (landx.limxdynamics.com), section "第一条主线", the paragraph after
 * Figure 3).
 *
 * kda_chunk_forward_states_count: host only.  *count = the number of state
 * slots kda_chunk_forward_states may write for this descriptor and
 * states_every (>= 1, in chunks): B * floor(T / (states_every * chunk)) for
 * a fixed-length batch, floor(T / (states_every * chunk)) for a packed one
 * (an upper bound there: the lengths live on the device).
 *
 * kda_chunk_forward_states: kda_chunk_forward_gated, and in addition, for
 * every sequence n in order and every m >= 1 with m * states_every * chunk
 * <= len_n, the state after the first m * states_every * chunk tokens of the
 * sequence (what ht would be for that prefix, so a later call can resume
 * from it as h0) is written to
 *   states[slot]  : [H, d_k, d_v] fp32, row-major like ht,
 *   slot = (slots of sequences 0 .. n-1) + m - 1,
 * i.e. states is [count, H, d_k, d_v] with the slots of each sequence
 * consecutive; slots past the last one written are left untouched.
 * states: device buffer of at least count * H * d_k * d_v floats, 16-byte
 * aligned, overlapping no other buffer; it may be NULL only when count is 0.
 * Returns what kda_chunk_forward_gated returns, and KDA_ERR_INVALID_ARGUMENT
 * for states_every < 1 or a states buffer that breaks the rules above.
 */
int kda_chunk_forward_states_count(const kda_chunk_desc_t* d, int states_every, size_t* count);
int kda_chunk_forward_states(const kda_chunk_desc_ex_t* d,
                             const void* q, const void* k, const void* v, const void* g,
                             const float* beta, const float* h0,
                             const int32_t* cu_seqlens,
                             void* o, float* ht,
                             float* states, int states_every,
                             void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * Backward pass of kda_chunk_forward_gated (training: K3's KDA layers are
 * trained chunk-parallel up to million-token contexts, "3 分钟看懂 Kimi K3"
 * (landx.limxdynamics.com), "第一条主线"; the pages give no gradient, so it is
 * derived from the recurrence above by the chain rule).
 *
 * Given dout = dL/do and dht = dL/dht for the forward with the same
 * descriptor and inputs, writes the gradients of L with respect to every
 * input:
 *   dq, dk  : [B, T, H, d_k]  dtype          dv: [B, T, H, d_v] dtype
 *   dg      : the layout of g (dtype), or NULL with KDA_GATE_NONE (ignored)
 *   dbeta   : [B, T, H] fp32
 *   dh0     : [S, H, d_k, d_v] fp32, or NULL (not written)
 * dout: [B, T, H, d_v] dtype; dht: [S, H, d_k, d_v] fp32 or NULL (= zero).
 * The floor max(g, g_floor) passes the gradient where g >= g_floor (on the
 * floor itself too: the derivative from above) and gives 0 where g is below.
 * The call replays the forward internally (its outputs are not needed).
 * The workspace (256-byte aligned) holds the replay's state after every
 * chunk (64 KiB per (chunk of 64 tokens, head) at d = 128) and, for the
 * chunks in flight, fp32 records and state gradients (about 0.27 MiB per
 * (chunk, head) at d = 128; at d = 64 also a scratch area).  Chunks are
 * processed in windows of W chunk indices of every sequence, from the last
 * window to the first; the call takes the widest window that fits
 * workspace_bytes (one window for the whole sequence when everything fits),
 * and the results do not depend on it.  kda_chunk_backward_workspace_size gives the default: one
 * window unless the in-flight areas of the whole call would pass 8192
 * (chunk, head) pairs, else windows of max(64, 8192 / (H rows)) chunks.
 * A workspace too small for windows of one chunk is
 * KDA_ERR_WORKSPACE_TOO_SMALL.  Outputs must not overlap each other, the
 * inputs or the workspace.  Other rules as kda_chunk_forward.
 */
int kda_chunk_backward_workspace_size(const kda_chunk_desc_t* d, size_t* bytes);
int kda_chunk_backward(const kda_chunk_desc_ex_t* d,
                       const void* q, const void* k, const void* v, const void* g,
                       const float* beta, const float* h0, const int32_t* cu_seqlens,
                       const void* dout, const float* dht,
                       void* dq, void* dk, void* dv, void* dg, float* dbeta, float* dh0,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * kda_chunk_backward with part of its work on a second stream.  Only the
 * local-gradient stage reads what the forward replay writes, so the replay
 * runs beside the state-gradient stage, which fills one CU per (sequence,
 * head, 16 state columns) and leaves the rest idle at small batch.  That stage
 * is then walked in several launches over ranges of the chunks, the last
 * chunks first (four ranges of the chunks, or of each window when the
 * workspace makes windows; two when that span is 64 chunks or fewer), and
 * the local gradients of each range but the
 * first run on the second stream beside the walk over the ranges before it.
 *   aux_stream : hipStream_t (NULL = the default stream) that work is
 *                enqueued on; it waits for `stream` at each fork, and
 *                `stream` waits for it before the call's last launch and
 *                once more at the end.
 *   fork_event, join_event : two distinct caller-created hipEvent_t; both are
 *                re-recorded by every call, so concurrent calls need their own.
 * Results are bit-identical to kda_chunk_backward.  Every work item the call
 * enqueues is ordered before later work on `stream`.  Arguments, workspace
 * and errors as kda_chunk_backward; NULL or equal events are
 * KDA_ERR_INVALID_ARGUMENT.
 */
int kda_chunk_backward_overlapped(const kda_chunk_desc_ex_t* d,
                                  const void* q, const void* k, const void* v, const void* g,
                                  const float* beta, const float* h0, const int32_t* cu_seqlens,
                                  const void* dout, const float* dht,
                                  void* dq, void* dk, void* dv, void* dg, float* dbeta, float* dh0,
                                  void* workspace, size_t workspace_bytes, void* stream,
                                  void* aux_stream, void* fork_event, void* join_event);

/*
 * Measurement twin of kda_chunk_backward: events[i] (5 caller-created
 * hipEvent_t, entries may be NULL) is recorded before stage i and events[4]
 * after the last.  Stages: 0 forward replay (its launches), 1 chunk records,
 * 2 state gradients (reverse over the chunks), 3 local gradients.  With
 * several windows of chunks (a workspace smaller than one window needs),
 * stages 1 to 3 are those of the first window processed (the last chunks)
 * and the interval from events[3] to events[4] also holds the later windows.
 */
int kda_chunk_backward_timed(const kda_chunk_desc_ex_t* d,
                             const void* q, const void* k, const void* v, const void* g,
                             const float* beta, const float* h0, const int32_t* cu_seqlens,
                             const void* dout, const float* dht,
                             void* dq, void* dk, void* dv, void* dg, float* dbeta, float* dh0,
                             void* workspace, size_t workspace_bytes, void* stream,
                             void* const* events);

/*
 * One decode step: one new token for each of N sequences, state resident
 * in device memory and updated IN PLACE.  For every (n, h):
 *     S' = diag(alpha) S;  u = beta (v - S'^T k);  S <- S' + k u^T;
 *     o  = S^T q
 * (the recurrence above for a single token; decode cost and state size do
 * not depend on how many tokens came before).
 *
 *   q, k, g : [N, H, d_k] dtype (g: log-decays per key channel)
 *   v       : [N, H, d_v] dtype
 *   beta    : [N, H] fp32            o: [N, H, d_v] dtype, written
 *   state   : [N, H, d_k, d_v] fp32, read and overwritten
 * d_k = d_v in {64, 128}.  state must not overlap any other argument and o
 * must not overlap any input.
 */
int kda_decode_step(int N, int H, int d_k, int d_v, kda_dtype_t dtype, float g_floor,
                    const void* q, const void* k, const void* v, const void* g,
                    const float* beta, float* state, void* o, void* stream);

/*
 * kda_decode_step for every gate variant: g is [N, H, d_k]
 * (KDA_GATE_CHANNEL), [N, H] (KDA_GATE_HEAD) dtype, or NULL (KDA_GATE_NONE:
 * not read).  With KDA_GATE_CHANNEL identical to kda_decode_step.
 */
int kda_decode_step_gated(int N, int H, int d_k, int d_v, kda_dtype_t dtype, kda_gate_t gate,
                          float g_floor, const void* q, const void* k, const void* v, const void* g,
                          const float* beta, float* state, void* o, void* stream);

/* ---- the operators around the recurrence --------------------------------
 *
 * What makes a layer's q, k and v from its projections (a short causal
 * convolution over the tokens, a norm and a position rotation for every
 * head), and the recurrence with a diagonal transition that hybrid models
 * put beside the delta rule (a selective state space scan).  The conventions
 * at the top of this header hold, with these differences:
 *   - Some inputs may be column slices of a wider row-major array (the output
 *     of one projection): `ld_*` is the distance between consecutive tokens'
 *     rows in elements (0: the row length, that is, contiguous rows), at
 *     least the row length.  Tokens are numbered through the whole batch, so
 *     one distance serves every batch row.  A row itself is contiguous.
 *   - Inputs and outputs need the alignment of their elements only (a slice
 *     starts anywhere); the workspace needs 256 bytes.
 *   - There is no floor and no sign rule on any input.  The scan's states may
 *     grow as well as shrink (rates above zero, steps of either sign): they
 *     are what the recurrence gives while that stays inside fp32.
 *   - Packed batches: cu_seqlens as kda_chunk_forward.  Sequences may be
 *     empty (their final state is their initial state).  Offsets that break
 *     those rules give wrong results, but no access outside the arrays; rows
 *     behind an offset cu[n_seqs] < T are not written.
 *   - Parameters (weight, A) are read, and not NULL, also without tokens.
 *   - KDA_ERR_UNSUPPORTED: 2^31 - 4096 tokens or more; what the descriptors
 *     state; more than 2^23 channels of a convolution; rows of x, dt or z
 *     more than 2^24 elements apart, or D N above 2^28, in a scan; a step of
 *     2^31 elements (convolution) or 2^27 channels (scan) or more; a batch
 *     that needs 2^32 threads or more along a launch's first dimension.
 *   - Sums, states and statistics are held in fp32, outputs are rounded once.
 *     Results do not depend on the launch: no atomics, every sum has a fixed
 *     order.
 */

typedef enum { KDA_ACT_NONE = 0, KDA_ACT_SILU = 1, KDA_ACT_SIGMOID = 2 } kda_act_t;
typedef enum { KDA_NORM_UNIT = 0, KDA_NORM_RMS = 1 } kda_norm_t;

/* Shape of one short convolution. */
typedef struct {
  int B;            /* batch; must be 1 when n_seqs > 0                      */
  int T;            /* tokens per batch row (packed total when n_seqs > 0)   */
  int D;            /* channels                                              */
  int width;        /* taps: 2, 3 or 4                                       */
  int n_seqs;       /* 0: B sequences of T tokens; > 0: packed sequences     */
  kda_dtype_t dtype;/* dtype of x, y, the states and their gradients         */
  kda_act_t activation; /* none or SiLU                                      */
  int64_t ld_x;     /* distance between token rows of x, in elements (0: D)  */
} kda_conv_desc_t;

/*
 * Short causal convolution, one filter per channel.  For every sequence,
 * with xe the sequence preceded by its initial state's width - 1 inputs:
 *     u_t = bias + sum_{j < width} weight[:, j] xe_{t + j}
 *         (the last tap meets token t, the ones before it earlier tokens)
 *     y_t = u_t, or u_t sigmoid(u_t) with KDA_ACT_SILU
 *   x       : [B, T, D] dtype, rows ld_x apart
 *   weight  : [D, width] fp32           bias: [D] fp32 or NULL
 *   initial_state : [S, width - 1, D] dtype, oldest input first, or NULL
 *             (zeros); S = n_seqs or B
 *   y       : [B, T, D] dtype, written
 *   final_state : [S, width - 1, D] dtype, written (the sequence's last
 *             width - 1 inputs, taken from the initial state where it has
 *             fewer), or NULL
 * Outputs must not overlap each other or any input.
 */
int kda_short_conv_forward(const kda_conv_desc_t* d, const void* x, const float* weight, const float* bias,
                           const void* initial_state, const int32_t* cu_seqlens, void* y, void* final_state,
                           void* stream);

/*
 * One new token for each of d->B sequences (d->T must be 1, d->n_seqs 0),
 * the state updated in place: x [B, D] (rows ld_x apart), y [B, D], state
 * [B, width - 1, D].  The same results as kda_short_conv_forward on one
 * token.  y and state must not overlap each other or any input.
 */
int kda_short_conv_step(const kda_conv_desc_t* d, const void* x, const float* weight, const float* bias, void* state,
                        void* y, void* stream);

/*
 * Gradients of <dy, y> + <dfinal, final_state>.
 *   dy      : [B, T, D] dtype;   dfinal : [S, width - 1, D] dtype or NULL (zero)
 *   dx      : [B, T, D] dtype;   dweight: [D, width] fp32
 *   dbias   : [D] fp32 or NULL;  dinitial: [S, width - 1, D] dtype or NULL
 * Every output given is written (dx, dweight are required).  The workspace
 * (kda_short_conv_backward_workspace_size) holds partial sums of dweight and
 * dbias over ranges of tokens.  Outputs must not overlap each other, the
 * inputs or the workspace.
 */
int kda_short_conv_backward_workspace_size(const kda_conv_desc_t* d, size_t* bytes);
int kda_short_conv_backward(const kda_conv_desc_t* d, const void* x, const float* weight, const float* bias,
                            const void* initial_state, const int32_t* cu_seqlens, const void* dy, const void* dfinal,
                            void* dx, float* dweight, float* dbias, void* dinitial, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Shape of one selective scan. */
typedef struct {
  int B;            /* batch; must be 1 when n_seqs > 0                      */
  int T;            /* tokens per batch row (packed total when n_seqs > 0)   */
  int D;            /* channels                                              */
  int N;            /* states per channel: 1 .. 64                           */
  int G;            /* groups of D / G channels that share B and C           */
  int n_seqs;       /* 0: B sequences of T tokens; > 0: packed sequences     */
  kda_dtype_t dtype;/* dtype of x, dt, z, B, C, o and their gradients        */
  int softplus;     /* nonzero: delta = softplus(dt + dt_bias), else dt + dt_bias */
  int64_t ld_x, ld_dt, ld_z; /* distances between token rows (0: D)          */
  int64_t ld_b, ld_c;        /* the same for B and C (0: G * N)              */
} kda_scan_desc_t;

/*
 * Selective state space scan.  Per sequence, channel c (of group g) and
 * state n, from h = h0 (or zeros):
 *     delta_t = softplus(dt_t + dt_bias_c)
 *     h_t[n]  = exp(delta_t A[c, n]) h_{t-1}[n] + delta_t B_t[g, n] x_t
 *     y_t     = sum_n C_t[g, n] h_t[n] + skip_c x_t
 *     o_t     = y_t z_t sigmoid(z_t)       (y_t when z is NULL)
 *   x, dt, z: [B, T, D] dtype (z may be NULL), rows ld_* apart
 *   A       : [D, N] fp32               skip, dt_bias: [D] fp32 or NULL (zero)
 *   Bm, Cm  : [B, T, G, N] dtype, token rows ld_b, ld_c apart
 *   h0      : [S, D, N] fp32 or NULL (zero state); S = n_seqs or B
 *   o       : [B, T, D] dtype, written
 *   ht      : [S, D, N] fp32, written, or NULL
 * Outputs must not overlap each other, the inputs or the workspace (in
 * particular ht is not h0: parts of a sequence are scanned at the same time).
 * A NaN or Inf reaches later tokens of its sequence, never another sequence.
 * The workspace (kda_selective_scan_workspace_size; 0 bytes when the batch
 * alone fills the device) holds the state of every range of tokens that the
 * call scans side by side.
 */
int kda_selective_scan_workspace_size(const kda_scan_desc_t* d, size_t* bytes);
int kda_selective_scan_forward(const kda_scan_desc_t* d, const void* x, const void* dt, const float* A,
                               const void* Bm, const void* Cm, const float* skip, const void* z,
                               const float* dt_bias, const float* h0, const int32_t* cu_seqlens, void* o, float* ht,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * One new token for each of d->B sequences (d->T must be 1, d->n_seqs 0),
 * the state [B, D, N] updated in place; o [B, D].  o and state must not
 * overlap each other or any input.
 */
int kda_selective_scan_step(const kda_scan_desc_t* d, const void* x, const void* dt, const float* A, const void* Bm,
                            const void* Cm, const float* skip, const void* z, const float* dt_bias, float* state,
                            void* o, void* stream);

/*
 * Gradients of <dout, o> + <dht, ht>.
 *   dout    : [B, T, D] dtype;           dht: [S, D, N] fp32 or NULL (zero)
 *   dx, ddt : [B, T, D] dtype;           dA : [D, N] fp32
 *   dB, dC  : [B, T, G, N] dtype, contiguous
 *   dskip, ddt_bias: [D] fp32 or NULL (not written)
 *   dz      : [B, T, D] dtype; required with z, ignored without
 *   dh0     : [S, D, N] fp32 or NULL (not written)
 * The workspace holds the state before every 16 tokens (N / 4 bytes per token
 * and channel), the dB and dC of every 16 channels in fp32 (N / 2 bytes per
 * token and channel), the states between ranges of tokens, and smaller sums:
 * some 3/4 N bytes per token and channel, 100 MB for 2 x 2048 tokens of 2048
 * channels with 16 states.  Long sequences are not cut into windows.
 * An infinity among dout reaches the earlier tokens of its sequence as an
 * infinity or, where the decays of 16 tokens together fall below 2^-126, as a
 * NaN.
 * Outputs must not overlap each other, the inputs or the workspace.
 */
int kda_selective_scan_backward_workspace_size(const kda_scan_desc_t* d, size_t* bytes);
int kda_selective_scan_backward(const kda_scan_desc_t* d, const void* x, const void* dt, const float* A,
                                const void* Bm, const void* Cm, const float* skip, const void* z,
                                const float* dt_bias, const float* h0, const int32_t* cu_seqlens, const void* dout,
                                const float* dht, void* dx, void* ddt, float* dA, void* dB, void* dC, float* dskip,
                                void* dz, float* ddt_bias, float* dh0, void* workspace, size_t workspace_bytes,
                                void* stream);

/* Shape of one norm of queries and keys. */
typedef struct {
  int n_tokens;     /* tokens of the whole batch                             */
  int Hq, Hk;       /* heads of q and of k                                   */
  int d;            /* channels per head: even, 2 .. 512                     */
  int rot;          /* channels rotated: even, 0 .. d (0: no rotation)       */
  kda_dtype_t dtype;
  kda_norm_t norm;
  int interleaved;  /* rotated pairs are channels (2i, 2i + 1), else (i, i + rot / 2) */
  float eps;        /* >= 0, finite                                          */
  float q_scale;    /* factor on q's output                                  */
  int64_t ld_q, ld_k;/* distances between token rows (0: Hq d, Hk d)         */
} kda_qk_norm_desc_t;

/*
 * Norm of every query and key head and the rotation by the token's position,
 * in one pass.  For each head x of d channels:
 *     r   = (sum x^2 + eps)^-1/2  (KDA_NORM_UNIT: unit vectors, as the delta
 *           rule's q and k) or (mean x^2 + eps)^-1/2  (KDA_NORM_RMS)
 *     v   = x r weight
 *     pair i < rot / 2 of v turned by the angle positions[t] inv_freq[i]:
 *           (a, b) -> (a cos - b sin, a sin + b cos)
 *     q_out = q_scale v,  k_out = v
 *   q, k    : [n_tokens, Hq, d], [n_tokens, Hk, d] dtype, token rows ld_* apart
 *   q_weight, k_weight: [d] fp32 or NULL (ones)
 *   positions: [n_tokens] int32, inv_freq: [rot / 2] fp32; NULL when rot is 0
 *   q_out, k_out: contiguous, written; must not overlap anything
 * The angle is reduced in 64 bits, so far positions keep their accuracy.
 */
int kda_qk_norm_forward(const kda_qk_norm_desc_t* d, const void* q, const void* k, const float* q_weight,
                        const float* k_weight, const int32_t* positions, const float* inv_freq, void* q_out,
                        void* k_out, void* stream);

/*
 * Gradients of <dq_out, q_out> + <dk_out, k_out>; dq_out, dk_out, dq, dk are
 * contiguous; dq_weight, dk_weight: [d] fp32 or NULL (not written; given
 * without the weight they are the gradient at a weight of ones).  The
 * workspace holds partial sums of the weights' gradients.
 */
int kda_qk_norm_backward_workspace_size(const kda_qk_norm_desc_t* d, size_t* bytes);
int kda_qk_norm_backward(const kda_qk_norm_desc_t* d, const void* q, const void* k, const float* q_weight,
                         const float* k_weight, const int32_t* positions, const float* inv_freq, const void* dq_out,
                         const void* dk_out, void* dq, void* dk, float* dq_weight, float* dk_weight, void* workspace,
                         size_t workspace_bytes, void* stream);

/* ---- linear attention with a decay for each head -------------------------
 *
 * The recurrence without the delta rule's erase step, as decayed linear
 * attention and state space layers in their attention form have it.  The
 * conventions of the operators above hold, with slices, alignment, packed
 * batches and unchecked offsets as there.
 */

typedef enum {
  KDA_DECAY_NONE = 0,  /* g NULL: nothing is forgotten                       */
  KDA_DECAY_HEAD = 1,  /* g [H] fp32: one log decay for each head            */
  KDA_DECAY_TOKEN = 2  /* g [B, T, H] dtype: one for each token and head     */
} kda_decay_t;

/* Shape of one linear attention. */
typedef struct {
  int B;            /* batch; must be 1 when n_seqs > 0                      */
  int T;            /* tokens per batch row (packed total when n_seqs > 0)   */
  int Hq;           /* heads of q and k                                      */
  int H;            /* heads of v: a multiple of Hq; head h reads q's and k's head h / (H / Hq) */
  int d_k, d_v;     /* channels of a head: 1 .. 128                          */
  int n_seqs;       /* 0: B sequences of T tokens; > 0: packed sequences     */
  kda_dtype_t dtype;/* dtype of q, k, v, g, o and their gradients            */
  kda_decay_t decay;
  float scale;      /* factor on o                                           */
  int64_t ld_q, ld_k, ld_v, ld_g; /* distances between token rows, in elements (0: Hq d_k, Hq d_k, H d_v, H) */
} kda_linear_desc_t;

/*
 * Per sequence and head, from S = h0 (or zeros):
 *     a_t = exp(min(g_t, 0))
 *     S_t = a_t S_{t-1} + k_t v_t^T          [d_k, d_v], fp32
 *     o_t = scale S_t^T q_t
 *   q, k    : [B, T, Hq, d_k] dtype, rows ld_q, ld_k apart
 *   v       : [B, T, H, d_v] dtype, rows ld_v apart
 *   g       : as the decay says; values above 0 count as 0, -infinity forgets
 *             everything.  Rows ld_g apart (KDA_DECAY_TOKEN).
 *   h0      : [S, H, d_k, d_v] fp32 or NULL (zero state); S = n_seqs or B
 *   o       : [B, T, H, d_v] dtype, written
 *   ht      : [S, H, d_k, d_v] fp32, written, or NULL
 * Tokens go through in chunks of 64 (fp32: 32): the decay from one token of a
 * chunk to another is one factor, which is 0 below 2^-126, and the products of
 * queries with keys are formed in fp32, where they have to be finite.
 * A NaN or Inf reaches its own and later tokens of its sequence and head (an
 * infinity as an infinity or a NaN), never an earlier token, another sequence
 * or another head.
 * Outputs must not overlap each other, the inputs or the workspace.  The
 * workspace (kda_linear_attn_workspace_size; 0 bytes when the batch alone
 * fills the device) holds the state of every range of tokens that the call
 * scans side by side: about three states for every compute unit at most.
 * Token rows (ld_q .. ld_g, and H d_k, H d_v) lie at most 2^22 elements apart,
 * and a batch has fewer than 2^31 - 4096 tokens (KDA_ERR_UNSUPPORTED).
 */
int kda_linear_attn_workspace_size(const kda_linear_desc_t* d, size_t* bytes);
int kda_linear_attn_forward(const kda_linear_desc_t* d, const void* q, const void* k, const void* v, const void* g,
                            const float* h0, const int32_t* cu_seqlens, void* o, float* ht, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * One new token for each of d->B sequences (d->T must be 1, d->n_seqs 0), the
 * state [B, H, d_k, d_v] updated in place; q, k [B, Hq, d_k], v, o [B, H, d_v],
 * g [B, H] with KDA_DECAY_TOKEN.  o and state must not overlap each other or
 * any input.
 */
int kda_linear_attn_step(const kda_linear_desc_t* d, const void* q, const void* k, const void* v, const void* g,
                         float* state, void* o, void* stream);

/*
 * Gradients of <dout, o> + <dht, ht>.
 *   dout    : [B, T, H, d_v] dtype;      dht: [S, H, d_k, d_v] fp32 or NULL (zero)
 *   dq, dk  : [B, T, Hq, d_k] dtype, summed over the heads that share them
 *   dv      : [B, T, H, d_v] dtype
 *   dg      : [B, T, H] dtype or NULL (not written); 0 where g is above 0.
 *             NULL unless the decay is KDA_DECAY_TOKEN (the others are constants)
 *   dh0     : [S, H, d_k, d_v] fp32 or NULL (not written)
 * dg is summed up from the end of its sequence: a token's is off by what the
 * roundings of later tokens' inner products (q . dq, k . dk) leave, back to the
 * last token whose factor is 0, whose own dg is 0.
 * A NaN or Inf reaches the gradients that the recurrence carries it to, and
 * may reach all of its sequence's and head's dg.
 * The workspace holds the states and their gradients between ranges of tokens
 * as the forward call's, 8 bytes per token and head, and for shared queries
 * and keys (H > Hq) their gradients by head in fp32, 8 d_k bytes per token and
 * head.  Outputs must not overlap each other, the inputs or the workspace.
 */
int kda_linear_attn_backward_workspace_size(const kda_linear_desc_t* d, size_t* bytes);
int kda_linear_attn_backward(const kda_linear_desc_t* d, const void* q, const void* k, const void* v, const void* g,
                             const float* h0, const int32_t* cu_seqlens, const void* dout, const float* dht, void* dq,
                             void* dk, void* dv, void* dg, float* dh0, void* workspace, size_t workspace_bytes,
                             void* stream);

/* ---- the norms at a block's end -------------------------------------------
 *
 * What follows the recurrence in its layer (the norm of every head with the
 * output gate), and what stands between that layer's output and the next
 * block (the residual sum and the norm of it).  Slices and alignment as
 * above.  KDA_ERR_UNSUPPORTED: norms over more than 8192 channels, more than
 * 65536 heads, 2^31 rows (tokens times heads) or more.  A row's sum of squares
 * is held in fp32: past its range (values of 2^64) the norm's factor is 0, and
 * without an epsilon below it (2^-75) an infinity.
 */

/* Shape of one gated norm. */
typedef struct {
  int n_tokens;     /* tokens of the whole batch                             */
  int H;            /* heads                                                 */
  int d;            /* channels per head: 1 .. 8192                          */
  kda_dtype_t dtype;
  kda_act_t activation; /* of the gate: KDA_ACT_SIGMOID or KDA_ACT_SILU      */
  float eps;        /* >= 0, finite                                          */
  int64_t ld_x, ld_gate; /* distances between token rows (0: H d)            */
} kda_gated_norm_desc_t;

/*
 * For each head x of d channels with its gate z:
 *     y = x (mean x^2 + eps)^-1/2 weight act(z)
 *   x, gate : [n_tokens, H, d] dtype, token rows ld_* apart
 *   weight  : [d] fp32 or NULL (ones)
 *   y       : contiguous, written; must not overlap anything
 */
int kda_gated_norm_forward(const kda_gated_norm_desc_t* d, const void* x, const void* gate, const float* weight,
                           void* y, void* stream);

/*
 * Gradients of <dy, y>: dy, dx, dgate [n_tokens, H, d] dtype, contiguous;
 * dweight [d] fp32 or NULL (not written; given without the weight it is the
 * gradient at a weight of ones).  The workspace holds partial sums of dweight.
 */
int kda_gated_norm_backward_workspace_size(const kda_gated_norm_desc_t* d, size_t* bytes);
int kda_gated_norm_backward(const kda_gated_norm_desc_t* d, const void* x, const void* gate, const float* weight,
                            const void* dy, void* dx, void* dgate, float* dweight, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Shape of one residual norm. */
typedef struct {
  int n_tokens;     /* tokens of the whole batch                             */
  int D;            /* channels: 1 .. 8192                                   */
  kda_dtype_t dtype;
  float scale;      /* on the block's output x                               */
  float eps;        /* >= 0, finite                                          */
  int64_t ld_x, ld_residual; /* distances between token rows (0: D)          */
} kda_residual_norm_desc_t;

/*
 * For each token:
 *     total = residual + scale channel_scale x
 *     y     = total (mean total^2 + eps)^-1/2 weight
 *   x, residual: [n_tokens, D] dtype, rows ld_* apart
 *   weight, channel_scale: [D] fp32 or NULL (ones)
 *   y, total: contiguous, written; must not overlap anything.  y is the norm
 *             of the sum before it is rounded to total's dtype.
 */
int kda_residual_norm_forward(const kda_residual_norm_desc_t* d, const void* x, const void* residual,
                              const float* weight, const float* channel_scale, void* y, void* total, void* stream);

/*
 * Gradients of <dy, y> + <dtotal, total>, from the total that the forward
 * call left (its rows ld_residual apart):
 *   dtotal  : [n_tokens, D] dtype, contiguous, or NULL (zero)
 *   dresidual: [n_tokens, D] dtype, written
 *   dx      : [n_tokens, D] dtype or NULL (not written: with a scale of 1 and
 *             no channel_scale it is dresidual)
 *   dweight, dchannel_scale: [D] fp32 or NULL (not written); the second needs
 *             x, which is not read otherwise and may be NULL
 * The workspace holds partial sums of the parameters' gradients.
 */
int kda_residual_norm_backward_workspace_size(const kda_residual_norm_desc_t* d, size_t* bytes);
int kda_residual_norm_backward(const kda_residual_norm_desc_t* d, const void* x, const void* total, const float* weight,
                               const float* channel_scale, const void* dy, const void* dtotal, void* dx,
                               void* dresidual, float* dweight, float* dchannel_scale, void* workspace,
                               size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */

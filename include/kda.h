/*
 * kda.h — C ABI of the MI355X (gfx950) Kimi Delta Attention (KDA) library.
 *
 * What is computed ("Kimi K3, explained", vibeengines.com/paper/kimi-k3,
 * sections "How Kimi Delta Attention works, step by step" and "The math",
 * gated delta rule equation; the page writes the state as d_v x d_k, this
 * library stores its transpose):
 *
 *   per sequence and head, state S in R^{d_k x d_v} (row = key channel,
 *   column = value channel), alpha_t = exp(g_t) per key channel:
 *       S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *       o_t = S_t^T q_t                      (read after the write)
 *
 * Prefill and append-prefill evaluate this recurrence in chunks of `chunk`
 * tokens ("Training in chunks": inside a chunk the product of decay-and-erase
 * transitions becomes dense products plus one triangular solve; only S
 * crosses chunk boundaries).  Decode applies one token per sequence at a cost
 * independent of the context length ("The decode wall"; "KDA: trade the cache
 * for a fixed-size state").
 *
 * Conventions shared by every entry point
 *   - Every tensor pointer is a DEVICE pointer owned by the caller; tensors are
 *     contiguous and row-major.  Alignment: for prefill and append, q, k and g
 *     16 bytes and the workspace 256 bytes; for decode, both states 16 bytes;
 *     every other pointer its element size.
 *   - Sizes: H * max(d_k, d_v) must be below 2^23 (a chunk's rows are
 *     addressed with 32-bit byte offsets); KDA_ERR_INVALID_ARG otherwise.
 *   - q, k, v and beta have the storage type `dtype` (KDA_F32: float,
 *     KDA_BF16: bfloat16).  g = log(alpha) is always float (fp32, values <= 0
 *     expected), states and outputs are always float.
 *   - Calls are asynchronous on `hip_stream` (a hipStream_t; NULL = the null
 *     stream).  The library never synchronises (unless KDA_DEBUG_SYNC=1 or
 *     KDA_DEBUG_CHECK=1 is set in the environment), never allocates or frees
 *     device memory, and keeps no pointer after returning.  The caller keeps
 *     every buffer alive until the stream has drained.
 *   - Return value: KDA_OK or a negative kda_status.  Arguments are validated
 *     on the host before any device work; a failed call launches nothing.
 *     kda_last_error() gives a message for the calling thread.
 *   - Device-resident data (cu_seqlens and snapshot_cu contents, gate ranges)
 *     is a caller contract and is not inspected by default.  With
 *     KDA_DEBUG_CHECK=1 in the environment every call first waits for its
 *     stream, copies those arrays to the host and checks them with the
 *     kda_validate_* functions below (cu_seqlens: cu[0] = 0, non-decreasing,
 *     cu[N] = T_total; snapshot_cu: consistent with cu_seqlens; g finite and
 *     <= 0, beta in [0, 1]; with the fused prologue, g and beta finite).  A
 *     violation returns KDA_ERR_INVALID_ARG before any launch.  Without the
 *     check, offsets that break the contract make the kernels read and write
 *     outside the caller's buffers.
 *   - bfloat16 path numerics (d_k = d_v = 128, chunk 64): products inside a
 *     chunk use fp16 matrix-core operands with fp32 accumulation; the state,
 *     the decays and all outputs are fp32.  Every value rounded to an fp16
 *     operand is first checked against the fp16 range (|x| < 65504; NaN and
 *     Inf fail too): q and k entries (which must not exceed 32768; unit-length
 *     q and k, as the DeltaNet family uses them, are far inside), the gated
 *     Gram matrix M, the UT transform T and the WY factor W per chunk, and
 *     beta*v, the per-token corrections and the state per chain.  A (sequence,
 *     head, 16-column value block) chain that meets a value outside the range
 *     is recomputed in the same call by the fp32 chunked evaluation (fp32
 *     accuracy, at that path's speed), so there is no range limit beyond
 *     fp32's.  Decays of any strength are exact up to rounding: a
 *     chunk in which some channel decays by more than e^10 over 8 tokens sums
 *     its diagonal 16x16 Gram tiles in fp32 with one exponential per token
 *     pair, which costs that chunk extra time.  The fp32 path has no such
 *     limits.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = -1, /* null pointer, negative size, bad cu_seqlens count, ... */
    KDA_ERR_UNSUPPORTED = -2, /* (dtype, d_k, d_v, chunk) combination not implemented */
    KDA_ERR_MISALIGNED = -3,  /* a pointer is not aligned as required (see Conventions) */
    KDA_ERR_ALIAS = -4,       /* outputs overlap inputs, or state_out partially overlaps state_in */
    KDA_ERR_WORKSPACE = -5,   /* workspace missing or smaller than kda_workspace_size() */
    KDA_ERR_HIP = -6          /* the HIP runtime reported an error (message in kda_last_error) */
} kda_status;

typedef enum { KDA_F32 = 0, KDA_BF16 = 1 } kda_dtype;

typedef enum { KDA_OP_PREFILL = 0, KDA_OP_APPEND = 1, KDA_OP_DECODE = 2, KDA_OP_BACKWARD = 3 } kda_op;

/*
 * Chunked prefill of B equal-length sequences of T tokens.
 *   q, k       [B, T, H, d_k]   dtype
 *   v          [B, T, H, d_v]   dtype
 *   g          [B, T, H, d_k]   float, log of the per-channel forget gate alpha
 *   beta       [B, T, H]        dtype, write strength
 *   state_in   [B, H, d_k, d_v] float, or NULL for a zero initial state
 *   out        [B, T, H, d_v]   float
 *   state_out  [B, H, d_k, d_v] float, or NULL; may equal state_in (in place),
 *              must not partially overlap it
 *   chunk      tokens per chunk: 16, 32 or 64 (64 for the bfloat16 d=128 path)
 *   workspace  device scratch of at least kda_workspace_size(KDA_OP_PREFILL, B, T, ...)
 *              bytes (NULL allowed when that size is 0), 256-byte aligned,
 *              overlapping no other argument (KDA_ERR_ALIAS); contents need no
 *              initialisation and are clobbered.
 * T = 0 copies state_in to state_out (zeros when state_in is NULL).
 */
int kda_prefill_chunked(const void* q, const void* k, const void* v, const float* g, const void* beta,
                        const float* state_in, float* out, float* state_out, int64_t B, int64_t T,
                        int32_t H, int32_t d_k, int32_t d_v, int32_t dtype, int32_t chunk,
                        void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * Append-prefill of N packed variable-length segments, each continuing from
 * its own carried state (the append-prefill workload: a long new segment on
 * top of a kept history).
 *   q, k, g    [T_total, H, d_k]; v [T_total, H, d_v]; beta [T_total, H]
 *   cu_seqlens DEVICE int32 [N + 1]: cu[0] = 0, non-decreasing, cu[N] = T_total
 *              (segment n is tokens cu[n] .. cu[n+1]-1; checked only with
 *              KDA_DEBUG_CHECK=1, see Conventions)
 *   state_in   [N, H, d_k, d_v] float or NULL (zeros); state_out as in prefill
 *   out        [T_total, H, d_v] float
 * Empty segments pass their state through unchanged.
 */
int kda_append_prefill(const void* q, const void* k, const void* v, const float* g, const void* beta,
                       const int32_t* cu_seqlens, int32_t N, int64_t T_total, const float* state_in,
                       float* out, float* state_out, int32_t H, int32_t d_k, int32_t d_v, int32_t dtype,
                       int32_t chunk, void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * One decode step: one new token for each of N sequences.
 *   q, k, g    [N, H, d_k]; v [N, H, d_v]; beta [N, H]
 *   state_in   [N, H, d_k, d_v] float (required)
 *   state_out  [N, H, d_k, d_v] float (required); may equal state_in for an
 *              in-place update, must not partially overlap it
 *   out        [N, H, d_v] float
 * Each state element is read once and written once.
 */
int kda_decode_step(const void* q, const void* k, const void* v, const float* g, const void* beta,
                    const float* state_in, float* state_out, float* out, int32_t N, int32_t H,
                    int32_t d_k, int32_t d_v, int32_t dtype, void* hip_stream);

/*
 * Extended calls: the same operations with options.
 *
 * Gate kind ("Kimi K3, explained", "How Kimi Delta Attention works, step by
 * step" and the comparison with Gated DeltaNet, whose forget gate is one
 * scalar per head and token rather than one value per key channel):
 *   KDA_GATE_CHANNEL  g has one log-decay per key channel: [..., H, d_k]
 *                     (KDA; the plain calls always use this).
 *   KDA_GATE_HEAD     g has one log-decay per token and head: [..., H], and
 *                     alpha_t = exp(g_t) multiplies every key channel (Gated
 *                     DeltaNet; g = 0 gives the plain delta rule).
 *
 * State snapshots ("Kimi K3 changed the memory math for agentic AI": keeping
 * the fixed-size state at checkpoints of a long context so that a session can
 * resume from one).  With snapshot_every = E > 0 (prefill and append only),
 * the state after every E * chunk tokens of a sequence is written, counted
 * from the start of the call's tokens for that sequence: snapshot m (m = 0,
 * 1, ...) is the state after the first (m + 1) * E * chunk tokens, for every
 * such count that does not exceed the sequence's length.  The final state
 * still goes to state_out.
 *   prefill: snapshots [B, T / (E * chunk), H, d_k, d_v] float (integer division)
 *   append:  snapshots [snapshot_cu[N], H, d_k, d_v] float, sequence n at rows
 *            snapshot_cu[n] .. snapshot_cu[n+1]-1; snapshot_cu is a DEVICE
 *            int32 [N + 1] with snapshot_cu[0] = 0 and snapshot_cu[n+1] -
 *            snapshot_cu[n] = (cu_seqlens[n+1] - cu_seqlens[n]) / (E * chunk)
 *            (a caller contract, not checked on the device).
 * snapshots must be 4-byte aligned and overlap no other argument.
 *
 * Fused input prologue ("Kimi K3, explained", "How Kimi Delta Attention
 * works, step by step": in the DeltaNet family queries and keys are
 * L2-normalised; beta is a write strength in (0, 1) and alpha a forget gate in
 * (0, 1)).  With prologue = 1 the inputs are the raw projections and the
 * kernels apply, per token and head:
 *   q <- q / ||q||,  k <- k / ||k||       (a zero vector stays zero)
 *   beta <- sigmoid(beta)                 (beta holds logits)
 *   g <- -gate_scale * softplus(g)        (g holds the raw gate input a, per
 *                                          key channel or per head)
 * so that no separate elementwise pass (and no extra round trip through
 * memory) is needed.  gate_scale must be finite and > 0.
 *
 * A NULL options pointer means { KDA_GATE_CHANNEL, 0, NULL, NULL, 0, 0 }.
 */
typedef enum { KDA_GATE_CHANNEL = 0, KDA_GATE_HEAD = 1 } kda_gate;

typedef struct kda_options {
    int32_t gate;               /* kda_gate */
    int32_t snapshot_every;     /* chunks between state snapshots; 0 = none (must be 0 for decode) */
    float* snapshots;           /* see above; NULL when snapshot_every = 0 */
    const int32_t* snapshot_cu; /* append only; NULL otherwise */
    int32_t prologue;           /* 1: raw q, k, beta logits and gate inputs (see above); 0: as stored */
    float gate_scale;           /* prologue only: g = -gate_scale * softplus(a) */
} kda_options;

int kda_prefill_chunked_ex(const void* q, const void* k, const void* v, const float* g, const void* beta,
                           const float* state_in, float* out, float* state_out, int64_t B, int64_t T,
                           int32_t H, int32_t d_k, int32_t d_v, int32_t dtype, int32_t chunk,
                           void* workspace, size_t workspace_bytes, const kda_options* options,
                           void* hip_stream);

int kda_append_prefill_ex(const void* q, const void* k, const void* v, const float* g, const void* beta,
                          const int32_t* cu_seqlens, int32_t N, int64_t T_total, const float* state_in,
                          float* out, float* state_out, int32_t H, int32_t d_k, int32_t d_v, int32_t dtype,
                          int32_t chunk, void* workspace, size_t workspace_bytes, const kda_options* options,
                          void* hip_stream);

int kda_decode_step_ex(const void* q, const void* k, const void* v, const float* g, const void* beta,
                       const float* state_in, float* state_out, float* out, int32_t N, int32_t H,
                       int32_t d_k, int32_t d_v, int32_t dtype, const kda_options* options, void* hip_stream);

/*
 * kda_append_prefill_noalloc — kda_append_prefill_ex without a workspace, for
 * callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc).  Same arguments,
 * results and errors as kda_append_prefill_ex with a workspace (the same
 * kernels), except:
 *   - The scratch the matrix-core path needs (kda_workspace_size(KDA_OP_APPEND,
 *     ...) bytes) comes from a fixed array of KDA_NOALLOC_SCRATCH_BYTES bytes
 *     in device memory that the library holds on each GPU it runs on, from
 *     its first use there until the process ends.  A call that needs more
 *     returns KDA_ERR_WORKSPACE before any launch; 128 MiB covers, e.g.,
 *     H = 32 with T_total / 64 + N <= 62 (one segment of up to 3,904 tokens).
 *     Shapes served by the fp32 kernel need no scratch.
 *   - The call allocates and frees nothing (no hipMalloc, hipFree or
 *     allocating library routine).  Its first call on a device looks up the
 *     array's address on that device once (hipGetSymbolAddress).
 *   - Every call on one GPU shares that GPU's array, which keeps the previous
 *     call's contents (nothing in it needs clearing: every word a call reads
 *     it has written first).  Calls that overlap in time on one GPU (several
 *     streams, or several host threads) race on it: serialise them, e.g. on
 *     one stream.
 *   - KDA_DEBUG_CHECK=1 (see Conventions) synchronises and copies through host
 *     memory, so it is for debugging only, not for the callers above.
 */
#define KDA_NOALLOC_SCRATCH_BYTES ((size_t)128 << 20)

int kda_append_prefill_noalloc(const void* q, const void* k, const void* v, const float* g, const void* beta,
                               const int32_t* cu_seqlens, int32_t N, int64_t T_total, const float* state_in,
                               float* out, float* state_out, int32_t H, int32_t d_k, int32_t d_v, int32_t dtype,
                               int32_t chunk, const kda_options* options, void* hip_stream);

/*
 * kda_chunked_backward — gradients of the chunked prefill (training).
 *
 * "Kimi K3, explained" ("How is KDA trained efficiently if it is a
 * recurrence?"; "Training in chunks") states that training runs the same
 * recurrence in chunks; it prints no gradient equations.  This call returns
 * the derivative of the recurrence of kda_append_prefill (same inputs, same
 * packed layout) with respect to every input, given the gradients of a loss L
 * with respect to its outputs:
 *   d_out        [T_total, H, d_v] float   dL/do (required when T_total > 0)
 *   d_state_out  [N, H, d_k, d_v] float    dL/dS_T, or NULL (zero)
 * and writes (all float, caller-owned, overlapping no input):
 *   dq, dk       [T_total, H, d_k]         dL/dq, dL/dk
 *   dv           [T_total, H, d_v]         dL/dv
 *   dg           [T_total, H, d_k]         dL/dg (g = log alpha); [T_total, H]
 *                                          with options->gate = KDA_GATE_HEAD
 *   dbeta        [T_total, H]              dL/dbeta
 *   d_state_in   [N, H, d_k, d_v]          dL/dS_0, or NULL (not wanted)
 * q, k, v, g, beta, cu_seqlens, state_in, dtype and chunk are as for
 * kda_append_prefill (a batch of B equal sequences is cu_seqlens = 0, T, 2T,
 * ...).  Accumulation is fp32 whatever dtype is; with KDA_BF16 at d = 128,
 * chunk 64 the chain and state-side products multiply split-bf16 operands
 * (each fp32 value as bf16 hi plus bf16 lo, three bf16 matrix-core steps per
 * product, within about 2^-16 of the fp32 product), the rest fp32 operands.
 * Supported shapes:
 * d_k = d_v in {16, 32, 64, 128}, chunk in {16, 32, 64}.  options may be NULL;
 * only options->gate is honoured, and snapshot_every and prologue must be 0
 * (KDA_ERR_UNSUPPORTED otherwise).  workspace: at least
 * kda_workspace_size(KDA_OP_BACKWARD, N, T_total, H, d_k, d_v, dtype, chunk)
 * bytes, 256-byte aligned, overlapping no argument; it holds the per-chunk
 * factors, the states entering each chunk and the state gradients leaving it.
 * That grows with T_total (about 545 KB per chunk and head at d = 128, chunk
 * 64); when it would exceed 20 GiB (or the byte count in the environment
 * variable KDA_BWD_WORKSPACE_CAP, read by both kda_workspace_size and the
 * call, which must agree), the chunks are taken in windows of a fixed number
 * of chunks of every sequence: the factors and the forward state chain run
 * twice (a forward sweep keeping the states at window boundaries, then a
 * reverse sweep that rebuilds each window from its checkpoint), and the
 * workspace is one window's records plus the checkpoints.  The results are
 * bitwise those of the one-pass evaluation.
 * The gradient outputs must not overlap one another either (KDA_ERR_ALIAS).
 * Repeated calls on the same inputs give bitwise equal results (no atomics).
 * Asynchronous on hip_stream; errors as for the other calls.
 */
int kda_chunked_backward(const void* q, const void* k, const void* v, const float* g, const void* beta,
                         const int32_t* cu_seqlens, int32_t N, int64_t T_total, const float* state_in,
                         const float* d_out, const float* d_state_out, float* dq, float* dk, float* dv,
                         float* dg, float* dbeta, float* d_state_in, int32_t H, int32_t d_k, int32_t d_v,
                         int32_t dtype, int32_t chunk, void* workspace, size_t workspace_bytes,
                         const kda_options* options, void* hip_stream);

/*
 * Host-side validators of the device-resident contract (the checks that
 * KDA_DEBUG_CHECK=1 applies to a call's data after copying it to the host).
 * Every pointer here is a HOST pointer; nothing is launched.  Each returns
 * KDA_OK, or KDA_ERR_INVALID_ARG with a message in kda_last_error().
 *   kda_validate_cu_seqlens   cu [N + 1]: cu[0] = 0, cu[n] <= cu[n+1],
 *                             cu[N] = T_total (the append-prefill layout).
 *   kda_validate_snapshot_cu  snapshot_cu [N + 1]: snapshot_cu[0] = 0 and
 *                             snapshot_cu[n+1] - snapshot_cu[n] =
 *                             (cu[n+1] - cu[n]) / (snapshot_every * chunk).
 *   kda_validate_gates        g [n_g] finite and <= 0 (alpha = exp(g) in
 *                             (0, 1]); beta [n_beta] finite and in [0, 1]
 *                             ("Kimi K3, explained", "How Kimi Delta
 *                             Attention works, step by step": both gates lie
 *                             in (0, 1)).  raw = 1 (fused prologue inputs):
 *                             finite only.  beta is given as float.
 */
int kda_validate_cu_seqlens(const int32_t* cu, int32_t N, int64_t T_total);
int kda_validate_snapshot_cu(const int32_t* cu, const int32_t* snapshot_cu, int32_t N, int32_t snapshot_every,
                             int32_t chunk);
int kda_validate_gates(const float* g, int64_t n_g, const float* beta, int64_t n_beta, int32_t raw);

/*
 * Serving next to the recurrence: paged key-value cache, branching, beam search
 * ==========================================================================
 *
 * A hybrid stack runs softmax-attention layers between its recurrent ones.
 * Their keys and values grow with the context, so a serving program keeps them
 * in pages of a fixed number of tokens, names the pages of a sequence in a
 * table, and shares pages between sequences that have a common beginning.  The
 * recurrent states have a fixed size and are copied instead.
 *
 * Layouts (all device memory owned by the caller; the Conventions above hold):
 *   k_pages, v_pages  [n_pages, H_kv, page_size, d] dtype: page p starts
 *                     p * page_stride elements behind the pointer and is
 *                     contiguous.  16-byte aligned, and so is the stride in
 *                     bytes; a stride larger than the page is allowed (several
 *                     layers, or keys and values, in one pool).
 *   page_size         tokens per page, a multiple of 16 (16 .. 4096)
 *   page_table        int32 [N, table_pages], row n starts n * table_stride
 *                     elements behind the pointer: entry j names the page that
 *                     holds tokens j * page_size .. of sequence n.  An entry
 *                     outside [0, n_pages) means that there is no page (write
 *                     -1): attention leaves its tokens out, writes to it are
 *                     dropped.
 *                     Strides of all calls are below 2^40 elements.
 *   lengths           int32 [N], tokens of each sequence
 *   refcount          int32 [n_pages]: how many table entries (of all tables of
 *                     the pool) name the page; 0 means that it is free.  There
 *                     is no other list of free pages.
 * Every index that a kernel reads from device memory (table entries, parents,
 * rows, copy pairs) is checked against its range there, so that a wrong one is
 * left out and never makes a kernel read or write outside the caller's buffers.
 * All calls are deterministic: integer results do not depend on the order in
 * which workgroups run, and free pages are taken lowest first.
 * A call that needs 2^32 or more threads in one launch is refused
 * (KDA_ERR_INVALID_ARG; some 2^24 sequences, table rows or query heads, or 2^28
 * short tokens); kda_pages_copy and kda_beam_reorder go on in further launches.
 */

/*
 * kda_cache_append — writes the keys and values of new tokens into the pages.
 *   k, v        token t at t * k_stride (v_stride) elements: [H_kv, d] dtype,
 *               contiguous; 16-byte aligned, strides too
 *   cu_seqlens  DEVICE int32 [N + 1] as in kda_append_prefill (tokens
 *               cu[n] .. cu[n+1]-1 belong to sequence n), or NULL: one token per
 *               sequence (T_total = N)
 *   start       int32 [N], the position of each sequence's first new token
 * Token i of sequence n goes to position start[n] + i.  A position without a
 * page (before 0, behind the table, or at an entry that names none) is dropped.
 * The pages written must belong to one sequence each (kda_cache_reserve sees to
 * that); two sequences that write the same slot leave either value.  k_pages and
 * v_pages must not overlap (they may for kda_paged_decode, which only reads them).
 * d in {64, 128, 256}.
 */
int kda_cache_append(const void* k, const void* v, int64_t k_stride, int64_t v_stride, const int32_t* cu_seqlens,
                     const int32_t* start, int32_t N, int64_t T_total, void* k_pages, void* v_pages,
                     int64_t k_page_stride, int64_t v_page_stride, int32_t n_pages, int32_t page_size,
                     const int32_t* page_table, int64_t table_stride, int32_t table_pages, int32_t H_kv, int32_t d,
                     int32_t dtype, void* hip_stream);

/*
 * kda_paged_decode — softmax attention of one new token per sequence over its
 * pages (the token's own key and value are in the pages already):
 *   s_t = scale * q . k_t,   out = sum_t softmax(s)_t v_t,   lse = log sum_t exp(s_t)
 * over the visible tokens t < lengths[n] of sequence n.
 *   q       sequence n at n * q_stride elements: [H_q, d] dtype, contiguous;
 *           16-byte aligned, stride too.  H_q is a multiple of H_kv, and query
 *           heads g * H_q / H_kv .. share key-value head g.
 *   window  0, or only the last `window` tokens are visible ...
 *   sinks   ... and the first `sinks` tokens (0 without a window)
 *   max_length  an upper bound of lengths that sizes the launch; 0: the table's
 *           table_pages * page_size (which has to be below 2^31 - 4096).  A longer
 *           sequence is cut there.
 *   out     [N, H_q, d] float; lse [N, H_q] float or NULL
 * A sequence without a visible token (or whose every visible score is -inf)
 * gives out = 0 and lse = -inf.  Tokens that are not visible are never used,
 * whatever bits their slots hold.  Products are exact in bf16 with fp32 sums;
 * with KDA_BF16 the softmax weights enter their product as the sum of three bf16
 * values, which is the fp32 weight itself (from 2^-103 up).  A visible key or value that is not
 * finite makes what it enters NaN, but for a score of -inf, which has weight 0.
 * workspace: kda_paged_decode_workspace bytes for the same arguments, 256-byte
 * aligned, overlapping no argument; holds the partial results where a sequence
 * is split over several workgroups.  Needs no initialisation.
 * d in {64, 128, 256}; lengths are a caller contract (checked with
 * KDA_DEBUG_CHECK=1: 0 <= lengths[n] <= the bound); values below 0 count as 0.
 */
int kda_paged_decode(const void* q, int64_t q_stride, const void* k_pages, const void* v_pages, int64_t k_page_stride,
                     int64_t v_page_stride, int32_t n_pages, int32_t page_size, const int32_t* page_table,
                     int64_t table_stride, int32_t table_pages, const int32_t* lengths, int32_t N, int32_t H_q,
                     int32_t H_kv, int32_t d, int32_t dtype, float scale, int32_t window, int32_t sinks,
                     int64_t max_length, float* out, float* lse, void* workspace, size_t workspace_bytes,
                     void* hip_stream);

/* Workspace bytes of kda_paged_decode, max_length being the smaller of the bound
 * given and table_pages * page_size (not 0 for "no bound" here); (size_t)-1 for an
 * unsupported or invalid combination. */
size_t kda_paged_decode_workspace(int32_t N, int32_t H_q, int32_t H_kv, int32_t d, int32_t dtype, int64_t max_length,
                                  int32_t window, int32_t sinks);

/*
 * kda_cache_fork — a new set of sequences from an old one, sharing its pages:
 * new sequence i is old sequence parents[i] (its table row and length), or empty
 * where parents[i] is outside [0, N).  The old set is released: refcount goes up
 * by what the new table names and down by what the old one named.  So the same
 * call branches (an index several times), reorders beams, keeps (i at place i)
 * and drops sequences.
 *   page_table, lengths          N rows, table_pages wide
 *   table_out, lengths_out       N_out rows, as wide; must not overlap the old
 * Tokens to come are written only after kda_cache_reserve has given the
 * branches pages of their own.
 */
int kda_cache_fork(const int32_t* page_table, int64_t table_stride, const int32_t* lengths, int32_t N,
                   int32_t table_pages, int32_t* refcount, int32_t n_pages, const int32_t* parents, int32_t N_out,
                   int32_t* table_out, int64_t table_out_stride, int32_t* lengths_out, void* hip_stream);

/*
 * kda_cache_free — drops sequences in place: for every r of rows [n_rows] (int32)
 * the pages of row r lose one reference, its entries become -1 and its length 0.
 * A row outside [0, N) is left out; one that is named twice is freed once.
 */
int kda_cache_free(int32_t* page_table, int64_t table_stride, int32_t* lengths, int32_t N, int32_t table_pages,
                   int32_t* refcount, int32_t n_pages, const int32_t* rows, int32_t n_rows, void* hip_stream);

/*
 * kda_cache_reserve — makes room for new_tokens[n] more tokens of every sequence
 * (int32 [N]; 0 or less: the sequence is left alone).  Every page that holds one
 * of the positions lengths[n] .. lengths[n] + new_tokens[n] - 1 is made the
 * sequence's own: an entry without a page, or with one that had more than one
 * reference when the call began, gets a free page (refcount 1) and gives its old
 * one back.  Where the old page held tokens of the sequence (a shared page that
 * is partly filled), the pair (old, new) is returned for kda_pages_copy.
 *   copies   int32 [N, 2]: the page to copy from and to, or -1, -1
 *   granted  int32 [N]: new_tokens[n], or 0 where nothing was reserved
 * lengths[n] grows by granted[n].  Free pages are taken lowest first, sequences
 * in order; a sequence is served if the pages needed by it and by those before it
 * are there, whether those were served or not, and if its table row is wide
 * enough; otherwise it is left as it was.
 * workspace: kda_cache_workspace_size(N, n_pages) bytes, 256-byte aligned.
 */
int kda_cache_reserve(int32_t* page_table, int64_t table_stride, int32_t* lengths, int32_t N, int32_t table_pages,
                      int32_t* refcount, int32_t n_pages, int32_t page_size, const int32_t* new_tokens,
                      int32_t* copies, int32_t* granted, void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * kda_cache_compact — plans the move of the pages in use to the front of the pool
 * with the fewest copies: with L pages in use, the i-th used page at or behind L
 * (ascending) takes the place of the i-th free one before L.
 *   table_out     page_table with the new places (may be page_table itself)
 *   refcount_out  refcount with the new places (may be refcount itself); pages
 *                 L .. are 0
 *   moves         int32 [n_pages / 2, 2]: (from, to) pairs for kda_pages_copy, in
 *                 ascending order, then -1, -1
 * The pages themselves are moved by kda_pages_copy with `moves`, for every pool
 * the table belongs to.  Entries of other tables of the same pool have to be
 * mapped in the same call (pass them as further rows).
 * workspace: kda_cache_workspace_size(N, n_pages) bytes, 256-byte aligned.
 */
int kda_cache_compact(const int32_t* page_table, int64_t table_stride, int32_t N, int32_t table_pages,
                      const int32_t* refcount, int32_t n_pages, int32_t* table_out, int64_t table_out_stride,
                      int32_t* refcount_out, int32_t* moves, void* workspace, size_t workspace_bytes,
                      void* hip_stream);

/* Workspace bytes of kda_cache_reserve and kda_cache_compact; (size_t)-1 for
 * negative sizes or n_pages >= 2^24. */
size_t kda_cache_workspace_size(int32_t N, int32_t n_pages);

/*
 * kda_pages_copy — copies pages inside each of n_pools pools: for every pair
 * (from, to) of pairs [n_pairs, 2] (DEVICE int32) the `page_bytes` bytes of page
 * `from` go to page `to`.  Pairs with an index outside [0, n_pages) are left out.
 * No page may be the target of two pairs, or the source of one and the target of
 * another (the pairs of kda_cache_reserve and kda_cache_compact are such).
 *   pools, page_strides, page_bytes  HOST arrays of n_pools entries: the pool's
 *            device address, bytes between pages, bytes of a page (all multiples
 *            of 16; a page below 4 GiB).  Read before the call returns.
 * Any rows of equal size are pages here, for instance recurrent states
 * [n_pages, H, d_k, d_v].
 */
int kda_pages_copy(void* const* pools, const int64_t* page_strides, const int64_t* page_bytes, int32_t n_pools,
                   int32_t n_pages, const int32_t* pairs, int64_t n_pairs, void* hip_stream);

/*
 * kda_beam_select — one step of beam search for B groups of K beams: the n_out
 * best continuations of each group over its beams and the vocabulary,
 *   c[k, v] = scores[k] + x[k, v] - log sum_u exp(x[k, u])
 *   logits     beam r = b * K + k at r * row_stride elements: [V] dtype.  NaN
 *              counts as -inf.
 *   scores     [B, K] float, the beams' sums of log-probabilities so far (-inf: a
 *              beam that does not take part yet)
 *   finished   uint8 [B, K] or NULL.  A beam with finished != 0 goes on with token
 *              `eos` alone, at its own score; its logits are not used.
 *   scores_out, parents, tokens  [B, n_out] float, int32, int32: the chosen c in
 *              descending order, the beam k it continues (0 .. K-1) and its token
 *   finished_out  uint8 [B, n_out], with finished only: the parent was finished, or
 *              the token is `eos`
 * Order: within a beam by logit, ties to the lower token; over the beams by c
 * (computed in fp64 from the logit and the beam's log-sum, a running fp32 sum:
 * beams whose c differ by less than its rounding, about 1e-7, may change places),
 * ties to the lower beam.  A c that is NaN counts as -inf; continuations of -inf fill the places
 * that no other one takes.
 * 1 <= K, n_out <= 64, n_out <= K * V, V < 2^24; eos in [0, V) with finished.
 * workspace: kda_beam_select_workspace bytes, 256-byte aligned.
 */
int kda_beam_select(const void* logits, int64_t row_stride, const float* scores, const uint8_t* finished, int32_t B,
                    int32_t K, int32_t V, int32_t n_out, int32_t eos, int32_t dtype, float* scores_out,
                    int32_t* parents, int32_t* tokens, uint8_t* finished_out, void* workspace, size_t workspace_bytes,
                    void* hip_stream);

/* Workspace bytes of kda_beam_select; (size_t)-1 for an invalid combination. */
size_t kda_beam_select_workspace(int32_t B, int32_t K, int32_t V, int32_t n_out);

/*
 * kda_beam_reorder — reorders fixed-size states to the beams they continue, in
 * place: row b * K + k of every state becomes what row b * K + parents[b, k] was.
 * Rows whose parent is their own index are neither read nor written for
 * themselves; a parent outside [0, K) leaves its row as it is.
 *   states, row_bytes  HOST arrays of n_states entries: the device address of
 *            [B * K] contiguous rows and the bytes of a row (multiples of 16,
 *            below 4 GiB).  Read before the call returns.
 *   parents  DEVICE int32 [B, K]; 1 <= K <= 64
 */
int kda_beam_reorder(void* const* states, const int64_t* row_bytes, int32_t n_states, const int32_t* parents,
                     int32_t B, int32_t K, void* hip_stream);

/*
 * Prompt chunks: rotary positions
 * ==========================================================================
 *
 * A chunk of new tokens (a prompt's segment, a chat turn, drafted tokens) goes
 * through an attention layer as rotated queries and keys.  Pair i < rotary_dim / 2
 * of a token at position p is turned by the angle a = p * freqs[i]:
 *     (x, y) -> amplitude * (x cos a - y sin a, x sin a + y cos a)
 *   layout KDA_ROTARY_HALVES       x, y are channels i and i + rotary_dim / 2
 *          KDA_ROTARY_INTERLEAVED  x, y are channels 2 i and 2 i + 1
 * Channels from rotary_dim on are copied as they are.
 *   freqs      DEVICE double [rotary_dim / 2], radians per token, 8-byte aligned: any
 *              base and any scaling for long contexts is a choice of them (and of
 *              amplitude)
 * The angle is an fp64 product reduced by multiples of 2 pi in fp64, its cosine and
 * sine and the rotation are fp32, and the result is rounded once to dtype.
 */
typedef enum { KDA_ROTARY_HALVES = 0, KDA_ROTARY_INTERLEAVED = 1 } kda_rotary_layout;

/*
 * kda_rotary — rotates queries and keys.
 *   q, k        token t at t * q_stride (k_stride) elements: [H_q, d], [H_k, d]
 *               dtype, contiguous; 16-byte aligned, strides too.  k and k_out are
 *               NULL with H_k = 0.
 *   positions   int32 [T], any value
 *   inverse     1: turn by -a, which (amplitude included) is the transpose of the
 *               rotation: applied to the gradients of q_out and k_out it gives those
 *               of q and k
 *   q_out, k_out  laid out as q and k; each is its input itself (same address and
 *               stride, in place) or does not overlap it.  No other overlap.
 * d: a multiple of 8 up to 512; rotary_dim even, 2 .. d; H_q <= 16384, H_k <= 1024.
 */
int kda_rotary(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const int32_t* positions,
               const double* freqs, int64_t T, int32_t H_q, int32_t H_k, int32_t d, int32_t rotary_dim,
               int32_t layout, float amplitude, int32_t inverse, int32_t dtype, void* q_out, int64_t q_out_stride,
               void* k_out, int64_t k_out_stride, void* hip_stream);

/*
 * kda_rotary_append — kda_rotary and kda_cache_append in one launch, with the same
 * results: token i of sequence n is at position start[n] + i; its rotated queries go
 * to q_out, its rotated keys and its values into the pages.
 *   q, k, v     token t at t * stride elements: [H_q, d], [H_kv, d], [H_kv, d]
 *   cu_seqlens, start, pages, table: as in kda_cache_append.  A position without a
 *               page is dropped (q_out is written); rows of q_out that belong to no
 *               sequence are left as they were.
 *   q_out       as in kda_rotary (may be q itself); overlaps neither pages nor k, v
 * d in {64, 128, 256}; the rest as in kda_rotary.
 */
int kda_rotary_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                      int64_t v_stride, const int32_t* cu_seqlens, const int32_t* start, int32_t N, int64_t T_total,
                      const double* freqs, int32_t rotary_dim, int32_t layout, float amplitude, void* q_out,
                      int64_t q_out_stride, void* k_pages, void* v_pages, int64_t k_page_stride,
                      int64_t v_page_stride, int32_t n_pages, int32_t page_size, const int32_t* page_table,
                      int64_t table_stride, int32_t table_pages, int32_t H_q, int32_t H_kv, int32_t d, int32_t dtype,
                      void* hip_stream);

/*
 * Prompt chunks: attention over pages
 * ==========================================================================
 *
 * kda_paged_prefill — softmax attention of the new tokens of every sequence (packed segments, any number of each)
 * over its pages, in which their own keys and values are already (kda_cache_append, kda_rotary_append):
 *   s_t = scale * q . k_t,   out = sum_t softmax(s)_t v_t,   lse = log sum_t exp(s_t)
 * The query of token i of sequence n, which has m = cu[n+1] - cu[n] new tokens, is at position
 * p = lengths[n] - m + i and sees the tokens t <= p of its sequence (none for p < 0).
 *   q          token r at r * q_stride elements: [H_q, d] dtype, contiguous; 16-byte
 *              aligned, stride too.  Heads as in kda_paged_decode.
 *   cu_seqlens DEVICE int32 [N + 1] as in kda_append_prefill
 *   lengths    int32 [N], tokens of each sequence, the new ones among them
 *   window     0, or of those only t > p - window ...
 *   sinks      ... and t < sinks (0 without a window)
 *   max_length an upper bound of lengths that sizes the launch; 0: table_pages * page_size (below 2^31 - 4096).
 *              Tokens behind it are not visible.
 *   out        [T_total, H_q, d] dtype, contiguous (unlike kda_paged_decode's: a prompt's rows go into a
 *              projection of their type next); lse [T_total, H_q] float or NULL.  16-byte aligned.  Rows that belong
 *              to no sequence are left as they were.
 * A query without a visible token (or whose every visible score is -inf) gives out = 0 and lse = -inf.  Tokens that a
 * query does not see never change its result, whatever bits their slots hold; a visible key or value that is not finite
 * makes what it enters not finite, but for a key with a score of -inf, which has weight 0.  Products are exact in
 * bf16 with fp32 sums.  With KDA_BF16 and T_total * H_q / H_kv > 32 N (many new tokens) the softmax weights are rounded
 * to bf16 for their product with the values (their sum is not), which adds to the output's own rounding about as much
 * again; with fewer they are two bf16 each.  This goes by the batch: a single token or a draft has two alone or with
 * others of its kind, and one next to a prompt that brings the average above 32.
 * workspace: kda_paged_prefill_workspace bytes for the same arguments, 256-byte aligned, overlapping no argument; holds
 * the partial results where the keys of some rows are split over several workgroups.  Needs no initialisation.  How they
 * are split goes by the lengths of all sequences, so that a sequence's last bits may depend on the others' lengths.
 * T_total * H_q / 32 + N * H_kv is below 2^24.
 * d in {64, 128, 256}; lengths and cu_seqlens are a caller contract (checked with KDA_DEBUG_CHECK=1).
 */
int kda_paged_prefill(const void* q, int64_t q_stride, const void* k_pages, const void* v_pages, int64_t k_page_stride,
                      int64_t v_page_stride, int32_t n_pages, int32_t page_size, const int32_t* page_table,
                      int64_t table_stride, int32_t table_pages, const int32_t* lengths, const int32_t* cu_seqlens,
                      int32_t N, int64_t T_total, int32_t H_q, int32_t H_kv, int32_t d, int32_t dtype, float scale,
                      int32_t window, int32_t sinks, int64_t max_length, void* out, float* lse, void* workspace,
                      size_t workspace_bytes, void* hip_stream);

/* Workspace bytes of kda_paged_prefill for a bound of max_length (or a table of as many tokens, if that is less); 0, no
 * bound: enough for a table of any width.  (size_t)-1 for an unsupported or invalid combination. */
size_t kda_paged_prefill_workspace(int32_t N, int64_t T_total, int32_t H_q, int32_t H_kv, int32_t d, int32_t dtype,
                                   int64_t max_length, int32_t window, int32_t sinks);

/*
 * Prompt chunks: log-probabilities of given tokens
 * ==========================================================================
 *
 * kda_token_logprobs — for every row x of logits (a prompt's tokens, drafted tokens, a training batch):
 *     lse = log sum_u exp(x_u),   logprob = x_token - lse,
 *     entropy = -sum_u p_u log p_u with p_u = exp(x_u - lse),
 *     and the `top` largest x - lse with their tokens, in descending order, ties to the lower token.
 *   logits     row r at r * row_stride elements: [V] dtype.  NaN counts as -inf.
 *   tokens     int32 [R], with logprobs (NULL without).  A token outside [0, V) is
 *              ignored: its logprob is 0.
 *   logprobs, lse, entropy   float [R], each may be NULL
 *   top_logprobs, top_tokens float, int32 [R, top]; NULL with top = 0
 * A row whose log-sum is not finite (all -inf, or a logit of +inf) has entropy 0, and a log-probability that is NaN
 * there counts as -inf.
 * V < 2^24, 0 <= top <= 64, top <= V, R < 2^24 (a workgroup is counted for every row, also where four share one).
 * workspace: kda_token_logprobs_workspace bytes, 256-byte aligned, overlapping no argument; needs no
 * initialisation.
 */
int kda_token_logprobs(const void* logits, int64_t row_stride, const int32_t* tokens, int64_t R, int32_t V,
                       int32_t top, int32_t dtype, float* logprobs, float* lse, float* entropy, float* top_logprobs,
                       int32_t* top_tokens, void* workspace, size_t workspace_bytes, void* hip_stream);

/* Workspace bytes of kda_token_logprobs; (size_t)-1 for an invalid combination. */
size_t kda_token_logprobs_workspace(int64_t R, int32_t V, int32_t top);

/*
 * kda_token_logprobs_grad — the gradient of kda_token_logprobs with respect to the logits:
 *     d_logits_v = p_v (d_lse - d_logprob - d_entropy (log p_v + entropy)) + d_logprob [v = token]
 *   logits, tokens   as given to kda_token_logprobs; lse, entropy float [R]: its results
 *   d_logprobs (with tokens), d_lse, d_entropy (with entropy)   float [R], each may be NULL (zero)
 *   d_logits   row r at r * out_stride elements: [V] dtype; may be logits itself (same address and stride),
 *              no other overlap
 * An ignored token's d_logprob counts as 0.  Where p_v is 0 (logits of -inf or NaN) it contributes nothing; rows whose
 * lse is not finite have gradient 0.  Computed in fp32, rounded once to dtype.
 */
int kda_token_logprobs_grad(const void* logits, int64_t row_stride, const int32_t* tokens, const float* lse,
                            const float* entropy, const float* d_logprobs, const float* d_lse, const float* d_entropy,
                            int64_t R, int32_t V, int32_t dtype, void* d_logits, int64_t out_stride,
                            void* hip_stream);

/* Host-side validator (as those above) of a page table and lengths, HOST arrays:
 * 0 <= lengths[n] <= min(max_length, table_pages * page_size) and entries that
 * are -1 or in [0, n_pages). */
int kda_validate_page_table(const int32_t* page_table, int64_t table_stride, const int32_t* lengths, int32_t N,
                            int32_t table_pages, int32_t page_size, int32_t n_pages, int64_t max_length);

/* Workspace bytes an op needs (B_or_N sequences, T tokens per sequence for
 * KDA_OP_PREFILL or T_total for KDA_OP_APPEND and KDA_OP_BACKWARD).  0 for
 * KDA_OP_DECODE.
 * Returns (size_t)-1 for an unsupported or invalid combination. */
size_t kda_workspace_size(int32_t op, int64_t B_or_N, int64_t T, int32_t H, int32_t d_k, int32_t d_v,
                          int32_t dtype, int32_t chunk);

/* 1 if (op, dtype, d_k, d_v, chunk) is implemented, else 0. */
int kda_is_supported(int32_t op, int32_t dtype, int32_t d_k, int32_t d_v, int32_t chunk);

/* Static description of a kda_status value. */
const char* kda_status_string(int status);

/* Message describing the last failed call on the calling thread ("" if none). */
const char* kda_last_error(void);

/* Library version string. */
const char* kda_version(void);

/*
 * Diagnostics: per-kernel timing with HIP events (the library's own tracing).
 * kda_timing_begin() starts recording, for calls made on the calling thread,
 * a HIP event immediately before and after every kernel the library launches,
 * on that call's stream.  kda_timing_end() stops recording, waits for the
 * recorded events, and writes up to max_records (kernel id, milliseconds)
 * pairs in launch order into kernel_ids / ms (either may be NULL to only
 * count).  Returns the number of kernels recorded, or a negative kda_status
 * (KDA_ERR_HIP if an event failed).  Event objects are created on first use and
 * reused; no device memory is allocated.  Kernel ids are kda_kernel values.
 */
typedef enum {
    KDA_KERNEL_PREP = 1,      /* chunk-parallel prep of the matrix-core prefill */
    KDA_KERNEL_STATE = 2,     /* sequential state pass of the matrix-core prefill */
    KDA_KERNEL_CHUNK_F32 = 3, /* fp32 chunked prefill */
    KDA_KERNEL_DECODE = 4,    /* decode step */
    KDA_KERNEL_BWD_FACTORS = 5,    /* backward: per-chunk factors */
    KDA_KERNEL_BWD_FWD_CHAIN = 6,  /* backward: states entering each chunk */
    KDA_KERNEL_BWD_REV_CHAIN = 7,  /* backward: state gradients, chunks in reverse */
    KDA_KERNEL_BWD_GRAD_STATE = 8, /* backward: products over the value axis */
    KDA_KERNEL_BWD_GRAD_CHUNK = 9, /* backward: in-chunk gradients */
    KDA_KERNEL_CACHE_APPEND = 10,  /* keys and values written into pages */
    KDA_KERNEL_PAGED_DECODE = 11,  /* attention over pages */
    KDA_KERNEL_PAGED_JOIN = 12,    /* attention over pages: join of the split parts */
    KDA_KERNEL_CACHE_FORK = 13,    /* tables of branched sequences */
    KDA_KERNEL_CACHE_FREE = 14,    /* sequences dropped */
    KDA_KERNEL_CACHE_SCAN = 15,    /* reserve, compact: counts of free or used pages */
    KDA_KERNEL_CACHE_RESERVE = 16, /* reserve: pages handed out */
    KDA_KERNEL_CACHE_PLAN = 17,    /* compact: moves */
    KDA_KERNEL_CACHE_REMAP = 18,   /* compact: tables and counts */
    KDA_KERNEL_PAGES_COPY = 19,    /* pages copied */
    KDA_KERNEL_BEAM_SCAN = 20,     /* beam search: best logits and log-sum of a part of a row */
    KDA_KERNEL_BEAM_JOIN = 21,     /* beam search: choice over the beams */
    KDA_KERNEL_BEAM_REORDER = 22,  /* states reordered */
    KDA_KERNEL_ROTARY = 23,        /* queries and keys rotated (and put into pages) */
    KDA_KERNEL_LOGPROB_SCAN = 24,  /* token log-probabilities: a row or a part of one */
    KDA_KERNEL_LOGPROB_JOIN = 25,  /* token log-probabilities: join of the split rows */
    KDA_KERNEL_LOGPROB_GRAD = 26,  /* gradient of token log-probabilities */
    KDA_KERNEL_PAGED_PREFILL = 27, /* attention of a chunk over pages */
    KDA_KERNEL_PREFILL_JOIN = 28   /* attention of a chunk over pages: join of the split parts */
} kda_kernel;

int kda_timing_begin(void);
int kda_timing_end(int32_t* kernel_ids, float* ms, int32_t max_records);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */

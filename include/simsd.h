/*
 * simsd.h -- C ABI of libsimsd.so: the SimSD speculative-verification step
 * for diffusion language models on one NVIDIA GB300 (sm_103a).
 *
 * Method: "SimSD: Simple Speculative Decoding in Diffusion Language Models"
 * (gist.science technical summaries of paper 2606.02544):
 *   section 1 "Input Layout"            -- prompt | D (B reference tokens) |
 *                                          D~ (B [MASK] prediction slots);
 *   section 2 "Temporal Attention Mask" -- step map tau, mask A_ij;
 *   section 3 "Position Encoding Alignment" -- D~_k reuses D_k's RoPE index;
 *   section 4 "Speculative Decoding Pipeline" -- one verification forward,
 *                                          rejection sampling along tau.
 *
 * Conventions shared by every call
 *   - Plain C types only.  "device" pointers are CUDA device memory of the
 *     current device; "host" pointers are ordinary host memory.
 *   - All memory is owned by the caller.  The device calls never allocate:
 *     scratch lives in a caller-provided workspace whose size the matching
 *     *_workspace_size function returns (256-byte aligned pointer required).
 *   - Device calls are asynchronous and stream-ordered on `stream` (a
 *     cudaStream_t; NULL is the legacy default stream).  They never
 *     synchronise the host.
 *   - Argument errors are detected on the host and returned before anything
 *     is launched.  A launch failure returns SIMSD_ERR_CUDA.  Kernels never
 *     trap: a bounded wait that runs out, or device arrays that disagree
 *     with the limits, set a bit in the workspace's status word (its first
 *     4 bytes).  The bits stay set across calls until simsd_read_status()
 *     reads and clears them (no call clears it on the hot path), so a new
 *     workspace must start zero-filled (or be passed to simsd_read_status
 *     once).
 *   - Token order inside a sequence with section length B is
 *     D_1..D_B, D~_1..D~_B (2B tokens); sequences are back to back, so
 *     sequence b's tokens start at row 2*cu_B[b].
 *   - Limits: head_dim in {64, 128}; num_q_heads % num_kv_heads == 0;
 *     1 <= B_b <= 32; page_size == 16; batch >= 1; one new token's raw
 *     q, k and v rows together at most 196,608 bytes
 *     ((num_q_heads + 2 num_kv_heads) * head_dim * element size).
 *   - Every device array of q, k, v, cache or output values starts on a
 *     16-byte boundary (SIMSD_ERR_ALIGN otherwise); logits may be unaligned
 *     (slower element-wise loads).
 *   - The library is stateless and re-entrant.  Calls on different streams
 *     must not share a workspace or write the same cache pages.
 */
#ifndef SIMSD_H
#define SIMSD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SIMSD_OK = 0,
  SIMSD_ERR_NULL = 1,      /* a required pointer is NULL                    */
  SIMSD_ERR_SHAPE = 2,     /* a size is out of range or inconsistent        */
  SIMSD_ERR_TAU = 3,       /* tau is not a permutation of 1..B              */
  SIMSD_ERR_DTYPE = 4,     /* unsupported dtype                             */
  SIMSD_ERR_WORKSPACE = 5, /* workspace missing, misaligned or too small    */
  SIMSD_ERR_CUDA = 6,      /* a CUDA runtime call or launch failed          */
  SIMSD_ERR_TIMEOUT = 7,   /* a device-side bounded wait ran out            */
  SIMSD_ERR_ALIGN = 8      /* a device array is not 16-byte aligned         */
} simsd_status;

typedef enum {
  SIMSD_F32 = 0,
  SIMSD_BF16 = 1,
  SIMSD_E4M3 = 2           /* simsd_kv4_read's rows only                      */
} simsd_dtype;

/* Static text for a status code; never NULL. */
const char *simsd_status_string(int status);

/* Library version as major*10000 + minor*100 + patch. */
int simsd_version(void);

/* ------------------------------------------------------------------------
 * simsd_layout -- host only.  Sections 1-3: paired layout, positions, mask.
 *   prompt_len  P >= 0
 *   B           1..32 (section length; also the draft length gamma)
 *   tau         host int32[B], tau[k] = step label of response position k+1
 *   positions   host int32[P+2B] out: prompt j -> j; D_k -> P+k-1;
 *               D~_k -> P+k-1 (copied RoPE index)
 *   mask        host uint8[2B][P+2B] out, may be NULL.  Row r < B is D_{r+1},
 *               row B+i is D~_{i+1}; column c < P is prompt token c, then D,
 *               then D~.  1 = may attend.  Slot rows: whole prompt, D_j with
 *               tau(j) < tau(i), D~_j with tau(j) >= tau(i).  Data rows (a
 *               convention: their outputs feed later layers, their logits
 *               are not consumed): prompt and D_j with tau(j) <= tau(i).
 * Errors: SIMSD_ERR_NULL, SIMSD_ERR_SHAPE, SIMSD_ERR_TAU.
 * ---------------------------------------------------------------------- */
simsd_status simsd_layout(int32_t prompt_len, int32_t B, const int32_t *tau,
                          int32_t *positions, uint8_t *mask);

/* ------------------------------------------------------------------------
 * simsd_verify_attn -- sections 2-4: one attention layer of the verification
 * forward over [prompt KV cache | D | D~] for a batch of sequences.
 *
 * Kernel sequence on `stream`:
 *   K1  rotate q (all query heads) and k_new at the layout positions (D~_k
 *       uses D_k's), write rotated k and raw v of the 2B new tokens into
 *       cache slots [lens[b], lens[b]+2B_b) of sequence b;
 *   K2  attention of all 2B_b x Hq query rows of a sequence and KV head
 *       against the cache, the temporal mask evaluated on the fly; a
 *       (sequence, KV head) unit runs whole or in key splits (every unit
 *       when the block-table width makes one unit long, or only the units
 *       of the last partial wave of CTAs, so that wave takes a split's
 *       time instead of a unit's);
 *   K3  merge of the split units' partial softmax states (launched only
 *       when some unit is split).
 * lens[] is NOT advanced: rolling back a rejected draft costs nothing, and
 * committing accepted tokens is the caller's business.
 *
 * Layouts (row-major, innermost last):
 *   q            device [T][Hq][hd]   raw queries, T = 2 * total_B
 *   k_new, v_new device [T][Hkv][hd]  raw keys / values of the new tokens
 *   k_cache, v_cache device [num_pages][Hkv][page_size][hd]; prompt slots
 *                hold keys already rotated at their own positions
 *   block_table  device int32[batch][max_pages_per_seq]; entries
 *                0 .. ceil((lens[b]+2B_b)/16)-1 of row b must be valid page
 *                ids < num_pages (the rest are never read)
 *   tau          device int32[total_B]; sequence b's labels at cu_B[b]..
 *   lens         device int32[batch]   prompt KV length P_b >= 0
 *   cu_B         device int32[batch+1] prefix sums of B_b (cu_B[0] = 0)
 *   out          device [T][Hq][hd]    attention output of every new row
 * dtype applies to q, k/v (new and cache) and out.
 * Host-side fields (total_B, B_max, max_pages_per_seq) must agree with the
 * device arrays.  A sequence whose device arrays disagree with them (cu_B
 * not within 0..total_B, B_b outside 1..B_max, lens[b]+2B_b beyond the
 * table row, a page id outside the cache) sets the status word's bad-input
 * bit (2) and is skipped: nothing is read or written out of range for it.
 * tau is trusted: a wrong tau gives a wrong mask, never an out-of-bounds
 * access.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t batch;
  int32_t num_q_heads;        /* Hq                                         */
  int32_t num_kv_heads;       /* Hkv                                        */
  int32_t head_dim;           /* hd: 64 or 128                              */
  int32_t page_size;          /* 16                                         */
  int32_t num_pages;          /* pages in each cache array                  */
  int32_t max_pages_per_seq;  /* row stride of block_table                  */
  int32_t total_B;            /* sum_b B_b (host copy)                      */
  int32_t B_max;              /* max_b B_b (host copy), 1..32               */
  simsd_dtype dtype;
  float rope_base;            /* RoPE base (e.g. 1e6)                       */
  float sm_scale;             /* score = sm_scale * q.k; finite, > 0        */
  const void *q;
  void *k_cache;
  void *v_cache;
  const int32_t *block_table;
  const void *k_new;
  const void *v_new;
  const int32_t *tau;
  const int32_t *lens;
  const int32_t *cu_B;
  void *out;
  void *workspace;            /* device, 256-byte aligned                   */
  size_t workspace_bytes;
  int32_t wait_polls;         /* polls a kernel's bounded wait makes before
                                 it gives up: 0 (a zero-filled descriptor)
                                 selects the default 2^24; a negative value
                                 gives up at once, which runs the timeout
                                 path (status bit 0, nothing written to the
                                 cache; out undefined) -- for tests        */
  int32_t node_size;          /* 0: SimSD's paired layout under the temporal
                                 mask (above).  > 0: Spiffy's draft-graph
                                 verification: a sequence's 2B_b new tokens
                                 are 2B_b / node_size candidate states of the
                                 block (nodes of node_size <= 32 tokens, node
                                 after node); token k of every node sits at
                                 position lens[b] + k; a row attends to the
                                 whole prompt and to every token of its own
                                 node, nothing of another node; tau is not
                                 read (may be NULL).  A sequence whose 2B_b
                                 is not a multiple of node_size sets the
                                 bad-input bit and is skipped                */
} simsd_verify_desc;

/* Bytes of workspace simsd_verify_attn needs for these sizes (reads only
 * the host-side fields).  Returns 0 if the sizes are invalid.  The size
 * follows the key-split plan, which depends on the current device's SM
 * count (152 when no device is visible): query it with the device that
 * will run the call current. */
size_t simsd_verify_workspace_size(const simsd_verify_desc *d);
simsd_status simsd_verify_attn(const simsd_verify_desc *d, void *stream);

/* Same as simsd_verify_attn, and records caller-created CUDA events (each a
 * cudaEvent_t, or NULL to skip) on `stream` at the kernel boundaries:
 * events[0] before K1, [1] after K1, [2] after K2, [3] after K3 (recorded
 * even when K3 is not needed).  For per-kernel timing; the events are not
 * waited on or destroyed. */
simsd_status simsd_verify_attn_timed(const simsd_verify_desc *d, void *stream,
                                     void *const events[4]);

/* ------------------------------------------------------------------------
 * simsd_prompt_append -- K1 on plain positions: rotate n_b raw keys of
 * sequence b at positions start[b] .. start[b]+n_b-1 and write them (and
 * the raw values) into the same cache slots.  Fills a prompt's cache, or
 * commits tokens after acceptance.
 *   k, v     device [sum n_b][Hkv][hd]   raw keys / values
 *   start    device int32[batch]         first slot (= position) per seq
 *   cu_n     device int32[batch+1]       prefix sums of n_b
 *   total_n  host: sum n_b
 *   block_table as above; every slot written must be covered.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t batch;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t page_size;
  int32_t num_pages;
  int32_t max_pages_per_seq;
  int32_t total_n;
  simsd_dtype dtype;
  float rope_base;
  const void *k;
  const void *v;
  const int32_t *start;
  const int32_t *cu_n;
  void *k_cache;
  void *v_cache;
  const int32_t *block_table;
} simsd_append_desc;

simsd_status simsd_prompt_append(const simsd_append_desc *d, void *stream);

/* ------------------------------------------------------------------------
 * simsd_accept -- section 4, acceptance: standard rejection sampling along
 * the temporal order tau.  For sequence b and steps t = 1..B_b, slot
 * k = tau^-1(t) with draft token x = draft_tokens[k]:
 *   p = softmax(target row k / T), q = softmax(draft row k / T) (fp32
 *   math; T = temperature, 1 by default);
 *   accept iff u[t-1] * q(x) < p(x);
 *   at the first rejection draw a token from max(0, p - q) normalised (p
 *   itself if that is empty) by inverse CDF with u[B_b], and stop.
 * Variant rule SIMSD_ACCEPT_GREEDY (the temperature -> 0 limit): step t
 * accepts iff x is the target row's argmax (the smallest index among equal
 * maxima); the first rejection emits that argmax.  It reads neither the
 * draft logits nor the uniforms (they may be NULL).
 * Variant rule SIMSD_ACCEPT_MATCH (sample matching, Spiffy's verification):
 * step t draws the target's own token y from p (at temperature T) by
 * inverse CDF with u[t-1] and accepts iff y = x; the first rejection emits
 * y (u[B_b] unused, draft logits not read and may be NULL).
 * Kernels: K4a, a chunk pass over (row, 32 KB chunk) items on every SM
 * (for the sampling rule's small batches a pass that loads each part
 * directly, a warp per part), writes per eighth of a chunk (a "part") its
 * maximum and sum of
 * exponentials -- of both rows of every slot for the sampling rule; of the
 * target rows and the mass below the draft token for sample matching; the
 * largest value and its index for the greedy rule -- and the logits at the
 * draft tokens, to the workspace.  K4b: sampling, up to two CTAs per SM
 * over the batch, each owning a range of a sequence's chunks: every CTA of
 * a sequence merges its slots' parts and walks the steps alike, computes
 * the residual masses of its chunks of the rejected slot's two rows, and
 * the last CTA of the sequence draws from them; greedy and matching, one
 * CTA per sequence merging each slot's parts (matching: a slot that
 * rejects draws its token from the part holding u S) and walking the
 * steps.  With a workspace smaller than simsd_accept_workspace_size, or
 * with `decided` (the blockwise loop: decided slots' rows are not read),
 * each rule's thread-block cluster kernel (C <= 16 CTAs per sequence, each
 * owning 1/C of the vocabulary) streams the rows itself in one launch.
 *   target_logits, draft_logits device [total_B][vocab] (dtype); row k of
 *                sequence b (at cu_B[b]+k) holds the logits read at D~_k
 *   draft_tokens device int32[total_B] in [0, vocab); a token outside
 *                sets the status word's bad-input bit and its step rejects
 * A sequence whose cu_B entries fall outside 0..total_B, whose B_b is
 * outside 1..B_max, or whose tau is not a permutation of 1..B_b sets the
 * bad-input bit and gets n_accept = 0, token = -1, pos = -1 without reading
 * its logits.  Logits must not be NaN (-inf is allowed; the greedy rule
 * gives index 0 for a row with no larger entry).
 *   tau, cu_B    device, as for simsd_verify_attn
 *   uniforms     device float32[batch][B_max+1], values in [0, 1)
 *   n_accept     device int32[batch] out: accepted prefix length (0..B_b)
 *   token        device int32[batch] out: token drawn at the rejection,
 *                -1 when every step was accepted (no bonus token: the
 *                layout has no slot after D~_B)
 *   pos          device int32[batch] out: response position (0-based k) of
 *                the rejected slot, -1 when none
 * Limits: 1 <= vocab <= 2^21; batch <= 65535.  Rows whose byte length is
 * a multiple of 16 (and 16-byte aligned logits) are streamed by bulk
 * copies; other vocabularies take a slower element-wise copy.
 * Workspace: simsd_accept_workspace_size returns the size of the
 * two-kernel path, with C = ceil(vocab / E) chunks of E = 16384 entries
 * (bf16) or 8192 (fp32) and each term rounded up to a multiple of 256:
 * sampling, 256 + 2 total_B C * 64 + 2 total_B * 4 + batch * 4 +
 * batch C * 256 bytes; greedy and matching, 256 + total_B C * 128 +
 * total_B * 4.  Any workspace of at least 256 bytes is accepted; one smaller
 * than that size runs the single-launch path.  A wait of the chunk pass
 * that gives up leaves every sequence of the call with n_accept = 0,
 * token = -1, pos = -1 (and the timeout bit set).
 * Errors: SIMSD_ERR_NULL, SIMSD_ERR_SHAPE (also: an unknown rule, or a
 * temperature that is negative or not finite), SIMSD_ERR_DTYPE,
 * SIMSD_ERR_WORKSPACE, SIMSD_ERR_CUDA.
 * ---------------------------------------------------------------------- */
typedef enum {
  SIMSD_ACCEPT_SAMPLE = 0,    /* rejection sampling at temperature T         */
  SIMSD_ACCEPT_GREEDY = 1,    /* accept iff x = argmax of the target row      */
  SIMSD_ACCEPT_MATCH = 2      /* accept iff x = the target's own sample       */
} simsd_accept_rule;

typedef struct {
  int32_t batch;
  int32_t vocab;
  int32_t total_B;            /* host copy                                  */
  int32_t B_max;              /* host copy, 1..32                           */
  simsd_dtype dtype;          /* of the logits                              */
  const void *target_logits;
  const void *draft_logits;
  const int32_t *draft_tokens;
  const int32_t *tau;
  const int32_t *cu_B;
  const float *uniforms;
  int32_t *n_accept;
  int32_t *token;
  int32_t *pos;
  void *workspace;            /* device, 256-byte aligned                   */
  size_t workspace_bytes;
  simsd_accept_rule rule;     /* 0 (a zero-filled descriptor): sampling      */
  float temperature;          /* > 0; 0 selects 1 (a zero-filled descriptor
                                 keeps the standard rule); the logits are
                                 divided by this float's exact value         */
  int32_t wait_polls;         /* as in simsd_verify_desc; a sequence whose
                                 wait gave up gets n_accept = 0, token = -1,
                                 pos = -1 (the sampling rule's chunk pass for
                                 small batches and the finishing kernels have
                                 no waits)                                   */
  const int32_t *decided;     /* device int32[batch] or NULL (all 0): steps
                                 1..decided[b] belong to positions decided
                                 in earlier passes of the block (the
                                 blockwise loop, simsd_commit); the walk
                                 starts at step decided[b]+1 and counts the
                                 earlier ones as accepted (0..B_b; B_b: no
                                 step is tested, n_accept = B_b)             */
} simsd_accept_desc;

size_t simsd_accept_workspace_size(const simsd_accept_desc *d);
simsd_status simsd_accept(const simsd_accept_desc *d, void *stream);

/* Same as simsd_accept, recording events (cudaEvent_t or NULL) on `stream`:
 * events[0] before K4, [1] after K4a (the chunk pass; recorded right after
 * [0] on the single-launch path), [2] after K4b. */
simsd_status simsd_accept_timed(const simsd_accept_desc *d, void *stream,
                                void *const events[3]);

/* ------------------------------------------------------------------------
 * simsd_draft_step -- section 4, drafting: the draft proposes the section's
 * tokens and their temporal order.  For each open slot k of sequence b
 * (every slot when decided is NULL; else those with tau_prev[k] >
 * decided[b]): q = softmax(draft row k / T); the token is the smallest v
 * whose running mass exceeds u[k] (inverse CDF; the last v with q > 0 if
 * rounding leaves none); the open slots take the step labels
 * decided[b]+1 .. B_b in order of the row's largest probability, max_v q(v)
 * (most confident first, equal ones in position order).  The order depends
 * on the draft rows only, not on the drawn tokens, which keeps the walk's
 * rejection sampling exact.  Decided slots keep their token and label.
 *   draft_logits device [total_B][vocab] (dtype)
 *   uniforms     device float32[batch][B_max], values in [0, 1): u[k]
 *                draws slot k
 *   decided      device int32[batch] or NULL
 *   tau_prev     device int32[total_B], read when decided is not NULL: the
 *                block's labels so far (decided slots: 1..decided[b])
 *   tokens       device int32[total_B] in/out: decided slots are kept,
 *                open slots get their drawn token
 *   tau          device int32[total_B] out (may be tau_prev itself)
 *   confidence   device float32[total_B] out or NULL: max_v q(v) of open
 *                slots, -1 at decided ones
 * Kernels: with a workspace of simsd_draft_workspace_size bytes and no
 * decided slots, a chunk pass over (row, 32 KB chunk) items on every SM
 * (per eighth of a chunk: maximum, sum of exponentials, largest logit),
 * then one CTA per sequence: a warp per slot merges its row's parts, finds
 * the part holding u*S and scans it; a wait of the chunk pass that gives
 * up sets the timeout bit and leaves every tokens and tau entry of the
 * call unwritten.  Otherwise one thread-block cluster per sequence (as
 * simsd_accept's rules): one pass over every open row for its normaliser,
 * then each slot's inverse-CDF scan in the vocabulary slice holding u*S.
 * Errors: as simsd_accept (SIMSD_ERR_SHAPE also for a negative or
 * non-finite temperature).  Bad device arrays (cu_B, decided outside
 * 0..B_b, tau_prev not a permutation) set the bad-input bit and leave the
 * sequence's tokens and tau unwritten.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t batch;
  int32_t vocab;
  int32_t total_B;            /* host copy                                  */
  int32_t B_max;              /* host copy, 1..32                           */
  simsd_dtype dtype;          /* of the logits                              */
  float temperature;          /* > 0; 0 selects 1                           */
  const void *draft_logits;
  const int32_t *cu_B;
  const float *uniforms;
  const int32_t *decided;
  const int32_t *tau_prev;
  int32_t *tokens;
  int32_t *tau;
  float *confidence;
  void *workspace;            /* device, 256-byte aligned: the status word,
                                 or simsd_draft_workspace_size bytes (256 +
                                 total_B ceil(vocab / E) * 128 rounded up to
                                 a multiple of 256, E as in simsd_accept)
                                 for the chunked path                      */
  size_t workspace_bytes;
} simsd_draft_desc;

size_t simsd_draft_workspace_size(const simsd_draft_desc *d);
simsd_status simsd_draft_step(const simsd_draft_desc *d, void *stream);

/* ------------------------------------------------------------------------
 * simsd_commit -- section 4: "the longest accepted prefix is committed, and
 * the process is repeated", with the KV cache and blockwise decoding
 * (section "Contributions").  One pass of the blockwise loop is
 * simsd_draft_step -> simsd_verify_attn -> simsd_accept (decided) ->
 * simsd_commit.  For sequence b, with the walk's n_accept, token, pos:
 *   - positions with tau <= n_accept stay decided with their tokens;
 *   - a rejection (pos >= 0) decides position pos with the drawn token
 *     (written to tokens[pos]); it holds label n_accept + 1, so
 *     decided[b] = n_accept + 1;
 *   - every position decided by a pass that drew nothing (n_accept = B_b,
 *     pos = -1): the cache slots [lens, lens+B_b) written by that pass's
 *     verification hold the final tokens' keys and values, so the block
 *     closes: lens[b] += B_b, decided[b] = 0, done[b] = 1 (the mask-slot
 *     slots past them are free again).  A block whose last position was
 *     decided by a draw stays open with decided[b] = B_b: its next pass
 *     tests nothing, rewrites the section's keys and values from the final
 *     tokens, and closes it.
 *   tau, cu_B, n_accept, token, pos  device, as written by simsd_accept
 *   tokens   device int32[total_B] in/out (the pass's data-section tokens)
 *   decided  device int32[batch] in/out
 *   lens     device int32[batch] in/out
 *   done     device int32[batch] out
 * A sequence whose arrays are inconsistent (cu_B outside 0..total_B, B_b
 * outside 1..B_max, a walk that does not fit its tau) sets the bad-input
 * bit and is left unchanged (done = 0).  One thread per sequence.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t batch;
  int32_t total_B;            /* host copy                                  */
  int32_t B_max;              /* host copy, 1..32                           */
  const int32_t *cu_B;
  const int32_t *tau;
  const int32_t *n_accept;
  const int32_t *token;
  const int32_t *pos;
  int32_t *tokens;
  int32_t *decided;
  int32_t *lens;
  int32_t *done;
  void *workspace;            /* device, 256-byte aligned (status word)     */
  size_t workspace_bytes;
} simsd_commit_desc;

size_t simsd_commit_workspace_size(const simsd_commit_desc *d);
simsd_status simsd_commit(const simsd_commit_desc *d, void *stream);

/* ------------------------------------------------------------------------
 * simsd_accept_noalloc -- simsd_accept for callers that cannot allocate
 * device memory.  (No counterpart in the SimSD paper: it is a deployment
 * convenience.)  Some callers never get to call cudaMalloc: a serving loop
 * that runs the acceptance step under a fixed memory budget and must not
 * allocate per request (an allocation can fail under memory pressure, or
 * stall the device mid-request), or a plugin whose host framework owns all
 * device memory and hands it only the input and output tensors.  This entry
 * point takes the same descriptor, ignores its workspace fields, and keeps
 * its scratch in a static device array of SIMSD_ACCEPT_NOALLOC_SCRATCH_BYTES
 * bytes that every GPU loading the library holds until the process exits.
 *   - It calls no cudaMalloc, cudaFree or allocating library routine.
 *   - It runs the two-kernel path where its chunk partials (which grow
 *     with total_B and vocab) fit the array, and the single-launch path,
 *     whose scratch is one status word for every size, otherwise; a
 *     scratch need beyond the array would be rejected with
 *     SIMSD_ERR_WORKSPACE before any launch.
 *   - The first call on each device looks up the array's device address
 *     (once per device, with that device current); make that first call
 *     before any stream capture.
 *   - Every call shares the one array per device (zero at load time) and it
 *     keeps the previous call's contents.  Calls that
 *     overlap on the GPU -- on different streams, or from several host
 *     threads -- race on it: serialise them.
 *   - The kernels' status word lives in that array, so simsd_read_status
 *     cannot read it; device-detected input errors are not reported here.
 *   - The address is cached per device ordinal for the life of the process:
 *     it assumes the device's primary context (the one the CUDA runtime
 *     uses) and no cudaDeviceReset in between.
 * ---------------------------------------------------------------------- */
#define SIMSD_ACCEPT_NOALLOC_SCRATCH_BYTES ((size_t)4096)
simsd_status simsd_accept_noalloc(const simsd_accept_desc *d, void *stream);

/* ------------------------------------------------------------------------
 * Rotary positions as the calls below take them.  Pair i < rotary_dim / 2 of
 * a head turns by position * w_i, w_i = base^(-2i / rotary_dim) scaled for
 * long contexts; elements from rotary_dim on pass unchanged.
 *   SIMSD_ROPE_LINEAR  w_i / factor
 *   SIMSD_ROPE_NTK     w_i of the base base * factor^(rd / (rd - 2))
 *   SIMSD_ROPE_YARN    w_i (1 - r) + w_i / factor * r, r rising in i from 0
 *                      at floor(i(fast)) to 1 at ceil(i(slow)), where i(n) =
 *                      rd ln(original_len / (2 pi n)) / (2 ln base) is the
 *                      pair that makes n turns over original_len positions
 *                      (the two ends kept within 0..rd-1 and at least 0.001
 *                      apart)
 *   SIMSD_ROPE_BANDED  w_i / factor * (1 - r) + w_i * r, r = (turns - slow)
 *                      / (fast - slow) kept within 0..1, turns =
 *                      original_len w_i / (2 pi)
 * attn_factor multiplies the cosines and sines (so scores grow by its
 * square); 0 selects 0.1 ln(factor) + 1 for YARN and 1 otherwise.
 * Angles are formed to ~3e-7 rad at every position (64 bits from 2^24 on).
 * ---------------------------------------------------------------------- */
typedef enum {
  SIMSD_ROPE_HALF = 0,        /* pairs (i, i + rotary_dim / 2)               */
  SIMSD_ROPE_INTERLEAVED = 1  /* pairs (2i, 2i + 1)                          */
} simsd_rope_style;

typedef enum {
  SIMSD_ROPE_PLAIN = 0,
  SIMSD_ROPE_LINEAR = 1,
  SIMSD_ROPE_NTK = 2,
  SIMSD_ROPE_YARN = 3,
  SIMSD_ROPE_BANDED = 4
} simsd_rope_scaling;

typedef struct {
  float base;                 /* > 1                                        */
  int32_t rotary_dim;         /* even, 2..head_dim; 0 selects head_dim
                                 (NTK: at least 4)                          */
  simsd_rope_style style;
  simsd_rope_scaling scaling;
  float factor;               /* >= 1; not read by PLAIN                    */
  int32_t original_len;       /* >= 1; read by YARN and BANDED              */
  float fast, slow;           /* 0 < slow < fast; read by YARN and BANDED   */
  float attn_factor;          /* >= 0                                       */
} simsd_rope_spec;

/* ------------------------------------------------------------------------
 * simsd_rope -- rotates rows of heads (a pass's queries and its keys in one
 * launch).  inverse = 1 turns by the negative angle: the gradient of the
 * rotation with respect to its input (attn_factor multiplies it as well).
 *   positions  device int32[rows], any value in -2^30..2^30
 *   x0, y0     device, num_heads0 heads of every row in and out; head h of
 *              row r starts at x0 + r * x0_row + h * x0_head (elements; a
 *              head's head_dim elements are contiguous).  y0 may be x0 with
 *              the same strides; other overlaps, and rows or heads of y that
 *              overlap one another, are not allowed
 *   x1, y1     the same for a second tensor; num_heads1 = 0: none
 * Arrays and strides that are multiples of 16 bytes, with rotary_dim a
 * multiple of 32 bytes, move in 16-byte vectors; others element by element
 * (each pointer aligned to its element, SIMSD_ERR_ALIGN otherwise).
 * rows = 0 returns SIMSD_OK (the arrays may be NULL then).  Limits: heads <=
 * 16384 each, rows <= 2^30.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t rows;
  int32_t num_heads0;         /* >= 1                                       */
  int32_t num_heads1;         /* >= 0                                       */
  int32_t head_dim;           /* 64 or 128                                  */
  simsd_dtype dtype;
  int32_t inverse;            /* 0 or 1                                     */
  simsd_rope_spec rope;
  const int32_t *positions;
  const void *x0;
  void *y0;
  const void *x1;
  void *y1;
  int64_t x0_row, x0_head, y0_row, y0_head;
  int64_t x1_row, x1_head, y1_row, y1_head;
} simsd_rope_desc;

simsd_status simsd_rope(const simsd_rope_desc *d, void *stream);

/* ------------------------------------------------------------------------
 * simsd_page_map -- block tables and slot maps from request lengths, on the
 * GPU.  Sequence b shall hold need_b = ceil((lens[b] + n_b) / 16) pages,
 * n_b = cu_n[b+1] - cu_n[b] its tokens about to be written.  Pages come from
 * and go back to a ring of free ones; what a call gives back can be taken
 * from the next call on.
 *   - need_b > held[b]: the row's entries held[b].. take the next free pages,
 *     in the order of the sequences.  A sequence that the pages free at the
 *     call's start do not reach to is not served (served[b] = 0, nothing of
 *     it changes, its slots are -1), and neither is any growing one after it;
 *   - need_b < held[b]: the entries need_b.. go to the ring's end, in the
 *     order of the sequences (a finished request: lens = n = 0);
 *   - slots[t] = page * 16 + offset of token t = cu_n[b] + i, at position
 *     lens[b] + i: for writers of their own; the calls of this library find a
 *     token's place by the table.  Tokens of no sequence's range are left as they were.
 * The ring: free_pages[(head + i) mod num_pages], i < count; queue holds
 * {head, count}.  Pages held and free together are at most num_pages.
 *   lens       device int32[batch]
 *   cu_n       device int32[batch+1], non-decreasing, within 0..total_n; may
 *              be NULL when total_n = 0 (n_b = 0)
 *   held       device int32[batch]; held_out (may be held) the new counts
 *   queue      device int32[2]; queue_out (may be queue) the new ring
 *   free_pages device int32[num_pages] in/out
 *   block_table device int32[batch][max_pages_per_seq] in/out
 *   served     device int32[batch] out
 *   slots      device int64[total_n] out, or NULL
 * A sequence whose numbers are out of range (lens < 0, lens + n_b >= 2^31,
 * need_b or held outside 0..max_pages_per_seq, a cu_n range that falls or
 * lies outside 0..total_n) sets the bad-input bit, is not served and is left
 * unchanged (its slots, where its cu_n range is valid, are -1); the others
 * are served all the same (a token in the ranges of two has the later one's
 * slot).  A ring out of range (head, count, or more free and given back pages
 * than num_pages) sets the bit and serves none.  A free page id outside
 * 0..num_pages-1 sets it and is handed on as it is.
 * Limits: batch <= 16384; batch * max_pages_per_seq < 2^31; num_pages < 2^30.
 * Workspace: 256 bytes (status word and a counter that each call leaves at
 * zero), one for each call that may run at the same time as another.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t batch;
  int32_t page_size;          /* 16                                         */
  int32_t num_pages;          /* pages of the cache = entries of the ring   */
  int32_t max_pages_per_seq;
  int32_t total_n;            /* entries of slots (host copy), >= 0         */
  const int32_t *lens;
  const int32_t *cu_n;
  const int32_t *held;
  const int32_t *queue;
  int32_t *free_pages;
  int32_t *block_table;
  int32_t *held_out;
  int32_t *queue_out;
  int32_t *served;
  int64_t *slots;
  void *workspace;            /* device, 256-byte aligned                   */
  size_t workspace_bytes;
} simsd_page_map_desc;

size_t simsd_page_map_workspace_size(const simsd_page_map_desc *d);
simsd_status simsd_page_map(const simsd_page_map_desc *d, void *stream);

/* ------------------------------------------------------------------------
 * The 8-bit cache.  k_cache, v_cache: device e4m3 [num_pages][Hkv][16][hd];
 * k_scale, v_scale: device uint8 [num_pages][Hkv], the exponent of a page
 * and head's scale plus 127 (an e8m0 value): a stored code c stands for
 * c * 2^(scale - 127).  The append's exponents lie in -64..7, so magnitudes up
 * to 57344 (an older byte beyond them is brought into the range); the
 * attention takes every byte as what it stands for.
 * 255 marks a page and head that got a NaN or an infinity: every value of it
 * reads as NaN.  A power of two changes no mantissa, so a page whose scale
 * grows keeps its older codes' values (those of the few smallest binades are
 * rounded again).
 *
 * simsd_kvq_append -- rotates n_b keys of sequence b at positions start[b]
 * .. start[b]+n_b-1 and writes them and the values into those cache slots.
 * A page's scale is the smallest one that covers its new tokens, and where
 * tokens before start[b] lie in the page, not below its present scale (their
 * codes are moved to the new one).  Slots at and past start[b]+n_b keep
 * their codes; a later append writes them.
 *   k, v     device; head h of row r at r * k_row + h * hd (elements; 0
 *            selects Hkv * hd), sequence b's rows at cu_n[b]..; 16-byte
 *            aligned arrays and strides
 *   start    device int32[batch]
 *   cu_n     device int32[batch+1] prefix sums of the rows (cu_n[0] >= 0: rows
 *            before it are no sequence's)
 *   take     device int32[batch] or NULL: n_b = take[b] <= the sequence's
 *            rows (the first take[b] of them are written; 0: none), e.g. the
 *            data section's tokens of a block that closed, or 0 for a sequence
 *            that simsd_page_map did not serve (its table has no page for them)
 *   total_n  host: rows of k and v; 0: nothing is written (k and v may be NULL)
 * A sequence whose numbers are out of range, or whose table row does not
 * cover its slots or holds a page id outside the cache, sets the workspace's
 * bad-input bit; nothing is written for that sequence, or of that page.  (Where
 * cu_n falls, other sequences may be left out as well.)
 * Two sequences must not write the same page in one call.
 * Limits: num_kv_heads <= 1024; batch <= 2^20; max_pages_per_seq <= 2^26.
 * Workspace: the status word (256 bytes).
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t batch;
  int32_t num_kv_heads;
  int32_t head_dim;           /* 64 or 128                                  */
  int32_t page_size;          /* 16                                         */
  int32_t num_pages;
  int32_t max_pages_per_seq;
  int32_t total_n;
  simsd_dtype dtype;          /* of k and v                                 */
  simsd_rope_spec rope;
  int64_t k_row, v_row;       /* row strides in elements; 0: Hkv * hd       */
  const void *k;
  const void *v;
  const int32_t *start;
  const int32_t *cu_n;
  const int32_t *take;
  void *k_cache;
  void *v_cache;
  uint8_t *k_scale;
  uint8_t *v_scale;
  const int32_t *block_table;
  void *workspace;            /* device, 256-byte aligned                   */
  size_t workspace_bytes;
} simsd_kvq_append_desc;

simsd_status simsd_kvq_append(const simsd_kvq_append_desc *d, void *stream);

/* ------------------------------------------------------------------------
 * simsd_kvq_verify -- one attention layer of a pass over [8-bit prompt cache
 * | new tokens].  The cache is only read: the new tokens' keys (rotated
 * here) and values take part as they are, unquantised, and a rejected draft
 * leaves no trace; simsd_kvq_append writes what is kept.
 *   SIMSD_ORDER_PAIRED  simsd_verify_attn's layout: sequence b's n_b = 2 B_b
 *                       new tokens are D_1..D_B, D~_1..D~_B, tokens k of
 *                       both sections at position lens[b] + k - 1, under the
 *                       temporal mask of tau; B_max <= 32
 *   SIMSD_ORDER_NODES   n_b = B_b tokens, nodes of node_size tokens one after
 *                       another, token k of every node at position lens[b] +
 *                       k; a row sees the prompt and its own node (one node:
 *                       a block that sees itself); B_max <= 64
 *   SIMSD_ORDER_CAUSAL  n_b = B_b tokens at positions lens[b].., a row sees
 *                       the prompt and the tokens up to itself (B_b = 1: a
 *                       decode step); B_max <= 64
 * With T = 2 total_B (paired) or total_B tokens:
 *   q            device [T][Hq][hd], raw; row stride q_row
 *   k_new, v_new device [T][Hkv][hd], raw; row strides k_row, v_row
 *   out          device [T][Hq][hd], contiguous
 *   block_table  device int32[batch][max_pages_per_seq]; entries
 *                0..ceil(lens[b]/16)-1 are read
 *   tau, lens, cu_B  as for simsd_verify_attn (tau: paired only)
 * Strides are in elements, 0 selects contiguous rows; arrays and strides are
 * multiples of 16 bytes (SIMSD_ERR_ALIGN).  The prompt's values in slots at
 * and past lens[b] are never used.  fp32: fp32 arithmetic throughout.  bf16:
 * on the tensor cores, scores from the codes themselves; sums, maxima and the
 * output's accumulation in fp32, and in fewer bits
 *   - the rotated query and each new key, in two e4m3 parts: an element is off
 *     by at most 2^-9 of itself (rounding it to bf16: 2^-8) or 2^-17 of the
 *     largest of its row, whichever is more;
 *   - the weights that multiply the values, in f16, times the power of two of
 *     the page's or new token's values: such a product is off by at most 2^-11
 *     of itself or 2^-32 of the row's largest one.  (One that lies 2^110 or more
 *     below the largest may be missing from the sum of weights as well: a row
 *     that sees a new value of 1e25 beside pages of values below 1e-8.)
 * Keys are split over the SMs by max_pages_per_seq, not by the lengths: one or
 * a few long prompts run fastest in a table not much wider than they are.
 * A sequence whose device arrays are out of range (cu_B, B_b outside 1..B_max,
 * lens[b] outside 0..16 max_pages_per_seq, n_b not a multiple of node_size)
 * sets the bad-input bit and its rows of out are not written; a page id outside
 * the cache sets it too, and that page counts as absent.  (B_b = 0 is out of
 * range: a finished request leaves the batch first.)
 * A row that sees a marked page, or a new token whose value holds a NaN or an
 * infinity, is NaN; a token that a row does not see has no effect on it.
 * Limits: Hq % Hkv == 0, Hq <= 65535, head_dim 64 or 128, max_pages_per_seq <
 * 2^26, total_B <= 2^28, 64 batch Hkv row tiles < 2^31 (a tile: 128 of a
 * sequence's rows for a KV head, fp32 16).  The workspace size follows the
 * key-split plan (the current device's SM count).
 * ---------------------------------------------------------------------- */
typedef enum {
  SIMSD_ORDER_PAIRED = 0,
  SIMSD_ORDER_NODES = 1,
  SIMSD_ORDER_CAUSAL = 2
} simsd_order;

typedef struct {
  int32_t batch;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;           /* 64 or 128                                  */
  int32_t page_size;          /* 16                                         */
  int32_t num_pages;
  int32_t max_pages_per_seq;
  int32_t total_B;            /* sum_b B_b (host copy)                      */
  int32_t B_max;              /* max_b B_b (host copy)                      */
  simsd_dtype dtype;          /* of q, k_new, v_new, out                    */
  simsd_order order;
  int32_t node_size;          /* SIMSD_ORDER_NODES: >= 1; otherwise 0       */
  simsd_rope_spec rope;
  float sm_scale;             /* finite, > 0                                */
  int32_t wait_polls;         /* as in simsd_verify_desc                    */
  int64_t q_row, k_row, v_row;
  const void *q;
  const void *k_cache;
  const void *v_cache;
  const uint8_t *k_scale;
  const uint8_t *v_scale;
  const int32_t *block_table;
  const void *k_new;
  const void *v_new;
  const int32_t *tau;
  const int32_t *lens;
  const int32_t *cu_B;
  void *out;
  void *workspace;            /* device, 256-byte aligned                   */
  size_t workspace_bytes;
} simsd_kvq_verify_desc;

size_t simsd_kvq_verify_workspace_size(const simsd_kvq_verify_desc *d);
simsd_status simsd_kvq_verify(const simsd_kvq_verify_desc *d, void *stream);

/* ------------------------------------------------------------------------
 * The 4-bit cache.  cache: device uint8 [num_pages][Hkv][18 hd], a page and
 * head's record of 16 tokens (hd = 128: 2304 bytes, 64: 1152):
 *   [0, 8 hd)        key codes: token i's row at i hd / 2; byte d / 2 holds
 *                    elements d (even: low four bits) and d + 1
 *   [8 hd, 16 hd)    value codes: element d of tokens i (even: low four bits)
 *                    and i + 1 in byte (d / 32) 256 + (i / 2) 32 + d % 32
 *   [16 hd, 17 hd)   key scales: group g of token i at i hd / 16 + g
 *   [17 hd, 18 hd)   value scales: at (i / 2) hd / 8 + 2 g + i % 2
 * A code is an e2m1 number (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives); a
 * group is 16 neighbouring elements of a token's head; a scale byte holds bits
 * 14..7 of a non-negative f16 number (five bits of exponent, three of
 * mantissa).  A code stands for code * scale, which f16 holds exactly.  A byte
 * of 0xf8 and above marks a group that got a NaN or an infinity (the append
 * writes 0xfc): its elements read as NaN or infinities.
 *
 * simsd_kv4_append -- simsd_kvq_append for this cache: rotates n_b keys of
 * sequence b at positions start[b].. and writes them and the values there.  A
 * group's scale is the one nearest to its largest magnitude / 6 (ties to the
 * even one), at most 10240 (magnitudes up to 61440); an element's code the one
 * nearest to element / scale (ties to the even one, saturating).  A group
 * below 6 * 2^-18 is zeros.  No other token's codes or scales change.
 * Arguments, checks and bad inputs as for simsd_kvq_append, and two sequences
 * must not write the same page in one call.
 * Limits: num_kv_heads <= 1024; batch <= 2^20; max_pages_per_seq <= 2^26;
 * total_n <= 2^30.
 * Workspace: the status word (256 bytes).
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t batch;
  int32_t num_kv_heads;
  int32_t head_dim;           /* 64 or 128                                  */
  int32_t page_size;          /* 16                                         */
  int32_t num_pages;
  int32_t max_pages_per_seq;
  int32_t total_n;
  simsd_dtype dtype;          /* of k and v: SIMSD_F32 or SIMSD_BF16        */
  simsd_rope_spec rope;
  int64_t k_row, v_row;       /* row strides in elements; 0: Hkv * hd       */
  const void *k;
  const void *v;
  const int32_t *start;
  const int32_t *cu_n;
  const int32_t *take;        /* or NULL                                    */
  void *cache;                /* 16-byte aligned                            */
  const int32_t *block_table;
  void *workspace;            /* device, 256-byte aligned                   */
  size_t workspace_bytes;
} simsd_kv4_append_desc;

simsd_status simsd_kv4_append(const simsd_kv4_append_desc *d, void *stream);

/* ------------------------------------------------------------------------
 * simsd_kv4_read -- the keys (rotated, as they lie) and values of positions
 * start[b] .. start[b]+n_b-1 of each sequence as rows: for a prefix that moves
 * elsewhere, or an attention that wants them plain.
 *   start    device int32[batch]
 *   cu_n     device int32[batch+1] prefix sums of the rows; rows of no
 *            sequence's range are left as they were
 *   k, v     device out, head h of row r at r * k_row + h * hd (elements; 0
 *            selects Hkv * hd); 16-byte aligned arrays and strides.  One of
 *            them may be NULL: not wanted.  SIMSD_F32 is exact, SIMSD_BF16
 *            too (scales below 2^-14 included); SIMSD_E4M3 rounds to nearest
 *            even, saturating at 448, NaN for what is not finite
 *   total_n  host: rows of k and v; 0: nothing is written
 * Limits and bad inputs as for simsd_kv4_append: that sequence's rows, or
 * those of that page, are left as they were.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t batch;
  int32_t num_kv_heads;
  int32_t head_dim;           /* 64 or 128                                  */
  int32_t page_size;          /* 16                                         */
  int32_t num_pages;
  int32_t max_pages_per_seq;
  int32_t total_n;
  simsd_dtype dtype;          /* of k and v                                 */
  int64_t k_row, v_row;       /* row strides in elements; 0: Hkv * hd       */
  const void *cache;          /* 16-byte aligned                            */
  const int32_t *block_table;
  const int32_t *start;
  const int32_t *cu_n;
  void *k;
  void *v;
  void *workspace;            /* device, 256-byte aligned                   */
  size_t workspace_bytes;
} simsd_kv4_read_desc;

simsd_status simsd_kv4_read(const simsd_kv4_read_desc *d, void *stream);

/* ------------------------------------------------------------------------
 * simsd_kv4_verify -- simsd_kvq_verify over the 4-bit cache: the same orders,
 * arrays, strides, limits, key splits and bad inputs.  fp32: fp32 arithmetic
 * throughout.  bf16: on the tensor cores in f16 with fp32 sums, maxima and
 * output; the cache's values are exact there.  In fewer bits
 *   - the rotated query and each new key, relative to a power of two of the
 *     row's: an element is off by at most 2^-11 of itself or 2^-33 of the
 *     largest of its row, whichever is more;
 *   - each new value, relative to a power of two of its token's, likewise (or
 *     2^-89, if that is more);
 *   - the weights that multiply the values: off by at most 2^-11 of themselves
 *     or 2^-32 of the row's largest product.  (The sum of weights has its own:
 *     no token's share depends on any value.  Only beside a new value beyond
 *     2^96 may it lack prompt keys that weigh less than 2^-29 of the largest.)
 * A row that sees a key of a marked group is NaN; one of a value, in that
 * group's elements; a row that sees a new token with a NaN or an infinity is
 * NaN.  A token that a row does not see has no effect on it.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t batch;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;           /* 64 or 128                                  */
  int32_t page_size;          /* 16                                         */
  int32_t num_pages;
  int32_t max_pages_per_seq;
  int32_t total_B;            /* sum_b B_b (host copy)                      */
  int32_t B_max;              /* max_b B_b (host copy)                      */
  simsd_dtype dtype;          /* of q, k_new, v_new, out                    */
  simsd_order order;
  int32_t node_size;          /* SIMSD_ORDER_NODES: >= 1; otherwise 0       */
  simsd_rope_spec rope;
  float sm_scale;             /* finite, > 0                                */
  int32_t wait_polls;         /* as in simsd_verify_desc                    */
  int64_t q_row, k_row, v_row;
  const void *q;
  const void *cache;          /* 16-byte aligned                            */
  const int32_t *block_table;
  const void *k_new;
  const void *v_new;
  const int32_t *tau;
  const int32_t *lens;
  const int32_t *cu_B;
  void *out;
  void *workspace;            /* device, 256-byte aligned                   */
  size_t workspace_bytes;
} simsd_kv4_verify_desc;

size_t simsd_kv4_verify_workspace_size(const simsd_kv4_verify_desc *d);
simsd_status simsd_kv4_verify(const simsd_kv4_verify_desc *d, void *stream);

/* ------------------------------------------------------------------------
 * simsd_token_logprobs -- what a request gets back beside its tokens.  For
 * each row r of logits l, p = softmax(l / T):
 *   logprob[r]  ln p of tokens[r]
 *   rank[r]     tokens ahead of it: #{v: l_v > l_t} + #{v < t: l_v = l_t}
 *   entropy[r]  -sum p ln p, in nats
 *   top_ids[r], top_logprobs[r]  the top_k likeliest tokens, likeliest first
 *               (equal ones in index order), and their ln p
 *   logits   device [rows] rows of vocab entries (dtype), row_stride elements
 *            apart (0: vocab); any alignment of their type
 *   tokens   device int32[rows] or NULL (then logprob and rank are NULL too).
 *            -1: the row is not read, its outputs stay as they were.  Another
 *            token outside 0..vocab-1 sets the bad-input bit; its logprob is
 *            NaN, its rank -1
 *   logprob, entropy  device float32[rows] or NULL; rank device int32[rows] or
 *            NULL; top_ids device int32[rows][top_k] and top_logprobs device
 *            float32[rows][top_k], both or none (top_k = 0)
 * -inf entries have probability 0 (ln p = -inf).  A row that is -inf
 * throughout or holds a NaN or +inf has NaN for logprob, entropy and
 * top_logprobs; its rank and ids are of no use (ids lie in 0..vocab-1).
 * Limits: 1 <= vocab <= 2^21; 0 <= rows <= 2^20; 0 <= top_k <= min(32, vocab);
 * T as in simsd_accept_desc, within 1e-30..1e30.  rows = 0 returns SIMSD_OK.
 * Workspace: simsd_token_logprobs_workspace_size, 256 + rows * C * 48 bytes
 * rounded up to a multiple of 256, with C = ceil(vocab / 2048) + 1.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t rows;
  int32_t vocab;
  int32_t top_k;
  simsd_dtype dtype;          /* of the logits: SIMSD_F32 or SIMSD_BF16     */
  float temperature;          /* > 0; 0 selects 1                           */
  int64_t row_stride;
  const void *logits;
  const int32_t *tokens;
  float *logprob;
  int32_t *rank;
  float *entropy;
  int32_t *top_ids;
  float *top_logprobs;
  void *workspace;            /* device, 256-byte aligned                   */
  size_t workspace_bytes;
} simsd_token_logprobs_desc;

size_t simsd_token_logprobs_workspace_size(const simsd_token_logprobs_desc *d);
simsd_status simsd_token_logprobs(const simsd_token_logprobs_desc *d, void *stream);

/* ------------------------------------------------------------------------
 * simsd_read_status -- synchronise `stream`, copy the device status word of
 * a workspace used by simsd_verify_attn / simsd_accept to *word_out (bit 0:
 * a bounded wait ran out) and clear it, together with the chunk pass's
 * control words (bytes 128..139 of a workspace, zero between calls).  Returns SIMSD_ERR_TIMEOUT when a
 * bit was set, SIMSD_OK otherwise, SIMSD_ERR_CUDA on a CUDA error.
 * ---------------------------------------------------------------------- */
simsd_status simsd_read_status(void *workspace, void *stream,
                               uint32_t *word_out);

#ifdef __cplusplus
}
#endif
#endif /* SIMSD_H */

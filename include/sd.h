/*
 * sd.h -- C ABI of the GB300 (sm_103a) speculative-decoding verify and P-EAGLE draft-batch
 * rebuild library (libsd_gb300.so).
 *
 * Three calls make one decoding step's hot path, in this order on one stream:
 *   sd_verify         lossless verification of K drafts per request (rejection sampling with a
 *                     residual resample, or greedy argmax at temperature 0);
 *   sd_pdraft_expand  rebuild of the drafter batch for the next parallel-drafting pass;
 *   sd_hidden_gather  drafter hidden states from the target's hidden states or h_shared.
 *
 * Conventions for every call:
 *   - Every pointer is a DEVICE pointer owned by the caller, or, for the read-only row inputs
 *     (target, draft, hidden states), host memory the GPU can address (page-locked or
 *     registered): the kernels then read over the host link only the parts the step needs.
 *     Outputs, the workspace and *err are device memory. The library allocates nothing and keeps
 *     no state between calls.
 *   - Calls only enqueue work on `stream` (a cudaStream_t; 0 = the legacy default stream) and
 *     never synchronise, so a step can be captured in a CUDA graph.
 *   - The return value is SD_OK or a negative SD_E_* code for errors the host can see (null
 *     pointer, bad size, misaligned pointer, launch failure). Nothing is enqueued on error.
 *   - Data errors found on the device (a draft token outside [0, V), a position the block table
 *     does not cover, ...) are OR-ed as SD_ERR_* bits into *err (a device int32 the caller
 *     zeroes; may be NULL). The kernel then takes the documented fallback. No kernel traps or
 *     asserts. One kernel waits on a value written by another CTA of the same launch: the
 *     single launch of sd_verify_prepare (see there), whose wait is bounded by time (20 ms on
 *     the GPU clock) and ends with SD_ERR_WAIT, never with a hang. The warps of a CTA of
 *     sd_kv_attend and of sd_kv_weights wait for one another and for their loads, each time about a
 *     second at most; SD_ERR_WAIT there too means that the call's output is incomplete.
 *
 * Notation: B requests, K drafts per request (1 <= K <= SD_K_MAX), V vocabulary entries,
 * H hidden size. Target rows p_0..p_K of request r are rows r*(K+1)+j of `target`; draft rows
 * q_0..q_{K-1} are rows r*K+j of `draft`; draft d_{j+1} (drafts[r*K+j]) is checked against row j.
 */
#ifndef SD_GB300_H
#define SD_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define SD_API __attribute__((visibility("default")))
#else
#define SD_API
#endif

#define SD_K_MAX 16

/* host-visible status codes */
#define SD_OK 0
#define SD_E_NULL (-1)     /* a required pointer is NULL */
#define SD_E_SHAPE (-2)    /* a size or stride is out of range, or arrays share memory that may not */
#define SD_E_DTYPE (-3)    /* unknown dtype */
#define SD_E_ALIGN (-4)    /* a pointer or stride breaks the stated alignment */
#define SD_E_LAUNCH (-5)   /* the CUDA launch failed (cudaGetLastError is left set) */
#define SD_E_DEVICE (-6)   /* no usable sm_103 device is current */
#define SD_E_NOALLOC_LIMIT (-7) /* B > SD_VERIFY_NOALLOC_MAX_B for sd_verify_noalloc */

/* device-side data error bits, OR-ed into *err */
#define SD_ERR_TOKEN_RANGE 1    /* a draft token outside [0, V): treated as rejected */
#define SD_ERR_BLOCK_TABLE 2    /* drafter position not covered by the block table: slot -1 */
#define SD_ERR_NUM_ACCEPTED 4   /* num_accepted outside [0, K]: clamped */
#define SD_ERR_MAP_RANGE 8      /* hidden_map row >= n_in_rows: h_shared written instead */
#define SD_ERR_ZERO_ROW 16      /* a race row without a positive key even on p, or a row to be cut
                                   without an entry to keep: token 0 */
#define SD_ERR_TOTAL_RANGE 32   /* total_out outside [0, capacity]: clamped */
#define SD_ERR_WAIT 64          /* sd_verify_prepare: a request's first drafter slot was not
                                   published within the bounded wait (20 ms); its final token is
                                   not written to input_ids. sd_kv_attend, sd_kv_weights: a wait
                                   inside the kernel ran out, outputs are incomplete */
#define SD_ERR_DRAFT_COUNT 128  /* cu_drafts gives a request a draft count outside [0, K_max]:
                                   clamped (sd_verify_ragged) */
#define SD_ERR_KV_SLOT 256      /* a slot beyond the cache: that token is not written */
#define SD_ERR_KV_RANGE 512     /* a length, a prefix entry or a block-table entry of a cache read
                                   is out of range: those tokens are left out (sd_kv_read writes
                                   zeros for them, sd_kv_evict takes them as such) */

/* input kinds for sd_verify */
#define SD_F32_PROBS 0    /* fp32 probabilities, already at the sampling temperature */
#define SD_BF16_LOGITS 1  /* bf16 logits; softmax(l / T_r) is taken inside the kernel */

/*
 * sd_verify -- batched lossless verification of K drafts per request.
 *
 * Speculative-decoding explainer (ainews.alishangtian.com), sections "核心思想" (verify K+1
 * positions, discard after the first rejection, K+1 tokens when all are accepted),
 * "修正拒绝采样" (accept with probability min(1, p(x)/q(x)); on rejection resample from the
 * normalised residual max(0, p - q)) and "边界与代价" (temperature 0 must equal greedy decoding).
 *
 * Per request r, with T_r = temperature[r] (NULL: every T_r = 1):
 *   T_r > 0: draft d_{j+1} is accepted iff u_j * Q < P, with P = p_j(d_{j+1}),
 *            Q = q_j(d_{j+1}), compared exactly in double, and u_j = (w >> 8) * 2^-24 where w
 *            is word 0 of Philox4x32-10 block (0, j, r, 0) under key (seed lo, seed hi).
 *            a_r = index of the first rejection, or K. The final token b_r is
 *              a_r < K:  argmax_x r(x) / E_x, r = max(0, p_{a_r} - q_{a_r}),
 *              a_r == K: argmax_x max(0, p_K(x)) / E_x   (the bonus token),
 *            with E_x = fp32(-log(v)) from the double log, v = (w + 0.5) * 2^-32 and w word
 *            (x & 3) of block (x >> 2, j, r, 1), j the race row. Keys are fp32 quotients for
 *            SD_F32_PROBS; ties go to the lowest x. If no key of the residual race is
 *            positive, the race is re-run on p of the same row with the same E_x; if that has
 *            none either, b_r = 0 and SD_ERR_ZERO_ROW is raised.
 *   T_r == 0: accept iff d_{j+1} == argmax_x p_j(x) (lowest x on ties); b_r = argmax p_{a_r}.
 * For SD_BF16_LOGITS, p_j = softmax(l^t_j / T_r) and q_j = softmax(l^d_j / T_r) are formed in
 * fp32 inside the kernel (results match a double-precision evaluation within the documented
 * tolerance, not bit for bit); T_r == 0 works on the raw logits (bit-exact).
 * Rows after the first rejection are never read.
 *
 * Arguments:
 *   B >= 0, 1 <= K <= SD_K_MAX, V >= 1; dtype SD_F32_PROBS or SD_BF16_LOGITS.
 *   target [B*(K+1) rows, stride ld_t elements], draft [B*K rows, stride ld_d elements]
 *     (fp32 or bf16 per dtype; ld >= V). Rows whose start is 16-byte aligned are read with
 *     128-bit loads, other layouts with scalar loads.
 *   drafts [B, K] int32; temperature [B] fp32 or NULL (every request samples at T = 1; for
 *     large probability rows the library then balances the race over the whole GPU);
 *   seed: Philox key; request_base: the request index that local request 0 has in the Philox
 *     counters (r in the blocks above is request_base + local index), so that a batch split
 *     over several GPUs by request draws exactly what one GPU would draw for the whole batch;
 *     request_base + B <= 2^32.
 * Outputs:
 *   out_tokens [B, K+1] int32: d_1..d_{a_r}, b_r, then -1.
 *   num_accepted [B] int32: a_r.
 *   p_at_draft, q_at_draft [B, K] fp32, each may be NULL: P and Q of every examined draft
 *     j <= min(a_r, K-1) (probabilities; raw target/draft values for T_r == 0; 0 for an
 *     out-of-range token), -1 for drafts never examined.
 *   workspace, workspace_bytes: device scratch of at least sd_verify_workspace_bytes(B, K, V,
 *     dtype) bytes, zeroed before first use and left zeroed by every call (see below).
 *   err: see above.
 */
SD_API int sd_verify(int B, int K, int V, int dtype, const void* target, long ld_t,
                     const void* draft, long ld_d, const int32_t* drafts,
                     const float* temperature, uint64_t seed, uint32_t request_base,
                     int32_t* out_tokens, int32_t* num_accepted, float* p_at_draft,
                     float* q_at_draft, void* workspace, size_t workspace_bytes, int32_t* err,
                     void* stream);

/*
 * sd_verify_ragged -- sd_verify with a number of drafts of its own for every request.
 *
 * Request r has K_r = cu_drafts[r+1] - cu_drafts[r] drafts (0 <= K_r <= K_max; cu_drafts is the
 * exclusive prefix [B+1] of the counts, on the device). Its rows are packed: target rows
 * p_0..p_{K_r} at rows cu_drafts[r] + r .. cu_drafts[r] + r + K_r of target, draft rows
 * q_0..q_{K_r - 1} and draft tokens at cu_drafts[r] .. of draft and drafts. Each request is
 * verified exactly as sd_verify verifies it with K = K_r (the same Philox counters: request
 * request_base + r, row j); K_r = 0 samples the bonus token from p_0 alone. Outputs keep the
 * stride of K_max: out_tokens [B, K_max+1] (-1 after b_r), p_at_draft / q_at_draft [B, K_max]
 * (-1 where no draft was examined). cu_drafts must be consistent with the arrays: rows are
 * addressed from its entries. A count outside [0, K_max] (a decreasing entry, a step beyond K_max)
 * is clamped and raises SD_ERR_DRAFT_COUNT; the rows it then addresses must still lie inside the
 * arrays. Other arguments, workspace and errors as for sd_verify (with K = K_max).
 */
SD_API int sd_verify_ragged(int B, int K_max, int V, int dtype, const void* target, long ld_t,
                            const void* draft, long ld_d, const int32_t* drafts,
                            const int32_t* cu_drafts, const float* temperature, uint64_t seed,
                            uint32_t request_base, int32_t* out_tokens, int32_t* num_accepted,
                            float* p_at_draft, float* q_at_draft, void* workspace,
                            size_t workspace_bytes, int32_t* err, void* stream);

/*
 * Size in bytes of the workspace sd_verify needs for B requests: 16 bytes per request, where the
 * CTAs that share a request's race row merge their results. The caller allocates it (16-byte
 * aligned) and zeroes it once; every sd_verify call leaves it zeroed again. Calls that may run
 * concurrently need separate workspaces.
 */
SD_API size_t sd_verify_workspace_bytes(int B, int K, int V, int dtype);

/*
 * Number of kernels one sd_verify (or sd_verify_noalloc) call with these sizes launches on the
 * current device: 0 for B == 0, else 1 (the cluster kernel, or for an all-sampled batch on large
 * probability rows the race kernel that balances the batch over every SM). A planning query for
 * callers that count launches (a CUDA-graph budget, a profiler filter); it launches nothing.
 * Returns a negative status for an unknown dtype or B < 0, V < 1.
 */
SD_API int sd_verify_kernels(int B, int V, int dtype, int has_temperature);

/*
 * sd_verify_noalloc -- sd_verify for callers that cannot allocate device memory. This call has
 * no counterpart in the method's sources; it exists for callers such as a plugin or engine
 * that is handed only its input and output buffers and may not call cudaMalloc (allocation
 * would stall or break the host runtime's memory pool, or happen inside a stream capture that
 * forbids it). Same arguments, semantics and results as sd_verify, minus the workspace: the
 * merge slots live in a fixed device array of SD_VERIFY_NOALLOC_MAX_B entries (16 bytes each)
 * that every GPU loading the library holds until the process exits.
 *   - B > SD_VERIFY_NOALLOC_MAX_B returns SD_E_NOALLOC_LIMIT and enqueues nothing.
 *   - The first call on a device looks the array's address up (cudaGetSymbolAddress) with that
 *     device current; make that first call before any stream capture.
 *   - Each call enqueues a clear of the slots it uses (one cudaMemsetAsync of B*16 bytes) and
 *     then the verify kernel: two stream operations, of which sd_verify_kernels counts only the
 *     kernel. It calls no allocator.
 *   - All calls on a device share the one array: calls that may overlap on the GPU (other
 *     streams, other host threads) race on it and must be serialised by the caller.
 */
#define SD_VERIFY_NOALLOC_MAX_B 4096
SD_API int sd_verify_noalloc(int B, int K, int V, int dtype, const void* target, long ld_t,
                             const void* draft, long ld_d, const int32_t* drafts,
                             const float* temperature, uint64_t seed, uint32_t request_base,
                             int32_t* out_tokens, int32_t* num_accepted, float* p_at_draft,
                             float* q_at_draft, int32_t* err, void* stream);

/*
 * sd_draft_sample -- the drafter's K new drafts per request, sampled from its output rows.
 *
 * P-EAGLE blog (vLLM), section "Triton Kernel": new_token_idx marks the drafter slots whose
 * logits become the next drafts; the drafter runs its head on those slots, giving one row per
 * (request, draft). Each row is sampled the way the verify step samples a bonus token
 * (speculative-decoding explainer, "修正拒绝采样": an exact sample of the row's distribution):
 * d_{k+1} of request r = argmax_x q(x) / E_x over row (r*K + k), E_x = fp32(-log((w + 0.5) 2^-32))
 * with w word (x & 3) of Philox4x32-10 block (x >> 2, k, request_base + r, 2) -- tag 2, a stream
 * separate from the verify races' tag 1 -- ties to the lowest x; temperature[r] == 0 takes the
 * argmax of the row (lowest x on ties).
 * Arguments:
 *   rows: [B*K, V] with row stride ld elements: SD_F32_PROBS probabilities (already at the
 *     sampling temperature; only temperature == 0 matters), or SD_BF16_LOGITS logits, sampled
 *     from softmax(l / temperature[r]) computed in the kernel.
 *   temperature: [B] fp32 or NULL (= 1); seed, request_base: as for sd_verify.
 *   drafts: [B, K] int32 output (may serve as the next step's sd_verify drafts).
 *   err: SD_ERR_ZERO_ROW when a sampled row has no positive entry (draft 0).
 * Returns SD_OK, or SD_E_SHAPE (K outside [1, SD_K_MAX], V < 1, ld < V, B*K rows beyond 2^31
 * CTAs, request_base + B > 2^32), SD_E_DTYPE, SD_E_NULL, SD_E_ALIGN (rows not aligned to its
 * element), SD_E_DEVICE, SD_E_LAUNCH.
 */
SD_API int sd_draft_sample(int B, int K, int V, int dtype, const void* rows, long ld,
                           const float* temperature, uint64_t seed, uint32_t request_base,
                           int32_t* drafts, int32_t* err, void* stream);

/*
 * sd_pdraft_expand -- rebuild of the drafter batch for P-EAGLE parallel drafting.
 *
 * P-EAGLE blog (vLLM), sections "核心方法" (drafter position i takes the token and hidden state
 * of position i-1; MASK positions take emb(mask) and h_shared), "并行草稿生成的挑战" (expand ids,
 * hidden states and positions with MASK slots, bump positions per request, recompute the slot
 * mapping and per-request start indices), "Triton Kernel" (one pass also emits the rejected-token
 * mask, the masked-token mask, the new-token indices and the hidden-state mapping) and
 * "Hidden State 管理" (PADDING_SLOT_ID = -1).
 *
 * Request r with a_r = num_accepted[r] gets L_r = a_r + K consecutive drafter slots starting at
 * start_loc[r] = sum_{r' < r} L_{r'}. Slot j of request r (i = start_loc[r] + j):
 *   input_ids[i]    = out_tokens[r][j] for j <= a_r (d_1..d_{a_r}, b_r), else mask_token_id
 *   positions[i]    = pos0[r] + 1 + j          (pos0[r] = position of verify slot 0)
 *   slot_mapping[i] = block_table[r][pos / block_size] * block_size + pos % block_size, or -1
 *                     with SD_ERR_BLOCK_TABLE when the table does not cover pos
 *   hidden_map[i]   = r*(K+1) + j for j <= a_r (target hidden row), else -1 (h_shared)
 *   is_masked[i]    = (j > a_r)
 * Slots total_out <= i < capacity are padding: id -1, position 0, slot -1, map -1, mask 0.
 * is_rejected [B, K+1]: 1 for verify slots 1 <= j <= K with j > a_r, else 0.
 * new_token_idx [B, K]: start_loc[r] + a_r + k, the slots whose drafter logits become the next
 *   drafts. start_loc has B+1 entries; start_loc[B] = *total_out = sum_r L_r.
 * Arguments: B >= 0, 1 <= K <= SD_K_MAX; out_tokens [B, K+1] and num_accepted [B] as written by
 *   sd_verify; pos0 [B]; block_table [B, max_blocks] int32 (entries < 0 unused);
 *   block_size >= 1; capacity >= 0 (B*2*K holds every outcome; a smaller capacity truncates
 *   with SD_ERR_TOTAL_RANGE). Outputs have `capacity` entries (is_masked uint8).
 */
SD_API int sd_pdraft_expand(int B, int K, const int32_t* out_tokens, const int32_t* num_accepted,
                     const int32_t* pos0, const int32_t* block_table, int max_blocks,
                     int block_size, int32_t mask_token_id, int capacity, int32_t* input_ids,
                     int32_t* positions, int32_t* slot_mapping, int32_t* hidden_map,
                     uint8_t* is_masked, uint8_t* is_rejected, int32_t* start_loc,
                     int32_t* new_token_idx, int32_t* total_out, int32_t* err, void* stream);

/*
 * sd_pdraft_prepare -- sd_pdraft_expand and the hidden-state gather of sd_hidden_gather in one
 * launch: every output of sd_pdraft_expand, plus out_hidden[i, :] for i < total_out (clamped to
 * capacity) = target_hidden[hidden_map[i], :], or h_shared[:] where hidden_map[i] == -1, as
 * sd_hidden_gather defines it (same sources: P-EAGLE blog, "Hidden State 管理"). Rows from
 * total_out on are not written. Arguments are those of the two calls; target_hidden has n_in_rows
 * rows of stride ld_in, out_hidden `capacity` rows of stride ld_out (both >= H), bf16.
 * When enqueued right after sd_verify it is launched as a programmatic dependent of it: it is
 * scheduled while sd_verify drains and waits on the device for sd_verify's results.
 */
SD_API int sd_pdraft_prepare(int B, int K, const int32_t* out_tokens, const int32_t* num_accepted,
                             const int32_t* pos0, const int32_t* block_table, int max_blocks,
                             int block_size, int32_t mask_token_id, int capacity,
                             int32_t* input_ids, int32_t* positions, int32_t* slot_mapping,
                             int32_t* hidden_map, uint8_t* is_masked, uint8_t* is_rejected,
                             int32_t* start_loc, int32_t* new_token_idx, int32_t* total_out,
                             int H, const void* target_hidden, long ld_in, int n_in_rows,
                             const void* h_shared, void* out_hidden, long ld_out, int32_t* err,
                             void* stream);

/*
 * sd_verify_prepare -- one step of the hot path in one call: sd_verify followed by
 * sd_pdraft_prepare on its outputs.
 *
 * The two operations are those of sd_verify (speculative-decoding explainer, sections "核心思想"
 * and "修正拒绝采样") and sd_pdraft_prepare (P-EAGLE blog, sections "Triton Kernel" and "Hidden
 * State 管理"), with sd_verify's out_tokens and num_accepted feeding the rebuild. When every
 * request samples (temperature NULL) on probability rows, the batch is small enough for one
 * wave of CTAs (B <= 192, and 2B no more than 5 CTAs per SM) and sd_verify would split each row
 * over a request's CTAs (rather than its large-batch race kernel), both run in a single launch:
 * B extra CTAs rebuild the drafter batch while the others race. The single launch is taken
 * only when every one of its CTAs fits on the device at once (the occupancy API's count of
 * resident CTAs per SM times the SMs).
 * A rebuild CTA recomputes the accept decisions of its request and of those before it (they
 * depend on the inputs only), takes its first drafter slot as their prefix, and writes its
 * request's rows and hidden states; only the final token at slot a_r waits for the race, and the
 * CTA that completes request r's race row writes it at the slot the rebuild CTA published in the
 * workspace. If that CTA finds nothing published, it polls for at most 20 ms of the GPU clock
 * (in practice it never waits: the slot appears microseconds after the launch starts, the race
 * rows complete tens of microseconds later; a rebuild CTA kept off the GPU, for instance by
 * other work on another stream filling the SMs, is the only way to run the wait out). When the
 * wait runs out, SD_ERR_WAIT is raised and that request's final token is not written to
 * input_ids (every other output is); the two CTAs still leave the workspace zeroed. Other
 * batches run the two kernels back to back. Either way every output is bit for bit what
 * sd_verify then sd_pdraft_prepare write.
 *
 * Arguments: sd_verify's (without cu_drafts) then sd_pdraft_prepare's from pos0 on (out_tokens
 * and num_accepted are this call's own outputs), with one workspace of at least
 * sd_verify_prepare_workspace_bytes(B) bytes (as much as sd_verify's), 16-byte aligned, zeroed
 * before first use and left zeroed by every call. Errors: those of both calls; SD_ERR_WAIT if a
 * request's published slot never appeared (its final token is then not written to input_ids).
 */
SD_API int sd_verify_prepare(
    int B, int K, int V, int dtype, const void* target, long ld_t, const void* draft, long ld_d,
    const int32_t* drafts, const float* temperature, uint64_t seed, uint32_t request_base,
    int32_t* out_tokens, int32_t* num_accepted, float* p_at_draft, float* q_at_draft,
    const int32_t* pos0, const int32_t* block_table, int max_blocks, int block_size,
    int32_t mask_token_id, int capacity, int32_t* input_ids, int32_t* positions,
    int32_t* slot_mapping, int32_t* hidden_map, uint8_t* is_masked, uint8_t* is_rejected,
    int32_t* start_loc, int32_t* new_token_idx, int32_t* total_out, int H,
    const void* target_hidden, long ld_in, int n_in_rows, const void* h_shared, void* out_hidden,
    long ld_out, void* workspace, size_t workspace_bytes, int32_t* err, void* stream);

/*
 * sd_verify_prepare_ragged -- sd_verify_ragged then sd_pdraft_prepare_ragged on its outputs, in
 * one call: a draft count per request (cu_drafts [B+1], rows packed as sd_verify_ragged reads
 * them, K_max the output stride), with the same single launch for all-sampled one-wave batches
 * (the rebuild CTAs recompute every request's decisions over its own K_r drafts). Every output is
 * bit for bit what the two ragged calls write; arguments and errors as for them and
 * sd_verify_prepare.
 */
SD_API int sd_verify_prepare_ragged(
    int B, int K_max, int V, int dtype, const void* target, long ld_t, const void* draft,
    long ld_d, const int32_t* drafts, const int32_t* cu_drafts, const float* temperature,
    uint64_t seed, uint32_t request_base, int32_t* out_tokens, int32_t* num_accepted,
    float* p_at_draft, float* q_at_draft, const int32_t* pos0, const int32_t* block_table,
    int max_blocks, int block_size, int32_t mask_token_id, int capacity, int32_t* input_ids,
    int32_t* positions, int32_t* slot_mapping, int32_t* hidden_map, uint8_t* is_masked,
    uint8_t* is_rejected, int32_t* start_loc, int32_t* new_token_idx, int32_t* total_out, int H,
    const void* target_hidden, long ld_in, int n_in_rows, const void* h_shared, void* out_hidden,
    long ld_out, void* workspace, size_t workspace_bytes, int32_t* err, void* stream);

/* Workspace of sd_verify_prepare (and _ragged): sd_verify's merge slots, one per request. */
SD_API size_t sd_verify_prepare_workspace_bytes(int B);

/* Kernels one sd_verify_prepare call with these sizes launches (0, 1 fused, or 2); a planning
 * query like sd_verify_kernels. */
SD_API int sd_verify_prepare_kernels(int B, int K, int V, int dtype, int has_temperature);

/*
 * sd_pdraft_prepare_ragged -- sd_pdraft_prepare with a draft count per request, the rebuild
 * that follows sd_verify_ragged (adaptive per-request k): request r with K_r = cu_drafts[r+1] -
 * cu_drafts[r] drafts (0 <= K_r <= K_max) gets L_r = a_r + K_r drafter slots (its accepted
 * drafts, its final token, K_r - 1 MASK slots); its target hidden rows are cu_drafts[r] + r ..
 * (the packing sd_verify_ragged reads). is_rejected [B, K_max+1] is 1 for 1 <= j <= K_r with
 * j > a_r; new_token_idx [B, K_max] is start_loc[r] + a_r + k for k < K_r and -1 after;
 * num_accepted outside [0, K_r] is clamped (SD_ERR_NUM_ACCEPTED), a count outside [0, K_max]
 * too (SD_ERR_DRAFT_COUNT). capacity B*2*K_max holds every outcome. Other arguments and outputs
 * as for sd_pdraft_prepare (with K = K_max).
 */
SD_API int sd_pdraft_prepare_ragged(int B, int K_max, const int32_t* out_tokens,
                                    const int32_t* num_accepted, const int32_t* cu_drafts,
                                    const int32_t* pos0, const int32_t* block_table,
                                    int max_blocks, int block_size, int32_t mask_token_id,
                                    int capacity, int32_t* input_ids, int32_t* positions,
                                    int32_t* slot_mapping, int32_t* hidden_map,
                                    uint8_t* is_masked, uint8_t* is_rejected, int32_t* start_loc,
                                    int32_t* new_token_idx, int32_t* total_out, int H,
                                    const void* target_hidden, long ld_in, int n_in_rows,
                                    const void* h_shared, void* out_hidden, long ld_out,
                                    int32_t* err, void* stream);

/*
 * sd_pdraft_prepare_padded -- the drafter batch in fixed-width rows, with its hidden states.
 *
 * P-EAGLE blog (vLLM), sections "并行草稿生成的挑战" and "Triton Kernel" (the rebuilt ids,
 * positions, slot mapping, masks and new-token indices) and "Hidden State 管理" (rejected tokens
 * map to PADDING_SLOT_ID = -1 so that they write no KV cache; the target hidden states are
 * scattered to their drafter rows; MASK rows take h_shared). In this form every request keeps a
 * row of W = 2K drafter slots whatever it accepted, so start indices are r*W, the batch size is
 * fixed at B*W and no prefix over the batch is needed. Slot j of request r (i = r*W + j):
 *   j < a_r + K: as sd_pdraft_expand defines slot j of request r (input_ids, positions =
 *     pos0 + 1 + j, slot_mapping, hidden_map, is_masked), rejected[i] = 0;
 *   j >= a_r + K (K - a_r rejected leftovers): input_ids = mask_token_id, positions =
 *     pos0 + 1 + j, slot_mapping = -1, hidden_map = -1, is_masked = 0, rejected[i] = 1.
 *   scatter_map [B*(K+1)]: target row r*(K+1)+j -> drafter row r*W + j for j <= a_r, else -1
 *     (the same copies as hidden_map, indexed by source).
 *   new_token_idx [B, K]: r*W + a_r + k.
 *   out_hidden (nullable: metadata only) [B*W, H] bf16 with row stride ld_out: row i =
 *     target_hidden[hidden_map[i]] or h_shared (also for map rows >= n_in_rows, with
 *     SD_ERR_MAP_RANGE). Every row is written.
 * Arguments as for sd_pdraft_prepare; outputs input_ids .. rejected have B*W entries.
 * Errors: SD_ERR_NUM_ACCEPTED (clamped), SD_ERR_BLOCK_TABLE (live slot not covered: -1).
 */
SD_API int sd_pdraft_prepare_padded(int B, int K, const int32_t* out_tokens,
                                    const int32_t* num_accepted, const int32_t* pos0,
                                    const int32_t* block_table, int max_blocks, int block_size,
                                    int32_t mask_token_id, int32_t* input_ids, int32_t* positions,
                                    int32_t* slot_mapping, int32_t* hidden_map,
                                    uint8_t* is_masked, uint8_t* rejected, int32_t* scatter_map,
                                    int32_t* new_token_idx, int H, const void* target_hidden,
                                    long ld_in, int n_in_rows, const void* h_shared,
                                    void* out_hidden, long ld_out, int32_t* err, void* stream);

/*
 * sd_verify_prepare_padded -- sd_verify then sd_pdraft_prepare_padded in one call.
 *
 * The step of sd_verify_prepare with the drafter batch in the fixed-width layout of
 * sd_pdraft_prepare_padded (P-EAGLE blog, "Hidden State 管理": rejected tokens on
 * PADDING_SLOT_ID, target hidden states scattered to their drafter rows). When every request
 * samples on probability rows (temperature NULL) and the batch fits one wave (the conditions of
 * sd_verify_prepare's single launch), this is one launch: CTA r (r < B) recomputes request r's
 * accept decisions from the inputs -- in this layout no request's rows depend on another's counts
 * -- and writes all 2K rows of request r but the token at row r*2K + a_r, which the CTA that
 * completes the request's race writes; nothing waits. Other batches run the verify kernel and
 * then the padded rebuild kernel. Either way every output is bit for bit what sd_verify then
 * sd_pdraft_prepare_padded write; sd_verify_prepare_kernels gives the number of launches.
 *
 * Arguments: sd_verify's (workspace of at least sd_verify_workspace_bytes(B, K, V, dtype),
 * 16-byte aligned, zeroed before first use and left zeroed by every call) then
 * sd_pdraft_prepare_padded's from pos0 on (out_tokens and num_accepted are this call's own
 * outputs). Errors: those of both calls.
 */
SD_API int sd_verify_prepare_padded(
    int B, int K, int V, int dtype, const void* target, long ld_t, const void* draft, long ld_d,
    const int32_t* drafts, const float* temperature, uint64_t seed, uint32_t request_base,
    int32_t* out_tokens, int32_t* num_accepted, float* p_at_draft, float* q_at_draft,
    const int32_t* pos0, const int32_t* block_table, int max_blocks, int block_size,
    int32_t mask_token_id, int32_t* input_ids, int32_t* positions, int32_t* slot_mapping,
    int32_t* hidden_map, uint8_t* is_masked, uint8_t* rejected, int32_t* scatter_map,
    int32_t* new_token_idx, int H, const void* target_hidden, long ld_in, int n_in_rows,
    const void* h_shared, void* out_hidden, long ld_out, void* workspace, size_t workspace_bytes,
    int32_t* err, void* stream);

/*
 * sd_hidden_gather -- drafter hidden states.
 *
 * P-EAGLE blog (vLLM), section "Hidden State 管理": target hidden states are copied to their
 * drafter slots and the learned h_shared fills the MASK slots. Written here in gather form:
 *   out_hidden[i, :] = hidden_map[i] >= 0 ? target_hidden[hidden_map[i], :] : h_shared[:]
 * for i < *total_out (read on the device, clamped to capacity with SD_ERR_TOTAL_RANGE). Rows
 * from *total_out on are not written. A map entry >= n_in_rows writes h_shared and raises
 * SD_ERR_MAP_RANGE. Rows are H bf16 values moved bit for bit; target_hidden has n_in_rows rows
 * of stride ld_in elements, out_hidden `capacity` rows of stride ld_out (both >= H).
 */
SD_API int sd_hidden_gather(int capacity, int H, const int32_t* total_out, const int32_t* hidden_map,
                     const void* target_hidden, long ld_in, int n_in_rows, const void* h_shared,
                     void* out_hidden, long ld_out, int32_t* err, void* stream);

/* ---- the paged 8-bit cache ----
 *
 * The slots, positions and block tables of the calls above index a paged KV cache; these calls
 * write, read and attend to one. Conventions for all of them:
 *   - A page is block_size tokens, a power of two from 8 to 128. K and V hold one e4m3 byte for
 *     each value: value d of head h of slot t of page b is at
 *     b*st_block + t*st_tok + h*st_head + d of k_cache and of v_cache (strides in elements; base
 *     addresses 16-byte aligned, strides multiples of 16). D is a multiple of 16 from 16 to 128,
 *     Hkv at most 2^22.
 *   - k_scale and v_scale [num_blocks, Hkv] fp32 hold one scale for each page and head: the byte q
 *     stands for e4m3(q) * scale. sd_kv_write makes powers of two, so that every product with a
 *     scale is exact; reads take any positive scale (sd_kv_attend V scales from 2^-100 to 2^120, which
 *     holds all that sd_kv_write makes). A scale of 0 means that the page holds zeros (a cache may
 *     start as zeroed memory, or as any with zeroed scales).
 *   - block_table [B, max_blocks] as for sd_pdraft_expand: position p of request r is slot
 *     p % block_size of page block_table[r][p / block_size].
 */

/*
 * sd_kv_write -- quantise the K and V of n tokens into the pages that slot_mapping names.
 *
 * Token i goes to slot s = slot_mapping[i]: page s / block_size, offset s % block_size; a
 * negative slot (PADDING_SLOT_ID: rejected and padding tokens) is skipped, one beyond the cache
 * too, with SD_ERR_KV_SLOT. For each page that receives tokens, and each head of K and of V:
 *   need  = the smallest power of two, 2^-100 at the least, with |x| <= 448 need for every finite
 *           value x that the call writes to the page;
 *   scale = max(old scale, need), the old scale counting as 0 when the call writes the page's
 *           slot 0 (the page then starts afresh: pages fill in order, so what a rewound or reused
 *           page held before is void; a page given to a new owner is therefore first written with its
 *           slot 0 among the tokens, or has its scales set to 0);
 *   the tokens written become e4m3(x / scale), to nearest even; infinities become +-448, NaN stays
 *   NaN; when the scale grew, what the page's other slots hold is rounded again to the new scale:
 *   e4m3(held * old / scale).
 * The tokens of one page stand next to one another in slot_mapping, up to 31 skipped entries in a
 * row between them (the slots of a request's consecutive positions do); of tokens with the same
 * slot the last is kept. Two stretches of the same page in one call race on its scale.
 * Arguments: k, v: bf16, value d of head h of token i at i*ld + h*hs + d (16-byte aligned,
 *   strides multiples of 8; they may be slices of one projection); slot_mapping [n] int32;
 *   num_blocks*block_size <= 2^31; n <= 2^31 - 1024.
 */
SD_API int sd_kv_write(int n, int Hkv, int D, const void* k, long ld_k, long hs_k, const void* v,
                       long ld_v, long hs_v, const int32_t* slot_mapping, void* k_cache,
                       void* v_cache, long st_block, long st_tok, long st_head, float* k_scale,
                       float* v_scale, int num_blocks, int block_size, int32_t* err,
                       void* stream);

/*
 * sd_kv_read -- what the cache holds, as bf16 rows.
 *
 * Row i of k_out and v_out, cu_tokens[r] <= i < cu_tokens[r+1], is request r's token at position
 * first_pos[r] + i - cu_tokens[r] (first_pos NULL: 0): e4m3(q) * scale rounded to bf16 (exact for
 * power-of-two scales, unless it leaves bf16's range). Rows outside [cu_tokens[0], cu_tokens[B])
 * are not written; a position that the table does not cover reads as 0 with SD_ERR_KV_RANGE.
 * Arguments: n rows, n <= 2^31 - 1024; cu_tokens [B+1], non-decreasing; k_out, v_out bf16, value d
 *   of head h of row i at i*ld_out + h*hs_out + d (16-byte aligned, strides multiples of 8).
 */
SD_API int sd_kv_read(int B, int n, int Hkv, int D, const void* k_cache, const void* v_cache,
                      long st_block, long st_tok, long st_head, const float* k_scale,
                      const float* v_scale, int num_blocks, int block_size,
                      const int32_t* block_table, int max_blocks, const int32_t* cu_tokens,
                      const int32_t* first_pos, void* k_out, void* v_out, long ld_out,
                      long hs_out, int32_t* err, void* stream);

/*
 * sd_kv_attend -- attention of each request's new tokens to its cached ones.
 *
 * Request r has the query tokens cu_q[r] .. cu_q[r+1]-1 of q (n_r of them: K+1 verify slots, a
 * drafter batch's a_r + K slots, one token, a chunk of a prompt) and ctx_lens[r] tokens in the
 * cache, its own new ones included (sd_kv_write before this call). Query token i of the request
 * stands at position ctx_lens[r] - n_r + i and, when causal, sees the tokens up to its own
 * position; else all ctx_lens[r]. Head h of Hq reads head h / (Hq / Hkv) of the cache.
 *   S = sm_scale * q . k,  out = sum_j softmax(S)_j v_j,  lse = ln sum_j e^(S_j)
 * q is taken exactly but for what lies below 2^-17 of its largest magnitude; exponentials, sums
 * and products are fp32; out is rounded to bf16 once. The weights of v have 8 significant bits. Among
 * 128 neighbouring tokens, weights far below the largest can have fewer, in steps of 2^-7 of it,
 * but keep 3 down to 2^-12 of it; beside a token that dominates the row the steps are 2^-19 of its
 * weight, and 3 bits are kept down to 2^-24 of it. So the rest of a long context counts to 8 bits
 * against a dominant token, too. The V scales of the pages that one token sees lie within 2^80 of
 * one another (a scale of 0 counts as 2^-60). A token that sees nothing gets out = 0 and lse =
 * -inf. NaN in tokens that a query token does not see has no effect on it, nor have the other
 * queries of the request. The same call gives the same bits: parts of a request are joined in a
 * fixed order.
 * A table entry outside [0, num_blocks) or a length outside [0, max_blocks*block_size] (or beyond
 * 2^31 - 256) raises SD_ERR_KV_RANGE; those tokens are left out. cu_q has B+1 non-decreasing entries
 * in [0, n] (others are clamped, SD_ERR_KV_RANGE); tokens outside [cu_q[0], cu_q[B]) are not written.
 * Arguments: q, out bf16, value d of head h of token i at i*ld + h*hs + d (16-byte aligned,
 *   strides multiples of 8); lse [n, Hq] fp32 or NULL; max_q: the most query tokens that a request
 *   is expected to have, which only chooses the kernel (any value >= 1 is right); Hq a multiple of
 *   Hkv; n*Hq and B <= 2^31 - 1024; num_blocks >= 1; sm_scale positive and finite; workspace: at
 *   least sd_kv_attend_workspace_bytes(D) bytes of device scratch, 16-byte aligned, its contents
 *   irrelevant before and after. Calls that may run concurrently need separate workspaces.
 */
SD_API int sd_kv_attend(int B, int n, int max_q, int Hq, int Hkv, int D, const void* q, long ld_q,
                        long hs_q, const void* k_cache, const void* v_cache, long st_block,
                        long st_tok, long st_head, const float* k_scale, const float* v_scale,
                        int num_blocks, int block_size, const int32_t* block_table,
                        int max_blocks, const int32_t* ctx_lens, const int32_t* cu_q,
                        float sm_scale, int causal, void* out, long ld_out, long hs_out,
                        float* lse, void* workspace, size_t workspace_bytes, int32_t* err,
                        void* stream);

/* Scratch of sd_kv_attend, where the parts of a request that several CTAs share wait to be joined
 * (it does not depend on the batch). */
SD_API size_t sd_kv_attend_workspace_bytes(int D);

/*
 * sd_kv_weights -- the attention weight that each cached token gets from a call's queries.
 *
 * Queries, lengths and cache as for sd_kv_attend, whose lse is an input: of the query tokens of
 * request r the first live[r] count (NULL: all; sd_verify's num_accepted + 1 leaves rejected drafts
 * out). For each KV head h and token t < ctx_lens[r]:
 *   w = sum over the tokens i that count and see t, and the heads of h's group, of
 *       e^(sm_scale q_i . k_t - lse_i)
 *   weights[t] = w                      for the request's own new tokens, or without `before`
 *   weights[t] = w + decay * before[t]  for the others
 * so that a token's number starts afresh in the call that brings it. weights and before are fp32
 * [num_blocks, Hkv, block_size], as the cache's pages lie; before may be weights itself (and else
 * shares nothing with it). Numbers of other slots are not written. A token whose page is not in the
 * table is left out (SD_ERR_KV_RANGE, as for ctx_lens, cu_q and a live[r] outside [0, n_r], which are
 * clamped). Rows with lse = -inf that see nothing add nothing. The same call gives the same bits; sums are fp32, q as for sd_kv_attend.
 * Arguments: as for sd_kv_attend; lse [n, Hq] fp32; decay finite and >= 0; B and Hkv at most 65535.
 *   Requests that share a page of the table race on its numbers.
 */
SD_API int sd_kv_weights(int B, int n, int max_q, int Hq, int Hkv, int D, const void* q, long ld_q,
                         long hs_q, const float* lse, const void* k_cache, long st_block,
                         long st_tok, long st_head, const float* k_scale, int num_blocks,
                         int block_size, const int32_t* block_table, int max_blocks,
                         const int32_t* ctx_lens, const int32_t* cu_q, const int32_t* live,
                         float sm_scale, int causal, float decay, const float* before,
                         float* weights, int32_t* err, void* stream);

/*
 * sd_kv_evict -- a cache cut to a budget of tokens a request, by their weights.
 *
 * A request of more than `budget` tokens keeps the first `sink`, the last `recent`, and of those
 * between them the ones with the largest weights (equal ones: the earlier; a NaN before all), so that
 * `budget` stay, in their order. Every KV head chooses for itself: slot j of head h then holds its
 * j-th token that stays. Shorter requests keep all.
 *   kept[r][h][j] = the position that the j-th token had, -1 from new_lens[r] on
 *   new_lens[r]   = min(ctx_lens[r], budget)
 * The tokens' K, V and weights move to the pages that to_table lists (fresh ones: none of any
 * request's table), or, to_table NULL, to the request's own from the first on (its pages not shared
 * with another request; those behind new_lens are then free). A page's new scale is the largest of its
 * tokens' old ones; a value becomes e4m3(held * old / new), to nearest even: unchanged but for what
 * becomes subnormal. Pages and slots behind new_lens, and a table's pages that tokens leave, stay as they
 * are. A position that a table does not cover raises SD_ERR_KV_RANGE: as a source it holds weight 0
 * and zeros, as a place it is not written; lengths beyond the table are clamped, with the bit.
 * Rotated keys keep the angle of the position they had: new tokens go on with positions of the text,
 * while slots, ctx_lens and sd_kv_attend's causal order go by place.
 * Arguments: cache as for sd_kv_write; weights fp32 [num_blocks, Hkv, block_size]; kept [B, Hkv,
 *   budget] and new_lens [B] int32 outputs, apart from each other, ctx_lens and the tables; budget >= 1;
 *   sink, recent >= 0, sink + recent <= budget; to_table [B, to_blocks], apart from block_table (in place:
 *   NULL); k_cache is not v_cache, nor k_scale v_scale, but for one cache and its scales given twice with
 *   to_table; B and Hkv at most 65535.
 */
SD_API int sd_kv_evict(int B, int Hkv, int D, void* k_cache, void* v_cache, long st_block,
                       long st_tok, long st_head, float* k_scale, float* v_scale, int num_blocks,
                       int block_size, float* weights, const int32_t* block_table, int max_blocks,
                       const int32_t* to_table, int to_blocks, const int32_t* ctx_lens, int budget,
                       int sink, int recent, int32_t* kept, int32_t* new_lens, int32_t* err,
                       void* stream);

/* ---- rotary positions ---- */
#define SD_ROPE_HALVES 0      /* pair i of a head: values i and i + rot / 2 */
#define SD_ROPE_NEIGHBOURS 1  /* pair i: values 2 i and 2 i + 1 */

/* frequencies of pair i, in radians a position; f_i = base^(-2 i / rot) */
#define SD_ROPE_PLAIN 0   /* f_i */
#define SD_ROPE_LINEAR 1  /* f_i / factor */
#define SD_ROPE_NTK 2     /* f_i of base * factor^(rot / (rot - 2)) */
#define SD_ROPE_BANDS 3   /* from f_i / factor to f_i as the turns over original_len go from low to high */
#define SD_ROPE_YARN 4    /* the same over the pairs between those that make `high` and `low` turns over
                             original_len (whole pairs), and a scale of 0.1 ln(factor) + 1 */

/*
 * sd_rope -- rotary positions of queries and keys.
 *
 * The first `rot` values of every head of token i turn by its position p = positions[i] (any int32):
 * with a = 2 pi p turns[j] / 2^64, pair j (x, y) becomes
 *   scale * (x cos a - y sin a),  scale * (y cos a + x sin a),
 * or, inverse, with -a and the same scale: the transposed map, which sends a gradient back (and, called
 * with 1 / scale, a rotated key to its unrotated one). The other values are copied. The angle is exact to 10^-7 at every position; values are fp32, rounded once.
 * Arguments: n >= 0 tokens, n <= 2^31 - 1024; Hq, Hk >= 0 heads of queries and keys (0: none; their
 *   pointers may then be NULL), Hq + Hk <= 2^20; D a multiple of 8 up to 512; rot even, 0 < rot <= D;
 *   pairs SD_ROPE_HALVES or SD_ROPE_NEIGHBOURS; turns [rot / 2] (sd_rope_table's, on the device); scale
 *   finite; q, k and their outputs bf16, value d of head h of token i at i*ld + h*hs + d (16-byte
 *   aligned, strides multiples of 8). An output may be its input itself, with the same strides, and
 *   else shares nothing with either input or the other output (slices of one array may lie side by side);
 *   no two of its own values share memory.
 */
SD_API int sd_rope(int n, int Hq, int Hk, int D, int rot, int pairs, const int32_t* positions,
                   const uint64_t* turns, float scale, int inverse, const void* q, long ld_q,
                   long hs_q, void* q_out, long ld_qo, long hs_qo, const void* k, long ld_k,
                   long hs_k, void* k_out, long ld_ko, long hs_ko, void* stream);

/*
 * sd_rope_table -- the turns a position of every pair as fractions of 2^64, and the scale, for
 * sd_rope. Host arithmetic: turns [rot / 2] and scale are HOST memory, and nothing is enqueued.
 * Arguments: rot even, 2..512; base > 1; kind SD_ROPE_*; factor > 0 (SD_ROPE_YARN: >= 1); original_len
 *   > 0 and 0 < low < high for SD_ROPE_BANDS and SD_ROPE_YARN (not looked at otherwise).
 */
SD_API int sd_rope_table(int rot, double base, int kind, double factor, double original_len,
                         double low, double high, uint64_t* turns, float* scale);

/* ---- rows cut by top-k, top-p and min-p ----
 *
 * A row's entries stand in order: larger first, equal ones by lower index. With their weights w (the
 * probabilities for SD_F32_PROBS; exp(l / T_r) for SD_BF16_LOGITS, T_r within 2^-100 and 2^100) those
 * kept are the first
 *   top_k[r] of them (<= 0: all),
 *   those of these before which less than top_p[r] of their sum lies (>= 1 or NaN: all),
 *   those with w >= min_p[r] w_max (<= 0 or NaN: all; above 1 as 1),
 * whichever is fewest, and the first entry always. T_r <= 0 (or NaN): the first entry alone. Entries of
 * weight 0 are never kept: probabilities <= 0, logits of -inf, all beside a +inf, and NaN. A
 * probability above 1 counts as 1. Which entries are kept, and which is drawn, is decided by sums that
 * are off by 2^-40 of the row's sum at most, however many entries and values there are. temperature,
 * top_k, top_p, min_p are [B] or NULL (1, and off).
 */
#define SD_CUT_MAX_V 524224

/*
 * sd_truncate -- rows cut as above, as probability rows: w / (the sum of those kept), else 0.
 *
 * The rows may serve as sd_verify's (target and draft rows cut by the same request's settings: the
 * answer is then distributed as the cut target rows), sd_draft_sample's or sd_token_logprobs's.
 * Arguments: B >= 0, J >= 1, 1 <= V <= SD_CUT_MAX_V; rows [B*J, V] of stride ld >= V (row r*J + j is
 *   request r's); probs [B*J, V] fp32 of stride ld_out >= V; kept [B, J] int32 or NULL: how many entries
 *   are kept; outputs in memory apart from each other, the rows and the settings. A row that keeps none:
 *   zeros, kept 0, SD_ERR_ZERO_ROW. B*J <= 2^27.
 */
SD_API int sd_truncate(int B, int J, int V, int dtype, const void* rows, long ld,
                       const float* temperature, const int32_t* top_k, const float* top_p,
                       const float* min_p, float* probs, long ld_out, int32_t* kept, int32_t* err,
                       void* stream);

/*
 * sd_sample -- one token drawn from each row cut as above, by a given random number.
 *
 * tokens[r][j] = the first entry, in the order above, up to and with which more than u[r][j] of the
 * sum of those kept lies (u taken within [0, 1]; NaN as 0).
 * Arguments: as for sd_truncate; u [B, J] fp32; tokens [B, J] int32; prob [B, J] fp32 or NULL: the
 *   token's probability among those kept (it may be u itself; outputs share nothing else). A row that
 *   keeps none: token 0, prob 0, SD_ERR_ZERO_ROW.
 */
SD_API int sd_sample(int B, int J, int V, int dtype, const void* rows, long ld,
                     const float* temperature, const int32_t* top_k, const float* top_p,
                     const float* min_p, const float* u, int32_t* tokens, float* prob,
                     int32_t* kept, int32_t* err, void* stream);

/*
 * sd_token_logprobs -- log probabilities of given tokens (a step's answer: sd_verify's
 * out_tokens on its target rows), with each row's entropy and best alternatives.
 *
 * Row r*J + j of rows belongs to tokens[r][j] (J = K+1 for sd_verify's outputs). SD_F32_PROBS:
 * p = the row. SD_BF16_LOGITS: p = softmax(l / T_r), T_r = temperature[r], taken within 2^-100 and
 * 2^100 (NULL, or 0: 1; a greedy request is reported at temperature 1).
 *   logprob[r][j] = ln p(token)
 *   entropy[r][j] = -sum p ln p
 *   rank[r][j]    = 1 + the entries that come before the token, larger ones first, equal ones by
 *                   lower index
 *   top_ids, top_logprobs [r][j][0..n_top): the first n_top entries in that order.
 * A row without a token (tokens -1, sd_verify's padding) is not read: logprob 0, entropy 0, rank 0,
 * top_ids -1, top_logprobs -inf. A token outside [-1, V) raises SD_ERR_TOKEN_RANGE: logprob -inf and
 * rank 0 for one >= V, a negative one counts as none.
 * Arguments: B >= 0, J >= 1, 1 <= V <= SD_TOP_MAX_V; rows [B*J, V] of stride ld >= V;
 *   0 <= n_top <= min(V, SD_TOP_MAX); entropy, rank may be NULL; top_ids and top_logprobs may be
 *   NULL if n_top is 0.
 */
#define SD_TOP_MAX 32
#define SD_TOP_MAX_V 33554432
SD_API int sd_token_logprobs(int B, int J, int V, int dtype, const void* rows, long ld,
                             const int32_t* tokens, const float* temperature, int n_top,
                             float* logprob, float* entropy, int32_t* rank, int32_t* top_ids,
                             float* top_logprobs, int32_t* err, void* stream);

/* ---- diagnostics (test support; same conventions) ---- */

/* Philox4x32-10 of n counters ctr[n][4] under key (seed lo, seed hi) -> out[n][4]. */
SD_API int sd_philox_words(int n, const uint32_t* ctr, uint64_t seed, uint32_t* out, void* stream);

/* The race variates E = fp32(-log((w + 0.5) * 2^-32)) of n words w[n] -> E[n] (the exact path
 * the kernels use). */
SD_API int sd_race_E(int n, const uint32_t* w, float* E, void* stream);

/* Worst relative error, over every w in [w_begin, w_begin + count), of the fast approximation
 * the race filter uses for -log(v) against the exact E above. Writes max_rel[0] (fp32,
 * caller-zeroed) with atomicMax on the float bits. */
SD_API int sd_race_E_approx_error(uint32_t w_begin, uint64_t count, float* max_rel, void* stream);

/* Bit-exactness check of the exact race variate: the kernels evaluate E from pairs of fp32 and
 * take the double path only near an fp32 rounding boundary. Over every w in
 * [w_begin, w_begin + count) adds to counts[0] (uint64, caller-zeroed) the words whose E differs
 * from the double path's fp32(-log((w + 0.5) * 2^-32)), and to counts[1] the words that took
 * the double path. */
SD_API int sd_race_E_check(uint32_t w_begin, uint64_t count, uint64_t* counts, void* stream);

/* sd_verify_prepare with its single launch's wait made to run out (test support for the
 * bounded wait; same arguments from B on): in the single launch, request withhold_request's
 * rebuild CTA publishes its first drafter slot only after the CTA completing that request's race
 * row has polled for wait_us microseconds (1..10^6) of the GPU clock and given up, so that the
 * call raises SD_ERR_WAIT and leaves that request's final token unwritten in input_ids while
 * every other output matches sd_verify_prepare's. Batches that take two kernels run as
 * sd_verify_prepare does (they have no wait). Returns SD_E_SHAPE for a request outside [0, B) or
 * wait_us outside the range. */
SD_API int sd_diag_verify_prepare_withheld(
    int withhold_request, uint32_t wait_us, int B, int K, int V, int dtype, const void* target,
    long ld_t, const void* draft, long ld_d, const int32_t* drafts, const float* temperature,
    uint64_t seed, uint32_t request_base, int32_t* out_tokens, int32_t* num_accepted,
    float* p_at_draft, float* q_at_draft, const int32_t* pos0, const int32_t* block_table,
    int max_blocks, int block_size, int32_t mask_token_id, int capacity, int32_t* input_ids,
    int32_t* positions, int32_t* slot_mapping, int32_t* hidden_map, uint8_t* is_masked,
    uint8_t* is_rejected, int32_t* start_loc, int32_t* new_token_idx, int32_t* total_out, int H,
    const void* target_hidden, long ld_in, int n_in_rows, const void* h_shared, void* out_hidden,
    long ld_out, void* workspace, size_t workspace_bytes, int32_t* err, void* stream);

/* Text for a status code (static storage). */
SD_API const char* sd_status_string(int status);

/* Library version (major * 100 + minor). */
SD_API int sd_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SD_GB300_H */

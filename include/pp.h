/*
 * pp.h - C ABI of libpp, exact softmax attention over a preference-packed sequence on B200 (sm_100a).
 *
 * Problem (pages: "Preference Packing: Efficient Preference Optimization for LLMs", abstract and method digest;
 * "prefix_grouper_utils.py", section 1 building position ids, section 2 building the grouper, and the
 * prefix-sharing diagram; "PackInfer: Compute- and I/O-Efficient Attention for Batched LLM Inference", abstract):
 * a batch of G groups is packed into one flat sequence of T tokens. Group g stores its prompt prefix P_g once,
 * followed by its k_g responses S_g1..S_gk. A prefix token attends causally within the prefix; a token of S_i
 * attends to the whole prefix and causally within S_i, never to a sibling response or to another group. Position
 * ids run 0..P_g-1 on the prefix and restart at P_g for every response.
 *
 * Conventions for every call
 *   - Ownership: the caller owns all memory. The library allocates nothing on the device or the host (apart from a
 *     few small static tables of its own); every buffer is passed in as a raw pointer with its size.
 *   - Pointers: "_d" names and every tensor argument are DEVICE pointers on the current CUDA device, except where a
 *     comment says host, aligned to their elements where nothing more is asked. Tensors are dense and row-major:
 *       Q, O, dO, dQ: [T, Hq, d]; K, V, dK, dV: [T, Hkv, d]; LSE: [Hq, T] fp32; pos ids: int32 [T].
 *     The packed order is group by group: prefix, then the responses in order.
 *   - Asynchrony: every call only enqueues work on `stream` (a cudaStream_t; NULL = legacy default stream) and
 *     returns without synchronising, except pp_get_status().
 *   - Errors: arguments are validated on the host before anything is enqueued; an invalid argument returns
 *     PP_ERR_INVALID_ARG (or PP_ERR_UNSUPPORTED / PP_ERR_WORKSPACE) and enqueues nothing. A failed launch returns
 *     PP_ERR_CUDA. Problems only the device can see (inconsistent descriptors, a bounded wait that ran out) set a
 *     device error word that pp_get_status() reads. pp_last_error() returns a message for the calling thread.
 *   - Limits: T < 2^31 - 256; d in {64, 128}; Hq % Hkv == 0; Hq <= 256.
 */
#ifndef PP_H_
#define PP_H_

#include <stdint.h>

#if defined(__GNUC__)
#define PP_API __attribute__((visibility("default")))
#else
#define PP_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    PP_OK = 0,
    PP_ERR_INVALID_ARG = -1,   /* host-side validation failed; nothing was enqueued */
    PP_ERR_UNSUPPORTED = -2,   /* valid but unsupported combination (e.g. backward in fp32) */
    PP_ERR_CUDA = -3,          /* a CUDA runtime/driver call failed */
    PP_ERR_DEVICE_TIMEOUT = -4,/* a kernel's bounded wait ran out (reported by pp_get_status) */
    PP_ERR_WORKSPACE = -5,     /* a buffer is smaller than the size the library asked for */
    PP_ERR_DEVICE_INPUT = -6   /* the device found inconsistent descriptors (reported by pp_get_status) */
} pp_status;

/* PP_E4M3 and PP_INT8 are the codes of a paged cache (pp_cache_store); every other argument takes the first two. */
typedef enum { PP_BF16 = 0, PP_FP32 = 1, PP_E4M3 = 2, PP_INT8 = 3 } pp_dtype;

/* One group's descriptor ("prefix_grouper_utils.py" section 1: each group carries its prefix length and its
 * responses' lengths). The response lengths themselves are the segments of cu_seqlens. */
typedef struct {
    int32_t prefix_len;    /* P_g >= 0 */
    int32_t num_suffixes;  /* k_g >= 0 */
} pp_group_desc;

/* Which pass a workspace size is asked for. */
enum { PP_PASS_FWD = 0, PP_PASS_BWD = 1 };

/* ---------------------------------------------------------------------------------------------------------------
 * pp_meta_bounds (host only, no device work)
 * Upper bound on the bytes of the metadata buffer that pp_build_meta fills, from the sizes alone.
 *   num_groups G >= 1, num_segments = sum_g (1 + k_g), total_tokens T >= 0, num_heads_q / num_heads_kv as for the
 *   attention calls. *meta_bytes (host pointer) receives the size. Errors: PP_ERR_INVALID_ARG.
 */
PP_API pp_status pp_meta_bounds(int32_t num_groups, int32_t num_segments, int64_t total_tokens, int32_t num_heads_q,
                         int32_t num_heads_kv, int64_t *meta_bytes);

/* ---------------------------------------------------------------------------------------------------------------
 * pp_build_meta: group descriptors + segment boundaries -> grouped position ids and the tile schedule.
 * ("prefix_grouper_utils.py" section 1 for the position ids; "PackInfer" abstract for building the attention work
 * directly over the packed query-key regions and balancing it across thread blocks.)
 *   groups_d      device pp_group_desc[num_groups]
 *   cu_seqlens_d  device int32[num_segments + 1]: packed segment boundaries in the packed order (for each group its
 *                 prefix, then each response); zero-length segments allowed. cu[0] must be 0, cu[nseg] must be T,
 *                 and num_segments must equal sum_g (1 + k_g); a violation found on the device sets
 *                 PP_ERR_DEVICE_INPUT (pp_get_status) and leaves the outputs undefined.
 *   pos_ids_d     device int32[T] out: position ids (prefix 0..P-1, every response restarts at P).
 *   meta_d        device buffer out, meta_bytes >= the pp_meta_bounds value, 256-byte aligned. Its content is
 *                 private to the library (read it only through the calls below); it holds the per-token segment
 *                 table, the forward query tiles (128 rows, aligned to each group's start) in cost order, and the
 *                 backward key/value tiles (128 rows) split into work chunks in cost order.
 * The buffers must stay alive and unchanged while attention calls that use them are in flight.
 */
PP_API pp_status pp_build_meta(const pp_group_desc *groups_d, int32_t num_groups, const int32_t *cu_seqlens_d,
                        int32_t num_segments, int64_t total_tokens, int32_t num_heads_q, int32_t num_heads_kv,
                        int32_t *pos_ids_d, void *meta_d, int64_t meta_bytes, void *stream);

/* ---------------------------------------------------------------------------------------------------------------
 * pp_meta_tiles: expand the schedule in meta_d into explicit tiles, for checking and inspection.
 *   which = PP_PASS_FWD: query tiles of 128 rows x key tiles of 128 rows; PP_PASS_BWD: key tiles of 128 rows x
 *   query tiles of 128 rows. Both are aligned to each group's start. Writes one int32 triple
 *   (q_row0, kv_row0, class) per non-empty tile into tiles_d (device int32[3 * capacity]), class 1 = every pair in
 *   the tile allowed (FULL), 2 = some allowed (PARTIAL); fully masked tiles are never listed. *count_d (device
 *   int32) receives the number of tiles (possibly > capacity; only the first `capacity` are written). The order is
 *   unspecified. The classification is the same device code the attention kernels use.
 */
PP_API pp_status pp_meta_tiles(const void *meta_d, int32_t which, int32_t *tiles_d, int64_t capacity, int32_t *count_d,
                        void *stream);

/* ---------------------------------------------------------------------------------------------------------------
 * pp_meta_schedule: the work lists the attention kernels execute, in their stored order, for checking.
 * ("PackInfer" abstract: attention work over the packed query-key regions, ordered to balance the thread blocks.)
 *   which = PP_PASS_FWD: the forward query tiles in cost order (the order pp_attn_fwd and the dQ half of
 *   pp_attn_bwd walk them); one record per key tile a query tile visits. which = PP_PASS_BWD: the backward work
 *   chunks (key tile x a range of its query tiles) in their stored order; one record per query tile of a chunk.
 *   Each record is five int32 (item, q_row0, kv_row0, class, split): item = position of the query tile (fwd) or of
 *   the chunk (bwd) in its list; class 1 = FULL, 2 = PARTIAL; split = 1 if the chunk's key tile is split over
 *   several chunks (its dK/dV partials are added in fp32), else 0 (always 0 for fwd). records_d: device
 *   int32[5 * capacity]; *count_d (device int32) receives the number of records (only the first `capacity` are
 *   written). The order of the records is unspecified; their item fields give the stored order.
 */
PP_API pp_status pp_meta_schedule(const void *meta_d, int32_t which, int32_t *records_d, int64_t capacity,
                                  int32_t *count_d, void *stream);

/* ---------------------------------------------------------------------------------------------------------------
 * pp_rope: rotary embedding at the grouped position ids, in place on q and k (v untouched).
 * Rotate-half form with base theta: for m < d/2, w_m = theta^(-2m/d), a = pos * w_m,
 *   y_m = x_m cos a - x_{m+d/2} sin a,  y_{m+d/2} = x_{m+d/2} cos a + x_m sin a
 * (the pages give the positions, "prefix_grouper_utils.py" section 1, but not the variant; rotate-half is the
 * reading taken). inverse != 0 rotates by -a, which maps gradients of the rotated tensors back.
 *   q: [T, hq, d], k: [T, hkv, d] (either may be NULL to skip it), dt = PP_BF16 or PP_FP32 storage; the angle is
 *   formed in fp64 and the rotation in fp32, rounded to nearest even on store. theta > 0 (0 means 10000).
 */
PP_API pp_status pp_rope(void *q, void *k, const int32_t *pos_ids_d, int64_t T, int32_t hq, int32_t hkv, int32_t d,
                  float theta, pp_dtype dt, int32_t inverse, void *stream);

/* ---------------------------------------------------------------------------------------------------------------
 * pp_workspace_bytes (host only): scratch bytes pp_attn_fwd (which = PP_PASS_FWD) or pp_attn_bwd
 * (PP_PASS_BWD) needs for these sizes. *bytes (host pointer) receives it.
 */
PP_API pp_status pp_workspace_bytes(int32_t which, int64_t T, int32_t hq, int32_t hkv, int32_t d, int64_t *bytes);

/* ---------------------------------------------------------------------------------------------------------------
 * pp_bwd_ds_bytes (host only): extra backward workspace, beyond pp_workspace_bytes(PP_PASS_BWD, ...), that lets
 * pp_attn_bwd keep one dS tile (128 keys x 128 queries, bf16, 32 KiB) per backward step and form dq from them
 * instead of recomputing the scores. A step is (key tile of 128 rows, query tile of 128 rows that attends it, q
 * head), for every kv head; the count follows the mask (same descriptors as pp_build_meta). groups_host,
 * cu_host: host copies of the descriptors and segment bounds; *bytes (host) receives 1024 + steps * 32768.
 * Returns PP_ERR_INVALID_ARG for descriptors that disagree with the segments or segment bounds that decrease.
 */
PP_API pp_status pp_bwd_ds_bytes(const pp_group_desc *groups_host, int32_t G, const int32_t *cu_host,
                                 int32_t nseg, int32_t hq, int32_t hkv, int64_t *bytes);

/* ---------------------------------------------------------------------------------------------------------------
 * pp_attn_fwd: O and the per-row log-sum-exp of exact packed attention.
 *   s_ij = softmax_scale * q_i . k_j over the allowed keys j of row i (q head h reads kv head h / (hq/hkv));
 *   lse_i = ln sum_j exp(s_ij) (natural log of the scaled scores); o_i = sum_j exp(s_ij - lse_i) v_j.
 *   q, k, v: inputs as above in dtype dt (PP_BF16: tcgen05 tensor-core path, fp32 accumulation;
 *   PP_FP32: fp32 CUDA-core path, meant for small checks). o: [T, hq, d] out in dt; lse: [hq, T] fp32 out.
 *   softmax_scale 0 means 1/sqrt(d). meta_d from pp_build_meta with the same T, hq, hkv.
 *   workspace: device scratch of ws_bytes >= pp_workspace_bytes(PP_PASS_FWD, ...), 256-byte aligned; contents
 *   need not be initialised. Rows of fully masked positions do not exist (every row attends at least itself).
 */
PP_API pp_status pp_attn_fwd(const void *q, const void *k, const void *v, const void *meta_d, int64_t T, int32_t hq,
                      int32_t hkv, int32_t d, float softmax_scale, pp_dtype dt, void *o, float *lse,
                      void *workspace, int64_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------------------------------------------
 * pp_attn_bwd: gradients of sum(O * dO) with respect to q, k and v (bf16 only).
 *   D_i = dO_i . o_i; p_ij = exp(s_ij - lse_i); dS_ij = p_ij (dO_i . v_j - D_i);
 *   dq_i = scale sum_j dS_ij k_j; dk_j = scale sum_h sum_i dS_ij q_i; dv_j = sum_h sum_i p_ij dO_i
 *   (sums over the q heads h that share kv head j's head). q, k, v, o, lse: the forward's inputs and outputs;
 *   dout: [T, hq, d]. dq, dk, dv: outputs in bf16 with the shapes of q, k, v (fully overwritten).
 *   workspace: ws_bytes >= pp_workspace_bytes(PP_PASS_BWD, ...), 256-byte aligned, contents need not be
 *   initialised. It holds (-lse/scale, -D) per row and q head, and fp32 dK/dV for the prefix key tiles, which are
 *   attended by every response of their group and so are split into chunks whose partials are added there (fp32
 *   reduction adds, one per element and chunk) before conversion to bf16. Each row tile of dq is produced by exactly
 *   one CTA (no reduction). If ws_bytes also covers pp_bwd_ds_bytes(...) for the batch, the dK/dV kernel keeps
 *   every step's dS tile after the base workspace and dq is formed from them (the fast path); otherwise the dq
 *   kernel recomputes the tile's scores and dP. The choice is made on the device from the batch's step count, so
 *   either size is valid. A batch of T tokens that could exceed 2^31 - 1 steps per kv head (about 4.2 M tokens at
 *   hq/hkv = 4) always takes the recompute path. The result is deterministic except for the order of the dK/dV adds.
 */
PP_API pp_status pp_attn_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                      const void *dout, const void *meta_d, int64_t T, int32_t hq, int32_t hkv, int32_t d,
                      float softmax_scale, void *dq, void *dk, void *dv, void *workspace, int64_t ws_bytes,
                      void *stream);

/* ---------------------------------------------------------------------------------------------------------------
 * pp_attn_bwd_noalloc: pp_attn_bwd for callers that cannot allocate device memory.
 * (The paper has no counterpart; this is a convenience of the library.)
 * Some callers cannot call cudaMalloc or ask anyone for a scratch buffer: a plugin or custom op handed only its
 * input and output pointers by a host framework whose caching allocator owns the device memory, or code that must
 * not allocate at that point. This entry point takes the same arguments as pp_attn_bwd minus the workspace, and
 * uses instead a scratch array compiled into the library (a file-scope __device__ array of
 * PP_NOALLOC_SCRATCH_BYTES = 64 MiB; every GPU that loads libpp holds it until the process exits). It calls no
 * allocator at all.
 *   Limit: the scratch a call needs (pp_workspace_bytes(PP_PASS_BWD, T, hq, hkv, d)) must fit in 64 MiB, e.g.
 *   T <= about 7,600 tokens at 32/8 heads and d = 128; a larger call returns PP_ERR_WORKSPACE and enqueues nothing.
 *   Set-up: the first call on each device looks up the array's device address (cudaGetSymbolAddress) with that
 *   device current; make that first call before any stream capture.
 *   Sharing: every call on a device uses the same array, which keeps the last call's contents; the call clears the
 *   parts that must start at zero itself. Calls that overlap on the GPU (other streams, other host threads) race
 *   on the array: serialise them.
 */
#define PP_NOALLOC_SCRATCH_BYTES (64ll << 20)
PP_API pp_status pp_attn_bwd_noalloc(const void *q, const void *k, const void *v, const void *o, const float *lse,
                              const void *dout, const void *meta_d, int64_t T, int32_t hq, int32_t hkv, int32_t d,
                              float softmax_scale, void *dq, void *dk, void *dv, void *stream);

/* ---------------------------------------------------------------------------------------------------------------
 * pp_decode_attn: one decoding step of every response over a group-contiguous KV cache.
 * The cache holds the packed layout of pp_build_meta (each group's prefix rows, then each response's rows), the
 * newest token of each response last. Each response has one query (its newest token), which attends to its group's
 * prefix and its own rows, the packed mask at the response's last row ("PackInfer" abstract: group-contiguous KV
 * and attention over packed query-key regions; "Preference Packing": the prompt is shared by its responses).
 * A prefix chunk is read from HBM once per group and serves all of the group's responses (flash-decoding in
 * 128-key chunks on the tensor cores: the chunk's queries, every response that sees it times the r q heads of a kv
 * head, form the rows of S = Q K^T and O = P V; fp32 partials are combined per query). hq / hkv <= 128.
 *   q: [n_resp, hq, d] bf16, n_resp = num_segments - num_groups (responses in packed order). k_cache, v_cache:
 *   [T, hkv, d] bf16. groups_d, cu_d: the device descriptors and segment bounds of the cache (as for
 *   pp_build_meta; every response of nonzero length has its query's K/V as its last row). d = 128.
 *   o: [n_resp, hq, d] bf16; lse: [hq, n_resp] fp32 (natural log); a response with no keys gets 0 and -inf.
 *   workspace: ws_bytes >= pp_decode_workspace_bytes for the same descriptors, 256-byte aligned. Descriptors that
 *   disagree with T, num_segments or the sized workspace set PP_ERR_DEVICE_INPUT and yield NaN outputs.
 */
PP_API pp_status pp_decode_workspace_bytes(const pp_group_desc *groups_host, int32_t num_groups,
                                           const int32_t *cu_seqlens_host, int32_t num_segments, int32_t num_heads_q,
                                           int64_t *bytes);
PP_API pp_status pp_decode_attn(const void *q, const void *k_cache, const void *v_cache, const pp_group_desc *groups_d,
                                int32_t num_groups, const int32_t *cu_seqlens_d, int32_t num_segments, int64_t T,
                                int32_t hq, int32_t hkv, int32_t d, float softmax_scale, void *o, float *lse,
                                void *workspace, int64_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------------------------------------------
 * pp_qk_norm_rope: RMS norm of every query and key head and the rotation of pp_rope in one pass.
 *   r = (mean_i x_i^2 + eps)^-1/2 over a row of d elements (one token, one head); z_i = x_i r w_i; the row is then
 *   rotated at the token's position as by pp_rope (inverse = 0). The norm is formed in fp32, the angle in fp64, and
 *   the result is rounded once, to nearest even. Squares and their sum are fp32: a row whose sum passes its range (elements
 *   of some 10^18 and more) gives zeros; with eps = 0 rows of elements below 10^-19 lose bits, and zeros give NaN.
 *   q: T tokens of [hq, d], k: T tokens of [hkv, d], dt PP_BF16 or PP_FP32; q_stride and k_stride are the elements
 *   from one token to the next (hq * d and hkv * d for a dense tensor; more for the heads of a fused projection), a
 *   multiple of 16 bytes. q_out, k_out likewise with qo_stride, ko_stride; an output may be its input (same pointer
 *   and stride) but may not overlap it otherwise. q or k may be NULL to skip that side. wq, wk: [d] in dt, shared by
 *   the side's heads, or NULL for ones. eps >= 0; theta > 0 (0 means 10000). Tensors are 16-byte aligned.
 */
PP_API pp_status pp_qk_norm_rope(const void *q, const void *k, int64_t q_stride, int64_t k_stride, const void *wq,
                                 const void *wk, const int32_t *pos_ids_d, int64_t T, int32_t hq, int32_t hkv,
                                 int32_t d, float eps, float theta, pp_dtype dt, void *q_out, void *k_out,
                                 int64_t qo_stride, int64_t ko_stride, void *stream);

/* pp_qk_norm_rope_bwd: its gradients. With g the gradient of an output row, dz the row g rotated back and
 * e_i = dz_i w_i: dx_i = r (e_i - x_i r mean_j(e_j x_j r)), dw_i = sum over tokens and heads of dz_i x_i r.
 *   q, k, wq, wk, pos_ids_d, eps, theta: the forward's. gq, gk: gradients of q_out and k_out with their token
 *   strides; dq, dk: gradients of q and k (dt), with theirs; dq may be gq itself (same pointer and stride). dwq, dwk:
 *   fp32 [d] out, or NULL. The sums are fp32 in an order that the sizes alone fix, so a call repeats bit for bit.
 *   workspace: device scratch of ws_bytes >= pp_qk_norm_rope_bwd_bytes (host only, from the sizes), 256-byte aligned,
 *   contents need not be initialised.
 */
PP_API pp_status pp_qk_norm_rope_bwd_bytes(int64_t T, int32_t hq, int32_t hkv, int32_t d, int64_t *bytes);
PP_API pp_status pp_qk_norm_rope_bwd(const void *q, const void *k, int64_t q_stride, int64_t k_stride, const void *wq,
                                     const void *wk, const int32_t *pos_ids_d, int64_t T, int32_t hq, int32_t hkv,
                                     int32_t d, float eps, float theta, pp_dtype dt, const void *gq, const void *gk,
                                     int64_t gq_stride, int64_t gk_stride, void *dq, void *dk, int64_t dq_stride,
                                     int64_t dk_stride, float *dwq, float *dwk, void *workspace, int64_t ws_bytes,
                                     void *stream);

/* ---------------------------------------------------------------------------------------------------------------
 * The paged cache: the packed layout's segments (each group's prefix, then its responses) held in pages, so that a
 * response can grow without moving its neighbours and a prefix is still stored once for its group.
 *   A page holds page_size tokens (16, 32, 64 or 128) of every kv head, as 8-bit codes (codes = PP_E4M3 or PP_INT8):
 *     k_pages [num_pages, hkv, page_size, 128],  v_pages [num_pages, hkv, 128, page_size]  (values transposed),
 *     k_scale, v_scale fp32 [num_pages, hkv]: one scale for each block of page_size tokens of one head.
 *   An element is its code times its block's scale. Segment s owns row s of the page table, int32 [num_segments,
 *   max_pages]: the token at place t of the segment lies in page table[s][t / page_size] at offset t % page_size, and
 *   its slot is page * page_size + offset. Entries past a segment's last page are not read.
 *   The groups are given by group_start_d, int32 [num_groups + 1] (segment group_start[g] is group g's prefix and
 *   the ones up to group_start[g + 1] its responses; group_start[0] = 0 and group_start[num_groups] = num_segments)
 *   and seg_group_d, int32 [num_segments], each segment's group. num_segments <= 8192.
 *   Lengths, page ids or slots that do not fit are found on the device, never followed out of bounds, and reported
 *   by pp_get_status as PP_ERR_DEVICE_INPUT.
 *
 * pp_pages_resize: give pages to segments that grow, take them back from segments that shrink, and map the new
 * tokens to slots.
 *   old_lens_d, new_lens_d: int32 [num_segments], tokens before and after. page_table_d is updated in place: a
 *   growing segment's new pages are written after its ceil(old / page_size) ones; a shrinking segment's last pages go
 *   back to the pool (their entries stay). free_pages_d: int32 [num_pages], the first *n_free_in of them the free
 *   pages. Pages given back are put at its end in the order of (segment, place), then the pages needed are taken off
 *   its end in that order. *n_free_out receives the new count (n_free_out may be n_free_in).
 *   slots_d, pos_ids_d: int32 [capacity] out, one entry for each new token, segment by segment: its slot and its
 *   grouped position (place in a prefix; the prefix's new length plus its place in a response). Entries past the last
 *   new token get slot -1 (which pp_cache_store skips) and position 0. counts_d: int32 [4] out: new tokens, pages
 *   taken, pages given back, and 1.
 *   Where the pool has too few pages, the new tokens exceed `capacity`, a length is negative or exceeds
 *   max_pages * page_size, or a page to be given back is none of the pool's, nothing changes: counts are {0, 0, 0, 0},
 *   every slot -1, *n_free_out = *n_free_in, and pp_get_status reports it, the first two, which a server may meet at any
 *   time, by a message of their own. A free page, or a growing segment's last page, that is none of the pool's is
 *   reported too, but the change stands: its tokens get slot -1.
 *   max_pages * page_size <= 2^30; num_pages * page_size < 2^31.
 */
PP_API pp_status pp_pages_resize(const int32_t *group_start_d, int32_t num_groups, const int32_t *seg_group_d,
                                 int32_t num_segments, const int32_t *old_lens_d, const int32_t *new_lens_d,
                                 int32_t page_size, int32_t *page_table_d, int64_t max_pages, int32_t *free_pages_d,
                                 int32_t num_pages, const int32_t *n_free_in, int32_t *n_free_out, int32_t *slots_d,
                                 int32_t *pos_ids_d, int64_t capacity, int32_t *counts_d, void *stream);

/* pp_cache_store: round rows of keys and values to 8 bits and write them at their slots.
 *   k, v: n rows of [hkv, 128] in dt (PP_BF16 or PP_FP32), k_stride and v_stride elements apart (a multiple of 16
 *   bytes); slots_d: int32 [n], a negative slot skips its row. The rows of one page stand together, as pp_pages_resize
 *   gives them: each within 256 rows of the one before, skipped rows between them and none of another page. Their slots
 *   may leave gaps and come in any order; of two rows with one slot the later stands (both count for the scale). A page in
 *   two places of one call is written in no defined order. Rows whose smallest offset is 0 start their page anew; with a
 *   smallest offset o they keep the o tokens before it. Codes past o that no row names stay, but stand for nothing.
 *   The scale of a (page, head) block is the smallest 2^e, -40 <= e <= 56, under which its largest finite value does
 *   not exceed the largest code (448 for e4m3, 127 for int8), or the block's scale so far if that is larger; when it
 *   grows, the codes of the tokens before are rounded again. Codes round to nearest even; values beyond the largest
 *   code, infinities among them, become it; NaN becomes e4m3's NaN, or 0 in int8. Scales must be written by this call
 *   (or be positive and finite) where o > 0.
 */
PP_API pp_status pp_cache_store(const void *k, const void *v, int64_t k_stride, int64_t v_stride, pp_dtype dt,
                                const int32_t *slots_d, int64_t n, int32_t hkv, int32_t d, void *k_pages,
                                void *v_pages, float *k_scale, float *v_scale, pp_dtype codes, int32_t num_pages,
                                int32_t page_size, void *stream);

/* pp_paged_decode: one decoding step of every response over a paged cache, as pp_decode_attn over a dense one.
 *   Response i (segment i + g + 1 in group g) has one query, which attends its group's prefix and its own segment, all
 *   lens_d[segment] tokens of each. q: [n_resp, hq, 128] bf16, n_resp = num_segments - num_groups; o the same (it may
 *   be q); lse: [hq, n_resp] fp32 (natural log). A response with no keys gets 0 and -inf. softmax_scale 0 means 1/sqrt(128).
 *   The codes enter their products exactly. A query row is scaled by a power of two and taken as f16: its bf16 elements
 *   stay exact, but for those more than 2^14 below the row's largest, which keep what is above 2^-24 of it. Scores,
 *   softmax and sums are fp32. p times its block's value scale is rounded to 11 significant bits for the product with the
 *   value codes, and what is below 2^-31 of the largest such product of the row is lost to o (not to lse). d = 128.
 *   workspace: device scratch of ws_bytes >= pp_paged_decode_bytes (host only, from the sizes), 256-byte aligned,
 *   contents need not be initialised. Descriptors or lengths that do not fit yield NaN outputs; a page id outside the
 *   pool yields undefined values in the responses that read it.
 */
PP_API pp_status pp_paged_decode_bytes(int32_t n_resp, int32_t hq, int32_t hkv, int64_t *bytes);
PP_API pp_status pp_paged_decode(const void *q, const void *k_pages, const void *v_pages, const float *k_scale,
                                 const float *v_scale, pp_dtype codes, int32_t num_pages, int32_t page_size,
                                 const int32_t *group_start_d, int32_t num_groups, const int32_t *seg_group_d,
                                 int32_t num_segments, const int32_t *lens_d, const int32_t *page_table_d,
                                 int64_t max_pages, int32_t hq, int32_t hkv, int32_t d, float softmax_scale, void *o,
                                 float *lse, void *workspace, int64_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------------------------------------------
 * pp_pack_batch: pack an ungrouped micro-batch on the device ("prefix_grouper_utils.py" section 2, building the
 * grouper from a micro-batch). Consecutive samples with equal uids form a group (a uid that reappears later starts a
 * new group); the group's prefix is the valid prompt tokens of its first sample; the packed sequence is, group by
 * group, the prefix followed by each sample's valid response tokens, in order, without padding.
 *   prompts int32 [bs, Lp] and prompt_mask uint8 [bs, Lp]; responses int32 [bs, Lr] and response_mask uint8 [bs, Lr]
 *   (nonzero mask = valid token; padding may be on either side); uids int64 [bs]. 0 <= bs <= 8192.
 *   Outputs: packed_ids int32 [capacity >= bs * (Lp + Lr)] (first T written); groups pp_group_desc [bs] (first G
 *   written: prefix_len, num_suffixes = group size); cu_seqlens int32 [2 * bs + 1] (first nseg + 1 written: each
 *   group's prefix, then each response, empty segments kept; the layout pp_build_meta takes); sample_offsets
 *   int32 [bs, 2] = (packed offset of the sample's prompt if it heads its group, else -1; packed offset of its
 *   response); counts int32 [3] = {G, nseg = G + bs, T}. All device pointers; nothing is allocated.
 *   The counts are device values: a caller reads them (a synchronising copy) to size and call pp_build_meta.
 *   Errors: PP_ERR_INVALID_ARG (sizes, NULL pointers, capacity), PP_ERR_UNSUPPORTED (bs > 8192).
 */
PP_API pp_status pp_pack_batch(const int32_t *prompts, const uint8_t *prompt_mask, int32_t Lp, const int32_t *responses,
                               const uint8_t *response_mask, int32_t Lr, const int64_t *uids, int32_t bs,
                               int32_t *packed_ids, int64_t capacity, pp_group_desc *groups, int32_t *cu_seqlens,
                               int32_t *sample_offsets, int32_t *counts, void *stream);

/* ---------------------------------------------------------------------------------------------------------------
 * pp_response_logprobs: log-probability of every response token under the packed logits (the read-out of
 * "prefix_grouper_utils.py" section 3: split_output(logits, include_prefix_last=1) puts the group's last prefix row
 * in front of each response's rows, the last row of each block is dropped, the rows are divided by the temperature,
 * and the log-softmax is read at each completion token).
 *   On the packed layout: the token at response row y is predicted by row y - 1, except a response's first token,
 *   which is predicted by its group's last prefix row (o_g + P_g - 1). out[y] = x[src, id_y] / temperature -
 *   ln sum_v exp(x[src, v] / temperature), computed in fp32 with one pass over the row.
 *   logits: [T, V] row-major, dt PP_BF16 or PP_FP32, aligned to its element size (rows need not be 16-byte
 *   aligned). token_ids: int32 [T], the packed input ids. meta_d from pp_build_meta for the same groups.
 *   temperature > 0. out: fp32 [T]; prefix rows, and a response's first token in a group with P_g = 0 (no row
 *   predicts it), get 0. All pointers are device pointers; nothing is allocated.
 *   A token id outside [0, V) writes NaN at its row and sets PP_ERR_DEVICE_INPUT (reported by pp_get_status).
 */
PP_API pp_status pp_response_logprobs(const void *logits, pp_dtype dt, int64_t V, const int32_t *token_ids,
                                      const void *meta_d, int64_t T, float temperature, float *out, void *stream);

/* ---------------------------------------------------------------------------------------------------------------
 * pp_plan_batches (host only): plan training batches of packed preference groups ("Preference Packing" abstract and
 * method digest: packing combined with batch sorting, batch size following the lengths). A group costs its packed
 * length group_tokens[g] (P_g + sum of its response lengths). With sort_by_length != 0 the groups are taken longest
 * first (stable: ties keep their input order), otherwise in input order; batches are filled greedily in that order
 * up to token_capacity tokens; a group longer than the capacity forms a batch of its own.
 *   group_tokens: int64 [num_groups] (host, >= 0). order: int32 [num_groups] out, the groups in batch order.
 *   batch_of_group: int32 [num_groups] out. *num_batches out. token_capacity >= 1.
 *   Errors: PP_ERR_INVALID_ARG (no message is recorded for this call; it touches no device state).
 */
PP_API pp_status pp_plan_batches(const int64_t *group_tokens, int32_t num_groups, int64_t token_capacity,
                                 int32_t sort_by_length, int32_t *order, int32_t *batch_of_group, int32_t *num_batches);

/* ---------------------------------------------------------------------------------------------------------------
 * pp_selftest_bounded_wait: exercise the error channel of the kernels' bounded waits without a fault.
 * (The pages have no counterpart; this checks the library's failure detection.) Every mbarrier wait in the attention
 * kernels gives up after a time limit (2 s), records PP_ERR_DEVICE_TIMEOUT in the device error word and returns, so
 * a stuck pipeline ends with an error status instead of a hung GPU. This call launches one small kernel whose single
 * wait, with the same wait code and the given limit, is on an mbarrier that nothing arrives on; it issues no copy and
 * no MMA, so nothing is in flight when the wait gives up. The next pp_get_status() returns PP_ERR_DEVICE_TIMEOUT
 * (and clears the word); the context stays usable.
 *   limit_ns in [1e3, 2e9]. waited_ns_d: device uint64 out, the time the wait took before it gave up (0 if it
 *   completed, which cannot happen here). Errors: PP_ERR_INVALID_ARG.
 */
PP_API pp_status pp_selftest_bounded_wait(int64_t limit_ns, unsigned long long *waited_ns_d, void *stream);

/* ---------------------------------------------------------------------------------------------------------------
 * pp_get_status: synchronises `stream`, then reads and clears this device's error word. Returns PP_OK,
 * PP_ERR_DEVICE_TIMEOUT, PP_ERR_DEVICE_INPUT or PP_ERR_CUDA (a sticky CUDA error is reported as such).
 */
PP_API pp_status pp_get_status(void *stream);

/* Message describing the last failure seen by the calling thread ("" if none). Valid until its next call. */
PP_API const char *pp_last_error(void);

/* Library version string. */
PP_API const char *pp_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PP_H_ */

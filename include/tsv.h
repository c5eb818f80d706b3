/*
 * tsv.h - C ABI of the tree speculative-decoding verify step on GB300 (sm_103a).
 *
 * One verify round of tree speculative decoding, as five calls on one CUDA
 * stream (mask -> attention for every layer -> LM head + argmax -> accept walk
 * -> KV compaction).  The operations follow these pages:
 *
 *   [1204] mlxcel issue #1204, "perf(speculative): draft a tree instead of a
 *          chain, so an MTP round emits more than 2.33 tokens"
 *   [1212] mlxcel PR #1212, "feat(speculative): draft and verify a token tree,
 *          behind a flag, default off" (its commit messages)
 *   [1185] mlxcel issue #1185, "perf(speculative): cut the MTP drafter's
 *          per-step cost, now the binding constraint on M5-class hardware"
 *   [728]  Splash issue #728, "Experiment: qualify shared-prefix tree
 *          verification and conservative admission"
 *
 * Conventions shared by every call
 * --------------------------------
 * Ownership: every array argument is caller-owned memory.  Unless a parameter
 *   says "host", it is DEVICE memory of the current CUDA device.  The library
 *   keeps no pointer after a call returns and allocates no device memory;
 *   scratch comes from a caller-provided workspace whose size the matching
 *   *_workspace_size() call returns.  Workspaces are 16-byte aligned, and each
 *   belongs to one call until that has run on the device: calls that may overlap
 *   (on several streams, or in graphs that are replayed at the same time) need
 *   one each.
 * Streams: every call only enqueues work on `stream` (0 = legacy default
 *   stream) and returns without synchronising.  Results are ready when the
 *   stream reaches them.  Calls are capturable in CUDA graphs.  Every kernel
 *   is launched with programmatic stream serialization: it waits for the
 *   kernel before it on the stream to complete before it touches memory, and
 *   lets the kernel after it be scheduled early.  A kernel of the caller's
 *   launched after a call with that attribute set must therefore wait
 *   (griddepcontrol.wait / cudaGridDependencySynchronize) before it reads the
 *   call's outputs; ordinary launches, copies and events need nothing.
 * Host errors: a call returns TSV_OK when its work was enqueued.  Any other
 *   status means nothing was enqueued; tsv_last_error() then names the reason
 *   (a per-thread string, valid until the next call on the same thread).
 *   TSV_EUNSUPPORTED is a refusal ([1212], gather_positions commit: a layout
 *   the operation cannot serve refuses with a message, and the caller must
 *   decline tree drafting rather than proceed).
 * Device errors: topology or path errors that only the device can see are
 *   written to `dev_status` (int32[4], device memory) and never trap: word 0
 *   receives the first TSV_DEV_* code (atomic compare-and-swap from 0, so it
 *   is sticky), words 1..2 the sequence and node/position where it was found.
 *   The caller zeroes the words once and reads them whenever it chooses;
 *   outputs of a sequence with an error are unspecified (but in bounds).
 *   dev_status may be NULL, in which case device errors are dropped.
 * Sizes: 1 <= T <= 64 (one 64-bit ancestor word per node; tsv_tree_mask also
 *   accepts T == 0).  Layout shapes are row-major, innermost last.
 */
#ifndef TSV_H
#define TSV_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TSV_OK = 0,
    TSV_EINVAL = 1,       /* bad argument: null pointer, size out of range, misaligned buffer */
    TSV_ETOPOLOGY = 2,    /* a host-visible topology error */
    TSV_EUNSUPPORTED = 3, /* a format or shape this build refuses (the caller must decline) */
    TSV_ECAPACITY = 4,    /* workspace too small, or a size above a compiled maximum */
    TSV_ECUDA = 5         /* the CUDA runtime reported an error while enqueueing */
} tsv_status;

typedef enum {
    TSV_F16 = 0,       /* IEEE binary16 */
    TSV_BF16 = 1,      /* bfloat16 */
    TSV_I8_SCALED = 2, /* int8 code x fp16 per-token scale (KV caches only) */
    TSV_Q4_G64 = 3,    /* 4-bit affine, groups of 64 input features (LM head only) */
    TSV_I4_G64 = 4,    /* 4-bit affine, groups of 64 features of a token's row (KV caches only) */
    TSV_E4M3_B128 = 5, /* e4m3 codes x fp32 scales, one per block of 128 x 128 (LM head, matmul weights) */
    TSV_F32 = 6        /* IEEE binary32 (norm rows, logits, products) */
} tsv_dtype;

/* Device status codes (dev_status word 0). */
#define TSV_DEV_OK 0
#define TSV_DEV_BAD_ROOT 1    /* parents[b][0] != -1 */
#define TSV_DEV_BAD_PARENT 2  /* parents[b][i] outside [0, i) for i >= 1 */
#define TSV_DEV_BAD_PATH 3    /* path not strictly increasing from 0, or path_len outside [1, T]; or a
                                 kept list / kept_len of tsv_gather_positions out of order or range */
#define TSV_DEV_BAD_KV_LEN 4  /* kv_len[b] < T (< 0 for tsv_gather_positions), or kv_len[b] > capacity */
#define TSV_DEV_TIMEOUT 5     /* a bounded wait inside a kernel expired (a library bug; outputs unspecified) */
#define TSV_DEV_BAD_SEQ_LEN 6 /* cu_len not ascending within [0, rows], or a sequence longer than max_len */

#define TSV_MAX_T 64
#define TSV_MAX_CANDIDATES 1024 /* candidate-tree nodes per sequence for tsv_tree_select */
#define TSV_MAX_LAYERS 64

/* Reason for the last non-TSV_OK status returned on this thread ("" if none). */
const char* tsv_last_error(void);

/*
 * tsv_selftest_bounded_wait - checks the failure path every tensor-core
 * kernel relies on (no page counterpart: a property of this implementation).
 * One CTA waits on a barrier that nothing completes; the library's bounded
 * wait gives up after 1 s, raises the CTA's abort flag (which ends the other
 * warps' waits) and records TSV_DEV_TIMEOUT in dev_status (words 1..2: the
 * flag, the warp).  The device stays usable.  dev_status: int32[4], device
 * memory, zeroed by the caller.
 */
tsv_status tsv_selftest_bounded_wait(int32_t* dev_status, cudaStream_t stream);

/* ABI version of this library (major * 100 + minor). */
int tsv_version(void);

/*
 * tsv_tree_mask - topology check, ancestor bitmask and depth of every node.
 *   [1204] "What this needs" item 1: each node attends to its ancestors only,
 *   rebuilt every round from the topology; [1204] "Increment 1": nodes in
 *   topological order with parents[i] < i; [1212] history-mask commit: the
 *   [n, offset + n] additive form, history columns attended in full; [1212]
 *   verify commit: blocked entries are -1e9, never -inf.
 *
 *   parents    int32 [B, T]   parents[b][0] == -1, 0 <= parents[b][i] < i.
 *   anc        uint64 [B, T]  out: bit j of anc[b][i] set iff node j is an
 *                             ancestor of node i or i itself.
 *   depth      int32 [B, T]   out: edges from the root (root = 0).
 *   dense_mask float [B, T, mask_offset + T] or NULL; out: the additive mask
 *                             (0 = attend, -1e9 = blocked) for a history of
 *                             mask_offset positions.  Provided for parity
 *                             checks; the attention call never reads it.
 *   Device errors: TSV_DEV_BAD_ROOT / TSV_DEV_BAD_PARENT; that sequence's anc
 *   and depth are then 0 / -1.
 */
tsv_status tsv_tree_mask(const int32_t* parents, int32_t B, int32_t T, uint64_t* anc, int32_t* depth,
                         float* dense_mask, int32_t mask_offset, int32_t* dev_status, cudaStream_t stream);

/*
 * tsv_sliding_band_mask - the mask a sliding-window layer attends with, in place.
 *   [1212], the commit on caller masks and the sliding-window band: a
 *   sliding-window layer takes the intersection of the caller's mask (here the
 *   dense tree mask of tsv_tree_mask) with its band, by element-wise minimum
 *   of the additive masks, and only where the two can disagree.  Query row q
 *   sits at position mask_offset + q; its band keeps columns c with
 *   mask_offset + q - window < c <= mask_offset + q, all else becomes
 *   min(mask, -1e9).  Every row keeps its own position.
 *   dense_mask float [B, T, mask_offset + T], in/out.  window >= 1; when
 *   mask_offset + T <= window the mask is left untouched (nothing is launched).
 *   The attention call applies the same band itself from tsv_attn_desc.window;
 *   this call is provided for parity checks.
 */
tsv_status tsv_sliding_band_mask(float* dense_mask, int32_t B, int32_t T, int32_t mask_offset, int32_t window,
                                 cudaStream_t stream);

/*
 * Building the draft tree from the drafter's confidence (two calls).
 *   [1204] "What this needs", the fourth decision: EAGLE-2 branches by the
 *   drafter's confidence, which needs the drafter's logits; [1212], the
 *   draft_tree commit: the runner-up at an uncertain step is the alternative
 *   worth a verify position; [728] "What it does": the chain plus likely
 *   alternatives from the draft's top-k selector.
 *
 * tsv_draft_children - for every expanded node (row of drafter logits
 *   [rows, V] fp32), its top_k tokens (ties to the lower index) and their
 *   log-probabilities log_softmax(logits)[token]: child_tokens int32 and
 *   child_logp float, [rows, top_k], largest first.  1 <= top_k <= min(64, V).
 * tsv_tree_select - the verified tree from a candidate tree (reading: the
 *   root plus the T - 1 candidates of highest cumulative log-probability,
 *   summed in fp32 from the root down, depth <= depth_max, ties to the earlier
 *   candidate - what best-first expansion by path probability selects).
 *   cand_parents int32 [B, N] (topological: [b][0] = -1, 0 <= [b][i] < i),
 *   cand_tokens int32 [B, N], cand_logp float [B, N] (log-probability of the
 *   candidate given its parent, <= 0; the root's is ignored).  N <= 1024.
 *   Out: parents, tokens, cand_index int32 [B, T] in selection order (descending
 *   score, so topological; the root first), sizes int32 [B] = nodes chosen
 *   (< T when fewer candidates qualify; the rest of the row is -1).
 *   Device errors: TSV_DEV_BAD_ROOT / TSV_DEV_BAD_PARENT for a candidate tree
 *   that is not topological (that sequence's outputs are -1, size 0) or whose
 *   chosen node's parent was not chosen (a log-probability above 0).
 */
size_t tsv_draft_children_workspace_size(int32_t rows, int32_t V, int32_t top_k);

tsv_status tsv_draft_children(const float* draft_logits, int32_t rows, int32_t V, int32_t top_k, int32_t* child_tokens,
                              float* child_logp, void* workspace, size_t ws_bytes, cudaStream_t stream);

tsv_status tsv_tree_select(const int32_t* cand_parents, const int32_t* cand_tokens, const float* cand_logp, int32_t B,
                           int32_t N, int32_t T, int32_t depth_max, int32_t* parents, int32_t* tokens,
                           int32_t* cand_index, int32_t* sizes, int32_t* dev_status, cudaStream_t stream);

/*
 * Tree-masked GQA attention of the verify block, for n_layers layers at once.
 *   [1204] "What this needs" item 1 and "Increment 3"; [1212] history-mask and
 *   verify_forward_with_mask commits; [728] "Earlier shader evidence" (split-KV
 *   attention with fp32 partials and statistics, 16 nodes x 24 heads x D256).
 *   For every layer l, sequence b, query head h and node i:
 *     O[b,i,h,:] = sum_c p_c V[b, h/G, c, :],  p = softmax_c( Q[b,i,h,:] . K[b,h/G,c,:] / sqrt(D) )
 *   over c in [0, S_b) and c = S_b + j for every j set in anc[b][i], where
 *   S_b = kv_len[b] - T (the block was appended in topological order at
 *   [S_b, S_b + T)).  G = HQ / HKV.  Int8: K = code * k_scale[c], V = code * v_scale[c].
 *   Sliding-window layers ([1212], the commit on caller masks and the
 *   sliding-window band): with window[l] > 0, node i (at cache position
 *   S_b + i) keeps only those of the keys above whose position c satisfies
 *   c > S_b + i - window[l]: the intersection of the tree mask with the
 *   layer's band.  Every node keeps itself.  window[l] == 0 is a full-attention layer.
 *   Accumulation is fp32; O is rounded to bf16 once.
 *   4-bit caches (TSV_I4_G64, [1185] Phase 3's affine groups of 64 on the cache): byte j of a row holds element 2j in
 *   its low nibble and 2j + 1 in its high nibble; value = scale * code + bias, with the fp16 pair (scale, bias) of
 *   its group of 64 features at k_scale[b][h][c][group] (v_scale likewise; the buffers 16-byte aligned).  Pairs of
 *   positions below kv_len[b] have to be finite and to stand for values within fp16's range, as tsv_tree_append writes
 *   them; what lies behind is not looked at.
 */
typedef struct {
    int32_t n_layers;   /* 1 .. TSV_MAX_LAYERS */
    int32_t B, T, HQ, HKV, D; /* HQ % HKV == 0; D in {64, 128, 256} */
    int64_t s_cap;      /* capacity of every cache buffer's sequence axis, in positions */
    int32_t max_kv_len; /* host-known upper bound of every kv_len[b] (<= s_cap); sizes the grid */
    int32_t kv_dtype;   /* TSV_F16, TSV_BF16, TSV_I8_SCALED or TSV_I4_G64 */
    int32_t splits;     /* key-range splits per (layer, sequence, kv head); 0 = automatic; at most 64 */
    int32_t path;       /* TSV_ATTN_AUTO, TSV_ATTN_SIMT or TSV_ATTN_TCGEN05 */
    const void* q[TSV_MAX_LAYERS];       /* per layer: bf16 [B, T, HQ, D] */
    const void* k[TSV_MAX_LAYERS];       /* per layer: [B, HKV, s_cap, D] in kv_dtype (int8 codes; 4-bit: D/2 bytes a row) */
    const void* v[TSV_MAX_LAYERS];       /* per layer: as k */
    const void* k_scale[TSV_MAX_LAYERS]; /* per layer: fp16 [B, HKV, s_cap] (Int8), fp16 [B, HKV, s_cap, D/64, 2]
                                            (4-bit: scale, bias), else NULL */
    const void* v_scale[TSV_MAX_LAYERS]; /* per layer: as k_scale */
    void* o[TSV_MAX_LAYERS];             /* per layer: bf16 [B, T, HQ, D], out */
    const int32_t* kv_len;               /* int32 [B]: S_b + T */
    const uint64_t* anc;                 /* uint64 [B, T] from tsv_tree_mask */
    int32_t window[TSV_MAX_LAYERS];      /* per layer: sliding window in positions, 0 = full attention */
} tsv_attn_desc;

/* Kernel choice.  AUTO takes the tensor-core (tcgen05) kernel where it applies
 * (D == 256) and the CUDA-core kernel elsewhere; 4-bit caches of up to 16 query
 * rows per K/V head, or of other head dimensions, take a kernel of their own.
 * TCGEN05 lets the library pick the tensor-core kernel's score-tile width (128
 * keys for Int8 caches and for units of more than 128 query rows, else 64);
 * TCGEN05_64 and TCGEN05_128 force one (both compute the same result; 4-bit
 * caches have 128-key tiles only).
 * On the tensor-core path Q is rounded to the cache's 16-bit type for the
 * Q K^T product (exact for bf16; for fp16, Int8 and 4-bit caches, whose products
 * are fp16, |q| must lie in fp16 range; there a row of q that is NaN or beyond it gives a row of NaN)
 * and the softmax weights P enter P V as 16-bit values. */
#define TSV_ATTN_AUTO 0
#define TSV_ATTN_SIMT 1
#define TSV_ATTN_TCGEN05 2
#define TSV_ATTN_TCGEN05_64 3
#define TSV_ATTN_TCGEN05_128 4

size_t tsv_attention_workspace_size(const tsv_attn_desc* d);

/* Device errors: TSV_DEV_BAD_KV_LEN (that sequence's outputs are left unwritten). */
tsv_status tsv_tree_verify_attention(const tsv_attn_desc* d, void* workspace, size_t ws_bytes,
                                     int32_t* dev_status, cudaStream_t stream);

/*
 * tsv_lm_head_argmax - LM-head projection fused with a greedy argmax; the
 * logits are never written.  [1185] "Phase 2" item 2a (fused projection and
 * argmax at temperature 0) and "Phase 3" (affine group-64 4-bit weights with
 * scales and biases); [1204] "What this needs" item 2 (one target argmax per
 * verified position).
 *   hidden  bf16 [rows, H]
 *   W       TSV_F16 / TSV_BF16: [V, H].  TSV_Q4_G64: uint8 [V, H/2], byte j of a
 *           row holds element 2j in its low nibble and 2j+1 in its high nibble;
 *           scales, biases: bf16 [V, H/64]; w = scale * q + bias, q in [0, 15].
 *   argmax  int32 [rows], out: index of the largest logit, ties -> lowest index.
 *           A logit that is NaN counts as larger than every number if its sign
 *           bit is clear, and as smaller if it is set.
 *   maxlogit float [rows] or NULL, out: that logit (fp32 accumulation).
 *   H % 64 == 0 (H % 256 == 0 for TSV_F16/TSV_BF16), 1 <= V < 2^31, rows >= 1.
 *   fp16 and bf16 heads with up to 4 rows stream the head once through CUDA
 *   cores; more rows, and 4-bit heads at any row count (H % 512 == 0, scales
 *   and biases 16-byte aligned), use the tcgen05 kernels (fp16 or bf16
 *   operands, fp32 accumulation; 4-bit weights are dequantised to fp16 with
 *   one rounding, and hidden is rounded to fp16 for fp16 and 4-bit heads).
 */
/* Workspace bytes for tsv_lm_head_argmax: 8 per hidden row (running bests), plus, when the tensor-core
 * kernel applies to an fp16 or 4-bit head, an fp16 copy of hidden (rows * H * 2, rounded up to 256).  A
 * smaller workspace (at least 8 bytes per row) is accepted and selects the CUDA-core kernel. */
size_t tsv_lm_head_workspace_size(int32_t rows, int32_t H, int32_t V, int32_t w_dtype);

tsv_status tsv_lm_head_argmax(const void* hidden, int32_t rows, int32_t H, int32_t V, int32_t w_dtype,
                              const void* W, const void* scales, const void* biases, int32_t* argmax,
                              float* maxlogit, void* workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * tsv_lm_head_logits - the same projection, writing every logit instead of the
 * argmax: logits float [rows, V] (fp32 accumulation, same kernels and
 * workspace as tsv_lm_head_argmax).  The input of sampled verification
 * (tsv_sample_nucleus): Splash issue #728, "What it does" - sampled requests
 * draw from the target's nucleus-filtered distribution at every node.
 */
tsv_status tsv_lm_head_logits(const void* hidden, int32_t rows, int32_t H, int32_t V, int32_t w_dtype,
                              const void* W, const void* scales, const void* biases, float* logits,
                              void* workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * tsv_sample_nucleus - each node's draw for sampled (temperature > 0)
 * verification.  Splash issue #728, "What it does": every node draws from
 * the nucleus-filtered distribution with its own uniform, which keeps the
 * chain verify's output distribution; the walk (tsv_tree_accept_walk, with
 * these tokens in place of the argmax) then follows the child whose draft
 * token equals the draw.  Filter order (reading; the page names the three
 * knobs): logits / temperature, the top_k largest (ties to the lower index),
 * softmax over them, the shortest descending prefix whose mass reaches top_p,
 * renormalised; the token is the first whose cumulative mass exceeds
 * uniforms[row] * (kept mass).
 *   logits   float [rows, V] (tsv_lm_head_logits); uniforms float [rows] in
 *            [0, 1), one per node, drawn by the caller; tokens int32 [rows], out.
 *   1 <= top_k <= 64 (TSV_EUNSUPPORTED above: the top-k selection is exact
 *   and bounded), temperature > 0, 0 < top_p <= 1, rows <= 65535.
 *   Arithmetic: softmax weights and prefix sums in fp32.
 */
size_t tsv_sample_workspace_size(int32_t rows, int32_t V, int32_t top_k);

tsv_status tsv_sample_nucleus(const float* logits, int32_t rows, int32_t V, float temperature, int32_t top_k,
                              float top_p, const float* uniforms, int32_t* tokens, void* workspace, size_t ws_bytes,
                              cudaStream_t stream);

/*
 * tsv_lm_head_argmax_noalloc - tsv_lm_head_argmax without a workspace argument.
 *   The pages have no counterpart: this entry point exists only in this
 *   library, for callers that cannot allocate device memory themselves -
 *   for example a plugin whose host framework owns every device buffer
 *   through its own pool, or a latency-critical caller that may not pay for
 *   cudaMalloc's implicit synchronisation.  Its scratch is a fixed array of
 *   TSV_NOALLOC_MAX_ROWS 64-bit entries (32 KiB) inside this library's device
 *   image, held by every GPU that loads the library until the process exits.
 *   Arguments, results and errors are those of tsv_lm_head_argmax, plus
 *   TSV_ECAPACITY when rows > TSV_NOALLOC_MAX_ROWS.  The library allocates
 *   nothing for it: the first call on each device looks up the array's
 *   device address (with that device current), and every call clears the
 *   entries it uses on `stream` before the projection.  All calls share the
 *   one array, so calls whose work overlaps on the GPU (on different streams,
 *   or from different host threads) race and give wrong results; serialise
 *   them on one stream.
 *   Speed: the array is also the call's workspace, and for fp16 and 4-bit
 *   heads the tensor-core kernel needs an fp16 copy of hidden beside the
 *   bests (rows * H * 2 bytes, rounded up to 256, after 8 bytes per row
 *   rounded up to 256).  When that does not fit the 32 KiB (H = 5120: more
 *   than 3 rows), the call takes the CUDA-core kernel instead, which streams
 *   the whole head once per 8 hidden rows and, for a 4-bit head, dequantises
 *   every weight again for each row (248,320 x 5120 4-bit head: about 2.1 ms
 *   per 8-row pass, so 4096 rows take about a second instead of a few ms).
 *   bf16 heads need no copy and keep the tensor-core kernel.  Callers with
 *   many rows and an fp16 or 4-bit head should use tsv_lm_head_argmax with a
 *   workspace.
 */
#define TSV_NOALLOC_MAX_ROWS 4096

tsv_status tsv_lm_head_argmax_noalloc(const void* hidden, int32_t rows, int32_t H, int32_t V, int32_t w_dtype,
                                      const void* W, const void* scales, const void* biases, int32_t* argmax,
                                      float* maxlogit, cudaStream_t stream);

/*
 * tsv_tree_accept_walk - descend the tree along the target's argmaxes.
 *   [1204] "What this needs" item 2 and "Increment 1" (the accepted set is a
 *   path, never a subtree); [1212] first commit; [728] "What it does" (every
 *   committed token is the target's selection at its path node).
 *   From u = 0: take the lowest-index child c of u with tokens[c] == argmax[u],
 *   append it, repeat; stop when no child matches.
 *   argmax, tokens, parents  int32 [B, T]
 *   path      int32 [B, T] out: accepted nodes from the root, -1 padded.
 *   path_len  int32 [B]    out: accepted + 1.
 *   emitted   int32 [B, T] out: argmax[path[j]] for j < path_len, -1 padded.
 *   Device errors: TSV_DEV_BAD_ROOT / TSV_DEV_BAD_PARENT (that sequence gets
 *   path = [0], path_len = 1).
 */
tsv_status tsv_tree_accept_walk(const int32_t* argmax, const int32_t* tokens, const int32_t* parents, int32_t B,
                                int32_t T, int32_t* path, int32_t* path_len, int32_t* emitted, int32_t* dev_status,
                                cudaStream_t stream);

/*
 * tsv_kv_gather_positions - compact the verify block of every cache to the
 * accepted path, in place.  [1204] "The rollback constraint, which decides
 * feasibility"; [1212] gather_positions commit (Int8 scale sidecars move with
 * their tokens; a prefix selection equals trim_to; the identity selection
 * short-circuits) and gather_within_tail commit (only [tail_start, tail_start
 * + kept_len) is rewritten; cost scales with the block, not the context).
 *   For every layer, sequence b and kv head, with S = kv_len[b] - T:
 *     rows S + j <- rows S + path[b][j] for j < path_len[b] (K, V and, for
 *     Int8, k_scale and v_scale); then kv_len[b] = S + path_len[b].
 *   Rows below S and at or beyond the new kv_len are not written.  When
 *   path[b][j] == j for every j, no cache byte is moved.
 *   path: strictly increasing with path[b][0] == 0 (every root path of a
 *   topological tree is), 1 <= path_len[b] <= T.
 *   Device errors: TSV_DEV_BAD_PATH, TSV_DEV_BAD_KV_LEN (that sequence is left
 *   untouched, kv_len included).
 */
typedef struct {
    int32_t n_layers, B, HKV, D;
    int64_t s_cap;
    int32_t kv_dtype; /* TSV_F16, TSV_BF16, TSV_I8_SCALED or TSV_I4_G64 */
    int32_t reserved;
    void* k[TSV_MAX_LAYERS];       /* per layer: [B, HKV, s_cap, D] (4-bit: D/2 bytes a row) */
    void* v[TSV_MAX_LAYERS];
    void* k_scale[TSV_MAX_LAYERS]; /* per layer: fp16 [B, HKV, s_cap] (Int8), fp16 [B, HKV, s_cap, D/64, 2] (4-bit) */
    void* v_scale[TSV_MAX_LAYERS];
} tsv_kv_desc;

tsv_status tsv_kv_gather_positions(const tsv_kv_desc* kv, int32_t* kv_len, const int32_t* path,
                                   const int32_t* path_len, int32_t T, int32_t* dev_status, cudaStream_t stream);

/*
 * tsv_gather_positions - the absolute form of the compaction: keep the cache
 * positions listed in kept, in order, and close them up from position 0.
 *   [1212] gather_positions commit: select and compact positions on the
 *   sequence axis (kept strictly increasing); Int8 scale sidecars move with
 *   their tokens; a prefix selection [0, 1, ..., n-1] equals trim_to(n) and
 *   the identity selection moves nothing.  tsv_kv_gather_positions is the
 *   tail form of the same selection ([1212] gather_within_tail commit) for
 *   kept = [0, S_b) followed by S_b + path[b][j].
 *   For every layer, sequence b and kv head:
 *     rows j <- rows kept[b][j] for j < kept_len[b] (K, V and, for Int8,
 *     k_scale and v_scale); then kv_len[b] = kept_len[b].
 *   Rows at or beyond the new kv_len are not written.  Rows below the first j
 *   with kept[b][j] != j are not written either, so a prefix or identity
 *   selection moves no cache byte.
 *   kept      int32 [B, max_kept] (row stride max_kept): kept[b][0..kept_len[b])
 *             strictly increasing within [0, kv_len[b]).  May be NULL when
 *             max_kept == 0.
 *   kept_len  int32 [B]: 0 <= kept_len[b] <= min(max_kept, kv_len[b]).
 *   kv_len    int32 [B], in/out: in, the current length (<= s_cap); out,
 *             kept_len[b].
 *   The list may be as long as the cache; every (layer, sequence, kv head)
 *   moves its rows in ascending chunks, so the cost is the rows moved.
 *   Device errors: TSV_DEV_BAD_PATH (a kept list that is not strictly
 *   increasing, leaves [0, kv_len[b]), or a kept_len out of range),
 *   TSV_DEV_BAD_KV_LEN (kv_len[b] outside [0, s_cap]); that sequence is left
 *   untouched, kv_len included.
 */
tsv_status tsv_gather_positions(const tsv_kv_desc* kv, int32_t* kv_len, const int32_t* kept, const int32_t* kept_len,
                                int32_t max_kept, int32_t* dev_status, cudaStream_t stream);

/*
 * tsv_tree_append - append the verify block to every layer's cache, each node
 * at its own position, ahead of the attention call.
 *   [1185], the closing comment's list of follow-ups: the tree path verifies
 *   the tree at its own positions (the title of the PR that added tree
 *   drafting there).  Node i is verified at position S_b + depth(i)
 *   (the root, the last committed token, at S_b; a chain gets S_b + i); its K
 *   and V rows still go to cache slot S_b + i, the topological block layout
 *   tsv_tree_verify_attention and tsv_kv_gather_positions use.  Rotary
 *   embedding (reading; the pages name only positions): the first rot_dim
 *   features are rotated in pairs (j, j + rot_dim/2) - or (2j, 2j + 1) when
 *   interleaved - by the angle pos * rope_base^(-2j / rot_dim); Q and K are
 *   rotated, V is not.  Int8 caches ([1212] gather_positions commit: one scale
 *   per token; a per-token scale maps every single-valued token to the same
 *   code): scale = fp16(absmax / 127) with the division in fp32, code =
 *   round-half-to-even(x / scale) in fp32, clamped to [-127, 127]; a token whose
 *   scale is 0 stores zero codes.  4-bit caches: per group of 64 features, with its minimum and maximum (over what is
 *   not NaN) cut to [-65000, 65000], bias = fp16(minimum), scale = fp16((maximum - minimum) / 15) with the division in
 *   fp32, code = round-half-to-even((x - bias) / scale) in fp32, clamped to [0, 15] (0 for NaN); a group whose scale is 0
 *   stores zero codes.  fp16 / bf16 caches store the rotated fp32
 *   values rounded to nearest even.  Angles are reduced in fp64, so positions
 *   up to 2^31 keep fp32 accuracy.
 *   kv_len: in, S_b per sequence; out, S_b + T.  depth: from tsv_tree_mask.
 *   Device errors: TSV_DEV_BAD_KV_LEN when S_b + T > s_cap; a sequence whose
 *   depth[b][0] != 0 (its mask call failed) is skipped.  Skipped sequences
 *   keep their caches and kv_len.
 */
typedef struct {
    int32_t n_layers;   /* 1 .. TSV_MAX_LAYERS */
    int32_t B, T, HQ, HKV, D; /* HQ % HKV == 0; D in {64, 128, 256} */
    int64_t s_cap;
    int32_t kv_dtype;   /* TSV_F16, TSV_BF16, TSV_I8_SCALED or TSV_I4_G64 */
    int32_t rot_dim;    /* even, 2 <= rot_dim <= D; features >= rot_dim are copied */
    int32_t interleaved; /* 0: pairs (j, j + rot_dim/2); 1: pairs (2j, 2j + 1) */
    int32_t reserved;
    double rope_base;   /* > 0, e.g. 1e4 or 1e6 */
    const void* q_in[TSV_MAX_LAYERS];  /* per layer: bf16 [B, T, HQ, D], not yet rotated */
    void* q_out[TSV_MAX_LAYERS];       /* per layer: bf16 [B, T, HQ, D], out (may equal q_in) */
    const void* k_new[TSV_MAX_LAYERS]; /* per layer: bf16 [B, T, HKV, D], not yet rotated */
    const void* v_new[TSV_MAX_LAYERS]; /* per layer: bf16 [B, T, HKV, D] */
    void* k[TSV_MAX_LAYERS];           /* per layer caches as in tsv_kv_desc */
    void* v[TSV_MAX_LAYERS];
    void* k_scale[TSV_MAX_LAYERS];
    void* v_scale[TSV_MAX_LAYERS];
    const int32_t* depth;              /* int32 [B, T] */
} tsv_append_desc;

tsv_status tsv_tree_append(const tsv_append_desc* d, int32_t* kv_len, int32_t* dev_status, cudaStream_t stream);

/*
 * The gated delta rule of a hybrid target's recurrent layers, for n_layers layers at once (three calls).
 *   [1204] on recurrent layers: recurrent layers cannot take a mask, and a
 *   flattened tree would leak state between siblings, so every node runs from its own parent's state; [728] "What it
 *   does": the selected path's recurrent state is the one retained.  The pages do not print the recurrence (reading:
 *   the published gated delta rule).  For one value head with state S [DV, DK] (fp32), log decay g <= 0, write
 *   strength beta:
 *     S <- e^g S;  u = beta (v - S k);  S <- S + u k^T;  o = scale * S q
 *   Value head h reads key head h / (HV / HK).  With norm_eps > 0 every row of q and k is divided by
 *   sqrt(sum x^2 + norm_eps) first.  Sums and the state are fp32.  Products on the tensor cores take their operands as
 *   fp16 with power-of-two scales: an hi + lo pair (within 2^-22 of the value) for what reaches the state, one fp16
 *   (2^-12) for what reaches o alone.  The scales are a value feature's, over a block (a tree, or 64 tokens): v, and the
 *   state's row as the block's first row leaves it (decayed), are held down to 2^-37 of the largest of them; so is the
 *   weight of one row's write in a later row (in o: 2^-33).  A block is computed in fp32 where its operands leave fp16's
 *   range, where a row of q or k is shorter than 2^-8, where a node or token sees (in its own v, the one before it and the
 *   state, times their beta and decay) less than 2^-24 of that largest, and where the new state is less than 2^-18 of it:
 *   values that a row does not see, or that were forgotten ahead of it, do not reach it.  o is rounded to
 *   bf16 once.  g may be -infinity (the state is forgotten).
 *
 * tsv_gdn_tree_verify - o of every node of each sequence's tree, node i starting from its parent's state and the
 *   root from state[l][b].  The state is read once and not written (state_out is ignored).  anc: uint64 [B, T] from
 *   tsv_tree_mask; bits at or above a node's own index are ignored.  A NaN or infinity in one node's inputs reaches
 *   that node and its descendants only.
 * tsv_gdn_commit - the state after the accepted path: state_out[l][b] = state[l][b] advanced over the block's rows
 *   path[b][0 .. path_len[b]).  path and path_len as for tsv_kv_gather_positions (path[b][0] == 0, strictly
 *   increasing, 1 <= path_len[b] <= T).  q and o are ignored.  Device errors: TSV_DEV_BAD_PATH (that sequence's
 *   state_out is not written).
 * tsv_gdn_scan - the state advanced over new tokens (a decoding step, a prompt, or a ragged batch of both), with
 *   every token's o.  q, k, v, g, beta and o hold T packed rows; sequence b owns rows cu_len[b] .. cu_len[b + 1]
 *   (int32 [B + 1] on the device, ascending, within [0, T]; a sequence without rows keeps its state, which is copied
 *   to state_out).  max_len: host-known upper bound of every sequence's rows (<= T); it picks the kernel.  Rows that
 *   no sequence owns are not read and their o is not written.  Device errors: TSV_DEV_BAD_SEQ_LEN (that sequence's
 *   o and state_out are not written).
 *
 * state_out[l] may equal state[l] (in place); otherwise they must not overlap, nor may o overlap an input, nor the
 * outputs of two layers each other.
 */
typedef struct {
    int32_t n_layers;   /* 1 .. TSV_MAX_LAYERS */
    int32_t B, T;       /* T: nodes per tree (verify, commit: 1 .. 64) or packed rows in all (scan) */
    int32_t HK, HV;     /* HV % HK == 0 */
    int32_t DK, DV;     /* each 64 or 128 */
    float norm_eps;     /* 0: q and k are taken as they are */
    float scale;        /* on q; 0: 1 / sqrt(DK) */
    int32_t reserved;
    const void* q[TSV_MAX_LAYERS];     /* per layer: bf16 [B, T, HK, DK] (scan: [T, HK, DK]) */
    const void* k[TSV_MAX_LAYERS];     /* per layer: as q */
    const void* v[TSV_MAX_LAYERS];     /* per layer: bf16 [B, T, HV, DV] */
    const float* g[TSV_MAX_LAYERS];    /* per layer: fp32 [B, T, HV], log decay */
    const float* beta[TSV_MAX_LAYERS]; /* per layer: fp32 [B, T, HV] */
    const float* state[TSV_MAX_LAYERS]; /* per layer: fp32 [B, HV, DV, DK] */
    float* state_out[TSV_MAX_LAYERS];   /* per layer: as state, out (commit, scan) */
    void* o[TSV_MAX_LAYERS];            /* per layer: bf16 as v, out (verify, scan) */
} tsv_gdn_desc;

tsv_status tsv_gdn_tree_verify(const tsv_gdn_desc* d, const uint64_t* anc, int32_t* dev_status, cudaStream_t stream);

tsv_status tsv_gdn_commit(const tsv_gdn_desc* d, const int32_t* path, const int32_t* path_len, int32_t* dev_status,
                          cudaStream_t stream);

tsv_status tsv_gdn_scan(const tsv_gdn_desc* d, const int32_t* cu_len, int32_t max_len, int32_t* dev_status,
                        cudaStream_t stream);

/*
 * What stands ahead of the LM head, and products, in 8 bits.  The pages have no counterpart: [1185] Phase 3 quantises the
 * head to 4 bits, and its cost model counts the projections among a verify's reads; these calls serve targets whose
 * weights are e4m3 with one fp32 scale per block of 128 x 128.
 *
 * 8-bit rows: codes e4m3 [rows, H] with float scale [rows, ceil(H / 128)]; per 128 features of a row (the last group may be
 *   shorter) scale = max |y| * (1 / 448) in fp32 (1 / 448 rounded to fp32) and code = e4m3(y / scale), the division in fp32,
 *   the code rounded to nearest even and held to +-448.  A group of zeros, or of values so small that the scale is 0, has
 *   scale 0 and zero codes; a NaN or an infinity among a group's values makes its scale that, and the codes follow.
 *
 * tsv_add_rms_norm - the residual's addition and the root-mean-square norm of every row:
 *     h = x + residual;  y = h / sqrt(mean(h^2) + eps) * (weight_offset + weight)
 *   x, residual, residual_out, weight, out: `dtype` (TSV_F16, TSV_BF16 or TSV_F32), [rows, H], weight [H].  residual may
 *   be NULL (h = x).  Outputs, each optional but one at least: residual_out = h, out = y, and y as 8-bit rows in out8
 *   (uint8 e4m3 [rows, H]) with out8_scale.  Everything between is fp32 and each output is rounded once from it: y is of
 *   the unrounded h, the codes of the unrounded y (their quotients within two units in the last place of fp32).  A row
 *   whose squares leave fp32's range is scaled by a power of two first.  residual_out may equal residual or x, out may
 *   equal x or residual; otherwise outputs overlap neither inputs nor each other.
 *   1 <= H <= 32768, 1e-30 <= eps, eps and weight_offset finite.  A NaN in a row makes all of its y NaN, an infinity makes
 *   y NaN there and 0 elsewhere.
 * tsv_quantize_e4m3 - 8-bit rows of x as it is: out8, out8_scale as above (H without an upper limit).
 */
tsv_status tsv_add_rms_norm(const void* x, const void* residual, const void* weight, int32_t rows, int32_t H, int32_t dtype,
                            float eps, float weight_offset, void* residual_out, void* out, void* out8, float* out8_scale,
                            cudaStream_t stream);

tsv_status tsv_quantize_e4m3(const void* x, int32_t rows, int32_t H, int32_t dtype, void* out8, float* out8_scale,
                             cudaStream_t stream);

/*
 * tsv_matmul_e4m3 - rows in 8 bits times weights in 8 bits:
 *     out[m, n] = sum over k of a[m, k] a_scale[m, k / 128] w[n, k] w_scale[n / 128, k / 128]
 *   a: e4m3 [rows, K], a_scale float [rows, ceil(K / 128)] (8-bit rows as above); w: e4m3 [N, K], w_scale float
 *   [ceil(N / 128), ceil(K / 128)]; out [rows, N] of out_dtype (TSV_BF16, TSV_F16 or TSV_F32).  The products of 128
 *   features are summed on the tensor cores into fp32, scaled, and summed in fp32; out is rounded once.  The same inputs
 *   give the same bits in every call.  A block's scale is a_scale w_scale rounded to fp32 ahead of its sums: below fp32's
 *   normal numbers (2^-126) it has fewer bits, beyond its range it is an infinity.
 *   K % 16 == 0, a and w 16-byte aligned, 0 <= rows <= 2^30, 1 <= N <= 2^30.
 *   Every wait inside the kernel is bounded.  These calls have no status word: should a wait run out, the part of out that it was
 *   for is NaN (of the argmax: those rows' maxval).
 * tsv_matmul_e4m3_argmax - the same product with its argmax, as tsv_lm_head_argmax: argmax int32 [rows] (ties to the lowest
 *   index), maxval float [rows] or NULL; the products are never written.  Workspace: tsv_matmul_e4m3_argmax_workspace_size.
 *   A product that is NaN counts as larger than every number if its sign bit is clear, and as smaller if it is set.
 * tsv_lm_head_argmax, tsv_lm_head_logits with w_dtype TSV_E4M3_B128: W as w, scales as w_scale, biases ignored; hidden
 *   (bf16) becomes 8-bit rows in the workspace first.  H % 16 == 0, H >= 64, rows and V at most 2^30.
 */
tsv_status tsv_matmul_e4m3(const void* a, const float* a_scale, int32_t rows, int32_t K, const void* w, const float* w_scale,
                           int32_t N, void* out, int32_t out_dtype, cudaStream_t stream);

size_t tsv_matmul_e4m3_argmax_workspace_size(int32_t rows);

tsv_status tsv_matmul_e4m3_argmax(const void* a, const float* a_scale, int32_t rows, int32_t K, const void* w,
                                  const float* w_scale, int32_t N, int32_t* argmax, float* maxval, void* workspace,
                                  size_t ws_bytes, cudaStream_t stream);

/*
 * tsv_token_logprobs - what a user asks about emitted tokens, from one read of the logits:
 *     z = logits / temperature;  logp(t) = z_t - log(sum exp(z));  entropy = -sum p log p with p = softmax(z)
 *   logits [rows, V] of logits_dtype (TSV_F32, TSV_BF16 or TSV_F16; each row may start anywhere: V needs no alignment),
 *   1 <= V <= 2^24.
 *   targets int32 [rows] or NULL; logp float [rows]: each target's log probability; rank int32 [rows] or NULL: how many
 *   tokens have a larger logit, or an equal one and a lower index (0: the greedy choice).  With targets NULL, logp and
 *   rank are NULL too.  entropy float [rows] or NULL.  top_tokens int32, top_logp float [rows, top_k]: the top_k largest,
 *   largest first, ties to the lower index; 0 <= top_k <= min(64, V) (0: both NULL).
 *   A logit of -infinity has probability 0 (and adds nothing to the entropy).  A row with a NaN or +infinity, or with
 *   nothing but -infinity, has no distribution: its floats are NaN and its rank and tokens -1.  A target outside [0, V)
 *   (the -1 that pads emitted tokens) gets logp NaN and rank -1.  1e-6 <= temperature <= 1e6.  Sums are fp32, in an order
 *   that the sizes and the rows' offsets from 16-byte boundaries fix, so the same call gives the same bits.
 */
size_t tsv_token_logprobs_workspace_size(int32_t rows, int32_t V, int32_t top_k);

tsv_status tsv_token_logprobs(const void* logits, int32_t logits_dtype, int32_t rows, int32_t V, const int32_t* targets,
                              float temperature, int32_t top_k, float* logp, int32_t* rank, float* entropy,
                              int32_t* top_tokens, float* top_logp, void* workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * tsv_greedy_tokens - what tsv_lm_head_argmax gives, of logits whose likeliest tokens tsv_token_logprobs has found: argmax
 *   int32 [rows], the first of each row's top_tokens [rows, top_k], and its logit in maxlogit (float [rows] or NULL).  Rows without a
 *   distribution, whose first token is -1, are searched: ties to the lower index, a NaN larger than every number if its
 *   sign bit is clear and smaller if it is set.  logits float [rows, V] as in that call; top_k >= 1.
 */
tsv_status tsv_greedy_tokens(const float* logits, int32_t rows, int32_t V, const int32_t* top_tokens, int32_t top_k,
                             int32_t* argmax, float* maxlogit, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TSV_H */

/*
 * mxsa -- block-sparse KV-outer attention over a paged KV cache, for one
 * GB300 (sm_103a).  C ABI: plain pointers and sizes, no C++ or torch types.
 *
 * The operation (fw-ai/minimax-kernels README, intro and "Quick start"):
 * every query token t of sequence s attends, per KV head g, only to the
 * 128-token logical KV blocks listed in selected[t, g, :] (-1 = none).  In
 * the KV-outer (KV-stationary) formulation each selected block is loaded
 * from HBM once and used for every (query, GQA query head) row that selected
 * it, producing per-row partial outputs and log-sum-exps that a combine step
 * merges.  The call sequence is
 *
 *     mxsa_build_index -> mxsa_schedule -> mxsa_kvouter_fwd -> mxsa_combine
 *
 * all asynchronous on the caller's CUDA stream, followed optionally by
 * mxsa_read_status.  For token t of sequence s (offset i = t - cu[s]) the
 * result is, with L = used_kv_lens[s], Tq_s = cu[s+1] - cu[s], pos(t) =
 * L - Tq_s + i, G = Hq / Hkv and g = h / G:
 *
 *     K(t,g)   = { p : p in a selected block b (128 b <= p < 128 b + 128),
 *                  p < L, and p <= pos(t) when causal }
 *     s_p      = softmax_scale * q[t,h,:] . k_p
 *     out[t,h] = sum_p softmax(s)_p * v_p            (0 when K(t,g) is empty)
 *     lse[h,t] = log sum_p exp(s_p)   (natural log; -inf when K is empty)
 *
 * Key p lives at k_cache[block_tables[s][p / page_size], g, p % page_size, :].
 *
 * Conventions shared by every entry point:
 *   - The caller owns every buffer; the library allocates nothing (no
 *     cudaMalloc, no host allocation) and keeps no state between calls.
 *   - "device" pointers must point to GPU memory of the current device;
 *     all must be 16-byte aligned and densely packed in the stated layout.
 *   - Host-side argument errors return synchronously with a status code; the
 *     library never falls back to another implementation silently.
 *   - Data errors found on the device (a selection outside [-1, nblk), a
 *     repeated block in one row, a bad page id, ...) set bits in a status
 *     word inside the index workspace and skip the offending slot or page;
 *     they never trap.  mxsa_read_status returns that word.
 *   - Calls on one workspace set must be ordered on one stream.
 */
#ifndef MXSA_H_
#define MXSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MXSA_OK = 0,
  MXSA_ERR_INVALID_ARG = 1, /* null/misaligned pointer, inconsistent shape */
  MXSA_ERR_UNSUPPORTED = 2, /* head_dim != 128, page_size not 64/128, G > 128, ... */
  MXSA_ERR_WORKSPACE = 3,   /* a workspace is smaller than mxsa_workspace_size says */
  MXSA_ERR_CUDA = 4,        /* a CUDA runtime/driver call failed */
  MXSA_ERR_DATA = 5         /* mxsa_read_status: the device flagged bad input data */
} mxsa_status;

typedef enum { MXSA_BF16 = 0, MXSA_FP16 = 1, MXSA_FP8_E4M3 = 2, MXSA_NVFP4 = 3 } mxsa_dtype;

/* MXSA_NVFP4 caches (the MSA summary page, "Highlighted Details", lists
 * NVFP4 among the formats of sparse attention and decoding; the layout and
 * the scaling are this library's): OCP MX FP4 E2M1 codes, each 16
 * consecutive elements of a row sharing one E4M3 scale (value = e2m1 *
 * scale, no per-tensor scale).  A cache is bytes [num_pages][Hkv][page_size
 * * 72]: per (page, kv head) slab, page_size rows of 64 code bytes (element
 * 2i in the low nibble of byte i, 2i + 1 in the high one) and then
 * page_size rows of 8 scale bytes (scale j for elements 16 j .. 16 j + 15). */

/* Bits of the device status word (mxsa_read_status). */
#define MXSA_FLAG_SEL_RANGE 1   /* selected block outside [-1, ceil(L/128)) : slot ignored */
#define MXSA_FLAG_SEL_DUP 2     /* block repeated in one (token, kv head) row: later slot ignored */
#define MXSA_FLAG_PAGE 4        /* a needed block_tables entry outside [0, num_pages): page skipped */
#define MXSA_FLAG_CAUSAL_LEN 8  /* causal with used_kv_len < new tokens of the sequence */
#define MXSA_FLAG_LEN 16        /* used_kv_len < 0 or > max_pages_per_seq * page_size: clamped */
#define MXSA_FLAG_TIMEOUT 32    /* an on-device wait gave up (result undefined) */
#define MXSA_FLAG_SCHEDULE 64   /* schedule and forward disagree on the CTA count */
#define MXSA_FLAG_CU 128        /* cu_seqlens_q is not a non-decreasing partition of total_q */
#define MXSA_FLAG_POS 256       /* a token's position lies past the rotation table: token left out */
#define MXSA_FLAG_GROUP 512     /* group_ptr is not a non-decreasing list of sequences: groups ignored */
#define MXSA_FLAG_TREE 1024     /* a drafted tree's parents, path or mask width do not fit it */
#define MXSA_FLAG_PAGES 2048    /* free list with too few pages, or one that does not fit, or what goes back is no
                                 * page of the cache: nothing given out */

/* Problem description (sizes and flags of one call).  The sources: the
 * Quick-start signature and the supported-feature list of the
 * fw-ai/minimax-kernels README. */
typedef struct {
  int32_t num_seqs;          /* B >= 1 */
  int32_t total_q;           /* Tq = cu_seqlens_q[B] >= 0 */
  int32_t num_q_heads;       /* Hq */
  int32_t num_kv_heads;      /* Hkv; Hq % Hkv == 0 and G = Hq / Hkv <= 128 */
  int32_t head_dim;          /* must be 128 */
  int32_t topk;              /* selection slots per (token, kv head), 1..256 */
  int32_t page_size;         /* 64 or 128 tokens */
  int32_t num_pages;         /* physical pages in k_cache / v_cache */
  int32_t max_pages_per_seq; /* row stride of block_tables */
  int32_t causal;            /* 0 or 1 (bottom-right aligned: pos(t) = L - Tq_s + i) */
  float softmax_scale;       /* 0 means 1/sqrt(128) */
  int32_t q_dtype;           /* MXSA_BF16 or MXSA_FP16; the output has this dtype */
  int32_t kv_dtype;          /* q_dtype, MXSA_FP8_E4M3 (unscaled e4m3fn) or MXSA_NVFP4 */
} mxsa_problem;

/* Library version, (major << 16) | minor.  (This library's own; the pages
 * describe no C API.) */
int32_t mxsa_version(void);

/* Human-readable name of a status code (static string).  (This library's
 * own; no passage.) */
const char* mxsa_status_string(mxsa_status status);

/* Workspace sizes (bytes) for a problem.  No passage of the pages defines
 * this call: the README's Quick-start API allocates internally, and this
 * caller-owned-workspace design is the library's own.  Upper bounds computed
 * from the shapes alone (independent of the CTA count: the schedule's
 * per-CTA arrays are sized for MXSA_MAX_CTAS), so one allocation serves
 * any selections / lengths of that shape.  index: inverted block index +
 * device status word; sched: work items and the per-CTA partition; partial:
 * partial outputs and lses, one row of 128 values plus one FP32 lse per
 * (selected block, query head) pair; the rows are FP32 when kv_dtype is
 * MXSA_FP8_E4M3 or MXSA_NVFP4, else in the 16-bit q_dtype.
 * Returns MXSA_ERR_INVALID_ARG / MXSA_ERR_UNSUPPORTED for bad problems. */
mxsa_status mxsa_workspace_size(const mxsa_problem* problem, size_t* index_bytes, size_t* sched_bytes,
                                size_t* partial_bytes);

/* Step 1 -- index builder ("index builder" in the README's test list; the
 * algorithm is this library's): inverts the query -> block selections into
 * block -> (token, head group) lists.  Keys are (kv head g, sequence s,
 * block b) in that order; within a key the entries are the selection slots
 * (t * Hkv + g) * topk + k in increasing t (bit-exact, deterministic).
 *   sel           device int32 [total_q, Hkv, topk], -1 = none
 *   cu_seqlens_q  device int64 [B + 1]
 *   used_kv_lens  device int32 [B]
 *   index_ws      device, index_bytes from mxsa_workspace_size (written)
 * Asynchronous on `stream` (a cudaStream_t; NULL = legacy default stream). */
mxsa_status mxsa_build_index(const mxsa_problem* problem, const int32_t* sel, const int64_t* cu_seqlens_q,
                             const int32_t* used_kv_lens, void* index_ws, size_t index_bytes, void* stream);

/* Step 1, cross-sequence variant.  The README's intro (fw-ai/minimax-kernels)
 * makes the KV block the unit that is loaded once for every query that
 * selected it; with a paged cache, sequences that share a cached prefix
 * point their block_tables at the same physical pages, and this build
 * keys such blocks by the pages, not by the sequence (the rule is this
 * library's reading of that passage):
 *   a block (s, b) is shareable when it is full (128 b + 128 <= L_s) and
 *   its pages (block_tables[s][b] for page_size 128, [2b] and [2b + 1] for
 *   64) lie in [0, num_pages); owner(s, b) = the smallest sequence s' whose
 *   block b is shareable with the same pages (s itself when none is
 *   smaller; a block that is not shareable owns itself); a selection of
 *   (s, b) becomes an entry of key g * NB + blk_off[owner] + b.
 * Everything else is mxsa_build_index's definition: keys (g, s, b) in that
 * order (a key whose rows moved to an owner holds no entries), entries by
 * slot within a key, the same flags and workspace.  A key then holds rows
 * of several sequences; each keeps its own causal position, which the
 * forward reads per row.  mxsa_schedule and mxsa_kvouter_fwd take the
 * result as they take the plain index; mxsa_plan builds the plain index
 * only.
 *   block_tables  device int32 [B, max_pages_per_seq]
 *   dedup_ws      device scratch, dedup_bytes from mxsa_dedup_workspace_size
 *                 (its contents need no initialisation and are not kept)
 * Other arguments as for mxsa_build_index.  Asynchronous on `stream`. */
mxsa_status mxsa_dedup_workspace_size(const mxsa_problem* problem, size_t* dedup_bytes);
mxsa_status mxsa_build_index_dedup(const mxsa_problem* problem, const int32_t* sel, const int64_t* cu_seqlens_q,
                                   const int32_t* used_kv_lens, const int32_t* block_tables, void* index_ws,
                                   size_t index_bytes, void* dedup_ws, size_t dedup_bytes, void* stream);

/* Step 2 -- load-balancing scheduler ("load-balancing scheduler" in the
 * README's test list; the split rule and cost model are this library's):
 * splits each key's entries into work items of at most 4 tiles of 128
 * (token, head) rows and partitions the items into `num_ctas` contiguous
 * ranges of near-equal integer cost.
 *   index_ws   device, written by mxsa_build_index on the same stream
 *   num_ctas   persistent CTAs of the forward; 0 = one per SM of the
 *              current device; at most 4096
 *   sched_ws   device, sched_bytes from mxsa_workspace_size (written) */
mxsa_status mxsa_schedule(const mxsa_problem* problem, const void* index_ws, size_t index_bytes,
                          int32_t num_ctas, void* sched_ws, size_t sched_bytes, void* stream);

/* Steps 1 and 2 in one launch: the same index and schedule as
 * mxsa_build_index followed by mxsa_schedule (bit-identical workspaces),
 * with one kernel launch instead of two.  Arguments as for those calls. */
mxsa_status mxsa_plan(const mxsa_problem* problem, const int32_t* sel, const int64_t* cu_seqlens_q,
                      const int32_t* used_kv_lens, void* index_ws, size_t index_bytes, int32_t num_ctas,
                      void* sched_ws, size_t sched_bytes, void* stream);

/* Step 3 -- KV-outer forward (the README's intro): every work item TMA-loads
 * its KV block (through block_tables) into shared memory once, gathers the
 * q rows of every (token, head) that selected it, and runs q k^T and p v on
 * the tcgen05 tensor cores with FP32 accumulators in tensor memory and the
 * softmax in registers.  Writes one partial row o = sum softmax * v over
 * the block's keys (accumulated in FP32; stored as FP32 with FP8 caches,
 * else rounded to nearest-even in q_dtype: o is a convex combination of V
 * rows, so it stays within their range) and its FP32 lse per (entry, head)
 * into partial_ws.
 *   q             device [total_q, Hq, 128] of q_dtype
 *   k_cache/v_cache device [num_pages, Hkv, page_size, 128] of kv_dtype
 *                 (MXSA_NVFP4: the byte slabs described at mxsa_dtype; FP8
 *                 and NVFP4 blocks are widened exactly to q_dtype before
 *                 the MMAs)
 *   block_tables  device int32 [B, max_pages_per_seq]
 *   num_ctas      must equal the value given to mxsa_schedule (0 = #SMs)
 *   partial_ws    device, partial_bytes from mxsa_workspace_size (written) */
mxsa_status mxsa_kvouter_fwd(const mxsa_problem* problem, const void* q, const void* k_cache,
                             const void* v_cache, const int32_t* block_tables, const void* index_ws,
                             size_t index_bytes, const void* sched_ws, size_t sched_bytes, int32_t num_ctas,
                             void* partial_ws, size_t partial_bytes, void* stream);

/* Step 4 -- combine ("combine" kernel in the README's "Tests" list; output
 * [Tq, Hq, 128] and FP32 lse [Hq, Tq] from its "Quick start"): for each
 * (t, h) merges the partials of the row's selected blocks with LSE weights,
 * in FP32: M = max lse_k, w_k = exp(lse_k - M),
 * out = sum w_k o_k / sum w_k (rounded to nearest-even into q_dtype),
 * lse = M + log sum w_k.  A row with no partial gets out 0 and lse -inf.
 *   out   [total_q, Hq, 128] of q_dtype (written): device memory, or pinned
 *         host memory mapped at the same address (unified addressing), which
 *         the kernel then writes directly over the host link
 *   lse   float [Hq, total_q] (written), same memory rules, or NULL to skip it
 * Pageable host memory or an unknown pointer for out/lse returns
 * MXSA_ERR_INVALID_ARG before any launch. */
mxsa_status mxsa_combine(const mxsa_problem* problem, const void* index_ws, size_t index_bytes,
                         const void* partial_ws, size_t partial_bytes, void* out, float* lse, void* stream);

/* This library's own (no passage; the README's "Backends" section only
 * asks that errors are raised rather than hidden).
 * Synchronises `stream`, then copies the device status word (MXSA_FLAG_*
 * bits) of index_ws into *device_flags.  Returns MXSA_ERR_DATA when any bit
 * is set, MXSA_OK otherwise. */
mxsa_status mxsa_read_status(const void* index_ws, void* stream, int32_t* device_flags);

/* Dense paged attention, the all-blocks-selected case computed directly (no
 * partials, no combine; the MSA project page lists a dense FMHA path next to
 * the sparse one): for token t of sequence s and query head h,
 *   out[t][h][:] = sum_p softmax_p(scale * q[t][h] . k_p) v_p,
 *   lse[h][t] = log sum_p exp(scale * q[t][h] . k_p)   (natural log),
 * over keys p < used_kv_lens[s] (and p <= pos(t) = L - Tq_s + i when causal),
 * k_p / v_p read through block_tables as in mxsa_kvouter_fwd.  No key: out 0,
 * lse -inf.  Same tensors and layouts as the sparse path (q, caches, out
 * [total_q][Hq][128] in q_dtype, lse [Hq][total_q] or NULL); topk is unused
 * and not checked, nor are the sparse index's size limits.
 * kv_dtype must equal q_dtype (BF16/FP16); num_seqs <= 1024.  Tokens outside
 * every sequence (cu_seqlens_q out of order or past total_q) are not written.
 * device_flags (device int32, may be NULL): MXSA_FLAG_PAGE when a needed
 * block_tables entry lies outside [0, num_pages) (that page is skipped and its
 * rows' results are undefined), MXSA_FLAG_TIMEOUT.  Device pointers; q, caches
 * and out 16-byte aligned.  One launch, asynchronous on `stream`;
 * MXSA_ERR_INVALID_ARG / MXSA_ERR_UNSUPPORTED before any launch. */
mxsa_status mxsa_dense_fwd(const mxsa_problem* problem, const void* q, const void* k_cache, const void* v_cache,
                           const int32_t* block_tables, const int64_t* cu_seqlens_q, const int32_t* used_kv_lens,
                           void* out, float* lse, int32_t* device_flags, void* stream);

/* Dense paged attention of a batch whose sequences share prefixes (this
 * library's own; the plain dense path is mxsa_dense_fwd, the sparse one with
 * shared blocks mxsa_build_index_dedup): out and lse of mxsa_dense_fwd, each
 * common key loaded once for all the sequences that have it, and every
 * sequence's keys split over the whole GPU (also without groups: a batch of
 * few sequences with many keys).  Group j is the sequences group_ptr[j] <= s <
 * group_ptr[j + 1]; its prefix is
 *   P_j = prefix_lens[j], at least 0 and at most the smallest used_kv_len
 *         among its sequences with new tokens (0 for a group of one sequence);
 *   keys p < P_j of all its sequences are read through the block_tables row
 *   of sequence group_ptr[j], keys p >= P_j through their own.
 * P_j need not fill a block or a page (a page that holds a prefix's end is
 * read twice, by both ways).  Entries of the other rows for pages wholly
 * below P_j are not read.  Sequences in no group have no prefix.
 *   group_ptr    device int32 [num_groups + 1], 0 <= non-decreasing <= B;
 *                else MXSA_FLAG_GROUP and no group at all
 *   prefix_lens  device int32 [num_groups]
 *   num_groups   0 (both may be NULL) .. num_seqs
 *   ws           device, shared_bytes from mxsa_shared_workspace_size: plan
 *                and partial rows (FP32); needs no initialisation, keeps
 *                nothing between calls
 * The other arguments and limits are mxsa_dense_fwd's: kv_dtype = q_dtype,
 * num_seqs <= 1024, topk unused; total_q * num_q_heads < 2^29 - 2^17 always
 * fits.  The softmax weights are rounded to q_dtype before they multiply V,
 * everything else is FP32.  A NaN or infinity at a key outside
 * [0, used_kv_len) of a sequence does not reach its rows; under causal masking
 * the V rows of keys that come after a token but that others of its group see
 * have to be finite.  An infinity in V at a key that a row sees makes its
 * column of the row infinite or NaN (a tile of few rows multiplies it by
 * zeros too).  Results do not depend on timing: the same call gives the
 * same bits.  Two calls that may run at the same time, captured graphs
 * included, need a ws each.
 * cu_seqlens_q must be non-decreasing within [0, total_q], else MXSA_FLAG_CU
 * and nothing is written; tokens before cu_seqlens_q[0] and from
 * cu_seqlens_q[B] on are not written.  device_flags (may be NULL) also gets
 * MXSA_FLAG_LEN (clamped length), MXSA_FLAG_PAGE and MXSA_FLAG_TIMEOUT as
 * for mxsa_dense_fwd.  Three launches, asynchronous on `stream`. */
mxsa_status mxsa_shared_workspace_size(const mxsa_problem* problem, size_t* shared_bytes);
mxsa_status mxsa_dense_shared_fwd(const mxsa_problem* problem, const void* q, const void* k_cache,
                                  const void* v_cache, const int32_t* block_tables, const int64_t* cu_seqlens_q,
                                  const int32_t* used_kv_lens, int32_t num_groups, const int32_t* group_ptr,
                                  const int32_t* prefix_lens, void* ws, size_t shared_bytes, void* out, float* lse,
                                  int32_t* device_flags, void* stream);

/* Attention of drafted token trees over the paged cache, the verification
 * step of speculative decoding (this library's own; the plain dense path is
 * mxsa_dense_shared_fwd).  A sequence's Tq_s new tokens are the nodes of a
 * tree (or of several) whose keys already stand in the cache, in the order of
 * the tokens, behind its base_s = L - Tq_s committed ones.  Token i of s sees
 *   every key p < base_s, and key base_s + j when bit j % 32 of
 *   tree_mask[t][j / 32] is set (its ancestors' and its own bit, as
 *   mxsa_tree_mask writes them, or any other set),
 * and out, lse are mxsa_dense_fwd's over those keys (none: out 0, lse -inf).
 * tree_mask is device uint32 [total_q][mask_words], 1 <= mask_words <= 64; a
 * sequence of more than 32 * mask_words new tokens sets MXSA_FLAG_TREE, and
 * the further ones' keys are seen by no row.  L < Tq_s sets
 * MXSA_FLAG_CAUSAL_LEN; the first Tq_s - L tokens then have no key.
 * Everything else is mxsa_dense_shared_fwd's: the groups (each prefix at most
 * the smallest base_s of the group's sequences with new tokens), the workspace
 * (mxsa_shared_workspace_size), limits, types, roundings and flags;
 * problem->causal is not used.  The V rows of drafted keys that a row does not
 * see, but others of its sequence do, have to be finite.  kv_dtype equals
 * q_dtype as there: rows of FP8 and NVFP4 caches, which mxsa_tree_commit does
 * take, have to be widened first (mxsa_load_kv).  One launch for few sequences
 * with tables (max_pages_per_seq, whatever the lengths) of moderate width and no
 * groups: ws is then given but not used; else three; asynchronous on `stream`. */
mxsa_status mxsa_tree_fwd(const mxsa_problem* problem, const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_tables, const int64_t* cu_seqlens_q, const int32_t* used_kv_lens,
                          const uint32_t* tree_mask, int32_t mask_words, int32_t num_groups,
                          const int32_t* group_ptr, const int32_t* prefix_lens, void* ws, size_t shared_bytes,
                          void* out, float* lse, int32_t* device_flags, void* stream);

/* Masks and positions of drafted trees (this library's own).  parents[t] is
 * the index of token t's parent among its sequence's new tokens, smaller than
 * t's own, or -1 for a token that follows the last committed one.
 *   tree_mask[t][w]: bit j of word w set when new token 32 w + j of the
 *                    sequence is t or an ancestor of t
 *   positions[t]   = used_kv_lens[s] - Tq_s + (number of t's ancestors), the
 *                    position that its rotation takes (NULL to skip it)
 *   parents        device int32 [total_q]
 *   positions      device int64 [total_q]
 * A parent outside [-1, own index) sets MXSA_FLAG_TREE and stands for -1; a
 * sequence of more than 32 * mask_words tokens (1..64 words) sets it too, its
 * further tokens' bits left out and, of a token with more than 2048 ancestors,
 * those beyond the nearest 2048 neither set nor counted.  MXSA_FLAG_LEN and
 * MXSA_FLAG_CAUSAL_LEN as for the calls that read the lengths (clamped; L <
 * Tq_s: positions below zero).
 * Tokens before cu_seqlens_q[0] and from cu_seqlens_q[B] on are not written;
 * cu_seqlens_q out of order: MXSA_FLAG_CU and nothing is.  The outputs overlap
 * neither an input nor one another.  Of the problem the call reads num_seqs
 * (<= 1024), total_q, page_size and max_pages_per_seq.  One launch,
 * asynchronous on `stream`. */
mxsa_status mxsa_tree_mask(const mxsa_problem* problem, const int32_t* parents, const int64_t* cu_seqlens_q,
                           const int32_t* used_kv_lens, int32_t mask_words, uint32_t* tree_mask, int64_t* positions,
                           int32_t* device_flags, void* stream);

/* The accepted tokens of drafted trees moved to their places (this library's
 * own): for each sequence s, with base_s = used_kv_lens[s] - Tq_s and the
 * accepted path p_0 < p_1 < ... of path_lens[s] token indices in path[s],
 * the K and V rows of every kv head (and the index keys' of every index head)
 * at position base_s + p_k become those at base_s + k, and
 *   kv_lens_out[s] = base_s + path_lens[s].
 * The result is that of reading every row before any is written.  Any cache
 * type; rows are copied as they are.  One call per layer's caches.
 *   path        device int32 [B][max_path], read up to path_lens[s]
 *   path_lens   device int32 [B], 0 .. max_path
 *   idx_cache   as for mxsa_store_kv, or NULL (idx_heads, idx_dim unused)
 *   kv_lens_out device int32 [B], apart from every other array, or NULL
 * A path that is not ascending within [0, Tq_s), or longer than max_path, sets
 * MXSA_FLAG_TREE; a length out of range MXSA_FLAG_LEN or, below Tq_s,
 * MXSA_FLAG_CAUSAL_LEN; cu_seqlens_q out of order MXSA_FLAG_CU: of such a
 * sequence nothing is moved, and kv_lens_out[s] is what is committed of it (0
 * at least).  A row whose page lies outside the cache is not moved
 * (MXSA_FLAG_PAGE).  Sequences must not share the pages that hold their
 * drafted tokens.  One launch, asynchronous on `stream`. */
mxsa_status mxsa_tree_commit(const mxsa_problem* problem, const int64_t* cu_seqlens_q, const int32_t* used_kv_lens,
                             const int32_t* block_tables, const int32_t* path, int32_t max_path,
                             const int32_t* path_lens, void* k_cache, void* v_cache, void* idx_cache,
                             int32_t idx_heads, int32_t idx_dim, int32_t* kv_lens_out, int32_t* device_flags,
                             void* stream);

/* Attention of whole prompts that have no cache yet (this library's own; the
 * paged form is mxsa_dense_fwd): sequence s is the tokens cu_seqlens[s] <= t <
 * cu_seqlens[s + 1] of q, k and v alike, and
 *   out[t][h][:] = sum_u softmax_u(scale * q[t][h] . k[u][g]) v[u][g],
 *   lse[h][t]    = log sum_u exp(scale * q[t][h] . k[u][g]),  g = h / G,
 * over its tokens u (u <= t when problem->causal).  q is [total_q][Hq][128], k
 * and v [total_q][Hkv][128] in q_dtype, a token's heads next to each other and
 * the tokens *_stride elements apart (a multiple of 8, at least heads * 128),
 * so they may be views of one packed projection; out [total_q][Hq][128] in
 * q_dtype and lse [Hq][total_q] (or NULL) are dense and overlap no input.
 *   ws   device, prompt_bytes from mxsa_prompt_workspace_size: the order of
 *        the work; needs no initialisation, keeps nothing between calls.  Two
 *        calls that may run at the same time need one each.
 * The softmax weights are rounded to q_dtype before they multiply V,
 * everything else is FP32; the same call gives the same bits.  NaN and
 * infinities of one sequence do not reach another; under causal masking the V
 * rows of a sequence's later tokens have to be finite.  kv_dtype must equal
 * q_dtype; num_seqs <= 1024; topk and the pages of the problem are not used.
 * Tokens before cu_seqlens[0] and from cu_seqlens[B] on are not written;
 * cu_seqlens out of order: MXSA_FLAG_CU in device_flags (may be NULL) and
 * nothing is written (MXSA_FLAG_TIMEOUT as everywhere).  Device pointers,
 * 16-byte aligned (ws 256).  One or two launches, asynchronous on `stream`. */
mxsa_status mxsa_prompt_workspace_size(const mxsa_problem* problem, size_t* prompt_bytes);
mxsa_status mxsa_prompt_fwd(const mxsa_problem* problem, const void* q, int64_t q_stride, const void* k,
                            int64_t k_stride, const void* v, int64_t v_stride, const int64_t* cu_seqlens, void* ws,
                            size_t prompt_bytes, void* out, float* lse, int32_t* device_flags, void* stream);

/* A serving step's tables, built on the GPU from the requests' lengths (this
 * library's own): what every paged call above takes.  Request s has kv_lens[s]
 * tokens in the cache, in pages_held[s] pages (the first entries of its row of
 * block_tables), and new_lens[s] >= 0 new ones in this step; new_lens[s] < 0:
 * it is finished.
 *   1. The pages of finished requests go back to the free list, behind its
 *      free_count[0] pages, in the order of the requests and of their rows.
 *   2. Every other request gets the pages that its kv_lens[s] + new_lens[s]
 *      tokens need beyond pages_held[s], in the order of the requests: the
 *      list's last page first, each into the next entry of its row.
 *   3. cu_seqlens_q = the running sums of the new tokens (0 of a finished
 *      request); used_kv_lens[s] = kv_lens[s] + new_lens[s] (finished: 0);
 *      positions[t] = kv_lens[s] + i and loc[t] = its slot page * page_size +
 *      offset for token t = cu_seqlens_q[s] + i; -1 in both from
 *      cu_seqlens_q[B] to total_q (padding to the calls that take them).
 *      pages_held_out and free_count_out: what the requests hold now, and the
 *      list's new length.
 *   kv_lens, new_lens, pages_held   device int32 [B]
 *   block_tables   device int32 [B][max_pages_per_seq] (updated)
 *   free_pages     device int32 [num_pages] (updated)
 *   free_count     device int32 [1]
 *   cu_seqlens_q   device int64 [B + 1]; used_kv_lens, pages_held_out device
 *                  int32 [B]; positions, loc device int64 [total_q]
 *                  (total_q: the step's capacity); free_count_out int32 [1]
 * The call does not look for pages that several rows hold: what a finished
 * request gives back is free from then on, whoever else reads it, and a page
 * given back twice is handed out twice.  So a page that goes back must be among
 * no other request's first pages_held entries, finished or not, nor in the free
 * list already.  Requests that share a prefix's pages (the groups of
 * mxsa_dense_shared_fwd and mxsa_tree_fwd) may have them in their rows and
 * counts as long as they run; before one of them is finished here while others
 * still read them, they have to leave its first pages_held[s] entries (its own
 * pages moved to the front and pages_held[s] their number; 0: nothing goes
 * back).  The last one gives them back.
 * used_kv_lens may be kv_lens, pages_held_out pages_held and free_count_out
 * free_count; otherwise no two arrays overlap.  When the new tokens are more
 * than total_q (MXSA_FLAG_CU), a length, a held count or a row does not fit
 * (MXSA_FLAG_LEN: kv_lens[s] < 0 or beyond the held pages, pages_held[s]
 * outside [0, max_pages_per_seq], more tokens than a row's pages hold), or the
 * list has too few pages or would outgrow num_pages, or an entry that a finished
 * request gives back lies outside [0, num_pages) (MXSA_FLAG_PAGES), no page
 * moves: cu_seqlens_q is all 0, positions and loc all -1, the lengths, held
 * counts and list as they came.  A slot in a page outside [0, num_pages) is -1
 * (MXSA_FLAG_PAGE).  Of the problem the call reads num_seqs (<= 1024), total_q,
 * page_size, num_pages and max_pages_per_seq.  positions and loc 16-byte
 * aligned.  One or two launches, asynchronous on `stream`. */
mxsa_status mxsa_build_tables(const mxsa_problem* problem, const int32_t* kv_lens, const int32_t* new_lens,
                              const int32_t* pages_held, int32_t* block_tables, int32_t* free_pages,
                              const int32_t* free_count, int64_t* cu_seqlens_q, int32_t* used_kv_lens,
                              int64_t* positions, int64_t* loc, int32_t* pages_held_out, int32_t* free_count_out,
                              int32_t* device_flags, void* stream);

/* Paged-cache store, the write side of the caches the forward reads (a
 * sglang pull request on these pages, "Summary": the fused K/V/index store
 * with an unscaled bf16-to-fp8_e4m3 cast).  For each of n_tokens new tokens
 * with slot loc[t] = page * page_size + offset (device int64; loc[t] < 0:
 * token t is not stored):
 *   k_cache[page][h][offset][:] = cast(k[t][h][:]) and likewise v, h < Hkv;
 *   idx_cache[page][j][offset][:] = cast(idx_k[t][j][:]), j < idx_heads.
 * k, v: [n_tokens][num_kv_heads][128] in problem->q_dtype (bf16 or fp16);
 * idx_k: [n_tokens][idx_heads][idx_dim], same dtype, idx_dim a multiple of 8.
 * Of the problem, the store reads the head counts, page size, page count and
 * dtypes; topk, total_q and the sequence fields are not checked.
 * Caches: [num_pages][heads][page_size][dim] in problem->kv_dtype, which is
 * q_dtype (bits copied), MXSA_NVFP4 or MXSA_FP8_E4M3.  MXSA_NVFP4 (the slab
 * layout at mxsa_dtype; no index keys): a group of 16 values stores the
 * scale e4m3(amax / 6) (amax over its non-NaN |x|, single-precision
 * division, rounded as below) and, with sd that scale's value, the E2M1
 * code nearest to x / sd (single precision), ties to even, saturating at
 * 6, with the quotient's sign; NaN elements and groups whose scale is 0
 * store code 0.  MXSA_FP8_E4M3: each value becomes x clamped to
 * [-448, 448] rounded to the nearest e4m3fn value, ties to even, NaN keeping
 * its sign -- bit-identical to x.float().clamp(-448, 448).to(float8_e4m3fn).
 * idx_k and idx_cache are both NULL (no index keys) or both set.
 * device_flags (device int32, may be NULL): MXSA_FLAG_PAGE is ORed in when a
 * slot lies at or past num_pages * page_size (that token is not stored).
 * Device pointers, 16-byte aligned (loc 8-byte); the caller owns all of them.
 * One launch, asynchronous on `stream`.  MXSA_ERR_INVALID_ARG /
 * MXSA_ERR_UNSUPPORTED for bad arguments, before any launch. */
mxsa_status mxsa_store_kv(const mxsa_problem* problem, int64_t n_tokens, const int64_t* loc, const void* k,
                          const void* v, void* k_cache, void* v_cache, const void* idx_k, void* idx_cache,
                          int32_t idx_heads, int32_t idx_dim, int32_t* device_flags, void* stream);

/* Paged-cache load, the read side of mxsa_store_kv (this library's own; no
 * passage): for each of n_tokens slots loc[t] = page * page_size + offset
 * (device int64; loc[t] < 0: the token's rows are left as they are)
 *   k[t][h][:] = widen(k_cache[page][h][offset][:]) and likewise v, h < Hkv;
 *   idx_k[t][j][:] = widen(idx_cache[page][j][offset][:]), j < idx_heads,
 * into [n_tokens][heads][dim] rows of problem->q_dtype (BF16 or FP16).  The
 * widening is exact: 16-bit caches are copied bit for bit, e4m3 values and
 * the NVFP4 products e2m1 * scale are values of both 16-bit types (a NaN
 * code or scale gives NaN).  The way from a quantised cache to the calls
 * that take 16-bit keys (mxsa_dense_fwd, mxsa_dense_shared_fwd), to another
 * cache type (mxsa_store_kv of the rows), or to a host.  A slot may occur
 * several times.
 * Of the problem, the load reads what the store reads; the index arguments
 * (both NULL or both set, no NVFP4) and device_flags (MXSA_FLAG_PAGE: a slot
 * past the cache, its token left as it is) are the store's too.
 * Device pointers, 16-byte aligned (loc 8-byte); the outputs must not overlap
 * the caches.  One launch, asynchronous on `stream`; MXSA_ERR_INVALID_ARG /
 * MXSA_ERR_UNSUPPORTED for bad arguments, before any launch. */
mxsa_status mxsa_load_kv(const mxsa_problem* problem, int64_t n_tokens, const int64_t* loc, const void* k_cache,
                         const void* v_cache, void* k, void* v, const void* idx_cache, void* idx_k,
                         int32_t idx_heads, int32_t idx_dim, int32_t* device_flags, void* stream);

/* The prologue of an attention layer (this library's own; no passage): the
 * RMS norm of every query and key head, the rotation by position and the
 * paged-cache store in one pass over a projection's output.  A head row x of
 * D values (D = 128; index rows: idx_dim) with weight row w becomes
 *   y_i = x_i / sqrt((1/D) sum x_j^2 + eps) * w_i      (no norm when w is NULL)
 *   (y_a, y_b) <- (y_a c_i - y_b s_i, y_b c_i + y_a s_i),  i < rot_dim / 2,
 * (a, b) = (i, i + rot_dim / 2), or (2 i, 2 i + 1) when interleaved; columns
 * from rot_dim on are not rotated.  c_i and s_i are cos_sin[pos][i] and
 * cos_sin[pos][rot_dim / 2 + i], pos = positions[t].  All in FP32 (so rows
 * whose squares sum past FP32's range give 0), rounded once:
 *   q_out[t][h][:]     = the row of q[t][h], in q_dtype, dense;
 *   k_cache, v_cache   = the rows of k, and v as it is, at slot loc[t], with
 *                        mxsa_store_kv's casts (applied to the FP32 row of k,
 *                        whose NaN have no sign: 0x7F in an FP8 cache);
 *   idx_q_out[t][g][:] = the row of idx_q[t][g], in kv_dtype, dense (what
 *                        mxsa_select_blocks takes), g < Hkv;
 *   idx_cache          = the rows of idx_k, at slot loc[t], in kv_dtype.
 * q, k, v, idx_q and idx_k are in q_dtype, the heads of a token next to each
 * other and the tokens *_stride elements apart (a multiple of 8, at least
 * heads * D), so they may be views of one packed projection.  Weights are in
 * q_dtype: [D], or [heads][D] when weight_per_head.
 * A token with positions[t] < 0 is padding: nothing of it is written.  One
 * at or past num_positions is left out too and sets MXSA_FLAG_POS.  loc[t] <
 * 0: its k, v and idx_k are not stored; past the cache: the same, and
 * MXSA_FLAG_PAGE.  Slots should be distinct: one that occurs twice holds a
 * mixture of its tokens' rows, each value (in an NVFP4 cache: each byte, so
 * that codes may stand under the other token's scale) one of theirs.
 * idx_dim 0: the idx_* pointers are NULL; else 64 or 128, none of idx_q,
 * idx_k, idx_q_out, idx_cache NULL, rot_dim <= idx_dim, kv_dtype not NVFP4.
 * Of the problem, the call reads what mxsa_store_kv reads and num_q_heads.
 * q_out may be q itself when q is dense; no other output may overlap an
 * input.  Device pointers, 16-byte aligned (positions, loc 8-byte).  One
 * launch, asynchronous on `stream`; MXSA_ERR_INVALID_ARG /
 * MXSA_ERR_UNSUPPORTED before any launch. */
typedef struct {
  int64_t q_stride, k_stride, v_stride; /* elements between tokens */
  int64_t idx_q_stride, idx_k_stride;
  int64_t num_positions;                /* rows of cos_sin, >= 1 */
  int32_t rot_dim;                      /* a multiple of 16, 16..128 */
  int32_t interleaved;                  /* 0 or 1 */
  int32_t weight_per_head;              /* 0 or 1 */
  int32_t idx_dim;                      /* 0 (none), 64 or 128 */
  float eps;                            /* >= 0 */
} mxsa_norm_rope;
mxsa_status mxsa_norm_rope_store(const mxsa_problem* problem, const mxsa_norm_rope* cfg, int64_t n_tokens,
                                 const int64_t* positions, const int64_t* loc, const float* cos_sin, const void* q,
                                 const void* k, const void* v, const void* q_weight, const void* k_weight,
                                 void* q_out, void* k_cache, void* v_cache, const void* idx_q, const void* idx_k,
                                 const void* idx_q_weight, const void* idx_k_weight, void* idx_q_out,
                                 void* idx_cache, int32_t* device_flags, void* stream);

/* Top-k block selection, the step before mxsa_build_index: which 128-token
 * blocks each (token, kv head) row attends to.  The MSA summary page ("How
 * It Works") names the "sparse top-k selection"; the sglang pull request
 * ("Summary") writes an index K cache beside K and V (mxsa_store_kv's
 * idx_cache).  The pages give no scoring rule; this library's reading:
 *   dot(t, g, p)   = the FP32 sum of idx_q[t][g][d] * ik_p[d] over d,
 *                    fused multiply-adds in the order d = 0 .. idx_dim-1
 *                    from +0, where ik_p = idx_cache[block_tables[s][p /
 *                    page_size]][g][p % page_size][:] (one index head per kv
 *                    head); a NaN dot counts as no key;
 *   score(t, g, b) = the largest dot over the block's visible positions:
 *                    128 b <= p < min(128 b + 128, L), p <= pos(t) when
 *                    causal, p on a page in [0, num_pages);
 *   sel[t][g][:]   = the blocks that have a score, by score descending and
 *                    then block ascending (+0 = -0), the first topk of them;
 *                    the remaining slots are -1.
 * The result is exact (bit-identical to a CPU statement of the definition);
 * its rows are valid input for mxsa_plan / mxsa_build_index.
 *   idx_q        device [total_q][Hkv][idx_dim] of kv_dtype (BF16, FP16 or
 *                FP8: an MXSA_NVFP4 problem is MXSA_ERR_UNSUPPORTED)
 *   idx_cache    device [num_pages][Hkv][page_size][idx_dim] of kv_dtype
 *   block_tables, cu_seqlens_q, used_kv_lens as for mxsa_build_index
 *   score_ws     device, score_bytes from mxsa_select_workspace_size: first
 *                the block scores [total_q][Hkv][ceil(max_pages_per_seq *
 *                page_size / 128)] FP32 (NaN: no score), kept for
 *                inspection (entries past a sequence's last block are not
 *                written), then a per-sequence table
 *   sel          device int32 [total_q][Hkv][topk] (written)
 *   device_flags device int32 or NULL: MXSA_FLAG_CU when cu_seqlens_q is not
 *                a non-decreasing partition of total_q (then every row is -1)
 * idx_dim is 64 or 128; num_seqs <= 1024; at most 4096 blocks per sequence.
 * Four launches, asynchronous on `stream`; MXSA_ERR_INVALID_ARG /
 * MXSA_ERR_UNSUPPORTED / MXSA_ERR_WORKSPACE before any launch. */
mxsa_status mxsa_select_workspace_size(const mxsa_problem* problem, int32_t idx_dim, size_t* score_bytes);
mxsa_status mxsa_select_blocks(const mxsa_problem* problem, int32_t idx_dim, const void* idx_q,
                               const void* idx_cache, const int32_t* block_tables, const int64_t* cu_seqlens_q,
                               const int32_t* used_kv_lens, void* score_ws, size_t score_bytes, int32_t* sel,
                               int32_t* device_flags, void* stream);

/* This library's own (no passage).
 * Byte offsets of the arrays inside the index workspace, for inspection
 * (tests compare them bit-exactly with an independent CPU statement).
 * header: int32[16] = {flags, NB (blocks over all sequences), nnz (entries),
 *   n_active (keys with entries), n_keys (Hkv * NB), ...};
 * row_ptr: int32 [n_keys + 1]; entries: int32 [nnz] slot ids;
 * slot_entry: int32 [total_q * Hkv * topk], position in entries or -1;
 * active_keys: int32 [n_active], keys with entries in increasing order. */
typedef struct {
  size_t header, seq_info, token_seq, slot_entry, bitmap, kmap, counts, row_ptr, entries, active_keys,
      active_valid, row_nnz, row_minb, row_maxb, cta_sums, total;
  int64_t keys_cap, nslots, bitmap_words_cap, kmap_bytes_cap, tiles_cap;
} mxsa_index_layout;
mxsa_status mxsa_index_layout_query(const mxsa_problem* problem, mxsa_index_layout* layout);

/* This library's own (no passage).  Byte offsets inside the schedule workspace.  header: int32[16] =
 * {n_items, num_ctas, total cost low, total cost high, (scan counter),
 *  n_dec_items, decode cost low, decode cost high, ...};
 * Two lists, each with int64 exclusive cost prefixes [n + 1] and its own
 * partition cta_ptr int32 [num_ctas + 1]:
 *   items:     int32[4] = {key, entry_begin, n_entries, 0}, keys of
 *              sequences with several new tokens (KV-stationary tiles);
 *   items_dec: int32[4] = {position in active_keys, entry, 1, n_keys}, runs
 *              of up to 8 consecutive decode keys of one sequence and kv
 *              head.  A decode key belongs to a sequence with one new token
 *              (G <= 16) and holds exactly one entry, of that token.  With
 *              the plain index every key of such a sequence is one; with the
 *              dedup index a shared block's key holds several sequences'
 *              entries and goes to the first list.
 * decode_bits: uint32 words, bit a set when active key a is a decode key. */
typedef struct {
  size_t header, items, cost_prefix, cta_ptr, items_dec, cost_prefix_dec, cta_ptr_dec, cta_sums, decode_bits, total;
  int64_t items_cap, tiles_cap;
} mxsa_sched_layout;
mxsa_status mxsa_sched_layout_query(const mxsa_problem* problem, mxsa_sched_layout* layout);

/* The whole call (index, schedule, forward, combine) without any
 * caller-provided workspace.  The pages describe no such entry point; it
 * exists for callers that may not allocate device memory themselves, such as
 * plug-ins of a host runtime that plans every buffer up front, or hot loops
 * that must not risk the device-wide synchronisation a cudaMalloc/cudaFree
 * can cause.  The caller passes inputs and outputs exactly as for the four
 * steps (same layouts and dtypes; lse may be NULL); all scratch lives in one
 * fixed 16 MiB device array inside the library, which every GPU that loads
 * the library keeps reserved until the process exits.  Problems whose three
 * workspaces (mxsa_workspace_size) add up to more than 16 MiB are rejected
 * with MXSA_ERR_WORKSPACE before anything runs.  Nothing is allocated.
 * The first call on a device looks up the array's device address: made
 * while `stream` is being captured it returns MXSA_ERR_INVALID_ARG, as does
 * a stream of another device than the current one (nothing runs).  Calls
 * share the array: calls that overlap on the GPU race and must be
 * serialised by the caller.  Asynchronous on `stream`; the device status
 * word of the last call (data errors, MXSA_FLAG_TIMEOUT) is read with
 * mxsa_noalloc_read_status. */
mxsa_status mxsa_attention_noalloc(const mxsa_problem* problem, const void* q, const void* k_cache,
                                   const void* v_cache, const int32_t* sel, const int32_t* block_tables,
                                   const int64_t* cu_seqlens_q, const int32_t* used_kv_lens, void* out, float* lse,
                                   void* stream);

/* This library's own (no passage), the companion of mxsa_attention_noalloc:
 * synchronises `stream`, then copies the status word (MXSA_FLAG_* bits) that
 * the last mxsa_attention_noalloc call on the current device left in the
 * library's array into *device_flags.  Returns MXSA_ERR_DATA when any bit
 * is set, MXSA_OK otherwise (MXSA_ERR_INVALID_ARG as for that call). */
mxsa_status mxsa_noalloc_read_status(void* stream, int32_t* device_flags);

/* Rows per tile, tiles per normal work item and blocks per decode work item
 * used by the scheduler. */
#define MXSA_TILE_ROWS 128
#define MXSA_ITEM_TILES 4
#define MXSA_DECODE_BLOCKS 8
#define MXSA_MAX_CTAS 4096

#ifdef __cplusplus
}
#endif
#endif /* MXSA_H_ */

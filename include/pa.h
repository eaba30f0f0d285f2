/*
 * pa.h -- paged-attention decode on GB300 (sm_103a): the C ABI of libpa103.so.
 *
 * The operation.  A decode step gives each sequence b a few new query tokens
 * (q_lens[b] <= max_q_len rows per query head) that attend over that
 * sequence's cached keys and values.  The cache is a pool of fixed-size
 * physical pages; sequence b reaches its logical page p at physical block
 * block_tables[b][p] ("HSTU Paged Attention", RecSDK issue 1281, background:
 * historical K/V are read page by page from the paged KV cache).  For query
 * head h (KV head g = h / (Hq / Hkv)) and new-token row i < q_lens[b]:
 *
 *     n   = context_lens[b]          (counts the q_lens[b] new tokens, which are
 *                                     the last q_lens[b] positions)
 *     L   = causal ? n - q_lens[b] + i + 1 : n     visible keys 0 .. L-1
 *     s_j = sm_scale * <q[b,i,h,:], k_j>           k_j = K[block_tables[b][j/bs], j%bs, g, :]
 *     out[b,i,h,:] = sum_j softmax(s)_j v_j ,  lse[b,i,h] = log sum_j exp(s_j)
 *
 * Rows i >= q_lens[b] are padding: out = 0, lse = -inf.
 *
 * The work is split as in "Optimize paged-attention metadata decode" (FlyDSL
 * PR #910, Summary and Changes): a planner emits a work list for a persistent
 * grid of one CTA per SM (times a grid multiplier, default 1); a persistent
 * decode kernel processes it, writing whole results directly and per-range
 * partials (o_s, lse_s) otherwise; a reducer merges the partials by
 *     m* = max_s lse_s,  w_s = exp(lse_s - m*),  out = sum_s w_s o_s / sum_s w_s.
 * fp8 caches hold OCP E4M3 codes with one fp32 scale per tensor, one per
 * (block, slot, kv-head) row (FlyDSL PR #910, per_token_kv scale mode) or one per
 * (block, kv-head).
 *
 * Calling convention.  The caller owns all memory.  pa_plan, pa_decode and
 * pa_reduce allocate nothing, never synchronise the host and never abort: each
 * validates its arguments on the host, enqueues its kernel on `stream` and
 * returns a status.  They are stream-ordered, so the three calls on one stream
 * with one workspace form one decode step and can be captured in a CUDA graph.
 * Problems in the device-resident lengths or block tables cannot be seen by the
 * host.  The planner flags bad lengths and empties the work list (the output is
 * then all zeros with lse = -inf); the decode kernel checks every block id before
 * it loads the page, skips a page outside the pool and flags it (the rows of that
 * sequence are then unspecified).  Either way no kernel touches memory outside the
 * inputs.  pa_read_flags (the one synchronising call) returns the flags.
 *
 * Device pointers: q, k_cache, v_cache, k_scale, v_scale, block_tables,
 * context_lens, q_lens, out, lse and ws.  q, k_cache, v_cache and out must be
 * 16-byte aligned; ws 256-byte aligned.
 *
 * Besides the step, pa_append_kv writes a step's new K/V rows into their pages
 * (quantising them to fp8 where the cache is fp8), and pa_gather_kv copies a batch's
 * cached K and V rows out of the pages into contiguous buffers (the workspace copy of
 * the HSTU paged attention), with the same calling convention.  pa_build_tables grows and
 * shrinks block tables from the requests' lengths.  pa_append_rotated makes a projection's queries and
 * keys ready (norms, rotary positions) as it appends, and pa_dequant_kv reads a quantised cache back as
 * 16-bit rows.  A step that attends over a part of its
 * cached pages keeps channel bounds of every page's keys (pa_update_bounds), scores the pages
 * with them (pa_score_blocks), selects pages by score (pa_select_blocks) and attends over the
 * selected ones (pa_decode_selected).
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Entry points are the only symbols the library exports. */
#if defined(__GNUC__)
#define PA_API __attribute__((visibility("default")))
#else
#define PA_API
#endif

/* The same type as cudaStream_t; 0 is the legacy default stream. */
typedef struct CUstream_st *pa_stream;

typedef enum {
  PA_OK = 0,
  PA_ERR_INVALID_ARG = 1, /* null pointer, misalignment, negative size, bad enum value */
  PA_ERR_UNSUPPORTED = 2, /* head_dim, block_size or dtype combination not supported */
  PA_ERR_WORKSPACE = 3,   /* ws_bytes below pa_workspace_size() */
  PA_ERR_CUDA = 4,        /* a CUDA runtime call or a kernel launch failed */
  PA_ERR_DEVICE = 5       /* pa_read_flags: the device recorded an input problem */
} pa_status;

/* PA_INT4 is a cache's type only: see "4-bit caches" below. */
typedef enum { PA_BF16 = 0, PA_FP16 = 1, PA_FP8_E4M3 = 2, PA_INT4 = 3 } pa_dtype;

typedef enum {
  PA_SCALE_NONE = 0,       /* 16-bit cache, or fp8 codes used as they are */
  PA_SCALE_PER_TENSOR = 1, /* k_scale, v_scale: one fp32 each */
  PA_SCALE_PER_TOKEN = 2,  /* k_scale, v_scale: fp32 [num_blocks, block_size, num_kv_heads] */
  PA_SCALE_PER_BLOCK = 3,  /* k_scale, v_scale: fp32 [num_blocks, num_kv_heads] */
  PA_SCALE_AFFINE = 4      /* PA_INT4 caches, and only they: k_scale, v_scale hold pairs (step, low)
                              of q_dtype, [num_blocks, num_kv_heads, block_size, 2] */
} pa_scale_mode;

/* 4-bit caches (kv_dtype PA_INT4 with PA_SCALE_AFFINE).  k_cache and v_cache are bytes
 * [num_blocks, block_size, num_kv_heads, head_dim / 2]: channel 2 j of a row (one token and kv
 * head) in the low half of byte j, channel 2 j + 1 in the high half, each a code c in 0 .. 15.
 * A row's pair (step, low) stands in the scale array of its cache, and its values are
 *     low + step * c.
 * A page's pairs of one kv head lie together, as its rows of one kv head are read together.
 * (The pages cited above have no counterpart of this cache.) */

/* Where the log-sum-exp merge of split units runs.  A unit cut into ns pieces can be merged
 * by the last CTA to finish one of its pieces, inside pa_decode (an atomic arrival counter
 * per unit; no CTA ever waits for another), or by pa_reduce's own kernel, which spreads the
 * rows of the unit over many CTAs.  The first costs no launch but runs on one SM, so it
 * suits units of a few pieces; the second suits units cut into many.
 *   PA_MERGE_AUTO (0, the default): the library's choice, currently that of
 *     PA_MERGE_IN_REDUCE (measured fastest: a merge inside the decode runs after the merging
 *     CTA's own work and lengthens the decode's tail).
 *   PA_MERGE_IN_DECODE: pa_decode merges every unit and pa_reduce launches nothing.
 *   PA_MERGE_IN_REDUCE: pa_decode only writes partials and pa_reduce merges them all.
 * The choice changes the order of no sum inside a merge: outputs agree to rounding. */
typedef enum { PA_MERGE_AUTO = 0, PA_MERGE_IN_DECODE = 1, PA_MERGE_IN_REDUCE = 2 } pa_split_merge;

/* Device-side input problems, OR-ed into the flags word. */
enum {
  PA_FLAG_BAD_LENGTHS = 1,   /* q_lens[b] outside [0, max_q_len], context_lens[b] < q_lens[b],
                                or context_lens[b] > max_blocks_per_seq * block_size */
  PA_FLAG_BAD_BLOCK_ID = 2,  /* a block_tables entry in use lies outside [0, num_blocks) */
  PA_FLAG_WAIT_TIMEOUT = 4,  /* a kernel gave up a bounded wait on its own copies */
  PA_FLAG_STALE_PLAN = 8,    /* pa_decode read lengths other than those pa_plan planned for
                                (they changed between the two calls); outputs unspecified */
  PA_FLAG_BAD_SELECTION = 16, /* pa_decode_selected: a page count outside [0, top_k] or a listed
                                page outside the sequence */
  PA_FLAG_NO_FREE_BLOCKS = 32, /* pa_build_tables: fewer free pages than the lengths need */
  PA_FLAG_BAD_FREE_LIST = 64, /* pa_build_tables: a held or free page count that cannot be */
  PA_FLAG_BAD_POSITION = 128 /* pa_append_rotated: a position outside [0, table_rows) */
};

typedef struct {
  int32_t batch;              /* B >= 1 */
  int32_t max_q_len;          /* Sq >= 1: query rows per sequence in q and out */
  int32_t num_q_heads;        /* Hq */
  int32_t num_kv_heads;       /* Hkv, divides Hq */
  int32_t head_dim;           /* D: 64, 128 or 256 */
  int32_t block_size;         /* tokens per page: a power of two in [16, 1024] */
  int32_t max_blocks_per_seq; /* columns of block_tables */
  int32_t num_blocks;         /* physical pages in the pool */
  int32_t q_dtype;            /* pa_dtype of q and out: PA_BF16 or PA_FP16 */
  int32_t kv_dtype;           /* pa_dtype of the cache: q_dtype, PA_FP8_E4M3 or PA_INT4 */
  int32_t kv_scale_mode;      /* pa_scale_mode; PA_SCALE_NONE for a 16-bit cache, PA_SCALE_AFFINE
                                 for PA_INT4 */
  int32_t causal;             /* 1: new token i sees keys up to its own position */
  float sm_scale;             /* logit scale, usually 1/sqrt(D) */
  int32_t num_ctas;           /* persistent grid size; 0: (SMs of the current device x grid_mult)
                                 x the decode CTAs that fit on one SM */
  int32_t grid_mult;          /* grid multiplier when num_ctas is 0; 0 means 1 */
  int32_t split_merge;        /* pa_split_merge: where units cut into several pieces are merged */
} pa_config;

/* Bytes of workspace a pa_plan/pa_decode/pa_reduce sequence needs for cfg:
 * the work list for (C + units) items and fp32 partials for as many splits,
 * where C is the persistent grid size and units = B * Hkv * row blocks.
 * May query the current device (num_ctas == 0).  Writes *bytes. */
PA_API pa_status pa_workspace_size(const pa_config *cfg, size_t *bytes);

/* Plan one decode step (device work, no host sync).  Reads context_lens[B] and
 * q_lens[B]; checks the lengths; writes the work list into ws.  Cuts the
 * concatenated token ranges of all (sequence, kv-head, row-block) units into C
 * contiguous tile-aligned pieces of equal size, one per CTA, so every CTA of the
 * persistent grid reads the same number of pages.  block_tables is not read here
 * (pa_decode checks every block id it uses) but must not be NULL. */
PA_API pa_status pa_plan(const pa_config *cfg, const int32_t *block_tables, const int32_t *context_lens,
                  const int32_t *q_lens, void *ws, size_t ws_bytes, pa_stream stream);

/* Run the persistent decode over the work list pa_plan left in ws.
 *   q        [B, Sq, Hq, D]            q_dtype
 *   k_cache  [num_blocks, block_size, Hkv, D]   kv_dtype (uint8 codes for fp8; see "4-bit caches")
 *   v_cache  same layout as k_cache
 *   k_scale, v_scale  NULL unless there is a scale mode (see pa_scale_mode); 16-byte aligned pairs for
 *            a 4-bit cache
 *   out      [B, Sq, Hq, D]            q_dtype; written for every unit done in one piece,
 *            with no keys, or merged here (see pa_split_merge)
 *   lse      [B, Sq, Hq] fp32 natural-log LSE, or NULL
 * The tables and lengths must be the ones given to pa_plan, with the same contents.  A CTA
 * of the tcgen05 decode (33 or more query rows per kv head; head dim 128 or 256, 128 for an
 * fp8 cache), of the streaming decode (PA_SCALE_PER_BLOCK with head dim 64, or with up to 32
 * query rows per kv head) and of the 4-bit decode derives its first work item from the lengths
 * (the planner's rules) and starts on it while the planner is still running; it waits for the
 * planner before the rest of its list and before writing anything, and raises
 * PA_FLAG_STALE_PLAN if the planner's first item differs.  Where the planner runs no longer, and
 * the other decode kernels always, a CTA first waits for the launch before it.
 * The kernels launch with programmatic dependent launch.  A kernel of the caller's between pa_plan and
 * pa_decode that writes q, the caches, the scales, the tables or the lengths may do so too, if it lets its
 * dependents start no earlier than its own wait on the launch before it.
 * A decode that completed leaves the merge counters as pa_plan set them, so pa_decode may run again on
 * the same plan: a model may plan once a step, and append, decode and reduce for each of its layers.
 *
 * Rounding.  Logits, the softmax's maxima and sums, and the outputs' accumulators are fp32.  A
 * weight is rounded once, to the type of the second product's operands: bf16 for a bf16 cache,
 * f16 for fp16 and fp8 caches (whose codes are exact there).  With PA_SCALE_PER_TOKEN it is rounded
 * with its token's V scale in it as that is, so V scales below 2^-14 cost it bits.  With
 * PA_SCALE_PER_BLOCK it keeps its bits whatever the scales are, unless pages that one row reads
 * differ in theirs by more than 2^60 (2^30 with 33 query rows and more per kv head at head dim
 * 128).  For an fp8 cache a bf16 query goes into f16: with PA_SCALE_PER_BLOCK times a power of two
 * that makes it fit, else as it is (past 65504 it becomes infinite); with 33 rows and more per kv
 * head at head dim 128 any query goes into two or three E4M3 terms, scaled to fit, where elements
 * below about a thousandth of the row's largest lose bits.  64-dim fp8 caches without page scales
 * run in fp32 throughout.  For a 4-bit cache the codes enter both products as the integers c - 8,
 * a bf16 query in f16 times a power of two that makes it fit (elements below 2^-22 of its row's
 * largest lose bits), a weight times its row's V step in f16
 * (11 bits kept as with PA_SCALE_PER_BLOCK), and what low + 8 step adds to logits and outputs is
 * fp32; an fp16 output is so off by up to a third more than its own rounding, a bf16 output is not.
 *
 * Keys that a row does not see may hold anything; the values (V) of a key that some of a
 * sequence's rows see and others do not have to be finite, as a weight of zero meets them in the
 * same product.  (Not so for a 4-bit cache, whose codes are finite: a pair that is not reaches the rows
 * that see its token, and no other.  A NaN logit is NaN in its row's out and lse, split or not.) */
PA_API pa_status pa_decode(const pa_config *cfg, const void *q, const void *k_cache, const void *v_cache,
                    const void *k_scale, const void *v_scale, const int32_t *block_tables,
                    const int32_t *context_lens, const int32_t *q_lens, void *out, float *lse,
                    void *ws, size_t ws_bytes, pa_stream stream);

/* Completes the step: merges the split partials pa_decode left in ws into out (and lse) for
 * every unit pa_decode did not merge itself (see pa_split_merge).  With PA_MERGE_IN_DECODE
 * there is none, and this call only validates its arguments and launches nothing. */
PA_API pa_status pa_reduce(const pa_config *cfg, void *out, float *lse, void *ws, size_t ws_bytes,
                    pa_stream stream);

/* Synchronise `stream` and return the device flags of the last plan/decode in ws
 * (PA_FLAG_* bits; 0 when the step was clean) in *flags.  Returns PA_ERR_DEVICE
 * when any flag is set, PA_OK otherwise. */
PA_API pa_status pa_read_flags(const void *ws, size_t ws_bytes, int32_t *flags, pa_stream stream);

/* Size of the device scratch array behind pa_decode_step_static (16 MiB). */
#define PA_STATIC_SCRATCH_BYTES ((size_t)16 << 20)

/* One whole decode step (plan, decode, reduce) that allocates nothing and needs no
 * workspace from the caller.  The pages have no counterpart: it exists for callers that
 * cannot allocate device memory -- code running under a framework or plugin interface that
 * hands out no allocator, loops that must not call cudaMalloc once serving has started
 * (cudaMalloc can synchronise the device and is not allowed during stream capture), and
 * deployments that forbid allocation after start-up.  Arguments are those of pa_decode
 * without ws/ws_bytes; the caller still provides q, the caches, scales, tables, lengths,
 * out and lse.
 *
 * The scratch is one file-scope __device__ array of PA_STATIC_SCRATCH_BYTES, reserved on
 * every GPU where the library's device code is loaded and held until the process exits.
 * The first call on a device looks up the array's device address (cudaGetSymbolAddress)
 * with that device current and caches it; make that first call before any stream capture.
 * The cached address belongs to the device's primary context: after cudaDeviceReset (or any
 * other teardown of that context) it names freed memory, so a process that resets a device
 * must not call this entry point on that device again.
 * A problem whose pa_workspace_size() exceeds PA_STATIC_SCRATCH_BYTES is rejected with
 * PA_ERR_WORKSPACE before anything is launched.  All calls on a device share the one array
 * and each call overwrites what the previous one left there: calls whose kernels overlap on
 * the GPU (different streams, or different host threads without ordering) race and corrupt
 * each other's results.  Calls on one stream are ordered and safe.  pa_read_flags is not
 * available for this scratch (its address is private); device-side input problems leave
 * out unspecified. */
PA_API pa_status pa_decode_step_static(const pa_config *cfg, const void *q, const void *k_cache,
                                       const void *v_cache, const void *k_scale,
                                       const void *v_scale, const int32_t *block_tables,
                                       const int32_t *context_lens, const int32_t *q_lens,
                                       void *out, float *lse, pa_stream stream);

/* Paged -> contiguous copy of a batch's cached K and V (the copy the HSTU paged attention
 * makes from its paged cache into its workspace before attending: "HSTU Paged Attention"
 * K/V double-buffering issue, background and optimisation plan).
 *
 * Sequence b's tokens 0 .. context_lens[b] - 1 are copied, in token order, to rows
 * row_off[b] .. row_off[b] + context_lens[b] - 1 of k_out and of v_out, where
 * row_off[b] = context_lens[0] + ... + context_lens[b - 1]; a row is one token's
 * [num_kv_heads, head_dim] values exactly as the cache stores them (bf16, fp16 or E4M3
 * codes; the scales of tokens or pages are not copied; pa_dequant_kv reads codes back as values,
 * those of 4-bit caches among them, which this call does not take).  Reads cfg's batch, num_kv_heads, head_dim,
 * block_size, max_blocks_per_seq, num_blocks and kv_dtype; the other fields are ignored.
 *
 *   k_cache, v_cache  device, [num_blocks, block_size, num_kv_heads, head_dim], 16-byte aligned
 *   block_tables      device int32 [batch, max_blocks_per_seq]
 *   context_lens      device int32 [batch]
 *   k_out, v_out      device, room for max_rows rows of num_kv_heads * head_dim elements,
 *                     16-byte aligned
 *   row_offsets       NULL, or device int32 [batch + 1] that receives row_off[0 .. batch]
 *                     (row_off[batch] = rows copied)
 *   flags             NULL, or a device int32 the call ORs PA_FLAG_* bits into:
 *                     PA_FLAG_BAD_LENGTHS when a length is negative or exceeds
 *                     max_blocks_per_seq * block_size (that sequence counts as empty) or the
 *                     rows exceed max_rows (nothing is copied), PA_FLAG_BAD_BLOCK_ID for a
 *                     page whose block id lies outside [0, num_blocks) (its rows are not
 *                     written)
 *
 * Stream-ordered, allocates nothing.  PA_ERR_UNSUPPORTED for batch > 8192, head_dim or
 * block_size outside the decode's sets, or problems whose row or copy counts exceed int32. */
PA_API pa_status pa_gather_kv(const pa_config *cfg, const void *k_cache, const void *v_cache,
                              const int32_t *block_tables, const int32_t *context_lens,
                              void *k_out, void *v_out, int64_t max_rows, int32_t *row_offsets,
                              int32_t *flags, pa_stream stream);

/* Quantise-on-write KV append: write a decode step's new K/V rows into their pages.
 *
 * New row i < q_lens[b] of sequence b is cache position pos = context_lens[b] - q_lens[b] + i
 * (the new tokens are the last q_lens[b] of the context_lens[b] tokens, the positions the
 * decode's causal mask gives them), i.e. slot pos % block_size of physical block
 * block_tables[b][pos / block_size] ("HSTU Paged Attention", RecSDK issue 1281, background:
 * the paged KV cache).  Call it with the tables and lengths of the pa_decode that is to read the rows,
 * before that call (and before or behind its pa_plan).
 *   16-bit cache (kv_dtype == q_dtype): the row's bits are copied unchanged.
 *   fp8 cache: OCP E4M3 codes of row / scale, rounded to nearest (ties to even), magnitudes
 *   past 448 saturating to 448; scale modes of "Optimize paged-attention metadata decode"
 *   (FlyDSL PR #910, Breaking Changes: per_token_kv):
 *     PA_SCALE_PER_TOKEN   scale = amax(|row|) / 448 (1 for an all-zero row), computed in fp32
 *                          and WRITTEN to k_scale / v_scale [num_blocks, block_size, Hkv];
 *     PA_SCALE_PER_TENSOR  scale = k_scale[0] / v_scale[0], READ (one fp32 each);
 *     PA_SCALE_NONE        scale 1; k_scale / v_scale may be NULL.
 *     PA_SCALE_PER_BLOCK   one scale for each (block, kv head) in k_scale / v_scale
 *                          [num_blocks, Hkv], READ and WRITTEN.  With w = the largest finite
 *                          magnitude among the call's new rows in the page / 448 (at least
 *                          2^-126; 0 if they are all zero): a page whose slot 0 is among the
 *                          new rows gets scale w (1 for w = 0); any other page keeps its scale
 *                          unless w is larger.  Then the page's scale becomes w and the codes c
 *                          of its older tokens become E4M3(c * old scale / w), the product and
 *                          the quotient each rounded to fp32.  A scale never falls while its
 *                          page is in use, so a page that begins with zeros holds what follows
 *                          no finer than E4M3 at scale 1 does (2^-9).  The older scale has to be
 *                          one that an earlier append wrote (positive and finite).  No two
 *                          sequences may append to one page in one call.
 *   Quotients are IEEE fp32 divisions.  A NaN element gives a NaN code (0x7f or 0xff).
 *   4-bit cache (PA_INT4): each row x gets, and its pair in k_scale / v_scale becomes,
 *     low  = the largest number of q_dtype that is <= min(x),
 *     step = the least number of q_dtype that is >= (max(x) - low) / 15 (fp32 difference and
 *            quotient, each rounded to nearest),
 *     c    = (x - low) / step (fp32 difference and IEEE quotient) rounded to the nearest integer,
 *            ties to even; 0 when step is 0.
 *   So low is the least element itself and a value is read back within step / 2, which is a
 *   thirtieth of the row's range (and half a step of q_dtype in that).  (The keys that
 *   pa_append_rotated quantises are fp32: there low may lie below the least element.)  A row that
 *   holds a NaN or an infinity, whose range passes fp32, or whose low or step passes q_dtype's
 *   largest number (fp16 keys that a rotation or a norm's weights take past 65504), gets step NaN
 *   and codes 0: all of it reads back NaN.
 * Reads cfg's batch, max_q_len, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
 * num_blocks, q_dtype, kv_dtype and kv_scale_mode.
 *
 *   k_new, v_new   device, [batch, max_q_len, num_kv_heads, head_dim] in q_dtype, 16-byte
 *                  aligned; rows i >= q_lens[b] are ignored
 *   block_tables, context_lens, q_lens   device int32, as for pa_plan
 *   k_cache, v_cache   device, [num_blocks, block_size, num_kv_heads, head_dim] in kv_dtype,
 *                  16-byte aligned; the new rows' slots are written, and with
 *                  PA_SCALE_PER_BLOCK also the older slots of a page whose scale grows
 *   k_scale, v_scale   device fp32 (see the scale modes), or pairs of q_dtype for a 4-bit cache
 *   flags          NULL, or a device int32 the call ORs PA_FLAG_* bits into:
 *                  PA_FLAG_BAD_LENGTHS for a sequence whose lengths break the rules of
 *                  pa_plan (none of its rows is written), PA_FLAG_BAD_BLOCK_ID for a new row
 *                  whose page lies outside [0, num_blocks) (that row is not written)
 *
 * Stream-ordered, allocates nothing, never synchronises.  PA_ERR_INVALID_ARG for NULL or
 * misaligned pointers (scales NULL with a scale mode), PA_ERR_UNSUPPORTED for head_dim,
 * block_size or dtype combinations the decode does not take. */
PA_API pa_status pa_append_kv(const pa_config *cfg, const void *k_new, const void *v_new,
                              const int32_t *block_tables, const int32_t *context_lens,
                              const int32_t *q_lens, void *k_cache, void *v_cache,
                              void *k_scale, void *v_scale, int32_t *flags, pa_stream stream);

/* How pa_append_rotated makes a projection's rows ready for attention. */
typedef struct {
  const void *q_weight;     /* q_dtype [head_dim], or NULL: queries are not normalised */
  const void *k_weight;     /* the same for keys */
  float eps;                /* added to the mean square; finite and >= 0 */
  int32_t rotary_dim;       /* channels that rotate, the first ones of a head: a multiple of 16, at
                               most head_dim; 0: none (cos_sin and positions are not read) */
  int32_t interleaved;      /* pair p is channels 2 p, 2 p + 1 (1) or p, p + rotary_dim / 2 (0) */
  const float *cos_sin;     /* fp32 [table_rows, rotary_dim], 16-byte aligned: the cosines of a
                               position's rotary_dim / 2 angles, then their sines */
  int32_t table_rows;
  const int32_t *positions; /* int32 [num_axes, batch, max_q_len], or NULL: every axis is at the
                               row's cache position */
  int32_t num_axes;         /* 1 to 3 */
  int32_t axis_pairs[3];    /* the first axis_pairs[0] pairs take their angle from the first axis's
                               position, the next axis_pairs[1] from the second's, ...; they add up
                               to rotary_dim / 2 */
  int64_t q_stride, k_stride, v_stride; /* elements from one token's rows of q, k_new and v_new to
                               the next token's, multiples of 8; 0: the rows lie dense */
} pa_rotary;

/* Normalise and rotate a step's queries and keys and write its K/V rows into their pages, in one
 * pass.  (The pages cited above have no counterpart.)
 *
 * For each new row i < q_lens[b] of each q and k head x (fp32 throughout, one rounding at the end):
 *     y_c = x_c / sqrt(mean(x^2) + eps) * weight_c          (with a weight; else y = x)
 *     (z_a, z_b) = (y_a cos - y_b sin, y_b cos + y_a sin)   for each pair (a, b), with the angle of
 *                                                           its axis's position
 * z of a query goes to q_out, z of a key to k_out (both rounded to q_dtype) and, quantised from fp32
 * as pa_append_kv quantises, into its page; values go into their pages as they are.  Keys, values,
 * scales, tables, lengths and the order of calls are those of pa_append_kv, for every cache but one with
 * PA_SCALE_PER_BLOCK (PA_ERR_UNSUPPORTED: a page's scale needs all its new rows; take k_out and give
 * it to pa_append_kv).
 *
 *   q [batch, max_q_len, num_q_heads, head_dim], k_new, v_new [batch, max_q_len, num_kv_heads,
 *                  head_dim] in q_dtype, 16-byte aligned; tokens may lie apart (the strides: slices
 *                  of one projection's output)
 *   q_out          dense, as q; may be q itself if that is dense.  Rows i >= q_lens[b] are left as
 *                  they were
 *   k_out          NULL, or dense, as k_new: the rotated keys (what pa_update_bounds wants); may be
 *                  k_new itself if that is dense
 *   k_cache, v_cache   both, or both NULL with k_out given: nothing goes into pages (v_new, scales
 *                  and block_tables are not read then and may be NULL)
 *   flags          NULL, or a device int32: PA_FLAG_BAD_LENGTHS (nothing of that sequence is
 *                  written), PA_FLAG_BAD_POSITION (nothing of that token is written),
 *                  PA_FLAG_BAD_BLOCK_ID (that token's K and V do not go into a page)
 * No other two arrays may overlap, where one of them is written.  Reads cfg's batch, max_q_len,
 * num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks, q_dtype, kv_dtype
 * and kv_scale_mode.  Stream-ordered, allocates nothing, never synchronises. */
PA_API pa_status pa_append_rotated(const pa_config *cfg, const pa_rotary *rotary, const void *q,
                                   const void *k_new, const void *v_new,
                                   const int32_t *block_tables, const int32_t *context_lens,
                                   const int32_t *q_lens, void *q_out, void *k_out, void *k_cache,
                                   void *v_cache, void *k_scale, void *v_scale, int32_t *flags,
                                   pa_stream stream);

/* Read a quantised cache back: the rows that pa_gather_kv copies, as values of q_dtype.
 *
 * Row row_off[b] + t of k_out (and v_out) holds the values of sequence b's token t: the code times
 * its scale (fp8), or low + step * code (4-bit), in fp32 and rounded to q_dtype once.  Arguments,
 * checks and flags are those of pa_gather_kv, with k_scale and v_scale as for pa_decode and q_dtype
 * the type of k_out and v_out.  PA_ERR_UNSUPPORTED for a 16-bit cache (pa_gather_kv copies it). */
PA_API pa_status pa_dequant_kv(const pa_config *cfg, const void *k_cache, const void *v_cache,
                               const void *k_scale, const void *v_scale,
                               const int32_t *block_tables, const int32_t *context_lens,
                               void *k_out, void *v_out, int64_t max_rows, int32_t *row_offsets,
                               int32_t *flags, pa_stream stream);

/* Grow and shrink block tables from the requests' lengths, on the GPU.  (The pages cited above
 * have no counterpart.)
 *
 * Row b of block_tables holds held_blocks[b] pages; sequence b needs ceil(context_lens[b] /
 * block_size).  A row that holds too many gives its last pages to the free list, one that holds
 * too few takes pages from it, and a finished request is a row with context_lens[b] =
 * q_lens[b] = 0.  The free list is a stack: free_blocks[0 .. free_count[0]).  The pages given
 * are pushed first (ascending b, then ascending page), then the pages taken are popped one by
 * one (ascending b, then ascending page), so the result does not depend on timing.
 * slot_map[b][i], for new token i < q_lens[b] at position p = context_lens[b] - q_lens[b] + i,
 * is block_tables[b][p / block_size] * block_size + p % block_size in the tables after the
 * call, and -1 for i >= q_lens[b].
 * Reads cfg's batch, max_q_len, block_size, max_blocks_per_seq and num_blocks.
 *
 *   context_lens, q_lens, held_blocks   device int32 [batch], read
 *   block_tables    device int32 [batch, max_blocks_per_seq]: the taken pages' entries are
 *                   written, all others (those of given pages too) are left as they were
 *   free_blocks     device int32 [num_blocks]: entries at and above free_count[0] may be written
 *   free_count      device int32, read
 *   new_held, new_free_count   device int32 [batch] and int32, written; the next call's
 *                   held_blocks and free_count.  They may not be the arrays of this call, so
 *                   that the call reads only what it does not write: with the same inputs it
 *                   can be run again and gives the same result
 *   slot_map        NULL, or device int64 [batch, max_q_len], written, 16-byte aligned
 *   flags           NULL, or a device int32 the call ORs PA_FLAG_* bits into.  PA_FLAG_BAD_LENGTHS
 *                   (lengths that break the rules of pa_plan), PA_FLAG_BAD_FREE_LIST (a held
 *                   count outside [0, max_blocks_per_seq], a free count outside [0, num_blocks],
 *                   or more free pages than num_blocks after the pushes) and
 *                   PA_FLAG_NO_FREE_BLOCKS: nothing is given or taken, new_held and
 *                   new_free_count are copies and every slot is -1.  PA_FLAG_BAD_BLOCK_ID: a page
 *                   given or taken (it moves all the same) or, with a slot_map, a page of a new
 *                   token lies outside [0, num_blocks); its tokens' slots are -1.  Pages that stay
 *                   where they are and hold no new token are not looked at
 *
 * Stream-ordered, allocates nothing, never synchronises.  No two arrays may overlap.
 * PA_ERR_UNSUPPORTED for batch > 4096, a block_size outside the decode's set, or tables or slot
 * maps of 2^31 entries or more. */
PA_API pa_status pa_build_tables(const pa_config *cfg, const int32_t *context_lens,
                                 const int32_t *q_lens, const int32_t *held_blocks,
                                 int32_t *block_tables, int32_t *free_blocks,
                                 const int32_t *free_count, int32_t *new_held,
                                 int32_t *new_free_count, int64_t *slot_map, int32_t *flags,
                                 pa_stream stream);

/* Channel bounds of a page's keys, kept as keys are appended.  (The pages cited above have no
 * counterpart of this call and the three below.)
 *
 * k_bounds [num_blocks, num_kv_heads, 2, head_dim] in q_dtype holds, for each page and kv head,
 * the least ([.., 0, :]) and the largest ([.., 1, :]) value of each channel over the page's keys
 * as they were given (before any quantisation).  A page whose slot 0 is among the new rows
 * starts afresh; any other page's bounds are widened by the new rows.  NaN stays NaN.
 * Arguments and flags are those of pa_append_kv, which may run before or after it.  Reads cfg's
 * batch, max_q_len, num_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks and
 * q_dtype. */
PA_API pa_status pa_update_bounds(const pa_config *cfg, const void *k_new,
                                  const int32_t *block_tables, const int32_t *context_lens,
                                  const int32_t *q_lens, void *k_bounds, int32_t *flags,
                                  pa_stream stream);

/* Scores of a sequence's pages for each new-token row and kv head.
 *
 * With L the keys that row i sees (as for the decode), page p < ceil(L / block_size) of row i
 * and kv head g scores
 *     max over the group's heads h of  sm_scale * sum_d (max(q_d, 0) hi_d + min(q_d, 0) lo_d)
 * with lo and hi the page's bounds.  For sm_scale >= 0 no key that went into the bounds has a
 * larger logit, but for rounding: the products are exact and their sums fp32, off by less than
 * (2 D + 1) 2^-23 of the sum of their magnitudes.  An fp8 cache does not hold those keys but their
 * codes, each value off by up to 2^-4 of itself (or half a step of E4M3's subnormals, 2^-10 of
 * the scale), and by as much again each time that its page's scale grows: such a key may score
 * above its page by what that comes to.
 * Other pages, and the rows i >= q_lens[b], score -inf.  Bounds or queries that are not finite
 * give scores that are not (NaN included).
 *   q        [B, Sq, Hq, D] q_dtype, 16-byte aligned
 *   k_bounds [num_blocks, num_kv_heads, 2, head_dim] q_dtype, 16-byte aligned
 *   scores   fp32 [B, Sq, Hkv, max_blocks_per_seq], written whole
 *   flags    NULL, or a device int32: PA_FLAG_BAD_LENGTHS (that sequence scores -inf),
 *            PA_FLAG_BAD_BLOCK_ID (that page scores -inf)
 * Reads cfg's sizes, q_dtype, causal and sm_scale.  PA_ERR_UNSUPPORTED for what the decode does
 * not take. */
PA_API pa_status pa_score_blocks(const pa_config *cfg, const void *q, const void *k_bounds,
                                 const int32_t *block_tables, const int32_t *context_lens,
                                 const int32_t *q_lens, float *scores, int32_t *flags,
                                 pa_stream stream);

/* The best pages of each row, in ascending order.
 *
 * Row (b, i, g) sees N = ceil(L / block_size) pages and gets min(top_k, N) of them: first the
 * pages below num_first and the last num_last of the N (num_first + num_last <= top_k), then
 * those with the highest scores; NaN ranks above every number, +0 and -0 are equal, and of
 * equal scores the lower page wins.
 *   scores        fp32 [B, Sq, Hkv, max_blocks_per_seq]; pages at and past N are not read
 *   selected      int32 [B, Sq, Hkv, top_k], written whole: the pages, ascending, then -1
 *   num_selected  int32 [B, Sq, Hkv]: min(top_k, N); 0 for rows i >= q_lens[b]
 *   flags         NULL, or a device int32: PA_FLAG_BAD_LENGTHS (that sequence selects nothing)
 * Reads cfg's batch, max_q_len, num_kv_heads, block_size, max_blocks_per_seq and causal. */
PA_API pa_status pa_select_blocks(const pa_config *cfg, const float *scores,
                                  const int32_t *context_lens, const int32_t *q_lens,
                                  int32_t top_k, int32_t num_first, int32_t num_last,
                                  int32_t *selected, int32_t *num_selected, int32_t *flags,
                                  pa_stream stream);

/* Attention of each row over its listed pages only.
 *
 * Row i of sequence b and the heads of kv head g attend over the keys of the logical pages
 * selected[b][i][g][0 .. num_selected[b][i][g]) that lie below L (the keys the row sees, as for
 * the decode): out and lse as for pa_decode with the softmax over those keys alone; a row with
 * none gets out = 0, lse = -inf.  The list may be in any order; a page listed twice counts
 * twice.  Any cache, scale mode and head grouping that pa_decode takes but a 4-bit cache
 * (PA_ERR_UNSUPPORTED).
 *   selected      int32 [B, Sq, Hkv, top_k] logical pages (columns of block_tables)
 *   num_selected  int32 [B, Sq, Hkv]
 *   lse           [B, Sq, Hq] fp32 or NULL
 *   flags         NULL, or a device int32: PA_FLAG_BAD_LENGTHS (that sequence's rows get out = 0,
 *                 lse = -inf), PA_FLAG_BAD_SELECTION (a count outside [0, top_k] is clamped, a
 *                 page outside the sequence's is skipped), PA_FLAG_BAD_BLOCK_ID (a listed page
 *                 whose block lies outside [0, num_blocks) is skipped)
 * One launch, no workspace; the split of a row's pages depends on the sizes alone, so equal
 * inputs give equal bits.  num_ctas, grid_mult and split_merge of cfg are not used.  Weights and
 * queries are rounded as pa_decode does with PA_SCALE_PER_BLOCK and up to 32 rows per kv head,
 * whatever the scale mode.  Keys and values that a row does not see may hold anything.
 * PA_ERR_UNSUPPORTED for what the decode does not take, and for lists of 2^31 tokens or more
 * (top_k * block_size). */
PA_API pa_status pa_decode_selected(const pa_config *cfg, const void *q, const void *k_cache,
                                    const void *v_cache, const float *k_scale,
                                    const float *v_scale, const int32_t *block_tables,
                                    const int32_t *context_lens, const int32_t *q_lens,
                                    const int32_t *selected, const int32_t *num_selected,
                                    int32_t top_k, void *out, float *lse, int32_t *flags,
                                    pa_stream stream);

/* A static, human-readable name of a status. */
PA_API const char *pa_status_string(pa_status status);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */

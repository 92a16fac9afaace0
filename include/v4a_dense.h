/*
 * v4a_dense.h - dense attention layers beside the compressed ones of v4a.h:
 * layers that keep every token's key and value, per KV head, in a paged
 * cache of the same 256-position logical blocks.
 *
 *   v4a_step_plan     request lengths -> positions, slot maps and block
 *                     tables, built on the GPU (pages from a device free ring)
 *   v4a_dense_insert  per-head RMSNorm of queries and keys, the position
 *                     rotation, and the keys' and values' cache insert, in one
 *                     pass
 *   v4a_dense_attn    attention of the step's tokens over the paged cache:
 *                     single-token decode (split over the cache's length and
 *                     joined) and chunked prefill, grouped query heads, an
 *                     optional sliding window with sinks
 *
 * A step calls them in this order; the layers of one model share the plan.
 * Beside them:
 *
 *   v4a_dense_insert_rows  the insert, which also gives the keys as packed rows;
 *                          the one for caches with a scale per group
 *   v4a_dense_read         cached keys and values as packed rows
 *   v4a_prompt_attn        attention of whole prompts over packed keys and values
 *                          (those that v4a_dense_insert_rows leaves, behind
 *                          prefixes that v4a_dense_read gives), no cache
 *
 * The general rules of v4a.h hold: device pointers, caller-owned buffers and
 * workspaces, no allocation, no synchronisation, the given stream only; a
 * nonzero return code launched nothing (except V4A_ERR_CUDA); problems only
 * the device can see set V4A_DEV_* bits in *status and skip the access.
 * Each call can be captured into a CUDA graph (a shape's first call on a
 * device may load its kernels: make it before the capture); two calls that may run at the
 * same time need workspaces of their own.  A sequence's compressed layers and
 * dense layers can use one page allocator (v4a_pages.h): a dense cache is a
 * V4A_PAGES_BLOCK kind of v4a_dense_block_bytes bytes.
 */
#ifndef V4A_DENSE_H
#define V4A_DENSE_H

#include <stddef.h>
#include <stdint.h>

#include "v4a.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- a format of dense caches alone (the others are in v4a.h) ----------------- */
#define V4A_KV_FP8_GROUP 3 /* e4m3 codes; one fp32 scale, a power of two, per KV head and group of 64
                              positions (a quarter of a block) of the keys and of the values */

/* ---- device status bit (the others are in v4a.h) ------------------------------ */
#define V4A_DEV_OUT_OF_PAGES 16 /* v4a_step_plan: the free ring holds too few pages */

/*
 * The step plan.  Sequence b (a row of every block table) holds `cached[b]`
 * positions and brings `fresh[b]` new tokens: 0 rests, -1 ends the sequence.
 * The step's tokens are packed in sequence order:
 *   token_starts[b] = sum of the new tokens of the sequences before b,
 *   token t of sequence b: seq_ids[t] = b,
 *                          positions[t] = cached[b] + t - token_starts[b],
 *                          slots[l][t] = page * 256 + positions[t] % 256 with
 *                          page = table l's entry for positions[t] / 256.
 * Tokens behind the last one (a step padded to max_tokens for a captured
 * graph) get -1 in all three.
 *
 * A sequence holds ceil(cached / 256) blocks; a fresh token in a block it does
 * not hold takes a new page in each of the num_tables tables (for instance one
 * table per layer, all in one page pool).  Free pages are a ring of page ids,
 * first in first out: free_in = {index of the first free page, number of free
 * pages}.  With n blocks taken before block k of sequence b, its page in table
 * l is free_ring[(first + n * num_tables + l) % ring_cap].  The pages of an
 * ended sequence go behind the last free page in the same order and can be
 * taken from the next call on; its table rows are left as they were (stale:
 * a new sequence in that row starts at cached = 0).  free_out receives the
 * ring's new state; it may be the same array as free_in.
 *
 * The call does all or nothing: if a length is out of range (cached < 0,
 * fresh < -1, more than max_blocks blocks), the tokens exceed max_tokens or
 * the given-back pages exceed the ring (V4A_DEV_BAD_BATCH), or the ring holds
 * too few pages (V4A_DEV_OUT_OF_PAGES), then every token is -1, token_starts
 * is 0 throughout, free_out = free_in and no table or ring entry changes, so
 * the step's other calls do nothing.  A page id outside [0, num_blocks) sets
 * V4A_DEV_BAD_BLOCK and gives the slot -1; it goes into the table, and back
 * behind the free pages when its sequence ends, as it is.
 *
 * The plan gives back whole sequences: all blocks that `cached` counts.  It
 * takes no part in giving back blocks behind a window, and a row with holes
 * must not be ended with fresh = -1 (its -1 entries would be counted as free
 * pages; V4A_DEV_BAD_BLOCK is set).  A caller that gives such blocks back does
 * so between two calls, behind the last free page: free_ring[(first + count) %
 * ring_cap] and so on, count grown by as many, the table's entries set to -1.
 * It ends the sequence in the same way, with the pages that are left; the row
 * then starts anew at cached = 0.
 */
typedef struct {
  int32_t num_seqs;            /* B: 0..8192 */
  int32_t num_tables;          /* L: 1..4096 */
  int32_t max_tokens;          /* T: entries of the per-token outputs, >= 0 */
  int32_t max_blocks;          /* columns of a table row, 1..2^22 */
  const int32_t* cached;       /* [B] */
  const int32_t* fresh;        /* [B] */
  int32_t* block_table;        /* table l, row b, block k at [l * table_stride + b * max_blocks + k] */
  int64_t table_stride;        /* >= B * max_blocks */
  int64_t num_blocks;          /* pages of the pool */
  int32_t* free_ring;          /* [ring_cap] page ids */
  int32_t ring_cap;            /* >= the pages that can ever be free, 1..2^30 */
  const int32_t* free_in;      /* [2] first, count */
  int32_t* free_out;           /* [2] */
  int32_t* seq_ids;            /* [T] */
  int32_t* positions;          /* [T] */
  int64_t* slots;              /* [L][T] or NULL */
  int32_t* token_starts;       /* [B + 1] */
  int32_t* status;             /* optional device word */
} v4a_plan_args;

/* Bytes of device workspace v4a_step_plan needs (0 on bad arguments); it is
 * 16-byte aligned and its contents need no initialisation. */
V4A_API size_t v4a_plan_workspace_size(const v4a_plan_args* args);
V4A_API int v4a_step_plan(const v4a_plan_args* args, void* workspace, size_t workspace_bytes, void* stream);

/*
 * A dense paged cache.  Block `block_table[b][n]` holds sequence b's positions
 * [256 n, 256 n + 256): first the keys [num_kv_heads][256][dim], then the
 * values in the same layout, then for V4A_KV_FP8_TOKEN the fp32 scales of the
 * key rows [num_kv_heads][256] and of the value rows.  Formats: V4A_KV_BF16
 * and V4A_KV_FP8_TOKEN (e4m3 codes, one scale amax/448 per row: 1 for a row of
 * zeros, at least 2^-126, and elements below 2^-126 may count as zeros), and
 * V4A_KV_FP8_GROUP, whose codes are followed by the fp32 scales of the keys'
 * groups [num_kv_heads][4] and of the values'.
 */
typedef struct {
  int32_t num_kv_heads;        /* >= 1, <= 1024 */
  int32_t dim;                 /* 64, 128, 192 or 256 */
  int32_t format;              /* V4A_KV_BF16, V4A_KV_FP8_TOKEN or V4A_KV_FP8_GROUP */
  void* pool;                  /* block n starts at n * block_bytes; 16-byte aligned */
  int64_t num_blocks;
  int64_t block_bytes;         /* stride of blocks: a multiple of 16, at least v4a_dense_block_bytes;
                                  0 = v4a_dense_block_bytes */
  const int32_t* block_table;  /* [num_seqs][max_blocks]; -1 = unallocated */
  int32_t max_blocks;          /* 1..2^22 */
} v4a_dense_cache;

/* Bytes of one block (0 on a bad shape). */
V4A_API int64_t v4a_dense_block_bytes(int32_t num_kv_heads, int32_t dim, int32_t format);

/* ---- the position rotation ----------------------------------------------------- */
#define V4A_ROPE_INTERLEAVED 0  /* pairs (first + 2j, first + 2j + 1) */
#define V4A_ROPE_HALF        1  /* pairs (first + j, first + dims/2 + j) */

#define V4A_ROPE_PLAIN  0  /* f_j = theta^(-2j/dims) */
#define V4A_ROPE_LINEAR 1  /* f_j / factor (positions interpolated) */
#define V4A_ROPE_YARN   2  /* with r_j = original f_j / (2 pi) turns over the original context and
                              g_j = clamp((r_j - beta_slow) / (beta_fast - beta_slow), 0, 1):
                              f_j (g_j + (1 - g_j) / factor)  (YaRN, Peng et al. 2023).  The ramp g is
                              linear in the turns, as in the paper; a model whose ramp is linear in the
                              pair index j, between the (rounded) indices whose r is beta_fast and
                              beta_slow, has other frequencies there and takes V4A_ROPE_TABLE */
#define V4A_ROPE_TABLE  3  /* f_j = inv_freq[j], for any other rule */

/*
 * Dims [first, first + dims) of a head are rotated in pairs: [a, b] at
 * position p becomes magnitude * [a cos - b sin, a sin + b cos] with the angle
 * p f_j; the other dims pass through.  Angles are formed in 64-bit turns, so
 * positions up to 2^31 - 1 keep fp32 accuracy.
 */
typedef struct {
  int32_t dims;                /* a multiple of 16, 0..256; 0 = no rotation */
  int32_t first;               /* a multiple of 8; first + dims <= head dim */
  int32_t layout;              /* V4A_ROPE_INTERLEAVED or V4A_ROPE_HALF */
  int32_t scaling;             /* V4A_ROPE_PLAIN .. V4A_ROPE_TABLE */
  double theta;                /* > 0 */
  double factor;               /* LINEAR, YARN: > 0 */
  double original;             /* YARN: original context length, > 0 */
  double beta_fast, beta_slow; /* YARN: beta_fast > beta_slow */
  double magnitude;            /* factor on cos and sin, finite in fp32 (1 for none; YaRN uses 0.1 ln(factor) + 1) */
  const double* inv_freq;      /* TABLE: HOST array [dims / 2], read during the call, each in [0, pi] */
} v4a_rope;

/*
 * Norm + rotation + insert.  For token t with slots[t] >= 0, at P = positions[t]:
 *   q_out[t][h] = rope_P(norm(q[t][h]; q_gamma)),   h < num_heads
 *   key         = rope_P(norm(k[t][h]; k_gamma)),   h < num_kv_heads
 *   value       = v[t][h]
 * norm(x; g) = x / sqrt(max(mean(x^2) + eps, 2^-126)) * g over the head's dims
 * (x itself when the gamma pointer is NULL), in fp32, where squares below
 * 2^-126 count as zeros, and rounded once.  Key and value are encoded into
 * slot slots[t] (block slots[t] / 256, row slots[t] % 256) of every KV head.  A token with slot -1 is skipped and its q_out row is left as
 * it was; a slot below -1 or past the pool sets V4A_DEV_BAD_BLOCK, a negative
 * position with a valid slot V4A_DEV_BAD_BATCH, and the token is skipped.  The
 * rows of a slot that two tokens of a call share hold pieces of either (an fp8
 * row perhaps one's codes with the other's scale): nothing is to be read there.
 * q, k and v are rows of bf16 with a stride between tokens (three views of one
 * projection's output, for instance); heads are contiguous.  All row pointers
 * must be 16-byte aligned, the token strides multiples of 8 elements, the
 * gammas 16-byte aligned.  q_out may be q (in place, with equal strides) and
 * must overlap nothing else.  num_heads may be 0 (keys and values only).
 */
typedef struct {
  int32_t num_tokens;          /* T >= 0 */
  const int32_t* positions;    /* [T] */
  const int64_t* slots;        /* [T], as v4a_step_plan writes them */
  int32_t num_heads;           /* H, a multiple of kv.num_kv_heads, <= 1024 */
  const uint16_t* q;           /* [T] rows of [H][dim] */
  int64_t q_stride;            /* elements between tokens, >= H * dim */
  uint16_t* q_out;
  int64_t q_out_stride;
  const uint16_t* k;           /* [T] rows of [num_kv_heads][dim] */
  int64_t k_stride;
  const uint16_t* v;
  int64_t v_stride;
  const float* q_gamma;        /* [dim] or NULL */
  const float* k_gamma;        /* [dim] or NULL */
  float eps;                   /* >= 0 */
  v4a_rope rope;
  v4a_dense_cache kv;          /* block_table is not read */
  int32_t* status;             /* optional device word */
} v4a_dense_insert_args;

V4A_API int v4a_dense_insert(const v4a_dense_insert_args* args, void* stream);

/*
 * The same call with the keys as packed rows too: k_out[t][h] = bf16(key), with
 * k_out_stride elements between tokens (16-byte aligned, a multiple of 8, at
 * least num_kv_heads * dim).  k_out may be k (in place, with equal strides) and
 * must overlap nothing else; a skipped token's row is left as it was.  The
 * cache receives what v4a_dense_insert writes.
 *
 * This is the call for V4A_KV_FP8_GROUP caches (v4a_dense_insert returns
 * V4A_ERR_UNSUPPORTED for them), which hold the rows k_out and v quantised as
 * they come, x standing for a row's elements:
 *   pow2(a) = the smallest power of two s with a / s <= 448, at least 2^-126
 *   for each group with rows W among the call's (keys and values and each KV head apart):
 *     old   = 2^-126 if row 0 is in W, else the stored scale
 *     scale = max(old, pow2(max |x| over the finite x of W))
 *     codes of W    = e4m3(x / scale)   (nearest even; infinities become +-448, a NaN its code)
 *     other codes c = e4m3(c * old / scale), if scale > old and row 0 is not in W
 * A group begins anew with its row 0: what its other rows held before is lost
 * then, unless the call writes them.  A stored scale is read by its exponent
 * (0 counts as 2^-126).  The tokens of a group lie within 64 consecutive tokens
 * of the call, as v4a_step_plan leaves them, with a slot each: of tokens farther
 * apart the group holds pieces of any.
 */
V4A_API int v4a_dense_insert_rows(const v4a_dense_insert_args* args, uint16_t* k_out, int64_t k_out_stride, void* stream);

/*
 * Cached rows as packed bf16 rows, each code times its scale rounded once (above
 * 2^-126; V4A_KV_BF16 rows and V4A_KV_FP8_GROUP products exactly).  Row r with
 * row_starts[b] <= r < row_starts[b + 1] receives sequence b's position
 * first[b] + r - row_starts[b].  A row whose block is unallocated or out of
 * range (V4A_DEV_BAD_BLOCK) or whose position is negative or past max_blocks
 * (V4A_DEV_BAD_BATCH) is left as it was, as are the rows before the first
 * sequence and behind the last one.  row_starts must not decrease (otherwise
 * which sequence a row is read from is not defined).  The outputs overlap
 * nothing else.
 */
typedef struct {
  int32_t num_rows;            /* N >= 0: rows of k and v */
  int32_t num_seqs;            /* B >= 0 */
  const int32_t* row_starts;   /* [B + 1] */
  const int32_t* first;        /* [B] first positions, or NULL: 0 */
  v4a_dense_cache kv;
  uint16_t* k;                 /* [N] rows of [num_kv_heads][dim], 16-byte aligned */
  int64_t k_stride;            /* elements between rows: a multiple of 8, at least num_kv_heads * dim */
  uint16_t* v;
  int64_t v_stride;
  int32_t* status;             /* optional device word */
} v4a_dense_read_args;

V4A_API int v4a_dense_read(const v4a_dense_read_args* args, void* stream);

/*
 * Attention.  Sequence b's tokens are t in [token_starts[b],
 * token_starts[b + 1]), at consecutive positions; their keys and values are in
 * the cache already.  For token t at position m and head h (its KV head is
 * h / (num_heads / num_kv_heads)):
 *   visible(j) = j <= m and (window == 0 or j > m - window or j < sinks)
 *   z_j = softmax_scale * q[t][h] . key_j
 *   out[t][h] = sum_j softmax(z)_j value_j over the visible j,
 *   lse[t][h] = ln sum_j exp(z_j).
 * Positions in a block that is unallocated or out of range are left out and
 * set V4A_DEV_BAD_BLOCK (blocks that no query sees are never looked up, so the
 * caller of a window layer may give them back, see v4a_step_plan); a query
 * with nothing left gets 0 and lse = -inf.  A sequence whose entries are inconsistent (starts not
 * increasing or past num_tokens, more than max_new_per_seq tokens, first
 * position negative, last position not first + tokens - 1 or past max_blocks)
 * sets V4A_DEV_BAD_BATCH and its rows are left as they were, as are the rows
 * behind the last sequence.  Cache rows that no query of the call sees do not
 * reach the outputs whatever they hold; a NaN or infinity in a row that one
 * query sees may reach the same sequence's other queries of the same call.
 * Dot products and sums are fp32; the probabilities are rounded as an operand
 * of the tensor cores: to f16 for fp8 caches, to 16 bits for bf16 caches, and
 * to bf16 for the sequences of a bf16 cache that bring more than 32 rows
 * (tokens x heads per KV head; 16 of dim 256) and in the full calls below.  The
 * sum over the values precedes the division: over a bf16 cache it holds while the
 * |value| of a row's visible keys sum up to less than 2^127 (2^119 for those
 * sequences and calls).
 * fp8 value scales below 2^-100 are read as 2^-100; sums over up to 2^26
 * positions of such scales hold (2^13 over a V4A_KV_FP8_TOKEN cache for the
 * sequences of more than 64 rows, 32 of dim 256, and in the full calls).  Keys of
 * an fp8 cache whose exp(z_j) times value scale is below 2^-120 of the largest one
 * may be left out, of lse too, and beside value scales above 2^96 (values past
 * 2^104) more of them.  Over a V4A_KV_FP8_GROUP cache the sequences of more
 * than 32 rows (16 of dim 256), and those of the full calls, take an element of a
 * query to within 2^-17 of its row's largest (exactly down to 2^-9 of that).
 * Sequences that share tokens (entries not increasing)
 * set V4A_DEV_BAD_BATCH once they are more than the call has room for, and
 * what their rows hold then is not defined.
 *
 * A batch may mix decoding sequences and chunks.  A call whose num_tokens
 * reaches num_seqs * max_new_per_seq is taken as one where every sequence
 * brings max_new_per_seq tokens and saves the launches for the other kind:
 * in a batch padded that far, sequences of few rows are attended to in the
 * form for chunks (probabilities in bf16 over bf16 caches, about twice the
 * time); a num_tokens below that, by one token of padding less for instance,
 * keeps each kind its own.  Over V4A_KV_FP8_GROUP caches chunks take
 * kv.max_blocks for the sequences' length when their work is divided: with a
 * table far wider than its sequences short ones take up to 1.7 times as long
 * (results are the same but for the order of sums).  V4A_ERR_UNSUPPORTED: max_new_per_seq
 * * num_heads / num_kv_heads of 2^30 rows or more, V4A_KV_FP8_GROUP blocks of
 * 2^40 bytes or more.
 */
typedef struct {
  int32_t num_tokens;          /* T >= 0: rows of q and out */
  int32_t num_seqs;            /* B >= 0 */
  int32_t max_new_per_seq;     /* host-side bound on one sequence's tokens, >= 1 */
  const int32_t* positions;    /* [T] */
  const int32_t* token_starts; /* [B + 1] */
  v4a_dense_cache kv;
  int32_t num_heads;           /* a multiple of kv.num_kv_heads, <= 1024 */
  const uint16_t* q;           /* [T][H][dim] bf16, 16-byte aligned */
  float softmax_scale;         /* > 0, and finite times log2(e) */
  int32_t window;              /* 0 = every earlier position; else >= 1 */
  int32_t sinks;               /* first positions that stay visible (>= 0; no effect without a window) */
  uint16_t* out;               /* [T][H][dim] bf16, 16-byte aligned; not q */
  float* lse;                  /* [T][H] or NULL */
  int32_t* status;             /* optional device word */
} v4a_dense_attn_args;

/* Bytes of device workspace v4a_dense_attn needs (0 on a bad shape); it is
 * 16-byte aligned and its contents need no initialisation. */
V4A_API size_t v4a_dense_attn_workspace_size(const v4a_dense_attn_args* args);
V4A_API int v4a_dense_attn(const v4a_dense_attn_args* args, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Attention of whole prompts over packed rows.  Sequence b's queries are the
 * tokens t in [token_starts[b], token_starts[b + 1]), n of them; its keys and
 * values the rows [kv_starts[b], kv_starts[b + 1]), N of them.  The queries are
 * the sequence's last positions: the i-th is at position m = N - n + i.
 *   causal:      visible(j) = j <= m and (window == 0 or j > m - window or j < sinks)
 *   not causal:  visible(j) = every j < N
 * with z, out, lse and the KV head of a head as v4a_dense_attn has them.  A query
 * that sees no key (N = 0, or m < 0 where n > N) gets 0 and lse = -inf.  A
 * sequence whose entries are inconsistent (starts decreasing, negative or past
 * num_tokens or num_kv_tokens, more than max_new_per_seq queries) sets
 * V4A_DEV_BAD_BATCH and its rows are left as they were, as are the rows behind
 * the last sequence.  Sequences may share keys, not queries (V4A_DEV_BAD_BATCH
 * once they are more than the call has room for, and what their rows hold then
 * is not defined).  Rows outside [kv_starts[b], kv_starts[b + 1]) do not reach
 * sequence b's outputs whatever they hold; a NaN or infinity inside may reach
 * any of them.  Dot products and sums are fp32; the probabilities are rounded
 * to bf16, the output once.  The sum over the values precedes the division: it
 * holds while the |value| of a row's visible keys sum up to less than 2^127, and
 * elements of an output below 2^-102 may be zeros.
 */
typedef struct {
  int32_t num_tokens;          /* T >= 0: rows of q and out */
  int32_t num_kv_tokens;       /* rows of k and v, 0..2^30 */
  int32_t num_seqs;            /* B >= 0 */
  int32_t max_new_per_seq;     /* host-side bound on one sequence's queries, 1..2^22 */
  const int32_t* token_starts; /* [B + 1] */
  const int32_t* kv_starts;    /* [B + 1], or NULL: token_starts */
  int32_t num_heads;           /* H, a multiple of num_kv_heads, <= 1024 */
  int32_t num_kv_heads;
  int32_t dim;                 /* 64, 128, 192 or 256 */
  int32_t causal;              /* 1 or 0 */
  int32_t window;              /* 0 = every earlier position; else >= 1 (causal only) */
  int32_t sinks;               /* first positions that stay visible (>= 0; no effect without a window) */
  float softmax_scale;         /* > 0, and finite times log2(e) */
  const uint16_t* q;           /* [T] rows of [H][dim] bf16; rows 16-byte aligned, strides multiples of 8 elements */
  int64_t q_stride;            /* elements between tokens, >= H * dim */
  const uint16_t* k;           /* [num_kv_tokens] rows of [num_kv_heads][dim] */
  int64_t k_stride;
  const uint16_t* v;
  int64_t v_stride;
  uint16_t* out;               /* [T][H][dim] bf16, 16-byte aligned; overlaps no input */
  float* lse;                  /* [T][H] or NULL */
  int32_t* status;             /* optional device word */
} v4a_prompt_attn_args;

/* Bytes of device workspace v4a_prompt_attn needs (0 on a bad shape); it is
 * 16-byte aligned and its contents need no initialisation. */
V4A_API size_t v4a_prompt_attn_workspace_size(const v4a_prompt_attn_args* args);
V4A_API int v4a_prompt_attn(const v4a_prompt_attn_args* args, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* V4A_DENSE_H */

/*
 * topkp_decode.h -- decoding with several hypotheses at once: the calls of
 * libtopkp.so that stand next to the logit filter of topkp.h when a request
 * is decoded with beams or with drafted tokens.
 *
 *   topkp_beam_select     the best continuations of each request's beams
 *   topkp_beam_reorder    the states (caches) of the beams follow them
 *   topkp_cache_write     new keys and values into a paged or plain cache,
 *                         in its own type or quantised to e4m3
 *   topkp_cache_read      the cache's entries back as dense rows
 *   topkp_tree_attention  attention of one token, a drafted chain or a
 *                         drafted tree of each request over its cache
 *
 * The conventions of topkp.h hold: device pointers owned by the caller, no
 * allocation per call, asynchronous launches on the caller's stream, host
 * checks that never synchronise, topkp_last_error_string() for the reason of
 * a refusal.  On a refusal nothing was launched; after TOPKP_ERR_LAUNCH of a
 * call of several launches, those before the failed one may have been.  Every
 * result is deterministic.
 */
#ifndef TOPKP_DECODE_H
#define TOPKP_DECODE_H

#include "topkp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest beams per request and candidates per request of topkp_beam_select. */
#define TOPKP_MAX_BEAMS 64
#define TOPKP_MAX_CANDIDATES 128
/* Largest head dimension, and largest number of nodes of a drafted tree that
 * is given by masks (a chain may be longer). */
#define TOPKP_MAX_HEAD_DIM 256
#define TOPKP_MAX_TREE 64

/*
 * topkp_beam_select -- one step of beam search.  For request b, beam k and
 * token v, with x = logits[b * K + k]:
 *   candidate(k, v) = scores[b][k] + x[v] - log(sum over u of exp(x[u])).
 * A beam whose finished flag is set has one candidate, (pad_token, its score
 * unchanged), and its logits are not read.  The n best candidates of each
 * request come out in descending order; equal candidates in increasing
 * k * V + v.  Logits of -inf (what the filter removed) are never candidates;
 * a beam whose score is -inf, or whose row holds no finite logit, has none.
 * An output slot j without a candidate holds score -inf, token -1 and parent
 * j mod K (so that it may be handed to topkp_beam_reorder).
 *
 *   logits     device, [B * K, V] of dtype, row stride ld_logits (>= V).
 *   B, K, V    requests, beams of each (1 .. TOPKP_MAX_BEAMS) and tokens;
 *              B == 0 returns TOPKP_SUCCESS without a launch.  V >= 1 and at
 *              most TOPKP_MAX_V.
 *   scores     device, [B, K] float: the beams' summed log-probabilities.
 *   finished   device, [B, K] uint8 (0 or not), or NULL (none finished).
 *   pad_token  in [0, V): the token a finished beam goes on with.
 *   n          candidates of each request, 1 .. TOPKP_MAX_CANDIDATES.
 *   out_score, out_parent, out_token
 *              device, [B, n] float, int32 (beam of the request), int32.
 *   workspace  device, at least topkp_beam_select_workspace_size(...) bytes,
 *              256-byte aligned; contents on entry do not matter.
 * Scores and logits may be any finite numbers (a dead beam's -1e9, a mask of
 * the type's lowest value).  Candidates are compared in 64-bit floating point,
 * those of one beam by their logits.  The normaliser of a row is summed from
 * fp32 exponentials: its error is below 1e-6, so two candidates of different
 * beams that lie nearer than that, or than a step of 64 bits, may change
 * places; those of one beam never do.  A candidate below fp32's range comes
 * out with score -inf.  NaN and +inf among logits or scores give unspecified
 * output.  Two launches.
 */
size_t topkp_beam_select_workspace_size(int64_t B, int64_t K, int64_t V, topkp_dtype dtype, int32_t n);
topkp_status topkp_beam_select(const void* logits, int64_t B, int64_t K, int64_t V, int64_t ld_logits,
                               topkp_dtype dtype, const float* scores, const uint8_t* finished, int32_t pad_token,
                               int32_t n, float* out_score, int32_t* out_parent, int32_t* out_token, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * One state of the beams for topkp_beam_reorder: rows of `blocks` blocks of
 * `entries` entries of `entry_bytes` bytes.  A cache [rows, time, heads, dim]
 * has one block of `time` entries; [rows, heads, time, dim] has `heads`
 * blocks.  Entries of a block are contiguous; strides are in bytes.
 * dst == src with equal strides reorders in place; otherwise dst must not
 * overlap any src of the call.  States may lie between each other's rows and
 * blocks (views of one tensor): no byte may be written that another state
 * reads or writes.  That is decided exactly for equal strides; states of two
 * block strides may not interleave within a row, nor states of two row
 * strides at all.
 */
typedef struct {
  const void* src;
  void* dst;
  int64_t src_row_stride, dst_row_stride;
  int64_t src_block_stride, dst_block_stride;
  int64_t blocks, entries, entry_bytes;
} topkp_state;

/*
 * topkp_beam_reorder -- row b * K + j of every state becomes row
 * b * K + parent[b][j] as it was before the call.
 *
 *   states   host array of `count` descriptors, read during the call.
 *   parent   device, [B, K] int32, entries in [0, K); a row whose entry lies
 *            outside is left as it is.
 *   lengths  device, [B, K] int32, or NULL: only the first
 *            lengths[b][parent[b][j]] entries of each block are live and
 *            move; the rest of the destination row keeps what it held.
 * In place a row that is its own parent costs nothing.  One launch for every
 * 32 states whose places and sizes are multiples of 16 bytes (4 where K is
 * above 32), of 4, and of neither.
 */
topkp_status topkp_beam_reorder(const topkp_state* states, int64_t count, int64_t B, int64_t K, const int32_t* parent,
                                const int32_t* lengths, void* stream);

/* Element types of a cache: that of the rows written, or e4m3 (1 sign, 4
 * exponent and 3 mantissa bits, largest value 448) with exponents. */
#define TOPKP_E4M3 3

/*
 * A cache of keys or of values: token t of page p, head h, element d is at
 * data[p * page_stride + t * token_stride + h * head_stride + d] (strides in
 * elements, the head's elements contiguous).  With dtype TOPKP_E4M3 the
 * element stands for its value times 2^(exponents[p * exp_page_stride +
 * t * exp_token_stride + h * exp_head_stride] - 127); otherwise exponents
 * is NULL.
 */
typedef struct {
  void* data;
  uint8_t* exponents;
  int32_t dtype; /* topkp_dtype or TOPKP_E4M3 */
  int64_t page_stride, token_stride, head_stride;
  int64_t exp_page_stride, exp_token_stride, exp_head_stride;
} topkp_cache;

/*
 * topkp_cache_write -- rows k[i], v[i] ([H, D], of dtype, strides in
 * elements) go to token slots[i] % page_size of page slots[i] / page_size.
 * A slot outside [0, pages * page_size) is skipped; rows with the same
 * slot race, and what is left there is unspecified.
 * Quantised, a (token, head) row shares one power of two: 2^e with e the
 * smallest integer >= -126 for which every finite |x| <= 448 * 2^e (e = -126
 * for a row of zeros); the stored value is x * 2^-e rounded to e4m3 once, to
 * the nearest, ties to even, and the stored exponent e + 127.  Infinities
 * become the largest value, NaN stays NaN.  As the scale is a power of two
 * the only error of the cache is that one rounding.  At the top of a type's
 * range it goes past it: fp16 magnitudes from 63488 stand for 65536, bf16 and
 * fp32 ones from 1.9375 * 2^127 for 2^128.
 *
 *   k, v        device, [N, H, D] of dtype (v NULL together with v_cache
 *               NULL: keys alone).
 *   slots       device, [N] int64.
 *   k_cache, v_cache  host descriptors, read during the call; their dtype
 *               is dtype or TOPKP_E4M3.
 * D is at most TOPKP_MAX_HEAD_DIM.  One launch.
 */
topkp_status topkp_cache_write(const void* k, const void* v, int64_t N, int64_t H, int64_t D, int64_t k_token_stride,
                               int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                               topkp_dtype dtype, const int64_t* slots, const topkp_cache* k_cache,
                               const topkp_cache* v_cache, int64_t pages, int64_t page_size, void* stream);

/*
 * topkp_cache_read -- the reverse: row i of k and v ([N, H, D] of dtype,
 * contiguous) gets the values at slots[i]; a slot outside the cache gives a
 * row of zeros.  A quantised cache is read as its exact values, rounded once
 * to dtype; a value beyond dtype's range is an infinity.
 */
topkp_status topkp_cache_read(const int64_t* slots, int64_t N, int64_t H, int64_t D, const topkp_cache* k_cache,
                              const topkp_cache* v_cache, int64_t pages, int64_t page_size, topkp_dtype dtype, void* k,
                              void* v, void* stream);

/*
 * topkp_tree_attention -- the drafted nodes of each request attend to its
 * cache and to each other.  Request b has context[b] tokens in the cache,
 * and its node i stands at token context[b] + i (written before the call).
 * Node i sees every token of the context, and node j iff bit j of
 * tree[b][i] is set; with tree NULL, iff j <= i (a chain; T = 1 is ordinary
 * decoding).  For query head h, with the keys and values of head
 * h / (Hq / Hkv):
 *   out = sum over seen t of softmax_t(scale * q . k_t) v_t,
 *   lse = log(sum over seen t of exp(scale * q . k_t)).
 * A node that sees nothing, and every node i >= nodes[b], gets zeros and an
 * lse of -inf.
 *
 *   q, out      device, [B, T, Hq, D] of dtype (TOPKP_F16 or TOPKP_BF16),
 *               strides in elements, a head's elements contiguous.
 *   lse         device, [B, T, Hq] contiguous float, or NULL.
 *   k, v        the caches (one dtype for both): dtype or TOPKP_E4M3.
 *   table       device, [B, max_pages] int32, row stride ld_table: token t of
 *               request b is token t % page_size of page
 *               table[b][t / page_size].  A page outside [0, pages) reads as
 *               zeros.  NULL: page b is request b's whole cache (page_size
 *               its capacity, pages == B, max_pages == 1).
 *   context     device, [B] int32; read as if clamped to [0, capacity],
 *               capacity = max_pages * page_size, at most 2^31 - 1024.
 *               Nodes beyond the capacity are seen by none.
 *   nodes       device, [B] int32 (1 .. T), or NULL (T for all).
 *   tree        device, [B, T] uint64, T <= TOPKP_MAX_TREE, or NULL.
 *   scale       of the products.
 *   max_context an upper bound of context[b] that plans how the work is
 *               split (results hold for any value, speed for a true one).
 *   workspace   device, at least topkp_tree_attention_workspace_size()
 *               bytes, 256-byte aligned.
 * D is a multiple of 8, at most TOPKP_MAX_HEAD_DIM; pointers and strides of
 * q, out and the caches are multiples of 16 bytes (8 for an e4m3 cache);
 * exponents are strided by less than 2^32.
 * Products and sums are fp32; probabilities are rounded to dtype before the
 * product with the values (fp16's weights below 2^-32 of the row's largest
 * become zero there, those below 2^-21 lose bits).  Over an e4m3 cache q is taken as a sum of e4m3
 * terms (an element is off by at most about 2^-18 of the largest of its row),
 * and cached values are rounded to dtype: exact within its range, an infinity
 * beyond it, and with fp16 rows in steps of 2^-24 below 2^-14.  A
 * value that is not finite spoils the rows of its request that do not see it
 * too, if it is that of a drafted node, and an infinite one may leave NaN;
 * tokens past the last node are never used.  One launch, or two where the
 * tokens are split.
 */
typedef struct {
  const void* q;
  void* out;
  float* lse;
  topkp_cache k, v;
  const int32_t* table;
  const int32_t* context;
  const int32_t* nodes;
  const uint64_t* tree;
  void* workspace;
  size_t workspace_bytes;
  int64_t B, T, Hq, Hkv, D;
  int64_t pages, page_size, max_pages, ld_table, max_context;
  int64_t q_batch_stride, q_token_stride, q_head_stride;
  int64_t out_batch_stride, out_token_stride, out_head_stride;
  topkp_dtype dtype;
  float scale;
} topkp_tree_attention_args;

/* Reads the shape fields (B, T, Hq, Hkv, D, max_context, page_size,
 * max_pages) and the dtypes of args only. */
size_t topkp_tree_attention_workspace_size(const topkp_tree_attention_args* args);
topkp_status topkp_tree_attention(const topkp_tree_attention_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TOPKP_DECODE_H */

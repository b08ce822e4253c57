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
 * and when several continuations share a prompt, or drafted tokens are tried:
 *
 *   topkp_shared_attention  the same where requests share a prefix, whose keys
 *                         and values are read once for all of them
 *   topkp_draft_verify    which drafted tokens the target's probabilities
 *                         accept, and the token to go on with
 *   topkp_cache_compact   the accepted tokens of a tree move up behind the
 *                         context
 *   topkp_cache_fork      block tables and pages follow the requests that go
 *                         on: forked, freed and grown
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
/* Largest number of rows of a block table that topkp_cache_fork takes or makes. */
#define TOPKP_MAX_ROWS 8192

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

/*
 * topkp_shared_attention -- topkp_tree_attention of requests that share a
 * prefix.  The B requests are `groups` runs of B / groups consecutive ones;
 * tokens [0, shared[g]) are the same for all requests of group g (the same
 * pages, or equal contents), and are read once for all of them, through the
 * block table of the group's first request that has a node.  The result is
 * that of topkp_tree_attention but for the order of the sums.
 *
 *   args        as for topkp_tree_attention; table is not NULL.
 *   shared      device, [groups] int32.  What is read once is the largest
 *               multiple of 64 tokens within shared[g] and within the context
 *               of every request of the group that has a node; a value of
 *               zero or less, or one that is too small, costs speed only.
 *   groups      at least 1, divides B.
 *   max_shared  an upper bound of shared[g] that plans how the work is split
 *               (results hold for any value).  The nearer the better: what
 *               it leaves of max_context is planned as the requests' own, so
 *               with a bound far above the truth few CTAs take those.
 * args->workspace has topkp_shared_attention_workspace_size() bytes.  Three
 * launches, or those of topkp_tree_attention where the plan finds too little
 * shared to be worth them.
 */
size_t topkp_shared_attention_workspace_size(const topkp_tree_attention_args* args, int64_t groups, int64_t max_shared);
topkp_status topkp_shared_attention(const topkp_tree_attention_args* args, const int32_t* shared, int64_t groups,
                                    int64_t max_shared, void* stream);

/*
 * topkp_draft_verify -- speculative decoding's choice.  Request b has T
 * drafted nodes, node 0 the last accepted token (its own token is not looked
 * at).  With p the softmax of the target's logits after node n, the children
 * of n are tried in increasing order, and the walk goes on at the first that
 * is accepted; where none is, one token is drawn, and the walk ends.
 *   draft given: the children's tokens are independent draws from q, the
 *     softmax of the draft's logits after n.  Child c with token x is accepted
 *     iff uniform[c] * q(x) < p(x); after a child that is not, p becomes
 *     max(p - q, 0) over its sum.
 *   draft NULL: the children are certain (q is 1 at the child's token): x is
 *     accepted iff uniform[c] < p(x), and otherwise taken out of p, whose rest
 *     is divided by its sum.
 *   The token drawn is the largest p(v) / (race[v] + eps), the lowest v of
 *     equal ones; with race i.i.d. from Exp(1) it is a draw from p.  Where
 *     nothing is left of p (which roundings alone can bring about) it is drawn
 *     from p as it was at first.
 *   uniform and race both NULL (greedy): a child is accepted iff its token is
 *     the lowest index of the largest logit after n, and that is the token
 *     drawn.  draft must be NULL.
 * With uniform numbers of [0, 1) the emitted tokens are distributed as the
 * target's own.  A token outside [0, V) is never accepted and changes nothing.
 *
 *   target     device, [B, T, V] of dtype, strides in elements (node_stride
 *              >= V), V contiguous; -inf is a token that the filter removed.
 *              Rows of nodes that are not accepted do not matter (those of
 *              first children may be read).
 *   draft      device, the same, or NULL; rows of nodes without children are
 *              not read.
 *   tokens     device, [B, T] int32.
 *   parent     device, [B, T] int32: node i (i > 0) is a child of
 *              parent[b][i] < i, other nodes are nobody's; NULL: a chain.
 *   nodes      device, [B] int32 (clamped to [0, T]), or NULL (T for all).
 *   uniform    device, [B, T] float (that of node 0 is not used).
 *   race       device, [B, V] float, row stride ld_race; expected >= 0.
 *   eps        added to every race, >= 0.
 *   T          1 .. TOPKP_MAX_TREE.  V at most TOPKP_MAX_V.
 *   count      device, [B] int32: nodes of the accepted path, node 0 included;
 *              0 for a request without nodes.
 *   path       device, [B, T] int32: the nodes of that path, then -1.
 *   token      device, [B] int32: the token drawn; -1 for a request without
 *              nodes, and where a row has no logit above -inf.
 *   logprob    device, [B, T] float, or NULL: log p (of the node's whole row)
 *              of the path's second token and on, and behind them of the token
 *              drawn; 0 elsewhere.
 * Probabilities and sums are fp32, and one below 2^-126 of its row's largest
 * counts as zero; otherwise a decision may differ from exact arithmetic where
 * its two sides lie within about 1e-6 (relative to p) of one another.
 * NaN and +inf give an unspecified result.  One launch.
 */
typedef struct {
  const void* target;
  const void* draft;
  const int32_t* tokens;
  const int32_t* parent;
  const int32_t* nodes;
  const float* uniform;
  const float* race;
  int32_t* count;
  int32_t* path;
  int32_t* token;
  float* logprob;
  int64_t B, T, V;
  int64_t target_batch_stride, target_node_stride, draft_batch_stride, draft_node_stride, ld_race;
  topkp_dtype dtype;
  float eps;
} topkp_draft_verify_args;
topkp_status topkp_draft_verify(const topkp_draft_verify_args* args, void* stream);

/*
 * One tensor of pages for topkp_cache_fork and topkp_cache_compact: page p
 * has `blocks` blocks of page_size entries of entry_bytes bytes, one after
 * another; strides in bytes.  A cache [pages, page_size, heads, dim] has one
 * block; [pages, heads, page_size, dim] has `heads`.  Keys, values and
 * exponents of every layer are states of one call.  States may lie between
 * each other's pages (views of one tensor) but share no byte, as in
 * topkp_beam_reorder.
 */
typedef struct {
  void* data;
  int64_t page_stride, block_stride;
  int64_t blocks, entry_bytes;
} topkp_pages;

/*
 * topkp_cache_fork -- new row n of the block table goes on from old row
 * source[n], whose first lengths[source[n]] tokens are live.
 *   - Whole pages are shared with the old row.  A partly filled last page
 *     stays with the first new row that continues it, if nobody else holds
 *     it; every other row gets a free page and a copy of the live tokens.
 *   - The row then grows by free pages to hold `grow` tokens more, but to no
 *     more than max_pages pages.  Its other entries become -1.
 *   - What the old rows held and no new row does is given up.  refs counts
 *     the holders of a page; one without any is free.  Holders outside the
 *     table (another table, a prefix kept for later) count like rows.
 *   - Free pages are given out in increasing order: row after row, a row's
 *     copy before its growth.
 * So one call forks, reorders, frees (a row that no source names), starts
 * (a source outside [0, R) is an empty row) and grows requests.  Where fewer
 * pages are free than wanted nothing happens: missing[0] is how many lack,
 * the new table is all -1, refs_out equals refs, no page is written.
 *
 *   states     host array of `count` descriptors, read during the call.
 *   table      device, [R, max_pages] int32, row stride ld_table; an entry
 *              outside [0, pages) holds nothing and goes on as -1.
 *   lengths    device, [R] int32, clamped to [0, max_pages * page_size].
 *   source     device, [N] int32.
 *   grow       device, [N] int32, or NULL: grow_all for every row.
 *   refs       device, [pages] int32, at least 1 for every entry of the table.
 *   table_out  device, [N, max_pages] int32, row stride ld_out; not table.
 *   refs_out   device, [pages] int32; refs itself, or apart from it.
 *   missing    device, [1] int32.
 *   workspace  device, at least topkp_cache_fork_workspace_size() bytes,
 *              256-byte aligned.
 * R and N are at most TOPKP_MAX_ROWS, R or N times max_pages at most 2^30;
 * N == 0 frees every row.  One launch, and one for every 128 states.
 */
typedef struct {
  const topkp_pages* states;
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* source;
  const int32_t* grow;
  const int32_t* refs;
  int32_t* table_out;
  int32_t* refs_out;
  int32_t* missing;
  void* workspace;
  size_t workspace_bytes;
  int64_t count, R, N, max_pages, ld_table, ld_out, pages, page_size, grow_all;
} topkp_cache_fork_args;
size_t topkp_cache_fork_workspace_size(int64_t N, int64_t pages);
topkp_status topkp_cache_fork(const topkp_cache_fork_args* args, void* stream);

/*
 * topkp_cache_compact -- of request b's tokens from start[b] on, those at
 * start[b] + keep[b][j] move to start[b] + j, j < kept[b] (topkp_draft_verify's
 * path and count, after which the request's length is start[b] + kept[b]).
 * All are read as they were before the call.  An entry with keep[b][j] <= j,
 * or of which either place lies outside the request's pages, is left alone,
 * and so is a request with start[b] < 0.
 *
 *   states     host array of `count` descriptors, read during the call.
 *   table      device, [B, max_pages] int32, row stride ld_table, or NULL:
 *              page b is request b's whole cache (pages == B, max_pages 1).
 *              No two requests hold a page that either moves tokens in.
 *   start, kept  device, [B] int32.
 *   keep       device, [B, W] contiguous int32, W at most TOPKP_MAX_TREE.
 * One launch for every 128 states.
 */
topkp_status topkp_cache_compact(const topkp_pages* states, int64_t count, int64_t B, int64_t W, const int32_t* table,
                                 int64_t ld_table, int64_t max_pages, int64_t pages, int64_t page_size,
                                 const int32_t* start, const int32_t* keep, const int32_t* kept, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TOPKP_DECODE_H */

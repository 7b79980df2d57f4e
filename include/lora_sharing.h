/*
 * lora_sharing.h - C ABI for requests that share what they have cached (parallel
 * samples, beams, a common system prompt) on GB300 (sm_103a), next to the
 * attention side of a serving step (lora_attention.h):
 *
 *   lora_beam_select    the best continuations of each request over its beams
 *                       and the vocabulary
 *   lora_kv_fork        block tables of the next batch from its rows' parents:
 *                       shared pages, copies on write, pages that come free
 *   lora_kv_compact     block tables after the pages in use have moved to the
 *                       front of the cache
 *   lora_kv_copy        the pages' data, all layers in one launch
 *   lora_attend_shared  lora_attend where groups of requests share a prefix,
 *                       which is read once a group
 *
 * Conventions are those of lora_attention.h: asynchronous on the caller's
 * stream, no allocation, no synchronisation, capturable in a CUDA graph; host
 * checks return a status before anything is enqueued, errors found in device
 * data go to the caller's word `err` (first error wins, never cleared here; it may
 * be null).  Values read from device memory never send an access out of the
 * buffers described by the arguments.  Outputs must not overlap inputs, unless said
 * otherwise.
 */
#ifndef LORA_SHARING_H
#define LORA_SHARING_H

#include "lora_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_MAX_BEAMS 64
#define LORA_MAX_VOCAB (1 << 24)
#define LORA_MAX_PAGES (1 << 20)
#define LORA_MAX_KV_LAYERS 128

/*
 * Selection of beam search.  Request r has rows r beams .. r beams + beams - 1
 * of logits, one a beam; beam b's candidates are the tokens v with
 *     c(b, v) = scores[b] + logits[b][v] - ln sum_u exp(logits[b][u])
 * and, for a beam that has ended (ended[b] != 0; its logits are not read), the
 * token eos alone with c = scores[b].  The `keep` best candidates of the request
 * are written in falling order, the lowest row and then the lowest token first
 * among equals:
 *   parents     int32 [n_req keep], the row of the beam (0 .. n_req beams - 1)
 *   tokens      int32 [n_req keep]
 *   out_scores  fp32  [n_req keep], c rounded once
 *   out_ended   int32 [n_req keep], 1 where the beam had ended or token = eos
 * Candidates of -inf are not taken (masked tokens, beams with a score of -inf);
 * places that are left get parent -1, token -1, score -inf, ended 0.  A beam with a
 * NaN or +inf among its logits, a score that is NaN or +inf, or no logit above -inf
 * has no candidates.  Candidates are compared in 64 bits; the sum in the logarithm
 * is taken in fp32, within 2^-17 of itself whatever the vocabulary (about 2^-21 as measured).
 *   logits  bf16 or fp32 [n_req beams, ld], `vocab` columns used; aligned to
 *           its elements, any ld >= vocab
 *   scores  fp32 [n_req beams]; ended int32 [n_req beams], or null: none has
 *   eos     the token that ends a beam; -1: none (ended must be null then)
 *   ws      lora_beam_select_workspace_bytes() bytes, 16-byte aligned, zeroed
 *           once before the first call; every call leaves its counters as it
 *           found them.  Calls that may overlap need a workspace each
 * Outputs must not overlap inputs, but where keep = beams out_scores may be
 * scores and out_ended ended.  Limits: 1 <= beams, keep <= LORA_MAX_BEAMS,
 * 1 <= vocab <= LORA_MAX_VOCAB, n_req <= LORA_MAX_SEQS (LORA_ERR_INVALID_ARG).
 * One launch.
 */
typedef enum { LORA_LOGITS_BF16 = 0, LORA_LOGITS_FP32 = 1 } lora_logits_t;

lora_status_t lora_beam_select_workspace_bytes(int32_t n_req, int32_t beams, int32_t keep, int32_t vocab,
                                               size_t *bytes);

lora_status_t lora_beam_select(const void *logits, int64_t ld, lora_logits_t type, int32_t n_req, int32_t beams,
                               int32_t vocab, int32_t keep, const float *scores, const int32_t *ended, int32_t eos,
                               int32_t *parents, int32_t *tokens, float *out_scores, int32_t *out_ended, void *ws,
                               size_t ws_bytes, lora_stream_t stream);

/*
 * The next batch's tables.  Row i of the new batch continues row p = parents[i]
 * of the old one (-1: an empty request); with pages(n) = ceil(n / page_size):
 *   dst_lens[i] = src_lens[p]
 *   dst_table[i][e] = src_table[p][e], e < pages(src_lens[p])
 * but a last page that is not full belongs to one row alone, because tokens will
 * be appended to it: the lowest i with parent p keeps it, each other one gets
 * the next free page in its place and a copy job:
 *   copies[i] = {source page, destination page, tokens in it}, {-1, -1, 0} where
 *               row i needs none: what lora_kv_copy takes
 * Entries of dst_table from pages(dst_lens[i]) on are left as they were.  (Old
 * rows are taken to hold their last page alone where it is not full, as they do
 * after this call and lora_kv_step.)  Pages that neither the new rows nor
 * `held` name are free; they serve the copies in rising order (row order), and
 * the others are listed:
 *   free_pages  int32 [n_pages], free ids rising, then -1
 *   n_free      int32 [1], how many
 * So pages of rows without a child come free here, and parents = 0, 1, 2, ... only
 * lists free pages.  lora_kv_step takes pages from the front of this list (its
 * entries of -1 are reported there if they are reached).
 *   held        int32 [n_held], pages in use outside the rows (prefix caches, other
 *               batches); -1 is passed over
 * dst_table and dst_lens must not overlap src_table and src_lens
 * (LORA_ERR_INVALID_ARG).  Limits: n_src, n_dst <= LORA_MAX_SEQS (LORA_ERR_INVALID_ARG),
 * n_pages <= LORA_MAX_PAGES (LORA_ERR_UNSUPPORTED).  Device errors:
 * LORA_ERR_INVALID_ARG (a parent outside [-1, n_src), a length that is negative or longer
 * than either table's row: the new row is empty), LORA_ERR_NO_PAGES (no page for a copy:
 * the row's length is cut to its full pages), LORA_ERR_SLOT_RANGE (a page id outside
 * [0, n_pages): the entry is copied and counts nowhere; as a source it is not copied).
 * One launch.
 */
lora_status_t lora_kv_fork(const int32_t *src_table, int64_t ld_src, int32_t src_width, const int32_t *src_lens,
                           int32_t n_src, const int32_t *parents, int32_t n_dst, int32_t page_size, int32_t n_pages,
                           const int32_t *held, int32_t n_held, int32_t *dst_table, int64_t ld_dst, int32_t dst_width,
                           int32_t *dst_lens, int32_t *copies, int32_t *free_pages, int32_t *n_free, int32_t *err,
                           lora_stream_t stream);

/*
 * Pages in use moved to the front of the cache.  With U the number of pages that the
 * rows' first pages(lens[i]) entries or `held` name: the k-th of them (rising) that
 * is >= U moves to the k-th id (rising) below U that is not in use.
 *   dst_table   the rows' first pages(lens[i]) entries after the move; others are
 *               left as they were; must not overlap src_table
 *   dst_held    int32 [n_held], held after the move (-1 stays)
 *   moves       int32 [n_pages / 2][3]: {source, destination, page_size} of move k,
 *               then {-1, -1, 0}: what lora_kv_copy takes
 *   n_moves     int32 [1]
 *   free_pages  int32 [n_pages]: U, U + 1, .., n_pages - 1, then -1; n_free int32 [1]
 * No destination is a source, so the moves can be copied in any order.  Limits and
 * device errors as for lora_kv_fork (a row with a bad length counts as empty; a bad
 * page id stays as it is).  One launch.
 */
lora_status_t lora_kv_compact(const int32_t *src_table, int64_t ld_src, int32_t width, const int32_t *lens,
                              int32_t n_seq, int32_t page_size, int32_t n_pages, const int32_t *held, int32_t n_held,
                              int32_t *dst_table, int64_t ld_dst, int32_t *dst_held, int32_t *moves, int32_t *n_moves,
                              int32_t *free_pages, int32_t *n_free, int32_t *err, lora_stream_t stream);

/*
 * Copies of pages' data in each of n_layers caches (host array kvs) of one
 * geometry: equal n_pages, page_size, n_kv, head_dim, strides and type
 * (LORA_ERR_INVALID_ARG), 1 <= n_layers <= LORA_MAX_KV_LAYERS.  For row {s, d, m} of
 * copies (int32 [n_copies][3]) the first m tokens of page s, k and v, all heads,
 * are written to page d; s = -1 or d = -1: nothing, whatever m.  count (device int32 [1], may be
 * null) bounds the rows that are looked at.  The rows are copied in no order: a page
 * that is the destination of one row must not be named by another, and pages that
 * overlap in memory race.  Device errors: LORA_ERR_SLOT_RANGE (a page outside
 * [-1, n_pages)), LORA_ERR_INVALID_ARG (m outside [0, page_size]): that row is not
 * copied; LORA_ERR_INVALID_ARG too for a count outside [0, n_copies], which is cut to it.
 * n_copies may be 0.  One launch.
 */
lora_status_t lora_kv_copy(const lora_kv_t *kvs, int32_t n_layers, const int32_t *copies, int32_t n_copies,
                           const int32_t *count, int32_t *err, lora_stream_t stream);

typedef enum { LORA_SHARE_AUTO = 0, LORA_SHARE_ALWAYS = 1 } lora_share_t;

/*
 * lora_attend for groups of requests that share a prefix.  Requests
 * [group_offsets[g], group_offsets[g + 1]) hold the same keys and values at their
 * positions below prefix_lens[g] (in the same or in different pages): those are
 * read once for all rows of the group, through the table row of its first request with
 * rows, and each request's other positions through its own row, by the decode path
 * whatever the number of rows.  The result is what lora_attend computes, up to rounding:
 * weights of a shared prefix are rounded to bf16 (over LORA_KV_E4M3 to f16, times 2^7)
 * before the product with v, as on lora_attend's prompt path, so that how a row's
 * weights are rounded depends on whether its group shares.  Where a request of the group
 * with rows has cached less before its own rows, the prefix is cut to that; groups with
 * fewer than two requests with rows, and requests outside every group, share nothing.
 *   group_offsets  int32 [n_groups + 1], non-decreasing, within [0, n_seq]
 *   prefix_lens    int32 [n_groups]
 *   n_groups       0 .. LORA_MAX_SEQS
 *   ws             lora_attend_shared_workspace_bytes() bytes for at least this T and
 *                  n_seq, 16-byte aligned, zeroed once before the first call; every
 *                  call leaves it as it found it, up to values that no call reads (but
 *                  zero it again after a call that reports LORA_ERR_TIMEOUT, which joins
 *                  nothing: rows of requests that share are not written, and calls
 *                  that share report it too until then).  Calls that may overlap need a
 *                  workspace each (LORA_ERR_WORKSPACE in err where that is noticed)
 *   mode           LORA_SHARE_AUTO: prefixes are read once where that is estimated to
 *                  save time, which short ones do not (decided on the device, from the
 *                  lengths; a call that turns out to share nothing takes longer than
 *                  lora_attend, 1 us with short tables and 11 with long ones as
 *                  measured); LORA_SHARE_ALWAYS: all of them
 * A NaN or infinity in a value of the prefix that some row of the group sees can reach
 * the group's other rows.  All other arguments, limits and device errors are lora_attend's;
 * LORA_ERR_INVALID_ARG in err also reports group offsets out of order or range and negative
 * prefix lengths (that group shares nothing).  Nothing is shared where offsets of groups or
 * of rows are out of order or range.  Made for few rows a request (decode, speculative
 * decode); any number is computed.
 */
typedef struct {
    const int32_t *group_offsets, *prefix_lens;
    int32_t n_groups;
    int32_t mode; /* lora_share_t */
} lora_prefix_t;

lora_status_t lora_attend_shared_workspace_bytes(const lora_attention_t *att, const lora_kv_t *kv, int32_t T,
                                                 int32_t n_seq, size_t *bytes);

lora_status_t lora_attend_shared(const void *q, int64_t ldq, void *out, int64_t ldo, float *lse, int32_t T,
                                 int32_t n_seq, const int32_t *q_offsets, const int32_t *kv_lens,
                                 const int32_t *block_table, int64_t ld_table, int32_t table_width,
                                 const lora_prefix_t *prefix, const lora_kv_t *kv, const lora_attention_t *att,
                                 int32_t max_q_hint, void *ws, size_t ws_bytes, int32_t *err, lora_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_SHARING_H */

/*
 * lora_attention.h - C ABI of the attention side of a serving step on GB300
 * (sm_103a): what runs between the packed QKV projection (with its LoRA
 * branch, lora_gemm.h) and the output projection.
 *
 *   lora_kv_step      block tables, slot map and positions of a step, from
 *                     request lengths
 *   lora_rope_append  rotary positions of q and k; k and v into the paged cache
 *   lora_attend       attention of the step's tokens over the paged cache
 *
 * Conventions are those of lora_gemm.h: asynchronous on the caller's stream, no
 * allocation, no synchronisation, capturable in a CUDA graph; host checks
 * return a status before anything is enqueued, errors found in device data go
 * to the caller's word `err` (first error wins, never cleared here).  Values
 * read from device memory (lengths, page ids, slots) never send an access out
 * of the buffers described by the arguments.
 */
#ifndef LORA_ATTENTION_H
#define LORA_ATTENTION_H

#include "lora_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_MAX_SEQS 4096
#define LORA_MAX_PAGE_SIZE 1024
#define LORA_MAX_HEAD_DIM 256
#define LORA_MAX_KV_LEN (1 << 25)

/* Element type of the cache. */
typedef enum {
    LORA_KV_BF16 = 0,
    LORA_KV_E4M3 = 1 /* float8_e4m3fn codes; a value is code * k_scale (v_scale) */
} lora_kv_type_t;

/*
 * A paged cache of keys and values: element (page, token, head, dim) of k is
 * k[page * page_stride + token * token_stride + head * head_stride + dim], v
 * alike (strides in elements, any order of page, token and head; dims are
 * contiguous).  Slot p * page_size + t names token t of page p.
 *   n_pages    >= 1
 *   page_size  tokens a page, a power of two up to LORA_MAX_PAGE_SIZE
 *   n_kv       key/value heads, >= 1
 *   head_dim   a multiple of 16 up to LORA_MAX_HEAD_DIM (lora_attend: 64 or 128)
 *   strides    multiples of 16 bytes; k and v 16-byte aligned
 *   scales     finite and > 0 (used with LORA_KV_E4M3 only)
 */
typedef struct {
    void *k, *v;
    int32_t n_pages, page_size, n_kv, head_dim;
    int64_t page_stride, token_stride, head_stride;
    int32_t type; /* lora_kv_type_t */
    float k_scale, v_scale;
} lora_kv_t;

/*
 * Where a step's tokens go.  Request i has ctx_lens[i] tokens in the cache and
 * brings new_lens[i] more (0 is allowed); its tokens are consecutive rows of the
 * step, requests in order.  With c = ctx_lens[i], m = new_lens[i], and
 * pages(n) = ceil(n / page_size):
 *   need_i = pages(c + m) - pages(c), e_i = sum of need_j over j < i
 *   request i is served when need_i = 0 or e_i + need_i <= n_free (so from the
 *   first request that does not fit on, none that needs a page is served)
 *   block_table[i][pages(c) + u] = free_pages[e_i + u], u < need_i, if served
 * Outputs (device):
 *   block_table  int32 [n_seq] rows of ld_table elements, table_width used;
 *                entries below pages(c) are read, new pages written
 *   q_offsets    int32 [n_seq + 1], first row of each request; the last entry
 *                is the number of tokens (saturating at INT32_MAX)
 *   kv_lens      int32 [n_seq], c + m where served, else c
 *   positions    int32 [T], c + (t - q_offsets[i])   (0 for padding rows)
 *   seq_ids      int32 [T], i                         (-1 for padding rows)
 *   slot_map     int64 [T], the token's cache slot    (-1 for padding rows and
 *                tokens of requests that were not served)
 *   taken        int32 [1], pages taken from the front of free_pages
 * T is the rows the step has room for; rows past the last token are padding.
 * Device errors: LORA_ERR_NO_PAGES (a request was not served for want of
 * pages), LORA_ERR_INVALID_ARG (a negative length, a request longer than its
 * table row - neither is served - or more tokens than T: the ones past T are
 * dropped, their requests' pages, kv_lens and q_offsets stand), LORA_ERR_SLOT_RANGE (a negative page id; its tokens get slot -1).
 * n_seq, n_free and T may be 0.  One launch.
 */
lora_status_t lora_kv_step(const int32_t *ctx_lens, const int32_t *new_lens, int32_t n_seq, int32_t page_size,
                           const int32_t *free_pages, int32_t n_free, int32_t *block_table, int64_t ld_table,
                           int32_t table_width, int32_t T, int32_t *q_offsets, int32_t *kv_lens, int32_t *positions,
                           int32_t *seq_ids, int64_t *slot_map, int32_t *taken, int32_t *err, lora_stream_t stream);

/* How a model's frequencies are scaled for contexts longer than it was trained on. */
typedef enum {
    LORA_ROPE_PLAIN = 0,
    LORA_ROPE_LINEAR = 1, /* f / factor */
    LORA_ROPE_NTK = 2,    /* theta * factor^(rot / (rot - 2)) in place of theta */
    LORA_ROPE_LLAMA3 = 3, /* f where it turns at least high_freq_factor times over `original` positions, f / factor
                             where it turns at most low_freq_factor times, linear in the turns between */
    LORA_ROPE_YARN = 4    /* a linear ramp over the pair index from f to f / factor, between the pairs that turn
                             beta_fast and beta_slow times over `original` positions (rounded outwards);
                             cos and sin times 0.1 ln(factor) + 1 */
} lora_rope_kind_t;

typedef struct {
    int32_t kind; /* lora_rope_kind_t */
    double factor, low_freq_factor, high_freq_factor, beta_fast, beta_slow, original;
} lora_rope_scaling_t;

/*
 * Rotary frequencies as phases (host): pair j of rot_dim / 2 turns f_j radians a
 * position, f_j = theta^(-2 j / rot_dim) before scaling (null: LORA_ROPE_PLAIN).
 * phases[j] = round(f_j / (2 pi) * 2^64) mod 2^64, so position * phases[j] mod
 * 2^64 is the angle in 2^-64 turns, exact for every position.  *mscale gets the
 * factor on cos and sin.  Errors: LORA_ERR_INVALID_ARG (null pointers, theta <= 1
 * or not finite, a bad kind, factor < 1 or not finite, factors out of order).
 * rot_dim: a multiple of 16 in [16, LORA_MAX_HEAD_DIM] (LORA_ERR_ALIGNMENT).
 */
lora_status_t lora_rope_phases(int32_t rot_dim, double theta, const lora_rope_scaling_t *scaling, uint64_t *phases,
                               float *mscale);

/*
 * Rotary embedding of q and k and the write of k and v into the cache.
 *   qkv        bf16 [T, ldqkv]: per row n_heads query heads, then n_kv key heads,
 *              then n_kv value heads of head_dim each (the packed projection's y)
 *   q_out      bf16 [T, ldq]: the rotated query heads; may be qkv itself with
 *              ldq = ldqkv (in place), else must not overlap it
 *   positions  int32 [T]
 *   slot_map   int64 [T]; -1: the token's k and v are not written (q is)
 * Of each query and key head the first rot_dim dims are rotated, the pairs
 * (j, j + rot_dim / 2), or (2 j, 2 j + 1) when interleaved:
 *   (a, b) -> mscale (a cos - b sin, b cos + a sin), angle positions[t] f_j,
 * in fp32, rounded once to bf16, or for LORA_KV_E4M3 divided by the scale in
 * fp32, clamped to +-448 and rounded once to e4m3 (NaN stays NaN).  Tokens
 * that share a slot race.  A slot >= n_pages * page_size or < -1 is reported as
 * LORA_ERR_SLOT_RANGE and not written.  Negative positions turn backwards.
 * phases: device uint64 [rot_dim / 2] of lora_rope_phases, 16-byte aligned.
 * Host checks: LORA_ERR_INVALID_ARG, LORA_ERR_ALIGNMENT as for lora_apply
 * (16-byte pointers, leading dimensions multiples of 8); rot_dim a multiple of
 * 16 in [16, head_dim]; n_heads >= 1.
 */
typedef struct {
    int32_t rot_dim, interleaved;
    float mscale;
    const uint64_t *phases;
} lora_rope_t;

lora_status_t lora_rope_append(const void *qkv, int64_t ldqkv, int32_t T, int32_t n_heads, const lora_rope_t *rope,
                               const int32_t *positions, const int64_t *slot_map, void *q_out, int64_t ldq,
                               const lora_kv_t *kv, int32_t *err, lora_stream_t stream);

/*
 * Attention of a step's tokens over the cache.  Request i owns rows
 * [q_offsets[i], q_offsets[i + 1]) of q, its last kv_lens[i] positions being in
 * the cache (the step's own tokens included): row t has position
 * p = kv_lens[i] - (q_offsets[i + 1] - t) and, for query head h (key head
 * h / (n_heads / n_kv)),
 *     s_j = scale * q . k_j                  (times k_scale for LORA_KV_E4M3)
 *     s_j = softcap * tanh(s_j / softcap)    if softcap > 0
 *     s_j = s_j + slopes[h] * (j - p)        if slopes
 *     out = sum_j softmax_j(s) v_j           over 0 <= j <= p, j > p - window if window > 0
 * softmax statistics and sums in fp32, one rounding to bf16.  A row that sees
 * no key (p < 0, a request without cached tokens) is 0, its lse -inf.  Rows
 * outside every request are not written.  Cache entries that no row of the
 * request's row tile sees are never used, whatever they hold; a NaN or
 * infinity in a value that some row of the tile sees can reach the tile's
 * other rows.
 *   q, out       bf16 [T, ld], head h in columns [h head_dim, (h + 1) head_dim)
 *   lse          fp32 [T][n_heads], ln sum_j exp(s_j); may be null
 *   q_offsets    int32 [n_seq + 1] non-decreasing from 0, at most T
 *   kv_lens      int32 [n_seq]
 *   block_table  int32 [n_seq] rows of ld_table elements, table_width used
 *   slopes       device fp32 [n_heads] (distance bias), or null
 *   max_q_hint   host-known upper bound on a request's rows (0: not known; the rows
 *                are taken as shared out evenly, T / n_seq rounded up).  It picks the
 *                path and the decode path's tile, no row depends on its being right
 *   ws           lora_attend_workspace_bytes() bytes, 16-byte aligned, zeroed once
 *                before the first call; every call leaves it as it found it (but
 *                zero it again after a call that reports LORA_ERR_TIMEOUT).
 *                Calls that may overlap need a workspace each
 * Limits (LORA_ERR_UNSUPPORTED): head_dim 64 or 128.  n_heads a multiple of
 * n_kv, n_seq <= LORA_MAX_SEQS, scale finite, softcap >= 0, window >= 0
 * (LORA_ERR_INVALID_ARG).  Device errors: LORA_ERR_INVALID_ARG (offsets out of
 * order or past T, kv_lens negative, beyond the table row or above
 * LORA_MAX_KV_LEN: that request is skipped), LORA_ERR_SLOT_RANGE (a page id outside
 * [0, n_pages): its keys and values read as zeros), LORA_ERR_TIMEOUT (a wait inside
 * the kernel gave up), LORA_ERR_UNSUPPORTED (decode path: more than 2^31 steps of 32 or
 * 64 keys over all requests, key heads and tiles of rows; nothing is written).
 */
typedef struct {
    int32_t n_heads;
    float scale, softcap;
    int32_t window;
    const float *slopes;
} lora_attention_t;

typedef enum {
    LORA_ATTEND_AUTO = 0,
    LORA_ATTEND_DECODE = 1, /* few rows a request: the cache's length is split over the GPU and joined */
    LORA_ATTEND_PROMPT = 2  /* many rows a request: row tiles on the tensor cores */
} lora_attend_path_t;

lora_status_t lora_attend_workspace_bytes(const lora_attention_t *att, const lora_kv_t *kv, size_t *bytes);

/* The path lora_attend takes for `requested`, this shape and n_seq requests of at most max_q_hint >= 1 rows (host
 * only; without a hint lora_attend asks for T / n_seq rounded up). */
lora_attend_path_t lora_attend_resolve_path(lora_attend_path_t requested, const lora_attention_t *att,
                                            const lora_kv_t *kv, int32_t n_seq, int32_t max_q_hint);

lora_status_t lora_attend(const void *q, int64_t ldq, void *out, int64_t ldo, float *lse, int32_t T, int32_t n_seq,
                          const int32_t *q_offsets, const int32_t *kv_lens, const int32_t *block_table,
                          int64_t ld_table, int32_t table_width, const lora_kv_t *kv, const lora_attention_t *att,
                          int32_t max_q_hint, lora_attend_path_t path, void *ws, size_t ws_bytes, int32_t *err,
                          lora_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_ATTENTION_H */

// extern "C" entry points of lora_sharing.h: argument checks and kernel dispatch.
#include "attention.cuh"

namespace lora {
size_t beam_select_workspace_bytes(int32_t n_req, int32_t beams, int32_t keep, int32_t vocab);
cudaError_t launch_beam_select(const void *logits, int64_t ld, bool fp32, int32_t n_req, int32_t beams, int32_t vocab,
                               int32_t keep, const float *scores, const int32_t *ended, int32_t eos, int32_t *parents,
                               int32_t *tokens, float *out_scores, int32_t *out_ended, void *ws, cudaStream_t stream);
cudaError_t launch_kv_fork(const int32_t *src, int64_t ld_src, int32_t src_width, const int32_t *lens, int32_t n_src,
                           const int32_t *parents, int32_t n_dst, int32_t shift, int32_t n_pages, const int32_t *held,
                           int32_t n_held, int32_t *dst, int64_t ld_dst, int32_t dst_width, int32_t *dst_lens,
                           int32_t *copies, int32_t *free_pages, int32_t *n_free, int32_t *err, cudaStream_t stream);
cudaError_t launch_kv_compact(const int32_t *src, int64_t ld_src, int32_t width, const int32_t *lens, int32_t n_seq,
                              int32_t shift, int32_t n_pages, const int32_t *held, int32_t n_held, int32_t *dst,
                              int64_t ld_dst, int32_t *dst_held, int32_t *moves, int32_t *n_moves, int32_t *free_pages,
                              int32_t *n_free, int32_t *err, cudaStream_t stream);
cudaError_t launch_kv_copy(const KvView *layers, int32_t n_layers, bool e4m3, const int32_t *copies, int32_t n_copies,
                           const int32_t *count, int32_t *err, cudaStream_t stream);
size_t shared_workspace_bytes(int32_t head_dim, int32_t n_heads, int32_t T, int32_t n_seq);
cudaError_t launch_attend_shared(const AttendArgs &a, bool e4m3, int32_t max_q, const lora_prefix_t &prefix, void *ws,
                                 cudaStream_t stream);
}  // namespace lora

using lora::aligned16;

namespace {

lora_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA; }

// Whether n rows of `width` int32, ld apart, and m of another table overlap in memory.
bool overlap(const int32_t *a, int64_t ld_a, int64_t n, int64_t width_a, const int32_t *b, int64_t ld_b, int64_t m,
             int64_t width_b) {
    if (n <= 0 || m <= 0 || width_a <= 0 || width_b <= 0) return false;
    return a < b + (m - 1) * ld_b + width_b && b < a + (n - 1) * ld_a + width_a;
}

lora_status_t check_pages(int32_t page_size, int32_t n_pages, const int32_t *held, int32_t n_held,
                          const int32_t *free_pages, const int32_t *n_free, int32_t *shift) {
    if (page_size < 1 || page_size > LORA_MAX_PAGE_SIZE || (page_size & (page_size - 1)) != 0)
        return LORA_ERR_INVALID_ARG;
    if (n_pages < 1 || n_held < 0 || (n_held > 0 && held == nullptr) || free_pages == nullptr || n_free == nullptr)
        return LORA_ERR_INVALID_ARG;
    if (n_pages > LORA_MAX_PAGES) return LORA_ERR_UNSUPPORTED;
    *shift = 0;
    while ((1 << *shift) < page_size) ++*shift;
    return LORA_OK;
}

}  // namespace

extern "C" {

lora_status_t lora_beam_select_workspace_bytes(int32_t n_req, int32_t beams, int32_t keep, int32_t vocab,
                                               size_t *bytes) {
    if (bytes == nullptr || n_req < 0 || n_req > LORA_MAX_SEQS || beams < 1 || beams > LORA_MAX_BEAMS || keep < 1 ||
        keep > LORA_MAX_BEAMS || vocab < 1 || vocab > LORA_MAX_VOCAB)
        return LORA_ERR_INVALID_ARG;
    *bytes = lora::beam_select_workspace_bytes(n_req, beams, keep, vocab);
    return LORA_OK;
}

lora_status_t lora_beam_select(const void *logits, int64_t ld, lora_logits_t type, int32_t n_req, int32_t beams,
                               int32_t vocab, int32_t keep, const float *scores, const int32_t *ended, int32_t eos,
                               int32_t *parents, int32_t *tokens, float *out_scores, int32_t *out_ended, void *ws,
                               size_t ws_bytes, lora_stream_t stream) {
    size_t need = 0;
    const lora_status_t st = lora_beam_select_workspace_bytes(n_req, beams, keep, vocab, &need);
    if (st != LORA_OK) return st;
    if (type != LORA_LOGITS_BF16 && type != LORA_LOGITS_FP32) return LORA_ERR_INVALID_ARG;
    if (ld < vocab || eos < -1 || eos >= vocab || (eos < 0 && ended != nullptr)) return LORA_ERR_INVALID_ARG;
    if (n_req > 0 && (logits == nullptr || scores == nullptr || parents == nullptr || tokens == nullptr ||
                      out_scores == nullptr || out_ended == nullptr))
        return LORA_ERR_INVALID_ARG;
    const bool fp32 = type == LORA_LOGITS_FP32;
    if (reinterpret_cast<uintptr_t>(logits) % (fp32 ? 4 : 2) != 0) return LORA_ERR_ALIGNMENT;
    if (ws == nullptr || ws_bytes < need) return LORA_ERR_WORKSPACE;
    if (!aligned16(ws)) return LORA_ERR_ALIGNMENT;
    if (n_req == 0) return LORA_OK;
    return from_cuda(lora::launch_beam_select(logits, ld, fp32, n_req, beams, vocab, keep, scores, ended, eos, parents,
                                              tokens, out_scores, out_ended, ws,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

lora_status_t lora_kv_fork(const int32_t *src_table, int64_t ld_src, int32_t src_width, const int32_t *src_lens,
                           int32_t n_src, const int32_t *parents, int32_t n_dst, int32_t page_size, int32_t n_pages,
                           const int32_t *held, int32_t n_held, int32_t *dst_table, int64_t ld_dst, int32_t dst_width,
                           int32_t *dst_lens, int32_t *copies, int32_t *free_pages, int32_t *n_free, int32_t *err,
                           lora_stream_t stream) {
    if (n_src < 0 || n_src > LORA_MAX_SEQS || n_dst < 0 || n_dst > LORA_MAX_SEQS || src_width < 0 || dst_width < 0 ||
        ld_src < src_width || ld_dst < dst_width)
        return LORA_ERR_INVALID_ARG;
    int32_t shift;
    const lora_status_t st = check_pages(page_size, n_pages, held, n_held, free_pages, n_free, &shift);
    if (st != LORA_OK) return st;
    if (n_src > 0 && (src_lens == nullptr || (src_width > 0 && src_table == nullptr))) return LORA_ERR_INVALID_ARG;
    if (n_dst > 0 && (parents == nullptr || dst_lens == nullptr || copies == nullptr ||
                      (dst_width > 0 && dst_table == nullptr)))
        return LORA_ERR_INVALID_ARG;
    if (overlap(src_table, ld_src, n_src, src_width, dst_table, ld_dst, n_dst, dst_width) ||
        overlap(src_lens, 1, n_src, 1, dst_lens, 1, n_dst, 1))
        return LORA_ERR_INVALID_ARG;
    return from_cuda(lora::launch_kv_fork(src_table, ld_src, src_width, src_lens, n_src, parents, n_dst, shift, n_pages,
                                          held, n_held, dst_table, ld_dst, dst_width, dst_lens, copies, free_pages,
                                          n_free, err, reinterpret_cast<cudaStream_t>(stream)));
}

lora_status_t lora_kv_compact(const int32_t *src_table, int64_t ld_src, int32_t width, const int32_t *lens,
                              int32_t n_seq, int32_t page_size, int32_t n_pages, const int32_t *held, int32_t n_held,
                              int32_t *dst_table, int64_t ld_dst, int32_t *dst_held, int32_t *moves, int32_t *n_moves,
                              int32_t *free_pages, int32_t *n_free, int32_t *err, lora_stream_t stream) {
    if (n_seq < 0 || n_seq > LORA_MAX_SEQS || width < 0 || ld_src < width || ld_dst < width) return LORA_ERR_INVALID_ARG;
    int32_t shift;
    const lora_status_t st = check_pages(page_size, n_pages, held, n_held, free_pages, n_free, &shift);
    if (st != LORA_OK) return st;
    if (n_seq > 0 && (lens == nullptr || (width > 0 && (src_table == nullptr || dst_table == nullptr))))
        return LORA_ERR_INVALID_ARG;
    if ((n_held > 0 && dst_held == nullptr) || (n_pages > 1 && moves == nullptr) || n_moves == nullptr)
        return LORA_ERR_INVALID_ARG;
    if (overlap(src_table, ld_src, n_seq, width, dst_table, ld_dst, n_seq, width)) return LORA_ERR_INVALID_ARG;
    return from_cuda(lora::launch_kv_compact(src_table, ld_src, width, lens, n_seq, shift, n_pages, held, n_held,
                                             dst_table, ld_dst, dst_held, moves, n_moves, free_pages, n_free, err,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

lora_status_t lora_kv_copy(const lora_kv_t *kvs, int32_t n_layers, const int32_t *copies, int32_t n_copies,
                           const int32_t *count, int32_t *err, lora_stream_t stream) {
    if (kvs == nullptr || n_layers < 1 || n_layers > LORA_MAX_KV_LAYERS || n_copies < 0) return LORA_ERR_INVALID_ARG;
    if (n_copies > 0 && copies == nullptr) return LORA_ERR_INVALID_ARG;
    lora::KvView views[LORA_MAX_KV_LAYERS];
    for (int32_t i = 0; i < n_layers; ++i) {
        const lora_status_t st = lora::check_kv(kvs + i, views + i);
        if (st != LORA_OK) return st;
        const lora_kv_t &a = kvs[0], &b = kvs[i];
        if (a.n_pages != b.n_pages || a.page_size != b.page_size || a.n_kv != b.n_kv || a.head_dim != b.head_dim ||
            a.page_stride != b.page_stride || a.token_stride != b.token_stride || a.head_stride != b.head_stride ||
            a.type != b.type)
            return LORA_ERR_INVALID_ARG;
    }
    if (n_copies == 0) return LORA_OK;
    return from_cuda(lora::launch_kv_copy(views, n_layers, kvs[0].type == LORA_KV_E4M3, copies, n_copies, count, err,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

lora_status_t lora_attend_shared_workspace_bytes(const lora_attention_t *att, const lora_kv_t *kv, int32_t T,
                                                 int32_t n_seq, size_t *bytes) {
    lora::KvView view;
    lora_status_t st;
    if (bytes == nullptr || T < 0 || n_seq < 0 || n_seq > LORA_MAX_SEQS) return LORA_ERR_INVALID_ARG;
    if ((st = lora::check_kv(kv, &view)) != LORA_OK) return st;
    if ((st = lora::check_attention(att, view)) != LORA_OK) return st;
    *bytes = lora::shared_workspace_bytes(view.head_dim, att->n_heads, T, n_seq);
    return LORA_OK;
}

lora_status_t lora_attend_shared(const void *q, int64_t ldq, void *out, int64_t ldo, float *lse, int32_t T,
                                 int32_t n_seq, const int32_t *q_offsets, const int32_t *kv_lens,
                                 const int32_t *block_table, int64_t ld_table, int32_t table_width,
                                 const lora_prefix_t *prefix, const lora_kv_t *kv, const lora_attention_t *att,
                                 int32_t max_q_hint, void *ws, size_t ws_bytes, int32_t *err, lora_stream_t stream) {
    lora::AttendArgs a;
    lora_status_t st;
    if ((st = lora::check_attend(q, ldq, out, ldo, lse, T, n_seq, q_offsets, kv_lens, block_table, ld_table, table_width,
                                 kv, att, err, &a)) != LORA_OK)
        return st;
    if (prefix == nullptr || prefix->n_groups < 0 || prefix->n_groups > LORA_MAX_SEQS) return LORA_ERR_INVALID_ARG;
    if (prefix->mode != LORA_SHARE_AUTO && prefix->mode != LORA_SHARE_ALWAYS) return LORA_ERR_INVALID_ARG;
    if (prefix->n_groups > 0 && (prefix->group_offsets == nullptr || prefix->prefix_lens == nullptr))
        return LORA_ERR_INVALID_ARG;
    if (ws == nullptr || ws_bytes < lora::shared_workspace_bytes(a.kv.head_dim, a.n_heads, T, n_seq))
        return LORA_ERR_WORKSPACE;
    if (!aligned16(ws)) return LORA_ERR_ALIGNMENT;
    if (T == 0 || n_seq == 0) return LORA_OK;
    return from_cuda(lora::launch_attend_shared(a, kv->type == LORA_KV_E4M3, lora::rows_hint(max_q_hint, T, n_seq),
                                                *prefix, ws, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

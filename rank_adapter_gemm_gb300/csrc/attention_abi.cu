// extern "C" entry points of lora_attention.h: argument checks, the rotary
// frequencies and kernel dispatch.
#include <algorithm>
#include <cmath>

#include "attention.cuh"

namespace lora {
cudaError_t launch_kv_step(const int32_t *ctx_lens, const int32_t *new_lens, int32_t n_seq, int32_t page_shift,
                           const int32_t *free_pages, int32_t n_free, int32_t *table, int64_t ld_table, int32_t width,
                           int32_t T, int32_t *q_offsets, int32_t *kv_lens, int32_t *positions, int32_t *seq_ids,
                           int64_t *slot_map, int32_t *taken, int32_t *err, cudaStream_t stream);
cudaError_t launch_rope_append(const uint16_t *qkv, int64_t ldqkv, int32_t T, int32_t n_heads, const lora_rope_t &rope,
                               const int32_t *positions, const int64_t *slots, uint16_t *q_out, int64_t ldq,
                               const KvView &kv, bool e4m3, int32_t *err, cudaStream_t stream);
size_t decode_workspace_bytes(int32_t head_dim);
cudaError_t launch_attend_decode(const AttendArgs &a, bool e4m3, int32_t max_q, void *ws, cudaStream_t stream);
cudaError_t launch_attend_prompt(const AttendArgs &a, bool e4m3, void *ws, cudaStream_t stream);
}  // namespace lora

using lora::aligned16;
using lora::check_attention;
using lora::check_kv;
using lora::check_rows;
using lora::KvView;

namespace {

lora_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA; }

}  // namespace

extern "C" {

lora_status_t lora_kv_step(const int32_t *ctx_lens, const int32_t *new_lens, int32_t n_seq, int32_t page_size,
                           const int32_t *free_pages, int32_t n_free, int32_t *block_table, int64_t ld_table,
                           int32_t table_width, int32_t T, int32_t *q_offsets, int32_t *kv_lens, int32_t *positions,
                           int32_t *seq_ids, int64_t *slot_map, int32_t *taken, int32_t *err, lora_stream_t stream) {
    if (n_seq < 0 || n_free < 0 || T < 0 || table_width < 0 || ld_table < table_width) return LORA_ERR_INVALID_ARG;
    if (page_size < 1 || page_size > LORA_MAX_PAGE_SIZE || (page_size & (page_size - 1)) != 0)
        return LORA_ERR_INVALID_ARG;
    if (q_offsets == nullptr || taken == nullptr) return LORA_ERR_INVALID_ARG;
    if (n_seq > 0 && (ctx_lens == nullptr || new_lens == nullptr || kv_lens == nullptr)) return LORA_ERR_INVALID_ARG;
    if (n_seq > 0 && table_width > 0 && block_table == nullptr) return LORA_ERR_INVALID_ARG;
    if (n_free > 0 && free_pages == nullptr) return LORA_ERR_INVALID_ARG;
    if (T > 0 && (positions == nullptr || seq_ids == nullptr || slot_map == nullptr)) return LORA_ERR_INVALID_ARG;
    int32_t shift = 0;
    while ((1 << shift) < page_size) ++shift;
    return from_cuda(lora::launch_kv_step(ctx_lens, new_lens, n_seq, shift, free_pages, n_free, block_table, ld_table,
                                          table_width, T, q_offsets, kv_lens, positions, seq_ids, slot_map, taken, err,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

lora_status_t lora_rope_phases(int32_t rot_dim, double theta, const lora_rope_scaling_t *scaling, uint64_t *phases,
                               float *mscale) {
    if (phases == nullptr || mscale == nullptr) return LORA_ERR_INVALID_ARG;
    if (rot_dim < 16 || rot_dim > LORA_MAX_HEAD_DIM || rot_dim % 16 != 0) return LORA_ERR_ALIGNMENT;
    if (!std::isfinite(theta) || theta <= 1.0) return LORA_ERR_INVALID_ARG;
    const double pi = std::acos(-1.0);
    const int32_t kind = scaling == nullptr ? LORA_ROPE_PLAIN : scaling->kind;
    if (kind < LORA_ROPE_PLAIN || kind > LORA_ROPE_YARN) return LORA_ERR_INVALID_ARG;
    const double factor = kind == LORA_ROPE_PLAIN ? 1.0 : scaling->factor;
    if (!std::isfinite(factor) || factor < 1.0) return LORA_ERR_INVALID_ARG;
    if (kind == LORA_ROPE_LLAMA3 || kind == LORA_ROPE_YARN) {
        const double lo = kind == LORA_ROPE_LLAMA3 ? scaling->low_freq_factor : scaling->beta_slow;
        const double hi = kind == LORA_ROPE_LLAMA3 ? scaling->high_freq_factor : scaling->beta_fast;
        if (!(lo > 0.0) || !(hi > lo) || !std::isfinite(hi)) return LORA_ERR_INVALID_ARG;
        if (!(scaling->original >= 1.0) || !std::isfinite(scaling->original)) return LORA_ERR_INVALID_ARG;
    }
    if (kind == LORA_ROPE_NTK) theta *= std::pow(factor, double(rot_dim) / (rot_dim - 2));
    // index of the pair that turns `turns` times over the original context
    const auto pair_of = [&](double turns) {
        return rot_dim * std::log(scaling->original / (turns * 2 * pi)) / (2 * std::log(theta));
    };
    double ramp_lo = 0.0, ramp_hi = 0.0;
    if (kind == LORA_ROPE_YARN) {
        ramp_lo = std::max(0.0, std::floor(pair_of(scaling->beta_fast)));
        ramp_hi = std::min(rot_dim - 1.0, std::ceil(pair_of(scaling->beta_slow)));
    }
    for (int32_t j = 0; j < rot_dim / 2; ++j) {
        double f = std::pow(theta, -2.0 * j / rot_dim);
        if (kind == LORA_ROPE_LINEAR) f /= factor;
        if (kind == LORA_ROPE_LLAMA3) {
            const double turns = scaling->original * f / (2 * pi);
            const double t = (turns - scaling->low_freq_factor) /
                             (scaling->high_freq_factor - scaling->low_freq_factor);
            const double keep = std::min(1.0, std::max(0.0, t));
            f = f * keep + f / factor * (1.0 - keep);
        }
        if (kind == LORA_ROPE_YARN) {
            const double r = std::min(1.0, std::max(0.0, (j - ramp_lo) / std::max(ramp_hi - ramp_lo, 1e-3)));
            f = f * (1.0 - r) + f / factor * r;
        }
        // f <= 1 radian, so the turn's fraction is below 1/2 and the product below 2^63
        phases[j] = static_cast<uint64_t>(std::nearbyint(std::ldexp(f / (2 * pi), 64)));
    }
    *mscale = kind == LORA_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return LORA_OK;
}

lora_status_t lora_rope_append(const void *qkv, int64_t ldqkv, int32_t T, int32_t n_heads, const lora_rope_t *rope,
                               const int32_t *positions, const int64_t *slot_map, void *q_out, int64_t ldq,
                               const lora_kv_t *kv, int32_t *err, lora_stream_t stream) {
    KvView view;
    lora_status_t st;
    if (T < 0 || n_heads < 1 || rope == nullptr || rope->phases == nullptr) return LORA_ERR_INVALID_ARG;
    if ((st = check_kv(kv, &view)) != LORA_OK) return st;
    const int64_t heads = int64_t(n_heads) + 2 * int64_t(view.n_kv);
    if (heads * view.head_dim > INT32_MAX) return LORA_ERR_INVALID_ARG;
    if ((st = check_rows(qkv, ldqkv, T, static_cast<int32_t>(heads * view.head_dim))) != LORA_OK) return st;
    if ((st = check_rows(q_out, ldq, T, n_heads * view.head_dim)) != LORA_OK) return st;
    if (rope->rot_dim < 16 || rope->rot_dim > view.head_dim || rope->rot_dim % 16 != 0 || !aligned16(rope->phases))
        return LORA_ERR_ALIGNMENT;
    if (T > 0 && (positions == nullptr || slot_map == nullptr)) return LORA_ERR_INVALID_ARG;
    if (T == 0) return LORA_OK;
    return from_cuda(lora::launch_rope_append(static_cast<const uint16_t *>(qkv), ldqkv, T, n_heads, *rope, positions,
                                              slot_map, static_cast<uint16_t *>(q_out), ldq, view,
                                              kv->type == LORA_KV_E4M3, err, reinterpret_cast<cudaStream_t>(stream)));
}

lora_status_t lora_attend_workspace_bytes(const lora_attention_t *att, const lora_kv_t *kv, size_t *bytes) {
    KvView view;
    lora_status_t st;
    if (bytes == nullptr) return LORA_ERR_INVALID_ARG;
    if ((st = check_kv(kv, &view)) != LORA_OK) return st;
    if ((st = check_attention(att, view)) != LORA_OK) return st;
    *bytes = lora::decode_workspace_bytes(view.head_dim);
    return LORA_OK;
}

// The decode path reads a request's cache once for every 32 of its rows, spread over
// the whole GPU; the prompt path gives 256 rows of a key head to one block, or with
// few such items up to 16 parts of their keys to a block each.  Its time does not grow
// with rows but steps with the waves of such blocks on the SMs (kSms, a GB300's: the choice
// is made without a device).  Measured a key: 16 rows of a key head on the decode path cost
// about 1/256 of a wave on the prompt path.  Both sides, us (decode / prompt, 32/8 heads of
// 128, graph replay): 64 requests of 100 to 8,000 tokens, 4 rows 86 / 114, 8 rows 113 / 115; 8
// requests of 4,096, 4 rows 38 / 38, 8 rows 47 / 38, 32 rows 104 / 54; one request of 16,384,
// 4 rows 29 / 37, 8 rows 41 / 38, 32 rows 64 / 38, 128 rows 171 / 55; one of 2,000, 4 rows
// 18 / 22, 16 rows 22 / 23; one of 131,071, 4 rows 99 / 115, 64 rows 597 / 145.
constexpr int64_t kSms = 152;

lora_attend_path_t lora_attend_resolve_path(lora_attend_path_t requested, const lora_attention_t *att,
                                            const lora_kv_t *kv, int32_t n_seq, int32_t max_q_hint) {
    if (requested != LORA_ATTEND_AUTO || att == nullptr || kv == nullptr || kv->n_kv < 1) return requested;
    const int64_t rows = int64_t(max_q_hint) * (att->n_heads / kv->n_kv), pairs = int64_t(n_seq) * kv->n_kv;
    const int64_t half_tiles = rows <= 16 ? 1 : 2 * ((rows + 31) / 32);
    const int64_t items = pairs * ((rows + 255) / 256), waves = (items + kSms - 1) / kSms;
    const int64_t parts = std::min<int64_t>(16, std::max<int64_t>(1, kSms / std::max<int64_t>(1, items)));
    return pairs * half_tiles * parts < 256 * waves ? LORA_ATTEND_DECODE : LORA_ATTEND_PROMPT;
}

lora_status_t lora_attend(const void *q, int64_t ldq, void *out, int64_t ldo, float *lse, int32_t T, int32_t n_seq,
                          const int32_t *q_offsets, const int32_t *kv_lens, const int32_t *block_table,
                          int64_t ld_table, int32_t table_width, const lora_kv_t *kv, const lora_attention_t *att,
                          int32_t max_q_hint, lora_attend_path_t path, void *ws, size_t ws_bytes, int32_t *err,
                          lora_stream_t stream) {
    lora::AttendArgs a;
    lora_status_t st;
    if (path < LORA_ATTEND_AUTO || path > LORA_ATTEND_PROMPT) return LORA_ERR_INVALID_ARG;
    if ((st = lora::check_attend(q, ldq, out, ldo, lse, T, n_seq, q_offsets, kv_lens, block_table, ld_table, table_width,
                                 kv, att, err, &a)) != LORA_OK)
        return st;
    size_t need = 0;
    if ((st = lora_attend_workspace_bytes(att, kv, &need)) != LORA_OK) return st;
    if (ws == nullptr || ws_bytes < need) return LORA_ERR_WORKSPACE;
    if (!aligned16(ws)) return LORA_ERR_ALIGNMENT;
    if (T == 0 || n_seq == 0) return LORA_OK;
    max_q_hint = lora::rows_hint(max_q_hint, T, n_seq);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool e4m3 = kv->type == LORA_KV_E4M3;
    if (lora_attend_resolve_path(path, att, kv, n_seq, max_q_hint) == LORA_ATTEND_DECODE)
        return from_cuda(lora::launch_attend_decode(a, e4m3, max_q_hint, ws, s));
    return from_cuda(lora::launch_attend_prompt(a, e4m3, ws, s));
}

}  // extern "C"

// Structures and host checks shared by the attention-side kernels
// (lora_attention.h, lora_sharing.h) and their C entry points.
#pragma once

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "../../include/lora_sharing.h"
#include "checks.cuh"

namespace lora {

// The paged cache, passed by value to kernels.  Strides in bytes.
struct KvView {
    unsigned char *k, *v;
    int64_t page_b, token_b, head_b;
    int32_t n_pages, page_shift, page_mask, n_kv, head_dim;
    float k_scale, v_scale;
};

// One attention call, passed by value to kernels.
struct AttendArgs {
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    int64_t ldq, ldo, ld_table;
    const int32_t *q_offsets, *kv_lens, *table;
    const float *slopes;
    int32_t *err;
    KvView kv;
    int32_t T, n_seq, width, n_heads, group, window;
    float scale, softcap, inv_softcap;  // inv_softcap: 0 without a cap
};

// Rows [q0, q0 + n) of request i, its last n of len positions; not ok (and
// n = 0) where the offsets or the length do not fit the arguments.
struct RequestRows {
    int32_t q0, n, len;
    bool ok;
};

__device__ __forceinline__ RequestRows check_request(const AttendArgs &a, int32_t q0, int32_t q1, int32_t len) {
    const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.T && len >= 0 && len <= LORA_MAX_KV_LEN &&
                    len <= (int64_t(a.width) << a.kv.page_shift);
    return {q0, ok ? q1 - q0 : 0, ok ? len : 0, ok};
}

__device__ __forceinline__ RequestRows load_rows(const AttendArgs &a, int32_t i) {
    return check_request(a, a.q_offsets[i], a.q_offsets[i + 1], a.kv_lens[i]);
}

// Past the first-level cache, for kernels that do not begin with a wait.
__device__ __forceinline__ RequestRows load_rows_cg(const AttendArgs &a, int32_t i) {
    return check_request(a, __ldcg(a.q_offsets + i), __ldcg(a.q_offsets + i + 1), __ldcg(a.kv_lens + i));
}

// The kernels of this file's users are launched as programmatic dependents of the
// kernel before them on the stream, which hides the launch's latency.  Each first
// waits until that kernel has finished and its writes are visible, so it may read
// and write what the kernel before it wrote (through coherent loads: the read-only
// path is for data that no one writes while a kernel's blocks are there); only then
// does it let its own dependent's blocks start.
__device__ __forceinline__ void wait_for_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The current device's SM count, after raising `kernel`'s shared memory limit to
// smem there: both looked up once a device (`seen`: one word a kernel, a bit a device).
template <class K>
cudaError_t prepare_kernel(K kernel, int smem, std::atomic<uint64_t> &seen, int *sms) {
    static std::atomic<int> counts[64];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const bool known = device < 64 && ((seen.load(std::memory_order_acquire) >> device) & 1);
    if (known) {
        *sms = counts[device].load(std::memory_order_relaxed);
        return cudaSuccess;
    }
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, device);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && device < 64) {
        counts[device].store(*sms, std::memory_order_relaxed);
        seen.fetch_or(uint64_t(1) << device, std::memory_order_release);
    }
    return e;
}

template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
                             A... args) {
    cudaLaunchAttribute attr[1] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

inline lora_status_t check_kv(const lora_kv_t *kv, KvView *out) {
    if (kv == nullptr || kv->k == nullptr || kv->v == nullptr) return LORA_ERR_INVALID_ARG;
    if (kv->n_pages < 1 || kv->n_kv < 1 || kv->type < LORA_KV_BF16 || kv->type > LORA_KV_E4M3)
        return LORA_ERR_INVALID_ARG;
    if (kv->page_size < 1 || kv->page_size > LORA_MAX_PAGE_SIZE || (kv->page_size & (kv->page_size - 1)) != 0)
        return LORA_ERR_INVALID_ARG;
    if (kv->head_dim < 16 || kv->head_dim > LORA_MAX_HEAD_DIM) return LORA_ERR_INVALID_ARG;
    if (kv->page_stride < 0 || kv->token_stride < 0 || kv->head_stride < 0) return LORA_ERR_INVALID_ARG;
    const int32_t size = kv->type == LORA_KV_E4M3 ? 1 : 2, per16 = 16 / size;
    if (kv->head_dim % 16 != 0 || !aligned16(kv->k) || !aligned16(kv->v)) return LORA_ERR_ALIGNMENT;
    if (kv->page_stride % per16 != 0 || kv->token_stride % per16 != 0 || kv->head_stride % per16 != 0)
        return LORA_ERR_ALIGNMENT;
    if (kv->type == LORA_KV_E4M3 && !(kv->k_scale > 0.0f && std::isfinite(kv->k_scale) && kv->v_scale > 0.0f &&
                                      std::isfinite(kv->v_scale)))
        return LORA_ERR_INVALID_ARG;
    out->k = static_cast<unsigned char *>(kv->k);
    out->v = static_cast<unsigned char *>(kv->v);
    out->page_b = kv->page_stride * size;
    out->token_b = kv->token_stride * size;
    out->head_b = kv->head_stride * size;
    out->n_pages = kv->n_pages;
    out->page_mask = kv->page_size - 1;
    out->page_shift = 0;
    while ((1 << out->page_shift) < kv->page_size) ++out->page_shift;
    out->n_kv = kv->n_kv;
    out->head_dim = kv->head_dim;
    out->k_scale = kv->type == LORA_KV_E4M3 ? kv->k_scale : 1.0f;
    out->v_scale = kv->type == LORA_KV_E4M3 ? kv->v_scale : 1.0f;
    return LORA_OK;
}

inline lora_status_t check_attention(const lora_attention_t *att, const KvView &kv) {
    if (att == nullptr || att->n_heads < 1 || att->n_heads % kv.n_kv != 0) return LORA_ERR_INVALID_ARG;
    if (!std::isfinite(att->scale) || !(att->softcap >= 0.0f) || !std::isfinite(att->softcap) || att->window < 0)
        return LORA_ERR_INVALID_ARG;
    if (kv.head_dim != 64 && kv.head_dim != 128) return LORA_ERR_UNSUPPORTED;
    return LORA_OK;
}

// The checks of an attention call, in lora_attend's order, and its arguments for the kernels.
inline lora_status_t check_attend(const void *q, int64_t ldq, void *out, int64_t ldo, float *lse, int32_t T,
                                  int32_t n_seq, const int32_t *q_offsets, const int32_t *kv_lens,
                                  const int32_t *block_table, int64_t ld_table, int32_t table_width,
                                  const lora_kv_t *kv, const lora_attention_t *att, int32_t *err, AttendArgs *a) {
    KvView view;
    lora_status_t st;
    if (T < 0 || n_seq < 0 || n_seq > LORA_MAX_SEQS || table_width < 0 || ld_table < table_width)
        return LORA_ERR_INVALID_ARG;
    if ((st = check_kv(kv, &view)) != LORA_OK) return st;
    if ((st = check_attention(att, view)) != LORA_OK) return st;
    if (int64_t(att->n_heads) * view.head_dim > INT32_MAX) return LORA_ERR_INVALID_ARG;
    if ((st = check_rows(q, ldq, T, att->n_heads * view.head_dim)) != LORA_OK) return st;
    if ((st = check_rows(out, ldo, T, att->n_heads * view.head_dim)) != LORA_OK) return st;
    if (q_offsets == nullptr || (n_seq > 0 && kv_lens == nullptr)) return LORA_ERR_INVALID_ARG;
    if (n_seq > 0 && table_width > 0 && block_table == nullptr) return LORA_ERR_INVALID_ARG;
    // a cap from 1e30 on changes no score below 1e25 by an fp32 rounding: none
    const float cap = att->softcap < 1e30f ? att->softcap : 0.0f;
    *a = AttendArgs{static_cast<const uint16_t *>(q), static_cast<uint16_t *>(out), lse, ldq, ldo, ld_table, q_offsets,
                    kv_lens, block_table, att->slopes, err, view, T, n_seq, table_width, att->n_heads,
                    att->n_heads / view.n_kv, att->window, att->scale, cap,
                    cap > 0.0f ? std::min(1.0f / cap, FLT_MAX) : 0.0f};
    return LORA_OK;
}

// A bound on a request's rows: without a hint T rows are taken as shared out evenly.
inline int32_t rows_hint(int32_t hint, int32_t T, int32_t n_seq) {
    return std::min(hint <= 0 ? (T - 1) / n_seq + 1 : hint, T);
}

}  // namespace lora

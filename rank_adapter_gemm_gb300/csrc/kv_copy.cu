// Copies of pages' data in all layers (lora_kv_copy).
//
// Every byte is read and written once, so HBM bounds it.  A unit is k or v of one page in
// one layer; its 16-byte pieces go to the threads of one block in the order in which
// they lie in memory (tokens or heads innermost, by their strides), four in flight a
// thread, and the grid walks the units of all layers.
#include <algorithm>

#include "attention.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256, kEach = 4;

struct CopyArgs {
    unsigned char *base[2 * LORA_MAX_KV_LAYERS];  // k and v of each layer
    const int32_t *copies, *count;
    int32_t *err;
    int64_t page_b, outer_b, inner_b;  // bytes; inner: the smaller stride of token and head
    int32_t n_copies, n_bases, n_pages, page_size, n_kv, pieces, token_inner;
};

__global__ void __launch_bounds__(kThreads) kv_copy_kernel(const __grid_constant__ CopyArgs a, int32_t slices) {
    wait_for_previous();
    int32_t n = a.n_copies;
    if (a.count != nullptr) {
        n = a.count[0];
        if (n < 0 || n > a.n_copies) {
            if (blockIdx.x == 0 && threadIdx.x == 0) report_error(a.err, LORA_ERR_INVALID_ARG);
            n = min(max(n, 0), a.n_copies);
        }
    }
    const int64_t units = int64_t(n) * a.n_bases * slices;
    for (int64_t x = blockIdx.x; x < units; x += gridDim.x) {
        const int32_t slice = static_cast<int32_t>(x % slices);
        const int64_t y = x / slices;
        const int32_t b = static_cast<int32_t>(y % a.n_bases), job = static_cast<int32_t>(y / a.n_bases);
        const int32_t s = a.copies[3 * int64_t(job)], d = a.copies[3 * int64_t(job) + 1], m = a.copies[3 * int64_t(job) + 2];
        const bool range = s >= -1 && s < a.n_pages && d >= -1 && d < a.n_pages, nothing = s == -1 || d == -1;
        if (!range || (!nothing && (m < 0 || m > a.page_size))) {
            if (threadIdx.x == 0) report_error(a.err, range ? LORA_ERR_INVALID_ARG : LORA_ERR_SLOT_RANGE);
            continue;
        }
        if (nothing || s == d) continue;
        const unsigned char *from = a.base[b] + s * a.page_b;
        unsigned char *to = a.base[b] + d * a.page_b;
        const uint32_t inner = static_cast<uint32_t>(a.token_inner ? m : a.n_kv) * a.pieces;
        const int64_t all = int64_t(m) * a.n_kv * a.pieces;
        for (int64_t p0 = int64_t(slice) * kThreads * kEach; p0 < all; p0 += int64_t(slices) * kThreads * kEach) {
            int64_t at[kEach];
            uint4 v[kEach];
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int64_t p = p0 + e * kThreads + threadIdx.x;
                at[e] = -1;
                if (p < all) {
                    const uint32_t o = static_cast<uint32_t>(p / inner), r = static_cast<uint32_t>(p % inner);
                    at[e] = o * a.outer_b + (r / a.pieces) * a.inner_b + (r % a.pieces) * 16;
                    v[e] = ldg_cg(from + at[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < kEach; ++e)
                if (at[e] >= 0) stg_u4(to + at[e], v[e]);
        }
    }
}

}  // namespace

cudaError_t launch_kv_copy(const KvView *layers, int32_t n_layers, bool e4m3, const int32_t *copies, int32_t n_copies,
                           const int32_t *count, int32_t *err, cudaStream_t stream) {
    const KvView &v = layers[0];
    CopyArgs a;
    for (int32_t i = 0; i < n_layers; ++i) {
        a.base[2 * i] = layers[i].k;
        a.base[2 * i + 1] = layers[i].v;
    }
    a.copies = copies;
    a.count = count;
    a.err = err;
    a.page_b = v.page_b;
    a.token_inner = v.token_b <= v.head_b;
    a.inner_b = a.token_inner ? v.token_b : v.head_b;
    a.outer_b = a.token_inner ? v.head_b : v.token_b;
    a.n_copies = n_copies;
    a.n_bases = 2 * n_layers;
    a.n_pages = v.n_pages;
    a.page_size = v.page_mask + 1;
    a.n_kv = v.n_kv;
    a.pieces = v.head_dim * (e4m3 ? 1 : 2) / 16;
    static std::atomic<uint64_t> seen{0};
    int sms = 0;
    const cudaError_t e = prepare_kernel(kv_copy_kernel, 0, seen, &sms);
    if (e != cudaSuccess) return e;
    const int64_t most = int64_t(a.page_size) * a.n_kv * a.pieces, units = int64_t(n_copies) * a.n_bases;
    const int64_t want = (most + kThreads * kEach - 1) / (kThreads * kEach), blocks = int64_t(sms) * 8;
    const int64_t slices = std::max<int64_t>(1, std::min<int64_t>(want, blocks / units));
    return launch_dependent(kv_copy_kernel, static_cast<unsigned>(std::min(units * slices, blocks)), kThreads, 0, stream,
                            a, static_cast<int32_t>(slices));
}

}  // namespace lora

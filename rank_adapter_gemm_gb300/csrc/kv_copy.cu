// Copies of pages' data in all layers (lora_kv_copy).
//
// Every byte is read and written once, so HBM bounds it.  A unit is k or v of one page in
// one layer (or, where there are few, a slice of its heads or tokens); its 16-byte pieces go
// to the threads of one block in the order in which they lie in memory (tokens or heads
// innermost, by their strides), four in flight a thread, and the grid walks the units of all
// layers.  A unit's start is a chain of two loads (its row of the list, its data), so blocks
// are many, and each loads the next unit's row ahead.
//
// Measured, graph replay: 91 part pages of 16 tokens (8 heads of 128, bf16, 2 KB runs) in 32 layers,
// 212 MB read and written, 37.9 us, 5.6 TB/s (a plain copy: 6.8); one of them in 4 layers 2.2 us (5.4 a
// call through the Python binding).
// 4 blocks an SM 37.9, 6 39.3, 8 40.3; 8 pieces in flight in a warp's own unit 48.8.
#include <algorithm>

#include "attention.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256, kEach = 4, kBlocks = 4;  // blocks an SM

struct CopyArgs {
    unsigned char *base[2 * LORA_MAX_KV_LAYERS];  // k and v of each layer
    const int32_t *copies, *count;
    int32_t *err;
    int64_t page_b, outer_b, inner_b;  // bytes; inner: the smaller stride of token and head
    int32_t n_copies, n_bases, n_pages, page_size, n_kv, pieces, token_inner;
};

__global__ void __launch_bounds__(kThreads, kBlocks)
kv_copy_kernel(const __grid_constant__ CopyArgs a, int32_t slices) {
    wait_for_previous();
    int32_t n = a.n_copies;
    if (a.count != nullptr) {
        n = a.count[0];
        if (n < 0 || n > a.n_copies) {
            if (blockIdx.x == 0 && threadIdx.x == 0) report_error(a.err, LORA_ERR_INVALID_ARG);
            n = min(max(n, 0), a.n_copies);
        }
    }
    // this block's first unit; from one to the next: whole jobs, and units within a job
    const int32_t per_job = a.n_bases * slices;
    int32_t job = blockIdx.x / per_job, unit = blockIdx.x % per_job;
    const int32_t job_step = gridDim.x / per_job, unit_step = gridDim.x % per_job;
    int32_t s = -1, d = -1, m = 0;
    const auto look_up = [&]() {
        if (job < n) {
            s = a.copies[3 * int64_t(job)];
            d = a.copies[3 * int64_t(job) + 1];
            m = a.copies[3 * int64_t(job) + 2];
        }
    };
    look_up();
    while (job < n) {
        const int32_t from_page = s, to_page = d, tokens = m, now = unit;
        job += job_step;
        unit += unit_step;
        if (unit >= per_job) unit -= per_job, ++job;
        look_up();
        const bool range = from_page >= -1 && from_page < a.n_pages && to_page >= -1 && to_page < a.n_pages;
        const bool nothing = from_page == -1 || to_page == -1;
        if (!range || (!nothing && (tokens < 0 || tokens > a.page_size))) {
            if (threadIdx.x == 0) report_error(a.err, range ? LORA_ERR_INVALID_ARG : LORA_ERR_SLOT_RANGE);
            continue;
        }
        if (nothing || from_page == to_page) continue;
        const int32_t b = now / slices, slice = now - b * slices;
        const unsigned char *from = a.base[b] + from_page * a.page_b;
        unsigned char *to = a.base[b] + to_page * a.page_b;
        // the outer rows of this slice (heads or tokens), and the pieces of each
        const int32_t outer = a.token_inner ? a.n_kv : tokens, inner = (a.token_inner ? tokens : a.n_kv) * a.pieces;
        const int32_t o1 = static_cast<int32_t>(int64_t(outer) * (slice + 1) / slices);
        int32_t o = static_cast<int32_t>(int64_t(outer) * slice / slices);
        if (inner == 0 || o >= o1) continue;
        const bool flat = a.inner_b == a.pieces * 16;  // a row's pieces lie in one run
        // this thread's piece: outer row, piece of it
        int32_t p = threadIdx.x;
        if (p >= inner) o += p / inner, p %= inner;
        const int32_t o_step = kThreads / inner, p_step = kThreads % inner;
        while (o < o1) {
            int64_t at[kEach];
            uint4 v[kEach];
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                at[e] = -1;
                if (o < o1) {
                    at[e] = o * a.outer_b + (flat ? int64_t(p) * 16 : p / a.pieces * a.inner_b + p % a.pieces * 16);
                    v[e] = ldg_cg(from + at[e]);
                }
                o += o_step;
                p += p_step;
                if (p >= inner) p -= inner, ++o;
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
    const int64_t rows = a.token_inner ? a.n_kv : a.page_size, most = int64_t(a.page_size) * a.n_kv * a.pieces;
    const int64_t blocks = int64_t(sms) * kBlocks, units = int64_t(n_copies) * a.n_bases;
    // slices where units alone do not fill the SMs, of no less than a block's pieces in flight
    const int64_t want = std::min(rows, (most + kThreads * kEach - 1) / (kThreads * kEach));
    const int64_t slices = std::max<int64_t>(1, std::min(want, blocks / units));
    return launch_dependent(kv_copy_kernel, static_cast<unsigned>(std::min(units * slices, blocks)), kThreads, 0, stream,
                            a, static_cast<int32_t>(slices));
}

}  // namespace lora

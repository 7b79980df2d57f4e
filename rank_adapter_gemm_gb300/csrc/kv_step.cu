// Block tables, slot map and positions of a step (lora_kv_step).
//
// Two prefix sums over the requests place everything: the new tokens before
// request i give its first row, the new pages before it give its pages in the
// free list.  The tokens then need no further communication: token t finds its
// request by a binary search in the row offsets, and its page either stands in
// the table already (position below the cached pages) or is
// free_pages[e_i + position / page_size - pages(c_i)]; the token at a page's
// first position writes that page's table entry, so no thread reads an entry
// that this launch writes.
//
// The work is a few bytes a token and a request, so the launch's latency bounds
// it at every size; one launch therefore, with no second pass that waits for
// the scan: every block repeats the scan over the lengths (8 bytes a request,
// from L2) and writes the tokens of its own window.
#include "attention.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 4;                  // requests a thread and scan chunk
constexpr int kChunk = kThreads * kPerThread;  // requests a scan chunk
constexpr int kWindow = 1024;                  // tokens a block

// Running sums over requests: tokens and pages.
struct Sums {
    int64_t tokens, pages;
};

__device__ __forceinline__ Sums shfl_up(Sums v, int o) {
    return {__shfl_up_sync(0xffffffffu, v.tokens, o), __shfl_up_sync(0xffffffffu, v.pages, o)};
}

// One request's lengths, checked: a negative length or a request longer than
// its table row brings no pages and is not served.
struct Request {
    int32_t ctx, fresh;
    int64_t need;
    bool ok;
};

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int32_t shift) {
    return (tokens + (int64_t(1) << shift) - 1) >> shift;
}

__device__ __forceinline__ Request load_request(const int32_t *ctx_lens, const int32_t *new_lens, int32_t i, int32_t n,
                                                int32_t shift, int32_t width) {
    Request r{0, 0, 0, true};
    if (i >= n) return r;
    const int32_t c = ctx_lens[i], m = new_lens[i];
    r.ok = c >= 0 && m >= 0 && pages_of(int64_t(c) + m, shift) <= width;
    r.ctx = max(c, 0);
    r.fresh = max(m, 0);
    r.need = r.ok ? pages_of(int64_t(c) + m, shift) - pages_of(c, shift) : 0;
    return r;
}

__global__ void __launch_bounds__(kThreads)
kv_step_kernel(const int32_t *ctx_lens, const int32_t *new_lens, int32_t n, int32_t shift,
               const int32_t *free_pages, int32_t n_free, int32_t *table, int64_t ld_table, int32_t width,
               int32_t T, int32_t *q_offsets, int32_t *kv_lens, int32_t *positions, int32_t *seq_ids, int64_t *slot_map,
               int32_t *taken, int32_t *err) {
    __shared__ int64_t s_row[kChunk + 1];  // first row of the chunk's requests, and of the next chunk
    __shared__ int64_t s_page[kChunk];     // pages before them; -1: not served
    __shared__ int32_t s_ctx[kChunk];
    __shared__ Sums s_warp[kThreads / 32];
    __shared__ unsigned long long s_taken;
    wait_for_previous();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t w0 = int64_t(blockIdx.x) * kWindow, w1 = min(w0 + kWindow, int64_t(T));
    if (tid == 0) s_taken = 0;
    Sums run{0, 0};
    for (int32_t base = 0; base < n; base += kChunk) {
        Request r[kPerThread];
        Sums mine{0, 0};
#pragma unroll
        for (int e = 0; e < kPerThread; ++e) {
            r[e] = load_request(ctx_lens, new_lens, base + tid * kPerThread + e, n, shift, width);
            mine.tokens += r[e].fresh;
            mine.pages += r[e].need;
        }
        Sums incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Sums u = shfl_up(incl, o);
            if (lane >= o) {
                incl.tokens += u.tokens;
                incl.pages += u.pages;
            }
        }
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        Sums at{run.tokens + incl.tokens - mine.tokens, run.pages + incl.pages - mine.pages};
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const Sums v = s_warp[w];
            if (w < warp) {
                at.tokens += v.tokens;
                at.pages += v.pages;
            }
            run.tokens += v.tokens;
            run.pages += v.pages;
        }
        // the requests of this chunk: block b writes the outputs of every gridDim-th chunk
        const bool writer = (base / kChunk) % gridDim.x == blockIdx.x;
#pragma unroll
        for (int e = 0; e < kPerThread; ++e) {
            const int32_t l = tid * kPerThread + e, i = base + l;
            const bool fits = r[e].need == 0 || at.pages + r[e].need <= n_free, served = r[e].ok && fits;
            s_row[l] = at.tokens;
            s_page[l] = served ? at.pages : -1;
            s_ctx[l] = r[e].ctx;
            if (i < n && writer) {
                q_offsets[i] = static_cast<int32_t>(min(at.tokens, int64_t(INT32_MAX)));
                kv_lens[i] = served ? r[e].ctx + r[e].fresh : r[e].ctx;
                if (!r[e].ok) report_error(err, LORA_ERR_INVALID_ARG);
                else if (!fits) report_error(err, LORA_ERR_NO_PAGES);
            }
            // served requests take a prefix of the free list: the last one's end is what is taken
            if (blockIdx.x == 0 && served && r[e].need > 0)
                atomicMax(&s_taken, static_cast<unsigned long long>(at.pages + r[e].need));
            at.tokens += r[e].fresh;
            at.pages += r[e].need;
        }
        if (tid == kThreads - 1) s_row[kChunk] = at.tokens;
        __syncthreads();
        // this window's tokens among the chunk's
        const int64_t t0 = max(w0, s_row[0]), t1 = min(w1, s_row[kChunk]);
        for (int64_t t = t0 + tid; t < t1; t += kThreads) {
            int lo = 0, hi = kChunk - 1;  // the last request that starts at or before t
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_row[mid] <= t) lo = mid;
                else hi = mid - 1;
            }
            const int32_t i = base + lo;
            const int64_t pos = s_ctx[lo] + (t - s_row[lo]);
            int64_t slot = -1;
            if (s_page[lo] >= 0) {
                const int64_t have = pages_of(s_ctx[lo], shift), p = pos >> shift;
                int32_t page;
                if (p < have) {
                    page = table[i * ld_table + p];
                } else {
                    page = free_pages[s_page[lo] + p - have];
                    if ((pos & ((int64_t(1) << shift) - 1)) == 0) table[i * ld_table + p] = page;
                }
                if (page < 0) report_error(err, LORA_ERR_SLOT_RANGE);
                else slot = (int64_t(page) << shift) + (pos & ((int64_t(1) << shift) - 1));
            }
            positions[t] = static_cast<int32_t>(min(pos, int64_t(INT32_MAX)));
            seq_ids[t] = i;
            slot_map[t] = slot;
        }
        __syncthreads();
    }
    for (int64_t t = max(w0, run.tokens) + tid; t < w1; t += kThreads) {
        positions[t] = 0;
        seq_ids[t] = -1;
        slot_map[t] = -1;
    }
    if (blockIdx.x == 0) {
        __syncthreads();
        if (tid == 0) {
            q_offsets[n] = static_cast<int32_t>(min(run.tokens, int64_t(INT32_MAX)));
            taken[0] = static_cast<int32_t>(s_taken);
            if (run.tokens > T) report_error(err, LORA_ERR_INVALID_ARG);
        }
    }
}

}  // namespace

cudaError_t launch_kv_step(const int32_t *ctx_lens, const int32_t *new_lens, int32_t n_seq, int32_t page_shift,
                           const int32_t *free_pages, int32_t n_free, int32_t *table, int64_t ld_table, int32_t width,
                           int32_t T, int32_t *q_offsets, int32_t *kv_lens, int32_t *positions, int32_t *seq_ids,
                           int64_t *slot_map, int32_t *taken, int32_t *err, cudaStream_t stream) {
    const int32_t grid = T > kWindow ? (T - 1) / kWindow + 1 : 1;
    return launch_dependent(kv_step_kernel, grid, kThreads, 0, stream, ctx_lens, new_lens, n_seq, page_shift,
                            free_pages, n_free, table, ld_table, width, T, q_offsets, kv_lens, positions, seq_ids,
                            slot_map, taken, err);
}

}  // namespace lora

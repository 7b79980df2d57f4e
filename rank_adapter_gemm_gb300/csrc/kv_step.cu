// Block tables, slot map and positions of a step (lora_kv_step).
//
// Two prefix sums over the requests place everything: the new tokens before
// request i give its first row, the new pages before it give its pages in the
// free list.  The tokens then need no further communication: token t finds its
// request by a binary search in the row offsets, and its page either stands in
// the table already (position below the cached pages) or is
// free_pages[e_i + position / page_size - pages(c_i)]; the token at a page's
// first position writes that page's table entry, so no thread reads an entry
// that this launch writes.  Entries of pages that begin past the step's last row, which
// have no such token, are written with their request's outputs.
//
// The work is a few bytes a token and a request, so chains of dependent loads
// bound it at every size; one launch therefore, with no second pass that waits
// for the scan: every block repeats the scan over the lengths (8 bytes a request,
// from L2) and writes the tokens of its own window.  Measured, graph replay: 32
// requests of one token 3.0 us, of which the launch is 2; 1,024 requests of 56,780
// tokens 3.5 us (windows of 256 tokens 3.8, of 1,024 4.2); one of 131,072 tokens 3.8
// (6.2, 3.6); 4,096 of one token 8.8.
#include "attention.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 4;                  // requests a thread and scan chunk
constexpr int kChunk = kThreads * kPerThread;  // requests a scan chunk
constexpr int kWindow = 512;                   // tokens a block
constexpr int kEach = kWindow / kThreads;      // tokens a thread

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

__device__ __forceinline__ Request make_request(int32_t c, int32_t m, int32_t shift, int32_t width) {
    Request r;
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
        // all loads first; requests past the last are empty
        int32_t c[kPerThread], m[kPerThread];
#pragma unroll
        for (int e = 0; e < kPerThread; ++e) {
            const int32_t i = min(base + tid * kPerThread + e, n - 1);
            c[e] = ctx_lens[i];
            m[e] = new_lens[i];
        }
        Request r[kPerThread];
        Sums mine{0, 0};
#pragma unroll
        for (int e = 0; e < kPerThread; ++e) {
            const bool here = base + tid * kPerThread + e < n;
            r[e] = make_request(here ? c[e] : 0, here ? m[e] : 0, shift, width);
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
        int64_t end = 0;  // of the pages that this thread's requests take
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
                if (served && r[e].need > 0 && at.tokens + r[e].fresh > T) {
                    // page have + u begins at the request's token ((have + u) << shift) - ctx
                    const int64_t have = pages_of(r[e].ctx, shift), cut = max(int64_t(0), T - at.tokens) + r[e].ctx;
                    for (int64_t p = max(have, pages_of(cut, shift)); p < have + r[e].need; ++p)
                        table[i * ld_table + p] = free_pages[at.pages + p - have];
                }
            }
            if (served && r[e].need > 0) end = at.pages + r[e].need;
            at.tokens += r[e].fresh;
            at.pages += r[e].need;
        }
        // served requests take a prefix of the free list: the last one's end is what is taken
        if (blockIdx.x == 0) {
            const uint32_t takers = __ballot_sync(0xffffffffu, end > 0);
            if (takers != 0 && lane == 31 - __clz(takers)) atomicMax(&s_taken, static_cast<unsigned long long>(end));
        }
        if (tid == kThreads - 1) s_row[kChunk] = at.tokens;
        __syncthreads();
        // this window's tokens among the chunk's
        const int64_t t0 = max(w0, s_row[0]), t1 = min(w1, s_row[kChunk]);
        // a thread's tokens side by side: searches, then page loads, then the writes
        int32_t at_request[kEach], page[kEach];
        int64_t pos[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) at_request[e] = 0;
#pragma unroll
        for (int step = kChunk / 2; step > 0; step >>= 1)
#pragma unroll
            for (int e = 0; e < kEach; ++e)  // the last request that starts at or before the token
                if (s_row[at_request[e] + step] <= t0 + tid + e * kThreads) at_request[e] += step;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int64_t t = t0 + tid + e * kThreads;
            const int32_t l = at_request[e];
            pos[e] = s_ctx[l] + (t - s_row[l]);
            page[e] = -1;
            if (t < t1 && s_page[l] >= 0) {
                const int64_t have = pages_of(s_ctx[l], shift), p = pos[e] >> shift;
                page[e] = p < have ? table[(base + l) * ld_table + p] : free_pages[s_page[l] + p - have];
            }
        }
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int64_t t = t0 + tid + e * kThreads;
            if (t >= t1) break;
            const int32_t l = at_request[e], i = base + l;
            const int64_t p = pos[e] >> shift, in_page = pos[e] & ((int64_t(1) << shift) - 1);
            if (s_page[l] >= 0) {
                if (in_page == 0 && p >= pages_of(s_ctx[l], shift)) table[i * ld_table + p] = page[e];
                if (page[e] < 0) report_error(err, LORA_ERR_SLOT_RANGE);
            }
            positions[t] = static_cast<int32_t>(min(pos[e], int64_t(INT32_MAX)));
            seq_ids[t] = i;
            slot_map[t] = page[e] < 0 ? -1 : (int64_t(page[e]) << shift) + in_page;
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

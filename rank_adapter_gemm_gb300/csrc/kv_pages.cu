// Block tables of requests that branch, end and move (lora_kv_fork, lora_kv_compact).
//
// Both calls ask which pages a set of table rows names, and then for the k-th page
// in use or free in rising order: a bitmap of the pages and its prefix sums.  The
// work is 4 bytes an entry, so chains of dependent loads and the steps between them
// bound it, not bandwidth.  One cluster therefore does all of it in one launch
// without a workspace: the entries of the rows are spread over its blocks, each of
// which marks the pages that it meets in a bitmap of its own in shared memory; the
// bitmaps are joined through distributed shared memory, every block taking one slice
// of the pages; and the slices' counts, exchanged the same way, give every page its
// rank.  The cluster's barriers are the only waits.
//
// Measured, graph replay: 128 rows of up to 4,000 tokens (pages of 16) forked in 7.5 us, 1,024 rows
// with 102,000 entries in 14.1 (8 blocks a cluster 19), 16 rows compacted in 10.4, 1,024 in 29.5.
// A barrier of the cluster and what it waits for take about 1 us each; 5 of them, and one
// chain of loads (parents, lengths, entries), are the small fork.  The large ones spend the
// rest on entries and lists, 16 SMs' loads and stores; the compaction asks for every entry where
// its page moves (a load that depends on one).
#include "attention.cuh"

namespace lora {

namespace {

constexpr int kCtas = 16, kThreads = 1024, kWarps = kThreads / 32;
constexpr int kSpan = 256;  // entries of a row that a warp takes at a time

struct PagesArgs {
    const int32_t *src, *lens, *parents, *held;
    int32_t *dst, *dst_lens, *dst_held, *copies, *n_copies, *free_pages, *n_free, *err;
    int64_t ld_src, ld_dst;
    int32_t src_width, dst_width, n_src, n_rows, n_held, n_pages, shift;
};

__device__ __forceinline__ uint32_t ld_peer(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// (Threads may arrive one by one: the loops before it end at different times.)
__device__ __forceinline__ void sync_cluster() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Sum over the block's threads before this one; *total gets all of it.
__device__ __forceinline__ int32_t scan_block(int32_t mine, int32_t *s_warp, int32_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int32_t w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += v;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int32_t before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return (warp > 0 ? before : 0) + incl - mine;
}

// Words of the bitmap in a block's slice: a multiple of 4, so that slices are read in 16 bytes.
__host__ __device__ constexpr int32_t slice_words(int32_t n_pages) {
    return ((n_pages + 32 * kCtas * 4 - 1) / (32 * kCtas * 4)) * 4;
}

// The bitmap, and the free pages before each word of the own slice; then by row (of
// the new batch): its source row and its entries; for a fork, each parent's first child and each copy's row.
__host__ __device__ constexpr size_t pages_smem(int32_t n_pages, int32_t n_src, int32_t n_rows, bool fork) {
    const size_t rows = static_cast<size_t>((n_rows + 3) & ~3), src = static_cast<size_t>((n_src + 3) & ~3);
    return size_t(4) * (slice_words(n_pages) * (kCtas + 1) + 2 * rows + (fork ? src + rows : 0));
}

template <bool FORK>
__global__ void __launch_bounds__(kThreads, 1) kv_pages_kernel(const PagesArgs a) {
    extern __shared__ __align__(16) uint32_t smem_words[];
    __shared__ int32_t s_warp[32];
    __shared__ int32_t s_free[1];  // free pages of this block's slice
    __shared__ int32_t s_most;     // entries of the longest row
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_ctarank();
    const int32_t per = slice_words(a.n_pages), words = per * kCtas;
    uint32_t *s_map = smem_words;
    int32_t *s_before = reinterpret_cast<int32_t *>(smem_words + words);
    int32_t *s_from = s_before + per, *s_have = s_from + ((a.n_rows + 3) & ~3);
    int32_t *s_first = s_have + ((a.n_rows + 3) & ~3), *s_job = s_first + ((a.n_src + 3) & ~3);

    for (int32_t w = tid; w < words; w += kThreads) s_map[w] = 0u;
    if (FORK)
        for (int32_t i = tid; i < a.n_src; i += kThreads) s_first[i] = INT32_MAX;
    if (tid == 0) s_most = 0;
    wait_for_previous();
    __syncthreads();

    // ---- the rows: where they come from, how many entries, which need a copy -------
    const int32_t in_page = (1 << a.shift) - 1;
    // a row's length; bad ones (reported by one block) are empty
    const auto length_of = [&](int32_t p) {
        const int32_t len = a.lens[p];
        const int32_t pages = len > 0 ? static_cast<int32_t>((int64_t(len) + in_page) >> a.shift) : 0;
        if (len < 0 || pages > a.src_width || pages > a.dst_width) {
            if (rank == 0) report_error(a.err, LORA_ERR_INVALID_ARG);
            return 0;
        }
        return len;
    };
    for (int32_t i = tid; i < a.n_rows; i += kThreads) {
        int32_t p = i;
        if (FORK) {
            p = a.parents[i];
            if (p < -1 || p >= a.n_src) {
                if (rank == 0) report_error(a.err, LORA_ERR_INVALID_ARG);
                p = -1;
            }
        }
        const int32_t len = p >= 0 ? length_of(p) : 0;
        s_from[i] = p;
        s_have[i] = len;  // until the entries are known
        if (FORK && p >= 0) atomicMin(&s_first[p], i);
        if (len > 0) atomicMax(&s_most, static_cast<int32_t>((int64_t(len) + in_page) >> a.shift));
    }
    __syncthreads();
    int32_t jobs = 0;  // copies of the call
    if (FORK) {
        for (int32_t base = 0; base < a.n_rows; base += kThreads) {
            const int32_t i = base + tid;
            const bool job = i < a.n_rows && (s_have[i] & in_page) != 0 && s_first[s_from[i]] != i;
            int32_t total;
            const int32_t at = jobs + scan_block(job, s_warp, &total);
            if (job) s_job[at] = i;
            jobs += total;
            if (i < a.n_rows && rank == 0) {
                a.dst_lens[i] = s_have[i];
                if (!job)
                    for (int e = 0; e < 3; ++e) a.copies[3 * int64_t(i) + e] = e < 2 ? -1 : 0;
            }
        }
    }

    // ---- the entries: copied, and marked in the block's bitmap ---------------------
    const auto mark = [&](int32_t page) {
        if (static_cast<uint32_t>(page) < static_cast<uint32_t>(a.n_pages)) {
            const uint32_t bit = 1u << (page & 31);
            if ((s_map[page >> 5] & bit) == 0) atomicOr(&s_map[page >> 5], bit);
            return true;
        }
        return false;
    };
    // entries of row i that are copied as they are
    const auto entries = [&](int32_t i) {
        const int32_t len = s_have[i], pages = static_cast<int32_t>((int64_t(len) + in_page) >> a.shift);
        return FORK && (len & in_page) != 0 && s_first[s_from[i]] != i ? pages - 1 : pages;
    };
    // calls f(row of the new batch, first entry, end) for this warp's spans, spread over the cluster
    constexpr int32_t kTakers = kWarps * kCtas;
    const int32_t id = warp * kCtas + rank;
    const auto each_span = [&](auto f) {
        for (int32_t c = 0; c < s_most; c += kSpan)
            // (spans of neighbouring rows, then of their next entries, go round the warps)
            for (int32_t i = ((id - c / kSpan * (a.n_rows % kTakers)) % kTakers + kTakers) % kTakers; i < a.n_rows;
                 i += kTakers) {
                const int32_t end = min(entries(i), c + kSpan);
                if (c < end) f(i, c, end);
            }
    };
    constexpr int kEach = kSpan / 32;  // entries a lane, all of whose loads are under way together
    each_span([&](int32_t i, int32_t e0, int32_t e1) {
        const int32_t *from = a.src + s_from[i] * a.ld_src;
        int32_t *to = a.dst + i * a.ld_dst;
        int32_t page[kEach];
#pragma unroll
        for (int u = 0; u < kEach; ++u) page[u] = from[min(e0 + u * 32 + lane, e1 - 1)];
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const int32_t e = e0 + u * 32 + lane;
            if (e >= e1) break;
            if (FORK) to[e] = page[u];
            if (!mark(page[u])) report_error(a.err, LORA_ERR_SLOT_RANGE);
        }
    });
    for (int32_t i = rank * kThreads + tid; i < a.n_held; i += kCtas * kThreads) {
        const int32_t page = a.held[i];
        if (page != -1 && !mark(page)) report_error(a.err, LORA_ERR_SLOT_RANGE);
    }
    sync_cluster();

    // ---- the bitmaps joined: this block's slice of the pages, free ones as ones ------
    const int32_t w0 = static_cast<int32_t>(rank) * per;
    for (int32_t v = tid; v < per; v += kThreads) {
        const uint32_t at = smem_addr(s_map + w0 + v);
        uint32_t x[kCtas], all = 0;
#pragma unroll
        for (int c = 0; c < kCtas; ++c) x[c] = ld_peer(map_to_rank(at, c));
#pragma unroll
        for (int c = 0; c < kCtas; ++c) all |= x[c];
        // (other blocks still read this slice of the bitmap: the joined words go elsewhere)
        s_before[v] = static_cast<int32_t>(all);
    }
    sync_cluster();
    const int32_t each = (per + kThreads - 1) / kThreads;  // words a thread
    int32_t mine = 0;
    for (int32_t j = 0; j < each; ++j) {
        const int32_t w = tid * each + j;
        if (w >= per) break;
        const int64_t left = int64_t(a.n_pages) - int64_t(w0 + w) * 32;  // pages from this word on
        const uint32_t real = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1 : 0u;
        const uint32_t word = ~static_cast<uint32_t>(s_before[w]) & real;
        s_map[w0 + w] = word;
        mine += __popc(word);
    }
    int32_t slice_free;
    int32_t at = scan_block(mine, s_warp, &slice_free);
    if (tid == 0) s_free[0] = slice_free;
    sync_cluster();
    // free pages in the slices before this one, and in all: a lane a block
    const int32_t theirs = lane < kCtas ? static_cast<int32_t>(ld_peer(map_to_rank(smem_addr(s_free), lane))) : 0;
    const int32_t free_before = __reduce_add_sync(0xffffffffu, lane < static_cast<int>(rank) ? theirs : 0);
    int32_t n_free = __reduce_add_sync(0xffffffffu, theirs);
    at += free_before;
    for (int32_t j = 0; j < each; ++j) {
        const int32_t w = tid * each + j;
        if (w >= per) break;
        s_before[w] = at;
        at += __popc(s_map[w0 + w]);
    }
    __syncthreads();

    if constexpr (FORK) {
        // ---- free pages in order: to the copies first, then to the list --------------
        for (int32_t w = warp; w < per; w += kWarps) {
            const uint32_t word = s_map[w0 + w];
            if (!((word >> lane) & 1)) continue;
            const int32_t f = s_before[w] + __popc(word & ((1u << lane) - 1)), page = (w0 + w) * 32 + lane;
            if (f >= jobs) {
                a.free_pages[f - jobs] = page;
                continue;
            }
            const int32_t i = s_job[f], len = s_have[i], last = len >> a.shift;
            const int32_t from = a.src[s_from[i] * a.ld_src + last];
            const bool ok = static_cast<uint32_t>(from) < static_cast<uint32_t>(a.n_pages);
            if (!ok) report_error(a.err, LORA_ERR_SLOT_RANGE);
            a.dst[i * a.ld_dst + last] = page;
            a.copies[3 * int64_t(i)] = ok ? from : -1;
            a.copies[3 * int64_t(i) + 1] = ok ? page : -1;
            a.copies[3 * int64_t(i) + 2] = ok ? len & in_page : 0;
        }
        if (rank == 0) {
            for (int32_t u = n_free + tid; u < jobs; u += kThreads) {  // copies without a page
                const int32_t i = s_job[u];
                report_error(a.err, LORA_ERR_NO_PAGES);
                a.dst_lens[i] = s_have[i] & ~in_page;
                for (int e = 0; e < 3; ++e) a.copies[3 * int64_t(i) + e] = e < 2 ? -1 : 0;
            }
        }
        n_free = max(0, n_free - jobs);
    } else {
        // ---- pages in use at or past their number: each to the free page of its rank --
        // The list of free pages, written last, holds on the way: in front, by rank, the pages that
        // are moved to (fewer than are in use); at page p >= used, where it moves.
        const int32_t used = a.n_pages - n_free;
        sync_cluster();  // every slice's words and counts are there
        int32_t n_moves = 0;  // free pages below `used`
        if (n_free > 0) {
            const int32_t w = used >> 5, owner = w / per;
            const uint32_t word = ld_peer(map_to_rank(smem_addr(s_map + w), owner));
            n_moves = static_cast<int32_t>(ld_peer(map_to_rank(smem_addr(s_before + w % per), owner))) +
                      __popc(word & ((1u << (used & 31)) - 1));
        }
        const int32_t all = static_cast<int32_t>(rank) * kThreads + tid;
        // calls f(page, free, free pages before it) for the pages of this slice
        const auto each_page = [&](auto f) {
            for (int32_t w = warp; w < per; w += kWarps) {
                const uint32_t word = s_map[w0 + w];
                const int32_t page = (w0 + w) * 32 + lane;
                if (page < a.n_pages) f(page, (word >> lane) & 1, s_before[w] + __popc(word & ((1u << lane) - 1)));
            }
        };
        each_page([&](int32_t page, bool is_free, int32_t f) {
            if (page < used && is_free) a.free_pages[f] = page;
        });
        for (uint32_t i = 3 * n_moves + all; i < 3u * (a.n_pages / 2); i += kCtas * kThreads)
            a.copies[i] = i % 3 < 2 ? -1 : 0;
        if (all == 0) a.n_copies[0] = n_moves;
        __threadfence();
        sync_cluster();
        each_page([&](int32_t page, bool is_free, int32_t f) {
            if (page < used || is_free) return;
            const int64_t i = page - f - (used - n_moves);  // its rank among those
            const int32_t to = __ldcg(a.free_pages + i);
            a.free_pages[page] = to;
            a.copies[3 * i] = page;
            a.copies[3 * i + 1] = to;
            a.copies[3 * i + 2] = in_page + 1;
        });
        __threadfence();
        sync_cluster();
        const auto moved = [&](int32_t p) { return p >= used && p < a.n_pages ? __ldcg(a.free_pages + p) : p; };
        each_span([&](int32_t i, int32_t e0, int32_t e1) {
            const int32_t *from = a.src + s_from[i] * a.ld_src;
            int32_t *to = a.dst + i * a.ld_dst;
            int32_t page[kEach];
#pragma unroll
            for (int u = 0; u < kEach; ++u) page[u] = from[min(e0 + u * 32 + lane, e1 - 1)];
#pragma unroll
            for (int u = 0; u < kEach; ++u) page[u] = moved(page[u]);
#pragma unroll
            for (int u = 0; u < kEach; ++u)
                if (e0 + u * 32 + lane < e1) to[e0 + u * 32 + lane] = page[u];
        });
        for (int32_t i = all; i < a.n_held; i += kCtas * kThreads) {
            const int32_t p = a.held[i];
            a.dst_held[i] = p == -1 ? -1 : moved(p);
        }
        sync_cluster();  // the ways have been read
        for (int32_t p = all; p < n_free; p += kCtas * kThreads) a.free_pages[p] = used + p;
    }
#pragma unroll 4
    for (int32_t p = n_free + static_cast<int32_t>(rank) * kThreads + tid; p < a.n_pages; p += kCtas * kThreads)
        a.free_pages[p] = -1;
    if (rank == 0 && tid == 0) a.n_free[0] = n_free;
    sync_cluster();  // no block's shared memory is read any more
}

template <bool FORK>
cudaError_t launch(const PagesArgs &a, cudaStream_t stream) {
    static std::atomic<uint64_t> seen{0};
    constexpr size_t kMost = pages_smem(LORA_MAX_PAGES, LORA_MAX_SEQS, LORA_MAX_SEQS, true);
    static_assert(kMost <= 227 * 1024 - 1024, "shared memory");
    int sms = 0;
    cudaError_t e = prepare_kernel(kv_pages_kernel<FORK>, static_cast<int>(kMost), seen, &sms);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> wide{0};  // a bit a device: clusters beyond 8 blocks allowed
    int device = 0;
    if ((e = cudaGetDevice(&device)) != cudaSuccess) return e;
    if (device >= 64 || ((wide.load(std::memory_order_acquire) >> device) & 1) == 0) {
        e = cudaFuncSetAttribute(kv_pages_kernel<FORK>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        if (device < 64) wide.fetch_or(uint64_t(1) << device, std::memory_order_release);
    }
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = pages_smem(a.n_pages, a.n_src, a.n_rows, FORK);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kv_pages_kernel<FORK>, a);
}

}  // namespace

cudaError_t launch_kv_fork(const int32_t *src, int64_t ld_src, int32_t src_width, const int32_t *lens, int32_t n_src,
                           const int32_t *parents, int32_t n_dst, int32_t shift, int32_t n_pages, const int32_t *held,
                           int32_t n_held, int32_t *dst, int64_t ld_dst, int32_t dst_width, int32_t *dst_lens,
                           int32_t *copies, int32_t *free_pages, int32_t *n_free, int32_t *err, cudaStream_t stream) {
    return launch<true>(PagesArgs{src, lens, parents, held, dst, dst_lens, nullptr, copies, nullptr, free_pages, n_free,
                                  err, ld_src, ld_dst, src_width, dst_width, n_src, n_dst, n_held, n_pages, shift},
                        stream);
}

cudaError_t launch_kv_compact(const int32_t *src, int64_t ld_src, int32_t width, const int32_t *lens, int32_t n_seq,
                              int32_t shift, int32_t n_pages, const int32_t *held, int32_t n_held, int32_t *dst,
                              int64_t ld_dst, int32_t *dst_held, int32_t *moves, int32_t *n_moves, int32_t *free_pages,
                              int32_t *n_free, int32_t *err, cudaStream_t stream) {
    return launch<false>(PagesArgs{src, lens, nullptr, held, dst, nullptr, dst_held, moves, n_moves, free_pages, n_free,
                                   err, ld_src, ld_dst, width, width, n_seq, n_seq, n_held, n_pages, shift},
                         stream);
}

}  // namespace lora

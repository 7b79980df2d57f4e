// Selection of beam search (lora_beam_select).
//
// What it must read is the logits, once: HBM bounds it, with one exponential an
// element.  A block takes kChunk neighbouring logits of a row into registers and
// leaves what a selection can need of them: maximum, sum of exponentials, and the
// `keep` largest.  The block that arrives last at a request joins them: the rows'
// logarithms, then the `keep` best of all lists.
//
// The largest of a set are found through a bound: of 64 groups of elements, the
// keep-th largest of the groups' maxima is one that at least `keep` elements
// reach.  The elements that reach it, usually little more than `keep`, in few threads,
// are gathered and ranked by counting; where many are equal they are taken one by one.
// All keys of a chunk differ (value, then the lower token first), so order never
// depends on timing.
//
// A chunk's sum is taken in fp32 (32 terms a thread, then a tree); a row's, and all
// comparisons of candidates, in 64 bits: scores of different beams meet there, and a
// rounding to fp32 would decide between candidates.
#include "attend.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256, kEach = 32, kChunk = kThreads * kEach;
constexpr int kGroups = 64;   // groups of 4 neighbouring threads
constexpr int kGather = 1024;  // gathered keys at most; more take the slow way

struct SelectArgs {
    const void *logits;
    int64_t ld;
    const float *scores;
    const int32_t *ended;
    int32_t *parents, *tokens, *out_ended;
    float *out_scores;
    int32_t *counters;   // a request
    float2 *sums;        // maximum and sum of each row's chunks
    float *values;       // the largest of each chunk
    int32_t *ids;        // and their tokens
    int32_t beams, vocab, keep, eos, chunks;
};

// Order of fp32 values as unsigned numbers; -0 counts as 0.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ uint64_t ordered(double x) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
    return (u >> 63) ? ~u : u | (uint64_t(1) << 63);
}

// A thread's elements in registers.  Keys of elements: the value, then the lower index first; 0 is
// below all.  Indexes within a chunk are below 2^16.
struct Bf16Logits {
    using Key = uint32_t;
    static constexpr int kVec = 8, kWords = kEach / 2;
    static constexpr uint32_t kNone = 0xff80ff80u;  // -inf
    __device__ static float value(const uint32_t (&w)[kWords], int e) {
        return (e & 1) ? bf16hi_to_f32(w[e / 2]) : bf16lo_to_f32(w[e / 2]);
    }
    __device__ static uint32_t element(const void *p, int64_t i) { return static_cast<const uint16_t *>(p)[i]; }
    // the elements of a vector that are there, one by one
    __device__ static void put(uint32_t *w, int e, uint32_t v) {
        w[e / 2] = __byte_perm(w[e / 2], v, (e & 1) ? 0x5410 : 0x3254);
    }
    __device__ static float top(const uint32_t (&w)[kWords]) {
        uint32_t m = w[0];
#pragma unroll
        for (int i = 1; i < kWords; ++i) asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(w[i]));
        return fmaxf(bf16lo_to_f32(m), bf16hi_to_f32(m));
    }
    __device__ static Key key(float x, int32_t i) {
        return (ordered(x) & 0xffff0000u) | static_cast<uint32_t>(0xffff - i);
    }
    // (a negative value's ordered form is its complement: the low half was ones)
    __device__ static float of_key(Key k) { return from_ordered((k & 0x80000000u) ? k & 0xffff0000u : k | 0xffffu); }
};

struct Fp32Logits {
    using Key = uint64_t;
    static constexpr int kVec = 4, kWords = kEach;
    static constexpr uint32_t kNone = 0xff800000u;
    __device__ static float value(const uint32_t (&w)[kWords], int e) { return __uint_as_float(w[e]); }
    __device__ static uint32_t element(const void *p, int64_t i) { return static_cast<const uint32_t *>(p)[i]; }
    __device__ static void put(uint32_t *w, int e, uint32_t v) { w[e] = v; }
    __device__ static float top(const uint32_t (&w)[kWords]) {
        float m = __uint_as_float(w[0]);
#pragma unroll
        for (int i = 1; i < kWords; ++i) m = fmaxf(m, __uint_as_float(w[i]));
        return m;
    }
    __device__ static Key key(float x, int32_t i) {
        return (static_cast<uint64_t>(ordered(x)) << 32) | static_cast<uint32_t>(0xffff - i);
    }
    __device__ static float of_key(Key k) { return from_ordered(static_cast<uint32_t>(k >> 32)); }
};

template <class K>
__device__ __forceinline__ K shfl_max(K v, int o) {
    const K u = __shfl_xor_sync(0xffffffffu, v, o);
    return u > v ? u : v;
}

// The keep-th largest of 64 group values (s_group), by counting; by the whole block, with a
// barrier in front and behind.  Groups without elements hold the least value.
template <class K>
__device__ __forceinline__ K bound_of(const K *s_group, K *s_bound, int32_t keep) {
    __syncthreads();
    if (threadIdx.x < kGroups) {
        const K me = s_group[threadIdx.x];
        int above = 0;
#pragma unroll 16
        for (int j = 0; j < kGroups; ++j) {
            const K other = s_group[j];
            above += other > me || (other == me && j < static_cast<int>(threadIdx.x));
        }
        if (above == keep - 1) *s_bound = me;
    }
    __syncthreads();
    return *s_bound;
}

// A candidate of the request: its value in order, then beam * vocab + token.
struct Candidate {
    uint64_t key;
    uint32_t id;
    __device__ bool before(const Candidate &o) const { return key > o.key || (key == o.key && id < o.id); }
};

// The keep best of the request's lists, in order, to the outputs.
__device__ void join_request(const SelectArgs &a, int32_t r) {
    __shared__ double s_base[LORA_MAX_BEAMS];  // score minus the logarithm; NaN: no candidates
    __shared__ bool s_ended[LORA_MAX_BEAMS];   // (outputs may take the inputs' place)
    __shared__ uint64_t s_group[kGroups], s_bound;
    __shared__ Candidate s_found[kGather], s_best[kThreads / 32];
    __shared__ int32_t s_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t lists = a.beams * a.chunks;
    const int64_t list0 = int64_t(r) * lists;
    if (tid == 0) s_n = 0;
    for (int32_t b = warp; b < a.beams; b += kThreads / 32) {
        const int32_t row = r * a.beams + b;
        const float2 *sums = a.sums + int64_t(row) * a.chunks;
        float2 mine = lane < a.chunks ? __ldcg(sums + lane) : make_float2(-INFINITY, 0.0f);
        const float score = lane == 0 ? a.scores[row] : 0.0f;
        const bool ended = lane == 0 && a.ended != nullptr && a.ended[row] != 0;
        float top = mine.x;
        for (int32_t c = lane + 32; c < a.chunks; c += 32) top = fmaxf(top, __ldcg(sums + c).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        double sum = 0.0;
        for (int32_t c = lane; c < a.chunks; c += 32) {
            if (c != lane) mine = __ldcg(sums + c);
            // (a chunk without a number above -inf has sum 0; a NaN or +inf makes the sum NaN)
            if (mine.y != 0.0f) sum += mine.y * exp(static_cast<double>(mine.x) - top);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) {
            double base = ended ? score : score - (top + log(sum));
            if (!(base > -INFINITY && base < INFINITY)) base = NAN;
            s_base[b] = base;
            s_ended[b] = ended;
        }
    }
    __syncthreads();
    // candidate k of a list; key 0: none
    const auto candidate = [&](int32_t list, int32_t k) {
        const int64_t at = (list0 + list) * a.keep + k;
        const int32_t b = list / a.chunks, token = __ldcg(a.ids + at);
        const double v = s_base[b] + __ldcg(a.values + at);
        return Candidate{token >= 0 && v > -INFINITY ? ordered(v) : 0, static_cast<uint32_t>(b) * a.vocab + token};
    };
    // a bound that `keep` candidates reach: of 64 groups of lists, their firsts
    uint64_t best = 0;
    for (int32_t l = tid; l < lists; l += kThreads) best = max(best, candidate(l, 0).key);
    best = shfl_max(shfl_max(best, 1), 2);
    if ((lane & 3) == 0) s_group[tid >> 2] = best;
    const uint64_t bound = max(bound_of(s_group, &s_bound, a.keep), uint64_t(1));
    for (int32_t l = tid; l < lists; l += kThreads) {
        for (int32_t k = 0; k < a.keep; ++k) {
            const Candidate c = candidate(l, k);
            if (c.key < bound) break;  // the list falls
            const int32_t at = atomicAdd(&s_n, 1);
            if (at < kGather) s_found[at] = c;
        }
    }
    __syncthreads();
    const int32_t found = s_n;
    const auto put = [&](int32_t k, const Candidate &c) {
        const int64_t to = int64_t(r) * a.keep + k;
        const bool there = c.key != 0;
        const int32_t b = there ? static_cast<int32_t>(c.id / a.vocab) : 0;
        const int32_t token = there ? static_cast<int32_t>(c.id - static_cast<uint32_t>(b) * a.vocab) : -1;
        const uint64_t u = c.key;
        const double v = __longlong_as_double(static_cast<long long>((u >> 63) ? u ^ (uint64_t(1) << 63) : ~u));
        a.parents[to] = there ? r * a.beams + b : -1;
        a.tokens[to] = token;
        a.out_scores[to] = there ? static_cast<float>(v) : -INFINITY;
        a.out_ended[to] = there && (token == a.eos || s_ended[b]);
    };
    if (found <= kGather) {
        for (int32_t i = tid; i < found; i += kThreads) {
            const Candidate me = s_found[i];
            int32_t above = 0;
            for (int32_t j = 0; j < found; ++j) above += s_found[j].before(me);
            if (above < a.keep) put(above, me);
        }
        for (int32_t k = found + tid; k < a.keep; k += kThreads) put(k, Candidate{0, 0});
        return;
    }
    // one after the other: the best behind the last one
    Candidate last{~uint64_t(0), 0};
    for (int32_t k = 0; k < a.keep; ++k) {
        Candidate now{0, 0xffffffffu};
        for (int32_t l = tid; l < lists; l += kThreads)
            for (int32_t j = 0; j < a.keep; ++j) {
                const Candidate c = candidate(l, j);
                if (c.key < bound) break;
                if (last.before(c) && c.before(now)) now = c;
            }
        const auto better = [&](uint64_t key, uint32_t id) {
            const Candidate c{key, id};
            if (c.before(now)) now = c;
        };
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            better(__shfl_xor_sync(0xffffffffu, now.key, o), __shfl_xor_sync(0xffffffffu, now.id, o));
        __syncthreads();
        if (lane == 0) s_best[warp] = now;
        __syncthreads();
        for (int w = 0; w < kThreads / 32; ++w) better(s_best[w].key, s_best[w].id);
        last = now;
        if (tid == 0) put(k, now);
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads, 4) beam_select_kernel(const SelectArgs a) {
    using Key = typename T::Key;
    constexpr int kVec = T::kVec, kVecs = kEach / kVec, kSize = 16 / kVec;
    __shared__ uint32_t s_top[kThreads / 32], s_group[kGroups], s_bound;
    __shared__ float s_sum[kThreads / 32];
    __shared__ Key s_keys[kGather], s_best[kThreads / 32];
    __shared__ int32_t s_n;
    __shared__ bool s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t row = static_cast<int32_t>(blockIdx.x / a.chunks), chunk = static_cast<int32_t>(blockIdx.x % a.chunks);
    const int32_t r = row / a.beams;
    if (tid == 0) s_n = 0;
    wait_for_previous();
    const bool ended = a.ended != nullptr && a.ended[row] != 0;
    const int64_t list = (int64_t(row) * a.chunks + chunk) * a.keep;
    if (ended) {
        for (int32_t k = tid; k < a.keep; k += kThreads) {
            const bool here = chunk == 0 && k == 0;
            a.values[list + k] = here ? 0.0f : -INFINITY;
            a.ids[list + k] = here ? a.eos : -1;
        }
        if (tid == 0) a.sums[int64_t(row) * a.chunks + chunk] = make_float2(0.0f, 1.0f);
    } else {
        const int32_t v0 = chunk * kChunk, n = min(kChunk, a.vocab - v0);
        const unsigned char *base = static_cast<const unsigned char *>(a.logits) + (row * a.ld + v0) * kSize;
        // thread t's vector u holds elements (u * 256 + t) * kVec - skew ..: whole vectors lie on 16
        // bytes.  A skewed chunk's last elements go one each to the first threads' last places, which
        // hold elements before the chunk or none (u = 0, t = 0: `skew` elements of 8 or 4).
        const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15) / kSize);
        uint32_t w[T::kWords];
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            const int32_t i = (u * kThreads + tid) * kVec - skew;
            uint32_t *to = w + u * (T::kWords / kVecs);
            if (i >= 0 && i + kVec <= n) {
                const uint4 v = ldg_cg(base + int64_t(i) * kSize);
                to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
            } else {
                to[0] = to[1] = to[2] = to[3] = T::kNone;
                if (i + kVec > 0 && i < n) {
#pragma unroll
                    for (int e = 0; e < kVec; ++e)
                        if (i + e >= 0 && i + e < n) T::put(to, e, T::element(base, i + e));
                }
            }
        }
        // thread 0's first vector has room for the elements that the skew pushes out at the end
        const int32_t tail = kChunk - skew;  // their first index
        if (tid == 0 && tail < n) {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (e < skew && tail + e < n) T::put(w, e, T::element(base, tail + e));
        }
        const auto index_of = [&](int e) {
            const int32_t i = (e / kVec * kThreads + tid) * kVec - skew + e % kVec;
            return i < 0 ? i + kChunk : i;
        };
        const float mine = T::top(w);
        const uint32_t order = ordered(mine);
        uint32_t best = shfl_max(shfl_max(order, 1), 2);
        if ((lane & 3) == 0) s_group[tid >> 2] = best;
        best = __reduce_max_sync(0xffffffffu, best);
        if (lane == 0) s_top[warp] = best;
        const float bound = from_ordered(bound_of(s_group, &s_bound, a.keep));
        best = s_top[0];
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) best = max(best, s_top[i]);
        const float top = from_ordered(best), ref = top == -INFINITY ? 0.0f : top;
        const uint64_t by2 = pack2(kLog2e, kLog2e), ref2 = pack2(-ref, -ref);
        uint64_t sums[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < kEach; e += 2) {
            // the difference first: it is exact near the maximum, where the terms count
            float d0, d1;
            unpack2(mul2(add2(pack2(T::value(w, e), T::value(w, e + 1)), ref2), by2), d0, d1);
            sums[e / 2 & 1] = add2(sums[e / 2 & 1], pack2(ex2(d0), ex2(d1)));
        }
        float sum, odd;
        unpack2(add2(sums[0], sums[1]), sum, odd);
        sum += odd;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s_sum[warp] = sum;
        // few threads have an element that reaches the bound
        if (mine >= bound && mine > -INFINITY) {
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const float x = T::value(w, e);
                if (x >= bound && x > -INFINITY) {
                    const int32_t at = atomicAdd(&s_n, 1);
                    if (at < kGather) s_keys[at] = T::key(x, index_of(e));
                }
            }
        }
        __syncthreads();
        if (tid == 0) {
            float all = 0.0f;
            for (int i = 0; i < kThreads / 32; ++i) all += s_sum[i];
            a.sums[int64_t(row) * a.chunks + chunk] = make_float2(top, all);
        }
        const int32_t found = s_n;
        const auto put = [&](int32_t k, Key key) {
            a.values[list + k] = T::of_key(key);
            a.ids[list + k] = v0 + 0xffff - static_cast<int32_t>(key & 0xffffu);
        };
        if (found <= kGather) {
            for (int32_t i = tid; i < found; i += kThreads) {
                const Key me = s_keys[i];
                int32_t above = 0;
                for (int32_t j = 0; j < found; ++j) above += s_keys[j] > me;
                if (above < a.keep) put(above, me);
            }
        } else {
            // one after the other: the largest below the last one
            Key last = ~Key(0);
            for (int32_t k = 0; k < a.keep; ++k) {
                Key now = 0;
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    const float x = T::value(w, e);
                    const Key key = x > -INFINITY ? T::key(x, index_of(e)) : 0;
                    if (key < last && key > now) now = key;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) now = shfl_max(now, o);
                __syncthreads();
                if (lane == 0) s_best[warp] = now;
                __syncthreads();
                for (int i = 0; i < kThreads / 32; ++i) now = s_best[i] > now ? s_best[i] : now;
                last = now;
                if (tid == 0) put(k, now);
            }
        }
        for (int32_t k = min(found, a.keep) + tid; k < a.keep; k += kThreads) {
            a.values[list + k] = -INFINITY;
            a.ids[list + k] = -1;
        }
    }
    // the last block of the request joins its lists
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        const int32_t all = a.beams * a.chunks;
        s_last = atomicAdd(a.counters + r, 1) == all - 1;
        if (s_last) a.counters[r] = 0;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    join_request(a, r);
}

int32_t chunks_of(int32_t vocab) { return (vocab + kChunk - 1) / kChunk; }
size_t up128(size_t b) { return (b + 127) & ~size_t(127); }

// Their place does not depend on the call, so calls of other sizes find them as they were.
constexpr size_t kCounters = size_t(LORA_MAX_SEQS) * 4;

}  // namespace

// Counters (a request), then sums (a chunk of a row), values and tokens (`keep` a chunk).
size_t beam_select_workspace_bytes(int32_t n_req, int32_t beams, int32_t keep, int32_t vocab) {
    const size_t lists = size_t(n_req) * beams * chunks_of(vocab);
    return kCounters + up128(lists * 8) + 2 * up128(lists * keep * 4);
}

cudaError_t launch_beam_select(const void *logits, int64_t ld, bool fp32, int32_t n_req, int32_t beams, int32_t vocab,
                               int32_t keep, const float *scores, const int32_t *ended, int32_t eos, int32_t *parents,
                               int32_t *tokens, float *out_scores, int32_t *out_ended, void *ws, cudaStream_t stream) {
    const int32_t chunks = chunks_of(vocab);
    const size_t lists = size_t(n_req) * beams * chunks;
    char *at = static_cast<char *>(ws);
    SelectArgs a{logits, ld, scores, ended, parents, tokens, out_ended, out_scores, reinterpret_cast<int32_t *>(at),
                 nullptr, nullptr, nullptr, beams, vocab, keep, eos, chunks};
    at += kCounters;
    a.sums = reinterpret_cast<float2 *>(at);
    at += up128(lists * 8);
    a.values = reinterpret_cast<float *>(at);
    a.ids = reinterpret_cast<int32_t *>(at + up128(lists * keep * 4));
    if (fp32)
        return launch_dependent(beam_select_kernel<Fp32Logits>, static_cast<unsigned>(lists), kThreads, 0, stream, a);
    return launch_dependent(beam_select_kernel<Bf16Logits>, static_cast<unsigned>(lists), kThreads, 0, stream, a);
}

}  // namespace lora

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
// reach.  The elements that reach it, usually little more than `keep`, are gathered
// and ranked by counting.  All keys of a chunk differ (value, then the lower token
// first), so order never depends on timing.
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

// Keys of a chunk's elements: the value, then the lower index first.  0 is below all.
struct Bf16Logits {
    using Key = uint32_t;
    static constexpr int kVec = 8;
    __device__ static float load(const void *p, int64_t i) {
        return bf16lo_to_f32(static_cast<const uint16_t *>(p)[i]);
    }
    __device__ static void unpack(uint4 v, float *x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) x[2 * e] = bf16lo_to_f32(w[e]), x[2 * e + 1] = bf16hi_to_f32(w[e]);
    }
    __device__ static Key key(float x, int32_t i) {
        return (ordered(x) & 0xffff0000u) | static_cast<uint32_t>(0xffff - i);
    }
    __device__ static int32_t index(Key k) { return 0xffff - static_cast<int32_t>(k & 0xffffu); }
    // (a negative value's ordered form is its complement: the low half was ones)
    __device__ static float value(Key k) {
        return from_ordered((k & 0x80000000u) ? k & 0xffff0000u : k | 0xffffu);
    }
};

struct Fp32Logits {
    using Key = uint64_t;
    static constexpr int kVec = 4;
    __device__ static float load(const void *p, int64_t i) { return static_cast<const float *>(p)[i]; }
    __device__ static void unpack(uint4 v, float *x) {
        x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    }
    __device__ static Key key(float x, int32_t i) {
        return (static_cast<uint64_t>(ordered(x)) << 32) | static_cast<uint32_t>(0xffff - i);
    }
    __device__ static int32_t index(Key k) { return 0xffff - static_cast<int32_t>(k & 0xffffu); }
    __device__ static float value(Key k) { return from_ordered(static_cast<uint32_t>(k >> 32)); }
};

template <class K>
__device__ __forceinline__ K shfl_max(K v, int o) {
    const K u = __shfl_xor_sync(0xffffffffu, v, o);
    return u > v ? u : v;
}

// The keep best of the request's lists, in order, to the outputs.
__device__ void join_request(const SelectArgs &a, int32_t r) {
    __shared__ double s_base[LORA_MAX_BEAMS];  // score minus the logarithm; NaN: no candidates
    __shared__ bool s_ended[LORA_MAX_BEAMS];   // (outputs may take the inputs' place)
    __shared__ uint64_t s_best, s_wkey[kThreads / 32];
    __shared__ uint32_t s_wid[kThreads / 32], s_id;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int32_t b = warp; b < a.beams; b += kThreads / 32) {
        const int32_t row = r * a.beams + b;
        const float2 *sums = a.sums + int64_t(row) * a.chunks;
        double top = -INFINITY, sum = 0.0;
        for (int32_t c = lane; c < a.chunks; c += 32) {
            const float2 v = __ldcg(sums + c);
            top = v.x > top ? v.x : top;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
        for (int32_t c = lane; c < a.chunks; c += 32) {
            const float2 v = __ldcg(sums + c);
            // (a chunk without a number above -inf has sum 0; a NaN or +inf makes the sum NaN)
            sum += v.y == 0.0f ? 0.0 : v.y * exp(v.x - top);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) {
            const double score = a.scores[row];
            const bool ended = a.ended != nullptr && a.ended[row] != 0;
            double base = ended ? score : score - (top + log(sum));
            if (!(base > -INFINITY && base < INFINITY)) base = NAN;
            s_base[b] = base;
            s_ended[b] = ended;
        }
    }
    __syncthreads();
    // one after the other: the best below the last one
    const int32_t per_row = a.chunks * a.keep, n = a.beams * per_row;
    uint64_t last_key = ~uint64_t(0);
    uint32_t last_id = 0;
    for (int32_t k = 0; k < a.keep; ++k) {
        uint64_t best = 0;
        uint32_t id = 0xffffffffu;  // beam * vocab + token
        for (int32_t i = tid; i < n; i += kThreads) {
            const int32_t b = i / per_row;
            const int64_t at = int64_t(r) * n + i;
            const int32_t token = __ldcg(a.ids + at);
            const double v = s_base[b] + __ldcg(a.values + at);
            if (token < 0 || !(v > -INFINITY)) continue;
            const uint64_t key = ordered(v);
            const uint32_t me = static_cast<uint32_t>(b) * a.vocab + token;
            if (!(key < last_key || (key == last_key && me > last_id && k > 0))) continue;
            if (key > best || (key == best && me < id)) best = key, id = me;
        }
        const auto better = [](uint64_t k2, uint32_t i2, uint64_t &k1, uint32_t &i1) {
            if (k2 > k1 || (k2 == k1 && i2 < i1)) k1 = k2, i1 = i2;
        };
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            better(__shfl_xor_sync(0xffffffffu, best, o), __shfl_xor_sync(0xffffffffu, id, o), best, id);
        if (lane == 0) s_wkey[warp] = best, s_wid[warp] = id;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < kThreads / 32; ++w) better(s_wkey[w], s_wid[w], best, id);
            s_best = best;
            s_id = id;
            const int64_t to = int64_t(r) * a.keep + k;
            const bool there = best != 0;
            const int32_t b = there ? static_cast<int32_t>(id / a.vocab) : 0, row = r * a.beams + b;
            const int32_t token = there ? static_cast<int32_t>(id - static_cast<uint32_t>(b) * a.vocab) : -1;
            const uint64_t u = best;
            const double v = __longlong_as_double(static_cast<long long>((u >> 63) ? u ^ (uint64_t(1) << 63) : ~u));
            a.parents[to] = there ? row : -1;
            a.tokens[to] = token;
            a.out_scores[to] = there ? static_cast<float>(v) : -INFINITY;
            a.out_ended[to] = there && (token == a.eos || s_ended[b]);
        }
        __syncthreads();
        last_key = s_best;
        last_id = s_id;
        __syncthreads();
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) beam_select_kernel(const SelectArgs a) {
    using Key = typename T::Key;
    constexpr int kVec = T::kVec;
    __shared__ float s_top[kThreads / 32], s_sum[kThreads / 32];
    __shared__ Key s_group[kGroups], s_keys[kGather], s_bound;
    __shared__ int32_t s_n;
    __shared__ bool s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t row = static_cast<int32_t>(blockIdx.x / a.chunks), chunk = static_cast<int32_t>(blockIdx.x % a.chunks);
    const int32_t r = row / a.beams;
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
        // thread t's vector u holds elements (u * 256 + t) * kVec - skew ..: whole vectors lie on 16 bytes
        const int64_t first = row * a.ld + v0;
        constexpr int kSize = 16 / kVec;
        const unsigned char *base = static_cast<const unsigned char *>(a.logits) + first * kSize;
        const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15) / kSize);
        constexpr int kVecs = kEach / kVec;
        float x[kEach + kVec];  // (one vector more: the skew)
        const auto load = [&](int u, int32_t v, float *to) {
            const int32_t i = v * kVec - skew;
            if (i >= 0 && i + kVec <= n) {
                T::unpack(ldg_cg(base + int64_t(i) * kSize), to);
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    to[e] = i + e >= 0 && i + e < n ? T::load(base, i + e) : -INFINITY;
            }
        };
#pragma unroll
        for (int u = 0; u < kVecs; ++u) load(u, u * kThreads + tid, x + u * kVec);
        // the last elements of a skewed chunk: one vector, one thread
        const bool more = skew > 0 && tid == 0;
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[kEach + e] = -INFINITY;
        if (more) load(kVecs, kVecs * kThreads, x + kEach);
        const auto index_of = [&](int e) {
            const int u = e / kVec;
            if (u == kVecs && !more) return -1;
            return (u * kThreads + tid) * kVec - skew + e % kVec;
        };
        float top = -INFINITY;
        Key best = 0;
#pragma unroll
        for (int e = 0; e < kEach + kVec; ++e) {
            top = fmaxf(top, x[e]);
            const int32_t i = index_of(e);
            const Key k = i >= 0 && i < n ? T::key(x[e], i) : 0;
            best = k > best ? k : best;
        }
        // groups' maxima, and the block's maximum and sum
        best = shfl_max(shfl_max(best, 1), 2);
        if ((lane & 3) == 0) s_group[tid >> 2] = best;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) s_top[warp] = top;
        if (tid == 0) s_n = 0;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, s_top[w]);
        const float ref = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < kEach + kVec; ++e) sum += ex2((x[e] - ref) * kLog2e);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s_sum[warp] = sum;
        // the keep-th largest of the groups' maxima
        if (tid < kGroups) {
            const Key me = s_group[tid];
            int above = 0;
            for (int j = 0; j < kGroups; ++j) above += s_group[j] > me || (s_group[j] == me && j < tid);
            if (above == a.keep - 1) s_bound = me;
        }
        __syncthreads();
        if (tid == 0) {
            float all = 0.0f;
            for (int w = 0; w < kThreads / 32; ++w) all += s_sum[w];
            a.sums[int64_t(row) * a.chunks + chunk] = make_float2(top, all);
        }
        const Key bound = s_bound > 0 ? s_bound : 1;  // fewer groups with elements than `keep`: all elements
#pragma unroll
        for (int e = 0; e < kEach + kVec; ++e) {
            const int32_t i = index_of(e);
            const Key k = i >= 0 && i < n ? T::key(x[e], i) : 0;
            if (k >= bound) {
                const int32_t at = atomicAdd(&s_n, 1);
                if (at < kGather) s_keys[at] = k;
            }
        }
        __syncthreads();
        const int32_t found = s_n;
        const auto put = [&](int32_t k, Key key) {
            a.values[list + k] = T::value(key);
            a.ids[list + k] = v0 + T::index(key);
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
                for (int e = 0; e < kEach + kVec; ++e) {
                    const int32_t i = index_of(e);
                    const Key key = i >= 0 && i < n ? T::key(x[e], i) : 0;
                    if (key < last && key > now) now = key;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) now = shfl_max(now, o);
                __syncthreads();
                if (lane == 0) s_group[warp] = now;
                __syncthreads();
                for (int w = 0; w < kThreads / 32; ++w) now = s_group[w] > now ? s_group[w] : now;
                last = now;
                if (tid == 0) put(k, now);
            }
        }
        for (int32_t k = min(n, a.keep) + tid; k < a.keep; k += kThreads) {
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

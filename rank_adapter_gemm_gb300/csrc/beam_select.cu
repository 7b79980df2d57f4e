// Selection of beam search (lora_beam_select).
//
// What it must read is the logits, once: HBM bounds it, with one exponential an
// element.  A block takes a part of a row, in chunks that its threads hold in
// registers, the next one loading meanwhile, and leaves what a selection can need of it:
// maximum, sum of exponentials, and the `keep` largest.  The block that arrives last at
// a request joins them: the rows' logarithms, then the `keep` best of all lists.
//
// The largest of a part are found through a bound: of 64 groups of threads, the keep-th
// largest of the groups' maxima over the first chunk is one that at least `keep` elements
// reach.  The elements that reach it, of all chunks a few times `keep`, in few threads,
// are gathered and ranked by counting; where there are too many (equal or rising ones, a first
// chunk full of a mask's finite value) they are taken one by one, a pass over the part each (the call
// below with all but 1 in 10,000 logits at the type's lowest value 131 us; with 99 in 100 as without).  All keys differ (value, then the lower token first), so order
// never depends on timing.  Between the first chunk and the last no thread waits for another.
//
// A thread's sum is two fp32 numbers (the second holds what adding up the chunks rounds off),
// against a reference that follows its maximum at a distance (kMove): neither the additions'
// roundings nor those of moving the reference pile up over a long row, and so for the parts of a
// row.  In one number against the maximum itself, equal logits below 512 larger ones were off by
// up to 2^-15 over 2^22 tokens and 2^-13 over 2^24; so they are within 2^-21 at every length, in the same
// time.  Candidates are compared in 64 bits: scores of different beams meet there, and a
// rounding to fp32 would decide between them.
//
// Measured, graph replay: 32 requests of 4 beams over 128,256 tokens (29 MB are read: a tenth of
// the beams has ended) 18.4 us, 1.6 TB/s over all: about 12 us pass until the last part is done
// (SMs with four blocks take longer than those with three, and exponentials 4 us), 5 in the
// request's join, a chain of loads, barriers and rankings.  One request of 4 beams over 32,000 fp32 logits
// 8.0 us.  A chunk a block instead of parts: 23.9.
#include <algorithm>

#include "attend.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kGroups = 64;   // groups of 4 neighbouring threads
constexpr int kGather = 1024;  // gathered keys at most; more take the slow way
// How far a thread's maximum may grow above its reference: terms stay below 2^6, and terms that a
// reference has moved k times for weigh at most e^(-k kMove), so few roundings count.
constexpr float kMove = 4.0f;

struct SelectArgs {
    const void *logits;
    int64_t ld;
    const float *scores;
    const int32_t *ended;
    int32_t *parents, *tokens, *out_ended;
    float *out_scores;
    int32_t *counters;   // a request
    float2 *sums;        // reference and sum of each row's parts
    float *values;       // the largest of each part, by request and rank
    int32_t *ids;        // and their tokens
    int32_t beams, vocab, keep, eos, parts, part_vecs;
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
    constexpr uint64_t kSign = uint64_t(1) << 63;
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x));  // (64-bit arithmetic is slow here)
    return u <= kSign ? u | kSign : ~u;
}

// A thread's elements of a chunk in 16 registers.
struct Bf16Logits {
    static constexpr int kVec = 8, kEach = 32;
    static constexpr uint32_t kNone = 0xff80ff80u;  // -inf
    __device__ static float value(const uint32_t (&w)[16], int e) {
        return (e & 1) ? bf16hi_to_f32(w[e / 2]) : bf16lo_to_f32(w[e / 2]);
    }
    __device__ static uint32_t element(const void *p, int64_t i) { return static_cast<const uint16_t *>(p)[i]; }
    // element e of a vector
    __device__ static void put(uint32_t *w, int e, uint32_t v) {
        w[e / 2] = __byte_perm(w[e / 2], v, (e & 1) ? 0x5410 : 0x3254);
    }
    __device__ static float top(const uint32_t (&w)[16]) {
        uint32_t m = w[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(w[i]));
        return fmaxf(bf16lo_to_f32(m), bf16hi_to_f32(m));
    }
};

struct Fp32Logits {
    static constexpr int kVec = 4, kEach = 16;
    static constexpr uint32_t kNone = 0xff800000u;
    __device__ static float value(const uint32_t (&w)[16], int e) { return __uint_as_float(w[e]); }
    __device__ static uint32_t element(const void *p, int64_t i) { return static_cast<const uint32_t *>(p)[i]; }
    __device__ static void put(uint32_t *w, int e, uint32_t v) { w[e] = v; }
    __device__ static float top(const uint32_t (&w)[16]) {
        float m = __uint_as_float(w[0]);
#pragma unroll
        for (int i = 1; i < 16; ++i) m = fmaxf(m, __uint_as_float(w[i]));
        return m;
    }
};

// An element's key: the value, then the lower token first; 0 is below all.
__device__ __forceinline__ uint64_t key_of(float x, int32_t token) {
    return (static_cast<uint64_t>(ordered(x)) << 32) | ~static_cast<uint32_t>(token);
}

template <class K>
__device__ __forceinline__ K shfl_max(K v, int o) {
    const K u = __shfl_xor_sync(0xffffffffu, v, o);
    return u > v ? u : v;
}

// The keep-th largest of 64 group values (s_group, 16-byte aligned), by counting; by the whole
// block, with a barrier in front and behind.  Groups without elements hold the least value.
__device__ __forceinline__ uint32_t bound_of(const uint32_t *s_group, uint32_t *s_bound, int32_t keep) {
    __syncthreads();
    if (threadIdx.x < kGroups) {
        const int tid = threadIdx.x;
        const uint32_t me = s_group[tid];
        int above = 0;
#pragma unroll
        for (int j = 0; j < kGroups; j += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(s_group + j);
            above += (v.x > me || (v.x == me && j < tid)) + (v.y > me || (v.y == me && j + 1 < tid)) +
                     (v.z > me || (v.z == me && j + 2 < tid)) + (v.w > me || (v.w == me && j + 3 < tid));
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

// A number >= 0 added to sum + low: low takes what sum rounds off.  (Exactly where the number is the
// smaller one; else it is off by half a unit of it, and the sum has at least doubled.)
__device__ __forceinline__ void add_to(float &sum, float &low, float x) {
    const float now = __fadd_rn(sum, x);
    low += __fsub_rn(x, __fsub_rn(now, sum));
    sum = now;
}

// top + ln sum, in 64 bits but for the logarithm of a number near 1 (2^-25).
__device__ __forceinline__ double log_sum(float top, float sum) {
    const int32_t bits = __float_as_int(sum), e = ((bits - 0x3f400000) >> 23);  // sum / 2^e in [3/4, 3/2)
    if (!(sum > 0.0f && sum < INFINITY)) return top + logf(sum);  // (a sum with a term of 1 is 0, NaN or at least 1)
    return top + (e * 0.693147180559945309417 + static_cast<double>(logf(__int_as_float(bits - (e << 23)))));
}

// The keep best of the request's lists, in order, to the outputs.
__device__ void join_request(const SelectArgs &a, int32_t r) {
    constexpr long long kNoBase = 0x7ff8000000000000;
    constexpr int kHeld = 8;                   // candidates a thread holds
    __shared__ double s_base[LORA_MAX_BEAMS];  // score minus the logarithm; kNoBase: no candidates
    __shared__ bool s_ended[LORA_MAX_BEAMS];   // (outputs may take the inputs' place)
    __shared__ __align__(16) uint32_t s_group[kGroups];
    __shared__ uint32_t s_bound;
    __shared__ Candidate s_found[kGather], s_best[kThreads / 32];
    __shared__ int32_t s_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t lists = a.beams * a.parts, all = lists * a.keep;
    const int64_t list0 = int64_t(r) * all;
    // the first candidates, loaded beside what makes values of them
    float value[kHeld];
    int32_t token[kHeld];
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
        const int32_t i = tid + h * kThreads;
        value[h] = i < all ? __ldcg(a.values + list0 + i) : -INFINITY;
        token[h] = i < all ? __ldcg(a.ids + list0 + i) : -1;
    }
    if (tid == 0) s_n = 0;
    for (int32_t b = warp; b < a.beams; b += kThreads / 32) {
        const int32_t row = r * a.beams + b;
        const float2 *sums = a.sums + int64_t(row) * a.parts;
        float2 mine = lane < a.parts ? __ldcg(sums + lane) : make_float2(-INFINITY, 0.0f);
        const float score = lane == 0 ? a.scores[row] : 0.0f;
        const bool ended = lane == 0 && a.ended != nullptr && a.ended[row] != 0;
        float top = mine.x;
        for (int32_t c = lane + 32; c < a.parts; c += 32) top = fmaxf(top, __ldcg(sums + c).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float sum = 0.0f, low = 0.0f;
        for (int32_t c = lane; c < a.parts; c += 32) {
            if (c != lane) mine = __ldcg(sums + c);
            // (a part without a number above -inf has sum 0; a NaN or +inf makes the sum NaN)
            if (mine.y != 0.0f) add_to(sum, low, mine.y * ex2((mine.x - top) * kLog2e));
        }
        sum += low;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) {
            double base = ended ? score : score - log_sum(top, sum);
            if (!(base > -INFINITY && base < INFINITY)) base = __longlong_as_double(kNoBase);
            s_base[b] = base;
            s_ended[b] = ended;
        }
    }
    __syncthreads();
    // candidate i of the request; key 0: none
    const auto made = [&](int32_t i, float x, int32_t id) {
        const int32_t b = i % lists / a.parts;
        const double base = s_base[b];
        const bool there = id >= 0 && x > -INFINITY && __double_as_longlong(base) != kNoBase;
        return Candidate{there ? ordered(base + x) : 0, static_cast<uint32_t>(b) * a.vocab + id};
    };
    const auto loaded = [&](int32_t i) { return made(i, __ldcg(a.values + list0 + i), __ldcg(a.ids + list0 + i)); };
    Candidate held[kHeld];
    uint64_t best = 0;
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
        held[h].key = 0;
        if (h * kThreads >= all) continue;
        held[h] = made(tid + h * kThreads, value[h], token[h]);
        best = max(best, held[h].key);
    }
#pragma unroll 4
    for (int32_t i = tid + kHeld * kThreads; i < all; i += kThreads) best = max(best, loaded(i).key);
    // a bound that `keep` candidates reach: of 64 groups of threads, their best (its upper half)
    const uint32_t group = shfl_max(shfl_max(static_cast<uint32_t>(best >> 32), 1), 2);
    if ((lane & 3) == 0) s_group[tid >> 2] = group;
    const uint64_t bound = max(uint64_t(bound_of(s_group, &s_bound, a.keep)) << 32, uint64_t(1));
    const auto gather = [&](const Candidate &c) {
        if (c.key < bound) return;
        const int32_t at = atomicAdd(&s_n, 1);
        if (at < kGather) s_found[at] = c;
    };
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
        if (h * kThreads < all) gather(held[h]);
#pragma unroll 4
    for (int32_t i = tid + kHeld * kThreads; i < all; i += kThreads) gather(loaded(i));
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
        for (int32_t i = tid; i < all; i += kThreads) {
            const Candidate c = loaded(i);
            if (c.key >= bound && last.before(c) && c.before(now)) now = c;
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
    constexpr int kVec = T::kVec, kEach = T::kEach, kVecs = kEach / kVec, kSize = 16 / kVec;
    __shared__ __align__(16) uint32_t s_group[kGroups];
    __shared__ uint32_t s_top[kThreads / 32], s_bound;
    __shared__ float s_sum[kThreads / 32];
    __shared__ uint64_t s_keys[kGather], s_best[kThreads / 32];
    __shared__ int32_t s_n;
    __shared__ bool s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t row = static_cast<int32_t>(blockIdx.x / a.parts), part = static_cast<int32_t>(blockIdx.x % a.parts);
    const int32_t r = row / a.beams;
    if (tid == 0) s_n = 0;
    wait_for_previous();
    const bool ended = a.ended != nullptr && a.ended[row] != 0;
    // where this part's k-th largest goes: lists stand side by side, so that neighbours are of one rank
    const int32_t lists = a.beams * a.parts;
    const int64_t list = int64_t(r) * lists * a.keep + (row - r * a.beams) * a.parts + part;
    const auto place = [&](int32_t k) { return list + int64_t(k) * lists; };
    if (ended) {
        for (int32_t k = tid; k < a.keep; k += kThreads) {
            const bool here = part == 0 && k == 0;
            a.values[place(k)] = here ? 0.0f : -INFINITY;
            a.ids[place(k)] = here ? a.eos : -1;
        }
        if (tid == 0) a.sums[int64_t(row) * a.parts + part] = make_float2(0.0f, 1.0f);
    } else {
        // Vectors lie on 16 bytes: the row's elements are counted from `skew` elements before it.  The
        // part's vectors start at v0; thread t's vector u of chunk c is v0 + c kChunkVecs + u 256 + t.
        const unsigned char *base = static_cast<const unsigned char *>(a.logits) + row * a.ld * kSize;
        const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15) / kSize);
        constexpr int kChunkVecs = kThreads * kVecs;
        const int32_t v0 = part * a.part_vecs, v1 = min(v0 + a.part_vecs, (a.vocab + skew + kVec - 1) / kVec);
        const int32_t chunks = (v1 - v0 + kChunkVecs - 1) / kChunkVecs;
        const auto load = [&](int32_t c, uint32_t (&w)[16]) {
#pragma unroll
            for (int u = 0; u < kVecs; ++u) {
                const int32_t v = v0 + c * kChunkVecs + u * kThreads + tid, i = v * kVec - skew;
                uint32_t *to = w + 4 * u;
                if (v < v1 && i >= 0 && i + kVec <= a.vocab) {
                    const uint4 x = ldg_cg(base + int64_t(i) * kSize);
                    to[0] = x.x, to[1] = x.y, to[2] = x.z, to[3] = x.w;
                } else {
                    to[0] = to[1] = to[2] = to[3] = T::kNone;
                    if (v < v1) {
#pragma unroll
                        for (int e = 0; e < kVec; ++e)
                            if (i + e >= 0 && i + e < a.vocab) T::put(to, e, T::element(base, i + e));
                    }
                }
            }
        };
        const auto token_of = [&](int32_t c, int e) {
            return (v0 + c * kChunkVecs + e / kVec * kThreads + tid) * kVec - skew + e % kVec;
        };
        uint32_t w[16], next[16];
        if (chunks > 0) load(0, w);
        float m = -INFINITY, sum = 0.0f, low = 0.0f, bound = INFINITY;  // of this thread: its reference, its terms' sum
        for (int32_t c = 0; c < chunks; ++c) {
            if (c + 1 < chunks) load(c + 1, next);
            const float top = T::top(w);
            if (c == 0) {
                const uint32_t best = shfl_max(shfl_max(ordered(top), 1), 2);
                if ((lane & 3) == 0) s_group[tid >> 2] = best;
                bound = from_ordered(bound_of(s_group, &s_bound, a.keep));
            }
            if (top > m + kMove) {
                const float f = m > -INFINITY ? ex2((m - top) * kLog2e) : 0.0f;
                sum *= f;
                low *= f;
                m = top;
            }
            const float ref = m == -INFINITY ? 0.0f : m;
            const uint64_t by2 = pack2(kLog2e, kLog2e), ref2 = pack2(-ref, -ref);
            uint64_t sums[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < kEach; e += 2) {
                // the difference first: it is exact near the maximum, where the terms count
                float d0, d1;
                unpack2(mul2(add2(pack2(T::value(w, e), T::value(w, e + 1)), ref2), by2), d0, d1);
                sums[e / 2 & 1] = add2(sums[e / 2 & 1], pack2(ex2(d0), ex2(d1)));
            }
            float even, odd;
            unpack2(add2(sums[0], sums[1]), even, odd);
            add_to(sum, low, even + odd);
            // few threads have an element that reaches the bound
            if (top >= bound && top > -INFINITY) {
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    const float x = T::value(w, e);
                    if (x >= bound && x > -INFINITY) {
                        const int32_t at = atomicAdd(&s_n, 1);
                        if (at < kGather) s_keys[at] = key_of(x, token_of(c, e));
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = next[i];
        }
        // the block's reference and sum
        sum += low;
        uint32_t best = __reduce_max_sync(0xffffffffu, ordered(m));
        if (lane == 0) s_top[warp] = best;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) best = max(best, s_top[i]);
        const float all_top = from_ordered(best);
        if (m > -INFINITY) sum *= ex2((m - all_top) * kLog2e);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s_sum[warp] = sum;
        __syncthreads();
        if (tid == 0) {
            float all = 0.0f;
#pragma unroll
            for (int i = 0; i < kThreads / 32; i += 4) all += (s_sum[i] + s_sum[i + 1]) + (s_sum[i + 2] + s_sum[i + 3]);
            a.sums[int64_t(row) * a.parts + part] = make_float2(all_top, all);
        }
        const int32_t found = s_n;
        const auto put = [&](int32_t k, uint64_t key) {
            a.values[place(k)] = from_ordered(static_cast<uint32_t>(key >> 32));
            a.ids[place(k)] = static_cast<int32_t>(~static_cast<uint32_t>(key));
        };
        if (found <= kGather) {
            for (int32_t i = tid; i < found; i += kThreads) {
                const uint64_t me = s_keys[i];
                int32_t above = 0;
                for (int32_t j = 0; j < found; ++j) above += s_keys[j] > me;
                if (above < a.keep) put(above, me);
            }
        } else {
            // one after the other: the largest below the last one
            uint64_t last = ~uint64_t(0);
            for (int32_t k = 0; k < a.keep; ++k) {
                uint64_t now = 0;
                for (int32_t c = 0; c < chunks; ++c) {
                    load(c, w);
#pragma unroll
                    for (int e = 0; e < kEach; ++e) {
                        const float x = T::value(w, e);
                        const uint64_t key = x > -INFINITY ? key_of(x, token_of(c, e)) : 0;
                        if (key < last && key > now) now = key;
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) now = shfl_max(now, o);
                __syncthreads();
                if (lane == 0) s_best[warp] = now;
                __syncthreads();
                for (int i = 0; i < kThreads / 32; ++i) now = max(now, s_best[i]);
                last = now;
                if (tid == 0) put(k, now);
            }
        }
        for (int32_t k = min(found, a.keep) + tid; k < a.keep; k += kThreads) {
            a.values[place(k)] = -INFINITY;
            a.ids[place(k)] = -1;
        }
    }
    // the last block of the request joins its lists
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        const int32_t all = a.beams * a.parts;
        s_last = atomicAdd(a.counters + r, 1) == all - 1;
        if (s_last) a.counters[r] = 0;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    join_request(a, r);
}

// Vectors of a row, at any alignment, and its parts: as many as fill the GPU's places for
// blocks once (4 an SM), of equal size, a chunk at least.  32 x 4 rows of 128,256: 4 parts 19.5
// us, 2 23.0, 8 20.5, 16 (a chunk each) 23.9; 4 x 16 fp32 rows of 131,072: 9 parts 26.3, 4 26.5, 38 52.
constexpr int32_t kPlaces = 4 * 152;
struct Parts {
    int32_t parts, vecs;
};
Parts parts_of(int32_t rows, int32_t vocab, bool fp32) {
    const int32_t vec = fp32 ? Fp32Logits::kVec : Bf16Logits::kVec;
    const int32_t chunk = kThreads * (fp32 ? Fp32Logits::kEach : Bf16Logits::kEach) / vec;
    const int32_t vecs = (vocab + 2 * vec - 2) / vec, chunks = (vecs + chunk - 1) / chunk;
    const int32_t parts = std::max(1, std::min(chunks, kPlaces / rows));
    return {parts, (vecs + parts - 1) / parts};
}
size_t up128(size_t b) { return (b + 127) & ~size_t(127); }

// Their place does not depend on the call, so calls of other sizes find them as they were.
constexpr size_t kCounters = size_t(LORA_MAX_SEQS) * 4;

}  // namespace

// Counters (a request), then sums (a part of a row), values and tokens (`keep` a part).
size_t beam_select_workspace_bytes(int32_t n_req, int32_t beams, int32_t keep, int32_t vocab) {
    const int32_t rows = std::max(1, n_req * beams);
    const size_t lists = size_t(n_req) * beams * parts_of(rows, vocab, true).parts;  // (bf16 rows have no more)
    return kCounters + up128(lists * 8) + 2 * up128(lists * keep * 4);
}

cudaError_t launch_beam_select(const void *logits, int64_t ld, bool fp32, int32_t n_req, int32_t beams, int32_t vocab,
                               int32_t keep, const float *scores, const int32_t *ended, int32_t eos, int32_t *parents,
                               int32_t *tokens, float *out_scores, int32_t *out_ended, void *ws, cudaStream_t stream) {
    const Parts p = parts_of(n_req * beams, vocab, fp32);
    const size_t lists = size_t(n_req) * beams * p.parts;
    char *at = static_cast<char *>(ws);
    SelectArgs a{logits, ld, scores, ended, parents, tokens, out_ended, out_scores, reinterpret_cast<int32_t *>(at),
                 nullptr, nullptr, nullptr, beams, vocab, keep, eos, p.parts, p.vecs};
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

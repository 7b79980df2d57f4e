// What lora_attend_shared shares, and which blocks compute it.  Worked out from the
// lengths by every block that needs it, alike: no launch and no wait for it.
#pragma once

#include "attend.cuh"

namespace lora {

constexpr int kPrefixRows = 256, kPrefixKeys = 128;  // of a step of the prefix kernel
constexpr int kPrefixBlocks = 160, kOwnWarps = 8 * 160;  // at most: of the prefix kernel, of the own keys' kernel

// Opening a piece (its queries, its result) costs a block of the prefix kernel about as
// much as kPrefixOpen steps: every segment counts as so many more, in front of the real ones.
constexpr int kPrefixOpen = 6;

// What sharing must save, of each SM, to be worth the prefix kernel and the join.
constexpr int32_t kSharedFixedNs = 3000;

// Calls that take an SM up to kSharedLongNs compute prefixes on some SMs and own keys on the
// others, so that one starts up beside the other; longer ones take all SMs for each in turn.
// (Measured, 32 groups of 4 requests behind 2,000 tokens: 97 us in turn, 107 beside each other; 8
// of 4 behind 8,000 80 and 74; 64 requests behind 8,000 73 and 54.)
constexpr int32_t kSharedLongNs = 50000, kSharedLateNs = 6000;

// The call's groups, and the costs that decide what is shared (ns, of one SM).
struct Groups {
    const int32_t *offsets, *lens;
    int32_t n_groups, tile_rows;       // rows a tile of the decode path
    bool always;                       // whatever they are
    int32_t step_one, step_two;        // a step of the prefix kernel with up to 128 rows, with more
    int32_t own, first;                // 128 keys of a tile of the decode path; and where no other tile reads them
    int32_t own_open;                  // keys that a tile of it counts more
};

// In shared memory: by request its first row; by group the rest.
struct GroupPlan {
    int32_t *rows;            // n_seq + 1
    int32_t *offsets;         // n_groups + 1
    int32_t *prefix, *lo, *lead;  // its keys' end (0: shares nothing) and first, the request whose table row holds them
    int32_t *tiles;           // of the decode path, over its requests
    __device__ GroupPlan(int32_t *scratch, int32_t n, int32_t n_seq)
        : rows(scratch), offsets(rows + n_seq + 1), prefix(offsets + n + 1), lo(prefix + n), lead(lo + n),
          tiles(lead + n) {}
    __host__ __device__ static constexpr size_t bytes(int32_t n, int32_t n_seq) { return (size_t(5) * n + n_seq + 2) * 4; }
};

// How many blocks compute prefixes (0: nothing is shared) and own keys.
struct Blocks {
    int32_t prefix, own;
};

// Steps of a group's prefix (any row tile and key head).
__device__ __forceinline__ int32_t prefix_steps(int32_t lo, int32_t prefix) {
    return prefix > lo ? (prefix - 1) / kPrefixKeys - lo / kPrefixKeys + 1 : 0;
}

// The last of n rising entries that is <= x, from 0.
template <class V>
__device__ __forceinline__ int32_t last_at_most(const V *rising, int32_t n, int64_t x) {
    int32_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (rising[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Units (steps and openings) of a group's prefix in the call's order of work: key head, row tile, step.
__device__ __forceinline__ int64_t prefix_units(const AttendArgs &a, const GroupPlan &p, int32_t g) {
    const int32_t steps = prefix_steps(p.lo[g], p.prefix[g]);
    if (steps == 0) return 0;
    const int64_t rows = int64_t(p.rows[p.offsets[g + 1]] - p.rows[p.offsets[g]]) * a.group;
    return (rows + kPrefixRows - 1) / kPrefixRows * a.kv.n_kv * (steps + kPrefixOpen);
}

// The request's group, -1: none.  (bad: the groups' or the rows' offsets are out of order or range.)
__device__ __forceinline__ int32_t group_of(const GroupPlan &p, int32_t n_groups, bool bad, int32_t i) {
    if (bad || n_groups == 0 || i < p.offsets[0] || i >= p.offsets[n_groups]) return -1;
    return last_at_most(p.offsets, n_groups, i);
}

// By the whole block of NT threads.  Sums over it are taken in s_sum (4 NT / 32 entries).  Sets
// the plan of every group; returns how many of `grid` blocks compute what.  Ends with a barrier.
template <int NT>
__device__ Blocks plan_groups(const AttendArgs &a, const Groups &w, const GroupPlan &p, int64_t *s_sum, int32_t grid,
                              bool report, bool *bad_out) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const auto len_at = [&](int32_t i) { return i < a.n_seq ? __ldcg(a.kv_lens + i) : 0; };
    const auto row_at = [&](int32_t i) { return i <= a.n_seq ? __ldcg(a.q_offsets + i) : 0; };
    int32_t len = len_at(tid), row = row_at(tid);  // (loads that need no other ones together)
    for (int32_t g = tid; g <= w.n_groups && w.n_groups > 0; g += NT) p.offsets[g] = __ldcg(w.offsets + g);
    for (int32_t g = tid; g < w.n_groups; g += NT) {
        p.prefix[g] = INT32_MAX;
        p.lead[g] = INT32_MAX;
        p.tiles[g] = 0;
        const int32_t given = __ldcg(w.lens + g);
        p.lo[g] = given;  // for now
        if (given < 0 && report) report_error(a.err, LORA_ERR_INVALID_ARG);
    }
    for (int32_t i = tid; i <= a.n_seq; i += NT) {
        p.rows[i] = row;
        row = row_at(i + NT);
    }
    __syncthreads();
    bool bad = false;
    for (int32_t g = tid; g < w.n_groups; g += NT)
        bad = bad || p.offsets[g] < 0 || p.offsets[g + 1] < p.offsets[g] || p.offsets[g + 1] > a.n_seq;
    bad = __syncthreads_or(bad);
    if (bad && report && tid == 0) report_error(a.err, LORA_ERR_INVALID_ARG);
    // requests: what each has cached before its rows, its tiles; and the cost of all own keys
    const auto tiles_of = [&](int32_t n) { return (int64_t(n) * a.group + w.tile_rows - 1) / w.tile_rows; };
    int64_t own = 0;  // tiles x keys of the decode path, all requests on their own
    // A group's rows are those between its ends, and a token's request is found by a search in the
    // offsets: both need them to rise all over the call, or nothing is shared.
    bool falls = false;
    for (int32_t i = tid; i < a.n_seq; i += NT) {
        falls = falls || p.rows[i] < 0 || p.rows[i + 1] < p.rows[i] || p.rows[i + 1] > a.T;
        const RequestRows r = check_request(a, p.rows[i], p.rows[i + 1], len);
        len = len_at(i + NT);
        if (r.n == 0) continue;
        const int64_t tiles = tiles_of(r.n);
        own += tiles * (w.own_open + (a.window > 0 ? min(int64_t(r.len), int64_t(a.window) + r.n) : r.len));
        const int32_t g = group_of(p, w.n_groups, bad, i);
        if (g < 0) continue;
        atomicMin(&p.prefix[g], r.len - r.n);
        atomicMin(&p.lead[g], i);
        atomicAdd(&p.tiles[g], static_cast<int32_t>(min(tiles, int64_t(1) << 18)));
    }
    bad = __syncthreads_or(falls) || bad;
    *bad_out = bad;
    // groups: the prefix, and what sharing it saves
    int64_t sums[4] = {0, 0, 0, own};  // ns saved, ns of prefixes, tiles x keys that are not own any more
    for (int32_t g = tid; g < w.n_groups; g += NT) {
        const int32_t ctx = p.prefix[g], given = p.lo[g];
        int32_t prefix = 0, lo = 0;
        const int32_t lead = p.lead[g], rows_of_group = bad ? 0 : p.rows[p.offsets[g + 1]] - p.rows[p.offsets[g]];
        // more rows than one request has (seen from the offsets: counting requests costs a call of 64 in a group 1 us)
        if (lead != INT32_MAX && rows_of_group > p.rows[lead + 1] - p.rows[lead]) {
            prefix = max(0, min(given, ctx));
            if (a.window > 0) lo = static_cast<int32_t>(max(int64_t(0), int64_t(ctx) - a.window + 1));
            if (lo >= prefix) prefix = lo = 0;  // no row sees any of it
            if (prefix > 0) {
                const int64_t rows = int64_t(rows_of_group) * a.group, steps = prefix_steps(lo, prefix);
                const int64_t here = (rows + kPrefixRows - 1) / kPrefixRows * (steps + kPrefixOpen) *
                                     (rows > kPrefixRows / 2 ? w.step_two : w.step_one);
                const int64_t keys = int64_t(p.tiles[g]) * (prefix - lo);
                const int64_t there = (keys * w.own + int64_t(prefix - lo) * w.first) / kPrefixKeys;
                if (here < there || w.always) {
                    sums[0] += there - here;
                    sums[1] += here;
                    sums[2] += keys;
                } else {
                    prefix = lo = 0;
                }
            }
        }
        p.prefix[g] = prefix;
        p.lo[g] = lo;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sums[e] += __shfl_xor_sync(0xffffffffu, sums[e], o);
        if (lane == 0) s_sum[e * (NT / 32) + warp] = sums[e];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        sums[e] = 0;
        for (int i = 0; i < NT / 32; ++i) sums[e] += s_sum[e * (NT / 32) + i];
    }
    __syncthreads();
    // not worth the prefix kernel's and the join's time
    if (sums[1] == 0 || grid < 2 || (!w.always && sums[0] * a.kv.n_kv < int64_t(kSharedFixedNs) * grid)) {
        for (int32_t g = tid; g < w.n_groups; g += NT) p.prefix[g] = p.lo[g] = 0;
        __syncthreads();
        return {0, grid};
    }
    const int64_t rest = max(int64_t(1), (sums[3] - sums[2]) * (w.own + w.first) / kPrefixKeys), all = sums[1] + rest;
    if (all * a.kv.n_kv > int64_t(kSharedLongNs) * grid) return {grid, grid};
    // (the prefix kernel's first scores come kSharedLateNs later than the other kernel's)
    const int64_t late = min(sums[1], rest) * kSharedLateNs / (all * a.kv.n_kv) * grid, cost = sums[1] + late;
    const int32_t blocks = max(1, min(grid - 1, static_cast<int32_t>((grid * cost + (cost + rest) / 2) / (cost + rest))));
    return {blocks, grid - blocks};
}

}  // namespace lora

// Attention of few rows a request over the paged cache (LORA_ATTEND_DECODE).
//
// What it must read is the cache: 2 head_dim elements a key and key head, for
// group * rows dot products each, so HBM bandwidth bounds it.  The split below
// therefore spreads the bytes evenly whatever the lengths, and keeps copies in
// flight at all times:
//   - A segment is one (request, key head, tile of up to ROWS query rows), a
//     step 32 of its keys.  All steps of the call, in order, are cut into equal
//     shares, one a warp: a long request spreads over the whole GPU, many short
//     ones share a warp.  Every block finds its shares by a prefix sum over the
//     requests' lengths, so no plan has to be built or kept.
//   - A warp streams its steps' k and v through a private ring of cp.async
//     stages with no barrier between warps; the copies run ahead over segment
//     boundaries.  Rows are gathered key by key through the block table, so any
//     page size and any strides go the same way.
//   - The running maximum, sum and output stay in fp32 registers; both products
//     are warp MMAs (m16n8k16), which at 16 rows a tile need a fraction of the
//     time of the copies.
//   - A segment that one warp covers is written at once.  The others leave
//     (maximum, sum, output) partials: after the last step the block joins those
//     of its own warps, and the last block to arrive at a segment joins the
//     blocks', always in the order of the keys, so results do not depend on
//     timing.  Nothing waits.
//
// Weights are rounded for the second product: to f16 (11 bits) against an e4m3
// cache, scaled by 2^12 so that weights down to 2^-26 of the largest keep them
// all; against a bf16 cache to two bf16 parts, value and remainder (16 bits).
// With at most 8 rows the remainder goes into the MMA's unused rows 8..15 and
// costs nothing.  An e4m3 code is exact in f16; a query row is scaled by a power
// of two into f16, exact to 2^-24 of its largest element.
//
// Measured, 32 / 8 heads of 128, one row a request, graph replay: 256 requests of
// 4,096 tokens over bf16 629 us, 6.8 TB/s (a plain copy: 6.8), over e4m3 335 us, 6.4;
// one request of 131,071 tokens 88 us, 6.1; 64 requests of 108,700 tokens together
// 76 us, 5.8: about 5 us pass until every SM streams and as many in the joins.  One
// request of 100 tokens 7.6 us: a chain of dependent loads.  With 16 rows a tile over
// e4m3 the work between the copies bounds it instead: 64 requests of 4 rows and
// 108,700 tokens 62 us, 3.6 TB/s.
//
// The same kernel computes the requests' own keys where a prefix is shared
// (lora_attend_shared, SHARED): a request's keys then start at its `shared`, and its
// rows go to partials for the join with the prefix's.
#pragma once

#include <type_traits>

#include <cuda_fp16.h>

#include "attend.cuh"
#include "shared_plan.cuh"
#include "tc.cuh"

namespace lora {

namespace {

constexpr int kMaxGrid = 160;
constexpr int kSmemMax = 227 * 1024;
constexpr int kWarps = 8;
static_assert(kMaxGrid * kWarps == kOwnWarps, "the join's bound");
constexpr int kPrefixMax = ((LORA_MAX_SEQS + 1) * 4 + 127) & ~127;  // the requests' step prefix

template <int HD, bool E4M3, int ROWS, bool SHARED = false>
struct Config {
    static constexpr int kRowB = HD * (E4M3 ? 1 : 2);  // bytes of a key
    static constexpr int kChunks = kRowB / 16;         // 16-byte pieces of a key
    // Keys a step: 8 KB of k where the scores' registers allow, so that the work
    // around the products (maxima, waits, addresses) is spread over more keys.
    static constexpr int kKeys = ROWS == 32 || kRowB == 256 ? 32 : 64;
    static constexpr int kTileB = kKeys * kRowB;       // k, or v, of a step
    // A partial: maxima and sums of ROWS rows, then their outputs, fp32.
    static constexpr int kPartial = ROWS * (HD + 2);
    // A warp's query fragments in shared memory: with 32 rows there are no registers for them.
    static constexpr int kQBytes = ROWS == 32 ? (HD / 16) * 2 * 512 : 0;
    // Tiles of a warp's ring: all the memory that the longest prefix leaves.
    static constexpr int kRoom = (kSmemMax - 1024 - (SHARED ? 2 : 1) * kPrefixMax) / kWarps - kQBytes;
    static constexpr int kTiles = kRoom / kTileB < 9 ? kRoom / kTileB : 9;
    static constexpr int kWarpB = kQBytes + kTiles * kTileB;
    static_assert(kTiles >= 2 && kPartial * 4 <= kWarpB, "ring");
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// Two e4m3 codes (low 16 bits) to two f16, exact.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Byte offset of a 16-byte piece inside a k or v tile: pieces are XORed with the
// row so that eight rows at one piece fall in different banks.
template <int CHUNKS>
__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
    if constexpr (CHUNKS == 4) return row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
    return row * (CHUNKS * 16) + ((piece ^ (row & 7)) << 4);
}

// The groups of requests that share a prefix, and the partials of their rows for the join with
// it.  Of row (head T + token) group + head in group, by the warp that has its segment's first
// step: reference, sum, (first of the warps with its other pieces) << 5 | row of the tile, and
// how many they are; and its outputs, four dims of all rows together.  The other warps leave
// theirs in the place of their partial: reference and sum of ROWS rows, outputs alike.
struct OwnRows {
    Groups groups;
    float4 *sums;
    float *outs;
    const int32_t *blocks;  // the prefix kernel's word on how many blocks take part, 0 until it is there; null:
                            // that kernel does not run, nothing is shared
    int32_t *live;          // the join's word on whether there is anything to join; written where this kernel refuses
};

struct DecodeRows : RequestRows {
    int32_t shared;
};

// Data that a kernel before wrote, where this kernel does not begin with a wait.
template <bool PAST, class V>
__device__ __forceinline__ V load_past_l1(const V *p) {
    return PAST ? __ldcg(p) : *p;
}

// shared: by request, the keys that are not this call's.
template <bool SHARED>
__device__ __forceinline__ DecodeRows load_request(const AttendArgs &a, const int32_t *shared, int32_t i) {
    DecodeRows r;
    static_cast<RequestRows &>(r) = SHARED ? load_rows_cg(a, i) : load_rows(a, i);
    r.shared = SHARED ? shared[i] : 0;
    return r;
}

// A segment: its request, key head and row tile, and its keys (in steps of KEYS).
struct Segment {
    int32_t seq, head, tile;  // tile: first of its rows, rows numbered token * group + head in group
    int32_t q0, n, len;       // the request's rows and length
    int32_t lo, base, steps;  // first key that a row sees, the multiple of KEYS at or before it, steps from there
    int32_t begin;            // index of its first step among all of the call
    int32_t shared;           // keys that are not this call's
};

// Opening a segment (its query, its lengths, closing it) costs a warp about as
// much as kOpen steps: it counts as so many, in front of the real ones.
constexpr int kOpen = 2;

// The first key of a request that any of its rows sees.
__device__ __forceinline__ int32_t first_key(const AttendArgs &a, const DecodeRows &r) {
    if (a.window <= 0) return r.shared;
    return static_cast<int32_t>(max(int64_t(r.shared), int64_t(r.len) - r.n - a.window + 1));
}

template <int KEYS>
__device__ __forceinline__ int32_t steps_of(const AttendArgs &a, const DecodeRows &r) {
    return r.n > 0 ? (r.len - (first_key(a, r) & ~(KEYS - 1)) + KEYS - 1) / KEYS : 0;
}

template <int ROWS>
__device__ __forceinline__ int32_t tiles_of(const AttendArgs &a, int32_t n) {
    return static_cast<int32_t>((int64_t(n) * a.group + ROWS - 1) / ROWS);
}

// Where every warp gets at most one step, a segment takes whole blocks instead (its
// steps rounded up to the warps of a block, no opening): up to 8 steps then need
// no join between blocks.  One request of 100 tokens: 7.6 us so, 10.5 with openings and shares across blocks.
__device__ __forceinline__ int32_t units_of(int32_t steps, bool whole_blocks) {
    return whole_blocks ? (steps + kWarps - 1) / kWarps * kWarps : steps + kOpen;
}

// Steps of all segments of a request, their openings or roundings included.
template <int ROWS, int KEYS>
__device__ __forceinline__ int64_t cost_of(const AttendArgs &a, const DecodeRows &r, bool whole_blocks) {
    const int32_t steps = steps_of<KEYS>(a, r);
    return steps > 0 ? int64_t(units_of(steps, whole_blocks)) * a.kv.n_kv * tiles_of<ROWS>(a, r.n) : 0;
}

// The segment of request `seq` that step x of the call belongs to.
template <int ROWS, int KEYS, bool SHARED>
__device__ __forceinline__ Segment segment_at(const AttendArgs &a, const int32_t *shared, const int32_t *s_pref, int32_t seq,
                                              int32_t x, bool whole_blocks) {
    const DecodeRows r = load_request<SHARED>(a, shared, seq);
    Segment s;
    s.seq = seq;
    s.q0 = r.q0;
    s.n = r.n;
    s.len = r.len;
    s.shared = r.shared;
    s.lo = first_key(a, r);
    s.base = s.lo & ~(KEYS - 1);
    s.steps = max(1, steps_of<KEYS>(a, r));
    const int32_t tiles = max(1, tiles_of<ROWS>(a, r.n)), units = units_of(s.steps, whole_blocks);
    const int32_t i = (x - s_pref[seq]) / units;
    s.head = i / tiles;  // tiles of one head are neighbours: they read the same keys
    s.tile = (i - s.head * tiles) * ROWS;
    s.begin = s_pref[seq] + i * units + (whole_blocks ? 0 : kOpen);
    return s;
}

// A row of a segment among all rows and heads.
__device__ __forceinline__ int64_t own_row(const AttendArgs &a, const Segment &s, int32_t row) {
    return (int64_t(s.head) * a.T + s.q0) * a.group + row;
}

// The request that step x (below the total) belongs to.
__device__ __forceinline__ int32_t find_seq(const int32_t *s_pref, int32_t n, int32_t x) {
    int32_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (s_pref[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Rows r0 .. r0 + R - 1 (below `rows`) joined over partials first..last, in order;
// part(i) is partial i's address, in shared or global memory; B of them are loaded at
// a time, the first while the weights are computed (one request of 4,096 tokens: 16 at
// a time 14.6 us, 4 after the weights 16.1).  Writes rows of `out`, or of the partial `to`.
template <int HD, int ROWS, int R, int B, class P>
__device__ __forceinline__ void join_rows(const AttendArgs &a, P part, int32_t first, int32_t last, const Segment &s,
                                          int r0, int rows, float shift, float *to, int lane) {
    constexpr int V = HD / 32;
    float top[R], sum[R], o[R][V];
#pragma unroll
    for (int q = 0; q < R; ++q) {
        top[q] = -INFINITY;
        sum[q] = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) o[q][e] = 0.0f;
    }
    for (int32_t c = first; c <= last; c += 32) {
        const int32_t n = min(32, last - c + 1);
        const float *mine = part(c + min(lane, n - 1));
        float w[R], l[R], x[B][R][V];
        const auto fetch = [&](int32_t j0) {
#pragma unroll
            for (int b = 0; b < B; ++b) {
                if (j0 + b >= n) break;
                const float *v = part(c + j0 + b) + 2 * ROWS + lane * V;
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    const float *from = v + min(r0 + q, rows - 1) * HD;
                    if constexpr (V == 4) {
                        const float4 y = *reinterpret_cast<const float4 *>(from);
                        x[b][q][0] = y.x, x[b][q][1] = y.y, x[b][q][2] = y.z, x[b][q][3] = y.w;
                    } else {
                        const float2 y = *reinterpret_cast<const float2 *>(from);
                        x[b][q][0] = y.x, x[b][q][1] = y.y;
                    }
                }
            }
        };
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int r = min(r0 + q, rows - 1);
            w[q] = lane < n ? mine[r] : -INFINITY;
            l[q] = lane < n ? mine[ROWS + r] : 0.0f;
        }
        fetch(0);
#pragma unroll
        for (int q = 0; q < R; ++q) {
            float now = w[q];
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, d));
            now = fmaxf(now, top[q]);
            const float ref = now == -INFINITY ? 0.0f : now, f = ex2(top[q] - ref);
            w[q] = ex2(w[q] - ref);
            sum[q] *= f;
#pragma unroll
            for (int e = 0; e < V; ++e) o[q][e] *= f;
            top[q] = now;
        }
#pragma unroll 1
        for (int32_t j0 = 0; j0 < n; j0 += B) {
            if (j0 > 0) fetch(j0);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                if (j0 + b >= n) break;
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    const float wj = __shfl_sync(0xffffffffu, w[q], j0 + b);
                    sum[q] += wj * __shfl_sync(0xffffffffu, l[q], j0 + b);
#pragma unroll
                    for (int e = 0; e < V; ++e) o[q][e] += wj * x[b][q][e];
                }
            }
        }
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
        const int r = r0 + q;
        if (r >= rows) break;
        if (to != nullptr) {
            if (lane == 0) {
                to[r] = top[q];
                to[ROWS + r] = sum[q];
            }
#pragma unroll
            for (int e = 0; e < V; ++e) to[2 * ROWS + r * HD + lane * V + e] = o[q][e];
            continue;
        }
        const int32_t row = s.tile + r, t = s.q0 + row / a.group, h = s.head * a.group + row % a.group;
        const float inv = sum[q] > 0.0f ? a.kv.v_scale / sum[q] : sum[q] == 0.0f ? 0.0f : sum[q];
        uint32_t w[V / 2];
#pragma unroll
        for (int e = 0; e < V / 2; ++e) w[e] = pack_bf16x2(o[q][2 * e] * inv, o[q][2 * e + 1] * inv);
        uint16_t *dst = a.out + t * a.ldo + h * HD + lane * V;
        if constexpr (V == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t *>(dst) = w[0];
        if (a.lse != nullptr && lane == 0)
            a.lse[int64_t(t) * a.n_heads + h] = sum[q] == 0.0f ? -INFINITY : kLn2 * (top[q] - shift) + logf(sum[q]);
    }
}

// A block that did not wait for the kernel before it does so at its end: the kernel after
// this one then finds both finished.
template <bool SHARED>
__device__ __forceinline__ void end_own() {
    if (SHARED) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int HD, bool E4M3, int ROWS, bool SHARED>
__global__ void __launch_bounds__(kWarps * 32, 1)
attend_decode_kernel(const AttendArgs a, float *parts, int32_t *counters, int pref_bytes, const OwnRows own) {
    using C = Config<HD, E4M3, ROWS, SHARED>;
    constexpr int kKeys = C::kKeys, NK = kKeys / 32, ST = kKeys / 8, KB = kKeys / 16, kTiles = C::kTiles;
    constexpr int NW = kWarps, NT = NW * 32, MB = ROWS == 32 ? 2 : 1, KK = HD / 16, DT = HD / 8;
    constexpr bool kHalf = ROWS == 8;      // only rows 0..7 of the MMA's 16 hold queries
    constexpr bool kQShared = ROWS == 32;  // query fragments in shared memory, else in registers
    constexpr float kShift = E4M3 ? 12.0f : 0.0f;
    extern __shared__ __align__(128) unsigned char smem[];
    int32_t *s_pref = reinterpret_cast<int32_t *>(smem);
    __shared__ int64_t s_warp[NW][2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c4 = lane & 3;

    int32_t grid = gridDim.x;  // blocks that take part
    const int32_t *s_shared = nullptr;
    if constexpr (SHARED) {
        int32_t *to = reinterpret_cast<int32_t *>(smem + pref_bytes);
        if (own.blocks == nullptr) {
            wait_for_previous();
            const Groups &w = own.groups;
            if (blockIdx.x == 0)
                for (int32_t g = tid; g < w.n_groups; g += NT)
                    if (w.offsets[g] < 0 || w.offsets[g + 1] < w.offsets[g] || w.offsets[g + 1] > a.n_seq || w.lens[g] < 0)
                        report_error(a.err, LORA_ERR_INVALID_ARG);
            for (int32_t i = tid; i < a.n_seq; i += NT) to[i] = 0;
        } else {
            // The prefix kernel lets this one start when all of its blocks run, that is after all
            // kernels before it: what they wrote may be read (past the first-level cache), and only
            // the end waits for the prefix kernel.  Its blocks compute on as many SMs as the
            // plan gives them, this kernel's on the others.
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            __shared__ int64_t s_sum[4 * NW];
            // (blocks without a part, which start when the prefix kernel's end, leave at once)
            const int32_t known = __ldcg(own.blocks);
            if (__syncthreads_and(known > 0 && static_cast<int32_t>(blockIdx.x) >= known)) {
                end_own<SHARED>();
                return;
            }
            bool bad;
            const GroupPlan plan(reinterpret_cast<int32_t *>(smem + 2 * pref_bytes), own.groups.n_groups, a.n_seq);
            grid = plan_groups<NT>(a, own.groups, plan, s_sum, grid, false, &bad).own;
            for (int32_t i = tid; i < a.n_seq; i += NT) {
                const int32_t g = group_of(plan, own.groups.n_groups, bad, i);
                to[i] = g >= 0 ? plan.prefix[g] : 0;
            }
        }
        s_shared = to;
        __syncthreads();
        if (static_cast<int32_t>(blockIdx.x) >= grid) {
            end_own<SHARED>();
            return;
        }
    } else {
        wait_for_previous();
    }
    // steps of every request: exclusive prefix in s_pref[0..n_seq], total behind it
    int32_t total;
    bool whole_blocks;
    {
        const int32_t per = (a.n_seq + NT - 1) / NT, i0 = min(a.n_seq, tid * per), i1 = min(a.n_seq, i0 + per);
        int64_t mine = 0, padded = 0;
        for (int32_t i = i0; i < i1; ++i) {
            const DecodeRows r = load_request<SHARED>(a, s_shared, i);
            if (!r.ok && blockIdx.x == 0) report_error(a.err, LORA_ERR_INVALID_ARG);
            mine += cost_of<ROWS, kKeys>(a, r, false);
            padded += cost_of<ROWS, kKeys>(a, r, true);
        }
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        int64_t incl2 = padded;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, incl2, o);
            if (lane >= o) incl2 += u;
        }
        if (lane == 31) s_warp[warp][0] = incl, s_warp[warp][1] = incl2;
        __syncthreads();
        int64_t run = incl - mine, sum = 0, run2 = incl2 - padded, sum2 = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) run += s_warp[w][0], run2 += s_warp[w][1];
            sum += s_warp[w][0], sum2 += s_warp[w][1];
        }
        whole_blocks = sum2 <= int64_t(grid) * NW;
        if (whole_blocks) run = run2, sum = sum2;
        if (sum > INT32_MAX) {  // the same in every block
            if (blockIdx.x == 0 && tid == 0) report_error(a.err, LORA_ERR_UNSUPPORTED);
            end_own<SHARED>();
            // (behind the prefix kernel, which has set the word)
            if (SHARED && own.blocks != nullptr && blockIdx.x == 0 && tid == 0) own.live[0] = 0;
            return;
        }
        for (int32_t i = i0; i < i1; ++i) {
            const DecodeRows r = load_request<SHARED>(a, s_shared, i);
            s_pref[i] = static_cast<int32_t>(run);
            run += cost_of<ROWS, kKeys>(a, r, whole_blocks);
        }
        total = static_cast<int32_t>(sum);
        if (tid == 0) s_pref[a.n_seq] = total;
        __syncthreads();
    }

    // rows of requests without cached tokens
    for (int32_t i = blockIdx.x; i < a.n_seq; i += grid) {
        if (s_pref[i + 1] != s_pref[i]) continue;
        const DecodeRows r = load_request<SHARED>(a, s_shared, i);
        for (int64_t e = tid; e < int64_t(r.n) * a.n_heads; e += NT) {
            const int64_t t = r.q0 + e / a.n_heads, h = e % a.n_heads;
            for (int d = 0; d < HD; d += 8) stg_u4(a.out + t * a.ldo + h * HD + d, make_uint4(0, 0, 0, 0));
            if (a.lse != nullptr) a.lse[t * a.n_heads + h] = -INFINITY;
        }
    }

    const int32_t shares = grid * NW;
    const int64_t share = (int64_t(total) + shares - 1) / shares;  // steps a warp
    const int32_t me = blockIdx.x * NW + warp;
    const int32_t x0 = static_cast<int32_t>(min(int64_t(total), me * share));
    const int32_t x1 = static_cast<int32_t>(min(int64_t(total), x0 + share));

    // this warp's memory: its query fragments and its ring of k and v tiles; the last
    // partial of its share takes their place in the end
    const int ring_at = (SHARED ? 2 : 1) * pref_bytes;
    unsigned char *const warp_ptr = smem + ring_at + warp * C::kWarpB;
    const uint32_t ring = tc::smem_u32(warp_ptr) + C::kQBytes;
    uint4 *s_q = reinterpret_cast<uint4 *>(warp_ptr);

    // ---- the copying side: where its next step is ------------------------------
    Segment ls{};
    int32_t lx = x0, lkey = 0, lend = 0, lpage[NK];
    const int32_t *ltab = nullptr;
    // whether this lane's key 32 i + lane of the next step is one that a row sees, and its page
    const auto has_key = [&](int i) { return lkey + 32 * i + lane >= ls.lo && lkey + 32 * i + lane < ls.len; };
    const auto look_up = [&]() {
        if (lx < x1) {
#pragma unroll
            for (int i = 0; i < NK; ++i)
                lpage[i] = has_key(i) ? load_past_l1<SHARED>(ltab + ((lkey + 32 * i + lane) >> a.kv.page_shift)) : -1;
        }
    };
    const auto open_load = [&](int32_t seq) {
        ls = segment_at<ROWS, kKeys, SHARED>(a, s_shared, s_pref, seq, lx, whole_blocks);
        lx = max(lx, ls.begin);
        lkey = ls.base + (lx - ls.begin) * kKeys;
        lend = ls.begin + ls.steps;
        ltab = a.table + ls.seq * a.ld_table;
    };
    if (x0 < x1) {
        open_load(find_seq(s_pref, a.n_seq, x0));
        if (lx >= lend) lx = x1;  // a unit behind a segment's steps: nothing to do
        look_up();
    }
    // copies the next tile, k and v of a step in turn
    constexpr int kRows = 32 / C::kChunks;  // keys a copy instruction
    const int piece = lane % C::kChunks, row0 = lane / C::kChunks;
    const int64_t lane_off = row0 * a.kv.token_b + piece * 16, row_stride = kRows * a.kv.token_b;
    bool lv = false, smooth = false;
    int64_t at[NK];  // byte offsets of this lane's keys, -1: none
    const auto issue = [&](int slot) {
        if (lx < x1) {
            if (!lv) {
                bool all = a.kv.page_shift >= 4;
#pragma unroll
                for (int i = 0; i < NK; ++i) {
                    const bool ok = lpage[i] >= 0 && lpage[i] < a.kv.n_pages;
                    if (!ok && has_key(i)) report_error(a.err, LORA_ERR_SLOT_RANGE);
                    at[i] = ok ? lpage[i] * a.kv.page_b + ((lkey + 32 * i + lane) & a.kv.page_mask) * a.kv.token_b +
                                     ls.head * a.kv.head_b
                               : -1;
                    all = all && ok;
                }
                smooth = __all_sync(0xffffffffu, all);
            }
            const unsigned char *from = lv ? a.kv.v : a.kv.k;
            const uint32_t dst = ring + slot * C::kTileB;
            if (smooth) {
                // 16 neighbouring keys share a page: one address for them
#pragma unroll
                for (int half = 0; half < 2 * NK; ++half) {
                    const unsigned char *src = from + __shfl_sync(0xffffffffu, at[half / 2], 16 * (half & 1)) + lane_off;
#pragma unroll
                    for (int i = 0; i < C::kChunks / 2; ++i) {
                        tc::cp16(dst + piece_at<C::kChunks>(16 * half + i * kRows + row0, piece), src, true);
                        src += row_stride;
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < NK * C::kChunks; ++i) {
                    const int row = i * kRows + row0;
                    const int64_t o = __shfl_sync(0xffffffffu, at[i / C::kChunks], row & 31);
                    tc::cp16(dst + piece_at<C::kChunks>(row, piece), from + (o >= 0 ? o : 0) + piece * 16, o >= 0);
                }
            }
            if (lv) {
                ++lx;
                lkey += kKeys;
                if (lx == lend && lx < x1) {
                    int32_t seq = ls.seq;
                    while (s_pref[seq + 1] <= lx) ++seq;
                    open_load(seq);
                }
                look_up();
            }
            lv = !lv;
        }
        tc::cp_commit();
    };

    // ---- the computing side ----------------------------------------------------
    Segment cs{};
    int32_t cx = x0, cend = 0, ckey = 0, pos_lo = 0, pos_hi = 0;
    int32_t pos[MB][2];
    uint32_t qf[kQShared ? 1 : KK][4];
    float m[MB][2], l[MB][2], mult[MB][2], slope[MB][2], acc[MB][DT][4];

    const auto open_compute = [&](int32_t seq) {
        cs = segment_at<ROWS, kKeys, SHARED>(a, s_shared, s_pref, seq, cx, whole_blocks);
        cx = max(cx, cs.begin);
        cend = cs.begin + cs.steps;
        if (cx >= cend) cx = x1;  // a unit behind the segment's steps
        if (cx >= x1) return;
        ckey = cs.base + (cx - cs.begin) * kKeys;
        const int32_t rows = min(ROWS, cs.n * a.group - cs.tile);
        pos_lo = cs.len - cs.n + cs.tile / a.group;
        pos_hi = cs.len - cs.n + (cs.tile + rows - 1) / a.group;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int i = 0; i < (kHalf ? 1 : 2); ++i) {
                const int32_t r = mb * 16 + i * 8 + g, row = cs.tile + r;
                const bool live = r < rows;
                const int32_t token = row / a.group, h = cs.head * a.group + row % a.group;
                pos[mb][i] = live ? cs.len - cs.n + token : -1;
                slope[mb][i] = live && a.slopes != nullptr ? load_past_l1<SHARED>(a.slopes + h) * kLog2e : 0.0f;
                m[mb][i] = -INFINITY;
                l[mb][i] = 0.0f;
                mult[mb][i] = a.scale * a.kv.k_scale;
                const uint16_t *src = a.q + (cs.q0 + token) * a.ldq + h * HD;
                uint32_t w[KK][2];
                if constexpr (E4M3) {
                    // dims 4 c4 .. 4 c4 + 3 of each 16: the order in which a lane gets the codes of k
                    float top = 0.0f;
                    float f[KK][4];
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        const uint2 u = live ? load_past_l1<SHARED>(reinterpret_cast<const uint2 *>(src + kk * 16 + 4 * c4))
                                             : make_uint2(0, 0);
                        f[kk][0] = bf16lo_to_f32(u.x), f[kk][1] = bf16hi_to_f32(u.x);
                        f[kk][2] = bf16lo_to_f32(u.y), f[kk][3] = bf16hi_to_f32(u.y);
#pragma unroll
                        for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(f[kk][e]));
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // 2^e <= top < 2^(e + 1): the row times 2^-e is below 2
                    const int e = top > 0.0f ? max(-126, min(126, static_cast<int>(__float_as_uint(top) >> 23) - 127)) : 0;
                    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                    mult[mb][i] *= __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        w[kk][0] = pack_f16x2(f[kk][0] * down, f[kk][1] * down);
                        w[kk][1] = pack_f16x2(f[kk][2] * down, f[kk][3] * down);
                    }
                } else {
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        w[kk][0] = live ? load_past_l1<SHARED>(reinterpret_cast<const uint32_t *>(src + kk * 16 + 2 * c4)) : 0u;
                        w[kk][1] = live ? load_past_l1<SHARED>(reinterpret_cast<const uint32_t *>(src + kk * 16 + 8 + 2 * c4)) : 0u;
                    }
                }
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    if constexpr (kQShared) {
                        uint32_t *to = reinterpret_cast<uint32_t *>(s_q + (kk * MB + mb) * 32 + lane);
                        to[i] = w[kk][0];
                        to[2 + i] = w[kk][1];
                    } else {
                        qf[kk][i] = w[kk][0];
                        qf[kk][2 + i] = w[kk][1];
                        if (kHalf) qf[kk][1] = qf[kk][3] = 0u;
                    }
                }
            }
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mb][d][e] = 0.0f;
    };

    uint32_t hi[MB][KB][4], lo[MB][KB][4];
    const int mat = lane >> 3, r8 = lane & 7;
    const bool plain = a.softcap == 0.0f && a.slopes == nullptr && a.scale > 0.0f;
    // weights p = 2^(score log2 e - maximum) of the step's keys, as the fragments of the second product
    const auto scores = [&](int slot) {
        const uint32_t kt = ring + slot * C::kTileB;
        float s[MB][ST][4] = {};
#pragma unroll
        for (int kk = 0; kk < KK; kk += E4M3 ? 4 : 2) {
#pragma unroll
            for (int t0 = 0; t0 < ST; t0 += 4) {
                uint32_t b[4][4];
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    ldsm4(b[t], kt + piece_at<C::kChunks>(8 * (t0 + t) + r8, (E4M3 ? kk : 2 * kk) + mat));
#pragma unroll
                for (int u = 0; u < (E4M3 ? 4 : 2); ++u) {
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb) {
                        uint4 q;
                        if constexpr (kQShared) q = s_q[((kk + u) * MB + mb) * 32 + lane];
                        else q = make_uint4(qf[kk + u][0], qf[kk + u][1], qf[kk + u][2], qf[kk + u][3]);
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            if constexpr (E4M3)
                                mma_f16_16816(s[mb][t0 + t], q.x, q.y, q.z, q.w, e4m3x2_f16x2(b[t][u]),
                                              e4m3x2_f16x2(b[t][u] >> 16));
                            else
                                mma_bf16_16816(s[mb][t0 + t], q.x, q.y, q.z, q.w, b[t][2 * u], b[t][2 * u + 1]);
                        }
                    }
                }
            }
        }
        const bool masked = ckey + kKeys - 1 > pos_lo || (a.window > 0 && pos_hi - ckey >= a.window);
        const bool before = SHARED && ckey < cs.lo;  // the step's first keys are the prefix's
        const bool fast = plain && !masked && !before;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int i = 0; i < (kHalf ? 1 : 2); ++i) {
                float top = -INFINITY, by = mult[mb][i] * kLog2e;
                if (fast) {
#pragma unroll
                    for (int t = 0; t < ST; ++t) top = fmaxf(top, fmaxf(s[mb][t][2 * i], s[mb][t][2 * i + 1]));
                    top *= by;
                } else {
                    float f[2 * ST];
#pragma unroll
                    for (int t = 0; t < ST; ++t) f[2 * t] = s[mb][t][2 * i], f[2 * t + 1] = s[mb][t][2 * i + 1];
                    finish_scores<2 * ST, 8>(f, a, mult[mb][i], slope[mb][i], ckey + 2 * c4 - pos[mb][i], masked);
                    if (SHARED && before) {
#pragma unroll
                        for (int e = 0; e < 2 * ST; ++e)
                            if (ckey + 2 * c4 + e / 2 * 8 + (e & 1) < cs.lo) f[e] = -INFINITY;
                    }
#pragma unroll
                    for (int t = 0; t < ST; ++t) {
                        s[mb][t][2 * i] = f[2 * t], s[mb][t][2 * i + 1] = f[2 * t + 1];
                        top = fmaxf(top, fmaxf(f[2 * t], f[2 * t + 1]));
                    }
                    by = 1.0f;
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float now = fmaxf(m[mb][i], top);
                const float ref = (now == -INFINITY ? 0.0f : now) - kShift;
                if (__any_sync(0xffffffffu, now != m[mb][i])) {
                    const float f = ex2(m[mb][i] - kShift - ref);
                    l[mb][i] *= f;
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        acc[mb][d][2 * i] *= f;
                        acc[mb][d][2 * i + 1] *= f;
                        if (kHalf && !E4M3) {  // the remainder's part of the same row
                            acc[mb][d][2] *= f;
                            acc[mb][d][3] *= f;
                        }
                    }
                    m[mb][i] = now;
                }
                float sum = 0.0f;
#pragma unroll
                for (int t = 0; t < ST; ++t) {
                    const float p0 = ex2(fmaf(s[mb][t][2 * i], by, -ref)), p1 = ex2(fmaf(s[mb][t][2 * i + 1], by, -ref));
                    sum += p0 + p1;
                    // keys 8 t + 2 c4, + 1: the A fragment's word of 16-key block t / 2
                    const int w = (t & 1) * 2 + i;
                    if constexpr (E4M3) {
                        hi[mb][t / 2][w] = pack_f16x2(p0, p1);
                        if (kHalf) hi[mb][t / 2][w + 1] = 0u;
                    } else {
                        const uint32_t h = pack_bf16x2(p0, p1);
                        const uint32_t r = pack_bf16x2(p0 - bf16lo_to_f32(h), p1 - bf16hi_to_f32(h));
                        hi[mb][t / 2][w] = h;
                        if (kHalf) hi[mb][t / 2][w + 1] = r;
                        else lo[mb][t / 2][w] = r;
                    }
                }
                l[mb][i] += sum;
            }
    };
    // output: 16 keys at a time, all dims
    const auto outputs = [&](int slot) {
        const uint32_t vt = ring + slot * C::kTileB;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int c = 0; c < C::kChunks; c += 2) {
                uint32_t b[4];
                ldsm4_t(b, vt + piece_at<C::kChunks>(kb * 16 + (mat & 1) * 8 + r8, c + (mat >> 1)));
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if constexpr (E4M3) {
                        // piece c + u, 16 dims: even dims in one MMA, odd dims in the next
                        const uint32_t e0 = e4m3x2_f16x2(__byte_perm(b[2 * u], 0, 0x4420));
                        const uint32_t e1 = e4m3x2_f16x2(__byte_perm(b[2 * u + 1], 0, 0x4420));
                        const uint32_t o0 = e4m3x2_f16x2(__byte_perm(b[2 * u], 0, 0x4431));
                        const uint32_t o1 = e4m3x2_f16x2(__byte_perm(b[2 * u + 1], 0, 0x4431));
#pragma unroll
                        for (int mb = 0; mb < MB; ++mb) {
                            const uint32_t(&p)[4] = hi[mb][kb];
                            mma_f16_16816(acc[mb][2 * (c + u)], p[0], p[1], p[2], p[3], e0, e1);
                            mma_f16_16816(acc[mb][2 * (c + u) + 1], p[0], p[1], p[2], p[3], o0, o1);
                        }
                    } else {
#pragma unroll
                        for (int mb = 0; mb < MB; ++mb) {
                            const uint32_t(&p)[4] = hi[mb][kb];
                            mma_bf16_16816(acc[mb][c + u], p[0], p[1], p[2], p[3], b[2 * u], b[2 * u + 1]);
                            if constexpr (!kHalf) {
                                const uint32_t(&r)[4] = lo[mb][kb];
                                mma_bf16_16816(acc[mb][c + u], r[0], r[1], r[2], r[3], b[2 * u], b[2 * u + 1]);
                            }
                        }
                    }
                }
            }
    };

    // ends a segment, or this warp's part of it: rows to `out`, or a partial (the
    // share's last one into the warp's own memory, which holds no more tiles then)
    const auto close = [&]() {
        const int32_t rows = min(ROWS, cs.n * a.group - cs.tile);
        const bool whole = cs.begin >= x0 && cend == cx;
        // a piece for the join with the prefix: at the rows' place or, of a segment that begins before, at the warp's
        const bool piece = SHARED && cs.shared > 0, first = cs.begin >= x0;
        float *const cut = parts + int64_t(me) * C::kPartial;
        const int64_t all_rows = int64_t(a.T) * a.n_heads;
        float *part = cend + kOpen >= x1 ? reinterpret_cast<float *>(warp_ptr) : parts + int64_t(me) * C::kPartial;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int i = 0; i < (kHalf ? 1 : 2); ++i) {
                float sum = l[mb][i];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                const int32_t r = mb * 16 + i * 8 + g, row = cs.tile + r;
                if (r >= rows) continue;
                const int32_t t = cs.q0 + row / a.group, h = cs.head * a.group + row % a.group;
                const int64_t at = piece ? own_row(a, cs, row) : 0;
                float *const to_piece = first ? own.outs + at * 4 : cut + 2 * ROWS + r * 4;
                const int64_t dims4 = first ? 4 * all_rows : 4 * ROWS;  // from four dims to the next
                const float inv = !whole || piece ? 1.0f : sum > 0.0f ? a.kv.v_scale / sum : sum == 0.0f ? 0.0f : sum;
                uint16_t *out = a.out + t * a.ldo + h * HD;
                float *to = part + 2 * ROWS + r * HD;
                if (c4 == 0) {
                    if (piece) {
                        const int32_t others = static_cast<int32_t>((int64_t(cend) - 1) / share - me);
                        if (first)
                            own.sums[at] = make_float4(m[mb][i] - kShift, sum, __int_as_float((me + 1) << 5 | r),
                                                       __int_as_float(others));
                        else
                            *reinterpret_cast<float2 *>(cut + 2 * r) = make_float2(m[mb][i] - kShift, sum);
                    } else if (!whole) {
                        part[r] = m[mb][i];
                        part[ROWS + r] = sum;
                    } else if (a.lse != nullptr) {
                        a.lse[int64_t(t) * a.n_heads + h] = sum == 0.0f ? -INFINITY
                                                                        : kLn2 * (m[mb][i] - kShift) + logf(sum);
                    }
                }
                if constexpr (E4M3) {
#pragma unroll
                    for (int c = 0; c < DT; c += 2) {  // dims 16 (c / 2) + 4 c4 + {0, 1, 2, 3}
                        const float4 v = make_float4(acc[mb][c][2 * i] * inv, acc[mb][c + 1][2 * i] * inv,
                                                     acc[mb][c][2 * i + 1] * inv, acc[mb][c + 1][2 * i + 1] * inv);
                        const int d = 8 * c + 4 * c4;
                        if (piece)
                            *reinterpret_cast<float4 *>(to_piece + (d >> 2) * dims4) = v;
                        else if (whole)
                            *reinterpret_cast<uint2 *>(out + d) = make_uint2(pack_bf16x2(v.x, v.y),
                                                                             pack_bf16x2(v.z, v.w));
                        else
                            *reinterpret_cast<float4 *>(to + d) = v;
                    }
                } else {
#pragma unroll
                    for (int d8 = 0; d8 < DT; ++d8) {  // dims 8 d8 + 2 c4 + {0, 1}
                        float v0 = acc[mb][d8][2 * i], v1 = acc[mb][d8][2 * i + 1];
                        if (kHalf) v0 += acc[mb][d8][2], v1 += acc[mb][d8][3];
                        const int d = 8 * d8 + 2 * c4;
                        if (piece)
                            *reinterpret_cast<float2 *>(to_piece + (d >> 2) * dims4 + (d & 3)) = make_float2(v0, v1);
                        else if (whole) *reinterpret_cast<uint32_t *>(out + d) = pack_bf16x2(v0 * inv, v1 * inv);
                        else *reinterpret_cast<float2 *>(to + d) = make_float2(v0, v1);
                    }
                }
            }
    };

    // ---- the stream --------------------------------------------------------------
    for (int u = 0; u < kTiles - 1; ++u) issue(u);
    int slot = 0;
    const auto next = [&]() {
        tc::cp_wait_group<kTiles - 2>();
        __syncwarp();
        issue(slot == 0 ? kTiles - 1 : slot - 1);
        const int now = slot;
        slot = slot + 1 == kTiles ? 0 : slot + 1;
        return now;
    };
    if (x0 < x1) open_compute(find_seq(s_pref, a.n_seq, x0));
    while (cx < x1) {
        scores(next());
        outputs(next());
        ckey += kKeys;
        ++cx;
        if (cx == cend || cx == x1) {
            __syncwarp();
            close();
            if (cx < x1) {
                int32_t seq = cs.seq;
                while (s_pref[seq + 1] <= cx) ++seq;
                open_compute(seq);
            }
        }
    }
    tc::cp_wait_all();

    // ---- joining -------------------------------------------------------------------
    // The segments that the block's share boundaries cut, each listed once; its rows go to
    // the warps, first over the block's own partials, then, for segments of
    // several blocks, by the block that arrives last over the blocks'.
    struct Cut {
        Segment s;
        int32_t w0, w1, c0, c1, rows;  // first and last warp of this block and block of the call, rows
        bool last;
    };
    __shared__ Cut s_cut[NW + 1];
    float *block_parts = parts + int64_t(grid) * NW * C::kPartial;
    const int64_t block_share = share * NW, b0 = min(int64_t(total), blockIdx.x * block_share);
    const int64_t b1 = min(int64_t(total), b0 + block_share);
    if (tid <= NW) {
        const int64_t x = min(int64_t(total), b0 + tid * share);
        Cut c{};
        if (x > 0 && x < total) {
            c.s = segment_at<ROWS, kKeys, SHARED>(a, s_shared, s_pref, find_seq(s_pref, a.n_seq, static_cast<int32_t>(x)),
                                          static_cast<int32_t>(x), whole_blocks);
            const int64_t end = int64_t(c.s.begin) + c.s.steps;
            if (c.s.shared == 0 && c.s.begin < x && x < end && (tid == 0 || c.s.begin >= x - share)) {
                c.rows = min(ROWS, c.s.n * a.group - c.s.tile);
                c.w0 = static_cast<int32_t>(max(int64_t(c.s.begin), b0) / share);
                c.w1 = static_cast<int32_t>((min(end, b1) - 1) / share);
                c.c0 = static_cast<int32_t>(c.s.begin / block_share);
                c.c1 = static_cast<int32_t>((end - 1) / block_share);
            }
        }
        s_cut[tid] = c;
    }
    __syncthreads();
    // a block's partial: its first segment begins before it, its last cut one inside
    const auto block_part = [&](const Segment &s, int32_t c) -> float * {
        return block_parts + (2 * int64_t(c) + (s.begin >= c * block_share ? 1 : 0)) * C::kPartial;
    };
    // calls f(cut, first row, rows at a time) for this warp's part of the cuts that pick()
    // takes: four rows at a time hide each other's latency, one at a time where there are
    // fewer rows than that gives warps
    const auto each = [&](auto pick, auto f) {
        int all = 0;
        for (int i = 0; i <= NW; ++i) all += pick(s_cut[i]) ? s_cut[i].rows : 0;
        const int by = all > 2 * NW ? 4 : 1;
        for (int i = 0, turn = 0; i <= NW; ++i)
            if (pick(s_cut[i]))
                for (int r = 0; r < s_cut[i].rows; r += by, ++turn)
                    if (turn % NW == warp) {
                        if (by == 4) f(s_cut[i], r, std::integral_constant<int, 4>());
                        else f(s_cut[i], r, std::integral_constant<int, 1>());
                    }
    };
    each([](const Cut &c) { return c.rows > 0; }, [&](const Cut &c, int r, auto by) {
        const int64_t end = int64_t(c.s.begin) + c.s.steps;
        // a warp's partial is in its own memory, unless more segments followed in its share
        const auto of_warp = [&](int32_t w) -> const float * {
            if (end + kOpen < min(int64_t(total), (w + 1) * share)) return parts + int64_t(w) * C::kPartial;
            return reinterpret_cast<const float *>(smem + ring_at + (w - blockIdx.x * NW) * C::kWarpB);
        };
        join_rows<HD, ROWS, by.value, ROWS == 32 ? 2 : 4>(a, of_warp, c.w0, c.w1, c.s, r, c.rows, kShift,
                                                          c.c0 == c.c1 ? nullptr : block_part(c.s, blockIdx.x), lane);
    });
    bool shared_cut = false;
    for (int i = 0; i <= NW; ++i) shared_cut = shared_cut || (s_cut[i].rows > 0 && s_cut[i].c0 != s_cut[i].c1);
    if (!shared_cut) {
        end_own<SHARED>();
        return;
    }
    __threadfence();
    __syncthreads();
    if (tid <= NW && s_cut[tid].rows > 0 && s_cut[tid].c0 != s_cut[tid].c1) {
        Cut &c = s_cut[tid];
        c.last = atomicAdd(counters + c.c0, 1) == c.c1 - c.c0;
        if (c.last) counters[c.c0] = 0;
    }
    __syncthreads();
    __threadfence();
    each([](const Cut &c) { return c.last; }, [&](const Cut &c, int r, auto by) {
        const auto of_block = [&](int32_t b) -> const float * { return block_part(c.s, b); };
        join_rows<HD, ROWS, by.value, ROWS == 32 ? 2 : by.value == 1 ? 16 : 4>(a, of_block, c.c0, c.c1, c.s, r, c.rows,
                                                                               kShift, nullptr, lane);
    });
    end_own<SHARED>();
}

template <int HD, bool E4M3, int ROWS, bool SHARED>
cudaError_t launch_decode(const AttendArgs &a, const OwnRows &own, void *ws, cudaStream_t stream) {
    using C = Config<HD, E4M3, ROWS, SHARED>;
    static std::atomic<uint64_t> seen{0};
    const auto kernel = attend_decode_kernel<HD, E4M3, ROWS, SHARED>;
    int sms = 0;
    constexpr int kLists = SHARED ? 2 : 1;  // of the requests: step prefixes; shared keys
    const cudaError_t e = prepare_kernel(kernel, kLists * kPrefixMax + kWarps * C::kWarpB, seen, &sms);
    if (e != cudaSuccess) return e;
    const int grid = sms < kMaxGrid ? sms : kMaxGrid;
    const int pref = ((a.n_seq + 1) * 4 + 127) & ~127;
    const int smem = kLists * pref + kWarps * C::kWarpB;
    static_assert(!SHARED || GroupPlan::bytes(LORA_MAX_SEQS, LORA_MAX_SEQS) <= size_t(kWarps) * C::kWarpB, "the plan's place");
    int32_t *counters = static_cast<int32_t *>(ws);
    float *parts = reinterpret_cast<float *>(static_cast<char *>(ws) + 1024);
    return launch_dependent(kernel, grid, kWarps * 32, smem, stream, a, parts, counters, pref, own);
}

template <int HD, bool E4M3, bool SHARED>
cudaError_t pick_rows(const AttendArgs &a, int64_t rows, const OwnRows &own, void *ws, cudaStream_t stream) {
    if (rows <= 8) return launch_decode<HD, E4M3, 8, SHARED>(a, own, ws, stream);
    if (rows <= 16) return launch_decode<HD, E4M3, 16, SHARED>(a, own, ws, stream);
    return launch_decode<HD, E4M3, 32, SHARED>(a, own, ws, stream);
}

template <bool SHARED>
cudaError_t pick_decode(const AttendArgs &a, bool e4m3, int64_t rows, const OwnRows &own, void *ws,
                        cudaStream_t stream) {
    if (a.kv.head_dim == 64)
        return e4m3 ? pick_rows<64, true, SHARED>(a, rows, own, ws, stream)
                    : pick_rows<64, false, SHARED>(a, rows, own, ws, stream);
    return e4m3 ? pick_rows<128, true, SHARED>(a, rows, own, ws, stream)
                : pick_rows<128, false, SHARED>(a, rows, own, ws, stream);
}

}  // namespace

}  // namespace lora

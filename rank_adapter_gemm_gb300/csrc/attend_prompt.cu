// Attention of many rows a request over the paged cache (LORA_ATTEND_PROMPT).
//
// Two products of 2 rows keys head_dim operations each bound it, so both run on
// the 5th-generation tensor cores with accumulators in tensor memory:
//   S = Q K^T (128 rows x 128 keys), P = softmax weights in bf16, O += P V,
// a block holding two tiles of 128 rows whose products and softmaxes alternate:
// while one tile's weights are computed, the tensor cores work on the other's.
// Rows are (token, query head of one key head), so a key tile is read once for
// all heads of its group.
//
//   warps 0-3, 4-7   softmax of tile 0 and 1, one row a thread: the row of S from
//                    tensor memory into registers, weights back into S's place
//                    as the left operand of the second product, in halves that
//                    it starts on at once.  Weights are taken against a reference
//                    that moves, and the sum and O with it, only when a step's
//                    maximum passes 2^8 times it: most steps never touch O.
//   warps 8-11       copy q rows and k and v tiles of 128 keys, key by key through
//                    the block table, into the swizzled layout that the tensor
//                    cores read (e4m3 codes are widened to f16 on the way)
//   warp 12          issues the products
//   warp 13          hands out the work
// One block an SM stays for the whole call.  The (request, row tiles, key head)
// items go to whichever block is free, those with the most keys first (of each
// request, where there are more than 32), and a block's copies and products begin
// its next item while the softmax warps still write the last one's output.  With
// few items a block takes one part of an item's keys, and the parts are joined pair
// by pair.  An item's keys are taken from the last tile down: with a bias that falls
// with distance the largest scores come first and O is not rescaled step after step.
// k and v tiles share one ring; every wait is bounded (2 s) and reports
// LORA_ERR_TIMEOUT.
//
// The instruction takes one type for both operands.  Over a bf16 cache weights
// are rounded to bf16 (sums use them unrounded).  Over an e4m3 cache everything is
// f16: codes are exact in it, a query row is scaled by a power of two to keep
// 2^-24 of its largest element, and weights, times 2^7, keep 11 bits down to 2^-21
// of the row's reference.
//
// Measured, causal, 32 / 8 heads of 128, back to back: 8,192 tokens 431 us, 1.28 PFLOP/s
// (over e4m3 453), 16,384 tokens 1,600 us, 1.37 PFLOP/s; cuBLAS reaches 1.92 on a large
// bf16 product.  64-wide heads: 8,192 tokens 357 us; there a product does half the
// operations in nearly the time.  With caps and a bias the softmax bounds it: 16 / 4 heads of
// 64, 6,546 ragged tokens over e4m3 74 us, without them 54.  A step of a long item takes
// 1.75 us (131,072 to 4,194,304 keys), 1.5 with 64-wide heads.
#include "attend_tc.cuh"

namespace lora {

namespace {

constexpr int kThreads = 16 * 32;

template <int HD>
struct PromptConfig {
    static constexpr int kTileB = kRows * HD * 2;
    static constexpr int kSlots = HD == 128 ? 5 : 8;  // k and v tiles in the ring
    static constexpr int kQ = HD == 128 ? 1 : 2;      // items whose q rows fit
    static constexpr int kSmem = (2 * kQ + kSlots) * kTileB + 1024;
    static constexpr uint32_t kHalfB = kRows * 128;   // 64 dims of all rows
    // Registers a thread: 128 at launch, then by role.  The four warpgroups' shares (two
    // of softmax, copies, products) add up to the launch's 4 x 128.  Measured on 8,192
    // tokens (184, 80, 64 against 168, 104, 72): 128-wide heads 450 against 431 us, over
    // e4m3 482 against 453; 64-wide heads 357 against 365, 8 ragged chunks 74 against 77.
    static constexpr int kSoftmaxRegs = HD == 128 ? 168 : 184;
    static constexpr int kCopyRegs = HD == 128 ? 104 : 80;
    static constexpr int kMmaRegs = HD == 128 ? 72 : 64;
    static_assert(2 * kSoftmaxRegs + kCopyRegs + kMmaRegs == 4 * 128, "registers of the block");
};

struct Barriers {
    uint64_t q_full[2], q_empty[2], full[8], empty[8], s_full[2], p_full[2][2], o_full[2], o_empty[2], item_full[2],
        item_empty[2], exp_full[2], claim, done;
};

// 256 rows (two tiles) of a request and key head, and their keys [key0, key1).
struct Item {
    int32_t seq, head, row0, rows;  // first row and rows (of the request's n * group)
    int32_t q0, n, len, lo, key0, steps;
    int32_t part, parts;            // of the item's keys; the fields above are the part's
    bool first, last;               // of the part's segments (kSegment)
    bool any;                       // none: the work is done
};

// The tensor cores cut off what does not fit when they add to O, so that O loses about
// 2^-24 of itself with every 16 keys: 0.5 % at a million keys, 2 % at four.  More steps than
// these (65,536 keys) are handed out as segments, whose rows are added up in fp32 in the block's
// partial result: 0.03 % at any length.  No wait then spans more than a segment either (3 ms
// with scores far beyond a cap).
constexpr int32_t kSegment = 512;

// Few items leave SMs idle: their keys are cut into up to kMaxParts parts, of at least
// kMinSteps steps each, a block each.  32 rows over 16,384 tokens: 38 us, whole items 187; 64
// rows 45 and 234; 16 rows over 2,000 tokens 23.6 us, in parts of at least 2 steps 24.8, of 1
// 26.9, whole 31.
constexpr int kMaxParts = 16, kMinSteps = 4, kMaxGrid = 160;

// A part's partial result: references and sums of its 256 rows, then their outputs,
// four dims of all rows together, fp32.
template <int HD>
constexpr int64_t kPartial = int64_t(2 * kRows) * (HD + 2);

// A warp's 32 rows (a lane each: reference m, sum l, outputs in tensor memory) joined
// with those of the item's other parts, two neighbouring groups of parts at a time:
// of two warps that meet, the one that comes first leaves its rows and ends, the
// other goes on with both.  The lower part stands on the left whoever comes first,
// so results do not depend on timing, and nothing waits.  True in the warp that
// has all parts.  flags: of an item a bit for every warp and pair of groups (8 or 16 a
// warp: 4 + 2 + 1, or 8 + 4 + 2 + 1), zero between calls.
template <int HD>
__device__ __forceinline__ bool join_parts(float *slots, uint32_t *flags, int32_t part, int32_t parts, int r,
                                           uint32_t o_at, float &m, float &l, int warp, int lane) {
    const int bits = parts > 8 ? 16 : 8;
    flags += warp * bits / 32;
#pragma unroll 1
    for (int level = 0; (1 << level) < parts; ++level) {
        const int32_t group = part >> level, other = group ^ 1;
        if ((other << level) >= parts) continue;
        const uint32_t bit = 1u << (warp * bits % 32 + (bits - (bits >> level)) + (group >> 1));
        bool second = *static_cast<volatile uint32_t *>(flags) & bit;
        second = __shfl_sync(0xffffffffu, static_cast<int>(second), 0);
        if (!second) {
            float *mine = slots + (group << level) * kPartial<HD>;
            mine[r] = m;
            mine[2 * kRows + r] = l;
            mine += 4 * kRows + r * 4;
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
                uint32_t x[32];
                tmem_ld32(o_at + 32 * c, x);
                tmem_wait(x);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    stg_u4(mine + (8 * c + e) * 8 * kRows, make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]));
            }
            __threadfence();
            __syncwarp();
        }
        uint32_t before = 0;
        if (lane == 0) before = atomicXor(flags, bit);
        if ((__shfl_sync(0xffffffffu, before, 0) & bit) == 0) return false;
        __threadfence();
        const float *theirs = slots + (other << level) * kPartial<HD>;
        const float m2 = __ldcg(theirs + r), l2 = __ldcg(theirs + 2 * kRows + r);
        theirs += 4 * kRows + r * 4;
        const float top = fmaxf(m, m2), ref = top == -INFINITY ? 0.0f : top, w = ex2(m - ref), w2 = ex2(m2 - ref);
        const bool left = group < other;
        const auto joined = [&](float v, float v2) {
            return left ? fmaf(w2, v2, w * v) : fmaf(w, v, w2 * v2);
        };
        m = top;
        l = joined(l, l2);
#pragma unroll 1
        for (int c = 0; c < HD / 64; ++c) {
            float4 y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = ldg_cg_f4(theirs + (16 * c + e) * 8 * kRows);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t x[32];
                tmem_ld32(o_at + 64 * c + 32 * h, x);
                tmem_wait(x);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float4 v = y[8 * h + e];
                    x[4 * e] = __float_as_uint(joined(__uint_as_float(x[4 * e]), v.x));
                    x[4 * e + 1] = __float_as_uint(joined(__uint_as_float(x[4 * e + 1]), v.y));
                    x[4 * e + 2] = __float_as_uint(joined(__uint_as_float(x[4 * e + 2]), v.z));
                    x[4 * e + 3] = __float_as_uint(joined(__uint_as_float(x[4 * e + 3]), v.w));
                }
                tmem_st32(o_at + 64 * c + 32 * h, x);
            }
        }
        tmem_wait_st();
    }
    return true;
}

// A warp's rows between the segments of an item: the lane's reference, sum and outputs left
// in the block's partial result, and joined with it again.  (16 dims at a time: registers.)
template <int HD>
__device__ __forceinline__ void leave_segments(float *carried, int r, uint32_t o_at, float m, float l) {
    carried[r] = m;
    carried[2 * kRows + r] = l;
    carried += 4 * kRows + r * 4;
#pragma unroll 1
    for (int c = 0; c < HD / 16; ++c) {
        uint32_t x[16];
        tc::tmem_ld16(o_at + 16 * c, x);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            stg_u4(carried + (4 * c + e) * 8 * kRows, make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]));
    }
}

template <int HD>
__device__ __forceinline__ void add_segments(const float *carried, int r, uint32_t o_at, float &m, float &l) {
    const float m2 = __ldcg(carried + r), l2 = __ldcg(carried + 2 * kRows + r);
    carried += 4 * kRows + r * 4;
    const float top = fmaxf(m, m2), ref = top == -INFINITY ? 0.0f : top, w = ex2(m - ref), w2 = ex2(m2 - ref);
    m = top;
    l = fmaf(w2, l2, w * l);
#pragma unroll 1
    for (int c = 0; c < HD / 16; ++c) {
        uint32_t x[16];
        tc::tmem_ld16(o_at + 16 * c, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 v = ldg_cg_f4(carried + (4 * c + e) * 8 * kRows);
            x[4 * e] = __float_as_uint(fmaf(w2, v.x, w * __uint_as_float(x[4 * e])));
            x[4 * e + 1] = __float_as_uint(fmaf(w2, v.y, w * __uint_as_float(x[4 * e + 1])));
            x[4 * e + 2] = __float_as_uint(fmaf(w2, v.z, w * __uint_as_float(x[4 * e + 2])));
            x[4 * e + 3] = __float_as_uint(fmaf(w2, v.w, w * __uint_as_float(x[4 * e + 3])));
        }
        tmem_st16(o_at + 16 * c, x);
    }
    tmem_wait_st();
}

// Claims on the call's items, zero between calls: items given out past the first
// one of each block, and blocks that are done.
struct Claims {
    int32_t given, done;
};

template <int HD, bool E4M3, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
attend_prompt_kernel(const AttendArgs a, Claims *claims, uint32_t *flags, float *partials) {
    using C = PromptConfig<HD>;
    constexpr float kShift = E4M3 ? 7.0f : 0.0f;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Barriers bar;
    __shared__ Item s_item[2];
    __shared__ int64_t s_warp[kThreads / 32];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int32_t s_abort;
    __shared__ int8_t s_qexp[2][E4M3 ? 2 * kRows : 1];  // of this and the next item: q rows' powers of two
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t q_base = (tc::smem_u32(smem_raw) + 1023) & ~1023u;  // q tiles of kQ items, then the ring
    const uint32_t ring = q_base + 2 * C::kQ * C::kTileB;

    wait_for_previous();
    const auto pairs_of = [&](const RequestRows &r) {
        return (int64_t(r.n) * a.group + 2 * kRows - 1) / (2 * kRows);
    };
    int64_t total = 0;  // pairs of row tiles
    {
        int64_t mine = 0;
        for (int32_t i = tid; i < a.n_seq; i += kThreads) {
            const RequestRows r = load_rows(a, i);
            if (!r.ok && blockIdx.x == 0) report_error(a.err, LORA_ERR_INVALID_ARG);
            mine += pairs_of(r);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
        if (lane == 0) s_warp[warp] = mine;
    }
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < C::kQ; ++i) {
            tc::mbar_init(&bar.q_full[i], 4);
            tc::mbar_init(&bar.q_empty[i], 1);
        }
        for (int i = 0; i < C::kSlots; ++i) {
            tc::mbar_init(&bar.full[i], 4);
            tc::mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bar.s_full[i], 1);
            tc::mbar_init(&bar.p_full[i][0], 4);
            tc::mbar_init(&bar.p_full[i][1], 4);
            tc::mbar_init(&bar.o_full[i], 1);
            tc::mbar_init(&bar.o_empty[i], 4);
            tc::mbar_init(&bar.item_full[i], 1);
            tc::mbar_init(&bar.exp_full[i], 4);
            tc::mbar_init(&bar.item_empty[i], 13);  // the copying, multiplying and softmax warps
        }
        tc::mbar_init(&bar.claim, 1);
        tc::mbar_init(&bar.done, 1);
        tc::mbar_init_fence();
    }
    if (warp == 12) tc::tmem_alloc(&s_tmem, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) total += s_warp[w];
    const uint32_t tmem = s_tmem;
    // Waits of a whole warp.  Their outcome is a lane's own, and the instructions around them
    // want all lanes, so it steers the warp by votes only.  wait() votes at once.  After follow()
    // a lane that gave up remembers it, ends the block's other waits and goes on - every
    // address stays in bounds, values no longer matter - until go_on() is asked: at an item's
    // start and end, and every kVote steps of the products, whose chain of waits has no time
    // for votes (8,192 tokens: 470 us with one in every wait, 433 so).
    constexpr int32_t kVote = 64;
    bool fine = true;
    const auto follow = [&](uint64_t *b, uint32_t parity) {
        if (!tc::mbar_wait(b, parity, &s_abort, kWaitNs)) {
            fine = false;
            s_abort = 1;
        }
    };
    const auto go_on = [&]() { return __all_sync(0xffffffffu, fine) != 0; };
    const auto wait = [&](uint64_t *b, uint32_t parity) {
        const bool there = __all_sync(0xffffffffu, tc::mbar_wait(b, parity, &s_abort, kWaitNs));
        fine = fine && there;
        return there;
    };
    // a warp lets go of the block's k-th item
    const auto release = [&](int32_t k) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar.item_empty[k & 1]);
    };

    if (warp >= 8 && warp < 12) {
        set_registers<C::kCopyRegs, false>();
        // ---- copies ---------------------------------------------------------------------
        const int w = warp - 8;
        constexpr int kPieces = HD / 8;                          // 16-byte pieces of a 16-bit row
        constexpr int kStep = 32 / kPieces;                      // rows a q (or bf16) instruction
        constexpr int kKvPieces = E4M3 ? HD / 16 : kPieces;      // pieces of a cache row
        constexpr int kKvStep = 32 / kKvPieces;
        const int piece = lane % kPieces, row_in = lane / kPieces;
        const int kv_piece = lane % kKvPieces, kv_row = lane / kKvPieces;
        const auto publish = [&](uint64_t *b) {
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(b);
        };
        int32_t u = 0, q_round = 0;  // tiles and items so far
        for (int32_t k = 0;; ++k) {
            follow(&bar.item_full[k & 1], (k >> 1) & 1);
            if (!go_on() || !s_item[k & 1].any) break;
            const Item &it = s_item[k & 1];
            const int32_t steps = it.steps, lo = it.lo;
            const int32_t last = it.len - it.n + (it.row0 + it.rows - 1) / a.group;
            const int32_t *table = a.table + it.seq * a.ld_table;
            const int64_t head = it.head * a.kv.head_b;
            // this lane's key of the step to copy (the last keys first) and, ahead of it, its page
            int32_t key = it.key0 + (steps - 1) * kKeys + w * 32 + lane, page = -1;
            const auto has_key = [&]() { return key >= lo && key <= last; };
            if (has_key()) page = table[key >> a.kv.page_shift];
            const int qb = q_round % C::kQ;
            const uint32_t q_at_base = q_base + qb * 2 * C::kTileB;
            const auto q_piece = [&](int r) { return q_at_base + (r / kRows) * C::kTileB + tile_at(r % kRows, piece); };
            if (steps > 0) {
                if (q_round >= C::kQ) follow(&bar.q_empty[qb], (q_round / C::kQ - 1) & 1);
                ++q_round;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    // 32 rows of q: a lane's row's offset, then a few rows an instruction
                    const int r0 = w * 64 + half * 32, row = it.row0 + r0 + lane;
                    int64_t q_at = -1;
                    if (r0 + lane < it.rows)
                        q_at = (it.q0 + row / a.group) * a.ldq + (it.head * a.group + row % a.group) * HD;
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        const int64_t o = __shfl_sync(0xffffffffu, q_at, i * kStep + row_in);
                        tc::cp16(q_piece(r0 + i * kStep + row_in), a.q + (o >= 0 ? o : 0) + piece * 8, o >= 0);
                    }
                }
                if constexpr (E4M3) {
                    // a lane turns a row into f16, in place, scaled to lie below 2
                    tc::cp_wait_all();
                    __syncwarp();
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        const int r = w * 64 + half * 32 + lane;
                        const uint32_t tile = q_at_base + (r / kRows) * C::kTileB;
                        uint32_t top2 = 0;  // the row's largest size, as a pair of bf16 bit patterns
#pragma unroll 4
                        for (int p = 0; p < kPieces; ++p) {
                            const uint4 v = lds16(tile + tile_at(r % kRows, p));
                            top2 = __vmaxu2(top2, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                                           __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
                        }
                        const uint32_t top = max(top2 & 0xffffu, top2 >> 16);  // (bf16 sizes order like integers)
                        // 2^e <= top < 2^(e + 1)
                        const int e2 = top > 0 ? max(-126, min(126, static_cast<int>(top >> 7) - 127)) : 0;
                        const float down = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
                        s_qexp[k & 1][r] = static_cast<int8_t>(e2);
#pragma unroll 4
                        for (int p = 0; p < kPieces; ++p) {
                            const uint32_t at = tile + tile_at(r % kRows, p);
                            const uint4 v = lds16(at);
                            uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                x[e] = pack_f16x2(bf16lo_to_f32(x[e]) * down, bf16hi_to_f32(x[e]) * down);
                            sts16(at, make_uint4(x[0], x[1], x[2], x[3]));
                        }
                    }
                }
                if (E4M3) publish(&bar.q_full[qb]);
                else tc::cp_commit();
            }
            if (E4M3 && lane == 0) tc::mbar_arrive(&bar.exp_full[k & 1]);
            release(k);  // nothing below reads the item

            int64_t at = -1;      // byte offset of this lane's key, -1: none
            bool smooth = false;  // all keys there, and 16 neighbours always in one page
            const auto next_keys = [&]() {
                const bool ok = page >= 0 && page < a.kv.n_pages, has = has_key();
                if (has && !ok) report_error(a.err, LORA_ERR_SLOT_RANGE);
                at = has && ok ? page * a.kv.page_b + (key & a.kv.page_mask) * a.kv.token_b + head : -1;
                smooth = __all_sync(0xffffffffu, at >= 0) && a.kv.page_shift >= 4;
                key -= kKeys;
                if (has_key()) page = table[key >> a.kv.page_shift];
            };
            // calls f(instruction, address or null) for this warp's 32 keys of k or v
            const auto each = [&](const unsigned char *from, auto f) {
                from += kv_piece * 16;
                if (smooth) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const unsigned char *src = from + __shfl_sync(0xffffffffu, at, 16 * h) + kv_row * a.kv.token_b;
#pragma unroll
                        for (int i = 0; i < kKvPieces / 2; ++i) {
                            f(h * (kKvPieces / 2) + i, src);
                            src += kKvStep * a.kv.token_b;
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kKvPieces; ++i) {
                        const int64_t o = __shfl_sync(0xffffffffu, at, i * kKvStep + kv_row);
                        f(i, o >= 0 ? from + o : nullptr);
                    }
                }
            };
            const auto slot_free = [&]() {
                return u < C::kSlots || wait(&bar.empty[u % C::kSlots], (u / C::kSlots - 1) & 1);
            };
            const int32_t tiles = 2 * steps;
            if constexpr (E4M3) {
                uint4 v[kKvPieces];
                const auto load = [&](int32_t t) {
                    if ((t & 1) == 0) next_keys();
                    each((t & 1) ? a.kv.v : a.kv.k, [&](int i, const unsigned char *src) {
                        v[i] = src != nullptr ? ldg_cg(src) : make_uint4(0, 0, 0, 0);
                    });
                };
                if (tiles > 0) load(0);
                for (int32_t t = 0; t < tiles; ++t, ++u) {
                    if (t == tiles - 2 && w == 0 && lane == 0) tc::mbar_arrive(&bar.claim);
                    if (!slot_free()) break;
                    const uint32_t dst = ring + (u % C::kSlots) * C::kTileB;
#pragma unroll
                    for (int i = 0; i < kKvPieces; ++i) {
                        const int row = w * 32 + i * kKvStep + kv_row;
                        uint4 x, y;
                        widen16(v[i], x, y);
                        sts16(dst + tile_at(row, 2 * kv_piece), x);
                        sts16(dst + tile_at(row, 2 * kv_piece + 1), y);
                    }
                    if (t + 1 < tiles) load(t + 1);
                    publish(&bar.full[u % C::kSlots]);
                }
            } else {
                for (int32_t t = 0; t < tiles; ++t, ++u) {
                    if (t == tiles - 2 && w == 0 && lane == 0) tc::mbar_arrive(&bar.claim);
                    if ((t & 1) == 0) next_keys();
                    if (!slot_free()) break;
                    const uint32_t dst = ring + (u % C::kSlots) * C::kTileB;
                    each((t & 1) ? a.kv.v : a.kv.k, [&](int i, const unsigned char *src) {
                        tc::cp16(dst + tile_at(w * 32 + i * kKvStep + kv_row, kv_piece), src != nullptr ? src : a.kv.k,
                                 src != nullptr);
                    });
                    tc::cp_commit();
                    // the tile two before this one (and q before all) has landed
                    tc::cp_wait_group<2>();
                    if (t == 1) publish(&bar.q_full[qb]);
                    if (t >= 2) publish(&bar.full[(u - 2) % C::kSlots]);
                }
                if (tiles > 0) {
                    tc::cp_wait_group<1>();
                    publish(&bar.full[(u - 2) % C::kSlots]);
                    tc::cp_wait_group<0>();
                    publish(&bar.full[(u - 1) % C::kSlots]);
                }
            }
            if (steps == 0 && w == 0 && lane == 0) tc::mbar_arrive(&bar.claim);
        }
        tc::cp_wait_all();
    } else if (warp >= 12) {
        set_registers<C::kMmaRegs, false>();
        if (warp == 12) {
            // ---- products ---------------------------------------------------------------
            // The warp stays together and one elected thread issues: the products' operands
            // then stay in uniform registers.
            constexpr uint32_t kType = E4M3 ? (1u << 7) | (1u << 10) : 0u;  // f16 has 0 where bf16 has 1
            constexpr uint32_t kS = tc::idesc_bf16(kRows, kKeys) ^ kType;
            constexpr uint32_t kO = (tc::idesc_bf16(kRows, HD) ^ kType) | (1u << 16);  // v: keys are strided
            // descriptors are a tile's plus a constant: addresses stay below 2^18, so nothing carries
            const uint64_t q_desc = desc128(q_base, 16, 1024), k_desc = desc128(ring, 16, 1024);
            const uint64_t v_desc = desc128(ring, C::kHalfB, 1024);
            // (elect_one brings the warp together after a wait)
            const auto full = [&](int32_t u) { follow(&bar.full[u % C::kSlots], (u / C::kSlots) & 1); };
            const auto commit = [&](uint64_t *b) {
                if (elect_one()) tc::mma_commit(b);
                __syncwarp();
            };
            const auto scores = [&](int qb, int i, int32_t u) {
                const uint64_t q = q_desc + (((2 * qb + i) * C::kTileB) >> 4), k = k_desc + (((u % C::kSlots) * C::kTileB) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk) {
                        const uint32_t off = ((kk / 4) * C::kHalfB + (kk % 4) * 32) >> 4;
                        tc::mma_bf16(tmem + i * kKeys, q + off, k + off, kS, kk > 0);
                    }
                    tc::mma_commit(&bar.s_full[i]);
                }
                __syncwarp();
            };
            // half of a step's keys, as soon as their weights are there
            const auto outputs = [&](int i, int32_t u, int half, bool first) {
                const uint64_t v = v_desc + (((u % C::kSlots) * C::kTileB) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < kKeys / 32; ++ks) {
                        const int k16 = half * (kKeys / 32) + ks;
                        mma_bf16_ts(tmem + 2 * kKeys + i * 128, tmem + i * kKeys + k16 * 8, v + ((k16 * 2048) >> 4),
                                    kO, !first || k16 > 0);
                    }
                }
                __syncwarp();
            };
            int32_t u = 0, q_round = 0;
            uint32_t p_parity = 0, o_parity = 0, o_used = 0;  // a bit a tile
            for (int32_t k = 0;; ++k) {
                follow(&bar.item_full[k & 1], (k >> 1) & 1);
                if (!go_on() || !s_item[k & 1].any) break;
                const int32_t steps = s_item[k & 1].steps;
                const int n_tiles = s_item[k & 1].rows > kRows ? 2 : 1;
                release(k);
                if (steps == 0) continue;
                const int qb = q_round % C::kQ;
                follow(&bar.q_full[qb], (q_round / C::kQ) & 1);
                full(u);
                ++q_round;
                tc::fence_after_sync();
                for (int i = 0; i < n_tiles; ++i) scores(qb, i, u);
                commit(&bar.empty[u % C::kSlots]);
                if (steps == 1) commit(&bar.q_empty[qb]);
                int32_t j = 0;
                for (int32_t stop = min(steps, kVote); j < steps && go_on(); stop = min(steps, stop + kVote)) {
                    for (; j < stop; ++j, u += 2) {
                        const bool more = j + 1 < steps;
                        for (int i = 0; i < n_tiles; ++i) {
                            const bool last = i == n_tiles - 1;
                            if (i == 0) full(u + 1);
                            // the last item's output has been read
                            if (j == 0 && ((o_used >> i) & 1)) follow(&bar.o_empty[i], ((o_parity >> i) & 1) ^ 1);
                            follow(&bar.p_full[i][0], (p_parity >> i) & 1);
                            tc::fence_after_sync();
                            outputs(i, u + 1, 0, j == 0);
                            follow(&bar.p_full[i][1], (p_parity >> i) & 1);
                            tc::fence_after_sync();
                            outputs(i, u + 1, 1, j == 0);
                            p_parity ^= 1u << i;
                            if (!more) {
                                commit(&bar.o_full[i]);
                                o_parity ^= 1u << i;
                                o_used |= 1u << i;
                            }
                            if (last) commit(&bar.empty[(u + 1) % C::kSlots]);
                            if (more) {
                                if (i == 0) full(u + 2);
                                tc::fence_after_sync();
                                scores(qb, i, u + 2);
                                if (last) {
                                    commit(&bar.empty[(u + 2) % C::kSlots]);
                                    if (j + 2 == steps) commit(&bar.q_empty[qb]);
                                }
                            }
                        }
                    }
                }
            }
            // every product has finished, and every arrival landed, before the block ends
            commit(&bar.done);
            if (!tc::mbar_wait_timed(&bar.done, 0, kWaitNs)) fine = false;
        } else if (warp == 13) {
            // ---- work -------------------------------------------------------------------
            // Items in order, key heads innermost.  Up to 32 requests, a lane each: the pairs of
            // row tiles with the most keys first, of any request, so that what is left at the
            // end is small (8 ragged chunks of 6,546 tokens: 83 us in the requests' order, 74 us so;
            // one of 8,192: 437 and 431).
            // More requests: pairs from the last request's last one down; the many items even
            // out by themselves.
            const int64_t items = total * a.kv.n_kv;
            const bool by_size = a.n_seq <= 32;
            // by size: this lane's request
            RequestRows rows{0, 0, 0, false};
            int32_t pairs_here = 0;
            const auto item_of = [&](int32_t seq, const RequestRows &r, int32_t pair) {
                Item it;
                it.seq = seq;
                it.head = 0;
                it.row0 = pair * 2 * kRows;
                it.rows = min(2 * kRows, r.n * a.group - it.row0);
                it.q0 = r.q0;
                it.n = r.n;
                it.len = r.len;
                const int32_t first = r.len - r.n + it.row0 / a.group;
                const int32_t last = r.len - r.n + (it.row0 + it.rows - 1) / a.group;
                it.lo = a.window > 0 ? static_cast<int32_t>(max(int64_t(0), int64_t(first) - a.window + 1)) : 0;
                it.key0 = it.lo & ~(kKeys - 1);
                it.steps = last < 0 ? 0 : (last - it.key0) / kKeys + 1;
                it.part = 0;
                it.parts = 1;
                it.any = true;
                return it;
            };
            if (by_size && lane < a.n_seq) {
                rows = load_rows(a, lane);
                pairs_here = static_cast<int32_t>(pairs_of(rows));
            }
            const int32_t longest = static_cast<int32_t>(
                __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(rows.len) / kKeys));
            // this lane's pairs whose last row's position is at least 128 b: it grows with the pair
            const auto at_least = [&](int32_t b) -> uint32_t {
                const int64_t x = (int64_t(b) * kKeys - (rows.len - rows.n)) * a.group;  // rows before it
                if (b <= 0 || x <= 0) return pairs_here;
                if (x >= int64_t(rows.n) * a.group) return 0;
                return pairs_here - min(pairs_here, static_cast<int32_t>(x / (2 * kRows)));
            };
            // in order: the pairs above the walk's request are `above`
            int64_t above = total;
            int32_t seq = a.n_seq;  // requests from here on have been passed
            int64_t idx = blockIdx.x;
            // where items are split: neighbouring blocks take an item's parts.  (Offsets out of
            // order, which are reported, can make more items than the rows of the call: then
            // whole ones, in turn.)
            const int32_t most = SPLIT ? static_cast<int32_t>(max(int64_t(1), min(int64_t(kMaxParts),
                                                                                  gridDim.x / max(items, int64_t(1))))) : 1;
            if (SPLIT) idx = blockIdx.x / most;
            int32_t rest = 0;  // steps of the last item still to be handed out, in the lane that found it
            for (int32_t k = 0;; ++k) {
                Item it{};
                const bool more = __any_sync(0xffffffffu, rest > 0);
                if (more) {
                    if (rest > 0) {
                        it = s_item[(k - 1) & 1];
                        it.steps = min(rest, kSegment);
                        it.key0 -= it.steps * kKeys;
                        it.first = false;
                    }
                } else if (idx < items && by_size) {
                    // the largest b with more than `want` pairs at or above it, by bisection
                    const uint32_t want = static_cast<uint32_t>(idx / a.kv.n_kv);
                    int32_t lo = 0, hi = longest;
                    while (lo < hi) {
                        const int32_t mid = (lo + hi + 1) >> 1;
                        if (__reduce_add_sync(0xffffffffu, at_least(mid)) > want) lo = mid;
                        else hi = mid - 1;
                    }
                    // among the pairs of that size: by request, then from the last down
                    const uint32_t beyond = at_least(lo + 1), same = at_least(lo) - beyond;
                    const uint32_t r = want - __reduce_add_sync(0xffffffffu, beyond);
                    uint32_t incl = same;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
                        if (lane >= o) incl += v;
                    }
                    if (r >= incl - same && r < incl) {
                        it = item_of(lane, rows, pairs_here - 1 - static_cast<int32_t>(beyond + (r - (incl - same))));
                        it.head = static_cast<int32_t>(idx % a.kv.n_kv);
                    }
                } else if (idx < items) {
                    const int64_t want = total - 1 - idx / a.kv.n_kv;
                    // 32 requests at a time: lane l holds request seq - 1 - l
                    while (seq > 0) {
                        const int32_t i = seq - 1 - lane;
                        RequestRows r{0, 0, 0, false};
                        if (i >= 0) r = load_rows(a, i);
                        const int64_t pairs = i >= 0 ? pairs_of(r) : 0;
                        int64_t incl = pairs;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
                            if (lane >= o) incl += v;
                        }
                        const bool ours = i >= 0 && pairs > 0 && want >= above - incl && want < above - incl + pairs;
                        const uint32_t who = __ballot_sync(0xffffffffu, ours);
                        if (who != 0) {
                            if (ours) {
                                it = item_of(i, r, static_cast<int32_t>(want - (above - incl)));
                                it.head = static_cast<int32_t>(idx % a.kv.n_kv);
                            }
                            // the requests before the one found stay passed over
                            const int l = __ffs(who) - 1;
                            above -= __shfl_sync(0xffffffffu, incl - pairs, l);
                            seq -= l;
                            break;
                        }
                        above -= __shfl_sync(0xffffffffu, incl, 31);
                        seq -= 32;
                    }
                }
                if (SPLIT && it.any && !more) {
                    it.parts = max(1, min(most, it.steps / kMinSteps));
                    it.part = blockIdx.x % most;
                    it.any = it.part < it.parts;
                    const int32_t from = it.steps * it.part / it.parts;
                    it.steps = it.steps * (it.part + 1) / it.parts - from;
                    it.key0 += from * kKeys;
                }
                if (it.any) {
                    if (!more) {
                        rest = it.steps;
                        it.steps = min(rest, kSegment);
                        it.key0 += (rest - it.steps) * kKeys;
                        it.first = true;
                    }
                    rest -= it.steps;
                    it.last = rest == 0;
                }
                if (k >= 2 && !wait(&bar.item_empty[k & 1], ((k >> 1) - 1) & 1)) break;
                const bool any = __any_sync(0xffffffffu, it.any);
                if (it.any || (!any && lane == 0)) {
                    s_item[k & 1] = it;
                    tc::mbar_arrive(&bar.item_full[k & 1]);
                }
                __syncwarp();
                if (!any) {
                    // the last block to come to the end leaves the claims as they were
                    if (lane == 0 && atomicAdd(&claims->done, 1) == static_cast<int32_t>(gridDim.x) - 1) {
                        claims->given = 0;
                        claims->done = 0;
                    }
                    break;
                }
                const bool done = !__any_sync(0xffffffffu, rest > 0);
                if (SPLIT) {  // a block has one item, unless there are more items than blocks
                    if (done) idx = most == 1 ? idx + gridDim.x : items;
                    continue;
                }
                // the next item is claimed when the copies come to this one's last step: late
                // enough that blocks with short items take more, early enough to hide the claim
                if (!wait(&bar.claim, k & 1)) break;
                if (!done) continue;
                int32_t next = 0;
                if (lane == 0) next = atomicAdd(&claims->given, 1);
                idx = int64_t(gridDim.x) + __shfl_sync(0xffffffffu, next, 0);
            }
        }
    } else {
        set_registers<C::kSoftmaxRegs, true>();
        // ---- softmax --------------------------------------------------------------------
        const int i = warp >> 2, r = i * kRows + (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + i * kKeys, o_at = tmem + lanes + 2 * kKeys + i * 128;
        const bool plain = a.softcap == 0.0f && a.slopes == nullptr && a.scale > 0.0f;
        int32_t round = 0, o_round = 0;
        for (int32_t k = 0;; ++k) {
            follow(&bar.item_full[k & 1], (k >> 1) & 1);
            if (!go_on() || !s_item[k & 1].any) break;
            // the item stays in shared memory: registers are scarce in the loop below
            const Item &it = s_item[k & 1];
            const int32_t steps = it.steps, key0 = it.key0, first_pos = it.len - it.n;
            const bool live = r < it.rows;
            if (it.rows <= i * kRows) {  // this tile has no rows
                release(k);
                continue;
            }
            const int32_t row = it.row0 + r;
            const int32_t pos = live ? first_pos + row / a.group : -1;
            const int32_t pos_lo = first_pos + (it.row0 + i * kRows) / a.group;
            const int32_t pos_hi = first_pos + (it.row0 + min(it.rows, (i + 1) * kRows) - 1) / a.group;
            const float slope = live && a.slopes != nullptr ? a.slopes[it.head * a.group + row % a.group] * kLog2e : 0.0f;
            float mult = a.scale * a.kv.k_scale;
            if constexpr (E4M3) {
                // (an item's exponents stay until the item is released)
                follow(&bar.exp_full[k & 1], (k >> 1) & 1);
                if (steps > 0) mult *= __uint_as_float(static_cast<uint32_t>(127 + s_qexp[k & 1][r]) << 23);
            }
            const float by0 = mult * kLog2e;
            float m = -INFINITY, l = 0.0f;  // the reference of the row's weights, and their sum
            for (int32_t j = 0; j < steps; ++j, ++round) {
                if (!wait(&bar.s_full[i], round & 1)) break;
                tc::fence_after_sync();
                const int32_t key = key0 + (steps - 1 - j) * kKeys;
                const bool masked = key + kKeys - 1 > pos_lo || (a.window > 0 && pos_hi - key >= a.window);
                const bool direct = plain && !masked;
                const float by = direct ? by0 : 1.0f;
                uint32_t x[128];
                const auto load_scores = [&]() {
                    tmem_ld64(s_at, x);
                    tmem_ld64(s_at + 64, x + 64);
                    tmem_wait128(x);
                };
                load_scores();
                bool final_form = direct;
                if (!masked && a.softcap > 0.0f) {
                    float far4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int e = 0; e < 128; e += 2)
                        far4[(e / 2) & 3] = fmaxf(fmaxf(far4[(e / 2) & 3], fabsf(__uint_as_float(x[e]))),
                                                  fabsf(__uint_as_float(x[e + 1])));
                    final_form = __all_sync(0xffffffffu, near_cap(a, mult, fmaxf(fmaxf(far4[0], far4[1]),
                                                                                 fmaxf(far4[2], far4[3]))));
                    if (final_form) {
                        const NearForm form(a, mult, slope, key - pos);
#pragma unroll
                        for (int e = 0; e < 128; e += 2) {
                            float s0, s1;
                            unpack2(form.capped(pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])),
                                                static_cast<float>(e)), s0, s1);
                            x[e] = __float_as_uint(s0);
                            x[e + 1] = __float_as_uint(s1);
                        }
                    }
                }
                if (!final_form) {
                    // masks, biases without a cap, scores beyond half their cap: in place, 64 at a time (one
                    // copy of the code)
#pragma unroll 1
                    for (int c = 0; c < 2; ++c) {
                        uint32_t y[64];
                        float s[64];
                        tmem_ld64(s_at + 64 * c, y);
                        tmem_wait64(y);
#pragma unroll
                        for (int e = 0; e < 64; ++e) s[e] = __uint_as_float(y[e]);
                        finish_scores<64, 2>(s, a, mult, slope, key + 64 * c - pos, masked);
#pragma unroll
                        for (int e = 0; e < 64; ++e) y[e] = __float_as_uint(s[e]);
                        tmem_st32(s_at + 64 * c, y);
                        tmem_st32(s_at + 64 * c + 32, y + 32);
                    }
                    tmem_wait_st();
                    load_scores();
                }
                float top8[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    top8[q] = fmaxf(__uint_as_float(x[2 * q]), __uint_as_float(x[2 * q + 1]));
#pragma unroll
                    for (int e = 16 + 2 * q; e < 128; e += 16)
                        top8[q] = fmaxf(fmaxf(top8[q], __uint_as_float(x[e])), __uint_as_float(x[e + 1]));
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) top8[q] = fmaxf(top8[q], top8[q + 4]);
                const float top = fmaxf(fmaxf(top8[0], top8[1]), fmaxf(top8[2], top8[3])) * by;
                // the reference only moves when it must; then the sum and O follow
                if (__any_sync(0xffffffffu, top > m + kGrow || (m == -INFINITY && top > m))) {
                    const float now = fmaxf(m, top), f = now == -INFINITY ? 1.0f : ex2(m - now);
                    m = now;
                    l *= f;
                    if (j > 0) rescale_output<HD>(o_at, f);
                }
                const float ref = kShift - (m == -INFINITY ? 0.0f : m);
                const uint64_t by2 = pack2(by, by), ref2 = pack2(ref, ref);
                uint64_t sum[2] = {0, 0};  // of the step, pairs of fp32: a long row's sum has no room for single weights
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float p0, p1;
                        const int k2 = 32 * c + 2 * e;
                        unpack2(fma2(pack2(__uint_as_float(x[k2]), __uint_as_float(x[k2 + 1])), by2, ref2), p0, p1);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        sum[e & 1] = add2(sum[e & 1], pack2(p0, p1));
                        p[e] = E4M3 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
                    }
                    tmem_st16(s_at + 16 * c, p);
                    if (c & 1) {  // half of the step's weights
                        tmem_wait_st();
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(&bar.p_full[i][c >> 1]);
                    }
                }
                float even, odd;
                unpack2(add2(sum[0], sum[1]), even, odd);
                l += even + odd;
            }
            if (steps > 0) follow(&bar.o_full[i], o_round & 1);
            if (!go_on()) break;
            tc::fence_after_sync();
            // the segments before this one, and for the one after it
            float *const carried = partials + blockIdx.x * kPartial<HD>;
            if (!it.first) add_segments<HD>(carried, r, o_at, m, l);
            if (!it.last) {
                leave_segments<HD>(carried, r, o_at, m, l);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar.o_empty[i]);
                ++o_round;
                release(k);
                continue;
            }
            // (a block has one item where items are in parts, and the parts are neighbouring blocks')
            if (SPLIT && it.parts > 1 &&
                !join_parts<HD>(partials + (blockIdx.x - it.part) * kPartial<HD>,
                                flags + (blockIdx.x - it.part), it.part, it.parts, r, o_at, m, l, warp, lane)) {
                release(k);
                continue;
            }
            const float inv = l > 0.0f ? a.kv.v_scale / l : l == 0.0f ? 0.0f : l;
            const int32_t out_row = it.row0 + r, h = it.head * a.group + out_row % a.group;
            const int64_t t = it.q0 + (live ? out_row / a.group : 0);
            uint16_t *dst = a.out + t * a.ldo + h * HD;
#pragma unroll
            for (int c = 0; c < HD / 32; ++c) {
                uint32_t x[32], o[16];
                if (steps > 0) {
                    tmem_ld32(o_at + 32 * c, x);
                    tmem_wait(x);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = 0u;
                }
                if (c == HD / 32 - 1 && steps > 0) {  // all of O is in registers
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bar.o_empty[i]);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    o[e] = pack_bf16x2(__uint_as_float(x[2 * e]) * inv, __uint_as_float(x[2 * e + 1]) * inv);
                if (live) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        stg_u4(dst + 32 * c + 8 * e, make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
                }
            }
            if (steps > 0) ++o_round;
            if (live && a.lse != nullptr)
                a.lse[t * a.n_heads + h] = l == 0.0f ? -INFINITY : kLn2 * (m - kShift) + logf(l);
            release(k);
        }
    }
    // a wait that gave up stops the block's other roles; what is in flight lands before
    // the tensor memory goes
    if (!__all_sync(0xffffffffu, fine)) {
        s_abort = 1;
        report_error(a.err, LORA_ERR_TIMEOUT);
        __nanosleep(1000000);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 12) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int HD, bool E4M3, bool SPLIT>
cudaError_t prepare(int *sms) {
    static std::atomic<uint64_t> seen{0};
    const cudaError_t e = prepare_kernel(attend_prompt_kernel<HD, E4M3, SPLIT>, PromptConfig<HD>::kSmem, seen, sms);
    if (*sms > kMaxGrid) *sms = kMaxGrid;
    return e;
}

template <int HD, bool E4M3>
cudaError_t launch(const AttendArgs &a, void *ws, cudaStream_t stream) {
    // flags (a word a block: an item has as many words as blocks, and needs 2, or 4 for more than
    // 8 parts) and partials take the places of the decode path's counters and partials
    char *bytes = static_cast<char *>(ws);
    Claims *claims = reinterpret_cast<Claims *>(bytes + 768);
    uint32_t *flags = reinterpret_cast<uint32_t *>(bytes);
    float *partials = reinterpret_cast<float *>(bytes + 1024);
    // every request's rows fill pairs of tiles but for one
    const int64_t items = (int64_t(a.T) * a.group / (2 * kRows) + a.n_seq) * a.kv.n_kv;
    constexpr int kSmem = PromptConfig<HD>::kSmem;
    int sms = 0;
    cudaError_t e = prepare<HD, E4M3, true>(&sms);
    if (e != cudaSuccess) return e;
    // with no more than half of the SMs busy, parts of items for the others
    if (2 * items <= sms)
        return launch_dependent(attend_prompt_kernel<HD, E4M3, true>, sms, kThreads, kSmem, stream, a, claims, flags,
                                partials);
    if ((e = prepare<HD, E4M3, false>(&sms)) != cudaSuccess) return e;
    return launch_dependent(attend_prompt_kernel<HD, E4M3, false>, static_cast<unsigned>(items < sms ? items : sms),
                            kThreads, kSmem, stream, a, claims, flags, partials);
}

}  // namespace

cudaError_t launch_attend_prompt(const AttendArgs &a, bool e4m3, void *ws, cudaStream_t stream) {
    if (a.kv.head_dim == 64) return e4m3 ? launch<64, true>(a, ws, stream) : launch<64, false>(a, ws, stream);
    return e4m3 ? launch<128, true>(a, ws, stream) : launch<128, false>(a, ws, stream);
}

}  // namespace lora

// Attention of requests that share a prefix (lora_attend_shared).
//
// The keys of a group's prefix are read once for all of its rows: with R rows of a
// key head (tokens x query heads of it) a key costs 4 head_dim bytes and 4 R head_dim
// operations, so that HBM bounds it up to about 256 rows and the tensor cores from
// there on.  Three kernels:
//   attend_prefix_kernel  partial results (reference, sum, output) of every row over its
//                         group's prefix: S = Q K^T, P, O += P V on tcgen05 with
//                         accumulators in tensor memory, two tiles of 128 rows a block
//   attend_decode_kernel  partial results of the rows over their requests' own keys, by
//                         the decode path, its keys starting behind the prefix; rows
//                         of requests that share nothing are finished there
//   attend_join_kernel    a row's partial results joined, in the order of the keys
//
// The prefix kernel spreads the keys: a segment is (group, key head, 256 rows), a step
// 128 of its keys; all steps of the call, in order, are cut into equal shares, one a
// block, so one long prefix fills the GPU and many short ones share a block.  Every
// block finds the groups' prefixes and the shares by itself, from the lengths.  A
// piece that starts with its segment leaves its result at the rows' own place, another
// one (a block has one at most) at the block's.  Nothing waits for another block.
//
// Short calls compute prefixes on some SMs and own keys on the others, in numbers that follow
// the estimated costs; long ones take all SMs for each in turn (shared_plan.cuh).  The own
// keys' kernel starts as soon as all blocks of the prefix kernel run, without a wait.
//
// Measured, 32/8 heads of 128 over bf16, one row a request, graph replay: 16 prompts of 20,000 to
// 30,000 tokens with 16 samples each 343 us, 5.9 TB/s of what has to be read (each prefix for each
// request: 3,361); the prefixes' part reads 1.64 GB in 263 us, 6.2 TB/s.  64 requests of 100 to 1,000
// own tokens behind one prompt of 8,000 54 us (each on its own 178), of which HBM needs 20: 11 us pass
// until the first scores (lengths, plan, queries, first keys), 8 to 10 at the end (results left,
// pieces joined, one launch), and a step takes 2.2 us where blocks start together, 1.6 later on.
// 4 requests behind 30,000 tokens 49 us (72).
//
// Blocks are organised like those of the prompt path: warps 0-3 and 4-7 softmax of a
// tile's rows, a row a thread; 8-11 copy; 12 issues the products; 13 hands out the
// pieces.  Weights are rounded to bf16 over a bf16 cache (the instruction takes one type
// for both operands; sums use them unrounded), to f16, times 2^7, over an e4m3 cache: as on the
// prompt path, and fewer bits than the decode path gives the own keys (16, f16 times 2^12).  With a
// second product for the weights' remainders the 64 requests above take 60.7 us in place of 53.9 and the 16
// prompts 351 in place of 341, and outputs lie 0.0016 and 0.0015 (rms, relative) from 64 bits in place of
// 0.0017 and 0.0016: the output's own rounding is 0.0016.
#include "attend_tc.cuh"
#include "shared_plan.cuh"

namespace lora {

size_t decode_workspace_bytes(int32_t head_dim);
cudaError_t launch_attend_own(const AttendArgs &a, bool e4m3, const Groups &groups, float4 *sums, float *outs,
                              const int32_t *blocks, int32_t *live, void *ws, cudaStream_t stream);
const float *own_pieces(const void *ws);

namespace {

constexpr int kThreads = 16 * 32, kMaxGrid = kPrefixBlocks;

static_assert(kPrefixRows == 2 * kRows && kPrefixKeys == kKeys, "a step");

// The tensor cores cut off what does not fit when they add to O, about 2^-24 of it with
// every 16 keys: more steps than these are taken one after the other and added up in fp32.
constexpr int32_t kSegment = 512;

template <int HD>
struct PrefixConfig {
    static constexpr int kTileB = kRows * HD * 2;
    static constexpr int kSlots = HD == 128 ? 5 : 8;  // k and v tiles in the ring
    static constexpr int kQ = HD == 128 ? 1 : 2;      // pieces whose q rows fit
    static constexpr int kSmem = (2 * kQ + kSlots) * kTileB + 1024;
    static constexpr uint32_t kHalfB = kRows * 128;   // 64 dims of all rows
    // registers a thread by role, as on the prompt path
    static constexpr int kSoftmaxRegs = HD == 128 ? 168 : 184;
    static constexpr int kCopyRegs = HD == 128 ? 104 : 80;
    static constexpr int kMmaRegs = HD == 128 ? 72 : 64;
    static_assert(2 * kSoftmaxRegs + kCopyRegs + kMmaRegs == 4 * 128, "registers of the block");
};

// What the kernels of a call hand over.  Every block of the prefix kernel writes the same
// lists of groups (and reads what it wrote itself, or what is equal to it).
struct SharedWork {
    Groups groups;
    int64_t *units;               // by group: steps (and openings) before it, n_groups + 1
    int32_t *prefix, *lo, *lead;  // by group, of its plan
    int32_t *own_blocks;          // that take part in the own keys; 0 between calls
    int32_t *gave_up;             // whether a wait did: pieces are missing; stays until the workspace is zeroed again
    int32_t *live;                // whether there is anything to join; then by token, whether its request shares
    float4 *own_sums;             // of a row over its own keys, see OwnRows
    float *own_outs;
    const float *own_cuts;
    float4 *heads;                // reference and sum over the prefix; place of the row's other pieces and their number
    float *outs;                  // its output, as above
    float4 *cut_heads;            // of a block's piece, 256 rows a block
    float *cut_outs;
};

struct Barriers {
    uint64_t q_full[2], q_empty[2], full[8], empty[8], s_full[2], p_full[2][2], o_full[2], o_empty[2], item_full[2],
        item_empty[2], exp_full[2], half_full, done;
};

// A piece: up to 256 rows of a group and key head, and the keys [lo, end) of its steps.
struct Item {
    int32_t lead, head;              // request whose table row is read, key head
    int32_t q0, row0, rows;          // the group's first token; first row and rows of the tiles
    int32_t key0, steps, lo, end;
    int32_t cut, first_cut, cuts;    // cut: the block's own place; of a segment's first piece, the other pieces
    bool first, last;                // of the piece's runs of kSegment steps
    bool any;                        // none: the work is done

    // With up to 128 rows the block's two halves share them, taking turns at the steps: one's softmax
    // runs beside the other's products.  64 groups of 2 requests behind 4,000 tokens 210 us, else 220;
    // 32 of 4 behind 2,000 90 and 96.  Not over e4m3, where widening the codes bounds a step and the ring, with
    // k a step ahead, has less room for it: 32 of 4 behind 2,000 126 us so, else 108.
    template <bool E4M3>
    __device__ bool split() const { return !E4M3 && rows <= kRows && steps > 1; }
};

// Tiles of a piece in the ring's order: k and v in turn; where halves take turns, k is a step
// ahead: k0 k1 v0 k2 v1 .. k(n-1) v(n-2) v(n-1).
__device__ __forceinline__ int32_t k_place(int32_t j, bool split) { return split ? max(0, 2 * j - 1) : 2 * j; }
__device__ __forceinline__ int32_t v_place(int32_t j, int32_t n, bool split) {
    return split ? min(2 * j + 2, 2 * n - 1) : 2 * j + 1;
}

// The group that a block's share begins in, and the units before it.
struct First {
    int64_t before;
    int32_t group;
};

// The lists of the call's groups in global memory, by the whole block, and where its share (of
// all units over `blocks`) begins; returns all units.
__device__ int64_t list_groups(const AttendArgs &a, const SharedWork &w, const GroupPlan &p, int64_t *s_sum,
                               int32_t blocks, First *s_first) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t n = w.groups.n_groups;
    const int32_t per = (n + kThreads - 1) / kThreads, g0 = min(n, tid * per), g1 = min(n, g0 + per);
    int64_t mine = 0;
    for (int32_t g = g0; g < g1; ++g) mine += prefix_units(a, p, g);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int64_t run = incl - mine, total = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) run += s_sum[i];
        total += s_sum[i];
    }
    const int64_t share = (total + blocks - 1) / blocks, x0 = blockIdx.x * share;
    for (int32_t g = g0; g < g1; ++g) {
        const int64_t units = prefix_units(a, p, g);
        if (run <= x0 && x0 < run + units) *s_first = {run, g};
        w.units[g] = run;
        w.prefix[g] = p.prefix[g];
        w.lo[g] = p.lo[g];
        w.lead[g] = p.lead[g];
        run += units;
    }
    if (tid == 0) w.units[n] = total;
    return total;
}

// The lane's row left at its place, or added to what it left there before.
template <int HD>
__device__ __forceinline__ void leave_row(float4 *head, float *out, int64_t stride, const Item &it, int r, uint32_t o_at,
                                          float m, float l, bool live, float kshift) {
    if (live) *head = make_float4(m - kshift, l, __int_as_float(it.first_cut << 8 | r), __int_as_float(it.cuts));
#pragma unroll 1
    for (int c = 0; c < HD / 16; ++c) {
        uint32_t x[16];
        tc::tmem_ld16(o_at + 16 * c, x);
        if (live) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                stg_u4(out + (4 * c + e) * stride, make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]));
        }
    }
}

template <int HD>
__device__ __forceinline__ void add_row(const float4 *head, const float *out, int64_t stride, uint32_t o_at, float &m,
                                        float &l, bool live, float kshift) {
    const float4 h = live ? ldg_cg_f4(reinterpret_cast<const float *>(head)) : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
    const float m2 = h.x + kshift;
    const float top = fmaxf(m, m2), ref = top == -INFINITY ? 0.0f : top, w = ex2(m - ref), w2 = ex2(m2 - ref);
    m = top;
    l = fmaf(w2, h.y, w * l);
#pragma unroll 1
    for (int c = 0; c < HD / 16; ++c) {
        uint32_t x[16];
        tc::tmem_ld16(o_at + 16 * c, x);
        if (live) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 v = ldg_cg_f4(out + (4 * c + e) * stride);
                x[4 * e] = __float_as_uint(fmaf(w2, v.x, w * __uint_as_float(x[4 * e])));
                x[4 * e + 1] = __float_as_uint(fmaf(w2, v.y, w * __uint_as_float(x[4 * e + 1])));
                x[4 * e + 2] = __float_as_uint(fmaf(w2, v.z, w * __uint_as_float(x[4 * e + 2])));
                x[4 * e + 3] = __float_as_uint(fmaf(w2, v.w, w * __uint_as_float(x[4 * e + 3])));
            }
        }
        tmem_st16(o_at + 16 * c, x);
    }
    tmem_wait_st();
}

template <int HD, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) attend_prefix_kernel(const AttendArgs a, const SharedWork w) {
    using C = PrefixConfig<HD>;
    constexpr float kShift = E4M3 ? 7.0f : 0.0f;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Barriers bar;
    __shared__ Item s_item[2];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int32_t s_abort;
    __shared__ float2 s_half[kRows];  // references and sums of the second half's rows; before, the plan's sums
    int64_t *const s_sum = reinterpret_cast<int64_t *>(s_half);
    static_assert(sizeof(s_half) >= 4 * kThreads / 32 * sizeof(int64_t), "sums");
    __shared__ int8_t s_qexp[2][E4M3 ? 2 * kRows : 1];  // of this and the next piece: q rows' powers of two
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t q_base = (tc::smem_u32(smem_raw) + 1023) & ~1023u;  // q tiles of kQ pieces, then the ring
    const uint32_t ring = q_base + 2 * C::kQ * C::kTileB;

    __shared__ First s_first;
    wait_for_previous();
    if (warp == 12) tc::tmem_alloc(&s_tmem, 512);
    const GroupPlan plan(reinterpret_cast<int32_t *>(smem_raw), w.groups.n_groups, a.n_seq);  // (the ring's place)
    bool bad;
    const Blocks counts = plan_groups<kThreads>(a, w.groups, plan, s_sum, gridDim.x, blockIdx.x == 0, &bad);
    const int32_t blocks = counts.prefix;
    if (blockIdx.x == 0 && tid == 0) {
        w.live[0] = blocks > 0;
        w.own_blocks[0] = counts.own;
    }
    // blocks without a share leave their SM to the next kernel
    if (static_cast<int32_t>(blockIdx.x) >= blocks) {
        __syncthreads();
        tc::fence_after_sync();
        if (warp == 12) tc::tmem_dealloc(s_tmem, 512);
        return;
    }
    const int64_t total = list_groups(a, w, plan, s_sum, blocks, &s_first);
    const int64_t share = (total + blocks - 1) / blocks;
    const int64_t x0 = min(total, blockIdx.x * share), x1 = min(total, x0 + share);
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
        tc::mbar_init(&bar.half_full, 4);
        tc::mbar_init(&bar.done, 1);
        tc::mbar_init_fence();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;
    // Waits of a whole warp; their outcome steers it by votes only (see the prompt path).  After
    // follow() a lane that gave up ends the block's other waits and goes on, in bounds, until go_on().
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
    // a warp lets go of the block's k-th piece
    const auto release = [&](int32_t k) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar.item_empty[k & 1]);
    };

    if (warp >= 8 && warp < 12) {
        set_registers<C::kCopyRegs, false>();
        // ---- copies ---------------------------------------------------------------------
        const int cw = warp - 8;
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
        int32_t u = 0, q_round = 0;  // tiles and pieces so far
        for (int32_t k = 0;; ++k) {
            follow(&bar.item_full[k & 1], (k >> 1) & 1);
            if (!go_on() || !s_item[k & 1].any) break;
            const Item &it = s_item[k & 1];
            const int32_t steps = it.steps, lo = it.lo, end = it.end;
            const bool split = it.template split<E4M3>();
            const int32_t *table = a.table + it.lead * a.ld_table;
            const int64_t head = it.head * a.kv.head_b;
            // this lane's key of the step to copy (the last keys first) and, ahead of it, its page
            int32_t key = it.key0 + (steps - 1) * kKeys + cw * 32 + lane, page = -1;
            const auto has_key = [&]() { return key >= lo && key < end; };
            if (has_key()) page = table[key >> a.kv.page_shift];
            const int qb = q_round % C::kQ;
            const uint32_t q_at_base = q_base + qb * 2 * C::kTileB;
            const auto q_piece = [&](int r) { return q_at_base + (r / kRows) * C::kTileB + tile_at(r % kRows, piece); };
            if (q_round >= C::kQ) follow(&bar.q_empty[qb], (q_round / C::kQ - 1) & 1);
            ++q_round;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                // 32 rows of q: a lane's row's offset, then a few rows an instruction
                const int r0 = cw * 64 + half * 32, row = it.row0 + r0 + lane;
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
                    const int r = cw * 64 + half * 32 + lane;
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
                publish(&bar.q_full[qb]);
                if (lane == 0) tc::mbar_arrive(&bar.exp_full[k & 1]);
            } else {
                tc::cp_commit();
            }
            release(k);  // nothing below reads the piece

            // byte offset of this lane's key, -1: none; of the last k tile's, and of the one before it
            int64_t at = -1, new_at = -1, old_at = -1;
            // all keys there, and 16 neighbours always in one page
            bool smooth = false, new_smooth = false, old_smooth = false;
            const auto next_keys = [&]() {
                old_at = new_at;
                old_smooth = new_smooth;
                const bool ok = page >= 0 && page < a.kv.n_pages, has = has_key();
                if (has && !ok) report_error(a.err, LORA_ERR_SLOT_RANGE);
                new_at = has && ok ? page * a.kv.page_b + (key & a.kv.page_mask) * a.kv.token_b + head : -1;
                new_smooth = __all_sync(0xffffffffu, new_at >= 0) && a.kv.page_shift >= 4;
                key -= kKeys;
                if (has_key()) page = table[key >> a.kv.page_shift];
            };
            // the t-th tile: whether it is v, and its keys
            const auto tile_is_v = [&](int32_t t) {
                const bool v = split ? t > 1 && ((t & 1) == 0 || t == 2 * steps - 1) : t & 1;
                if (!v) next_keys();
                const bool old = v && split && t < 2 * steps - 1;
                at = old ? old_at : new_at;
                smooth = old ? old_smooth : new_smooth;
                return v;
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
                    const bool is_v = tile_is_v(t);
                    each(is_v ? a.kv.v : a.kv.k, [&](int i, const unsigned char *src) {
                        v[i] = src != nullptr ? ldg_cg(src) : make_uint4(0, 0, 0, 0);
                    });
                };
                load(0);
                for (int32_t t = 0; t < tiles; ++t, ++u) {
                    if (!slot_free()) break;
                    const uint32_t dst = ring + (u % C::kSlots) * C::kTileB;
#pragma unroll
                    for (int i = 0; i < kKvPieces; ++i) {
                        const int row = cw * 32 + i * kKvStep + kv_row;
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
                    const bool is_v = tile_is_v(t);
                    if (!slot_free()) break;
                    const uint32_t dst = ring + (u % C::kSlots) * C::kTileB;
                    each(is_v ? a.kv.v : a.kv.k, [&](int i, const unsigned char *src) {
                        tc::cp16(dst + tile_at(cw * 32 + i * kKvStep + kv_row, kv_piece), src != nullptr ? src : a.kv.k,
                                 src != nullptr);
                    });
                    tc::cp_commit();
                    // the tile two before this one (and q before all) has landed
                    tc::cp_wait_group<2>();
                    if (t == 1) publish(&bar.q_full[qb]);
                    if (t >= 2) publish(&bar.full[(u - 2) % C::kSlots]);
                }
                tc::cp_wait_group<1>();
                publish(&bar.full[(u - 2) % C::kSlots]);
                tc::cp_wait_group<0>();
                publish(&bar.full[(u - 1) % C::kSlots]);
            }
        }
        tc::cp_wait_all();
    } else if (warp >= 12) {
        set_registers<C::kMmaRegs, false>();
        if (warp == 12) {
            // ---- products ---------------------------------------------------------------
            constexpr uint32_t kType = E4M3 ? (1u << 7) | (1u << 10) : 0u;  // f16 has 0 where bf16 has 1
            constexpr uint32_t kS = tc::idesc_bf16(kRows, kKeys) ^ kType;
            constexpr uint32_t kO = (tc::idesc_bf16(kRows, HD) ^ kType) | (1u << 16);  // v: keys are strided
            // descriptors are a tile's plus a constant: addresses stay below 2^18, so nothing carries
            const uint64_t q_desc = desc128(q_base, 16, 1024), k_desc = desc128(ring, 16, 1024);
            const uint64_t v_desc = desc128(ring, C::kHalfB, 1024);
            const auto full = [&](int32_t u) { follow(&bar.full[u % C::kSlots], (u / C::kSlots) & 1); };
            const auto commit = [&](uint64_t *b) {
                if (elect_one()) tc::mma_commit(b);
                __syncwarp();
            };
            const auto scores = [&](int q_tile, int i, int32_t u) {
                const uint64_t q = q_desc + ((q_tile * C::kTileB) >> 4), k = k_desc + (((u % C::kSlots) * C::kTileB) >> 4);
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
                const bool split = s_item[k & 1].template split<E4M3>();
                release(k);
                const int qb = q_round % C::kQ;
                follow(&bar.q_full[qb], (q_round / C::kQ) & 1);
                full(u);
                ++q_round;
                tc::fence_after_sync();
                for (int i = 0; i < n_tiles; ++i) scores(2 * qb + i, i, u);
                commit(&bar.empty[u % C::kSlots]);
                if (steps == 1) commit(&bar.q_empty[qb]);
                int32_t j = 0;
                if (split) {
                    full(u + 1);
                    tc::fence_after_sync();
                    scores(2 * qb, 1, u + 1);
                    commit(&bar.empty[(u + 1) % C::kSlots]);
                    if (steps == 2) commit(&bar.q_empty[qb]);
                    for (int32_t stop = min(steps, kVote); j < steps && go_on(); stop = min(steps, stop + kVote)) {
                        for (; j < stop; ++j) {
                            const int i = j & 1;
                            const int32_t v = u + v_place(j, steps, true);
                            full(v);
                            // the last piece's output has been read
                            if (j < 2 && ((o_used >> i) & 1)) follow(&bar.o_empty[i], ((o_parity >> i) & 1) ^ 1);
                            follow(&bar.p_full[i][0], (p_parity >> i) & 1);
                            tc::fence_after_sync();
                            outputs(i, v, 0, j < 2);
                            follow(&bar.p_full[i][1], (p_parity >> i) & 1);
                            tc::fence_after_sync();
                            outputs(i, v, 1, j < 2);
                            p_parity ^= 1u << i;
                            if (j + 2 >= steps) {
                                commit(&bar.o_full[i]);
                                o_parity ^= 1u << i;
                                o_used |= 1u << i;
                            }
                            commit(&bar.empty[v % C::kSlots]);
                            if (j + 2 < steps) {
                                const int32_t kt = u + k_place(j + 2, true);
                                full(kt);
                                tc::fence_after_sync();
                                scores(2 * qb, i, kt);
                                commit(&bar.empty[kt % C::kSlots]);
                                if (j + 3 == steps) commit(&bar.q_empty[qb]);
                            }
                        }
                    }
                    u += 2 * steps;
                    continue;
                }
                for (int32_t stop = min(steps, kVote); j < steps && go_on(); stop = min(steps, stop + kVote)) {
                    for (; j < stop; ++j, u += 2) {
                        const bool more = j + 1 < steps;
                        for (int i = 0; i < n_tiles; ++i) {
                            const bool last = i == n_tiles - 1;
                            if (i == 0) full(u + 1);
                            // the last piece's output has been read
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
                                scores(2 * qb + i, i, u + 2);
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
            // ---- work: the block's pieces in order (every lane works out the same) ---------
            int64_t x = x0;
            int32_t g = 0, rest = 0;  // rest: steps of the last piece still to be handed out
            Item it{};
            // the piece of group g (whose units begin at `before`) that x lies in; x goes on to the next
            const auto open = [&](int64_t before, int32_t lo, int32_t end, int32_t lead, int32_t q0, int32_t q1) {
                const int32_t steps = prefix_steps(lo, end);
                const int64_t rows = int64_t(q1 - q0) * a.group, tiles = (rows + 2 * kRows - 1) / (2 * kRows);
                const int64_t i = (x - before) / (steps + kPrefixOpen), head = i / tiles, tile = i - head * tiles;
                const int64_t begin = before + i * (steps + kPrefixOpen) + kPrefixOpen;  // its first step
                const int64_t from = max(x, begin), to = min(x1, begin + steps);
                x = begin + steps;
                if (from >= to) return;  // only the opening lies in this share
                it.lead = lead;
                it.head = static_cast<int32_t>(head);
                it.q0 = q0;
                it.row0 = static_cast<int32_t>(tile * 2 * kRows);
                it.rows = static_cast<int32_t>(min(int64_t(2 * kRows), rows - tile * 2 * kRows));
                it.lo = lo;
                it.end = end;
                rest = static_cast<int32_t>(to - from);
                it.key0 = (lo & ~(kKeys - 1)) + static_cast<int32_t>(from - begin) * kKeys;
                it.cut = from == begin ? 0 : 1;
                it.first_cut = static_cast<int32_t>(blockIdx.x) + 1;
                it.cuts = static_cast<int32_t>((begin + steps - 1) / share - from / share);
                it.first = true;
                it.any = true;
                it.steps = min(rest, kSegment);
                it.key0 += (rest - it.steps) * kKeys;
            };
            for (int32_t k = 0;; ++k) {
                if (rest > 0) {
                    it.steps = min(rest, kSegment);
                    it.key0 -= it.steps * kKeys;
                    it.first = false;
                } else {
                    it.any = false;
                    if (k == 0 && x < x1) {
                        // the first one from the plan, in shared memory until its copies begin
                        g = s_first.group;
                        open(s_first.before, plan.lo[g], plan.prefix[g], plan.lead[g], plan.rows[plan.offsets[g]],
                             plan.rows[plan.offsets[g + 1]]);
                    }
                    while (!it.any && x < x1) {
                        // (of groups that begin at x the last is the one with units)
                        if (w.units[g + 1] <= x) g = last_at_most(w.units, w.groups.n_groups + 1, x);
                        open(w.units[g], w.lo[g], w.prefix[g], w.lead[g], a.q_offsets[w.groups.offsets[g]],
                             a.q_offsets[w.groups.offsets[g + 1]]);
                    }
                }
                rest -= it.any ? it.steps : 0;
                it.last = rest == 0;
                if (k >= 2 && !wait(&bar.item_empty[k & 1], ((k >> 1) - 1) & 1)) break;
                if (lane == 0) {
                    s_item[k & 1] = it;
                    tc::mbar_arrive(&bar.item_full[k & 1]);
                }
                __syncwarp();
                if (!it.any) break;
            }
        } else {
            // ---- the tokens whose rows are to be joined: the two warps left -------------------
            const int32_t n = w.groups.n_groups;
            for (int64_t t = blockIdx.x * 64 + (warp - 14) * 32 + lane; t < a.T; t += int64_t(blocks) * 64) {
                const int32_t i = last_at_most(a.q_offsets, a.n_seq, t);
                const RequestRows r = load_rows(a, i);
                const bool in = t >= r.q0 && t < r.q0 + r.n && i >= w.groups.offsets[0] && i < w.groups.offsets[n];
                w.live[1 + t] = in && w.prefix[last_at_most(w.groups.offsets, n, i)] > 0;
            }
        }
    } else {
        set_registers<C::kSoftmaxRegs, true>();
        // ---- softmax --------------------------------------------------------------------
        const int i = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + i * kKeys, o_at = tmem + lanes + 2 * kKeys + i * 128;
        const bool plain = a.softcap == 0.0f && a.slopes == nullptr && a.scale > 0.0f;
        int32_t round = 0, o_round = 0, half_round = 0;
        for (int32_t k = 0;; ++k) {
            follow(&bar.item_full[k & 1], (k >> 1) & 1);
            if (!go_on() || !s_item[k & 1].any) break;
            // the piece stays in shared memory: registers are scarce in the loop below
            const Item &it = s_item[k & 1];
            const int32_t steps = it.steps, key0 = it.key0, end = it.end;
            const bool split = it.template split<E4M3>();
            const int r = (split ? 0 : i * kRows) + (warp & 3) * 32 + lane;
            const bool live = r < it.rows;
            if (it.rows <= i * kRows && !split) {  // this tile has no rows
                release(k);
                continue;
            }
            const int32_t row = it.row0 + (live ? r : 0);
            int32_t pos = end;
            if (live && (a.window > 0 || a.slopes != nullptr)) {
                const int32_t t = it.q0 + row / a.group, seq = last_at_most(a.q_offsets, a.n_seq, t);
                const int64_t p = int64_t(a.kv_lens[seq]) - (int64_t(a.q_offsets[seq + 1]) - t);
                pos = static_cast<int32_t>(max(int64_t(end), min(p, int64_t(LORA_MAX_KV_LEN))));
            }
            const float slope = live && a.slopes != nullptr ? a.slopes[it.head * a.group + row % a.group] * kLog2e : 0.0f;
            float mult = a.scale * a.kv.k_scale;
            if constexpr (E4M3) {
                // (a piece's exponents stay until it is released)
                follow(&bar.exp_full[k & 1], (k >> 1) & 1);
                mult *= __uint_as_float(static_cast<uint32_t>(127 + s_qexp[k & 1][r]) << 23);
            }
            const float by0 = mult * kLog2e;
            float m = -INFINITY, l = 0.0f;  // the reference of the row's weights, and their sum
            const int32_t j0 = split ? i : 0, j_step = split ? 2 : 1;
            for (int32_t j = j0; j < steps; j += j_step, ++round) {
                if (!wait(&bar.s_full[i], round & 1)) break;
                tc::fence_after_sync();
                const int32_t key = key0 + (steps - 1 - j) * kKeys;
                const bool masked = key + kKeys > end ||
                                    __any_sync(0xffffffffu, a.window > 0 && pos - key >= a.window);
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
                    const int32_t first = a.window > 0 ? max(0, (pos - key) - (a.window - 1)) : 0;  // keys before it are not seen
#pragma unroll 1
                    for (int c = 0; c < 2; ++c) {
                        uint32_t y[64];
                        float s[64];
                        tmem_ld64(s_at + 64 * c, y);
                        tmem_wait64(y);
#pragma unroll
                        for (int e = 0; e < 64; ++e) s[e] = __uint_as_float(y[e]);
                        finish_scores<64, 2>(s, a, mult, slope, key + 64 * c - pos, false);
                        const int32_t from = first - 64 * c, to = end - key - 64 * c;
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            y[e] = __float_as_uint(masked && (e < from || e >= to) ? -INFINITY : s[e]);
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
                    if (j > j0) rescale_output<HD>(o_at, f);
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
            follow(&bar.o_full[i], o_round & 1);
            if (!go_on()) break;
            tc::fence_after_sync();
            if (split && i == 1) {
                // this half's references and sums; the first half goes on with both
                s_half[r] = make_float2(m, l);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar.half_full);
                ++o_round;
                release(k);
                continue;
            }
            if (split) {
                follow(&bar.half_full, half_round & 1);
                ++half_round;
                if (!go_on()) break;
                tc::fence_after_sync();
                const float2 other = s_half[r];
                const float top = fmaxf(m, other.x), ref = top == -INFINITY ? 0.0f : top;
                const float w0 = ex2(m - ref), w1 = ex2(other.x - ref);
                m = top;
                l = fmaf(w1, other.y, w0 * l);
#pragma unroll 1
                for (int c = 0; c < HD / 16; ++c) {
                    uint32_t x[16], y[16];
                    tc::tmem_ld16(o_at + 16 * c, x);
                    tc::tmem_ld16(o_at + 128 + 16 * c, y);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        x[e] = __float_as_uint(fmaf(w1, __uint_as_float(y[e]), w0 * __uint_as_float(x[e])));
                    tmem_st16(o_at + 16 * c, x);
                }
                tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar.o_empty[1]);
            }
            // the rows' own place, or the block's
            const int64_t at = it.cut ? int64_t(blockIdx.x) * 2 * kRows + r
                                      : (int64_t(it.head) * a.T + it.q0) * a.group + it.row0 + r;
            const int64_t stride = it.cut ? 8 * kRows : 4 * int64_t(a.T) * a.n_heads;
            float4 *head = (it.cut ? w.cut_heads : w.heads) + at;
            float *out = it.cut ? w.cut_outs + blockIdx.x * int64_t(2 * kRows * HD) + r * 4 : w.outs + at * 4;
            if (!it.first) add_row<HD>(head, out, stride, o_at, m, l, live, kShift);
            leave_row<HD>(head, out, stride, it, r, o_at, m, l, live, kShift);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar.o_empty[i]);
            ++o_round;
            release(k);
        }
    }
    // a wait that gave up stops the block's other roles; what is in flight lands before
    // the tensor memory goes
    if (!__all_sync(0xffffffffu, fine)) {
        s_abort = 1;
        *w.gave_up = 1;
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

// Joins the partial results of 32 neighbouring rows (of a key head: token, query head), a
// lane each; a warp takes every eighth group of 8 dims.
template <int HD>
__global__ void __launch_bounds__(256) attend_join_kernel(const AttendArgs a, const SharedWork w) {
    wait_for_previous();
    const int64_t rows = int64_t(a.T) * a.n_heads, row = min(int64_t(blockIdx.x) * 32 + (threadIdx.x & 31), rows - 1);
    const int64_t per = int64_t(a.T) * a.group, kv_head = row / per;
    const int32_t of_head = static_cast<int32_t>(row - kv_head * per), t = of_head / a.group;
    const int32_t h = static_cast<int32_t>(kv_head) * a.group + of_head % a.group;
    // (of a row that is not joined these are of another call)
    const float4 first = __ldcg(w.heads + row), own = __ldcg(w.own_sums + row);
    const bool live = w.live[1 + t] != 0 && int64_t(blockIdx.x) * 32 + (threadIdx.x & 31) < rows;
    const bool any = w.live[0] != 0, gave_up = *w.gave_up != 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        w.own_blocks[0] = 0;
        if (gave_up) report_error(a.err, LORA_ERR_TIMEOUT);  // (of an earlier call, the workspace not zeroed since)
    }
    if (!any || !live || gave_up) return;
    // The row's pieces, in the order of the keys: of the prefix the first and the others, by block;
    // its own first one and the others, by warp of the decode path.
    const int32_t tile = w.groups.tile_rows, own_size = tile * (HD + 2);
    const int32_t c0 = __float_as_int(first.z) >> 8, n0 = 1 + __float_as_int(first.w), r = __float_as_int(first.z) & 255;
    const int32_t w0 = __float_as_int(own.z) >> 5, n1 = 1 + __float_as_int(own.w), r1 = __float_as_int(own.z) & 31;
    const int32_t n = n0 + n1;
    // (what another call writes into this one's workspace at the same time sends no access out of it)
    const auto within = [](int32_t from, int32_t pieces, int32_t most) {
        return pieces >= 1 && pieces <= most && from >= 0 && from <= most - (pieces - 1);
    };
    if (!within(c0, n0, kMaxGrid) || !within(w0, n1, kOwnWarps)) {
        report_error(a.err, LORA_ERR_WORKSPACE);
        return;
    }
    constexpr int kBatch = 4;         // pieces whose loads are under way together
    constexpr int kGroups = HD / 64;  // of 8 dims, a warp
    const int warp = threadIdx.x >> 5;
    float o[kGroups][8], top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e) o[g][e] = 0.0f;
    for (int32_t p0 = 0; p0 < n; p0 += kBatch) {
        float2 head[kBatch];
        float4 x[kBatch][kGroups][2];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int32_t i = p0 + b;
            if (i >= n) {
                head[b] = make_float2(-INFINITY, 0.0f);
#pragma unroll
                for (int g = 0; g < kGroups; ++g) x[b][g][0] = x[b][g][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                continue;
            }
            const bool pre = i < n0;
            const int32_t c = pre ? c0 + i - 1 : w0 + i - n0 - 1;
            const float *from, *at;  // reference and sum; dims 4 i at from + i * stride
            int64_t stride = 4 * rows;
            if (i == 0) {
                at = reinterpret_cast<const float *>(w.heads + row);
                from = w.outs + row * 4;
            } else if (i == n0) {
                at = reinterpret_cast<const float *>(w.own_sums + row);
                from = w.own_outs + row * 4;
            } else if (pre) {
                at = reinterpret_cast<const float *>(w.cut_heads + int64_t(c) * 2 * kRows + r);
                from = w.cut_outs + int64_t(c) * 2 * kRows * HD + r * 4;
                stride = 8 * kRows;
            } else {
                at = w.own_cuts + int64_t(c) * own_size + 2 * r1;
                from = w.own_cuts + int64_t(c) * own_size + 2 * tile + r1 * 4;
                stride = 4 * tile;
            }
            head[b] = __ldcg(reinterpret_cast<const float2 *>(at));
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    x[b][g][e] = __ldcg(reinterpret_cast<const float4 *>(from + (2 * (g * 8 + warp) + e) * stride));
        }
        float now = top;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) now = fmaxf(now, head[b].x);
        const float ref = now == -INFINITY ? 0.0f : now, f = ex2(top - ref);
        top = now;
        sum *= f;
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
            for (int e = 0; e < 8; ++e) o[g][e] *= f;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const float v = ex2(head[b].x - ref);
            sum = fmaf(v, head[b].y, sum);
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    o[g][4 * e] = fmaf(v, x[b][g][e].x, o[g][4 * e]);
                    o[g][4 * e + 1] = fmaf(v, x[b][g][e].y, o[g][4 * e + 1]);
                    o[g][4 * e + 2] = fmaf(v, x[b][g][e].z, o[g][4 * e + 2]);
                    o[g][4 * e + 3] = fmaf(v, x[b][g][e].w, o[g][4 * e + 3]);
                }
        }
    }
    const float inv = sum > 0.0f ? a.kv.v_scale / sum : sum == 0.0f ? 0.0f : sum;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        uint32_t x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = pack_bf16x2(o[g][2 * e] * inv, o[g][2 * e + 1] * inv);
        stg_u4(a.out + t * a.ldo + h * HD + (g * 8 + warp) * 8, make_uint4(x[0], x[1], x[2], x[3]));
    }
    if (a.lse != nullptr && warp == 0)
        a.lse[int64_t(t) * a.n_heads + h] = sum == 0.0f ? -INFINITY : kLn2 * top + logf(sum);
}

constexpr int kSms = 152;  // a GB300's

size_t up128(size_t b) { return (b + 127) & ~size_t(127); }

// The word that has to be 0 when a call begins: behind the decode path's counters, at a place
// that does not depend on the call; and the one that says that a wait gave up.
constexpr size_t kOwnBlocks = 1020, kGaveUp = 1016;

// The parts of a call's workspace behind the decode path's.  Nothing in them outlives a call.
struct Layout {
    size_t units, prefix, lo, lead, live, own_sums, own_outs, heads, outs, cut_heads, cut_outs, end;
    Layout(int32_t head_dim, int32_t n_heads, int32_t T) {
        const size_t rows = size_t(T) * n_heads;
        size_t at = up128(decode_workspace_bytes(head_dim));
        const auto take = [&](size_t bytes) {
            const size_t here = at;
            at += up128(bytes);
            return here;
        };
        units = take((LORA_MAX_SEQS + 1) * 8);
        prefix = take(LORA_MAX_SEQS * 4);
        lo = take(LORA_MAX_SEQS * 4);
        lead = take(LORA_MAX_SEQS * 4);
        live = take((size_t(T) + 1) * 4);
        own_sums = take(rows * 16);
        own_outs = take(rows * head_dim * 4);
        heads = take(rows * 16);
        outs = take(rows * head_dim * 4);
        cut_heads = take(size_t(kMaxGrid) * 2 * kRows * 16);
        cut_outs = take(size_t(kMaxGrid) * 2 * kRows * head_dim * 4);
        end = at;
    }
};

template <int HD, bool E4M3>
cudaError_t launch(const AttendArgs &a, const SharedWork &w, void *ws, cudaStream_t stream) {
    static std::atomic<uint64_t> seen{0};
    int sms = 0;
    cudaError_t e = prepare_kernel(attend_prefix_kernel<HD, E4M3>, PrefixConfig<HD>::kSmem, seen, &sms);
    if (e != cudaSuccess) return e;
    e = launch_dependent(attend_prefix_kernel<HD, E4M3>, sms < kMaxGrid ? sms : kMaxGrid, kThreads,
                         PrefixConfig<HD>::kSmem, stream, a, w);
    if (e != cudaSuccess) return e;
    e = launch_attend_own(a, E4M3, w.groups, w.own_sums, w.own_outs, w.own_blocks, w.live, ws, stream);
    if (e != cudaSuccess) return e;
    return launch_dependent(attend_join_kernel<HD>, static_cast<unsigned>((int64_t(a.T) * a.n_heads + 31) / 32), 256, 0,
                            stream, a, w);
}

// Costs of the two ways, ns of one SM, from calls long enough to show them; a cap or a bias
// lengthens the softmax of both.  Shared always / never, us, 32/8 heads of 128 over bf16, one row a
// request: 4 requests behind 2,000 tokens 25 / 16, behind 30,000 49 / 74; 64 behind 500 27 / 35; 8
// groups of 4 behind 8,000 73 / 127; 64 of 2 behind 1,000 103 / 89, behind 4,000 210 / 324; over e4m3
// 32 of 4 behind 2,000 108 / 109, 8 of 16 63 / 98.
Groups costs(const lora_prefix_t &prefix, int32_t tile_rows, const AttendArgs &a, bool e4m3) {
    const bool wide = a.kv.head_dim == 128;
    const int32_t more = a.softcap == 0.0f && a.slopes == nullptr ? 0 : 800;
    const int32_t one = (e4m3 ? wide ? 2300 : 1650 : wide ? 1650 : 1400) + more;
    const int32_t two = one + (wide ? 550 : 400) + more;
    int32_t own = e4m3 ? wide ? 800 : 450 : wide ? 700 : 400;
    const int32_t first = e4m3 ? 0 : wide ? 750 : 350;
    if (tile_rows == 16) own = own * 5 / 4;
    if (tile_rows == 32) own = own * 5 / 2;
    return {prefix.group_offsets, prefix.prefix_lens, prefix.n_groups, tile_rows, prefix.mode == LORA_SHARE_ALWAYS,
            one, two, own + more / 4, first, e4m3 ? 128 : 64};
}

}  // namespace

size_t shared_workspace_bytes(int32_t head_dim, int32_t n_heads, int32_t T, int32_t) {
    return Layout(head_dim, n_heads, T).end;
}

cudaError_t launch_attend_shared(const AttendArgs &a, bool e4m3, int32_t max_q, const lora_prefix_t &prefix, void *ws,
                                 cudaStream_t stream) {
    const Layout at(a.kv.head_dim, a.n_heads, a.T);
    char *base = static_cast<char *>(ws);
    const auto ints = [&](size_t o) { return reinterpret_cast<int32_t *>(base + o); };
    const auto floats = [&](size_t o) { return reinterpret_cast<float *>(base + o); };
    const int64_t rows = int64_t(max_q) * a.group;
    const int32_t tile_rows = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
    const Groups groups = costs(prefix, tile_rows, a, e4m3);
    // Short tables cannot hold prefixes worth sharing, whatever the lengths: one group of all requests,
    // its prefix as long as a row of the table, would save most.  The own keys' kernel then does it all
    // (4 samples of 500 to 700 tokens 13.7 us, 21.6 with a prefix kernel that finds nothing to do).  It is
    // lora_attend's decode kernel with one more list in shared memory and some more registers (12.5 us there; of
    // the 12 instances five spill, 4 to 296 bytes, and one there), whatever the number of rows.
    const int64_t keys = int64_t(a.width) << a.kv.page_shift, tiles = int64_t(a.T) * a.group / tile_rows + a.n_seq;
    const int64_t most = (tiles * groups.own + groups.first - groups.step_one) * (keys / kKeys + 1) * a.kv.n_kv;
    if (prefix.n_groups == 0 || a.n_seq < 2 || (!groups.always && most < int64_t(kSharedFixedNs) * kSms))
        return launch_attend_own(a, e4m3, groups, nullptr, nullptr, nullptr, nullptr, ws, stream);
    const SharedWork w{groups, reinterpret_cast<int64_t *>(base + at.units), ints(at.prefix), ints(at.lo), ints(at.lead),
                       ints(kOwnBlocks), ints(kGaveUp), ints(at.live), reinterpret_cast<float4 *>(base + at.own_sums),
                       floats(at.own_outs), own_pieces(ws),
                       reinterpret_cast<float4 *>(base + at.heads), floats(at.outs),
                       reinterpret_cast<float4 *>(base + at.cut_heads), floats(at.cut_outs)};
    if (a.kv.head_dim == 64)
        return e4m3 ? launch<64, true>(a, w, ws, stream) : launch<64, false>(a, w, ws, stream);
    return e4m3 ? launch<128, true>(a, w, ws, stream) : launch<128, false>(a, w, ws, stream);
}

}  // namespace lora

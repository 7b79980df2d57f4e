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
//                    cores read (e4m3 codes are widened to bf16, exactly, on the way)
//   warps 12-15      one thread issues the products
// k and v tiles share one ring; every wait is bounded (2 s) and reports
// LORA_ERR_TIMEOUT.  Blocks take the (request, row tile, key head) items with the
// most keys of a request first, and an item's keys from the last tile down: with a
// bias that falls with distance the largest scores come first and O is not rescaled
// step after step.
//
// Weights are rounded to bf16 for the second product (the cache's type: the
// instruction takes one type for both operands); sums use them unrounded.
#include <cuda_fp16.h>

#include "attend.cuh"
#include "tc.cuh"

namespace lora {

namespace {

constexpr int kRows = 128, kKeys = 128;    // a tile
constexpr int kThreads = 16 * 32;
// Registers a thread: 128 at launch, then by role.  The four warpgroups' shares
// (two of softmax, copies, products) add up to the launch's 4 x 128.
constexpr int kSoftmaxRegs = 200, kCopyRegs = 56, kMmaRegs = 56;
static_assert(2 * kSoftmaxRegs + kCopyRegs + kMmaRegs == 4 * 128, "registers of the block");
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kGrow = 8.0f;              // log2 by which a row's maximum may grow before O is rescaled

template <int HD>
struct PromptConfig {
    static constexpr int kTileB = kRows * HD * 2;
    static constexpr int kSlots = HD == 128 ? 5 : 8;  // k and v tiles in the ring
    static constexpr int kSmem = (2 + kSlots) * kTileB + 1024;
    static constexpr uint32_t kHalfB = kRows * 128;   // 64 dims of all rows
};

struct Barriers {
    uint64_t q_full, full[8], empty[8], s_full[2], p_full[2][2], o_full[2], done;
};

// Shared-memory matrix descriptor, 128-byte swizzle: 64 elements of the
// contiguous dimension a row, 8 rows (1024 bytes) a group `sbo` apart, and for
// an operand whose contiguous dimension is not the summed one (v) blocks of 64
// of it `lbo` apart.
__device__ __forceinline__ uint64_t desc128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFF) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3FFF) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(tc::kLayoutSW128) << 61);
}

// Whole warpgroup: registers a thread from here on.
template <int N, bool MORE>
__device__ __forceinline__ void set_registers() {
    if constexpr (MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N));
}

// True in one thread of the (whole) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// D[tmem] (+)= A[tmem] * B[smem], issued by one thread.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        :: "r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u) : "memory");
}

#define LORA_R8(r, o) "+r"(r[o]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), "+r"(r[o + 4]), "+r"(r[o + 5]), \
                      "+r"(r[o + 6]), "+r"(r[o + 7])
#define LORA_W8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), \
                      "=r"(r[o + 6]), "=r"(r[o + 7])
#define LORA_I8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), \
                      "r"(r[o + 6]), "r"(r[o + 7])

// Whole warp: 32 columns of the warp's lanes, without waiting (tmem_wait).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : LORA_W8(r, 0), LORA_W8(r, 8), LORA_W8(r, 16), LORA_W8(r, 24) : "r"(taddr));
}

// Whole warp: 64 columns of the warp's lanes into r[0..63], without waiting.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
        : LORA_W8(r, 0), LORA_W8(r, 8), LORA_W8(r, 16), LORA_W8(r, 24), LORA_W8(r, 32), LORA_W8(r, 40), LORA_W8(r, 48),
          LORA_W8(r, 56)
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_wait64(uint32_t (&r)[64]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : LORA_R8(r, 0), LORA_R8(r, 8), LORA_R8(r, 16), LORA_R8(r, 24), LORA_R8(r, 32), LORA_R8(r, 40),
                   LORA_R8(r, 48), LORA_R8(r, 56)
                 : : "memory");
}

__device__ __forceinline__ void tmem_wait128(uint32_t (&r)[128]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : LORA_R8(r, 0), LORA_R8(r, 8), LORA_R8(r, 16), LORA_R8(r, 24), LORA_R8(r, 32), LORA_R8(r, 40),
                   LORA_R8(r, 48), LORA_R8(r, 56), LORA_R8(r, 64), LORA_R8(r, 72), LORA_R8(r, 80), LORA_R8(r, 88),
                   LORA_R8(r, 96), LORA_R8(r, 104), LORA_R8(r, 112), LORA_R8(r, 120)
                 : : "memory");
}

// Waits for this thread's loads; names the registers they fill.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : LORA_R8(r, 0), LORA_R8(r, 8), LORA_R8(r, 16), LORA_R8(r, 24) : : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
        :: LORA_I8(r, 0), LORA_I8(r, 8), LORA_I8(r, 16), LORA_I8(r, 24), "r"(taddr) : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
        :: LORA_I8(r, 0), LORA_I8(r, 8), "r"(taddr) : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int HD>
__device__ __forceinline__ void rescale_output(uint32_t o_at, float f) {
#pragma unroll 1
    for (int c = 0; c < HD / 16; ++c) {
        uint32_t o[16];
        tc::tmem_ld16(o_at + 16 * c, o);
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tmem_st16(o_at + 16 * c, o);
    }
}

// Sixteen e4m3 codes as bf16, exactly (through f16 and fp32).
__device__ __forceinline__ void widen16(uint4 w, uint4 &lo, uint4 &hi) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t pair = u[i >> 1] >> (16 * (i & 1));
        uint32_t h;
        asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(pair));
        const __half2 h2 = *reinterpret_cast<const __half2 *>(&h);
        o[i] = pack_bf16x2(__low2float(h2), __high2float(h2));
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

// Byte offset of the 8-element piece of a row in a tile: 64 dims a 128-byte row.
__device__ __forceinline__ uint32_t tile_at(int row, int piece) {
    return (piece >> 3) * (kRows * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
}

// A block's item: 256 rows (two tiles) of a request and key head, keys [key0, key1).
struct Item {
    int32_t seq, head, row0, rows;  // first row and rows (of the request's n * group)
    int32_t q0, n, len, lo, key0, key1;
    bool any;
};

template <int HD, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) attend_prompt_kernel(const AttendArgs a) {
    using C = PromptConfig<HD>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Barriers bar;
    __shared__ Item s_item;
    __shared__ int64_t s_warp[kThreads / 32];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int32_t s_abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = (tc::smem_u32(smem_raw) + 1023) & ~1023u;  // two q tiles, then the ring

    wait_for_previous();
    // ---- this block's item: the requests' row-tile pairs, last ones first --------------
    {
        const int32_t per = (a.n_seq + kThreads - 1) / kThreads, i0 = min(a.n_seq, tid * per),
                      i1 = min(a.n_seq, i0 + per);
        const auto pairs_of = [&](const RequestRows &r) {
            return (int64_t(r.n) * a.group + 2 * kRows - 1) / (2 * kRows);
        };
        int64_t mine = 0;
        for (int32_t i = i0; i < i1; ++i) {
            const RequestRows r = load_rows(a, i);
            if (!r.ok && blockIdx.x == 0) report_error(a.err, LORA_ERR_INVALID_ARG);
            mine += pairs_of(r);
        }
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) s_warp[warp] = incl;
        if (tid == 0) {
            s_item.any = false;
            s_abort = 0;
        }
        __syncthreads();
        int64_t run = incl - mine, total = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) run += s_warp[w];
            total += s_warp[w];
        }
        const int64_t want = total - 1 - blockIdx.x / a.kv.n_kv;
        for (int32_t i = i0; i < i1 && want >= run; ++i) {
            const RequestRows r = load_rows(a, i);
            const int64_t pairs = pairs_of(r);
            if (want < run + pairs) {
                Item it;
                it.seq = i;
                it.head = blockIdx.x % a.kv.n_kv;
                it.row0 = static_cast<int32_t>(want - run) * 2 * kRows;
                it.rows = min(2 * kRows, r.n * a.group - it.row0);
                it.q0 = r.q0;
                it.n = r.n;
                it.len = r.len;
                const int32_t first = r.len - r.n + it.row0 / a.group;
                const int32_t last = r.len - r.n + (it.row0 + it.rows - 1) / a.group;
                it.lo = a.window > 0 ? static_cast<int32_t>(max(int64_t(0), int64_t(first) - a.window + 1)) : 0;
                it.key0 = it.lo & ~(kKeys - 1);
                it.key1 = last + 1;
                it.any = true;
                s_item = it;
            }
            run += pairs;
        }
    }
    if (tid == 0) {
        tc::mbar_init(&bar.q_full, 4);
        for (int i = 0; i < C::kSlots; ++i) {
            tc::mbar_init(&bar.full[i], 4);
            tc::mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bar.s_full[i], 1);
            tc::mbar_init(&bar.p_full[i][0], 4);
            tc::mbar_init(&bar.p_full[i][1], 4);
            tc::mbar_init(&bar.o_full[i], 1);
        }
        tc::mbar_init(&bar.done, 1);
        tc::mbar_init_fence();
    }
    __syncthreads();
    const Item it = s_item;
    if (!it.any) return;
    if (it.key1 <= 0) {  // no row sees a key
        for (int32_t e = tid; e < it.rows * (HD / 8); e += kThreads) {
            const int32_t row = it.row0 + e / (HD / 8), t = it.q0 + row / a.group;
            const int32_t h = it.head * a.group + row % a.group;
            stg_u4(a.out + t * a.ldo + h * HD + e % (HD / 8) * 8, make_uint4(0, 0, 0, 0));
            if (a.lse != nullptr && e % (HD / 8) == 0) a.lse[int64_t(t) * a.n_heads + h] = -INFINITY;
        }
        return;
    }
    if (warp == 12) tc::tmem_alloc(&s_tmem, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;
    const int n_tiles = it.rows > kRows ? 2 : 1;
    const int32_t steps = (it.key1 - it.key0 + kKeys - 1) / kKeys;
    const uint32_t q_base = base, ring = base + 2 * C::kTileB;
    bool fine = true;
    const auto wait = [&](uint64_t *b, uint32_t parity) {
        fine = fine && tc::mbar_wait(b, parity, &s_abort, kWaitNs);
        return fine;
    };

    if (warp >= 8 && warp < 12) {
        set_registers<kCopyRegs, false>();
        // ---- copies ---------------------------------------------------------------------
        const int w = warp - 8;
        constexpr int kPieces = HD / 8;  // 16-byte pieces of a bf16 row
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            // 32 rows: a lane's row's offset, then a few rows a copy instruction
            constexpr int kStep = 32 / kPieces;
            const int piece = lane % kPieces, r0 = w * 64 + half * 32;
            const int32_t row = it.row0 + r0 + lane;
            int64_t at = -1;
            if (r0 + lane < it.rows)
                at = (it.q0 + row / a.group) * a.ldq + (it.head * a.group + row % a.group) * HD;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int r = r0 + i * kStep + lane / kPieces;
                const int64_t o = __shfl_sync(0xffffffffu, at, i * kStep + lane / kPieces);
                tc::cp16(q_base + (r / kRows) * C::kTileB + tile_at(r % kRows, piece),
                         a.q + (o >= 0 ? o : 0) + piece * 8, o >= 0);
            }
        }
        tc::cp_commit();
        const int32_t *table = a.table + it.seq * a.ld_table;
        const int32_t end = min(it.len, it.key1);
        // the byte offset of this lane's key of a step, -1: none
        const auto offset_of = [&](int32_t step) -> int64_t {
            const int32_t key = it.key0 + (steps - 1 - step) * kKeys + w * 32 + lane;  // last keys first
            if (key < it.lo || key >= end) return -1;
            const int32_t page = __ldg(table + (key >> a.kv.page_shift));
            if (page < 0 || page >= a.kv.n_pages) {
                report_error(a.err, LORA_ERR_SLOT_RANGE);
                return -1;
            }
            return page * a.kv.page_b + (key & a.kv.page_mask) * a.kv.token_b + it.head * a.kv.head_b;
        };
        const int32_t tiles = 2 * steps;
        const auto slot_free = [&](int32_t u) {
            return u < C::kSlots || wait(&bar.empty[u % C::kSlots], (u / C::kSlots - 1) & 1);
        };
        const auto publish = [&](uint64_t *b) {
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(b);
        };
        if constexpr (E4M3) {
            constexpr int kCodes = HD / 16;        // 16-byte pieces of a row of codes
            constexpr int kStep = 32 / kCodes;     // keys a load instruction
            const int piece = lane % kCodes;
            uint4 v[kCodes];
            int64_t at = offset_of(0), next_at = -1;
            const auto load = [&](int32_t u) {
                const unsigned char *from = (u & 1) ? a.kv.v : a.kv.k;
#pragma unroll
                for (int i = 0; i < kCodes; ++i) {
                    const int64_t o = __shfl_sync(0xffffffffu, at, i * kStep + lane / kCodes);
                    v[i] = o >= 0 ? ldg_stream(from + o + piece * 16) : make_uint4(0, 0, 0, 0);
                }
            };
            load(0);
            tc::cp_wait_all();
            publish(&bar.q_full);
            for (int32_t u = 0; u < tiles; ++u) {
                if ((u & 1) == 0 && u + 2 < tiles) next_at = offset_of(u / 2 + 1);
                if (!slot_free(u)) break;
                const uint32_t dst = ring + (u % C::kSlots) * C::kTileB;
#pragma unroll
                for (int i = 0; i < kCodes; ++i) {
                    const int row = w * 32 + i * kStep + lane / kCodes;
                    uint4 lo, hi;
                    widen16(v[i], lo, hi);
                    sts16(dst + tile_at(row, 2 * piece), lo);
                    sts16(dst + tile_at(row, 2 * piece + 1), hi);
                }
                if (u & 1) at = next_at;
                if (u + 1 < tiles) load(u + 1);
                publish(&bar.full[u % C::kSlots]);
            }
        } else {
            constexpr int kStep = 32 / kPieces;    // keys a copy instruction
            const int piece = lane % kPieces, row0 = lane / kPieces;
            int64_t at = offset_of(0), next_at = -1;
            int32_t u = 0;
            for (; u < tiles; ++u) {
                if ((u & 1) == 0 && u + 2 < tiles) next_at = offset_of(u / 2 + 1);
                if (!slot_free(u)) break;
                const unsigned char *from = (u & 1) ? a.kv.v : a.kv.k;
                const uint32_t dst = ring + (u % C::kSlots) * C::kTileB;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int row = i * kStep + row0;
                    const int64_t o = __shfl_sync(0xffffffffu, at, row);
                    tc::cp16(dst + tile_at(w * 32 + row, piece), from + (o >= 0 ? o : 0) + piece * 16, o >= 0);
                }
                tc::cp_commit();
                if (u & 1) at = next_at;
                // the tile two before this one (and q before all) has landed
                tc::cp_wait_group<2>();
                if (u == 1) publish(&bar.q_full);
                if (u >= 2) publish(&bar.full[(u - 2) % C::kSlots]);
            }
            if (fine) {
                tc::cp_wait_group<1>();
                publish(&bar.full[(tiles - 2) % C::kSlots]);
                tc::cp_wait_group<0>();
                publish(&bar.full[(tiles - 1) % C::kSlots]);
            }
            tc::cp_wait_all();
        }
    } else if (warp >= 12) {
        set_registers<kMmaRegs, false>();
        // ---- products -------------------------------------------------------------------
        if (warp == 12) {
            // The warp stays together and one elected thread issues: the products' operands
            // then stay in uniform registers.
            constexpr uint32_t kS = tc::idesc_bf16(kRows, kKeys);
            constexpr uint32_t kO = tc::idesc_bf16(kRows, HD) | (1u << 16);  // v: keys are the strided dimension
            // descriptors are a tile's plus a constant: addresses stay below 2^18, so nothing carries
            const uint64_t q_desc = desc128(q_base, 16, 1024), k_desc = desc128(ring, 16, 1024);
            const uint64_t v_desc = desc128(ring, C::kHalfB, 1024);
            const auto full = [&](int32_t u) { return wait(&bar.full[u % C::kSlots], (u / C::kSlots) & 1); };
            const auto scores = [&](int i, int32_t u, bool last) {
                const uint64_t q = q_desc + ((i * C::kTileB) >> 4), k = k_desc + (((u % C::kSlots) * C::kTileB) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk) {
                        const uint32_t off = ((kk / 4) * C::kHalfB + (kk % 4) * 32) >> 4;
                        tc::mma_bf16(tmem + i * kKeys, q + off, k + off, kS, kk > 0);
                    }
                    tc::mma_commit(&bar.s_full[i]);
                    if (last) tc::mma_commit(&bar.empty[u % C::kSlots]);
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
            const auto commit = [&](uint64_t *b) {
                if (elect_one()) tc::mma_commit(b);
                __syncwarp();
            };
            if (wait(&bar.q_full, 0) && full(0)) {
                tc::fence_after_sync();
                for (int i = 0; i < n_tiles; ++i) scores(i, 0, i == n_tiles - 1);
            }
            for (int32_t j = 0; j < steps && fine; ++j) {
                const bool more = j + 1 < steps;
                for (int i = 0; i < n_tiles && fine; ++i) {
                    const bool last = i == n_tiles - 1;
                    if (i == 0 && !full(2 * j + 1)) break;
                    if (!wait(&bar.p_full[i][0], j & 1)) break;
                    tc::fence_after_sync();
                    outputs(i, 2 * j + 1, 0, j == 0);
                    if (!wait(&bar.p_full[i][1], j & 1)) break;
                    tc::fence_after_sync();
                    outputs(i, 2 * j + 1, 1, j == 0);
                    if (!more) commit(&bar.o_full[i]);
                    if (last) commit(&bar.empty[(2 * j + 1) % C::kSlots]);
                    if (more) {
                        if (i == 0 && !full(2 * j + 2)) break;
                        tc::fence_after_sync();
                        scores(i, 2 * j + 2, last);
                    }
                }
            }
            // every product has finished, and every arrival landed, before the block ends
            commit(&bar.done);
            if (!tc::mbar_wait_timed(&bar.done, 0, kWaitNs)) fine = false;
        }
        fine = __all_sync(0xffffffffu, fine);
    } else {
        set_registers<kSoftmaxRegs, true>();
        // ---- softmax --------------------------------------------------------------------
        const int i = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + i * kKeys, o_at = tmem + lanes + 2 * kKeys + i * 128;
        if (i < n_tiles) {
            // the row's place is worked out again for the output: registers are scarce between
            const auto place = [&](bool &live, int32_t &token, int32_t &h) {
                const int32_t r = i * kRows + (warp & 3) * 32 + lane, row = s_item.row0 + r;
                live = r < s_item.rows;
                token = live ? row / a.group : 0;
                h = s_item.head * a.group + (live ? row % a.group : 0);
            };
            bool live;
            int32_t token, h;
            place(live, token, h);
            const int32_t first_pos = it.len - it.n, key0 = it.key0;
            const int32_t pos = live ? first_pos + token : -1;
            const int32_t pos_lo = first_pos + (it.row0 + i * kRows) / a.group;
            const int32_t pos_hi = first_pos + (it.row0 + min(it.rows, (i + 1) * kRows) - 1) / a.group;
            const float mult = a.scale * a.kv.k_scale, by0 = mult * kLog2e;
            const float slope = live && a.slopes != nullptr ? a.slopes[h] * kLog2e : 0.0f;
            const bool plain = a.softcap == 0.0f && a.slopes == nullptr && a.scale > 0.0f;
            float m = -INFINITY;  // the reference of the row's weights
            uint64_t sum[2] = {0, 0};  // pairs of fp32
            for (int32_t j = 0; j < steps; ++j) {
                if (!wait(&bar.s_full[i], j & 1)) break;
                tc::fence_after_sync();
                const int32_t key = key0 + (steps - 1 - j) * kKeys;
                const bool masked = key + kKeys - 1 > pos_lo || (a.window > 0 && pos_hi - key >= a.window);
                const bool direct = plain && !masked;
                const float by = direct ? by0 : 1.0f;
                if (!direct) {
                    // the final form of the scores, in place, 64 at a time (one copy of the code)
#pragma unroll 1
                    for (int c = 0; c < 2; ++c) {
                        uint32_t r[64];
                        float s[64];
                        tmem_ld64(s_at + 64 * c, r);
                        tmem_wait64(r);
#pragma unroll
                        for (int e = 0; e < 64; ++e) s[e] = __uint_as_float(r[e]);
                        finish_scores<64, 2>(s, a, mult, slope, key + 64 * c - pos, masked);
#pragma unroll
                        for (int e = 0; e < 64; ++e) r[e] = __float_as_uint(s[e]);
                        tmem_st32(s_at + 64 * c, r);
                        tmem_st32(s_at + 64 * c + 32, r + 32);
                    }
                    tmem_wait_st();
                }
                uint32_t x[128];
                tmem_ld64(s_at, x);
                tmem_ld64(s_at + 64, x + 64);
                tmem_wait128(x);
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
                    const uint64_t f2 = pack2(f, f);
#pragma unroll
                    for (int q = 0; q < 2; ++q) sum[q] = mul2(sum[q], f2);
                    if (j > 0) rescale_output<HD>(o_at, f);
                }
                const float ref = m == -INFINITY ? 0.0f : -m;
                const uint64_t by2 = pack2(by, by), ref2 = pack2(ref, ref);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float p0, p1;
                        const int k = 32 * c + 2 * e;
                        unpack2(fma2(pack2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), by2, ref2), p0, p1);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        sum[e & 1] = add2(sum[e & 1], pack2(p0, p1));
                        p[e] = pack_bf16x2(p0, p1);
                    }
                    tmem_st16(s_at + 16 * c, p);
                    if (c & 1) {  // half of the step's weights
                        tmem_wait_st();
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(&bar.p_full[i][c >> 1]);
                    }
                }
            }
            float l, l1;
            unpack2(add2(sum[0], sum[1]), l, l1);
            l += l1;
            if (fine && wait(&bar.o_full[i], 0)) {
                tc::fence_after_sync();
                const float inv = l > 0.0f ? a.kv.v_scale / l : l == 0.0f ? 0.0f : l;
                place(live, token, h);
                const int64_t t = s_item.q0 + token;
                uint16_t *dst = a.out + t * a.ldo + h * HD;
                uint32_t x[32];
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    tmem_ld32(o_at + 32 * c, x);
                    tmem_wait(x);
                    uint32_t o[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        o[e] = pack_bf16x2(__uint_as_float(x[2 * e]) * inv, __uint_as_float(x[2 * e + 1]) * inv);
                    if (live) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            stg_u4(dst + 32 * c + 8 * e, make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
                    }
                }
                if (live && a.lse != nullptr) a.lse[t * a.n_heads + h] = l == 0.0f ? -INFINITY : kLn2 * m + logf(l);
            }
        }
    }
    // a wait that gave up stops the block's other roles; what is in flight lands before
    // the tensor memory goes
    if (!fine) {
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

template <int HD, bool E4M3>
cudaError_t launch(const AttendArgs &a, cudaStream_t stream) {
    using C = PromptConfig<HD>;
    const auto kernel = attend_prompt_kernel<HD, E4M3>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    // every request's rows fill pairs of tiles but for one
    const int64_t pairs = int64_t(a.T) * a.group / (2 * kRows) + a.n_seq;
    if (pairs * a.kv.n_kv > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_dependent(kernel, static_cast<unsigned>(pairs * a.kv.n_kv), kThreads, C::kSmem, stream, a);
}

}  // namespace

cudaError_t launch_attend_prompt(const AttendArgs &a, bool e4m3, cudaStream_t stream) {
    if (a.kv.head_dim == 64) return e4m3 ? launch<64, true>(a, stream) : launch<64, false>(a, stream);
    return e4m3 ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
}

}  // namespace lora

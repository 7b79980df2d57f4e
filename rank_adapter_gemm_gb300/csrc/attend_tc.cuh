// Device helpers shared by the attention kernels on the 5th-generation tensor cores.
#pragma once

#include <cuda_fp16.h>

#include "attend.cuh"
#include "tc.cuh"

namespace lora {

constexpr int kRows = 128, kKeys = 128;    // a tile
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kGrow = 8.0f;              // log2 by which a row's maximum may grow before O is rescaled

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

// Sixteen e4m3 codes as f16, exactly.
__device__ __forceinline__ void widen16(uint4 w, uint4 &lo, uint4 &hi) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
            : "=r"(o[i]) : "r"(u[i >> 1] >> (16 * (i & 1))));
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr)
                 : "memory");
    return v;
}

// Byte offset of the 8-element piece of a row in a tile: 64 dims a 128-byte row.
__device__ __forceinline__ uint32_t tile_at(int row, int piece) {
    return (piece >> 3) * (kRows * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
}

}  // namespace lora

// Device arithmetic shared by the two attention kernels.
#pragma once

#include "attention.cuh"

namespace lora {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 in a 64-bit register, for the packed fp32 instructions.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}

// tanh of two numbers up to 1 in size, times `scale`: z (1 + z^2 (c1 + z^2 (c2 + ...))),
// the coefficients a minimax fit on [-1, 1]: within 2^-24 of tanh, and relatively so.
// Scores are seldom larger than the cap, and packed products cost a third of
// the exponential and the reciprocal that the general form needs.
__device__ __forceinline__ uint64_t tanh2_near(uint64_t z, uint64_t scale) {
    const uint64_t w = mul2(z, z);
    uint64_t r = pack2(0.0010059071f, 0.0010059071f);
    r = fma2(r, w, pack2(-0.0060955156f, -0.0060955156f));
    r = fma2(r, w, pack2(0.020165906f, 0.020165906f));
    r = fma2(r, w, pack2(-0.05339197f, -0.05339197f));
    r = fma2(r, w, pack2(0.13323739f, 0.13323739f));
    r = fma2(r, w, pack2(-0.33332753f, -0.33332753f));
    r = fma2(r, w, pack2(1.0f, 1.0f));
    return mul2(mul2(z, scale), r);
}

// tanh of any number to 2^-22: good relatively too for |z| >= 1/2.
__device__ __forceinline__ float tanh_far(float z) {
    return 1.0f - __fdividef(2.0f, ex2(z * (2.0f * kLog2e)) + 1.0f);
}

// N products s in their final form, times log2 e, in fp32: scaled, capped,
// biased by distance, masked.  back: first one's key minus the row's position;
// consecutive pairs lie STEP keys apart.  by = mult * log2 e, slope alike.
// Called by whole warps.
template <int N, int STEP>
__device__ __forceinline__ void finish_scores(float (&s)[N], const AttendArgs &a, float mult, float slope, int32_t back,
                                              bool masked) {
    if (a.softcap > 0.0f) {
        const float in = mult / a.softcap, cap = a.softcap * kLog2e;
        float top = 0.0f;
#pragma unroll
        for (int e = 0; e < N; ++e) top = fmaxf(top, fabsf(s[e]));
        if (__any_sync(0xffffffffu, !(top * fabsf(in) <= 1.0f))) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                float near, other;
                unpack2(tanh2_near(pack2(s[e] * in, 0.0f), pack2(cap, cap)), near, other);
                s[e] = fabsf(s[e] * in) < 0.75f ? near : cap * tanh_far(s[e] * in);
            }
        } else {
            const uint64_t in2 = pack2(in, in), cap2 = pack2(cap, cap);
#pragma unroll
            for (int e = 0; e < N; e += 2)
                unpack2(tanh2_near(mul2(pack2(s[e], s[e + 1]), in2), cap2), s[e], s[e + 1]);
        }
    } else {
        const uint64_t by2 = pack2(mult * kLog2e, mult * kLog2e);
#pragma unroll
        for (int e = 0; e < N; e += 2) unpack2(mul2(pack2(s[e], s[e + 1]), by2), s[e], s[e + 1]);
    }
    if (a.slopes != nullptr) {
        const float at = slope * static_cast<float>(back);
        const uint64_t at2 = pack2(at, at), slope2 = pack2(slope, slope);
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float d = static_cast<float>(e / 2 * STEP);
            unpack2(add2(pack2(s[e], s[e + 1]), fma2(slope2, pack2(d, d + 1.0f), at2)), s[e], s[e + 1]);
        }
    }
    if (masked) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int32_t b = back + e / 2 * STEP + (e & 1);
            if (b > 0 || (a.window > 0 && -b >= a.window)) s[e] = -INFINITY;
        }
    }
}

}  // namespace lora

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

// tanh z = z (1 + c1 z^2 + c2 z^4 + ...): minimax fits with the first coefficient
// held at 1 (so that small z keep their relative accuracy too), within 2^-22 for
// |z| <= 1/2 and 2^-21 for |z| <= 1.  Scores seldom reach half their cap, and the
// short polynomial costs a fifth of the exponential and the reciprocal that the
// general form needs.
#define LORA_TANH_HALF {1.0f, -0.33326461f, 0.13185862f, -0.04422929f}
#define LORA_TANH_ONE {1.0f, -0.3332867f, 0.13275616f, -0.05142535f, 0.016532812f, -0.002983080f}

// tanh of any number to 2^-22.
__device__ __forceinline__ float tanh_far(float z) {
    return 1.0f - __fdividef(2.0f, ex2(z * (2.0f * kLog2e)) + 1.0f);
}

// N products s in their final form, times log2 e, in fp32: scaled by mult, capped,
// biased by distance (slope: times log2 e), masked.  back: the first one's key minus
// the row's position; consecutive pairs lie STEP keys apart.  Called by whole warps.
template <int N, int STEP>
__device__ __forceinline__ void finish_scores(float (&s)[N], const AttendArgs &a, float mult, float slope, int32_t back,
                                              bool masked) {
    const uint64_t slope2 = pack2(slope, slope), at2 = pack2(slope * back, slope * back);
    const float by = mult * kLog2e;
    bool near = a.softcap > 0.0f;
    if (near) {
        float top = 0.0f;
#pragma unroll
        for (int e = 0; e < N; e += 2) top = fmaxf(fmaxf(top, fabsf(s[e])), fabsf(s[e + 1]));
        // (a cap below 1e-6 of mult would overflow the coefficients)
        near = __all_sync(0xffffffffu, top * fabsf(mult) <= 0.5f * a.softcap && fabsf(mult) <= 1e6f * a.softcap);
        if (!near) {
            constexpr float kTanh[6] = LORA_TANH_ONE;
            const float in = mult * a.inv_softcap, cap = a.softcap * kLog2e;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float z = s[e] * in, w = z * z;
                const float poly = z * (1.0f + w * (kTanh[1] + w * (kTanh[2] + w * (kTanh[3] + w * (kTanh[4] +
                                                                                                     w * kTanh[5])))));
                s[e] = cap * (fabsf(z) <= 1.0f ? poly : tanh_far(z));
            }
        }
    }
    if (near) {
        // by s + by c1 in^2 s^3 + ...: the scales are in the coefficients
        const float in = mult * a.inv_softcap, in2 = in * in;
        float c = by;
        constexpr float kTanh[4] = LORA_TANH_HALF;
        uint64_t k[4];
#pragma unroll
        for (int i = 0; i < 4; ++i, c *= in2) k[i] = pack2(c * kTanh[i], c * kTanh[i]);
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const uint64_t x = pack2(s[e], s[e + 1]), w = mul2(x, x);
            uint64_t r = fma2(k[3], w, k[2]);
#pragma unroll
            for (int i = 1; i >= 0; --i) r = fma2(r, w, k[i]);
            if (a.slopes != nullptr) {
                const float d = static_cast<float>(e / 2 * STEP);
                r = fma2(x, r, fma2(slope2, pack2(d, d + 1.0f), at2));
            } else {
                r = mul2(x, r);
            }
            unpack2(r, s[e], s[e + 1]);
        }
    } else {
        const float scale = a.softcap > 0.0f ? 1.0f : by;
        const uint64_t scale2 = pack2(scale, scale);
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float d = static_cast<float>(e / 2 * STEP);
            unpack2(fma2(pack2(s[e], s[e + 1]), scale2, fma2(slope2, pack2(d, d + 1.0f), at2)), s[e], s[e + 1]);
        }
    }
    if (masked) {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (back > -(e / 2 * STEP + (e & 1))) s[e] = -INFINITY;
        if (a.window > 0) {
            const int32_t first = -back - a.window;  // keys up to this one's index are out of the window
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (first >= e / 2 * STEP + (e & 1)) s[e] = -INFINITY;
        }
    }
}

}  // namespace lora

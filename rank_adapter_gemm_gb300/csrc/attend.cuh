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

// Whether products of size `top` lie within half the cap, and NearForm's coefficients in
// fp32's range: its last one is about |mult| (mult / cap)^6 and is wanted with all its
// bits.  (A product's square is finite then too.)  Other scales take the general form.
__device__ __forceinline__ bool near_cap(const AttendArgs &a, float mult, float top) {
    const float in = mult * a.inv_softcap, in2 = in * in, last = fabsf(mult) * in2 * in2 * in2;
    return top * fabsf(mult) <= 0.5f * a.softcap && last >= 0x1p-120f && last <= 0x1p120f;
}

// A pair of products in their final form (finish_scores), the scales in the coefficients:
// under a near cap, x (k0 + k1 x^2 + k2 x^4 + k3 x^6) + bias; without one x k0 + bias.
struct NearForm {
    uint64_t k[4], slope2, at2;

    __device__ __forceinline__ NearForm(const AttendArgs &a, float mult, float slope, int32_t back) {
        constexpr float kTanh[4] = LORA_TANH_HALF;
        const float in = mult * a.inv_softcap, in2 = in * in;  // 0 without a cap
        float c = mult * kLog2e;
#pragma unroll
        for (int i = 0; i < 4; ++i, c *= in2) k[i] = pack2(c * kTanh[i], c * kTanh[i]);
        slope2 = pack2(slope, slope);
        at2 = pack2(slope * back, slope * back);
    }

    __device__ __forceinline__ uint64_t bias(float d) const { return fma2(slope2, pack2(d, d + 1.0f), at2); }

    // keys d and d + 1 after the first
    __device__ __forceinline__ uint64_t capped(uint64_t x, float d) const {
        const uint64_t w = mul2(x, x);
        return fma2(x, fma2(fma2(fma2(k[3], w, k[2]), w, k[1]), w, k[0]), bias(d));
    }

    __device__ __forceinline__ uint64_t linear(uint64_t x, float d) const { return fma2(x, k[0], bias(d)); }
};

// N products s in their final form, times log2 e, in fp32: scaled by mult, capped,
// biased by distance (slope: times log2 e), masked.  back: the first one's key minus
// the row's position; consecutive pairs lie STEP keys apart.  Called by whole warps.
template <int N, int STEP>
__device__ __forceinline__ void finish_scores(float (&s)[N], const AttendArgs &a, float mult, float slope, int32_t back,
                                              bool masked) {
    bool capped = a.softcap > 0.0f;
    if (capped) {
        float top = 0.0f;
#pragma unroll
        for (int e = 0; e < N; e += 2) top = fmaxf(fmaxf(top, fabsf(s[e])), fabsf(s[e + 1]));
        if (!__all_sync(0xffffffffu, near_cap(a, mult, top))) {
            constexpr float kTanh[6] = LORA_TANH_ONE;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float z = s[e] * mult * a.inv_softcap, w = z * z;
                const float poly = z * (1.0f + w * (kTanh[1] + w * (kTanh[2] + w * (kTanh[3] + w * (kTanh[4] +
                                                                                                     w * kTanh[5])))));
                s[e] = fabsf(z) <= 1.0f ? poly : tanh_far(z);
            }
            capped = false;
            mult = a.softcap;
        }
    }
    const NearForm form(a, mult, slope, back);
    if (capped) {
#pragma unroll
        for (int e = 0; e < N; e += 2)
            unpack2(form.capped(pack2(s[e], s[e + 1]), static_cast<float>(e / 2 * STEP)), s[e], s[e + 1]);
    } else {
#pragma unroll
        for (int e = 0; e < N; e += 2)
            unpack2(form.linear(pack2(s[e], s[e + 1]), static_cast<float>(e / 2 * STEP)), s[e], s[e + 1]);
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

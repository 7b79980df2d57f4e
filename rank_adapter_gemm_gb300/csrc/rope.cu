// Rotary positions of q and k and the write of k and v into the paged cache
// (lora_rope_append).
//
// The angle of pair j at position p is p f_j.  As a fixed-point fraction of a
// turn, phase_j = f_j / (2 pi) in units of 2^-64, the product p * phase_j
// modulo 2^64 is the angle modulo one turn with no rounding at any position;
// its upper 32 bits, read as a signed number, are the angle in [-1/2, 1/2)
// turns to 2^-32.  On that interval the hardware sine and cosine are within
// 2^-20 of the true ones, far inside the 2^-9 of the bf16 result, and no table
// of cosines is read from memory.
//
// A unit is 16 elements of a head that are rotated among themselves: two
// 8-element (16-byte) pieces j and j + rot / 16 of the half layout, or two
// adjacent pieces (interleaved pairs, and the dims past rot).  A thread keeps one
// unit index for all its heads, so its eight sines and cosines are computed once
// a token: with many tokens a token gets only as many threads as leave each about
// six heads, so that the angles cost less than the bytes; with few tokens each gets
// a whole block, for latency.  Measured, graph replay, heads of 128 dims, 32 of q and 8
// of k and of v (in brackets the other choice): one token 2.2 us (2.7), 256 into e4m3
// 3.4 (4.2), 2,048 10.4 (10.4), 16,384 61.5 (64.3).
// Bound by HBM: 402.9 MB of q, k and v in and out at 16,384 tokens, 6.55 TB/s; into e4m3 (369.3 MB,
// and a rounded division an element) 61.6 us, 6.0.
#include <cuda_fp8.h>

#include "attention.cuh"

namespace lora {

namespace {

constexpr int kThreads = 128;
constexpr int kManyTokens = 2048;  // from here on blocks fill the GPU several times over

struct RopeArgs {
    const uint16_t *qkv;
    uint16_t *q_out;
    int64_t ldqkv, ldq;
    const uint64_t *phases;
    const int32_t *positions;
    const int64_t *slots;
    int32_t *err;
    KvView kv;
    int32_t T, n_heads, rot, interleaved;
    float mscale;
    int32_t per_pass, tokens;  // heads that a token's threads take at a time, tokens a block
};

__device__ __forceinline__ void unpack8(uint4 w, float *f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16lo_to_f32(u[i]);
        f[2 * i + 1] = bf16hi_to_f32(u[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float *f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// Eight e4m3 codes of f / scale, clamped to +-448 by the conversion.
__device__ __forceinline__ uint2 pack8_e4m3(const float *f, float scale) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f[4 * i], scale),
                                                                 __fdiv_rn(f[4 * i + 1], scale)),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f[4 * i + 2], scale),
                                                                 __fdiv_rn(f[4 * i + 3], scale)),
                                                     __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads, 8) rope_append_kernel(RopeArgs a) {
    wait_for_previous();
    const int32_t hd = a.kv.head_dim, units = hd / 16, per_pass = a.per_pass, group = units * per_pass;
    int32_t r = threadIdx.x;
    int64_t t = blockIdx.x;
    if (a.tokens > 1) {
        const int32_t i = r / group;
        r -= i * group;
        t = t * a.tokens + i;
        if (i >= a.tokens || t >= a.T) return;
    }
    if (r >= group) return;
    const int32_t h0 = r / units, u = r - h0 * units;
    const int32_t pos = a.positions[t];
    const int64_t slot = a.slots[t];
    const int32_t nk = a.kv.n_kv, H = a.n_heads, total = H + 2 * nk;
    // the unit's two pieces, in elements from the head's start
    const bool turned = 16 * u < a.rot;
    const bool half = turned && !a.interleaved;
    const int32_t c0 = half ? 8 * u : 16 * u, c1 = half ? 8 * u + a.rot / 2 : 16 * u + 8;
    const uint16_t *row = a.qkv + t * a.ldqkv;
    // a head's loads are issued one head ahead, the first before the angles are known
    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
    if (h0 < total) {
        w0 = ldg_cg(row + h0 * hd + c0);
        w1 = ldg_cg(row + h0 * hd + c1);
    }
    float cs[8], sn[8];
    if (turned) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t turns = static_cast<uint64_t>(static_cast<int64_t>(pos)) * a.phases[8 * u + i];
            const float angle = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
            cs[i] = __cosf(angle) * a.mscale;
            sn[i] = __sinf(angle) * a.mscale;
        }
    }
    const bool slot_ok = slot >= 0 && slot < (int64_t(a.kv.n_pages) << a.kv.page_shift);
    if (!slot_ok && slot != -1 && r == 0) report_error(a.err, LORA_ERR_SLOT_RANGE);
    const int64_t at = slot_ok ? (slot >> a.kv.page_shift) * a.kv.page_b + (slot & a.kv.page_mask) * a.kv.token_b : 0;
    for (int32_t h = h0; h < total; h += per_pass) {
        float x[8], y[8];
        unpack8(w0, x);
        unpack8(w1, y);
        if (h + per_pass < total) {
            w0 = ldg_cg(row + (h + per_pass) * hd + c0);
            w1 = ldg_cg(row + (h + per_pass) * hd + c1);
        }
        if (turned && h < H + nk) {
            if (a.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = x[2 * i], q = x[2 * i + 1], r = y[2 * i], s = y[2 * i + 1];
                    x[2 * i] = p * cs[i] - q * sn[i];
                    x[2 * i + 1] = q * cs[i] + p * sn[i];
                    y[2 * i] = r * cs[4 + i] - s * sn[4 + i];
                    y[2 * i + 1] = s * cs[4 + i] + r * sn[4 + i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = x[i], q = y[i];
                    x[i] = p * cs[i] - q * sn[i];
                    y[i] = q * cs[i] + p * sn[i];
                }
            }
        }
        if (h < H) {
            uint16_t *o = a.q_out + t * a.ldq + h * hd;
            stg_u4(o + c0, pack8(x));
            stg_u4(o + c1, pack8(y));
        } else if (slot_ok) {
            const bool is_k = h < H + nk;
            const int32_t kh = h - H - (is_k ? 0 : nk);
            unsigned char *o = (is_k ? a.kv.k : a.kv.v) + at + kh * a.kv.head_b;
            if constexpr (E4M3) {
                const float scale = is_k ? a.kv.k_scale : a.kv.v_scale;
                *reinterpret_cast<uint2 *>(o + c0) = pack8_e4m3(x, scale);
                *reinterpret_cast<uint2 *>(o + c1) = pack8_e4m3(y, scale);
            } else {
                stg_u4(o + 2 * c0, pack8(x));
                stg_u4(o + 2 * c1, pack8(y));
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope_append(const uint16_t *qkv, int64_t ldqkv, int32_t T, int32_t n_heads, const lora_rope_t &rope,
                               const int32_t *positions, const int64_t *slots, uint16_t *q_out, int64_t ldq,
                               const KvView &kv, bool e4m3, int32_t *err, cudaStream_t stream) {
    const int32_t units = kv.head_dim / 16, total = n_heads + 2 * kv.n_kv, most = kThreads / units;
    int32_t per_pass = total < most ? total : most;
    if (T >= kManyTokens && per_pass > total / 6) per_pass = total / 6 > 1 ? total / 6 : 1;
    // a token of 64 threads or more has its own block: half a wide block would wait for the other half
    const int32_t group = units * per_pass, threads = group >= 64 ? (group + 31) & ~31 : kThreads;
    const int32_t tokens = threads < 2 * group ? 1 : threads / group;
    const RopeArgs a{qkv, q_out, ldqkv, ldq, rope.phases, positions, slots, err, kv, T, n_heads, rope.rot_dim,
                     rope.interleaved, rope.mscale, per_pass, tokens};
    return launch_dependent(e4m3 ? rope_append_kernel<true> : rope_append_kernel<false>, (T - 1) / tokens + 1, threads,
                            0, stream, a);
}

}  // namespace lora

// Attention of a step's tokens over the paged cache (lora_attend): one warp a
// (row, query head), each lane holding head_dim / 32 dims, one key at a time
// with the running maximum and sum of the softmax.
#include <cuda_fp8.h>

#include "attention.cuh"

namespace lora {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float kv_value(const unsigned char *p, int32_t d, bool e4m3) {
    if (e4m3) return __half2float(__half(__nv_cvt_fp8_to_halfraw(p[d], __NV_E4M3)));
    return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[d]) << 16);
}

__global__ void __launch_bounds__(kWarps * 32) attend_rows_kernel(AttendArgs a, bool e4m3) {
    const int lane = threadIdx.x & 31;
    const int32_t h = blockIdx.y * kWarps + (threadIdx.x >> 5), t = blockIdx.x;
    if (h >= a.n_heads) return;
    if (h == 0 && t == 0 && lane == 0)
        for (int32_t i = 0; i < a.n_seq; ++i)
            if (!load_rows(a, i).ok) report_error(a.err, LORA_ERR_INVALID_ARG);
    // the request that owns row t
    int32_t lo = 0, hi = a.n_seq;
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (a.q_offsets[mid] <= t) lo = mid;
        else hi = mid;
    }
    const RequestRows r = load_rows(a, lo);
    if (t < r.q0 || t >= r.q0 + r.n) return;
    const int32_t p = r.len - (r.q0 + r.n - t);
    const int32_t hd = a.kv.head_dim, per = hd / 32, kh = h / a.group;
    float q[4], acc[4];
    for (int e = 0; e < per; ++e) {
        q[e] = __uint_as_float(static_cast<uint32_t>(a.q[t * a.ldq + h * hd + lane * per + e]) << 16);
        acc[e] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    for (int32_t j = a.window > 0 ? max(0, p - a.window + 1) : 0; j <= p; ++j) {
        const int32_t page = a.table[lo * a.ld_table + (j >> a.kv.page_shift)];
        const bool ok = page >= 0 && page < a.kv.n_pages;
        if (!ok) report_error(a.err, LORA_ERR_SLOT_RANGE);
        const int64_t at = page * a.kv.page_b + (j & a.kv.page_mask) * a.kv.token_b + kh * a.kv.head_b;
        float s = 0.0f;
        for (int e = 0; e < per; ++e) s += ok ? q[e] * kv_value(a.kv.k + at, lane * per + e, e4m3) : 0.0f;
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= a.scale * a.kv.k_scale;
        if (a.softcap > 0.0f) s = a.softcap * tanhf(s / a.softcap);
        if (a.slopes != nullptr) s += a.slopes[h] * static_cast<float>(j - p);
        const float m2 = fmaxf(m, s), w = expf(s - m2), f = expf(m - m2);
        l = l * f + w;
        for (int e = 0; e < per; ++e)
            acc[e] = acc[e] * f + (ok ? w * kv_value(a.kv.v + at, lane * per + e, e4m3) : 0.0f);
        m = m2;
    }
    for (int e = 0; e < per; ++e) {
        const float o = l > 0.0f ? acc[e] / l * a.kv.v_scale : 0.0f;
        a.out[t * a.ldo + h * hd + lane * per + e] = static_cast<uint16_t>(pack_bf16x2(o, 0.0f) & 0xffffu);
    }
    if (a.lse != nullptr && lane == 0) a.lse[int64_t(t) * a.n_heads + h] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_attend_rows(const AttendArgs &a, bool e4m3, cudaStream_t stream) {
    attend_rows_kernel<<<dim3(a.T, (a.n_heads + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(a, e4m3);
    return cudaGetLastError();
}

}  // namespace lora

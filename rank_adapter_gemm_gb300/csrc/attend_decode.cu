// The decode path of lora_attend: instances of the kernel in attend_decode.cuh.
#include "attend_decode.cuh"

namespace lora {

// Counters (one a block), then a partial a warp and two a block, of up to 32 rows: 320
// rows a block, of which the prompt path takes 256.
size_t decode_workspace_bytes(int32_t head_dim) {
    return 1024 + size_t(kMaxGrid) * (kWarps + 2) * 32 * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_attend_decode(const AttendArgs &a, bool e4m3, int32_t max_q, void *ws, cudaStream_t stream) {
    return pick_decode<false>(a, e4m3, int64_t(max_q) * a.group, OwnRows{}, ws, stream);
}

}  // namespace lora

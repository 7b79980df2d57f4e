// The requests' own keys of lora_attend_shared: instances of the kernel in attend_decode.cuh.
#include "attend_decode.cuh"

namespace lora {

cudaError_t launch_attend_own(const AttendArgs &a, bool e4m3, int32_t max_q, const int32_t *shared, float2 *sums,
                              float *outs, int32_t *started, void *ws, cudaStream_t stream) {
    return pick_decode<true>(a, e4m3, max_q, OwnRows{shared, sums, outs, started}, ws, stream);
}

}  // namespace lora

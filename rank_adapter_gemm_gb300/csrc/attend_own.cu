// The requests' own keys of lora_attend_shared: instances of the kernel in attend_decode.cuh.
#include "attend_decode.cuh"

namespace lora {

// The other pieces of rows are left in ws, behind the counters: see OwnRows.
cudaError_t launch_attend_own(const AttendArgs &a, bool e4m3, const Groups &groups, float4 *sums, float *outs,
                              const int32_t *blocks, int32_t *live, void *ws, cudaStream_t stream) {
    return pick_decode<true>(a, e4m3, groups.tile_rows, OwnRows{groups, sums, outs, blocks, live}, ws, stream);
}

const float *own_pieces(const void *ws) { return reinterpret_cast<const float *>(static_cast<const char *>(ws) + 1024); }

}  // namespace lora

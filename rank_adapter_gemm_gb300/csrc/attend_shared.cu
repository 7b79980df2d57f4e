// Attention of requests that share a prefix (lora_attend_shared).
#include "attend.cuh"

namespace lora {

size_t decode_workspace_bytes(int32_t head_dim);
cudaError_t launch_attend_decode(const AttendArgs &a, bool e4m3, int32_t max_q, void *ws, cudaStream_t stream);

namespace {

__global__ void __launch_bounds__(1024) check_groups_kernel(const int32_t *offsets, const int32_t *lens, int32_t n,
                                                            int32_t n_seq, int32_t *err) {
    wait_for_previous();
    for (int32_t g = threadIdx.x; g < n; g += blockDim.x)
        if (offsets[g] < 0 || offsets[g + 1] < offsets[g] || offsets[g + 1] > n_seq || lens[g] < 0)
            report_error(err, LORA_ERR_INVALID_ARG);
}

}  // namespace

size_t shared_workspace_bytes(int32_t head_dim, int32_t, int32_t, int32_t) { return decode_workspace_bytes(head_dim); }

// Every request's keys through its own row, on the decode path.
cudaError_t launch_attend_shared(const AttendArgs &a, bool e4m3, int32_t max_q, const lora_prefix_t &prefix, void *ws,
                                 cudaStream_t stream) {
    const cudaError_t e = launch_dependent(check_groups_kernel, 1, 1024, 0, stream, prefix.group_offsets,
                                           prefix.prefix_lens, prefix.n_groups, a.n_seq, a.err);
    return e != cudaSuccess ? e : launch_attend_decode(a, e4m3, max_q, ws, stream);
}

}  // namespace lora

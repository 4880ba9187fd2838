// decode_state_e4m3.cu -- split-KV decode kernels for e4m3 K/V pools whose
// results another pass joins.
#include "decode_dispatch.cuh"

namespace fd {

cudaError_t launch_decode_state_e4m3(const fd_problem &p, const KernelShape &ks, const DecodeParams &dp,
                                    const CUtensorMap &tmk, const CUtensorMap &tmv, int grid, size_t smem,
                                    cudaStream_t stream) {
    if (p.q_dtype == FD_BF16)
        return launch_decode_kind<KV_E4M3, true, kState>(p, ks, dp, tmk, tmv, grid, smem, stream);
    return launch_decode_kind<KV_E4M3, false, kState>(p, ks, dp, tmk, tmv, grid, smem, stream);
}

cudaError_t decode_occupancy_state_e4m3(const fd_problem &p, const KernelShape &ks, size_t smem, bool scr, int *blocks) {
    if (p.q_dtype == FD_BF16) return occupancy_kind<KV_E4M3, true, kState>(p, ks, smem, scr, blocks);
    return occupancy_kind<KV_E4M3, false, kState>(p, ks, smem, scr, blocks);
}

}  // namespace fd

// decode_scores_bf16.cu -- split-KV decode kernels for bf16 K/V pools that also
// write every score for the attention-weight totals.
#include "decode_dispatch.cuh"

namespace fd {

cudaError_t launch_decode_scores_bf16(const fd_problem &p, const KernelShape &ks, const DecodeParams &dp,
                                      const CUtensorMap &tmk, const CUtensorMap &tmv, int grid, size_t smem,
                                      cudaStream_t stream) {
    return launch_decode_kind<KV_BF16, true, kScores>(p, ks, dp, tmk, tmv, grid, smem, stream);
}

cudaError_t decode_occupancy_scores_bf16(const fd_problem &p, const KernelShape &ks, size_t smem, bool scr, int *blocks) {
    return occupancy_kind<KV_BF16, true, kScores>(p, ks, smem, scr, blocks);
}

}  // namespace fd

// decode_diff_bf16.cu -- split-KV decode kernels for bf16 K/V pools of
// differential attention.
#include "decode_dispatch.cuh"

namespace fd {

cudaError_t launch_decode_diff_bf16(const fd_problem &p, const KernelShape &ks, const DecodeParams &dp,
                                    const CUtensorMap &tmk, const CUtensorMap &tmv, int grid, size_t smem,
                                    cudaStream_t stream) {
    return launch_decode_kind<KV_BF16, true, kDiff>(p, ks, dp, tmk, tmv, grid, smem, stream);
}

}  // namespace fd

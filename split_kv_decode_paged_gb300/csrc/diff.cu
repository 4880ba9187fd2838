// diff.cu -- differential attention around the decode kernel.  Head h has two
// queries q1, q2 of width d = D / 2 and the cache holds K = [k1 | k2]: both
// score maps are products of full K rows with a query padded by zeros,
// q1 k1^T = [q1 | 0] K^T and q2 k2^T = [0 | q2] K^T, so one pass over K and V
// serves both maps (2 G query rows per KV head instead of G).
//   out_h = o1 - lambda_h o2, then out * rsqrt(mean(out^2) + eps) * w * scale.
#include "fd_internal.h"
#include "ptx.cuh"

namespace fd {

constexpr int kDiffWarps = 4;

// [rows, D] 16-bit -> [2 rows, D]: row 2r = [q1 | 0], row 2r + 1 = [0 | q2].
__global__ void fd_diff_expand_kernel(const uint4 *q, uint4 *out, long long rows, int upr) {
    const long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x;  // 16-byte unit of q
    if (u >= rows * upr) return;
    const long long r = u / upr;
    const int x = (int)(u - r * upr);
    const uint4 v = q[u], z = make_uint4(0u, 0u, 0u, 0u);
    const bool first = x < upr / 2;
    out[2 * r * upr + x] = first ? v : z;
    out[(2 * r + 1) * upr + x] = first ? z : v;
}

// One warp per output row: o [2 rows, D] fp32 -> out [rows, D].
template <int D>
__global__ void __launch_bounds__(kDiffWarps * 32) fd_diff_combine_kernel(const __grid_constant__ DiffCombineParams p) {
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * kDiffWarps + (threadIdx.x >> 5);
    if (row >= p.rows) return;
    const float lam = __ldg(p.lambda + row % p.Hq);
    const float *o1 = p.o + 2 * row * D + lane * PER, *o2 = o1 + D;
    float v[PER], ss = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        v[e] = fmaf(-lam, o2[e], o1[e]);
        ss = fmaf(v[e], v[e], ss);
    }
    float mul = p.out_scale;
    if (p.w) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += shfl_xor(ss, o);
        mul *= rsqrtf(ss * (1.f / D) + p.eps);
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const int d = lane * PER + e;
        float x = v[e] * mul;
        if (p.w) {
            float w;
            if (p.w_dtype == FD_F32) w = __ldg(reinterpret_cast<const float *>(p.w) + d);
            else if (p.w_dtype == FD_BF16) w = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p.w)[d]);
            else w = __half2float(reinterpret_cast<const __half *>(p.w)[d]);
            x *= w;
        }
        if (p.out_dtype == FD_F32) reinterpret_cast<float *>(p.out)[row * D + d] = x;
        else if (p.out_dtype == FD_BF16) reinterpret_cast<__nv_bfloat16 *>(p.out)[row * D + d] = __float2bfloat16_rn(x);
        else reinterpret_cast<__half *>(p.out)[row * D + d] = __float2half_rn(x);
    }
}

cudaError_t launch_diff_expand(const void *q, void *out, long long rows, int D, cudaStream_t stream) {
    const int upr = D * 2 / 16;
    const long long blocks = (rows * upr + 255) / 256;
    fd_diff_expand_kernel<<<(unsigned)blocks, 256, 0, stream>>>(reinterpret_cast<const uint4 *>(q),
                                                               reinterpret_cast<uint4 *>(out), rows, upr);
    return cudaGetLastError();
}

cudaError_t launch_diff_combine(const DiffCombineParams &p, int D, cudaStream_t stream) {
    const unsigned blocks = (unsigned)((p.rows + kDiffWarps - 1) / kDiffWarps);
    if (D == 128)
        fd_diff_combine_kernel<128><<<blocks, kDiffWarps * 32, 0, stream>>>(p);
    else
        fd_diff_combine_kernel<64><<<blocks, kDiffWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace fd

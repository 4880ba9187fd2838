// rows.cu -- launches of the rows kernel (rows_kernel.cuh) and the merge of the
// partial states of KV rows that it took in several chunks.
#include <math.h>

#include "fd_internal.h"
#include "ptx.cuh"
#include "rows_kernel.cuh"

namespace fd {

namespace {

// One warp a query row (sequence, token, head): the partial states of its chunks
// and, where there is one, the state over its own tokens.  Rows that the main
// kernel finished itself, or never had, have row_splits = 0.
//     out = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) d_s,  m = max_s m_s
// with o_s and d_s relative to their own reference m_s.  Bound by the latency of a
// row's loads (a warp has its counts, then its weights, then eight chunks at once):
// 16384 rows of 7 chunks 20.6 us, 3.3 TB/s; 12288 of 2 chunks 9.3 us.
template <int D>
__global__ void __launch_bounds__(128) fd_rows_merge_kernel(const RowsParams p) {
    constexpr int E = D / 32;
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + warp;
    if (row >= (long long)p.seqs * p.T * p.Hq) return;
    const int n = __ldcg(p.row_splits + row);
    if (n == 0) return;
    __syncwarp();
    if (lane == 0) p.row_splits[row] = 0;
    const float *pm = p.part_m + row * p.S, *pd = p.part_d + row * p.S;
    // Lane s has chunk s's weight (and s + 32's); then the outputs with eight
    // chunks' loads under way.
    float m0 = lane < n ? __ldcg(pm + lane) : -INFINITY, m1 = lane + 32 < n ? __ldcg(pm + lane + 32) : -INFINITY;
    const float d0 = lane < n ? __ldcg(pd + lane) : 0.f, d1 = lane + 32 < n ? __ldcg(pd + lane + 32) : 0.f;
    float mx = fmaxf(m0, m1);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, shfl_xor(mx, o));
    const float base = mx == -INFINITY ? 0.f : mx;
    const float a0 = d0 == 0.f ? 0.f : ex2(m0 - base), a1 = d1 == 0.f ? 0.f : ex2(m1 - base);  // 0: an empty state
    float sum = a0 * d0 + a1 * d1, y[E];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += shfl_xor(sum, o);
#pragma unroll
    for (int x = 0; x < E; ++x) y[x] = 0.f;
    const float *po = p.part_o + (size_t)row * p.S * D + lane * E;
    for (int s0 = 0; s0 < n; s0 += 8) {
        float v[8][E];
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int x = 0; x < E; x += 2) {
                const float2 f = s0 + k < n ? __ldcg(reinterpret_cast<const float2 *>(po + (size_t)(s0 + k) * D + x))
                                            : make_float2(0.f, 0.f);
                v[k][x] = f.x;
                v[k][x + 1] = f.y;
            }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int s = s0 + k;
            const float a = __shfl_sync(0xffffffffu, s < 32 ? a0 : a1, s & 31);
            const float d = __shfl_sync(0xffffffffu, s < 32 ? d0 : d1, s & 31);
#pragma unroll
            for (int x = 0; x < E; ++x)
                if (s < n && d != 0.f) y[x] = fmaf(a, v[k][x], y[x]);
        }
    }
    const bool empty = sum == 0.f;
    float lse = empty ? -INFINITY : (mx + __log2f(sum)) * kRowsLn2;
    float mul = empty ? 0.f : 1.f / sum, own = 0.f;
    if (p.own_out) {
        const float lo = __ldcg(p.own_lse + row), m = fmaxf(lse, lo);
        const float wa = lse == -INFINITY ? 0.f : __expf(lse - m), wb = lo == -INFINITY ? 0.f : __expf(lo - m);
        const float inv = wa + wb > 0.f ? 1.f / (wa + wb) : 0.f;
        mul *= wa * inv;
        own = wb * inv;
        lse = m == -INFINITY ? -INFINITY : m + logf(wa + wb);
    }
    if (lane == 0 && p.lse) p.lse[row] = lse;
#pragma unroll
    for (int x = 0; x < E; ++x) {
        y[x] *= mul;
        if (p.own_out) y[x] = fmaf(own, __ldcg(p.own_out + row * D + lane * E + x), y[x]);
    }
    uint32_t *dst = reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(p.out) + row * D + lane * E);
#pragma unroll
    for (int x = 0; x < E; x += 2) dst[x / 2] = p.q_bf16 ? pack_bf16x2(y[x], y[x + 1]) : pack_f16x2(y[x], y[x + 1]);
}

template <typename Kernel, typename... Args>
cudaError_t launch_after(Kernel kern, unsigned grid, unsigned threads, size_t smem, cudaStream_t stream, Args... args) {
    // Programmatic dependent launch: the prologue may run while the previous
    // grid of the stream drains; the kernel waits before it reads anything.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int KV, int D, bool QBF16, int PARTS>
cudaError_t launch_rows_t(const RowsParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid, cudaStream_t stream) {
    using Sh = RowsShape<KV, D>;
    auto kern = fd_rows_kernel<KV, D, QBF16, PARTS>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
    if (e != cudaSuccess) return e;
    return launch_after(kern, (unsigned)grid, Sh::THREADS, Sh::SMEM, stream, p, tmk, tmv);
}

template <int KV, bool QBF16, int PARTS = 1>
cudaError_t launch_rows_d(const RowsParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid, cudaStream_t stream) {
    return p.D == 128 ? launch_rows_t<KV, 128, QBF16, PARTS>(p, tmk, tmv, grid, stream)
                      : launch_rows_t<KV, 64, QBF16, PARTS>(p, tmk, tmv, grid, stream);
}

}  // namespace

cudaError_t launch_rows(const RowsParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid, cudaStream_t stream) {
    if (p.kv_kind == KV_BF16)
        return p.weight_parts == 2 ? launch_rows_d<KV_BF16, true, 2>(p, tmk, tmv, grid, stream)
                                   : launch_rows_d<KV_BF16, true, 1>(p, tmk, tmv, grid, stream);
    if (p.kv_kind == KV_F16) return launch_rows_d<KV_F16, false>(p, tmk, tmv, grid, stream);
    return p.q_bf16 ? launch_rows_d<KV_E4M3, true>(p, tmk, tmv, grid, stream)
                    : launch_rows_d<KV_E4M3, false>(p, tmk, tmv, grid, stream);
}

cudaError_t launch_rows_merge(const RowsParams &p, cudaStream_t stream) {
    const long long rows = (long long)p.seqs * p.T * p.Hq;
    const unsigned blocks = (unsigned)((rows + 3) / 4);
    return p.D == 128 ? launch_after(fd_rows_merge_kernel<128>, blocks, 128, 0, stream, p)
                      : launch_after(fd_rows_merge_kernel<64>, blocks, 128, 0, stream, p);
}

}  // namespace fd

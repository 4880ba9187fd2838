// rows.cu -- attention of many query rows over KV rows that all of them see:
// cross attention and the pass over shared prefixes (fd_cross_paged,
// fd_decode_paged_prefix).
//
// A warp takes one query row (sequence, token, head).  A lane scores every
// 32nd token, the warp takes one online-softmax step over 32 tokens, and each
// lane adds up its D / 32 outputs.
#include <math.h>

#include "fd_internal.h"
#include "ptx.cuh"
#include "rows_kernel.cuh"

namespace fd {

namespace {

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void flag(int *status, int bit) {
    if (status) atomicOr(status, bit);
}

__device__ __forceinline__ float as_float(const void *p, size_t i, int kind) {
    if (kind == KV_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
    if (kind == KV_F16) return __half2float(reinterpret_cast<const __half *>(p)[i]);
    const uint32_t h = e4m3x2_to_f16x2(reinterpret_cast<const uint8_t *>(p)[i]);
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffff)));
}

// offsets[s], made to rise within [0, seqs].
__device__ int group_end(const RowsParams &p, int s) {
    int at = 0;
    for (int i = 0; i <= s && i <= p.kv_rows; ++i) {
        const int o = p.offsets[i];
        const int cut = min(max(o, at), p.seqs);
        if (o != cut || (i == 0 && o != 0)) flag(p.status, FD_DEV_BAD_PAGE);
        at = i == 0 ? 0 : cut;
    }
    return at;
}

template <int D>
__global__ void __launch_bounds__(128) fd_rows_plain_kernel(const RowsParams p) {
    constexpr int E = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 4 + warp;
    if (w >= (long long)p.seqs * p.T * p.Hq) return;
    const int h = (int)(w % p.Hq);
    const int t = (int)(w / p.Hq % p.T);
    const int i = (int)(w / ((long long)p.Hq * p.T));
    const int b = p.members ? p.members[i] : i;
    if (b < 0 || b >= p.seqs) {
        flag(p.status, FD_DEV_BAD_PAGE);
        return;
    }
    if (p.q_lens) {
        const int n = p.q_lens[b];
        if (n < 0 || n > p.T) flag(p.status, FD_DEV_CAPACITY);
        if (n > p.T || t >= n) return;
    }
    int s = p.kv_rows;
    if (p.offsets) {
        for (int k = 0; k < p.kv_rows && s == p.kv_rows; ++k)
            if (i < group_end(p, k + 1)) s = k;
    } else {
        s = i / p.beams;
    }
    int L = s < p.kv_rows ? p.kv_lens[s] : 0;
    if (L < 0 || L > p.cap) {
        flag(p.status, FD_DEV_CAPACITY);
        L = L < 0 ? 0 : p.cap;
    }
    const int kvh = h / p.G;
    const size_t tok = (size_t)b * p.T + t;
    float q[D];
#pragma unroll
    for (int d = 0; d < D; ++d)
        q[d] = as_float(p.q, tok * p.q_stride + (size_t)h * D + d, p.q_bf16 ? KV_BF16 : KV_F16);
    float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int j0 = 0; j0 < L; j0 += 32) {
        const int j = j0 + lane;
        float x = -INFINITY, vs = 0.f;
        size_t at = 0;
        bool live = false;
        if (j < L) {
            const int page = p.block_table[(size_t)s * p.max_blocks + j / p.page_size];
            if (page < 0 || page >= p.num_pages) {
                flag(p.status, FD_DEV_BAD_PAGE);
            } else {
                live = true;
                at = (((size_t)page * p.page_size + j % p.page_size) * p.Hkv + kvh) * D;
                float dot = 0.f;
#pragma unroll
                for (int d = 0; d < D; ++d) dot = fmaf(q[d], as_float(p.k_pages, at + d, p.kv_kind), dot);
                const float ks = p.k_scale ? p.k_scale[(size_t)page * p.Hkv + kvh] : 1.f;
                vs = p.v_scale ? p.v_scale[(size_t)page * p.Hkv + kvh] : 1.f;
                x = dot * ks * p.scale_log2;
            }
        }
        float mx = x;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, shfl_xor(mx, k));
        const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.f : mn;
        const float a = exp2f(m - ref), w8 = live ? exp2f(x - ref) : 0.f;
        m = mn;
        l = l * a + w8;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= a;
        const unsigned any = __ballot_sync(0xffffffffu, live);
        for (int k = 0; k < 32; ++k) {
            if (!((any >> k) & 1u)) continue;
            const float pk = __shfl_sync(0xffffffffu, w8 * vs, k);
            const size_t ak = __shfl_sync(0xffffffffu, (unsigned long long)at, k);
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = fmaf(pk, as_float(p.v_pages, ak + lane * E + e, p.kv_kind), o[e]);
        }
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) l += shfl_xor(l, k);
    const size_t row = tok * p.Hq + h;
    float lse = m == -INFINITY ? -INFINITY : (m + log2f(l)) * kLn2;
    float wa = m == -INFINITY ? 0.f : 1.f / l, wb = 0.f;
    if (p.own_out) {
        const float lb = p.own_lse[row], mx = fmaxf(lse, lb);
        const float ea = lse == -INFINITY ? 0.f : expf(lse - mx), eb = lb == -INFINITY ? 0.f : expf(lb - mx);
        const float sum = ea + eb;
        wa = sum > 0.f ? wa * ea / sum : 0.f;
        wb = sum > 0.f ? eb / sum : 0.f;
        lse = mx == -INFINITY ? -INFINITY : mx + logf(sum);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float y = o[e] * wa + (p.own_out ? p.own_out[row * D + lane * E + e] * wb : 0.f);
        const size_t at = row * D + lane * E + e;
        if (p.q_bf16)
            reinterpret_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(y);
        else
            reinterpret_cast<__half *>(p.out)[at] = __float2half_rn(y);
    }
    if (lane == 0 && p.lse) p.lse[row] = lse;
}

// One warp a query row (sequence, token, head): the partial states of its chunks
// and, where there is one, the state over its own tokens.  Rows that the main
// kernel finished itself, or never had, have row_splits = 0.
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
    float mx = -INFINITY;
    for (int s = lane; s < n; s += 32) mx = fmaxf(mx, __ldcg(pm + s));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, shfl_xor(mx, o));
    const float base = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, y[E];
#pragma unroll
    for (int x = 0; x < E; ++x) y[x] = 0.f;
    for (int s = 0; s < n; ++s) {
        const float d = __ldcg(pd + s);
        if (d == 0.f) continue;  // an empty state
        const float a = ex2(__ldcg(pm + s) - base);
        sum = fmaf(a, d, sum);
        const float *po = p.part_o + (row * p.S + s) * D + lane * E;
#pragma unroll
        for (int x = 0; x < E; ++x) y[x] = fmaf(a, __ldcg(po + x), y[x]);
    }
    const bool empty = sum == 0.f;
    float lse = empty ? -INFINITY : (mx + __log2f(sum)) * kLn2;
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

template <int KV, int D>
cudaError_t launch_rows_t(const RowsParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid, cudaStream_t stream) {
    using Sh = RowsShape<KV, D>;
    auto kern = fd_rows_kernel<KV, D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
    if (e != cudaSuccess) return e;
    return launch_after(kern, (unsigned)grid, Sh::THREADS, Sh::SMEM, stream, p, tmk, tmv);
}

}  // namespace

cudaError_t launch_rows(const RowsParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid, cudaStream_t stream) {
    if (p.kv_kind == KV_BF16)
        return p.D == 128 ? launch_rows_t<KV_BF16, 128>(p, tmk, tmv, grid, stream)
                          : launch_rows_t<KV_BF16, 64>(p, tmk, tmv, grid, stream);
    if (p.kv_kind == KV_F16)
        return p.D == 128 ? launch_rows_t<KV_F16, 128>(p, tmk, tmv, grid, stream)
                          : launch_rows_t<KV_F16, 64>(p, tmk, tmv, grid, stream);
    const long long rows = (long long)p.seqs * p.T * p.Hq;
    const unsigned blocks = (unsigned)((rows + 3) / 4);
    if (p.D == 128)
        fd_rows_plain_kernel<128><<<blocks, 128, 0, stream>>>(p);
    else
        fd_rows_plain_kernel<64><<<blocks, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_rows_merge(const RowsParams &p, cudaStream_t stream) {
    const long long rows = (long long)p.seqs * p.T * p.Hq;
    const unsigned blocks = (unsigned)((rows + 3) / 4);
    return p.D == 128 ? launch_after(fd_rows_merge_kernel<128>, blocks, 128, 0, stream, p)
                      : launch_after(fd_rows_merge_kernel<64>, blocks, 128, 0, stream, p);
}

}  // namespace fd

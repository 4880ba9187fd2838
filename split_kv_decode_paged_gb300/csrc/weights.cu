// weights.cu -- attention weight of every cached token, added to its running
// total: total[b][kvh][t] += sum over the query rows r of the KV head (its
// query heads, and the query tokens of a multi-token call) of
// exp(s_r(t) - lse_r).  The decode kernel that ran before left the scores
// s_r(t) in log2 units (-inf where row r does not see t), R of them a token,
// and lse.  A weight cannot be formed before the row's lse is known, and the
// scores are 4 R bytes a token and KV head, out and back, where K's row, to be
// read again otherwise, is 64 to 256: less for few rows, more for many (25 rows
// over E4M3 take 9 times the time of their bytes).
//
// Only rows that the decode kernel split (or whose query rows take several
// work items) come here; it finishes the others itself, from scores that are
// still in L2.  One sequence of 131072 tokens, 8 heads: 8 us of the call's 96
// (the decode alone 84).
#include "weights.cuh"

namespace fd {

constexpr int kWeightThreads = 128;
constexpr int kWeightFly = 8;  // tokens per thread: one round of loads a CTA
constexpr int kWeightChunk = kWeightThreads * kWeightFly;
constexpr float kLog2e = 1.4426950408889634f;

__global__ void __launch_bounds__(kWeightThreads) fd_weights_kernel(const __grid_constant__ WeightParams p, int chunks) {
    grid_dependency_wait();
    extern __shared__ float lse2[];  // the rows' lse in log2 units, then ones
    const int stride = score_stride(p.R);
    const long long bh = blockIdx.x / chunks;
    const int chunk = (int)(blockIdx.x % chunks);
    const int b = (int)(bh / p.Hkv), h = (int)(bh % p.Hkv);
    int L = p.seq_lens[b];
    if (L > p.cap) L = p.cap;  // flagged by the decode kernel
    if (L <= p.skip_to) return;
    if (L > p.weights_stride) {
        if (threadIdx.x == 0 && chunk == 0 && h == 0 && p.status) atomicOr(p.status, FD_DEV_CAPACITY);
        L = p.weights_stride;
    }
    const int t0 = chunk * kWeightChunk, t1 = min(L, t0 + kWeightChunk);
    if (t0 >= t1) return;
    for (int r = threadIdx.x; r < p.R; r += kWeightThreads) {
        const size_t row = ((size_t)b * p.fold + r / p.G) * p.Hq + (size_t)h * p.G + r % p.G;
        const float l = p.lse[row];
        lse2[r] = l == -INFINITY ? 0.f : l * kLog2e;
        lse2[stride + r] = 1.f;
    }
    __syncthreads();
    const size_t at = (size_t)bh * p.weights_stride;
    sum_weights<kWeightThreads, kWeightFly>(p.scores + (size_t)bh * p.cap * stride, p.R, lse2, lse2 + stride,
                                            p.in ? p.in + at : nullptr, p.out + at, t0, t1, threadIdx.x);
}

bool weights_launchable(int Bkv, int Hkv, long long cap, long long R) {
    const long long chunks = (cap + kWeightChunk - 1) / kWeightChunk;
    // the rows' lse and ones in the 48 KB of shared memory that every launch may have
    constexpr long long kMaxRows = 48 * 1024 / (2 * sizeof(float));
    return chunks <= 0x7fffffffLL / ((long long)Bkv * Hkv) && R <= kMaxRows && score_stride((int)R) <= kMaxRows;
}

// For sizes that weights_launchable() takes.
cudaError_t launch_weights(const WeightParams &wp, cudaStream_t stream) {
    const long long chunks = (wp.cap + kWeightChunk - 1) / kWeightChunk;
    const long long blocks = (long long)wp.Bkv * wp.Hkv * chunks;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kWeightThreads);
    cfg.dynamicSmemBytes = (size_t)score_stride(wp.R) * 2 * sizeof(float);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fd_weights_kernel, wp, (int)chunks);
}

}  // namespace fd

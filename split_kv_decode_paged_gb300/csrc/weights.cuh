// weights.cuh -- attention weights of a run of cached tokens from their scores.
#pragma once

#include "fd_internal.h"
#include "ptx.cuh"

namespace fd {

// Floats a token's R scores take: whole 16-byte groups from 3 on (the padding
// columns hold the scores of absent query rows, NaN over an infinite key, and
// are not read).
__host__ __device__ constexpr int score_stride(int R) { return R <= 2 ? R : (R + 3) / 4 * 4; }

// out[t] = in[t] + sum over r < R of 2^(sc[t][r] - row_max[r]) * row_inv[r] for
// t in [t0, t1), by THREADS threads (tid).  FLY tokens a thread are in flight:
// the loop is a chain of L2 (in: DRAM) round trips otherwise.  A token's scores
// are score_stride(R) apart, read 16 bytes at a time where that is a multiple
// of 4 (sc 16-byte aligned), the last R % 4 by themselves.  A row that sees
// nothing has all scores -inf and a finite row_max: it adds 0.
template <int THREADS, int FLY>
__device__ __forceinline__ void sum_weights(const float *sc, int R, const float *row_max, const float *row_inv,
                                            const float *in, float *out, int t0, int t1, int tid) {
    const int stride = score_stride(R);
    for (int tb = t0 + tid; tb < t1; tb += FLY * THREADS) {
        float sum[FLY], old[FLY];
#pragma unroll
        for (int k = 0; k < FLY; ++k) {
            const int t = tb + k * THREADS;
            sum[k] = 0.f;
            old[k] = (in && t < t1) ? in[t] : 0.f;
        }
        int r = 0;
        if ((stride & 3) == 0) {
            for (; r + 4 <= R; r += 4) {
                float4 s[FLY];
#pragma unroll
                for (int k = 0; k < FLY; ++k) {
                    const int t = tb + k * THREADS;
                    s[k] = t < t1 ? __ldcg(reinterpret_cast<const float4 *>(sc + (size_t)t * stride + r))
                                  : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                }
#pragma unroll
                for (int k = 0; k < FLY; ++k) {
                    sum[k] = fmaf(ex2(s[k].x - row_max[r]), row_inv[r], sum[k]);
                    sum[k] = fmaf(ex2(s[k].y - row_max[r + 1]), row_inv[r + 1], sum[k]);
                    sum[k] = fmaf(ex2(s[k].z - row_max[r + 2]), row_inv[r + 2], sum[k]);
                    sum[k] = fmaf(ex2(s[k].w - row_max[r + 3]), row_inv[r + 3], sum[k]);
                }
            }
        }
        for (; r < R; ++r) {
            float s[FLY];
#pragma unroll
            for (int k = 0; k < FLY; ++k) {
                const int t = tb + k * THREADS;
                s[k] = t < t1 ? __ldcg(sc + (size_t)t * stride + r) : -INFINITY;
            }
#pragma unroll
            for (int k = 0; k < FLY; ++k) sum[k] = fmaf(ex2(s[k] - row_max[r]), row_inv[r], sum[k]);
        }
#pragma unroll
        for (int k = 0; k < FLY; ++k) {
            const int t = tb + k * THREADS;
            if (t < t1) out[t] = old[k] + sum[k];
        }
    }
}

}  // namespace fd

// append_norm.cu -- new tokens on their way into the paged cache in one pass:
// the RMS norm of every query and key head, the rotary embedding, and the
// write of K and V into the pools (E4M3 pools: quantised as fd_append_kv does).
//
//   y = x * rsqrt(mean(x^2) + eps) * w      per head row of D, in fp32
//   pair (a, b) of y at angle index i: (a cos - b sin, b cos + a sin)
//
// rounded once, to the type it is stored in.  A row of D 16-bit elements is
// D / 8 lanes of 16 bytes, so a warp takes 2 rows (D = 128) or 4 (D = 64) a
// step; a lane keeps its place in the row, so the token's cosines and sines
// and the norm weights stay in its registers over all the token's heads.
#include "fd_internal.h"
#include "ptx.cuh"

namespace fd {

constexpr int kNormWarps = 4;
constexpr int kNormUnroll = 2;  // steps of a warp whose rows are requested together

enum RotKind { ROT_NONE = 0, ROT_PAIRS = 1, ROT_HALVES = 2, ROT_HALVES_ANY = 3 };

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &r, float *x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (BF16) {
            x[2 * k] = __uint_as_float(w[k] << 16);
            x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
            x[2 * k] = f.x;
            x[2 * k + 1] = f.y;
        }
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float *y) {
    uint4 r;
    uint32_t *w = reinterpret_cast<uint32_t *>(&r);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        w[k] = BF16 ? pack_bf16x2(y[2 * k], y[2 * k + 1]) : pack_f16x2(y[2 * k], y[2 * k + 1]);
    return r;
}

template <bool BF16>
__device__ __forceinline__ void load_weight8(const void *w, int f32, int d0, float *out) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (f32) {
            out[e] = __ldg(reinterpret_cast<const float *>(w) + d0 + e);
        } else {
            const uint16_t b = __ldg(reinterpret_cast<const uint16_t *>(w) + d0 + e);
            out[e] = BF16 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
        }
    }
}

template <int D, bool BF16, bool FP8, int ROT>
__global__ void __launch_bounds__(kNormWarps * 32) fd_append_kv_norm_kernel(const __grid_constant__ NormAppendParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / LPR, d0 = (lane % LPR) * 8;
    const long long job = (long long)blockIdx.x * kNormWarps + warp;  // (token, part of its rows)
    const long long tok = job / p.parts;
    const int part = (int)(job - tok * p.parts);
    if (tok >= (long long)p.B * p.T) return;
    const int b = (int)(tok / p.T), i = (int)(tok - (long long)b * p.T);
    const int nrows = p.Hq + 2 * p.Hkv;
    const int step = p.parts * RPW;

    auto load_row = [&](int row) -> uint4 {
        if (row >= nrows) return make_uint4(0u, 0u, 0u, 0u);
        const uint16_t *src;
        if (row < p.Hq)
            src = reinterpret_cast<const uint16_t *>(p.q) + tok * p.q_stride + (size_t)row * D;
        else if (row < p.Hq + p.Hkv)
            src = reinterpret_cast<const uint16_t *>(p.k) + tok * p.k_stride + (size_t)(row - p.Hq) * D;
        else
            src = reinterpret_cast<const uint16_t *>(p.v) + tok * p.v_stride + (size_t)(row - p.Hq - p.Hkv) * D;
        return *reinterpret_cast<const uint4 *>(src + d0);
    };
    // The first rows do not depend on where they go: requested before the
    // lengths, positions and page id.
    uint4 raw[kNormUnroll];
#pragma unroll
    for (int u = 0; u < kNormUnroll; ++u) raw[u] = load_row(part * RPW + sub + u * step);

    const int fresh = p.new_lens ? __ldg(p.new_lens + b) : p.T;
    const int len = __ldg(p.seq_lens + b);
    const long long pos = (long long)(p.positions ? __ldg(p.positions + b) : len) + i;
    if (fresh < 0 || fresh > p.T) {
        if (lane == 0 && part == 0 && i == 0 && p.status) atomicOr(p.status, FD_DEV_CAPACITY);
        return;
    }
    if (i >= fresh) return;
    if (ROT != ROT_NONE && (pos < 0 || pos >= p.max_pos)) {
        if (lane == 0 && part == 0 && p.status) atomicOr(p.status, FD_DEV_CAPACITY);
        return;
    }
    const long long at = (long long)len + i;
    const long long col = len >= 0 ? at / p.page_size : -1;
    int page = -1;
    if (col >= 0 && col < p.max_blocks) page = __ldg(p.block_table + (size_t)b * p.max_blocks + col);
    const bool stored = page >= 0 && page < p.num_pages;
    if (!stored && lane == 0 && part == 0 && p.status) atomicOr(p.status, FD_DEV_BAD_PAGE);
    const size_t dst_tok = stored ? ((size_t)page * p.page_size + (size_t)(at - col * p.page_size)) * p.Hkv : 0;

    // This lane's cosines and sines: element e of the row turns with angle
    // index ai(e); elements from rotary_dim on pass through.
    const int half = p.rotary_dim >> 1;
    float c[8], s[8];
    if constexpr (ROT != ROT_NONE) {
        const float *cr = p.cos + (size_t)pos * half, *sr = p.sin + (size_t)pos * half;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int d = d0 + e;
            const int ai = ROT == ROT_PAIRS ? d >> 1 : (d < half ? d : d - half);
            const bool in = d < p.rotary_dim;
            c[e] = in ? __ldg(cr + ai) : 1.f;
            s[e] = in ? __ldg(sr + ai) : 0.f;
        }
    }
    float wq[8], wk[8];
    if (p.qw) load_weight8<BF16>(p.qw, p.w_f32, d0, wq);
    if (p.kw) load_weight8<BF16>(p.kw, p.w_f32, d0, wk);
    __shared__ float xch[ROT == ROT_HALVES_ANY ? kNormWarps * RPW * D : 1];

    for (int r0 = part * RPW; r0 < nrows; r0 += kNormUnroll * step) {
        if (r0 != part * RPW) {
#pragma unroll
            for (int u = 0; u < kNormUnroll; ++u) raw[u] = load_row(r0 + sub + u * step);
        }
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
            if (r0 + u * step >= nrows) break;  // the same for the whole warp
            const int row = r0 + sub + u * step;
            const int kind = row < p.Hq ? 0 : (row < p.Hq + p.Hkv ? 1 : 2);  // q, k, v
            float x[8];
            unpack8<BF16>(raw[u], x);
            // every lane takes part in the row sums; v rows drop them
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += shfl_xor(ss, o);
            const bool normed = kind == 0 ? p.qw != nullptr : (kind == 1 && p.kw != nullptr);
            if (normed) {
                const float inv = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * (kind == 0 ? wq[e] : wk[e]);
            }
            if constexpr (ROT != ROT_NONE) {
                float y[8];
                if constexpr (ROT == ROT_PAIRS) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
                } else if constexpr (ROT == ROT_HALVES) {
                    // half a multiple of 8: element e's partner is element e
                    // of the lane half / 8 places on (or back)
                    const int hl = half >> 3, l = lane % LPR;
                    const int from = lane - l + (l < hl ? l + hl : (l < 2 * hl ? l - hl : l));
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], from);
                } else {
                    float *buf = xch + (warp * RPW + sub) * D;
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e) buf[d0 + e] = x[e];
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int d = d0 + e;
                        y[e] = d < p.rotary_dim ? buf[d < half ? d + half : d - half] : 0.f;
                    }
                }
                if (kind < 2) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int d = d0 + e;
                        const bool first = ROT == ROT_PAIRS ? (e & 1) == 0 : d < half;
                        // each product and the sum rounded by itself, as in fd_append_kv_rotary
                        const float r = first ? __fsub_rn(__fmul_rn(x[e], c[e]), __fmul_rn(y[e], s[e]))
                                              : __fadd_rn(__fmul_rn(x[e], c[e]), __fmul_rn(y[e], s[e]));
                        if (d < p.rotary_dim) x[e] = r;
                    }
                }
            }
            if (row >= nrows) continue;
            if (kind == 0) {
                uint16_t *out = reinterpret_cast<uint16_t *>(p.q_out) + tok * p.q_out_stride + (size_t)row * D + d0;
                *reinterpret_cast<uint4 *>(out) = pack8<BF16>(x);
                continue;
            }
            if (!stored) continue;
            const int h = row - p.Hq - (kind == 2 ? p.Hkv : 0);
            const size_t dst = (dst_tok + h) * D + d0;
            void *pool = kind == 1 ? p.k_pages : p.v_pages;
            if constexpr (FP8) {
                const float sc = __ldg((kind == 1 ? p.k_scale : p.v_scale) + (size_t)page * p.Hkv + h);
                uint2 codes;
                uint32_t *cw = reinterpret_cast<uint32_t *>(&codes);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t lo = f32x2_to_e4m3x2(__fdiv_rn(x[4 * k + 1], sc), __fdiv_rn(x[4 * k], sc));
                    const uint32_t hi = f32x2_to_e4m3x2(__fdiv_rn(x[4 * k + 3], sc), __fdiv_rn(x[4 * k + 2], sc));
                    cw[k] = lo | (hi << 16);
                }
                *reinterpret_cast<uint2 *>(reinterpret_cast<uint8_t *>(pool) + dst) = codes;
            } else {
                *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(pool) + dst) = pack8<BF16>(x);
            }
        }
    }
}

namespace {

template <int D, bool BF16, bool FP8>
cudaError_t launch_rot(const NormAppendParams &p, int rot, unsigned blocks, cudaStream_t stream) {
    const int threads = kNormWarps * 32;
    switch (rot) {
    case ROT_NONE: fd_append_kv_norm_kernel<D, BF16, FP8, ROT_NONE><<<blocks, threads, 0, stream>>>(p); break;
    case ROT_PAIRS: fd_append_kv_norm_kernel<D, BF16, FP8, ROT_PAIRS><<<blocks, threads, 0, stream>>>(p); break;
    case ROT_HALVES: fd_append_kv_norm_kernel<D, BF16, FP8, ROT_HALVES><<<blocks, threads, 0, stream>>>(p); break;
    default: fd_append_kv_norm_kernel<D, BF16, FP8, ROT_HALVES_ANY><<<blocks, threads, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_kind(const NormAppendParams &p, int rot, unsigned blocks, cudaStream_t stream) {
    if (p.kv_kind == KV_E4M3)
        return p.is_bf16 ? launch_rot<D, true, true>(p, rot, blocks, stream)
                         : launch_rot<D, false, true>(p, rot, blocks, stream);
    return p.is_bf16 ? launch_rot<D, true, false>(p, rot, blocks, stream)
                     : launch_rot<D, false, false>(p, rot, blocks, stream);
}

}  // namespace

// D: 64 or 128 (validated); p.parts is set here.  A grid that CUDA cannot
// launch is cudaErrorInvalidConfiguration.
cudaError_t launch_append_norm(NormAppendParams p, int D, int interleaved, cudaStream_t stream) {
    const long long tokens = (long long)p.B * p.T;
    const int rpw = 256 / D;
    const int steps = (p.Hq + 2 * p.Hkv + rpw - 1) / rpw;
    p.parts = steps;  // one step a warp
    if (tokens * steps > 16384) p.parts = (steps + 7) / 8;
    const long long blocks = (tokens * p.parts + kNormWarps - 1) / kNormWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    int rot = ROT_NONE;
    if (p.cos) rot = interleaved ? ROT_PAIRS : (p.rotary_dim % 16 == 0 ? ROT_HALVES : ROT_HALVES_ANY);
    return D == 128 ? launch_kind<128>(p, rot, (unsigned)blocks, stream)
                    : launch_kind<64>(p, rot, (unsigned)blocks, stream);
}

}  // namespace fd

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
// Where the rotary part turns in halves its lanes hold four elements of each
// half instead of eight neighbours: their pairs are their own, no lane exchange,
// and they need four cosines and sines, not eight (half of D turning, the tokens
// below: 89 -> 72 us).
//
// One pass: every input is read and every output written once.  Many tokens
// are bound by instruction issue (63% of the slots) about as much as by DRAM:
// 16.6K tokens of 32 + 8 + 8 heads, D = 128, bf16, 411 MB in 70 us, 5.9 TB/s,
// 86% of the copy rate.  A loop per kind of row halved the instructions (no
// selects between q, k and v): 105 -> 75 us.  Few tokens are a chain of
// latencies (lengths, page id, cosines): 1 token 3.6 us, 256 tokens of 64 + 8 +
// 8 heads into E4M3 6.5 us.  The many tokens into E4M3: 84 us of 55 for their
// bytes, a division by the page's scale for every element of K and V.
#include <algorithm>

#include "fd_internal.h"
#include "ptx.cuh"

namespace fd {

constexpr int kNormWarps = 4;
constexpr int kNormUnroll = 4;  // steps of a warp whose rows are requested together

// How the pairs of a row lie in the lanes.
enum RotKind {
    ROT_NONE = 0,
    ROT_PAIRS = 1,   // (2i, 2i + 1): in the lane
    ROT_HALVES = 2,  // halves, rotary_dim a multiple of 8: four elements of each half in the lane
    ROT_ANY = 3      // other halves: through shared memory
};

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

// Four norm weights from element d on (w16: 8-byte aligned 16-bit weights).
template <bool BF16>
__device__ __forceinline__ void load_weight4(const void *w, int f32, bool w16, int d, float *out) {
    if (!f32 && w16) {
        const uint2 r = __ldg(reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(w) + d));
        float x[8];
        unpack8<BF16>(make_uint4(r.x, r.y, 0u, 0u), x);
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] = x[e];
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (f32) {
            out[e] = __ldg(reinterpret_cast<const float *>(w) + d + e);
        } else {
            const uint16_t b = __ldg(reinterpret_cast<const uint16_t *>(w) + d + e);
            out[e] = BF16 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
        }
    }
}

// ONE: a warp has one step (few tokens: the latency of a call); its rows are
// requested before the length, position and page id that say where they go, in
// a padded batch once new_lens says that the token is there: what lies behind a
// sequence's tokens is not read.  Otherwise a warp goes through every p.parts-th
// step of its token.
template <int D, bool BF16, bool FP8, int ROT, bool ONE>
__global__ void __launch_bounds__(kNormWarps * 32) fd_append_kv_norm_kernel(const __grid_constant__ NormAppendParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    constexpr int NCS = ROT == ROT_NONE ? 1 : (ROT == ROT_ANY ? 8 : 4);  // cosines a lane holds
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();    // launched while the kernel before drains
    grid_launch_dependents();  // and the next one (the decode) may be, too
    const int sub = lane / LPR, l = lane % LPR;
    // elements 0-3 of the lane are da .. da + 3 of the row, 4-7 db .. db + 3
    const bool split = ROT == ROT_HALVES && 8 * l < p.rotary_dim;  // four of each half, else eight neighbours
    const int da = split ? 4 * l : 8 * l, db = split ? (p.rotary_dim >> 1) + 4 * l : 8 * l + 4;
    const long long job = (long long)blockIdx.x * kNormWarps + warp;  // (token, part of its rows)
    const long long tok = job / p.parts;
    const int part = (int)(job - tok * p.parts);
    if (tok >= (long long)p.B * p.T) return;
    const int b = (int)(tok / p.T), i = (int)(tok - (long long)b * p.T);
    // Steps of this token: those of q, then k, then v (a step has one kind).
    const int sq = (p.Hq + RPW - 1) / RPW, sk = (p.Hkv + RPW - 1) / RPW;

    auto load8 = [&](const uint16_t *src) -> uint4 {
        if constexpr (ROT == ROT_HALVES) {
            const uint2 x = *reinterpret_cast<const uint2 *>(src + da), y = *reinterpret_cast<const uint2 *>(src + db);
            return make_uint4(x.x, x.y, y.x, y.y);
        } else {
            return *reinterpret_cast<const uint4 *>(src + da);
        }
    };
    const uint16_t *qrow = reinterpret_cast<const uint16_t *>(p.q) + tok * p.q_stride;
    const uint16_t *krow = reinterpret_cast<const uint16_t *>(p.k) + tok * p.k_stride;
    const uint16_t *vrow = reinterpret_cast<const uint16_t *>(p.v) + tok * p.v_stride;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    if (p.new_lens) {
        const int fresh = __ldg(p.new_lens + b);
        if (fresh < 0 || fresh > p.T) {
            if (lane == 0 && part == 0 && i == 0 && p.status) atomicOr(p.status, FD_DEV_CAPACITY);
            return;
        }
        if (i >= fresh) return;
    }
    uint4 first = none;
    if constexpr (ONE) {
        const int kind = part < sq ? 0 : (part < sq + sk ? 1 : 2);
        const int row = (part - (kind == 0 ? 0 : (kind == 1 ? sq : sq + sk))) * RPW + sub;
        if (row < (kind == 0 ? p.Hq : p.Hkv)) first = load8((kind == 0 ? qrow : (kind == 1 ? krow : vrow)) + row * D);
    }
    const int len = __ldg(p.seq_lens + b);
    const long long pos = (long long)(p.positions ? __ldg(p.positions + b) : len) + i;
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

    // This lane's cosines and sines; elements from rotary_dim on pass through.
    const int rd = p.rotary_dim, half = rd >> 1;
    float c[NCS], s[NCS];
    if constexpr (ROT != ROT_NONE) {
        const float *cr = p.cos + (size_t)pos * half, *sr = p.sin + (size_t)pos * half;
        if constexpr (ROT == ROT_ANY) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int d = da + e;
                const int ai = d < half ? d : d - half;
                c[e] = d < rd ? __ldg(cr + ai) : 1.f;
                s[e] = d < rd ? __ldg(sr + ai) : 0.f;
            }
        } else if (p.cs_vec) {
            // angle indices of the lane's pairs: 4 l .. 4 l + 3 either way
            if (8 * l < rd) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(cr + 4 * l));
                const float4 y = __ldg(reinterpret_cast<const float4 *>(sr + 4 * l));
                c[0] = x.x; c[1] = x.y; c[2] = x.z; c[3] = x.w;
                s[0] = y.x; s[1] = y.y; s[2] = y.z; s[3] = y.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                c[e] = 4 * l + e < half ? __ldg(cr + 4 * l + e) : 1.f;
                s[e] = 4 * l + e < half ? __ldg(sr + 4 * l + e) : 0.f;
            }
        }
    }
    float w[8];  // norm weights of the kind at hand
    auto load_weights = [&](const void *src) {
        if (src) {
            load_weight4<BF16>(src, p.w_f32, p.w_vec, da, w);
            load_weight4<BF16>(src, p.w_f32, p.w_vec, db, w + 4);
        }
    };
    __shared__ float xch[ROT == ROT_ANY ? kNormWarps * RPW * D : 1];

    // each product and the sum rounded by itself, as in fd_append_kv_rotary
    auto turn_first = [](float x, float y, float cc, float ss) { return __fsub_rn(__fmul_rn(x, cc), __fmul_rn(y, ss)); };
    auto turn_second = [](float x, float y, float cc, float ss) { return __fadd_rn(__fmul_rn(x, cc), __fmul_rn(y, ss)); };
    // Norm and rotation of a q or k row; every lane of the warp takes part.
    auto norm_turn = [&](bool normed, float *x) {
        if (normed) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += shfl_xor(ss, o);
            const float inv = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * w[e];
        }
        if constexpr (ROT == ROT_HALVES) {
            if (split) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a = x[e], bb = x[e + 4];
                    x[e] = turn_first(a, bb, c[e], s[e]);
                    x[e + 4] = turn_second(bb, a, c[e], s[e]);
                }
            }
        } else if constexpr (ROT == ROT_PAIRS) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float a = x[2 * e], bb = x[2 * e + 1];
                const float ra = turn_first(a, bb, c[e], s[e]), rb = turn_second(bb, a, c[e], s[e]);
                if (4 * l + e < half) {
                    x[2 * e] = ra;
                    x[2 * e + 1] = rb;
                }
            }
        } else if constexpr (ROT == ROT_ANY) {
            float y[8];
            float *buf = xch + (warp * RPW + sub) * D;
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; ++e) buf[da + e] = x[e];
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int d = da + e;
                y[e] = d < rd ? buf[d < half ? d + half : d - half] : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int d = da + e;
                const float r = d < half ? turn_first(x[e], y[e], c[e], s[e]) : turn_second(x[e], y[e], c[e], s[e]);
                if (d < rd) x[e] = r;
            }
        }
    };

    // 16 bytes of a q row, or of a cache row in its 16-bit type.
    auto store8 = [&](uint16_t *out, const uint4 &v) {
        if constexpr (ROT == ROT_HALVES) {
            *reinterpret_cast<uint2 *>(out + da) = make_uint2(v.x, v.y);
            *reinterpret_cast<uint2 *>(out + db) = make_uint2(v.z, v.w);
        } else {
            *reinterpret_cast<uint4 *>(out + da) = v;
        }
    };
    auto store_codes = [&](uint8_t *out, const float *x, float sc) {
        uint32_t cw[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t lo = f32x2_to_e4m3x2(__fdiv_rn(x[4 * k + 1], sc), __fdiv_rn(x[4 * k], sc));
            const uint32_t hi = f32x2_to_e4m3x2(__fdiv_rn(x[4 * k + 3], sc), __fdiv_rn(x[4 * k + 2], sc));
            cw[k] = lo | (hi << 16);
        }
        if constexpr (ROT == ROT_HALVES) {
            *reinterpret_cast<uint32_t *>(out + da) = cw[0];
            *reinterpret_cast<uint32_t *>(out + db) = cw[1];
        } else {
            *reinterpret_cast<uint2 *>(out + da) = make_uint2(cw[0], cw[1]);
        }
    };
    // One row (live: there is one here): v rows keep their bits in a 16-bit cache.
    uint16_t *qo = reinterpret_cast<uint16_t *>(p.q_out) + tok * p.q_out_stride;
    auto do_q = [&](uint4 bits, int row, bool live) {
        float x[8];
        unpack8<BF16>(bits, x);
        norm_turn(p.qw != nullptr, x);
        if (live) store8(qo + row * D, pack8<BF16>(x));
    };
    auto do_k = [&](uint4 bits, int row, bool live) {
        float x[8];
        unpack8<BF16>(bits, x);
        norm_turn(p.kw != nullptr, x);
        if (!live || !stored) return;
        if constexpr (FP8)
            store_codes(reinterpret_cast<uint8_t *>(p.k_pages) + (dst_tok + row) * D, x,
                        __ldg(p.k_scale + (size_t)page * p.Hkv + row));
        else
            store8(reinterpret_cast<uint16_t *>(p.k_pages) + (dst_tok + row) * D, pack8<BF16>(x));
    };
    auto do_v = [&](uint4 bits, int row, bool live) {
        if (!live || !stored) return;
        if constexpr (FP8) {
            float x[8];
            unpack8<BF16>(bits, x);
            store_codes(reinterpret_cast<uint8_t *>(p.v_pages) + (dst_tok + row) * D, x,
                        __ldg(p.v_scale + (size_t)page * p.Hkv + row));
        } else {
            store8(reinterpret_cast<uint16_t *>(p.v_pages) + (dst_tok + row) * D, bits);
        }
    };
    if constexpr (ONE) {
        if (part < sq) {
            load_weights(p.qw);
            do_q(first, part * RPW + sub, part * RPW + sub < p.Hq);
        } else if (part < sq + sk) {
            load_weights(p.kw);
            do_k(first, (part - sq) * RPW + sub, (part - sq) * RPW + sub < p.Hkv);
        } else {
            do_v(first, (part - sq - sk) * RPW + sub, (part - sq - sk) * RPW + sub < p.Hkv);
        }
    } else {
        // This warp's steps of one kind with n rows, steps base and on.
        auto each = [&](int base, int n, const uint16_t *rows, auto &&work) {
            int j = part - base % p.parts;
            if (j < 0) j += p.parts;  // the first step of the kind that is this warp's
            for (int r0 = j * RPW; r0 < n; r0 += kNormUnroll * p.parts * RPW) {
                uint4 raw[kNormUnroll];
#pragma unroll
                for (int u = 0; u < kNormUnroll; ++u) {
                    const int row = r0 + u * p.parts * RPW + sub;
                    raw[u] = row < n ? load8(rows + row * D) : none;
                }
#pragma unroll
                for (int u = 0; u < kNormUnroll; ++u) {
                    const int row = r0 + u * p.parts * RPW + sub;
                    if (row - sub < n) work(raw[u], row, row < n);  // the same for the whole warp
                }
            }
        };
        load_weights(p.qw);
        each(0, p.Hq, qrow, do_q);
        load_weights(p.kw);
        each(sq, p.Hkv, krow, do_k);
        each(sq + sk, p.Hkv, vrow, do_v);
    }
}

namespace {

template <int D, bool BF16, bool FP8, int ROT>
cudaError_t launch_rot(const NormAppendParams &p, bool one, unsigned blocks, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kNormWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (one) return cudaLaunchKernelEx(&cfg, fd_append_kv_norm_kernel<D, BF16, FP8, ROT, true>, p);
    return cudaLaunchKernelEx(&cfg, fd_append_kv_norm_kernel<D, BF16, FP8, ROT, false>, p);
}

template <int D, bool BF16, bool FP8>
cudaError_t launch_types(const NormAppendParams &p, int rot, bool one, unsigned blocks, cudaStream_t stream) {
    switch (rot) {
    case ROT_NONE: return launch_rot<D, BF16, FP8, ROT_NONE>(p, one, blocks, stream);
    case ROT_PAIRS: return launch_rot<D, BF16, FP8, ROT_PAIRS>(p, one, blocks, stream);
    case ROT_HALVES: return launch_rot<D, BF16, FP8, ROT_HALVES>(p, one, blocks, stream);
    default: return launch_rot<D, BF16, FP8, ROT_ANY>(p, one, blocks, stream);
    }
}

template <int D>
cudaError_t launch_width(const NormAppendParams &p, int rot, bool one, unsigned blocks, cudaStream_t stream) {
    if (p.kv_kind == KV_E4M3)
        return p.is_bf16 ? launch_types<D, true, true>(p, rot, one, blocks, stream)
                         : launch_types<D, false, true>(p, rot, one, blocks, stream);
    return p.is_bf16 ? launch_types<D, true, false>(p, rot, one, blocks, stream)
                     : launch_types<D, false, false>(p, rot, one, blocks, stream);
}

}  // namespace

// D: 64 or 128 (validated); p.parts, p.w_vec and p.cs_vec are set here.  A grid
// that CUDA cannot launch is cudaErrorInvalidConfiguration.
cudaError_t launch_append_norm(NormAppendParams p, int D, cudaStream_t stream) {
    const long long tokens = (long long)p.B * p.T;
    const int rpw = 256 / D;
    const int steps = (p.Hq + rpw - 1) / rpw + 2 * ((p.Hkv + rpw - 1) / rpw);
    // Few tokens: a step a warp.  Many: a warp per token (measured on 16.6K
    // tokens of 24 steps: 70 us; 2 warps a token 75, 4 warps 97); between, as
    // many as give every SM 12 warps (1000 tokens of 24 steps 8.7 us; 64 warps
    // an SM 11.7, a step a warp 11.1).
    const bool one = tokens * steps <= 16384;
    p.parts = one ? steps : (int)std::min<long long>(steps, (152 * 12 + tokens - 1) / tokens);
    const long long blocks = (tokens * p.parts + kNormWarps - 1) / kNormWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto al = [](const void *x, size_t n) { return reinterpret_cast<uintptr_t>(x) % n == 0; };
    p.w_vec = al(p.qw, 8) && al(p.kw, 8);
    int rot = ROT_NONE;
    if (p.cos) {
        p.cs_vec = al(p.cos, 16) && al(p.sin, 16) && p.rotary_dim % 8 == 0;  // every row of four
        rot = p.interleaved ? ROT_PAIRS : (p.rotary_dim % 8 == 0 ? ROT_HALVES : ROT_ANY);
    }
    return D == 128 ? launch_width<128>(p, rot, one, (unsigned)blocks, stream)
                    : launch_width<64>(p, rot, one, (unsigned)blocks, stream);
}

}  // namespace fd

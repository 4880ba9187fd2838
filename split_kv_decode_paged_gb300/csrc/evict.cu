// evict.cu -- cut a sequence back to its budget of cached tokens: the first
// `sinks` tokens, the last `recent` ones and, of those between, the ones with
// the largest accumulated attention weight stay, in their order; K, V and the
// weights move up into the first n = min(L, budget) slots.  Every KV head
// chooses its own tokens.
//
// Two launches.  fd_evict_select_kernel, one CTA per (sequence, KV head),
// finds the smallest weight that stays (radix select over an order-preserving
// 32-bit key, 8 bits a round) and lists the tokens that stay with a running
// scan (ties: lowest index first).  fd_evict_move_*_kernel copies the rows.
#include "fd_internal.h"
#include "ptx.cuh"

namespace fd {

constexpr int kSelThreads = 1024;
constexpr int kSelPer = 4;  // consecutive tokens per thread and tile of the scan
constexpr int kMoveThreads = 256;

// Unsigned key in the order of the weights: -0 counts as +0, NaN as the smallest.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    uint32_t u = __float_as_uint(w);
    if (u == 0x80000000u) u = 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) fd_evict_select_kernel(const __grid_constant__ EvictParams p) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t warp_sum[kSelThreads / 32];
    __shared__ uint32_t sh_bin, sh_left;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = (int)(blockIdx.x / p.Hkv), h = (int)(blockIdx.x % p.Hkv);
    const size_t row = (size_t)b * p.Hkv + h;
    const float *w = p.weights + row * p.weights_stride;
    float *wo = p.weights_out ? p.weights_out + row * p.weights_stride : nullptr;
    int32_t *kept = p.kept + row * p.budget;
    const int L = p.seq_lens[b];
    if (L < 0 || L > p.weights_stride || (long long)L > (long long)p.max_blocks * p.page_size) {
        // nothing of this sequence is touched
        for (int t = tid; t < p.budget; t += kSelThreads) kept[t] = -1;
        if (tid == 0 && h == 0) {
            p.new_lens[b] = L;
            if (p.status) atomicOr(p.status, FD_DEV_CAPACITY);
        }
        return;
    }
    const int n = min(L, p.budget);
    if (tid == 0 && h == 0) p.new_lens[b] = n;
    for (int t = n + tid; t < p.budget; t += kSelThreads) kept[t] = -1;
    if (L <= p.budget) {
        for (int t = tid; t < L; t += kSelThreads) {
            kept[t] = t;
            if (wo && wo != w) wo[t] = w[t];
        }
        return;
    }
    const int mid0 = p.sinks, mid1 = L - p.recent;
    const int many = p.budget - p.sinks - p.recent;  // stay of [mid0, mid1); fewer than there are
    uint32_t cut = 0xffffffffu;  // keys above it stay, and the first `ties` equal to it
    uint32_t ties = 0;
    if (many > 0) {
        uint32_t prefix = 0, mask = 0, left = (uint32_t)many;
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int t = mid0 + tid; t < mid1; t += kSelThreads) {
                const uint32_t k = weight_key(w[t]);
                if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (warp == 0) {
                // bins from the top, 8 per lane: the one where the count reaches `left`
                uint32_t c[8], sum = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    c[e] = hist[255 - (lane * 8 + e)];
                    sum += c[e];
                }
                uint32_t incl = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += v;
                }
                uint32_t above = incl - sum;
                if (above < left && incl >= left) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (above < left && above + c[e] >= left) {
                            sh_bin = 255u - (uint32_t)(lane * 8 + e);
                            sh_left = left - above;
                        }
                        above += c[e];
                    }
                }
            }
            __syncthreads();
            prefix |= sh_bin << shift;
            mask |= 255u << shift;
            left = sh_left;
        }
        cut = prefix;
        ties = left;
    }
    // Places in order: a token that stays goes to (tokens before it that stay
    // for certain) + min(equal ones before it, ties).
    uint32_t sure_run = 0, tie_run = 0;
    for (int base = 0; base < L; base += kSelThreads * kSelPer) {
        float wv[kSelPer];
        bool sure[kSelPer], tie[kSelPer];
        uint32_t mine = 0;  // certain ones in the low half, ties in the high half
#pragma unroll
        for (int e = 0; e < kSelPer; ++e) {
            const int t = base + tid * kSelPer + e;
            wv[e] = t < L ? w[t] : 0.f;
            const bool inside = t >= mid0 && t < mid1;
            const uint32_t k = weight_key(wv[e]);
            sure[e] = t < L && (!inside || (many > 0 && k > cut));
            tie[e] = t < L && inside && many > 0 && k == cut;
            mine += (sure[e] ? 1u : 0u) + (tie[e] ? 0x10000u : 0u);
        }
        uint32_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();  // also: every weight of this tile has been read
        uint32_t before = 0, total = 0;
#pragma unroll
        for (int k = 0; k < kSelThreads / 32; ++k) {
            const uint32_t v = warp_sum[k];
            before += k < warp ? v : 0u;
            total += v;
        }
        uint32_t sure_at = sure_run + ((before + incl - mine) & 0xffffu);
        uint32_t tie_at = tie_run + ((before + incl - mine) >> 16);
#pragma unroll
        for (int e = 0; e < kSelPer; ++e) {
            if (sure[e] || (tie[e] && tie_at < ties)) {
                const uint32_t to = sure_at + min(tie_at, ties);
                kept[to] = base + tid * kSelPer + e;
                if (wo) wo[to] = wv[e];
            }
            sure_at += sure[e] ? 1u : 0u;
            tie_at += tie[e] ? 1u : 0u;
        }
        sure_run += total & 0xffffu;
        tie_run += total >> 16;
        __syncthreads();  // warp_sum is used again
    }
    if (wo)
        for (int t = n + tid; t < L; t += kSelThreads) wo[t] = 0.f;
}

struct RowPlace {
    long long src, dst;  // row index (page * page_size + slot) * Hkv + h; src < 0: nothing to copy
    float k_from, k_to, v_from, v_to;
};

// Where row j of (b, h) comes from and goes to.
__device__ __forceinline__ RowPlace place_row(const EvictParams &p, int b, int h, const int32_t *kept, int j, bool fp8) {
    RowPlace r;
    r.src = r.dst = -1;
    r.k_from = r.k_to = r.v_from = r.v_to = 1.f;
    const int t = kept[j];
    if (t < 0) return r;
    const int c0 = t / p.page_size, c1 = j / p.page_size;
    const int p0 = __ldg(p.block_table + (size_t)b * p.max_blocks + c0);
    const int p1 = __ldg(p.dst_table + (size_t)b * p.max_blocks + c1);
    if (p0 < 0 || p0 >= p.num_pages || p1 < 0 || p1 >= p.num_pages) {
        if (p.status) atomicOr(p.status, FD_DEV_BAD_PAGE);
        return r;
    }
    const long long src = ((long long)p0 * p.page_size + (t - c0 * p.page_size)) * p.Hkv + h;
    const long long dst = ((long long)p1 * p.page_size + (j - c1 * p.page_size)) * p.Hkv + h;
    if (src == dst) return r;
    r.src = src;
    r.dst = dst;
    if (fp8) {
        r.k_from = __ldg(p.k_scale + (size_t)p0 * p.Hkv + h);
        r.k_to = __ldg(p.k_scale + (size_t)p1 * p.Hkv + h);
        r.v_from = __ldg(p.v_scale + (size_t)p0 * p.Hkv + h);
        r.v_to = __ldg(p.v_scale + (size_t)p1 * p.Hkv + h);
    }
    return r;
}

// 16 E4M3 codes of a page with scale `from`, as codes of a page with scale `to`.
__device__ __forceinline__ uint4 rescale16(uint4 v, float from, float to) {
    uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t out = 0;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const uint32_t h2 = e4m3x2_to_f16x2((uint16_t)(w[k] >> (16 * hh)));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
            out |= (uint32_t)f32x2_to_e4m3x2(__fdiv_rn(__fmul_rn(f.y, from), to), __fdiv_rn(__fmul_rn(f.x, from), to))
                   << (16 * hh);
        }
        w[k] = out;
    }
    return v;
}

constexpr int kCopyRows = 64;

// Into other pages: no row is read and written, so every CTA copies kCopyRows
// rows of K and V at their full width.
__global__ void __launch_bounds__(kMoveThreads) fd_evict_copy_kernel(const __grid_constant__ EvictParams p, int chunks) {
    __shared__ RowPlace rows[kCopyRows];
    const long long bh = blockIdx.x / chunks;
    const int j0 = (int)(blockIdx.x % chunks) * kCopyRows;
    const int b = (int)(bh / p.Hkv), h = (int)(bh % p.Hkv);
    const int n = min(p.new_lens[b], p.budget);
    if (j0 >= n) return;
    const bool fp8 = p.row_bytes == p.D;
    const int32_t *kept = p.kept + (size_t)bh * p.budget;
    if (threadIdx.x < kCopyRows) {
        const int j = j0 + threadIdx.x;
        if (j < n) rows[threadIdx.x] = place_row(p, b, h, kept, j, fp8);
        else rows[threadIdx.x].src = -1;
    }
    __syncthreads();
    const int upr = p.row_bytes / 16;  // 16-byte units per row
    const int units = kCopyRows * upr;
    for (int u = threadIdx.x; u < 2 * units; u += kMoveThreads) {
        const bool is_v = u >= units;
        const int x = is_v ? u - units : u;
        const RowPlace &r = rows[x / upr];
        if (r.src < 0) continue;
        uint8_t *pool = reinterpret_cast<uint8_t *>(is_v ? p.v_pages : p.k_pages);
        const int off = (x % upr) * 16;
        uint4 v = *reinterpret_cast<const uint4 *>(pool + r.src * p.row_bytes + off);
        if (fp8) {
            const float from = is_v ? r.v_from : r.k_from, to = is_v ? r.v_to : r.k_to;
            if (from != to) v = rescale16(v, from, to);
        }
        *reinterpret_cast<uint4 *>(pool + r.dst * p.row_bytes + off) = v;
    }
}

// In place: row j comes from row kept[j] >= j of the same sequence, so rows
// are moved in order, a chunk of them read before any of it is written.  What
// can run at once is the width: a CTA takes one slice of K's or V's row.
__global__ void __launch_bounds__(kMoveThreads) fd_evict_shift_kernel(const __grid_constant__ EvictParams p, int slices) {
    __shared__ RowPlace rows[kMoveThreads];
    const long long bh = blockIdx.x / (2 * slices);
    const int part = (int)(blockIdx.x % (2 * slices));
    const bool is_v = part >= slices;
    const int sl = is_v ? part - slices : part;
    const int b = (int)(bh / p.Hkv), h = (int)(bh % p.Hkv);
    const int n = min(p.new_lens[b], p.budget);
    const bool fp8 = p.row_bytes == p.D;
    const int32_t *kept = p.kept + (size_t)bh * p.budget;
    if (n <= 0 || kept[n - 1] <= n - 1) return;  // nothing left out: nothing moves
    // the first row that moves (kept[j] - j never falls)
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (kept[mid] > mid) hi = mid; else lo = mid + 1;
    }
    uint8_t *pool = reinterpret_cast<uint8_t *>(is_v ? p.v_pages : p.k_pages);
    const int ups = p.row_bytes / slices / 16;  // 16-byte units of the slice
    const int per = kMoveThreads / ups;         // rows per chunk
    const int rl = threadIdx.x / ups, off = sl * (p.row_bytes / slices) + (threadIdx.x % ups) * 16;
    for (int j0 = lo; j0 < n; j0 += per) {
        __syncthreads();
        if (threadIdx.x < per) {
            const int j = j0 + threadIdx.x;
            if (j < n) rows[threadIdx.x] = place_row(p, b, h, kept, j, fp8);
            else rows[threadIdx.x].src = -1;
        }
        __syncthreads();
        const RowPlace r = rows[rl];
        uint4 v;
        if (r.src >= 0) v = *reinterpret_cast<const uint4 *>(pool + r.src * p.row_bytes + off);
        __syncthreads();  // the chunk is read
        if (r.src >= 0) {
            if (fp8) {
                const float from = is_v ? r.v_from : r.k_from, to = is_v ? r.v_to : r.k_to;
                if (from != to) v = rescale16(v, from, to);
            }
            *reinterpret_cast<uint4 *>(pool + r.dst * p.row_bytes + off) = v;
        }
    }
}

cudaError_t launch_evict(const EvictParams &p, int sms, cudaStream_t stream) {
    const long long bh = (long long)p.B * p.Hkv;
    if (bh > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const bool in_place = p.dst_table == p.block_table;
    const long long chunks = (p.budget + kCopyRows - 1) / kCopyRows;
    int slices = 1;
    while (slices * 32 < p.row_bytes && bh * 2 * slices < 2LL * sms) slices *= 2;
    const long long blocks = in_place ? bh * 2 * slices : bh * chunks;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    fd_evict_select_kernel<<<(unsigned)bh, kSelThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (in_place)
        fd_evict_shift_kernel<<<(unsigned)blocks, kMoveThreads, 0, stream>>>(p, slices);
    else
        fd_evict_copy_kernel<<<(unsigned)blocks, kMoveThreads, 0, stream>>>(p, (int)chunks);
    return cudaGetLastError();
}

}  // namespace fd

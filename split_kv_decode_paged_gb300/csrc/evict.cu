// evict.cu -- cut a sequence back to its budget of cached tokens: the first
// `sinks` tokens, the last `recent` ones and, of those between, the ones with
// the largest accumulated attention weight stay, in their order; K, V and the
// weights move up into the first n = min(L, budget) slots.  Every KV head
// chooses its own tokens.
//
// Two launches.  fd_evict_select_kernel finds the smallest weight that stays
// (radix select over an order-preserving 32-bit key, 11 + 11 + 10 bits) and
// lists the tokens that stay in order (ties: lowest index first).
// fd_evict_copy_kernel or fd_evict_shift_kernel moves the rows; it is launched
// while the first still runs and waits for it.
//
// Selection is bound by instructions and by the rounds' latency, not by bytes:
// a row's tokens are dealt to the CTAs of a cluster in tiles of 8192, one CTA
// for short rows or many of them, up to 8 for few long ones, and a tile that
// is a CTA's only one is read once and kept in registers as keys.  The CTAs
// add up their histograms and counts through distributed shared memory.
//
// Measured: 64 sequences x 8 heads of 512-8192 tokens to at most 4096, bf16, D =
// 128, into other pages 274 us (1.72 GB, 6.3 TB/s, 93% of the copy rate): the
// copy 249, the selection 25.  Four E4M3 sequences x 8 heads of 60000-65536
// tokens halved 114 us: the copy 89 (floor 79), the selection 25.  A digit of
// the radix select costs 1.2 us in one CTA; through the cluster 6 with every
// CTA reading all the others' bins, 3 with their sums read first.  In
// place 238 and 331 us: few rows leave few slices to work on at once.
#include <algorithm>

#include "fd_internal.h"
#include "ptx.cuh"

namespace fd {

constexpr int kSelPer = 16;       // tokens per thread and tile: token base + k * threads + tid
constexpr int kMaxSelCtas = 8;    // portable cluster size

// Threads of a selecting CTA and bits of a round's digit: 512 threads and
// 11 + 11 + 10 bits; rows of at most 2048 tokens, of which there are often
// many, 128 threads and 9 + 9 + 9 + 5 bits (eight CTAs an SM instead of two).
template <int THREADS>
struct SelShape {
    static constexpr int WARPS = THREADS / 32, TILE = THREADS * kSelPer;
    static constexpr int BITS = THREADS == 512 ? 11 : 9, BINS = 1 << BITS, ROUNDS = (32 + BITS - 1) / BITS;
    static constexpr int PLACES = kSelPer * WARPS;  // counts of a tile: one per (k, warp)
    static_assert(BINS == 4 * THREADS && PLACES <= THREADS && WARPS <= 32, "bins and places per thread");
};
constexpr int kMoveThreads = 256;

// Unsigned keys in the order of the weights: -0 counts as +0, NaN (key 1) as
// the smallest; the smallest number, -inf, has 0x007fffff, the largest 0xff800000.
constexpr uint32_t kKeyNan = 1u;
__device__ __forceinline__ uint32_t weight_key(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
    const uint32_t key = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return w == w ? key : kKeyNan;
}
// The weight of a key (a NaN loses its payload, -0 its sign).
__device__ __forceinline__ float key_weight(uint32_t key) {
    if (key == kKeyNan) return __uint_as_float(0x7fffffffu);
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// Exclusive prefix over the warp of v.
__device__ __forceinline__ uint32_t warp_prefix(uint32_t v, int lane) {
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    return incl - v;
}

// Exclusive prefix over the CTA of v (one value a thread) and its total; two
// barriers, sums is scratch of WARPS words.
template <int WARPS>
__device__ __forceinline__ uint32_t cta_prefix(uint32_t v, uint32_t *sums, int warp, int lane, uint32_t &total) {
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    const uint32_t s = lane < WARPS ? sums[lane] : 0u;
    uint32_t all = s;
#pragma unroll
    for (int o = 1; o < WARPS; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, all, o);
        if (lane >= o) all += x;
    }
    total = __shfl_sync(0xffffffffu, all, WARPS - 1);
    const uint32_t before = __shfl_sync(0xffffffffu, all - s, warp);
    __syncthreads();  // sums may be used again
    return before + incl - v;
}

// A barrier of the cluster's CTAs that also publishes their shared memory.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Words at this CTA's shared address p, in the cluster's CTA `rank`.  (No
// memory clobber: cluster_sync orders them, and several are to be in flight.)
__device__ __forceinline__ uint32_t cluster_addr(const uint32_t *p, uint32_t rank) {
    uint32_t addr;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
    return addr;
}
__device__ __forceinline__ uint32_t cluster_read(const uint32_t *p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(p, rank)));
    return v;
}
__device__ __forceinline__ uint4 cluster_read4(const uint32_t *p, uint32_t rank) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(cluster_addr(p, rank)));
    return v;
}

// One cluster of `ctas` CTAs (a power of two; CLUSTER: more than one) per
// (sequence, KV head); tile i * ctas + rank of the row is CTA rank's in round
// i.  All branches that hold a barrier depend on the row alone, so the
// cluster's CTAs take them together.  64 registers: three or four CTAs of 512
// threads an SM instead of two spill and measured 1 to 2% slower.
template <int THREADS, bool CLUSTER>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
    fd_evict_select_kernel(const __grid_constant__ EvictParams p, int ctas_in) {
    const int ctas = CLUSTER ? ctas_in : 1;
    using Sh = SelShape<THREADS>;
    constexpr int kSelThreads = THREADS, kSelWarps = Sh::WARPS, kSelTile = Sh::TILE, kBins = Sh::BINS;
    __shared__ __align__(16) uint32_t hist[kBins];
    __shared__ uint32_t places[Sh::PLACES];  // counts of every (k, warp) of a tile, then their prefix
    __shared__ uint32_t sums[kSelWarps];
    __shared__ uint32_t tile_total[2];       // of rounds i and i + 1
    __shared__ uint32_t sh_bin, sh_left;
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long bh = blockIdx.x / ctas;
    const int rank = (int)(blockIdx.x % ctas);
    const int b = (int)(bh / p.Hkv), h = (int)(bh % p.Hkv);
    const float *w = p.weights + (size_t)bh * p.weights_stride;
    float *wo = p.weights_out ? p.weights_out + (size_t)bh * p.weights_stride : nullptr;
    int32_t *kept = p.kept + (size_t)bh * p.budget;
    const int L = p.seq_lens[b];
    const int part = rank * kSelThreads + tid, parts = ctas * kSelThreads;  // of the cluster's threads
    if (L < 0 || L > p.weights_stride || (long long)L > (long long)p.max_blocks * p.page_size) {
        // nothing of this sequence is touched
        for (int t = part; t < p.budget; t += parts) kept[t] = -1;
        if (part == 0 && h == 0) {
            p.new_lens[b] = L;
            if (p.status) atomicOr(p.status, FD_DEV_CAPACITY);
        }
        return;
    }
    const int n = min(L, p.budget);
    if (part == 0 && h == 0) p.new_lens[b] = n;
    for (int t = n + part; t < p.budget; t += parts) kept[t] = -1;
    if (L <= p.budget) {
        for (int t = part; t < L; t += parts) kept[t] = t;
        if (wo && wo != w)
            for (int t = part; t < L; t += parts) wo[t] = w[t];
        return;
    }
    const int mid0 = p.sinks, mid1 = L - p.recent;
    const int many = p.budget - p.sinks - p.recent;  // stay of [mid0, mid1); fewer than there are
    const int round_tokens = ctas * kSelTile, first = rank * kSelTile;
    const bool one_round = L <= round_tokens;
    // Keys of the tile at hand; bit k of mid: token k is one to choose from, of
    // always: it is among the first or last ones and stays.
    uint32_t keys[kSelPer], mid = 0, always = 0;
    auto load_tile = [&](int base) {
        mid = always = 0;
#pragma unroll
        for (int k = 0; k < kSelPer; ++k) {
            const int t = base + k * kSelThreads + tid;
            keys[k] = t < L ? weight_key(w[t]) : 0u;
            const bool in = t >= mid0 && t < mid1;
            mid |= in ? 1u << k : 0u;
            always |= (t < L && !in) ? 1u << k : 0u;
        }
    };
    load_tile(first);
    uint32_t cut = 0xffffffffu;  // keys above it stay, and the first `ties` equal to it
    uint32_t ties = 0;
    if (many > 0) {
        uint32_t prefix = 0, mask = 0, left = (uint32_t)many;
#pragma unroll 1
        for (int digits = 0; digits < Sh::ROUNDS; ++digits) {
            const int shift = max(0, 32 - Sh::BITS * (digits + 1));
            const uint32_t digit = digits == Sh::ROUNDS - 1 ? (1u << (32 - Sh::BITS * (Sh::ROUNDS - 1))) - 1u : kBins - 1u;
            *reinterpret_cast<uint4 *>(&hist[4 * tid]) = make_uint4(0u, 0u, 0u, 0u);
            __syncthreads();
#pragma unroll 1
            for (int base = first; base < L; base += round_tokens) {
                if (!one_round) load_tile(base);
#pragma unroll
                for (int k = 0; k < kSelPer; ++k) {
                    const uint32_t key = keys[k];
                    if ((mid >> k & 1u) && ((key ^ prefix) & mask) == 0u)
                        atomicAdd(&hist[(key >> shift) & digit], 1u);
                }
            }
            __syncthreads();
            // The bin, from the top, where the count reaches `left`.  Thread i
            // has the bins kBins - 1 - 4 i and down.
            const uint4 own = *reinterpret_cast<const uint4 *>(&hist[kBins - 4 - 4 * tid]);
            if constexpr (!CLUSTER) {
                const uint32_t c[4] = {own.w, own.z, own.y, own.x};
                uint32_t total;
                uint32_t above = cta_prefix<kSelWarps>(c[0] + c[1] + c[2] + c[3], sums, warp, lane, total);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (above < left && above + c[e] >= left) {
                        sh_bin = (uint32_t)(kBins - 1 - 4 * tid - e);
                        sh_left = left - above;
                    }
                    above += c[e];
                }
                __syncthreads();  // read: hist may be cleared
            } else {
                // Every CTA's sums of a warp's 128 bins first, then the bins of
                // the one warp that holds the place: little goes between the SMs.
                uint32_t s = own.x + own.y + own.z + own.w;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (lane == 0) sums[warp] = s;
                cluster_sync();
                if (warp == 0) {
                    static_assert(kSelWarps <= 32, "a lane per warp's sum");
                    uint32_t x[kMaxSelCtas];
#pragma unroll
                    for (int r = 0; r < kMaxSelCtas; ++r)
                        x[r] = r < ctas && lane < kSelWarps ? cluster_read(&sums[lane], (uint32_t)r) : 0u;
                    uint32_t sum = 0;
#pragma unroll
                    for (int r = 0; r < kMaxSelCtas; ++r) sum += x[r];
                    const uint32_t above_w = warp_prefix(sum, lane);
                    const unsigned hit = __ballot_sync(0xffffffffu, above_w < left && above_w + sum >= left);
                    const int at_warp = __ffs(hit) - 1;
                    const uint32_t base = __shfl_sync(0xffffffffu, above_w, at_warp);
                    const int i = at_warp * 32 + lane;
                    uint4 v[kMaxSelCtas];
#pragma unroll
                    for (int r = 0; r < kMaxSelCtas; ++r)
                        v[r] = r < ctas ? cluster_read4(&hist[kBins - 4 - 4 * i], (uint32_t)r) : make_uint4(0u, 0u, 0u, 0u);
                    uint32_t c[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int r = 0; r < kMaxSelCtas; ++r) {
                        c[0] += v[r].w;
                        c[1] += v[r].z;
                        c[2] += v[r].y;
                        c[3] += v[r].x;
                    }
                    uint32_t above = base + warp_prefix(c[0] + c[1] + c[2] + c[3], lane);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (above < left && above + c[e] >= left) {
                            sh_bin = (uint32_t)(kBins - 1 - 4 * i - e);
                            sh_left = left - above;
                        }
                        above += c[e];
                    }
                }
                cluster_sync();  // read everywhere: hist and sums may be cleared
            }
            prefix |= sh_bin << shift;
            mask |= digit << shift;
            left = sh_left;
        }
        cut = prefix;
        ties = left;
    }
    // Places in order: a token that stays goes to (tokens before it that stay
    // for certain) + min(equal ones before it, ties).  Place and weight of a
    // token never lie behind it, and every weight of a round is read before
    // any is written, so the weights may move up in place.
    uint32_t sure_run = 0, tie_run = 0;
    int parity = 0;
#pragma unroll 1
    for (int round = 0; round < L; round += round_tokens, parity ^= 1) {
        const int base = round + first;
        if (!one_round) load_tile(base);
        uint32_t stay = always, tied = 0;  // bit k: token k stays for certain, or ties
#pragma unroll
        for (int k = 0; k < kSelPer; ++k) {
            stay |= keys[k] > cut ? mid & 1u << k : 0u;
            tied |= keys[k] == cut ? mid & 1u << k : 0u;
        }
        // counts of both (low and high half), at most kSelTile of each
#pragma unroll
        for (int k = 0; k < kSelPer; ++k) {
            const uint32_t both = (uint32_t)__popc(__ballot_sync(0xffffffffu, stay >> k & 1u)) |
                                  ((uint32_t)__popc(__ballot_sync(0xffffffffu, tied >> k & 1u)) << 16);
            if (lane == 0) places[k * kSelWarps + warp] = both;
        }
        __syncthreads();
        uint32_t total;
        const uint32_t mine = tid < Sh::PLACES ? places[tid] : 0u;
        const uint32_t at = cta_prefix<kSelWarps>(mine, sums, warp, lane, total);
        if (tid < Sh::PLACES) places[tid] = at;
        if (tid == 0) tile_total[parity] = total;
        if constexpr (CLUSTER) cluster_sync(); else __syncthreads();
        uint32_t sure0 = sure_run, tie0 = tie_run;  // of this CTA's tile
        if constexpr (CLUSTER) {
            uint32_t x[kMaxSelCtas];
#pragma unroll
            for (int r = 0; r < kMaxSelCtas; ++r) x[r] = r < ctas ? cluster_read(&tile_total[parity], (uint32_t)r) : 0u;
#pragma unroll
            for (int r = 0; r < kMaxSelCtas; ++r) {
                sure_run += x[r] & 0xffffu;
                tie_run += x[r] >> 16;
                if (r < rank) {
                    sure0 = sure_run;
                    tie0 = tie_run;
                }
            }
        } else {
            sure_run += total & 0xffffu;
            tie_run += total >> 16;
        }
#pragma unroll
        for (int k = 0; k < kSelPer; ++k) {
            const bool sure = stay >> k & 1u, tie = tied >> k & 1u;
            const unsigned sb = __ballot_sync(0xffffffffu, sure), tb = __ballot_sync(0xffffffffu, tie);
            const unsigned below = (1u << lane) - 1u;
            const uint32_t start = places[k * kSelWarps + warp];
            const uint32_t tie_at = tie0 + (start >> 16) + __popc(tb & below);
            if (sure || (tie && tie_at < ties)) {
                const uint32_t to = sure0 + (start & 0xffffu) + __popc(sb & below) + min(tie_at, ties);
                kept[to] = base + k * kSelThreads + tid;
                if (wo) wo[to] = key_weight(keys[k]);
            }
        }
        __syncthreads();  // places are used again
    }
    if (wo)
        for (int t = n + part; t < L; t += parts) wo[t] = 0.f;
    if constexpr (CLUSTER) cluster_sync();  // no CTA leaves while its counts are read
}

struct RowPlace {
    long long src, dst;      // byte offsets in the pools; src < 0: nothing to copy
    float k_ratio, v_ratio;  // E4M3: scale of the old page / scale of the new one (1: the codes stay)
};

// What codes are multiplied by between pages of these scales; equal ones (0
// and infinity too, of which there is no quotient) leave them as they are.
__device__ __forceinline__ float scale_ratio(float from, float to) { return from == to ? 1.f : __fdiv_rn(from, to); }

// Where row j of (b, h) comes from and goes to.
template <int RB, bool FP8>
__device__ __forceinline__ RowPlace place_row(const EvictParams &p, int b, int h, const int32_t *kept, int j) {
    RowPlace r;
    r.src = r.dst = -1;
    r.k_ratio = r.v_ratio = 1.f;
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
    r.src = src * RB;
    r.dst = dst * RB;
    if constexpr (FP8) {
        const size_t s0 = (size_t)p0 * p.Hkv + h, s1 = (size_t)p1 * p.Hkv + h;
        r.k_ratio = scale_ratio(__ldg(p.k_scale + s0), __ldg(p.k_scale + s1));
        r.v_ratio = scale_ratio(__ldg(p.v_scale + s0), __ldg(p.v_scale + s1));
    }
    return r;
}

// 16 E4M3 codes times the ratio of their pages' scales, rounded to codes again.
// One product per code: a division for each instead made the copy of E4M3
// rows twice as slow as its bytes.
__device__ __forceinline__ uint4 rescale16(uint4 v, float ratio) {
    uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t out = 0;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const uint32_t h2 = e4m3x2_to_f16x2((uint16_t)(w[k] >> (16 * hh)));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
            out |= (uint32_t)f32x2_to_e4m3x2(f.y * ratio, f.x * ratio) << (16 * hh);
        }
        w[k] = out;
    }
    return v;
}

constexpr int kCopyRows = 64;

// Into other pages: no row is both read and written, so every CTA copies
// kCopyRows rows of K and V at their full width, all of them in flight.
template <int RB, bool FP8>
__global__ void __launch_bounds__(kMoveThreads) fd_evict_copy_kernel(const __grid_constant__ EvictParams p, int chunks) {
    constexpr int UPR = RB / 16;                        // 16-byte units of a row
    constexpr int ROWS = kMoveThreads / UPR;            // rows of one step
    constexpr int STEPS = (kCopyRows + ROWS - 1) / ROWS;
    __shared__ RowPlace rows[kCopyRows];
    grid_dependency_wait();
    const long long bh = blockIdx.x / chunks;
    const int j0 = (int)(blockIdx.x % chunks) * kCopyRows;
    const int b = (int)(bh / p.Hkv), h = (int)(bh % p.Hkv);
    const int n = min(p.new_lens[b], p.budget);
    if (j0 >= n) return;
    const int32_t *kept = p.kept + (size_t)bh * p.budget;
    if (threadIdx.x < kCopyRows) {
        const int j = j0 + threadIdx.x;
        if (j < n) rows[threadIdx.x] = place_row<RB, FP8>(p, b, h, kept, j);
        else rows[threadIdx.x].src = -1;
    }
    __syncthreads();
    const int off = (threadIdx.x % UPR) * 16, first = threadIdx.x / UPR;
    uint8_t *kp = reinterpret_cast<uint8_t *>(p.k_pages) + off, *vp = reinterpret_cast<uint8_t *>(p.v_pages) + off;
    uint4 k[STEPS], v[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int r = first + s * ROWS;
        const long long src = r < kCopyRows ? rows[r].src : -1;
        if (src >= 0) {
            k[s] = *reinterpret_cast<const uint4 *>(kp + src);
            v[s] = *reinterpret_cast<const uint4 *>(vp + src);
        }
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int r = first + s * ROWS;
        if (r >= kCopyRows || rows[r].src < 0) continue;
        if constexpr (FP8) {
            if (rows[r].k_ratio != 1.f) k[s] = rescale16(k[s], rows[r].k_ratio);
            if (rows[r].v_ratio != 1.f) v[s] = rescale16(v[s], rows[r].v_ratio);
        }
        const long long dst = rows[r].dst;
        *reinterpret_cast<uint4 *>(kp + dst) = k[s];
        *reinterpret_cast<uint4 *>(vp + dst) = v[s];
    }
}

// In place: row j comes from row kept[j] >= j of the same sequence, so rows
// are moved in order, a chunk of them read before any of it is written (what a
// chunk writes no later chunk reads).  What can run at once is the width: a
// CTA takes one slice of K's or V's row, kShiftUnits 16-byte units a thread in
// flight, and finds the next chunk's places while they are.
constexpr int kShiftUnits = 8;
constexpr int kShiftRows = kMoveThreads * kShiftUnits / 2;  // of the narrowest slice, 32 bytes

template <int RB, bool FP8>
__global__ void __launch_bounds__(kMoveThreads) fd_evict_shift_kernel(const __grid_constant__ EvictParams p, int slices) {
    __shared__ long long src_at[2][kShiftRows], dst_at[2][kShiftRows];
    __shared__ float ratio_at[2][FP8 ? kShiftRows : 1];
    grid_dependency_wait();
    const long long bh = blockIdx.x / (2 * slices);
    const int part = (int)(blockIdx.x % (2 * slices));
    const bool is_v = part >= slices;
    const int sl = is_v ? part - slices : part;
    const int b = (int)(bh / p.Hkv), h = (int)(bh % p.Hkv);
    const int n = min(p.new_lens[b], p.budget);
    const int32_t *kept = p.kept + (size_t)bh * p.budget;
    if (n <= 0 || kept[n - 1] <= n - 1) return;  // nothing left out: nothing moves
    // the first row that moves (kept[j] - j never falls)
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (kept[mid] > mid) hi = mid; else lo = mid + 1;
    }
    const int ups = RB / slices / 16;                    // 16-byte units of the slice
    const int step = kMoveThreads / ups;                 // rows of one unit a thread
    const int chunk = step * kShiftUnits;
    const int rl = threadIdx.x / ups;
    uint8_t *pool = reinterpret_cast<uint8_t *>(is_v ? p.v_pages : p.k_pages) + sl * (RB / slices) +
                    (threadIdx.x % ups) * 16;
    auto find = [&](int j0, int buf) {
        for (int i = threadIdx.x; i < chunk; i += kMoveThreads) {
            long long s = -1, d = -1;
            float f = 1.f;
            if (j0 + i < n) {
                const RowPlace r = place_row<RB, FP8>(p, b, h, kept, j0 + i);
                s = r.src;
                d = r.dst;
                f = is_v ? r.v_ratio : r.k_ratio;
            }
            src_at[buf][i] = s;
            dst_at[buf][i] = d;
            if constexpr (FP8) ratio_at[buf][i] = f;
        }
    };
    find(lo, 0);
    __syncthreads();
    int buf = 0;
    for (int j0 = lo; j0 < n; j0 += chunk, buf ^= 1) {
        uint4 v[kShiftUnits];
#pragma unroll
        for (int u = 0; u < kShiftUnits; ++u) {
            const long long s = src_at[buf][rl + u * step];
            if (s >= 0) v[u] = *reinterpret_cast<const uint4 *>(pool + s);
        }
        if (j0 + chunk < n) find(j0 + chunk, buf ^ 1);
        __syncthreads();  // the chunk is read, the next one's places are known
#pragma unroll
        for (int u = 0; u < kShiftUnits; ++u) {
            const int r = rl + u * step;
            if (src_at[buf][r] < 0) continue;
            if constexpr (FP8) {
                if (ratio_at[buf][r] != 1.f) v[u] = rescale16(v[u], ratio_at[buf][r]);
            }
            *reinterpret_cast<uint4 *>(pool + dst_at[buf][r]) = v[u];
        }
        __syncthreads();  // these places are overwritten next
    }
}

namespace {

template <int RB, bool FP8>
cudaError_t launch_move(const EvictParams &p, bool in_place, int per_row, unsigned blocks, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (in_place) return cudaLaunchKernelEx(&cfg, fd_evict_shift_kernel<RB, FP8>, p, per_row);
    return cudaLaunchKernelEx(&cfg, fd_evict_copy_kernel<RB, FP8>, p, per_row);
}

}  // namespace

// cudaErrorInvalidConfiguration: sizes that cannot be launched, and nothing was.
cudaError_t launch_evict(const EvictParams &p, int sms, cudaStream_t stream) {
    const long long bh = (long long)p.B * p.Hkv;
    if (bh > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const bool in_place = p.dst_table == p.block_table;
    const long long chunks = (p.budget + kCopyRows - 1) / kCopyRows;
    int slices = 1;
    while (slices * 32 < p.row_bytes && bh * 2 * slices < 2LL * sms) slices *= 2;
    const long long blocks = in_place ? bh * 2 * slices : bh * chunks;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    // CTAs per row: up to one per tile of the longest row there can be, while
    // all of them still run at once.
    const long long longest = std::min<long long>(p.weights_stride, (long long)p.max_blocks * p.page_size);
    const bool short_rows = longest <= SelShape<128>::TILE;
    int ctas = 1;
    while (!short_rows && ctas < kMaxSelCtas && (long long)ctas * SelShape<512>::TILE < longest &&
           bh * ctas * 2 <= 2LL * sms)
        ctas *= 2;
    if (bh * ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    {
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)ctas;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(bh * ctas));
        cfg.blockDim = dim3(short_rows ? 128 : 512);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = ctas > 1 ? 2 : 1;
        const cudaError_t e = short_rows ? cudaLaunchKernelEx(&cfg, fd_evict_select_kernel<128, false>, p, ctas)
                              : ctas > 1 ? cudaLaunchKernelEx(&cfg, fd_evict_select_kernel<512, true>, p, ctas)
                                         : cudaLaunchKernelEx(&cfg, fd_evict_select_kernel<512, false>, p, ctas);
        if (e != cudaSuccess) return e;
    }
    const int per_row = in_place ? slices : (int)chunks;
    const auto move = p.row_bytes == 256 ? launch_move<256, false>
                      : p.row_bytes == 64  ? launch_move<64, true>
                      : p.row_bytes == p.D ? launch_move<128, true>
                                           : launch_move<128, false>;
    const cudaError_t e = move(p, in_place, per_row, (unsigned)blocks, stream);
    // the selection is on its way: no refusal any more
    return e == cudaErrorInvalidConfiguration ? cudaErrorUnknown : e;
}

}  // namespace fd

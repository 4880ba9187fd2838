// rows_kernel.cuh -- attention of many query rows over KV rows that all of them
// see (cross attention, the pass over shared prefixes), on tcgen05.
//
// The mathematics.  For the query rows r of a KV head (its G query heads, times
// the query tokens of every sequence that reads the KV row) and its n tokens:
//   S = Q K^T,  P = exp2(S c - m_r),  l_r = sum P,  O = P V,  out = O / l_r,
// c = log2(e) / sqrt(D), in one pass over K and V: m_r is a running reference
// that moves only when a score passes it by more than kSlack, and then l_r and
// O are scaled.  No row hides a token from another, so a tile of 128 rows is a
// plain matrix product, whatever sequences, tokens and heads its rows are.
//
// A work item is (KV row, KV head, chunk of its tokens, up to 256 query rows):
// two tiles of 128 rows, each with its own S / P and O in tensor memory, that
// take the same K and V tiles of 128 tokens.  While the softmax of one tile
// runs, the tensor cores work on the other's products.
//
// CTA (one an SM, persistent; items claimed from a counter):
//   warps 0-3, 4-7  softmax of tile 0 and 1: a thread has one row; reads its
//                   128 scores, writes P over them (16 bits), scales O when the
//                   reference moves, and finishes the item's rows
//   warp 8          issues the products
//   warp 9          claims items, loads K and V tiles by TMA into a ring
//   warps 10-11     gather the query rows (any sequence, token and head order,
//                   any token stride) into swizzled shared memory
//   warps 12-15     (E4M3 pools) turn the loaded codes into 16-bit tiles
// E4M3: codes become f16 values, exactly, and all products are in f16.  K's scale
// (one a page and KV head) multiplies the scores, V's the weights before their
// one rounding, relative to a power of two R at or above the chunk's largest
// scale (O is multiplied by it at the end).  Where a chunk's scales differ by more
// than kScaleRange, small ones times R^-1 would leave f16's normal range: V and
// the weights are bf16 there, the weights as pairs (two products), so that what
// other pages' scales are does not cost bits.  A bf16 query row enters times a
// power of two that brings its largest element below 2^15 (elements down to 2^-31
// of it are exact), undone on the scores.
// Every wait is bounded; one that runs out sets FD_DEV_TIMEOUT and its warp
// leaves the loop, which ends the others' waits the same way.  The limit is for
// what does not come, not for how long an item is: the query warps, which wait
// for the next item all through this one, start theirs anew while tiles are loaded
// and lists of counts read.
//
// Bounds, measured on GB300 (one pass among others).  D = 128, 16 bits, two row
// tiles: the products, 4 x 2048 queries over 8192 states of 32/8 heads 735 us =
// 1.50 PFLOP/s, 79% of a large library product's rate (two parts a weight 1032).
// D = 64: the softmax, whose work is the same for half of the products' (32 x 448
// over 1500, 16 heads 135 us, 0.65 PFLOP/s).  E4M3: the conversion, 1370 cycles for
// a tile of K or V, of some 3850 for a pair of them; the softmax warps of these
// instances spill 210 to 260 bytes at their 184 registers.  Few rows over long KV
// rows: memory (64 x 4 rows a KV head over 512-8192 states 201 us, 84% of the copy
// rate; the decode kernel, which takes such calls, 168).
// Tiles of 128 rows and tokens: the largest whose scores and outputs, twice, fill
// tensor memory; two of them, so that one's softmax hides the other's products.
#pragma once

#include <limits.h>
#include <math.h>

#include <type_traits>

#include "fd_internal.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace fd {

constexpr int kTileTokens = 128;
constexpr int kTileRows = 128;   // query rows of one tile; two tiles an item
constexpr int kItemSlots = 2;
constexpr float kRowsLn2 = 0.6931471805599453f;
constexpr float kScaleRange = 8.f;  // E4M3: ratio of V's scales within a chunk up to which the product is in f16
constexpr float kSlack = 8.f;    // log2 headroom of the softmax reference

struct RowsItem {
    int seg;      // KV row; kv_rows: none; -1: no more items
    int kvh;
    int row0;     // first query row of the item within (segment, KV head)
    int nrows;    // 1 .. 256
    int first;    // member place of the segment's first sequence
    int tok0;     // first token of the chunk
    int ntok;     // tokens of the chunk (0: an empty KV row)
    int split;
    int nsplit;
    int n0, g0;   // row0's token of the segment and head of the group
    float v_unit; // E4M3: R, or 0 where V's scales differ by too much for it
};

template <int KV, int D>
struct RowsShape {
    static constexpr bool FP8 = KV == KV_E4M3;
    static constexpr int HALVES = D / 64;                   // 128-byte spans of a row
    static constexpr int TILE = kTileTokens * D * 2;        // bytes of a Q, K or V tile (16 bits)
    static constexpr int SPAN = kTileTokens * 128;          // bytes of one half of a Q tile
    // K and V tiles: eight tokens' 128-byte spans, half after half, then the next
    // eight tokens, so that one TMA box brings all of a page's tokens
    static constexpr int GROUP = HALVES * 1024;
    static constexpr int RAW = FP8 ? kTileTokens * D : 0;   // bytes of a tile of codes
    // stages of 16-bit K and V tiles, and of codes
    static constexpr int STAGES = (FP8 ? 3 : 5) * (128 / D);
    static constexpr int RAW_STAGES = FP8 ? 4 * (128 / D) : 0;
    static constexpr int LOADS = FP8 ? RAW_STAGES : STAGES; // what TMA fills
    static constexpr int THREADS = FP8 ? 512 : 384;
    // 65536 registers dealt out evenly at launch, then anew
    static constexpr int REGS_LAUNCH = FP8 ? 128 : 168;
    static constexpr int REGS_SOFTMAX = FP8 ? 184 : 208, REGS_OTHER = FP8 ? 72 : 88;
    static_assert(256 * REGS_SOFTMAX + (THREADS - 256) * REGS_OTHER <= THREADS * REGS_LAUNCH, "the launch's registers");
    // shared memory: control block, two Q tiles, the rings
    static constexpr int CONTROL = (D == 128 ? 3 : 4) * 1024;
    static constexpr int RING = CONTROL + 2 * TILE, RAW_RING = RING + STAGES * TILE;
    static constexpr int SMEM = RAW_RING + RAW_STAGES * RAW;
    static_assert(SMEM <= 232448, "shared memory of a CTA");
    static_assert(3 * (kMaxBatch + 2) * 4 <= SMEM - CONTROL, "room for the segments' counts");
};

template <typename Sh>
struct RowsControl {
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], pv_done[2];
    uint64_t item_full[kItemSlots], item_empty[kItemSlots], rows_full, rows_empty, rows_read, join_full, join_empty, drain;
    uint64_t kv_full[Sh::STAGES], kv_empty[Sh::STAGES];              // 16-bit tiles
    uint64_t raw_full[Sh::RAW_STAGES + 1], raw_empty[Sh::RAW_STAGES + 1];  // tiles of codes
    uint32_t tmem;
    int held[kItemSlots];      // softmax warps that are done with the stage held for the item's epilogue
    RowsItem item[kItemSlots];
    // q token (sequence * T + token) of every row of the item, -1 past the end; E4M3
    // under bf16 queries: with 127 plus the exponent of the row's factor above 22 bits
    int tok[2 * kTileRows];
    float2 join[kTileRows];    // reference and denominator that tile 1's warps hand to tile 0's
    float raw_scale[Sh::RAW_STAGES + 1][16];  // of a stage's groups of 16 tokens: K's, then V's
    alignas(16) float scale[Sh::FP8 ? Sh::STAGES : 1][16];
    // Last, as the items' place decides how they are read: between tmem and held
    // this word cost D = 64 prompts 4% (32 x 448 over 1500 136 -> 142 us).
    uint32_t beat;             // tiles loaded and counts read on so far
};

// The segments of a call: query tokens and KV length of each, in the kernel's
// dispatch order.  Lengths, counts and offsets that are out of range are cut.
struct Segments {
    const RowsParams &p;
    __device__ int count() const { return p.kv_rows + (p.offsets ? 1 : 0); }
    // offsets[s] before it is made to rise
    __device__ int raw_offset(int s) const { return s > p.kv_rows ? p.seqs : (s == 0 ? 0 : __ldcg(p.offsets + s)); }
    __device__ int q_len(int b, bool &bad) const {
        const int n = __ldcg(p.q_lens + b);
        const bool out = n < 0 || n > p.T;
        bad |= out;
        return out ? 0 : n;
    }
    __device__ int kv_len(int s) const {
        if (s >= p.kv_rows) return 0;
        return min(max(__ldcg(p.kv_lens + s), 0), p.cap);
    }
    // query tokens of sequences [first, end) of the member order, by one thread
    __device__ int tokens(int first, int end, bool &bad) const {
        if (!p.q_lens) return (end - first) * p.T;
        int n = 0;
#pragma unroll 4
        for (int b = first; b < end; ++b) n += q_len(b, bad);
        return n;
    }
    // by a whole warp
    __device__ int warp_tokens(int first, int end, bool &bad, int lane) const {
        int n = 0;
#pragma unroll 4
        for (int b = first + lane; b < end; b += 32) n += q_len(b, bad);
        return __reduce_add_sync(0xffffffffu, n);
    }
    // Whether a warp on every segment takes fewer rounds of loads than a thread on
    // every one, four loads a round, the threads' scattered ones twice as long: 8
    // KV rows of 64 sequences with counts 16.6 us a call by warps, 19.4 by threads.
    __device__ bool by_warp(int segments, int warps, int threads) const {
        return p.q_lens && (segments + warps - 1) / warps * ((p.beams + 127) >> 7) <
                               2 * ((segments + threads - 1) / threads) * ((p.beams + 3) >> 2);
    }
    // The q tokens (sequence * T + token) of a segment's query tokens n[0 .. 3]
    // (-1: none) of every lane, whose sequences are [first, end), by a whole warp:
    // the sums of 256 sequences at a time, running sums where one of n may be among
    // them.  Its loops stay loops: unrolled, this code, which few calls reach, cost
    // others 2% by its size alone (32 x 448 over 1500, D = 64, 134.4 -> 137.9 us).
    __device__ void find(int first, int end, const int (&n)[4], int (&q)[4], int lane, uint32_t *beat) const {
        int high = max(max(n[0], n[1]), max(n[2], n[3])), low = INT_MAX;
#pragma unroll
        for (int k = 0; k < 4; ++k) low = min(low, n[k] < 0 ? INT_MAX : n[k]);
        low = __reduce_min_sync(0xffffffffu, low);
        high = __reduce_max_sync(0xffffffffu, high);
        int base = 0;      // tokens of the sequences before
        bool bad = false;  // said at the start
        for (int b0 = first; b0 < end && base <= high; b0 += 8 * 32) {
            if (lane == 0) atomicAdd(beat, 1u);
            const int sum = end - first > 32 ? warp_tokens(b0, min(b0 + 8 * 32, end), bad, lane) : INT_MAX - base;
            if (base + sum <= low) {
                base += sum;
                continue;
            }
#pragma unroll 1
            for (int b1 = b0; b1 < min(b0 + 8 * 32, end) && base <= high; b1 += 32) {
                int incl = b1 + lane < end ? q_len(b1 + lane, bad) : 0;
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const int t = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += t;
                }
                const int total = __shfl_sync(0xffffffffu, incl, 31);
                if (base + total > low) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int left = n[k] - base;
                        int at = 0;  // the lane's sequence: the first whose running sum is above left
#pragma unroll 1
                        for (int o = 16; o > 0; o >>= 1)
                            if (__shfl_sync(0xffffffffu, incl, at + o - 1) <= left) at += o;
                        const int before = __shfl_sync(0xffffffffu, incl, max(at - 1, 0));
                        if (left >= 0 && left < total) q[k] = (b1 + at) * p.T + left - (at ? before : 0);
                    }
                }
                base += total;
            }
        }
    }
    // items of a segment with that many query tokens
    __device__ int items(int tokens, int len) const {
        const int mt = (tokens * p.G + 2 * kTileRows - 1) / (2 * kTileRows);
        const int ns = len == 0 ? 1 : (len + p.chunk - 1) / p.chunk;
        return mt * ns * p.Hkv;
    }
};

__device__ __forceinline__ void rows_flag(int *status, int bit) {
    if (status) atomicOr(status, bit);
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, bool live) {
    const int n = live ? 16 : 0;  // 0: zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// n / G for n < G + 256, by the factor ceil(2^32 / G) (0: G = 1).  Exact while
// n G < 2^32, and G is at most 2^15.
__device__ __forceinline__ int small_div(int n, uint32_t magic) {
    return magic ? (int)__umulhi((uint32_t)n, magic) : n;
}

// RowsItem::v_unit of a chunk, by a whole warp: the scales of its pages.
__device__ __forceinline__ float scale_unit(const RowsParams &p, const RowsItem &it, int lane) {
    const int pages = (it.ntok + it.tok0 % p.page_size + p.page_size - 1) / p.page_size;
    const int *table = p.block_table + (size_t)it.seg * p.max_blocks + it.tok0 / p.page_size;
    float lo = INFINITY, hi = 0.f;
    bool fine = true;
    for (int k0 = lane; k0 < pages; k0 += 8 * 32) {
        int pg[8];
        float s[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) pg[u] = k0 + 32 * u < pages ? __ldcg(table + k0 + 32 * u) : -1;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            s[u] = pg[u] >= 0 && pg[u] < p.num_pages ? __ldcg(p.v_scale + (size_t)pg[u] * p.Hkv + it.kvh) : -1.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (pg[u] < 0 || pg[u] >= p.num_pages) continue;  // not loaded either
            fine = fine && s[u] > 0.f;                        // no NaN
            lo = fminf(lo, s[u]);
            hi = fmaxf(hi, s[u]);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    fine = __all_sync(0xffffffffu, fine) && lo > 1e-30f && hi < 1e30f && hi <= kScaleRange * lo;
    // the power of two at or above hi
    return fine ? __uint_as_float((__float_as_uint(hi) + 0x7fffffu) & 0xff800000u) : 0.f;
}

// Four neighbouring outputs, rounded to nearest even.
template <bool BF16>
__device__ __forceinline__ void put4(void *out, size_t at, float a, float b, float c, float d) {
    *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(out) + at) =
        BF16 ? make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d)) : make_uint2(pack_f16x2(a, b), pack_f16x2(c, d));
}

// A whole warp's wait, for at most limit nanoseconds: the same answer in every
// lane.  The clock's read between two looks is as good as a pause: looks back to
// back, or without suspending, cost 4 x 2048 queries over 8192 states 5% to 9%.
__device__ __forceinline__ bool warp_wait(uint64_t &bar, uint32_t parity, uint64_t limit) {
    const uint32_t at = smem_u32(&bar);
    if (__all_sync(0xffffffffu, mbar_try_wait(at, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    bool late = false;
#pragma unroll 1
    while (!late) {
        if (__all_sync(0xffffffffu, mbar_try_wait(at, parity))) return true;
        late = __any_sync(0xffffffffu, global_timer_ns() - t0 > limit);
    }
    return false;
}

// The query warps' waits, which may take as long as an item: false once the limit
// has passed twice without a tile loaded in between.  (In every role's waits the
// look at it cost 2% to 6%, over E4M3 pools 25%: it is code between their steps.
// Theirs take a tile's time or two.)
template <typename Control>
__device__ __forceinline__ bool warp_wait_item(Control &c, uint64_t &bar, uint32_t parity, uint64_t limit) {
    uint32_t seen = ~0u;
    while (!warp_wait(bar, parity, limit)) {
        uint32_t beat;
        asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(beat) : "r"(smem_u32(&c.beat)) : "memory");
        if (__all_sync(0xffffffffu, beat == seen)) return false;
        seen = beat;
    }
    return true;
}

// PARTS: bf16 pools, bf16 parts of a weight.  One, as wide as the output, rounds a
// weight to 8 bits; two (16 bits) cost a third product of the size of the first two.
template <int KV, int D, bool QBF16, int PARTS>
__global__ void __launch_bounds__(RowsShape<KV, D>::THREADS, 1)
    fd_rows_kernel(const __grid_constant__ RowsParams p, const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv) {
    using Sh = RowsShape<KV, D>;
    constexpr bool FP8 = Sh::FP8;
    constexpr bool B16 = KV == KV_BF16;    // products in bf16 (else f16)
    constexpr bool PAIR = FP8 || PARTS == 2;  // bf16 weights (E4M3: chunks of wide scales) as pairs
    static_assert(PARTS == 1 || B16, "parts of bf16 weights");
    constexpr bool QSCALE = FP8 && QBF16;  // query rows scaled into f16
    static_assert(FP8 || QBF16 == (KV == KV_BF16), "16-bit pools have q's type");
    constexpr int HALVES = Sh::HALVES, NST = Sh::STAGES;
    constexpr uint32_t TMEM_S = 0, TMEM_O = 256;  // columns: S (and P) of both tiles, then O
    extern __shared__ __align__(1024) uint8_t smem[];
    static_assert(sizeof(RowsControl<Sh>) <= Sh::CONTROL, "the control block's room");
    RowsControl<Sh> &c = *reinterpret_cast<RowsControl<Sh> *>(smem);
    const uint32_t q_base = smem_u32(smem) + Sh::CONTROL, ring = smem_u32(smem) + Sh::RING;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t limit = p.timeout_ns;

    if (smem_u32(smem) & 1023) {  // the swizzled tiles' alignment: the launch has no static shared memory
        rows_flag(p.status, FD_DEV_TIMEOUT);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&c.q_full[i]), 64);
            mbar_init(smem_u32(&c.q_empty[i]), 1);
            mbar_init(smem_u32(&c.s_full[i]), 1);
            mbar_init(smem_u32(&c.p_full[i]), 4);
            mbar_init(smem_u32(&c.pv_done[i]), 1);
        }
        for (int i = 0; i < kItemSlots; ++i) {
            mbar_init(smem_u32(&c.item_full[i]), 1);
            mbar_init(smem_u32(&c.item_empty[i]), 8 + 1 + 2 + (FP8 ? 4 : 0));  // all warps but the producer's
        }
        mbar_init(smem_u32(&c.rows_full), 64);
        mbar_init(smem_u32(&c.rows_empty), 8);
        mbar_init(smem_u32(&c.rows_read), 64);
        mbar_init(smem_u32(&c.join_full), 4);
        mbar_init(smem_u32(&c.join_empty), 4);
        c.held[0] = c.held[1] = 0;
        c.beat = 0;
        for (int i = 0; i < NST; ++i) {
            mbar_init(smem_u32(&c.kv_full[i]), FP8 ? 4 : 1);
            mbar_init(smem_u32(&c.kv_empty[i]), 1);
        }
        for (int i = 0; i < Sh::RAW_STAGES; ++i) {
            mbar_init(smem_u32(&c.raw_full[i]), 1);
            mbar_init(smem_u32(&c.raw_empty[i]), 4);
        }
        mbar_init(smem_u32(&c.drain), 1);
        fence_barrier_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(&c.tmem), 512);
        tmem_relinquish();
    }
    if (warp == 9 && lane == 0) {
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = c.tmem;
    // Only shared memory, tensor memory and parameters so far; what follows
    // reads what the preceding grid may still be writing.  Behind the pass over
    // the sequences' own tokens only that pass's results may: they are waited
    // for where they are joined (its launch waited for everything before it).
    // Reads before such a wait go to L2, as L1 may hold an earlier call's lines;
    // not so the E4M3 scales' small copies, which therefore wait here.
    if (FP8 || !p.own_out) grid_dependency_wait();

    // ---- Items of every segment, counted by all threads into the ring (not in
    // use yet): the producer warp keeps their sums over 32 runs of segments.
    const Segments seg{p};
    const int nseg = seg.count();
    int *scratch = reinterpret_cast<int *>(smem + Sh::CONTROL);  // offsets that rise, items, query tokens: nseg + 1 each
    int *s_off = scratch, *s_items = scratch + nseg + 1, *s_tokens = scratch + 2 * (nseg + 1);
    if (p.offsets) {
        // offsets made to rise within [0, seqs]: a running maximum, by one warp
        if (warp == 0) {
            int high = 0;
            bool bad = __ldcg(p.offsets) != 0;
            for (int s0 = 0; s0 <= nseg; s0 += 32) {
                const int s = s0 + lane;
                const int raw = s <= nseg ? seg.raw_offset(s) : 0;
                int v = min(max(raw, high), p.seqs);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int t = __shfl_up_sync(0xffffffffu, v, o);
                    if (lane >= o) v = max(v, t);
                }
                if (s <= nseg) {
                    s_off[s] = v;
                    bad |= v != raw;
                }
                high = __shfl_sync(0xffffffffu, v, 31);
            }
            if (__any_sync(0xffffffffu, bad) && lane == 0) rows_flag(p.status, FD_DEV_BAD_PAGE);
        }
    } else {
        for (int s = threadIdx.x; s <= nseg; s += Sh::THREADS) s_off[s] = s * p.beams;
    }
    __syncthreads();
    const bool by_warp = seg.by_warp(nseg, Sh::THREADS / 32, Sh::THREADS);
    if (by_warp) {
        bool bad = false;
        for (int s = warp; s < nseg; s += Sh::THREADS / 32) {
            const int n = seg.warp_tokens(s_off[s], s_off[s + 1], bad, lane);
            if (lane == 0) s_tokens[s] = n;
        }
        if (bad) rows_flag(p.status, FD_DEV_CAPACITY);
        __syncthreads();
    }
    for (int s = threadIdx.x; s < nseg; s += Sh::THREADS) {
        bool bad = false;
        if (!by_warp) s_tokens[s] = seg.tokens(s_off[s], s_off[s + 1], bad);
        s_items[s] = seg.items(s_tokens[s], seg.kv_len(s));
        if (s < p.kv_rows) {
            const int L = __ldcg(p.kv_lens + s);
            bad |= L < 0 || L > p.cap;
        }
        if (bad) rows_flag(p.status, FD_DEV_CAPACITY);
    }
    __syncthreads();
    // Run of segments of each lane of the producer warp: [lane * per, ...).
    const int per = (nseg + 31) >> 5;
    int run_items = 0, run_before = 0, run_off = 0, run_end = 0, run_len = 0, run_tokens = 0, run_seg = 0, total = 0;
    if (warp == 9) {
        const int s0 = min(lane * per, nseg), s1 = min(s0 + per, nseg);
        for (int s = s0; s < s1; ++s) run_items += s_items[s];
        run_off = s_off[s0];
        run_end = s_off[s1];
        if (per == 1 && s1 > s0) {
            run_len = seg.kv_len(s0);
            run_tokens = s_tokens[s0];
        }
        if (per == 1) {
            // longest KV rows first, so that the short ones fill the end
            int rank = 0, src = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int len = __shfl_sync(0xffffffffu, run_len, i);
                rank += len > run_len || (len == run_len && i < lane);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (__shfl_sync(0xffffffffu, rank, i) == lane) src = i;
            run_seg = src;
            run_items = __shfl_sync(0xffffffffu, run_items, src);
            run_off = __shfl_sync(0xffffffffu, run_off, src);
            run_end = __shfl_sync(0xffffffffu, run_end, src);
            run_len = __shfl_sync(0xffffffffu, run_len, src);
            run_tokens = __shfl_sync(0xffffffffu, run_tokens, src);
        }
        int incl = run_items;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        run_before = incl - run_items;
        total = __shfl_sync(0xffffffffu, incl, 31);
    }
    fence_proxy_async_shared();
    __syncthreads();  // the ring and Q tiles are free now

    if (warp >= 8) {  // (the roles below are not indented for it)
    regs_down<Sh::REGS_OTHER>();
    if (warp == 9) {
        // ============================================================ producer
        const int bsh = __ffs(p.boxr) - 1;  // boxr is a power of two
        const int BPT = kTileTokens >> bsh;
        const uint64_t policy = l2_policy_evict_normal();  // other items of the KV head read the tiles too
        uint32_t e = 0;        // ring entries issued
        int n_item = 0;        // items published
        bool ok = true;
        if (p.stall_ns) {      // test hook: late loads
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < p.stall_ns) __nanosleep(1000);
        }
        // The item of a claim (seg -1: there are no more), and a page id for every
        // lane of its first 64 boxes.
        RowsItem nx;
        int npg0 = -1, npg1 = -1;
        auto page_of = [&](const RowsItem &it, int k) -> int {
            const int at = k << bsh;
            return at < it.ntok ? __ldcg(p.block_table + (size_t)it.seg * p.max_blocks + (it.tok0 + at) / p.page_size) : -1;
        };
        auto look_up = [&](int claim) {
            RowsItem it;
            it.seg = -1;
            it.ntok = 0;
            it.v_unit = 0.f;
            if (claim < total) {
                // the lane's run that holds it, then the segment within the run
                const unsigned has = __ballot_sync(0xffffffffu, run_before <= claim && claim < run_before + run_items);
                const int src = __ffs(has) - 1;
                // its items before this one (one segment a run: of all runs)
                int left = per == 1 ? claim : claim - __shfl_sync(0xffffffffu, run_before, src);
                int high = __shfl_sync(0xffffffffu, run_off, src);
                const int s_end = per == 1 ? nseg : min((src + 1) * per, nseg);
                for (int s0 = per == 1 ? 0 : src * per;; s0 += 32) {
                    const int s = s0 + lane;
                    int first = 0, end = 0;
                    if (per == 1) {  // a lane's run is one segment: its first and last place are here
                        first = run_off;
                        end = run_end;
                    } else if (p.offsets) {
                        int v = s < s_end ? min(max(seg.raw_offset(s + 1), high), p.seqs) : 0;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int t = __shfl_up_sync(0xffffffffu, v, o);
                            if (lane >= o) v = max(v, t);
                        }
                        end = v;
                        const int before = __shfl_up_sync(0xffffffffu, v, 1);
                        first = lane == 0 ? high : before;
                        high = __shfl_sync(0xffffffffu, v, 31);
                    } else {
                        first = s * p.beams;
                        end = first + p.beams;
                    }
                    const int len = per == 1 ? run_len : (s < s_end ? seg.kv_len(s) : 0);
                    int ntokens = run_tokens;
                    [[maybe_unused]] bool bad = false;  // said at the start
                    if (per > 1 && seg.by_warp(min(32, s_end - s0), 1, 32)) {
                        const int f0 = __shfl_sync(0xffffffffu, first, 0);
                        for (int x = 0; x < 32 && s0 + x < s_end; ++x) {
                            if (lane == 0) atomicAdd(&c.beat, 1u);
                            const int t = seg.warp_tokens(f0 + x * p.beams, f0 + (x + 1) * p.beams, bad, lane);
                            if (lane == x) ntokens = t;
                        }
                        if (s >= s_end) ntokens = 0;
                    } else if (per > 1) {
                        ntokens = s < s_end ? seg.tokens(first, end, bad) : 0;
                    }
                    const int n = per == 1 ? run_items : (s < s_end ? seg.items(ntokens, len) : 0);
                    int incl = n;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int t = __shfl_up_sync(0xffffffffu, incl, o);
                        if (lane >= o) incl += t;
                    }
                    const unsigned in = __ballot_sync(0xffffffffu, left < incl);
                    if (!in && s0 + 32 < s_end) {
                        left -= __shfl_sync(0xffffffffu, incl, 31);
                        continue;
                    }
                    const int ln = in ? __ffs(in) - 1 : 31;
                    // tile of rows fastest: the items that read the same K and V
                    // run at the same time and meet them in L2
                    const int L = __shfl_sync(0xffffffffu, len, ln);
                    const int rows = __shfl_sync(0xffffffffu, ntokens, ln) * p.G;
                    const int mt = max(1, (rows + 2 * kTileRows - 1) / (2 * kTileRows));
                    int k = left - __shfl_sync(0xffffffffu, incl - n, ln);
                    it.seg = per == 1 ? __shfl_sync(0xffffffffu, run_seg, ln) : s0 + ln;
                    it.first = __shfl_sync(0xffffffffu, first, ln);
                    it.row0 = (k % mt) * 2 * kTileRows;
                    k /= mt;
                    it.kvh = k % p.Hkv;
                    it.split = k / p.Hkv;
                    it.nsplit = L == 0 ? 1 : (L + p.chunk - 1) / p.chunk;
                    it.nrows = min(2 * kTileRows, rows - it.row0);
                    it.n0 = it.row0 / p.G;
                    it.g0 = it.row0 - it.n0 * p.G;
                    it.tok0 = it.split * p.chunk;
                    it.ntok = min(L - it.tok0, p.chunk);
                    break;
                }
            }
            if (it.seg >= 0) {
                npg0 = page_of(it, lane);
                npg1 = page_of(it, 32 + lane);
            }
            if constexpr (FP8) {
                if (it.ntok > 0) it.v_unit = scale_unit(p, it, lane);
            }
            nx = it;
        };
        look_up((int)blockIdx.x);
        while (true) {
            const int slot = n_item % kItemSlots;
            if (!warp_wait(c.item_empty[slot], ((n_item / kItemSlots) & 1) ^ 1, limit)) {
                ok = false;
                break;
            }
            const RowsItem it = nx;
            if (lane == 0) {
                c.item[slot] = it;
                mbar_arrive(smem_u32(&c.item_full[slot]));
            }
            __syncwarp();
            ++n_item;
            if (it.seg < 0) break;
            int next = 0;
            if (lane == 0) next = atomicAdd(p.counters, 1);
            // K and V tiles in turn, page ids 32 boxes ahead; the next item is
            // looked up two tiles before the end, while the ring is full.
            const int nbox = (it.ntok + p.boxr - 1) >> bsh;
            const int ahead = max(0, (it.ntok - 1) / kTileTokens - 1) * BPT;
            int pg_cur = npg0, pg_nxt = npg1, batch = 0;
            if (it.ntok == 0) look_up((int)gridDim.x + __shfl_sync(0xffffffffu, next, 0));
            for (int k0 = 0; k0 < nbox && ok; k0 += BPT) {
                if (lane == 0) atomicAdd(&c.beat, 1u);
                if (k0 == ahead) look_up((int)gridDim.x + __shfl_sync(0xffffffffu, next, 0));
                if (k0 >= (batch + 1) * 32) {
                    ++batch;
                    pg_cur = pg_nxt;
                    pg_nxt = page_of(it, (batch + 1) * 32 + lane);
                }
                const int pg = __shfl_sync(0xffffffffu, pg_cur, (k0 + (lane & (BPT - 1))) & 31);
                const bool live = lane < BPT && k0 + lane < nbox;
                const bool good = live && pg >= 0 && pg < p.num_pages;
                if (live && !good) rows_flag(p.status, FD_DEV_BAD_PAGE);
                const unsigned mask = __ballot_sync(0xffffffffu, good);
                const int at = (it.tok0 + ((k0 + lane) << bsh)) % p.page_size;
                // the page of this lane's group of 16 tokens, for the scales
                const int box = (lane & 7) >> (bsh - 4);
                [[maybe_unused]] const int pg16 = __shfl_sync(0xffffffffu, good ? pg : -1, box);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const int st = e % Sh::LOADS;
                    uint64_t &full = FP8 ? c.raw_full[st] : c.kv_full[st];
                    if (!warp_wait(FP8 ? c.raw_empty[st] : c.kv_empty[st], ((e / Sh::LOADS) & 1) ^ 1, limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = smem_u32(&full);
                    if constexpr (FP8) {
                        // both scales of every group with V's codes; the stage's
                        // barrier also waits for them
                        if (kv == 1 && lane < 8) {
                            float *ks = &c.raw_scale[st][lane], *vs = ks + 8;
                            if (pg16 >= 0) {
                                cp_async_4(smem_u32(ks), p.k_scale + (size_t)pg16 * p.Hkv + it.kvh);
                                cp_async_4(smem_u32(vs), p.v_scale + (size_t)pg16 * p.Hkv + it.kvh);
                                cp_async_mbar_arrive(fb);
                            } else {
                                *ks = *vs = 1.f;
                            }
                        }
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive_expect_tx(fb, (uint32_t)__popc(mask) * p.boxr * D * (FP8 ? 1 : 2));
                    __syncwarp();
                    if (good) {
                        if constexpr (FP8) {
                            const uint32_t dst = smem_u32(smem) + Sh::RAW_RING + st * Sh::RAW + (lane << bsh) * D;
                            tma_load_5d(dst, kv ? &tmv : &tmk, fb, 0, at, 0, it.kvh, pg, policy);
                        } else {
                            tma_load_4d(ring + st * Sh::TILE + (lane << bsh) * D * 2, kv ? &tmv : &tmk, fb, 0, 0, it.kvh * HALVES,
                                        pg * (p.page_size >> 3) + (at >> 3), policy);
                        }
                    }
                    ++e;
                }
            }
            if (!ok) break;
        }
        grid_launch_dependents();
        if (!ok && lane == 0) rows_flag(p.status, FD_DEV_TIMEOUT);
        // No copy may be in flight when the CTA ends: the latest entry of every stage.
        for (uint32_t k = 1; k <= Sh::LOADS && k <= e; ++k) {
            const uint32_t st = (e - k) % Sh::LOADS;
            if (!warp_wait(FP8 ? c.raw_full[st] : c.kv_full[st], ((e - k) / Sh::LOADS) & 1, limit) && lane == 0)
                rows_flag(p.status, FD_DEV_TIMEOUT);
        }
        // The last producer out resets the counters for the next launch.
        if (lane == 0 && atom_add_acq_rel_gpu(p.counters + 1, 1) == (int)gridDim.x - 1) {
            atomicExch(p.counters, 0);
            atomicExch(p.counters + 1, 0);
        }
    } else if (FP8 && warp >= 12) {
        if constexpr (FP8) {
            // ================================================ codes to values
            // A thread turns 16 codes of a row at a time into two 16-byte pieces.
            // Eight neighbouring lanes have four pieces of a 64-code half of one
            // row and of the other half of the next row (D = 64: of two rows):
            // their loads and stores meet no bank twice.
            const int t = threadIdx.x - 384;  // 0 .. 127
            constexpr int ROWS = D == 128 ? 16 : 32;  // rows a pass over the 128 threads
            const int pr = (t >> 2) & 1;              // row of the pair
            const int r0 = D == 128 ? (t >> 4) * 2 + pr : t >> 2;
            const int half = D == 128 ? ((t >> 3) & 1) ^ pr : 0, ch = t & 3;
            int n_item = 0;
            uint32_t rs = 0, rpar = 0, st = 0, par = 0;  // stages and parities of the next entry
            bool here = false;                           // both were ready at a look ahead
            bool ok = true;
            while (ok) {
                const int slot = n_item % kItemSlots;
                if (!(ok = warp_wait(c.item_full[slot], (n_item / kItemSlots) & 1, limit))) break;
                const int sg = c.item[slot].seg, ntok = c.item[slot].ntok;
                const bool wide = c.item[slot].v_unit == 0.f;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c.item_empty[slot]));
                ++n_item;
                if (sg < 0) break;
                const int entries = 2 * ((ntok + kTileTokens - 1) / kTileTokens);
                for (int x = 0; x < entries; ++x) {
                    const bool is_v = x & 1;
                    const int nvalid = ntok - (x >> 1) * kTileTokens;
                    if (!__all_sync(0xffffffffu, here)) {
                        if (!(ok = warp_wait(c.raw_full[rs], rpar, limit))) break;
                        if (!(ok = warp_wait(c.kv_empty[st], par ^ 1, limit))) break;
                    }
                    const uint8_t *src = smem + Sh::RAW_RING + rs * Sh::RAW + r0 * D + half * 64 + ch * 16;
                    uint8_t *dst = smem + Sh::RING + st * Sh::TILE + (r0 >> 3) * Sh::GROUP + half * 1024 + (r0 & 7) * 128;
                    // r & 7 is the same in every pass (ROWS is a multiple of 8)
                    const int c0 = ((2 * ch) ^ (r0 & 7)) << 4, c1 = ((2 * ch + 1) ^ (r0 & 7)) << 4;
                    auto convert = [&](auto to_bf16) {
                        constexpr bool BF16 = decltype(to_bf16)::value;
#pragma unroll
                        for (int r = 0; r < kTileTokens / ROWS; ++r) {
                            const uint4 w = *reinterpret_cast<const uint4 *>(src + r * ROWS * D);
                            const uint32_t in[4] = {w.x, w.y, w.z, w.w};
                            uint32_t o[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                o[k] = e4m3x2_to_f16x2((uint16_t)(in[k >> 1] >> (16 * (k & 1))));
                                if constexpr (BF16) {
                                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&o[k]));
                                    o[k] = pack_bf16x2(f.x, f.y);
                                }
                            }
                            uint8_t *row = dst + r * (ROWS / 8) * Sh::GROUP;
                            *reinterpret_cast<uint4 *>(row + c0) = make_uint4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<uint4 *>(row + c1) = make_uint4(o[4], o[5], o[6], o[7]);
                        }
                    };
                    if (is_v && wide)
                        convert(std::true_type());
                    else
                        convert(std::false_type());
                    if (is_v && nvalid < kTileTokens) {
                        // V behind the last token: zeros, whatever the codes were
#pragma unroll 1
                        for (int r = 0; r < kTileTokens / ROWS; ++r)
                            if (r0 + r * ROWS >= nvalid) {
                                uint8_t *row = dst + r * (ROWS / 8) * Sh::GROUP;
                                *reinterpret_cast<uint4 *>(row + c0) = make_uint4(0, 0, 0, 0);
                                *reinterpret_cast<uint4 *>(row + c1) = make_uint4(0, 0, 0, 0);
                            }
                    }
                    if (is_v && t < 16) c.scale[st][t] = c.raw_scale[rs][t];
                    const uint32_t raw_done = smem_u32(&c.raw_empty[rs]), kv_done = smem_u32(&c.kv_full[st]);
                    if (++rs == Sh::RAW_STAGES) {
                        rs = 0;
                        rpar ^= 1;
                    }
                    if (++st == NST) {
                        st = 0;
                        par ^= 1;
                    }
                    here = mbar_test_wait(smem_u32(&c.raw_full[rs]), rpar) && mbar_test_wait(smem_u32(&c.kv_empty[st]), par ^ 1);
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(kv_done);
                        mbar_arrive(raw_done);
                    }
                }
            }
            if (!ok && lane == 0) rows_flag(p.status, FD_DEV_TIMEOUT);
        }
    } else if (warp >= 10) {
        // ========================================================= query rows
        const int t = threadIdx.x - 320;  // 0 .. 63
        int n_item = 0;
        uint32_t n_q[2] = {0, 0};         // tiles loaded
        while (true) {
            const int slot = n_item % kItemSlots;
            if (!warp_wait_item(c, c.item_full[slot], (n_item / kItemSlots) & 1, limit)) {
                rows_flag(p.status, FD_DEV_TIMEOUT);
                break;
            }
            const RowsItem it = c.item[slot];
            if (it.seg < 0) break;
            if (!warp_wait_item(c, c.rows_empty, (n_item & 1) ^ 1, limit)) {
                rows_flag(p.status, FD_DEV_TIMEOUT);
                break;
            }
            int *tok = c.tok;
            if (p.q_lens && p.beams > 1) {
                int n[4], q4[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int r = t + 64 * u;
                    n[u] = r < it.nrows ? it.n0 + small_div(it.g0 + r, p.g_magic) : -1;  // token of the segment
                    q4[u] = -1;
                }
                seg.find(it.first, it.first + p.beams, n, q4, lane, &c.beat);
#pragma unroll
                for (int u = 0; u < 4; ++u) tok[t + 64 * u] = q4[u];
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int r = t + 64 * u;
                    int q = -1;
                    if (r < it.nrows) {
                        const int n = it.n0 + small_div(it.g0 + r, p.g_magic);
                        // place of its sequence in the segment (counts of queries: it has one)
                        const int k = p.q_lens ? 0 : p.T == 1 ? n : n / p.T, i = it.first + k;
                        const int b = p.members ? __ldcg(p.members + i) : i;
                        if (b >= 0 && b < p.seqs)
                            q = b * p.T + (n - k * p.T);
                        else
                            rows_flag(p.status, FD_DEV_BAD_PAGE);
                    }
                    tok[r] = q;
                }
            }
            // what the loaders need of each other's rows; the softmax warps get them
            // now, or with the rows' factors
            mbar_arrive(smem_u32(QSCALE ? &c.rows_read : &c.rows_full));
            bool ok = warp_wait(QSCALE ? c.rows_read : c.rows_full, n_item & 1, limit);
            const int tiles = it.nrows > kTileRows ? 2 : 1;
            for (int i = 0; i < tiles && ok; ++i) {
                ok = warp_wait_item(c, c.q_empty[i], (n_q[i] & 1) ^ 1, limit);
                if (ok && it.ntok > 0) {
                    constexpr int CH = D / 8;  // 16-byte pieces of a row
                    const int ch = t % CH;
                    const uint32_t dst = q_base + i * Sh::TILE + (ch / 8) * Sh::SPAN;
                    const uint16_t *src = reinterpret_cast<const uint16_t *>(p.q) + (size_t)it.kvh * p.G * D + ch * 8;
                    if constexpr (QSCALE) {
#pragma unroll 1
                        for (int r0 = t / CH; r0 < kTileRows; r0 += 8 * (64 / CH)) {
                            uint4 w[8];
                            int q[8];
#pragma unroll
                            for (int u = 0; u < 8; ++u) {
                                const int row = i * kTileRows + r0 + u * (64 / CH);
                                q[u] = tok[row];
                                const int g = it.g0 + row - small_div(it.g0 + row, p.g_magic) * p.G;
                                w[u] = q[u] >= 0 ? __ldcg(reinterpret_cast<const uint4 *>(src + (size_t)q[u] * p.q_stride + g * D))
                                                 : make_uint4(0, 0, 0, 0);
                            }
#pragma unroll
                            for (int u = 0; u < 8; ++u) {
                                const int r = r0 + u * (64 / CH);
                                uint32_t in[4] = {w[u].x, w[u].y, w[u].z, w[u].w}, o[4];
                                // exponent of the row's largest element, as a bf16 pattern
                                uint32_t top = 0;
#pragma unroll
                                for (int k = 0; k < 4; ++k) top = max(top, max(in[k] & 0x7fffu, (in[k] >> 16) & 0x7fffu));
#pragma unroll
                                for (int o2 = CH / 2; o2 > 0; o2 >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o2));
                                const int f = top ? 127 + max(-126, min(126, 141 - (int)(top >> 7))) : 127;
                                const float up = __uint_as_float((uint32_t)f << 23);
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    o[k] = pack_f16x2(__uint_as_float(in[k] << 16) * up, __uint_as_float(in[k] & 0xffff0000u) * up);
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + r * 128 + (((ch & 7) ^ (r & 7)) << 4)),
                                             "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                                             : "memory");
                                if (ch == 0 && q[u] >= 0) tok[i * kTileRows + r] = q[u] | (f << 22);
                            }
                        }
                    } else
#pragma unroll 8
                    for (int r = t / CH; r < kTileRows; r += 64 / CH) {
                        const int row = i * kTileRows + r, q = tok[row];
                        const int g = it.g0 + row - small_div(it.g0 + row, p.g_magic) * p.G;
                        cp_async_16(dst + r * 128 + (((ch & 7) ^ (r & 7)) << 4),
                                    src + (size_t)max(q, 0) * p.q_stride + g * D, q >= 0);
                    }
                }
                cp_async_commit();
            }
            // hand the tiles over as they land
            for (int i = 0; i < tiles && ok; ++i) {
                if (i + 1 < tiles)
                    cp_async_wait<1>();
                else
                    cp_async_wait<0>();
                fence_proxy_async_shared();
                mbar_arrive(smem_u32(&c.q_full[i]));
                ++n_q[i];
            }
            if (QSCALE) mbar_arrive(smem_u32(&c.rows_full));
            if (!ok) rows_flag(p.status, FD_DEV_TIMEOUT);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&c.item_empty[slot]));
            ++n_item;
            if (!ok) break;
        }
        cp_async_wait<0>();
    } else if (warp == 8) {
        // ============================================================ products
        // The whole warp goes round, so that descriptors and addresses stay in
        // uniform registers; one lane issues.
        constexpr uint32_t idesc_qk = mma_idesc(kTileRows, kTileTokens, B16, false);
        constexpr uint32_t idesc_f16 = mma_idesc(kTileRows, D, false, true), idesc_bf16 = mma_idesc(kTileRows, D, true, true);
        uint32_t idesc_pv = B16 ? idesc_bf16 : idesc_f16;
        const bool leader = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t q_desc = smem_desc(q_base, 16, 1024), k_desc = smem_desc(ring, 16, Sh::GROUP);
        const uint64_t v_desc = smem_desc(ring, 1024, Sh::GROUP);
        int n_item = 0;
        uint32_t st = 0, par = 0;  // ring stage and parity of the next entry
        uint32_t n_q0 = 0, n_q1 = 0, n_p0 = 0, n_p1 = 0;
        bool ok = true;
        auto next = [&]() {
            if (++st == NST) {
                st = 0;
                par ^= 1;
            }
        };
        auto qk = [&](int i, int tile, uint32_t stage) {  // scores i of that query tile
            const uint64_t a0 = q_desc + (uint64_t)(tile * (Sh::TILE >> 4)), b0 = k_desc + (uint64_t)(stage * (Sh::TILE >> 4));
            if (leader) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    mma_ss(tm + TMEM_S + i * 128, a0 + (((k / 4) * Sh::SPAN + (k % 4) * 32) >> 4),
                           b0 + (((k / 4) * 1024 + (k % 4) * 32) >> 4), idesc_qk, k > 0);
                }
                mma_commit(smem_u32(&c.s_full[i]));
            }
        };
        // O += P V of one tile.  All of the weights at once: handing three quarters
        // over while the rest is worked out keeps the products of the other row
        // tile waiting behind the last quarter (4 x 2048 queries over 8192 states
        // 737 -> 792 us).
        auto output = [&](int i, uint32_t stage, int steps, bool more, uint32_t phase) {
            if (!warp_wait(c.p_full[i], phase & 1, limit)) return false;
            tmem_fence_after();
            const uint64_t b0 = v_desc + (uint64_t)(stage * (Sh::TILE >> 4));
            const uint32_t d = tm + TMEM_O + i * 128, a0 = tm + TMEM_S + i * 128;
            if (leader) {
                if (steps == kTileTokens / 16) {
#pragma unroll
                    for (int k = 0; k < kTileTokens / 16; ++k)
                        mma_ts(d, a0 + k * 8, b0 + k * (2 * Sh::GROUP >> 4), idesc_pv, k > 0 || more);
                } else {
                    for (int k = 0; k < steps; ++k) mma_ts(d, a0 + k * 8, b0 + k * (2 * Sh::GROUP >> 4), idesc_pv, k > 0 || more);
                }
                if (PARTS == 2 && steps == kTileTokens / 16) {
#pragma unroll
                    for (int k = 0; k < kTileTokens / 16; ++k)
                        mma_ts(d, a0 + 64 + k * 8, b0 + k * (2 * Sh::GROUP >> 4), idesc_pv, true);
                } else if (PAIR && idesc_pv == idesc_bf16)  // the weights' low parts
                    for (int k = 0; k < steps; ++k) mma_ts(d, a0 + 64 + k * 8, b0 + k * (2 * Sh::GROUP >> 4), idesc_pv, true);
                mma_commit(smem_u32(&c.pv_done[i]));
            }
            return true;
        };
        auto release = [&](uint64_t &bar) {
            if (leader) mma_commit(smem_u32(&bar));
        };
        while (ok) {
            const int slot = n_item % kItemSlots;
            if (!(ok = warp_wait(c.item_full[slot], (n_item / kItemSlots) & 1, limit))) break;
            const int sg = __shfl_sync(0xffffffffu, c.item[slot].seg, 0);
            const int nrows = __shfl_sync(0xffffffffu, c.item[slot].nrows, 0);
            const int ntok = __shfl_sync(0xffffffffu, c.item[slot].ntok, 0);
            if constexpr (FP8) idesc_pv = __shfl_sync(0xffffffffu, c.item[slot].v_unit, 0) == 0.f ? idesc_bf16 : idesc_f16;
            if (lane == 0) mbar_arrive(smem_u32(&c.item_empty[slot]));
            ++n_item;
            if (sg < 0) break;
            const bool two = nrows > kTileRows;
            const int nt = (ntok + kTileTokens - 1) / kTileTokens;
            if (!(ok = warp_wait(c.q_full[0], n_q0++ & 1, limit))) break;
            if (two && !(ok = warp_wait(c.q_full[1], n_q1++ & 1, limit))) break;
            if (nt == 0) {
                if (lane == 0) {
                    mbar_arrive(smem_u32(&c.q_empty[0]));
                    if (two) mbar_arrive(smem_u32(&c.q_empty[1]));
                }
                __syncwarp();
                continue;
            }
            if (!(ok = warp_wait(c.kv_full[st], par, limit))) break;
            tmem_fence_after();
            if (two) {
                qk(0, 0, st);
                qk(1, 1, st);
                if (nt > 1)  // the last K tile's stage is released by the softmax warps
                    release(c.kv_empty[st]);
                else {
                    release(c.q_empty[0]);
                    release(c.q_empty[1]);
                }
                next();
                // V of a tile and K of the next one: looked for as the tile before
                // them is issued, so that the look costs nothing.
                bool v_here = false, k_here = false;
                for (int j = 0; j < nt; ++j) {
                    const uint32_t sv = st;
                    const bool more = j + 1 < nt;
                    if (!__all_sync(0xffffffffu, v_here) && !(ok = warp_wait(c.kv_full[sv], par, limit))) break;
                    next();
                    const uint32_t sk = st;
                    if (more) {
                        if (!__all_sync(0xffffffffu, k_here) && !(ok = warp_wait(c.kv_full[sk], par, limit))) break;
                        next();
                    }
                    const int steps = more ? kTileTokens / 16 : (ntok - j * kTileTokens + 15) / 16;
                    if (!(ok = output(0, sv, steps, j > 0, n_p0++))) break;
                    if (more) qk(0, 0, sk);
                    v_here = k_here = false;
                    if (more) {
                        v_here = mbar_test_wait(smem_u32(&c.kv_full[st]), par);
                        const uint32_t s2 = st + 1 == NST ? 0 : st + 1;
                        if (j + 2 < nt) k_here = mbar_test_wait(smem_u32(&c.kv_full[s2]), s2 ? par : par ^ 1);
                    }
                    if (!(ok = output(1, sv, steps, j > 0, n_p1++))) break;
                    release(c.kv_empty[sv]);
                    if (more) {
                        qk(1, 1, sk);
                        if (j + 2 < nt)
                            release(c.kv_empty[sk]);
                        else {
                            release(c.q_empty[0]);
                            release(c.q_empty[1]);
                        }
                    }
                }
            } else {
                // One row tile: its KV tiles in turn to the two halves of the
                // softmax, two of them under way at a time.
                qk(0, 0, st);
                if (nt > 1)
                    release(c.kv_empty[st]);
                else
                    release(c.q_empty[0]);
                next();
                uint32_t sv = st, pv_par = par;  // V of tile 0
                if (nt > 1) {
                    next();                      // K of tile 1
                    if (!(ok = warp_wait(c.kv_full[st], par, limit))) break;
                    tmem_fence_after();
                    qk(1, 0, st);
                    if (nt > 2)
                        release(c.kv_empty[st]);
                    else
                        release(c.q_empty[0]);
                }
                next();
                for (int j = 0; j < nt; ++j) {
                    const int steps = min(kTileTokens / 16, (ntok - j * kTileTokens + 15) / 16), i = j & 1;
                    if (!(ok = warp_wait(c.kv_full[sv], pv_par, limit))) break;
                    if (!(ok = output(i, sv, steps, j > 1, i ? n_p1++ : n_p0++))) break;
                    release(c.kv_empty[sv]);
                    // entries from here: V of tile j + 1 at st, K of tile j + 2 behind it
                    sv = st;
                    pv_par = par;
                    if (j + 2 < nt) {
                        next();
                        if (!(ok = warp_wait(c.kv_full[st], par, limit))) break;
                        tmem_fence_after();
                        qk(i, 0, st);
                        if (j + 3 < nt)
                            release(c.kv_empty[st]);
                        else
                            release(c.q_empty[0]);
                    }
                    if (j + 1 < nt) next();
                }
            }
        }
        if (!ok && lane == 0) rows_flag(p.status, FD_DEV_TIMEOUT);
        // every product is complete before shared and tensor memory go
        release(c.drain);
        if (!warp_wait(c.drain, 0, limit) && lane == 0) rows_flag(p.status, FD_DEV_TIMEOUT);
    }
    } else {
        // ============================================================= softmax
        regs_up<Sh::REGS_SOFTMAX>();
        const int i = warp >> 2;                           // tile
        const int r = (warp & 3) * 32 + lane;              // row of the tile
        const uint32_t lanes = (uint32_t)(warp & 3) << 21; // first tensor-memory lane of the warp << 16
        const uint32_t ts = tmem + lanes + TMEM_S + i * 128, to = tmem + lanes + TMEM_O + i * 128;
        const float sc = p.scale_log2;
        int n_item = 0;
        uint32_t e = 0, n_s = 0, n_join = 0;  // ring entries, score tiles and joined items so far
        bool handed = false;  // tile 1's state of a joined item may still be read
        while (true) {
            const int slot = n_item % kItemSlots;
            if (!warp_wait(c.item_full[slot], (n_item / kItemSlots) & 1, limit)) {
                rows_flag(p.status, FD_DEV_TIMEOUT);
                break;
            }
            const RowsItem it = c.item[slot];
            if (it.seg < 0) break;
            const int nt = (it.ntok + kTileTokens - 1) / kTileTokens;
            bool ok = warp_wait(c.rows_full, n_item & 1, limit);
            // With one row tile both halves have its rows, and every other KV tile.
            const bool solo = it.nrows <= kTileRows;
            const int row0 = solo ? 0 : i * kTileRows, step = solo ? 2 : 1, j0 = solo ? i : 0;
            int q = c.tok[row0 + r];  // this thread's row
            float row_sc = sc;
            if constexpr (QSCALE) {
                if (q >= 0) {
                    row_sc = sc * __uint_as_float((uint32_t)(254 - (q >> 22)) << 23);  // the row's factor undone
                    q &= (1 << 22) - 1;
                }
            }
            const bool wide = FP8 && it.v_unit == 0.f;
            const float v_inv = wide || !FP8 ? 1.f : 1.f / it.v_unit;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&c.rows_empty));
            const bool warp_live = row0 + (warp & 3) * 32 < it.nrows;
            const bool join = solo && nt > 1;
            float ref = -INFINITY, l = 0.f;
            if (ok) {
                for (int j = j0; j < nt; j += step, ++n_s) {
                    if (!warp_wait(c.s_full[i], n_s & 1, limit)) {
                        ok = false;
                        break;
                    }
                    const int nvalid = min(kTileTokens, it.ntok - j * kTileTokens);
                    [[maybe_unused]] const uint32_t es = (e + 2 * j + 1) % NST;  // V's stage
                    if constexpr (FP8) {  // its scales
                        if (!(ok = warp_wait(c.kv_full[es], ((e + 2 * j + 1) / NST) & 1, limit))) break;
                    } else if ((solo || i == 0) && (nvalid & 15)) {
                        // V rows behind the last token, up to the product's step of
                        // 16: their weight is 0, but they may hold infinities or NaN.
                        const uint32_t ev = e + 2 * j + 1;
                        if (!warp_wait(c.kv_full[ev % NST], (ev / NST) & 1, limit)) {
                            ok = false;
                            break;
                        }
                        const int z0 = nvalid, z1 = (nvalid + 15) & ~15;
                        uint8_t *vt = smem + Sh::RING + (ev % NST) * Sh::TILE;
                        for (int x = r; x < (z1 - z0) * HALVES * 8; x += 128) {
                            const int z = z0 + x / (HALVES * 8), y = x % (HALVES * 8);
                            *reinterpret_cast<uint4 *>(vt + (z >> 3) * Sh::GROUP + (y >> 3) * 1024 + (z & 7) * 128 + (y & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_shared();
                    }
                    if (handed) {  // O of the joined item before this one has been read
                        if (!(ok = warp_wait(c.join_empty, (n_join - 1) & 1, limit))) break;
                        handed = false;
                    }
                    if (warp_live) {
                        tmem_fence_after();
                        uint32_t s[128];
#pragma unroll
                        for (int k = 0; k < 4; ++k) tmem_ld32(ts + 32 * k, s + 32 * k);
                        tmem_wait_ld();
                        tmem_loaded<128>(s);
                        // E4M3: a group's scale goes into its factor; where a factor
                        // is not positive (a scale that is not, or a product that
                        // underflows) into the scores, before hidden ones are set
                        // to -inf (the highest score would be the lowest product,
                        // or -inf times 0).
                        [[maybe_unused]] float fs[8], vs[8];
                        if constexpr (FP8) {
                            const float4 *cs = reinterpret_cast<const float4 *>(c.scale[es]);
                            const float4 k0 = cs[0], k1 = cs[1], v0 = cs[2], v1 = cs[3];
                            fs[0] = k0.x; fs[1] = k0.y; fs[2] = k0.z; fs[3] = k0.w;
                            fs[4] = k1.x; fs[5] = k1.y; fs[6] = k1.z; fs[7] = k1.w;
                            vs[0] = v0.x; vs[1] = v0.y; vs[2] = v0.z; vs[3] = v0.w;
                            vs[4] = v1.x; vs[5] = v1.y; vs[6] = v1.z; vs[7] = v1.w;
                            bool odd = false;
#pragma unroll
                            for (int k = 0; k < 8; ++k) odd |= !(row_sc * fs[k] > 0.f);
                            if (odd) {
#pragma unroll
                                for (int k = 0; k < 128; ++k) s[k] = __float_as_uint(__uint_as_float(s[k]) * fs[k >> 4]);
                            }
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                fs[k] = odd ? row_sc : row_sc * fs[k];
                                vs[k] *= v_inv;
                            }
                        }
                        if (nvalid < kTileTokens) {
#pragma unroll
                            for (int k = 0; k < 128; ++k)
                                if (k >= nvalid) s[k] = 0xff800000u;  // -inf
                        }
                        float top;
                        if constexpr (FP8) {
                            top = -INFINITY;
#pragma unroll
                            for (int k = 0; k < 128; k += 16) {
                                float m = fmaxf(__uint_as_float(s[k]), __uint_as_float(s[k + 1]));
#pragma unroll
                                for (int x = 2; x < 16; x += 2) m = max3(m, __uint_as_float(s[k + x]), __uint_as_float(s[k + x + 1]));
                                top = k < nvalid ? fmaxf(top, m * fs[k >> 4]) : top;
                            }
                        } else {
                            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                            for (int k = 0; k < 128; k += 2)
                                mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
                            top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
                        }
                        if (__any_sync(0xffffffffu, top > ref + kSlack)) {
                            const float now = fmaxf(ref, top);
                            const float a = now == -INFINITY ? 1.f : ex2(ref - now);
                            ref = now;
                            l *= a;
                            if (j > j0) {
                                // O so far, once the product before this one is complete
                                if (!warp_wait(c.pv_done[i], (n_s - 1) & 1, limit)) {
                                    ok = false;
                                } else {
                                    tmem_fence_after();
#pragma unroll 1
                                    for (int k = 0; k < D; k += 8) {
                                        uint32_t o[8];
                                        tmem_ld8(to + k, o);
                                        tmem_wait_ld();
                                        tmem_loaded<8>(o);
#pragma unroll
                                        for (int x = 0; x < 8; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * a);
                                        tmem_st8(to + k, o);
                                    }
                                    tmem_wait_st();
                                }
                            }
                        }
                        const float base = ref == -INFINITY ? 0.f : ref;
                        const uint64_t base2 = pair(-base, -base);
                        uint64_t sum[2] = {0, 0};
                        // Weights in place of the scores (two a word), or straight to
                        // tensor memory where they are pairs.
                        auto weights = [&](auto in_bf16) {
                            constexpr bool to_bf16 = decltype(in_bf16)::value;
                            [[maybe_unused]] uint32_t hi[16], lo[16];
#pragma unroll
                            for (int k = 0; k < kTileTokens; k += 2) {
                                float x0, x1;
                                const float f = FP8 ? fs[k >> 4] : sc;
                                unpair(fma2(pair(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), pair(f, f), base2), x0, x1);
                                x0 = ex2(x0);
                                x1 = ex2(x1);
                                sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], pair(x0, x1));
                                if constexpr (FP8) {
                                    unpair(mul2(pair(x0, x1), pair(vs[k >> 4], vs[k >> 4])), x0, x1);
                                }
                                if (to_bf16 && !PAIR) {
                                    s[k >> 1] = pack_bf16x2(x0, x1);
                                } else if (to_bf16) {
                                    const uint32_t w = pack_bf16x2(x0, x1);
                                    const int n = (k & 31) >> 1;
                                    hi[n] = w;
                                    lo[n] = pack_bf16x2(x0 - __uint_as_float(w << 16), x1 - __uint_as_float(w & 0xffff0000u));
                                    if (n == 15) {
                                        tmem_st16(ts + (k >> 5) * 16, hi);
                                        tmem_st16(ts + 64 + (k >> 5) * 16, lo);
                                    }
                                } else {
                                    s[k >> 1] = pack_f16x2(x0, x1);
                                }
                            }
                        };
                        auto all = [&](auto in_bf16) {
                            weights(in_bf16);
                            if constexpr (!(PAIR && decltype(in_bf16)::value)) {  // weights() stored pairs itself
                                tmem_st32(ts, s);
                                tmem_st32(ts + 32, s + 32);
                            }
                        };
                        if constexpr (FP8) {
                            if (wide)
                                all(std::true_type());
                            else
                                all(std::false_type());
                        } else {
                            all(std::bool_constant<B16>());
                        }
                        float l0, l1;
                        unpair(add2(sum[0], sum[1]), l0, l1);
                        l += l0 + l1;
                        tmem_wait_st();
                    }
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&c.p_full[i]));
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                }
                // ------------------------------------------------- the item's rows
                if (ok && j0 < nt) ok = warp_wait(c.pv_done[i], (n_s - 1) & 1, limit);
            }
            if (ok && join && i == 1) {
                // this half's O stays where it is; the other half's warps, which
                // read the same lanes of tensor memory, take it from there
                c.join[r] = make_float2(ref, l);
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c.join_full));
                ++n_join;
                handed = true;
            } else if (ok && !(solo && i == 1)) {
                float a0 = 1.f, a1 = 0.f;
                if (join) {
                    ok = warp_wait(c.join_full, n_join & 1, limit);
                    ++n_join;
                    const float2 o = c.join[r];
                    const float top = fmaxf(ref, o.x), base = top == -INFINITY ? 0.f : top;
                    a0 = ex2(ref - base);
                    a1 = ex2(o.x - base);
                    l = a0 * l + a1 * o.y;
                    ref = top;
                }
                if (ok && warp_live) {
                    tmem_fence_after();
                    const int g = it.g0 + row0 + r;
                    const int h = it.kvh * p.G + g - small_div(g, p.g_magic) * p.G;
                    const int at = q < 0 ? -1 : q * p.Hq + h;  // row of out
                    const bool empty = l == 0.f;               // no token, or every score -inf
                    float mul = empty ? 0.f : 1.f / l, own = 0.f;
                    const bool part = it.nsplit > 1;
                    if (p.own_out && !part) grid_dependency_wait();
                    if (at >= 0) {
                        if (part) {
                            mul = 1.f;
                            p.part_m[(size_t)at * p.S + it.split] = ref;
                            p.part_d[(size_t)at * p.S + it.split] = l;
                            if (it.split == 0) p.row_splits[at] = it.nsplit;
                        } else {
                            float lse = empty ? -INFINITY : (ref + __log2f(l)) * kRowsLn2;
                            if (p.own_out) {
                                const float lo = __ldcg(p.own_lse + at), m = fmaxf(lse, lo);
                                const float wa = lse == -INFINITY ? 0.f : __expf(lse - m);
                                const float wb = lo == -INFINITY ? 0.f : __expf(lo - m);
                                const float inv = wa + wb > 0.f ? 1.f / (wa + wb) : 0.f;
                                mul *= wa * inv;
                                own = wb * inv;
                                lse = m == -INFINITY ? -INFINITY : m + logf(wa + wb);
                            }
                            if (p.lse) p.lse[at] = lse;
                        }
                    }
                    if (FP8 && !wide) mul *= it.v_unit;
                    a0 *= mul;
                    a1 *= mul;
                    if (nt > 0) {
                        // O through shared memory, so that neighbouring lanes write
                        // neighbouring bytes of a row: W columns at a time, in the
                        // stage of the item's last K tile (all its products are
                        // complete; the warps release it below).
                        constexpr int W = D / 4, CH = W / 4, RPI = 32 / CH;  // columns, 16-byte pieces, rows a pass
                        uint8_t *stage = smem + Sh::RING + ((e + 2 * (nt - 1)) % NST) * Sh::TILE + warp * (32 * W * 4);
                        // where piece ch of a row lies: eight lanes meet no bank twice
                        auto piece = [&](int row, int ch) {
                            return stage + row * (W * 4) + ((ch ^ (CH == 8 ? row & 7 : (row >> 1) & 3)) << 4);
                        };
                        const int my_ch = lane % CH;
                        int to_row[CH];  // this lane's rows of out, one a pass
#pragma unroll
                        for (int x = 0; x < CH; ++x) to_row[x] = __shfl_sync(0xffffffffu, at, x * RPI + lane / CH);
#pragma unroll 1
                        for (int k = 0; k < D; k += W) {
                            uint32_t o[W];
                            tmem_ldw<W>(to + k, o);
                            if (join) {
                                uint32_t o1[W];
                                tmem_ldw<W>(to + 128 + k, o1);
                                tmem_wait_ld();
                                tmem_loaded<W>(o);
                                tmem_loaded<W>(o1);
#pragma unroll
                                for (int x = 0; x < W; ++x)
                                    o[x] = __float_as_uint(fmaf(__uint_as_float(o1[x]), a1, __uint_as_float(o[x]) * a0));
                            } else {
                                tmem_wait_ld();
                                tmem_loaded<W>(o);
#pragma unroll
                                for (int x = 0; x < W; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * a0);
                            }
                            if (empty) {
#pragma unroll
                                for (int x = 0; x < W; ++x) o[x] = 0u;
                            }
#pragma unroll
                            for (int x = 0; x < CH; ++x)
                                *reinterpret_cast<uint4 *>(piece(lane, x)) = make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                            __syncwarp();
                            float4 v[CH];
#pragma unroll
                            for (int x = 0; x < CH; ++x) v[x] = *reinterpret_cast<const float4 *>(piece(x * RPI + lane / CH, my_ch));
                            const int col = k + 4 * my_ch;
                            if (part) {
#pragma unroll
                                for (int x = 0; x < CH; ++x)
                                    if (to_row[x] >= 0)
                                        *reinterpret_cast<float4 *>(p.part_o + ((size_t)to_row[x] * p.S + it.split) * D + col) = v[x];
                            } else {
                                if (p.own_out) {
                                    float4 f[CH];
#pragma unroll
                                    for (int x = 0; x < CH; ++x)
                                        f[x] = to_row[x] >= 0 ? __ldcg(reinterpret_cast<const float4 *>(p.own_out + (size_t)to_row[x] * D + col))
                                                              : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                                    for (int x = 0; x < CH; ++x) {
                                        const float w = __shfl_sync(0xffffffffu, own, x * RPI + lane / CH);
                                        v[x].x = fmaf(f[x].x, w, v[x].x);
                                        v[x].y = fmaf(f[x].y, w, v[x].y);
                                        v[x].z = fmaf(f[x].z, w, v[x].z);
                                        v[x].w = fmaf(f[x].w, w, v[x].w);
                                    }
                                }
#pragma unroll
                                for (int x = 0; x < CH; ++x)
                                    if (to_row[x] >= 0) put4<QBF16>(p.out, (size_t)to_row[x] * D + col, v[x].x, v[x].y, v[x].z, v[x].w);
                            }
                            __syncwarp();
                        }
                    } else if (at >= 0) {
                        // no tokens: the own tokens' state, or zeros
#pragma unroll 1
                        for (int k = 0; k < D; k += 4) {
                            const float4 f = p.own_out ? __ldcg(reinterpret_cast<const float4 *>(p.own_out + (size_t)at * D + k))
                                                       : make_float4(0.f, 0.f, 0.f, 0.f);
                            put4<QBF16>(p.out, (size_t)at * D + k, f.x * own, f.y * own, f.z * own, f.w * own);
                        }
                    }
                    __syncwarp();
                }
                if (join) {
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&c.join_empty));
                }
                tmem_fence_before();
            }
            if (ok && nt > 0) {
                // the last warp that is done with the held stage gives it back
                // (counted by item: one half may be an item ahead of the other)
                fence_proxy_async_shared();
                __threadfence_block();
                __syncwarp();
                if (lane == 0 && atomicAdd(&c.held[slot], 1) == 7) {
                    c.held[slot] = 0;
                    __threadfence_block();
                    mbar_arrive(smem_u32(&c.kv_empty[(e + 2 * (nt - 1)) % NST]));
                }
            }
            if (!ok) {
                if (lane == 0) rows_flag(p.status, FD_DEV_TIMEOUT);
                break;
            }
            e += 2 * nt;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&c.item_empty[slot]));
            ++n_item;
        }
        tmem_fence_before();
    }
    // What waits for this grid may read the own tokens' state as well.
    if (p.own_out) grid_dependency_wait();
    __syncthreads();
    tmem_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

}  // namespace fd

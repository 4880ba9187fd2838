// rows_api.cu -- C entry points of cross attention and of decode behind shared
// prefixes (declared in include/fd_api.h): checks, plans and launches.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <numeric>
#include <queue>
#include <vector>

#include "fd_internal.h"

using namespace fd;

namespace {

constexpr int kMaxBeams = 1 << 16;
constexpr long long kMaxTokens = 1LL << 22;  // query tokens of a call
constexpr long long kMaxRows = 1LL << 28;    // query tokens * heads
constexpr int kMaxGroup = 1 << 15;           // query heads of a KV head
constexpr int kMaxRowSms = 1 << 16;
constexpr uint64_t kRowsTimeoutNs = 2000000000ull;  // 2 s limit on any device-side wait
// Added to it where the pass over prefixes starts while the own tokens' pass ends
// (16-bit pools) and waits for that, without a limit, to join its state: what is
// left of it, its last stages and merges, takes tens of us, and other warps' waits
// last as long.
constexpr uint64_t kOwnEndNs = 1000000ull;
// Query rows of a KV head up to which the decode kernel takes a cross-attention
// call, decode and rows kernel in us.  16 bits (64 sequences, 512-8192 tokens, 4
// heads a KV head): 4 rows 172, 203; 16 rows 178, 211; 24 rows 300, 214 (16 rows a
// pass over K and V).  E4M3 (16 of 2048-16384 tokens, 8 heads), whose codes the
// rows kernel converts for 128 rows whatever their number: 8 rows 58, 156; 32
// rows 136, 156; 64 rows 263, 161.  2 to 64 sequences of 512 or 4096 tokens, D = 64
// and 128: the decode kernel is the faster one up to both limits but for 32 E4M3
// rows of 64 x 4096 tokens (143, 126; D = 64 99, 91) and 16 of 16 bits at D = 64 (64,
// 63).
constexpr int kFewRows = 16, kFewRowsE4m3 = 32;
constexpr int kPlanCross = 2, kPlanPrefix = 3;      // fd_cross_plan_t::reserved[0]

bool on(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// One work item: up to kItemRows query rows of a KV head over a chunk of a KV
// row, in tiles of kTile tokens and kTile rows.
constexpr int kTile = 128, kItemRows = 256;
constexpr int kMaxRowSplits = 64;
constexpr size_t kMaxPartialBytes = size_t(256) << 20;
// Times of the cost model, in ns: what an item costs beside its tiles (query
// rows, epilogue), what a split one costs more (its partial state), and the
// second launch that merges: its own time and the partial states it reads (bytes
// a ns).
constexpr double kItemNs = 2500, kSplitNs = 1000, kMergeNs = 3000, kMergeRate = 4000;

// Time of one CTA for a tile of 128 tokens: its share of the memory's rate, or
// what one and two row tiles measured (E4M3 codes are converted first).
double tile_ns(const fd_problem &p, int row_tiles, int weight_parts) {
    const bool fp8 = p.kv_dtype == FD_E4M3;
    // (two parts a weight, 4 x 2048 over 8192: 1.42 times at D = 128, 1.39 at D = 64)
    const double parts = p.kv_dtype == FD_BF16 && weight_parts == 2 ? 1.4 : 1.0;
    const double bytes = 2.0 * kTile * p.D * (fp8 ? 1 : 2) / 44.0;
    const double busy = (row_tiles == 2 ? (p.D == 128 ? 1450.0 : 1350.0) : (p.D == 128 ? 1000.0 : 800.0)) * (fp8 ? 1.5 : parts);
    return std::max(bytes, busy);
}

// Shared by both planners.  tokens_of(s): query tokens of segment s (segment
// kv_rows: those without a prefix).
template <typename TokensOf>
fd_status plan_rows(const fd_problem &p, int kv_rows, int seqs, int tokens, int max_blocks, const int32_t *kv_lens,
                    const fd_cross_options &opt, TokensOf tokens_of, fd_cross_plan_t *plan) {
    if (opt.num_splits < 0 || opt.num_sms < 0 || opt.num_sms > kMaxRowSms || opt.max_kv_len < 0 || opt.timeout_us < 0 ||
        opt.debug_stall_us < 0 || opt.debug_stall_us > 1000000 || opt.weight_parts < 1 || opt.weight_parts > 2)
        return FD_ERR_INVALID_ARG;
    if (p.out_dtype != p.q_dtype) return FD_ERR_UNSUPPORTED;
    if (p.Hq / p.Hkv > kMaxGroup) return FD_ERR_UNSUPPORTED;
    if (kv_rows > kMaxBatch || (long long)seqs * tokens > kMaxTokens || (long long)seqs * tokens * p.Hq > kMaxRows)
        return FD_ERR_UNSUPPORTED;
    int longest = 1, sms = opt.num_sms;
    for (int s = 0; s < kv_rows; ++s) {
        if (kv_lens[s] < 0) return FD_ERR_INVALID_ARG;
        longest = std::max(longest, (int)kv_lens[s]);
    }
    const int room = std::max(longest, opt.max_kv_len);
    if (room > (long long)p.page_size * max_blocks) return FD_ERR_INVALID_ARG;
    if (sms == 0) {
        DeviceInfo di;
        const fd_status st = device_info(di);
        if (st != FD_OK) return st;
        sms = di.sms;
    }
    // Chunks: the count that the cost model finds cheapest (fewest of equals).
    const size_t rows = (size_t)seqs * tokens * p.Hq;
    const int G = p.Hq / p.Hkv;
    auto chunk_of = [&](int S) { return (int)(((long long)longest + S - 1) / S + kTile - 1) / kTile * kTile; };
    auto fits = [&](int C) {
        const long long S = ((long long)room + C - 1) / C;
        return S == 1 || (S <= kMaxRowSplits && rows * S * (p.D + 2) * sizeof(float) <= kMaxPartialBytes);
    };
    // the kernel's order: longest rows first where it has few of them
    std::vector<int> order(kv_rows + 1);
    std::iota(order.begin(), order.end(), 0);
    if (kv_rows < 32)
        std::stable_sort(order.begin(), order.end() - 1, [&](int a, int b) { return kv_lens[a] > kv_lens[b]; });
    // items of all KV heads with chunks of C tokens, and their time on sms CTAs
    auto cost = [&](int C, long long *items_out) {
        std::vector<std::pair<double, long long>> items;  // time, how many of it
        double total = 0;
        long long count = 0;
        bool split = false;
        auto add = [&](double ns, long long n) {
            if (n < 1) return;
            items.push_back({ns, n});
            total += ns * n;
            count += n;
        };
        for (int s : order) {
            const long long r = (long long)tokens_of(s) * G;
            const int L = s < kv_rows ? kv_lens[s] : 0;
            const int ns = L == 0 ? 1 : (L + C - 1) / C;
            split |= ns > 1;
            const long long whole = r / kItemRows * p.Hkv;
            const int rest = (int)(r % kItemRows);
            const int last = L - (ns - 1) * C;  // tokens of the last chunk
            const double more = kItemNs + (ns > 1 ? kSplitNs : 0);
            for (int part = 0; part < 2; ++part) {
                const double tiles = (part ? last : C) / (double)kTile;
                const long long n = part ? 1 : ns - 1;
                add(std::ceil(tiles) * tile_ns(p, 2, opt.weight_parts) + more, n * whole);
                if (rest) add(std::ceil(tiles) * tile_ns(p, rest > kTile ? 2 : 1, opt.weight_parts) + more, n * p.Hkv);
            }
        }
        if (items_out) *items_out = count;
        const double merge = split ? kMergeNs + (double)rows * ((longest + C - 1) / C) * p.D * 4.0 / kMergeRate : 0.0;
        double longest_item = 0;
        for (const auto &it : items) longest_item = std::max(longest_item, it.first);
        if (count > 64LL * sms)  // plenty: the tail is about half an item
            return total / sms + 0.5 * longest_item + merge;
        std::priority_queue<double, std::vector<double>, std::greater<double>> q;
        for (int i = 0; i < sms; ++i) q.push(0.0);
        double worst = 0;
        for (const auto &it : items)
            for (long long k = 0; k < it.second; ++k) {
                const double t = q.top() + it.first;
                q.pop();
                worst = std::max(worst, t);
                q.push(t);
            }
        return worst + merge;
    };
    int best = chunk_of(std::max(1, std::min(opt.num_splits, kMaxRowSplits)));
    if (opt.num_splits == 0) {
        double best_cost = -1;
        int last = 0;
        for (int S = 1; S <= kMaxRowSplits; ++S) {
            const int C = chunk_of(S);
            if (C == last || !fits(C)) continue;
            last = C;
            const double t = cost(C, nullptr);
            if (best_cost < 0 || t < best_cost * 0.98) {
                best_cost = t;
                best = C;
            }
        }
    }
    while (!fits(best))
        best = (int)std::min((best + best / 2LL + kTile - 1) / kTile * kTile, (room + kTile - 1LL) / kTile * kTile);
    long long items = 0;
    cost(best, &items);
    // other lengths or groups than the planned ones may make more items
    items = std::max(items, (long long)sms);
    std::memset(plan, 0, sizeof(*plan));
    plan->problem = p;
    plan->problem.max_blocks_per_seq = max_blocks;
    plan->kv_rows = kv_rows;
    plan->seqs = seqs;
    plan->tokens = tokens;
    plan->num_splits = (room + best - 1) / best;
    plan->chunk_tokens = best;
    plan->capacity_tokens = room;
    plan->weight_parts = opt.weight_parts;
    plan->grid_ctas = (int)std::min<long long>(items, sms);
    plan->num_sms = sms;
    plan->timeout_us = opt.timeout_us;
    plan->debug_stall_us = opt.debug_stall_us;
    const size_t S = plan->num_splits > 1 ? (size_t)plan->num_splits : 0;
    size_t at = 0;
    plan->ws_partial_o = at;
    at += up256(rows * S * p.D * sizeof(float));
    plan->ws_partial_md = at;
    at += up256(2 * rows * S * sizeof(float));
    plan->ws_counters = at;
    at += 256 + (S ? up256(rows * sizeof(int)) : 0);
    plan->workspace_bytes = at;
    return FD_OK;
}

// The launch of a planned pass; pointers were checked.
fd_status run_rows(const fd_cross_plan_t &plan, RowsParams rp, const void *k_pages, const void *v_pages,
                   uint8_t *workspace, void *stream) {
    const fd_problem &p = plan.problem;
    rp.kv_rows = plan.kv_rows;
    rp.seqs = plan.seqs;
    rp.T = plan.tokens;
    rp.beams = plan.beams;
    rp.Hq = p.Hq;
    rp.Hkv = p.Hkv;
    rp.G = p.Hq / p.Hkv;
    rp.D = p.D;
    rp.page_size = p.page_size;
    rp.max_blocks = p.max_blocks_per_seq;
    rp.num_pages = p.num_pages;
    rp.S = plan.num_splits;
    rp.chunk = plan.chunk_tokens;
    rp.cap = plan.capacity_tokens;
    rp.q_bf16 = p.q_dtype == FD_BF16;
    rp.weight_parts = plan.weight_parts;
    rp.kv_kind = p.kv_dtype == FD_F16 ? KV_F16 : (p.kv_dtype == FD_BF16 ? KV_BF16 : KV_E4M3);
    rp.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)p.D));
    rp.timeout_ns = plan.timeout_us > 0 ? (uint64_t)plan.timeout_us * 1000ull : kRowsTimeoutNs;
    if (rp.own_out && p.kv_dtype != FD_E4M3) rp.timeout_ns += kOwnEndNs;
    rp.stall_ns = (uint64_t)plan.debug_stall_us * 1000ull;
    const size_t rows = (size_t)plan.seqs * plan.tokens * p.Hq;
    rp.part_o = reinterpret_cast<float *>(workspace + plan.ws_partial_o);
    rp.part_m = reinterpret_cast<float *>(workspace + plan.ws_partial_md);
    rp.part_d = rp.part_m + rows * plan.num_splits;
    rp.counters = reinterpret_cast<int *>(workspace + plan.ws_counters);
    rp.row_splits = rp.counters + 64;
    rp.boxr = std::gcd(p.page_size, kTile);
    rp.g_magic = rp.G > 1 ? (uint32_t)(((1ull << 32) + rp.G - 1) / rp.G) : 0;
    CUtensorMap tmk, tmv;
    const bool ok = p.kv_dtype == FD_E4M3
                        ? encode_pool_map(&tmk, k_pages, p, rp.boxr, true) && encode_pool_map(&tmv, v_pages, p, rp.boxr, true)
                        : encode_pool_map_grouped(&tmk, k_pages, p, rp.boxr) && encode_pool_map_grouped(&tmv, v_pages, p, rp.boxr);
    if (!ok) return FD_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (launch_rows(rp, tmk, tmv, plan.grid_ctas, s) != cudaSuccess) return FD_ERR_CUDA;
    if (plan.num_splits > 1 && launch_rows_merge(rp, s) != cudaSuccess) return FD_ERR_CUDA;
    return FD_OK;
}

// Both describe the same heads, types and pools (they may have another block
// table and output type).
bool same_pools(const fd_problem &a, const fd_problem &b) {
    return a.Hq == b.Hq && a.Hkv == b.Hkv && a.D == b.D && a.q_dtype == b.q_dtype && a.kv_dtype == b.kv_dtype &&
           a.page_size == b.page_size && a.num_pages == b.num_pages;
}

// What a plan handed in must satisfy for its launch to stay in bounds.
bool plan_ok(const fd_cross_plan_t &plan, int kind) {
    const fd_problem &p = plan.problem;
    fd_problem one = p;  // problem.B counts sequences or KV rows: both are bounded below
    one.B = 1;
    if (validate_problem(&one) != FD_OK || plan.reserved[0] != kind) return false;
    if (p.Hq / p.Hkv > kMaxGroup) return false;
    if (plan.kv_rows < 1 || plan.kv_rows > kMaxBatch || plan.seqs < 1 || plan.tokens < 1 || plan.num_splits < 1 ||
        (long long)plan.seqs * plan.tokens > kMaxTokens || (long long)plan.seqs * plan.tokens * p.Hq > kMaxRows)
        return false;
    if (kind == kPlanCross && (plan.beams < 1 || (long long)plan.kv_rows * plan.beams != plan.seqs)) return false;
    // (chunks of at most 2^30 tokens: length + chunk - 1 stays within an int)
    if (plan.chunk_tokens < kTile || plan.chunk_tokens > (1 << 30) || plan.chunk_tokens % kTile ||
        plan.num_splits > kMaxRowSplits || plan.grid_ctas < 1 ||
        plan.grid_ctas > kMaxRowSms ||
        plan.capacity_tokens > (long long)plan.num_splits * plan.chunk_tokens)
        return false;
    const size_t rows = (size_t)plan.seqs * plan.tokens * p.Hq, S = plan.num_splits > 1 ? (size_t)plan.num_splits : 0;
    if ((plan.ws_partial_o | plan.ws_partial_md | plan.ws_counters) % 256 || plan.ws_partial_md < plan.ws_partial_o ||
        plan.ws_partial_md - plan.ws_partial_o < rows * S * p.D * sizeof(float) || plan.ws_counters < plan.ws_partial_md ||
        plan.ws_counters - plan.ws_partial_md < 2 * rows * S * sizeof(float) || plan.workspace_bytes < plan.ws_counters ||
        plan.workspace_bytes - plan.ws_counters < 256 + (S ? rows * sizeof(int) : 0))
        return false;
    if (plan.has_few) {
        const fd_plan_t &f = plan.few;
        if (kind != kPlanCross || f.kv_rows != plan.kv_rows || f.row_fold != plan.beams * plan.tokens || f.q_len > 1 ||
            !same_pools(f.problem, p) || f.problem.out_dtype != p.out_dtype ||
            f.problem.max_blocks_per_seq != p.max_blocks_per_seq ||
            plan.ws_few % 256 || plan.workspace_bytes < plan.ws_few || plan.workspace_bytes - plan.ws_few < f.workspace_bytes ||
            plan.ws_few < plan.ws_counters || plan.ws_few - plan.ws_counters < 256 + (S ? rows * sizeof(int) : 0))
            return false;
    }
    if (plan.capacity_tokens < 1 || plan.capacity_tokens > (long long)p.page_size * p.max_blocks_per_seq) return false;
    return plan.timeout_us >= 0 && plan.debug_stall_us >= 0 && plan.debug_stall_us <= 1000000 && plan.weight_parts >= 1 &&
           plan.weight_parts <= 2;
}

bool pools_ok(const fd_problem &p, const void *k_pages, const void *v_pages, const float *k_scale, const float *v_scale) {
    const bool fp8 = p.kv_dtype == FD_E4M3;
    if (!k_pages || !v_pages || fp8 != (k_scale != nullptr) || fp8 != (v_scale != nullptr)) return false;
    return on(k_pages, 16) && on(v_pages, 16) && on(k_scale, 4) && on(v_scale, 4);
}

}  // namespace

extern "C" {

fd_status fd_plan_cross(const fd_problem *problem, const int32_t *kv_lens_host, const fd_cross_options *options,
                        fd_cross_plan_t *plan) {
    if (!plan || !kv_lens_host) return FD_ERR_INVALID_ARG;
    const fd_status st = validate_problem(problem);
    if (st != FD_OK) return st;
    fd_cross_options opt = {};
    if (options) opt = *options;
    if (opt.tokens < 0 || opt.beams < 0) return FD_ERR_INVALID_ARG;
    // One bf16 part: a prompt's time is its products' (4 x 2048 queries over 8192
    // states 740 us, with two 1032).
    if (opt.weight_parts == 0) opt.weight_parts = 1;
    opt.tokens = std::max(1, opt.tokens);
    opt.beams = std::max(1, opt.beams);
    if (opt.beams > kMaxBeams || opt.tokens > kMaxTokens) return FD_ERR_UNSUPPORTED;
    if ((long long)problem->B * opt.beams > kMaxTokens) return FD_ERR_UNSUPPORTED;
    fd_status r = FD_ERR_UNSUPPORTED;
    try {
        r = plan_rows(*problem, problem->B, problem->B * opt.beams, opt.tokens, problem->max_blocks_per_seq, kv_lens_host,
                      opt, [&](int s) { return s < problem->B ? (long long)opt.beams * opt.tokens : 0LL; }, plan);
    } catch (...) {  // no memory for the items
    }
    if (r != FD_OK) return r;
    plan->beams = opt.beams;
    plan->reserved[0] = kPlanCross;
    // Few query rows: the decode kernel, whose 8 or 16 columns of queries waste
    // less of an SM's time on them than tiles of 128 rows.
    const long long few = (long long)opt.beams * opt.tokens * (problem->Hq / problem->Hkv);
    if (few <= (problem->kv_dtype == FD_E4M3 ? kFewRowsE4m3 : kFewRows) && (long long)problem->B * opt.beams * opt.tokens <= kMaxBatch) {
        fd_plan_options po = {};
        po.fuse_merge = 1;
        po.num_splits = opt.num_splits;
        po.num_sms = opt.num_sms;
        po.max_seq_len = opt.max_kv_len;
        po.timeout_us = opt.timeout_us;
        po.debug_stall_us = opt.debug_stall_us;
        po.debug_stall_role = opt.debug_stall_us > 0 ? 1 : 0;
        if (plan_state(problem, kv_lens_host, &po, opt.beams * opt.tokens, &plan->few) == FD_OK) {
            plan->has_few = 1;
            plan->ws_few = plan->workspace_bytes;
            plan->workspace_bytes += up256(plan->few.workspace_bytes);
        }
    }
    return FD_OK;
}

fd_status fd_cross_paged(const fd_cross_plan_t *plan, const void *q, long long q_stride, const int32_t *q_lens,
                         const void *k_pages, const void *v_pages, const float *k_scale, const float *v_scale,
                         const int32_t *block_table, const int32_t *kv_lens, void *out, float *lse, void *workspace,
                         size_t workspace_bytes, int32_t *status_dev, void *stream) {
    if (!plan || !plan_ok(*plan, kPlanCross)) return FD_ERR_INVALID_ARG;
    const fd_problem &p = plan->problem;
    if (!q || !block_table || !kv_lens || !out || !workspace || !pools_ok(p, k_pages, v_pages, k_scale, v_scale))
        return FD_ERR_INVALID_ARG;
    if (!on(q, 16) || !on(out, 16) || !on(lse, 4) || !on(q_lens, 4) || !on(block_table, 4) || !on(kv_lens, 4) ||
        !on(workspace, 256) || !on(status_dev, 4))
        return FD_ERR_INVALID_ARG;
    if (q_stride < (long long)p.Hq * p.D || q_stride % 8) return FD_ERR_INVALID_ARG;
    if (workspace_bytes < plan->workspace_bytes) return FD_ERR_WORKSPACE_TOO_SMALL;
    if (plan->has_few && !q_lens && q_stride == (long long)p.Hq * p.D)
        return decode_state(&plan->few, q, k_pages, v_pages, k_scale, v_scale, block_table, kv_lens, out, lse,
                            static_cast<uint8_t *>(workspace) + plan->ws_few, plan->few.workspace_bytes, status_dev,
                            stream);
    RowsParams rp;
    std::memset(&rp, 0, sizeof(rp));
    rp.q = q;
    rp.q_stride = q_stride;
    rp.q_lens = q_lens;
    rp.block_table = block_table;
    rp.kv_lens = kv_lens;
    rp.k_scale = k_scale;
    rp.v_scale = v_scale;
    rp.out = out;
    rp.lse = lse;
    rp.status = status_dev;
    return run_rows(*plan, rp, k_pages, v_pages, static_cast<uint8_t *>(workspace), stream);
}

fd_status fd_plan_prefix(const fd_problem *problem, const int32_t *seq_lens_host, int prefixes, int prefix_max_blocks,
                         const int32_t *prefix_lens_host, const int32_t *offsets_host, const fd_plan_options *options,
                         const fd_cross_options *prefix_options, fd_prefix_plan_t *plan) {
    if (!plan || !seq_lens_host || !prefix_lens_host || !offsets_host) return FD_ERR_INVALID_ARG;
    const fd_status st = validate_problem(problem);
    if (st != FD_OK) return st;
    const fd_problem &p = *problem;
    if (prefixes < 1 || prefix_max_blocks < 1 || (long long)p.page_size * prefix_max_blocks > (1LL << 30))
        return FD_ERR_INVALID_ARG;
    if (prefixes > kMaxBatch) return FD_ERR_UNSUPPORTED;
    if (offsets_host[0] != 0 || offsets_host[prefixes] > p.B) return FD_ERR_INVALID_ARG;
    for (int s = 0; s < prefixes; ++s)
        if (offsets_host[s + 1] < offsets_host[s]) return FD_ERR_INVALID_ARG;
    if (p.out_dtype != p.q_dtype) return FD_ERR_UNSUPPORTED;
    fd_plan_options own = {0, 0, 1, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    if (options) own = *options;
    if (own.shared_kv) return FD_ERR_UNSUPPORTED;
    fd_cross_options opt = {};
    if (prefix_options) opt = *prefix_options;
    std::memset(plan, 0, sizeof(*plan));
    fd_problem po = p;
    po.out_dtype = FD_F32;  // a state that the other pass joins
    fd_status r = plan_state(&po, seq_lens_host, &own, 0, &plan->own);
    if (r != FD_OK) return r;
    // Two bf16 parts, as in the decode of whole sequences (64 behind 8170 tokens 69 us,
    // with one 66; 512 behind 32768 406 and 338).
    if (opt.weight_parts == 0) opt.weight_parts = 2;
    opt.num_sms = own.num_sms;
    opt.timeout_us = own.timeout_us;
    const int T = std::max(1, own.q_len);
    r = FD_ERR_UNSUPPORTED;
    try {
        r = plan_rows(p, prefixes, p.B, T, prefix_max_blocks, prefix_lens_host, opt,
                      [&](int s) { return (long long)T * ((s < prefixes ? offsets_host[s + 1] : p.B) - offsets_host[s]); },
                      &plan->shared);
    } catch (...) {  // no memory for the items
    }
    if (r != FD_OK) return r;
    plan->shared.reserved[0] = kPlanPrefix;
    plan->prefixes = prefixes;
    const size_t rows = (size_t)p.B * T * p.Hq;
    size_t at = 0;
    plan->ws_own_out = at;
    at += up256(rows * p.D * 4);
    plan->ws_own_lse = at;
    at += up256(rows * 4);
    plan->ws_own = at;
    at += up256(plan->own.workspace_bytes);
    plan->ws_shared = at;
    at += up256(plan->shared.workspace_bytes);
    plan->workspace_bytes = at;
    return FD_OK;
}

fd_status fd_decode_paged_prefix(const fd_prefix_plan_t *plan, const void *q, const void *k_pages, const void *v_pages,
                                 const float *k_scale, const float *v_scale, const int32_t *prefix_table,
                                 const int32_t *prefix_lens, const int32_t *members, const int32_t *offsets,
                                 const int32_t *block_table, const int32_t *seq_lens, void *out, float *lse,
                                 void *workspace, size_t workspace_bytes, int32_t *status_dev, void *stream) {
    if (!plan || !plan_ok(plan->shared, kPlanPrefix)) return FD_ERR_INVALID_ARG;
    const fd_cross_plan_t &sh = plan->shared;
    const fd_problem &p = sh.problem;
    if (plan->prefixes != sh.kv_rows || plan->own.kv_rows != sh.seqs || std::max(1, plan->own.q_len) != sh.tokens ||
        plan->own.row_fold != sh.tokens || !same_pools(plan->own.problem, p) || plan->own.problem.out_dtype != FD_F32)
        return FD_ERR_INVALID_ARG;
    const size_t rows = (size_t)sh.seqs * sh.tokens * p.Hq;
    if (plan->ws_own_lse < plan->ws_own_out || plan->ws_own_lse - plan->ws_own_out < rows * p.D * 4 ||
        plan->ws_own < plan->ws_own_lse || plan->ws_own - plan->ws_own_lse < rows * 4 || plan->ws_shared < plan->ws_own ||
        plan->ws_shared - plan->ws_own < plan->own.workspace_bytes || plan->workspace_bytes < plan->ws_shared ||
        plan->workspace_bytes - plan->ws_shared < sh.workspace_bytes ||
        (plan->ws_own_out | plan->ws_own_lse | plan->ws_own | plan->ws_shared) % 256)
        return FD_ERR_INVALID_ARG;
    if (!q || !prefix_table || !prefix_lens || !members || !offsets || !block_table || !seq_lens || !out || !workspace ||
        !pools_ok(p, k_pages, v_pages, k_scale, v_scale))
        return FD_ERR_INVALID_ARG;
    if (!on(q, 16) || !on(out, 16) || !on(lse, 4) || !on(prefix_table, 4) || !on(prefix_lens, 4) || !on(members, 4) ||
        !on(offsets, 4) || !on(block_table, 4) || !on(seq_lens, 4) || !on(workspace, 256) || !on(status_dev, 4))
        return FD_ERR_INVALID_ARG;
    if (workspace_bytes < plan->workspace_bytes) return FD_ERR_WORKSPACE_TOO_SMALL;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    float *own_out = reinterpret_cast<float *>(ws + plan->ws_own_out);
    float *own_lse = reinterpret_cast<float *>(ws + plan->ws_own_lse);
    const fd_status st = decode_state(&plan->own, q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens,
                                      own_out, own_lse, ws + plan->ws_own, plan->own.workspace_bytes, status_dev,
                                      stream);
    if (st != FD_OK) return st;
    RowsParams rp;
    std::memset(&rp, 0, sizeof(rp));
    rp.q = q;
    rp.q_stride = (long long)p.Hq * p.D;
    rp.members = members;
    rp.offsets = offsets;
    rp.block_table = prefix_table;
    rp.kv_lens = prefix_lens;
    rp.k_scale = k_scale;
    rp.v_scale = v_scale;
    rp.out = out;
    rp.lse = lse;
    rp.own_out = own_out;
    rp.own_lse = own_lse;
    rp.status = status_dev;
    return run_rows(sh, rp, k_pages, v_pages, ws + plan->ws_shared, stream);
}

}  // extern "C"

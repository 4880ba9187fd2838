// fd_internal.h -- parameters shared between the C ABI layer (fd_api.cu) and
// the kernel translation units.  Not part of the public interface.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/fd_api.h"

namespace fd {

// Consumer warps per CTA, tokens per consumer warp per stage, and the
// pipeline tile (tokens per stage) that follows from them.
constexpr int kTokensPerWarp = 16;
constexpr int kMaxConsumerWarps = 8;
constexpr int kMaxBoxesPerTile = 8;  // tile / gcd(page_size, tile) <= 128 / 16
constexpr int kMaxSplits = 512;      // partial slots per (b, hq)
constexpr int kMaxBatch = 8192;
constexpr int kMinChunkTokens = 256; // below this a sequence is not split

enum KvKind { KV_F16 = 0, KV_BF16 = 1, KV_E4M3 = 2 };

struct DecodeParams {
    const void *q;             // [B, Hq, D]
    const int32_t *block_table;
    const int32_t *seq_lens;
    const int32_t *batch_idx;  // [B] cache row of q row b, or null (row b)
    const int32_t *leftpad;    // [cache rows] first attended token, or null (0)
    int cache_rows;            // rows of block_table / seq_lens / leftpad
    const float *k_scale;      // [num_pages, Hkv] or null
    const float *v_scale;
    void *out;                 // [B, Hq, D]
    float *lse;                // [B, Hq] or null
    float *part_o;             // [B, Hq, S, D]
    float *part_m;             // [B, Hq, S]
    float *part_d;             // [B, Hq, S]
    int *merge_ctr;            // [B, Hkv]
    int *work_ctr;             // 1
    int *done_ctr;             // 1
    int *status;               // null allowed
    int B, Hq, Hkv, G;
    // Query rows of one work item: the G*fold rows that read KV head kvh of
    // KV row bkv (fold > 1: several q sequences share one KV row), sliced
    // into nhg sub-groups of at most 8*NT rows.  Row i of the group is q
    // sequence bkv*fold + i/G, head kvh*G + i%G.
    int fold, nhg, Bkv;
    int page_size, max_blocks, num_pages;
    int S;                     // partial slots per (b, hq)
    int chunk;                 // tokens per split
    int cap;                   // S * chunk
    int boxr;                  // token rows per TMA box: gcd(page_size, tile)
    int out_dtype;             // fd_dtype
    int fuse_merge;
    int stages;
    int scr_in_stage;          // epilogue scratch in the item's last stage (16-bit K/V)
    float scale_log2;          // log2(e) / sqrt(D)
    uint64_t timeout_ns;       // limit of every device-side wait
    uint64_t stall_ns;         // test hook (0 = off): idle time of stall_role
    int stall_role;            // 1: producer before its first load; 2: consumers before the first release
    int qn;                    // query tokens per KV row, causal among them (1: one-token decode)
    // Score-writing instances (attention-weight totals) only.
    float *scores;             // [Bkv, Hkv, cap, score_stride(G * fold)] log2-unit scores of rows that are split (or not w_fused)
    float *cta_scores;         // w_fused: [grid, chunk, score_stride(G * fold)], each CTA's scores of its current whole row
    const float *w_in;         // [Bkv, Hkv, w_stride] or null (zeros)
    float *w_out;
    int w_stride;
    int w_fused;               // rows that are not split: totals formed by the decode kernel (nhg == 1)
    // Differential instances only.
    const float *lambda;       // [Hq / 2] (Hq counts the padded query rows)
    const void *norm_w;        // [D] or null: no norm
    int norm_w_dtype;
    float norm_eps, out_scale;
};

// Attention-weight totals from the scores and lse of a decode call.
struct WeightParams {
    const float *scores;       // [Bkv, Hkv, cap, score_stride(R)]
    const float *lse;          // [Bkv * fold, Hq]
    const float *in;           // [Bkv, Hkv, weights_stride] or null (zeros)
    float *out;                // [Bkv, Hkv, weights_stride]
    const int32_t *seq_lens;
    int *status;
    int Bkv, Hq, Hkv, G, fold, R, cap, weights_stride;
    int skip_to;               // rows of at most this length were done by the decode kernel
};

struct NormAppendParams {
    const void *q, *k, *v;     // [B, T, heads, D] 16-bit, token strides in elements
    void *q_out;
    long long q_stride, k_stride, v_stride, q_out_stride;
    const void *qw, *kw;       // [D] or null: no norm
    int w_f32;                 // norm weights in fp32 (else in q's type)
    float eps;
    const float *cos, *sin;    // null: no rotation
    int rotary_dim, max_pos, interleaved;
    void *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const int32_t *block_table, *seq_lens, *positions, *new_lens;
    int *status;
    int B, T, Hq, Hkv;         // Hq = 0: no queries
    int page_size, max_blocks, num_pages;
    int kv_kind, is_bf16;
    int parts;                 // warps per token (set at launch)
    int w_vec;                 // both norm weights 8-byte aligned (set at launch)
    int cs_vec;                // cosines and sines in groups of four 16-byte aligned (set at launch)
};

struct EvictParams {
    void *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const int32_t *block_table, *dst_table, *seq_lens;
    const float *weights;
    float *weights_out;        // null: not kept
    int32_t *new_lens, *kept;  // [B], [B, Hkv, budget]
    int *status;
    int B, Hkv, D, page_size, max_blocks, num_pages, row_bytes;
    int weights_stride, budget, sinks, recent;
};

// Query rows over KV rows that all of them see (rows.cu).  Segment s: the query
// tokens of the sequences i in [off(s), off(s + 1)) of the member order, which
// read KV row s; the last segment of a grouped call reads none.
struct RowsParams {
    const void *q;             // [seqs, T, Hq, D]
    long long q_stride;        // elements between tokens
    const int32_t *q_lens;     // [seqs] or null (T each)
    const int32_t *members;    // [seqs] sequences in group order, or null (in order)
    const int32_t *offsets;    // [kv_rows + 1], or null (beams sequences a KV row)
    const int32_t *block_table, *kv_lens;  // [kv_rows, max_blocks], [kv_rows]
    const float *k_scale, *v_scale;        // [num_pages, Hkv] or null
    void *out;                 // [seqs, T, Hq, D]
    float *lse;                // [seqs, T, Hq] or null
    const float *own_out;      // [seqs, T, Hq, D] and [seqs, T, Hq]: a state over other
    const float *own_lse;      // tokens that joins every row's, or null
    float *part_o;             // [seqs * T * Hq, S, D]: unnormalised; m in log2 units
    float *part_m, *part_d;    // [seqs * T * Hq, S]
    int *row_splits;           // [seqs * T * Hq] partial states to merge, 0: none (zeros between calls)
    int *counters;             // 2, zeros between calls
    int *status;
    int kv_rows, seqs, T, beams, Hq, Hkv, G;
    int page_size, max_blocks, num_pages;
    int S, chunk, cap;
    int boxr;                  // token rows per TMA box: gcd(page_size, tile)
    uint32_t g_magic;          // ceil(2^32 / G), 0: G = 1
    int q_bf16, kv_kind, D;
    int weight_parts;          // bf16 pools: bf16 parts of a weight
    float scale_log2;          // log2(e) / sqrt(D)
    uint64_t timeout_ns, stall_ns;
};

struct MergeParams {
    const float *part_o, *part_m, *part_d;
    void *out;
    float *lse;
    const int32_t *seq_lens;   // non-null: per-sequence split counts from lengths
    const int32_t *batch_idx;  // as in DecodeParams (with seq_lens only)
    const int32_t *leftpad;
    int cache_rows;
    int B, Hq, S, D, chunk, cap;
    int fold;                  // q sequences per KV row
    int out_dtype;
};

struct AppendParams {
    const void *k_new, *v_new;
    void *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const int32_t *block_table, *seq_lens;
    int *status;
    int B, Hkv, D, page_size, max_blocks, num_pages;
    int kv_kind;               // KvKind
    int new_is_bf16;           // for E4M3 caches: input dtype bf16 (1) or f16 (0)
    // Rotary embedding (cos == null: none): tables [max_pos, rotary_dim/2].
    const float *cos, *sin;
    int rotary_dim, max_pos, interleaved;
    void *q_inout;             // [B, Hq, D] rotated in place, or null
    int Hq;
    int q_is_bf16;
};

// MODE of a decode kernel instance: the plain decode, the one that also writes
// its scores (attention-weight totals), differential attention, the plain decode
// whose results join other states or go by their lse (its denominators sum the
// weights unrounded).
constexpr int kPlain = 0, kScores = 1, kDiff = 2, kState = 3;

// Kernel configuration chosen at plan time.
struct KernelShape {
    int consumer_warps;  // 4 or 8
    int subtiles;        // 16-token sub-tiles per consumer warp per stage: 1 or 2
    int tile;            // tokens per stage = consumer_warps * subtiles * 16
    int nt;              // 8-wide head tiles: 1 (G <= 8) or 2 (G <= 16)
};

// tile_tokens: 64, 128 or 256 (0 = default for the K/V type); fold: q
// sequences per KV row (1 = ordinary decode); ctas_per_sm: persistent CTAs
// per SM (E4M3 128-token stages with two or more CTAs per SM take 4 consumer
// warps x 2 sub-tiles, which fit two to an SM).
KernelShape kernel_shape(const fd_problem &p, int tile_tokens, int fold, int ctas_per_sm);
// Dynamic shared memory of the decode kernel of this shape with `stages`
// stages (p.B = KV rows: the dispatch tables); scr_in_stage: the epilogue
// scratch in the item's last stage (16-bit K/V; 0 where a stage cannot hold it).
size_t decode_smem_bytes(const fd_problem &p, const KernelShape &ks, int stages, bool scr_in_stage);

cudaError_t launch_merge(const MergeParams &mp, cudaStream_t stream);
cudaError_t launch_append(const AppendParams &ap, cudaStream_t stream);
// Whether launch_weights can launch for these sizes (R: query rows per KV head).
bool weights_launchable(int Bkv, int Hkv, long long cap, long long R);
cudaError_t launch_weights(const WeightParams &wp, cudaStream_t stream);
cudaError_t launch_append_norm(NormAppendParams p, int D, cudaStream_t stream);
cudaError_t launch_evict(const EvictParams &p, int sms, cudaStream_t stream);
cudaError_t launch_rows(const RowsParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid, cudaStream_t stream);
// The merge of the rows that it left in partial states.
cudaError_t launch_rows_merge(const RowsParams &p, cudaStream_t stream);

// The decode kernel's kState instances over KV rows that `fold` query rows a head
// read whole (fold 0: as the options say): fd_plan and fd_decode_paged for them.
fd_status plan_state(const fd_problem *problem, const int32_t *seq_lens_host, const fd_plan_options *options, int fold,
                     fd_plan_t *plan);
fd_status decode_state(const fd_plan_t *plan, const void *q, const void *k_pages, const void *v_pages,
                       const float *k_scale, const float *v_scale, const int32_t *block_table, const int32_t *seq_lens,
                       void *out, float *lse, void *workspace, size_t workspace_bytes, int32_t *status_dev, void *stream);

// Checks and encodings that the entry points share (fd_api.cu).
struct DeviceInfo {
    int sms = 0;
    int smem_optin = 0;     // per CTA (opt-in maximum)
    int smem_per_sm = 0;    // per SM
    int smem_reserved = 0;  // set aside per resident CTA
};
fd_status device_info(DeviceInfo &di);
fd_status validate_problem(const fd_problem *p);
// Tensor map of a K or V pool with boxes of boxr token rows of one KV head, all
// 128-byte spans of a row, one after the other, swizzled or plain.
bool encode_pool_map(CUtensorMap *map, const void *pool, const fd_problem &p, int boxr, bool plain = false);
// The same of a 16-bit pool with a box's tokens in groups of eight.
bool encode_pool_map_grouped(CUtensorMap *map, const void *pool, const fd_problem &p, int boxr);

cudaError_t launch_merge_two(const float *oa, const float *la, const float *ob, const float *lb, int rows, int D,
                             int out_dtype, void *out, float *lse, cudaStream_t stream);

}  // namespace fd

// fa_internal.h -- parameter blocks and launchers shared by the C-ABI layer and
// the kernel translation units.  Not part of the public interface.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "../../include/fa.h"

namespace fa {

// Forward kernel tile: 128 query rows (the tcgen05 M) x 128 keys.
constexpr int kBlockM = 128;
constexpr int kBlockN = 128;

struct FwdParams {
    CUtensorMap tm_q;  // bf16 [B*H][N][d], box {min(d,64), 128, 1}
    CUtensorMap tm_k;  // bf16 [B*H][Nk][d]
    CUtensorMap tm_v;  // bf16 [B*H][Nk][dv]
    CUtensorMap tm_o;  // O [B*H][N][dv] (bf16 or fp32), box {128 bytes of a row (64 for bf16 d = 32), 32, 1}
    void* o;           // [B*H][N][dv], bf16 or fp32
    float* lse;        // [B*H][N] or nullptr
    int* status;       // device status word
    int BH, N, Nk;
    int n_qp;           // query tile pairs per head: ceil(N / 256)
    int n_items;        // BH * n_qp work items
    int num_ctas;       // persistent CTAs (one per SM)
    float scale_log2;   // scale * log2(e)
    unsigned long long wait_limit_ns;
    // set by the launcher from its grid size G: the step between a CTA's item rounds (G items
    // without a causal mask, 2G - 1 from the second item of a pair under one) as whole heads
    // and a remainder, so that the kernel advances (head, position) without a division
    int step_heads, step_rem;
    int pairs;          // items go out in heavy/light pairs (causal, more items than CTAs) or singly
    // Without a mask: pairs per head with rows in both query tiles (all but a last pair of at most
    // 128 rows).  Items 0 .. BH * n_full - 1 are those pairs, head-major; the BH one-tile last
    // pairs (if any) come after them, so that they fill the last round instead of lengthening it.
    int n_full;
    // Split mode (fa_fwd_splitkv): the keys are cut into n_splits ranges of split_tiles key
    // tiles, an item is (head, query pair, split), n_qp counts the (query pair, split) items of a
    // head (pair-major), and each item writes its rows' normalised partial O (fp32) and natural-log
    // LSE to o_part [B*H*N][n_splits][dv] and lse_part [B*H*N][n_splits] instead of o / lse.
    int n_splits, split_tiles;
    float* o_part;
    float* lse_part;
};

// Launch the forward kernel for head size d (= dv), causal flag and output type.
cudaError_t launch_fwd(const FwdParams& p, int d, bool causal, fa_dtype o_dtype, cudaStream_t st);
// The same kernel in split mode (fp32 partials; FwdParams::n_splits, split_tiles, o_part, lse_part).
cudaError_t launch_fwd_split(const FwdParams& p, int d, bool causal, cudaStream_t st);

// Backward.  Work item: one head and one 128-key tile; the CTA walks every query tile
// that sees a key of it.  Per-row vectors and the dQ accumulator are padded to whole
// query tiles (Tr * 128 rows per head).
struct BwdParams {
    CUtensorMap tm_q;   // bf16 [B*H][N][d], box {min(d,64), 128, 1}
    CUtensorMap tm_k;   // bf16 [B*H][Nk][d]
    CUtensorMap tm_v;   // bf16 [B*H][Nk][d]
    CUtensorMap tm_do;  // bf16 [B*H][N][d]
    CUtensorMap tm_dk;  // dK [B*H][Nk][d] (gradient dtype), box {128 bytes of a row (64 for bf16 d = 32), 128, 1}
    CUtensorMap tm_dv;  // dV, the same
    const float* lse2;  // [B*H][Tr*128]: LSE * log2(e); +inf past N and where no key is visible
    const float* dsc;   // [B*H][Tr*128]: scale * sum_c dO[c] O[c]; 0 past N
    float* dq_acc;      // [B*H][Tr] tiles of 128 x d fp32 (layout: see dq_bulk), zeroed before the kernel
    void* dk;           // [B*H][Nk][d], gradient dtype
    void* dv;           // [B*H][Nk][d]
    int* status;
    int BH, N, Nk, Tr, Tc;
    int num_ctas;       // persistent CTAs (one per SM)
    float scale_log2;   // scale * log2(e)
    float scale;
    unsigned long long wait_limit_ns;
    // set by the launcher from its grid size G: G = step_heads * Tc + step_jr, and step_heads mod Tc
    // (the causal rotation), so that the kernel advances its items without a division
    int step_heads, step_jr, step_rot;
};

#ifndef FA_DQ_BULK
#define FA_DQ_BULK 1
#endif
// d <= 64: the tensor-core kernel adds its dQ tiles into the accumulator with bulk reductions from
// shared memory, and the accumulator of a (head, query tile) is laid out [row quarter w][d/4][32][4]
// (row q: w = q / 32, lane q mod 32), so that each warp's 16-column block is 2 KB contiguous.
// d = 128 (no shared memory left for the staging) keeps vector atomics and the [d/4][128][4] layout.
constexpr bool dq_bulk(int d) { return FA_DQ_BULK != 0 && d <= 64; }

struct BwdPrepParams {
    const void* o;      // [B*H][N][d], bf16 or fp32 (forward output)
    const void* d_o;    // bf16 [B*H][N][d]
    const float* lse;   // [B*H][N] (forward output, natural log)
    float* lse2;
    float* dsc;
    float* dq_acc;
    int BH, N, Tr, d;
    float scale;
    int* counter;       // set to 0 (fa_rules_bwd_kernel's items); nullptr: none
};

struct BwdDqParams {
    const float* dq_acc;
    void* dq;           // [B*H][N][d], gradient dtype
    int BH, N, Tr, d;
    // blocks from dq_blocks on add up parts of dK and dV (fa_bwd_rules): out[i] = sum over parts of part[p][i], in order,
    // for i < n_sum (a multiple of 32)
    const float *dk_part, *dv_part;
    void *dk, *dv;
    long long n_sum;
    int parts;          // 0: none
    int dq_blocks, sum_blocks;  // set by the launcher
};

cudaError_t launch_bwd(const BwdParams& p, int d, bool causal, fa_dtype grad_dtype, cudaStream_t st);
cudaError_t launch_bwd_prep(const BwdPrepParams& p, fa_dtype o_dtype, cudaStream_t st);
struct RangesParams;
// The same, and the documents' intervals of every key.
cudaError_t launch_bwd_prep_ranges(const BwdPrepParams& p, const RangesParams& r, fa_dtype o_dtype, cudaStream_t st);
cudaError_t launch_bwd_dq(const BwdDqParams& p, fa_dtype grad_dtype, cudaStream_t st);

// Split-KV on the tensor core: one CTA per (key split, 128-row query tile, group).  A group is
// a head (prefill: its N query rows) or a key/value head with its R packed query heads (decode).
struct SplitParams {
    CUtensorMap tm_q;   // bf16 [n_groups][rows_per_group][d], box {min(d,64), 128, 1}
    CUtensorMap tm_k;   // bf16 [n_groups][Nk][d]
    CUtensorMap tm_v;   // bf16 [n_groups][Nk][d]
    float* o_part;      // [n_groups * rows_per_group][n_splits][d] fp32
    float* lse_part;    // [n_groups * rows_per_group][n_splits] fp32
    const int* seqlens; // decode: keys per sequence (group / groups_per_batch); nullptr: Nk for all
    int* status;
    int n_groups, rows_per_group, n_qtiles, groups_per_batch;
    int Nk, n_splits, chunk;  // chunk: keys per split, a multiple of 128
    int causal_off;           // Nk - N: query row i sits at position causal_off + i
    float scale_log2;
    unsigned long long wait_limit_ns;
};

cudaError_t launch_splitkv(const SplitParams& p, int d, bool causal, bool varlen, cudaStream_t st);

// Decode: keys per block of the split kernel's inner loop; a split is a whole
// number of such blocks.
constexpr int kDecodeKeyBlock = 64;

struct DecodeParams {
    const void* q;        // bf16 [B*H][d]
    const void* k;        // bf16 [B*Hkv][Nk_max][d]
    const void* v;        // bf16 [B*Hkv][Nk_max][dv]
    const int* seqlens;   // int32 [B]
    float* o_part;        // fp32 [B*H][n_splits][dv]
    float* lse_part;      // fp32 [B*H][n_splits]
    void* o;              // [B*H][dv]
    float* lse;           // [B*H] or nullptr
    int* status;
    int B, H, Nk_max, n_splits, chunk;
    int Hkv;              // key/value heads; query head h reads key/value head h / (H / Hkv)
    float scale_log2;
    // Fused combine: non-null = per-(b, key/value head) arrival counters (zero on entry, left
    // zero); the last split CTA of a (b, key/value head) merges its rows into o / lse.
    unsigned int* counters;
    fa_dtype o_dtype;
};

cudaError_t launch_decode(const DecodeParams& p, int d, fa_dtype o_dtype, cudaStream_t st);

struct MergeParams {
    const float* o_parts;   // partial outputs
    const float* lse_parts; // partial log-sum-exps
    long long o_part_stride, o_row_stride;     // elements between parts / rows of o_parts
    long long lse_part_stride, lse_row_stride; // elements between parts / rows of lse_parts
    int n_parts, rows, dv;
    // optional per-row count of valid parts: ceil(clamp(seqlens[row / H]) / chunk)
    const int* seqlens;
    int H, chunk, Nk_max;
    void* o;     // [rows][dv]
    float* lse;  // [rows] or nullptr
    int* status;
};

cudaError_t launch_merge(const MergeParams& p, fa_dtype o_dtype, cudaStream_t st);

// Tree decode (fa_tree_kernel.cuh).  A group is a (sequence, key/value head) with its
// rows = (Hq / Hkv) * T query rows, row = head within the group * T + node; a unit is a block of
// part_rows of them.
constexpr int kTreeMaxShares = 320;  // of a call, and so parts of a unit

// What the merge has to join: the unit that a share began and did not finish.
struct TreeJoin {
    long long first_row;  // in the output
    int rows, parts;      // parts = 0: none.  (Decode behind a prefix: of each unit, rows is the share that begins it.)
};

struct TreeParams {
    CUtensorMap tm_q;    // bf16 [B*Hkv][rows][d], box {min(d,64), 128, 1}
    CUtensorMap tm_k;    // bf16 [B*Hkv][Nk_max][d]
    CUtensorMap tm_v;    // bf16 [B*Hkv][Nk_max][d]
    const int* seqlens;  // int32 [B]: cached tokens, without the tree
    const int* parents;  // int32 [B][T] or nullptr (a chain)
    const int* n_nodes;  // int32 [B] or nullptr (T everywhere)
    void* o;             // [B*Hkv][rows][d]
    float* lse;          // [B*Hkv][rows] or nullptr
    float* o_part;       // fp32 [2 * num_shares][part_rows][d]
    float* lse_part;     // fp32 [2 * num_shares][part_rows]
    TreeJoin* joins;     // [num_shares]
    int* status;
    int B, Hkv, rows, T, Nk_max;
    int part_rows;       // min(rows, 128), or 256 for more than 128 rows (PAIR form)
    int n_qp;            // units per group: ceil(rows / part_rows)
    int num_ctas;        // one per SM
    int num_shares;      // num_ctas, or two for each CTA (up to 128 rows)
    int unit_cost;       // a unit's start and end, in key tiles
    float scale_log2;
    fa_dtype o_dtype;
    unsigned long long wait_limit_ns;
};

cudaError_t launch_tree_32(const TreeParams& p, cudaStream_t st);
cudaError_t launch_tree_64(const TreeParams& p, cudaStream_t st);
cudaError_t launch_tree_128(const TreeParams& p, cudaStream_t st);

// Query/key norm with rotation (fa_qk_rope.cu).  A row is one head of one token, d elements.
struct RopeParams {
    const void *q, *k, *v;                       // bf16 [B*N tokens][heads][d]; v may be nullptr
    long long q_stride, k_stride, v_stride;      // elements between tokens
    const void *wq, *wk;                         // [d], bf16 or fp32
    const float *cos_t, *sin_t;                  // fp32 [max_pos][rot / 2]
    const int* positions;                        // int32 [B*N] or nullptr (token index in its sequence)
    void *q_out, *k_out, *v_out;                 // bf16 [B][heads][N][d], or the caches [B][Hkv][Nk_max][d]
    const int *seqlens, *parents, *n_nodes;      // append: as TreeParams
    int* status;
    int B, N, Hq, Hkv, rot, max_pos, Nk_max;
    int copies;                                  // times each key/value head is written (Hq / Hkv expanded, else 1)
    float eps;
    fa_dtype w_dtype;
};

struct RopeBwdParams {
    const void *dq, *dk, *dv;                    // [B][heads][N][d] of g_dtype; dv may be nullptr
    const void *q, *k;                           // as RopeParams
    long long q_stride, k_stride;
    const void *wq, *wk;
    const float *cos_t, *sin_t;
    const int* positions;
    void *gq, *gk, *gv;                          // [B*N][heads][d] of out_dtype
    long long gq_stride, gk_stride, gv_stride;
    float *gwq, *gwk;                            // fp32 [d]
    float* part;                                 // fp32 [CTAs][2][d]
    int* status;
    int B, N, Hq, Hkv, rot, max_pos, copies;
    float eps;
    fa_dtype w_dtype, g_dtype, out_dtype;
};

// CTAs of the backward kernel, and so partial rows of the weights' gradients, at most.
constexpr int kRopeBwdCtas = 1024;

cudaError_t launch_qk_rope(const RopeParams& p, int d, bool interleaved, bool append, int sms, cudaStream_t st);
cudaError_t launch_qk_rope_bwd(const RopeBwdParams& p, int d, bool interleaved, int sms, cudaStream_t st);

// Cache compaction (fa_cache.cu).
struct CompactParams {
    void *k, *v;                                 // bf16 [L][B][Hkv][Nk_max][d]
    const int *seqlens, *accepted, *n_accepted;  // int32 [B], [B][T], [B]
    int* seqlens_out;                            // int32 [B] or nullptr
    int* status;
    int L, B, Hkv, Nk_max, d, T;
};

cudaError_t launch_cache_compact(const CompactParams& p, cudaStream_t st);

// Attention under score rules (fa_rules_*.cu, fa_rules_*.cuh).  Scores are scale q.k, capped by a tanh and lowered
// by slope * distance; what a query sees is one interval of keys, what sees a key one interval of queries.
struct ScoreRules {
    float cap_in;         // scale / cap, so that cap * tanh(cap_in * S) is the capped score; 0: no cap
    float mult;           // capped scores in base 2 are mult * tanh, others mult * S: cap or scale, times log2(e)
    const float* slopes;  // fp32 [Hq] or nullptr
    float bias_in;        // log2(e) / mult: slopes[h] * bias_in * distance is taken off what mult multiplies
    // tanh(cap_in * S), times mult in forward kernels without a bias, as S P(S^2) (fa_rules_common.cuh, cap_factor)
    float2 near[3], mid[4], wide[6];  // (each twice, as the two-wide operations take them)
    bool far;  // the cap is above kFarCap
    float near_in, mid_in, wide_in;  // cap_in over the polynomials' ranges: |S| times it is at most 1 where they hold; +inf: nowhere
};

// A run of equal document numbers, and what a query or a key has of it (fa_rules_ranges_kernel).
struct RangesParams {
    const int* docs;    // int32 [B][Nk]
    const int* prefix;  // int32 [B] or nullptr
    int2* each;         // [B][n]: keys [x, y) of query x, or queries [x, y) of key x; empty: (0, 0)
    int2* tile;         // [B][tiles]: 128-tiles [x, y) of the other side that one of its 128 has to do with
    int* counter;       // of work items, set to 0 (by fa_rules_ranges_kernel)
    int* status;
    int B, N, Nk, tiles, causal;
};

// The documents' intervals of every query.
cudaError_t launch_rules_ranges(const RangesParams& p, cudaStream_t st);

struct FwdRulesParams {
    FwdParams f;        // without splits; tm_k and tm_v over B * Hkv heads
    ScoreRules rules;
    const int* prefix;  // int32 [B] or nullptr
    const int2* each;   // with documents: keys of each query [B][N], key tiles of each query tile [B][ceil(N / 128)]
    const int2* tile;
    int* counter;       // with documents: work items handed out
    int Hq, Hkv, causal;
    int chunk;          // causal, without documents: items go out by as many query heads at a time, longest first
};

// The kernels under score rules are compiled for each head size and kind of rules: kCap, kBias, both or neither.
enum RuleKinds { kNoRules = 0, kCap = 1, kBias = 2 };
inline int rule_kind(const ScoreRules& r) { return (r.cap_in > 0.f ? kCap : 0) + (r.slopes != nullptr ? kBias : 0); }

template <int D, int RULES>
cudaError_t launch_fwd_rules(const FwdRulesParams& p, fa_dtype o_dtype, cudaStream_t st);

struct BwdRulesParams {
    BwdParams b;        // BH = B * Hq; tm_k, tm_v, tm_dk, tm_dv over B * Hkv heads
    ScoreRules rules;
    const int* prefix;
    const int2* each;   // with documents: queries of each key [B][Nk], query tiles of each key tile [B][ceil(Nk / 128)]
    const int2* tile;
    int* counter;       // work items handed out, 0 at the start
    int B, Hq, Hkv, causal;
    int parts, part_heads;  // items that share a key tile's query heads, and query heads of each; with parts > 1 tm_dk,
                            // tm_dv, dk and dv are fp32 sums [parts][B * Hkv][Nk][d]
    int n_items;            // B * Hkv * parts * Tc
    int chunk;              // items go out by as many (key/value head, part)s at a time: of all of these the first key tile,
                            // then the second ..; 1: head by head
};

template <int D, int RULES>
cudaError_t launch_bwd_rules(const BwdRulesParams& p, fa_dtype grad_dtype, cudaStream_t st);

// Decode behind a shared prefix (fa_tree_kernel.cuh, SHARED).  Units are a key/value head's prefix with a query tile of the
// batch's rows, and then a sequence's own keys with its R rows.  Of the tree's parameters rows, T, parents and n_nodes
// have no meaning, joins holds a record for each unit.
struct PrefixParams : TreeParams {
    CUtensorMap tm_q1;      // bf16 [B][Hkv][R][d], box {min(d,64), R, 1, 1}; tm_q: box {min(d,64), R, 1, seqs}
    CUtensorMap tm_kp;      // bf16 [Hkv][P_max][d]
    CUtensorMap tm_vp;      // bf16 [Hkv][P_max][d]
    const int* prefix_len;  // int32 [1] or nullptr (P_max)
    ScoreRules rules;
    int P_max, R;
    int seqs;               // sequences of a query tile of the prefix: min(B, 128 / R)
    int n_pre;              // prefix units, Hkv * n_qp, or 0
    int rows_all;           // B * R
    // where whole units go, fp32: prefix ones [Hkv][B * R] rows, others [B][Hkv][R] rows (or, as they are, to o and
    // lse where there is no prefix: o_own = nullptr)
    float *o_pre, *lse_pre, *o_own, *lse_own;
};

// Joins what prefix and own keys gave each row.
struct PrefixSide {
    const TreeJoin* units;  // {-, first share, parts}
    const float *o_whole, *lse_whole;
};
struct PrefixMergeParams {
    PrefixSide pre, own;  // pre.units = nullptr: no prefix
    const float *o_part, *lse_part;
    int part_rows, num_shares;
    void* o;
    float* lse;
    int B, Hkv, R, seqs, n_qp;
    fa_dtype o_dtype;
};

template <int D, int RULES>
cudaError_t launch_prefix(const PrefixParams& p, cudaStream_t st);
cudaError_t launch_prefix_merge(const PrefixMergeParams& p, int d, cudaStream_t st);

// Host helpers of the C ABI files (fa_api.cu).
cudaError_t device_status_word(int** out);  // the current device's status word
cudaError_t device_sm_count(int* out);
unsigned long long wait_limit_ns();
// Tensor map of a bf16 tensor [BH][rows][d] with boxes of 128 (or box_rows) rows, from the thread's cache when possible.
bool bf16_tile_map(CUtensorMap* m, const void* ptr, int BH, int rows, int d, int box_rows = kBlockM);
// Tensor map of q [B][Hkv][R][d] whose box is the R rows of one key/value head of `seqs` sequences, the same way.
bool bf16_group_map(CUtensorMap* m, const void* ptr, int B, int Hkv, int R, int d, int seqs);
// Tensor map of an output [BH][rows][d] for bulk stores of box_rows rows (encode_out_map), the same way.
bool out_tile_map(CUtensorMap* m, void* ptr, int BH, int rows, int d, fa_dtype t, int box_rows);

// Status word helpers (device side records the first failure only).
enum : int { kStatusOk = 0 };

}  // namespace fa

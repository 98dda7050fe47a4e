/*
 * fa.h -- C ABI of libfa: exact tiled attention on GB300 (sm_103a).
 *
 * Operations (page titles and sections they follow):
 *   fa_fwd              exact attention forward, tiled with an online softmax
 *                       ("flash_lab.py -- FlashAttention, flash-decoding and
 *                       megakernel in numpy", section 3 `flash_fwd`, FlashAttention-2
 *                       loop order; the value it reaches is section 2
 *                       `standard_attention`).
 *   fa_decode_splitkv   single-query decode split over the key/value length, each
 *                       split's normalised output and log-sum-exp merged afterwards
 *                       ("flash_lab.py", section 4 `split_kv_decode`).
 *   fa_bwd              gradients dQ, dK, dV of exact attention, P recomputed tile by
 *                       tile from the forward's log-sum-exp ("flash_lab.py", section 3
 *                       `flash_bwd`, FlashAttention-2 form; the value it reaches is
 *                       section 2 `standard_attention_bwd`).
 *   fa_decode_splitkv_gqa  the same with the query heads of a key/value group packed
 *                       together ("flash_lab.py", section 4: GQA packs a group's query heads
 *                       as the rows of q; `decode_attention_time` method "fd").
 *   fa_fwd_splitkv      the forward with the keys split and merged, for few query tiles
 *                       ("flash_lab.py", section 4 applied to a query tile).
 *   fa_decode_splitkv_fused  the decode with the combine done by the last split of each
 *                       (b, h) instead of a second kernel.
 *   fa_merge_states     the log-sum-exp combine of partial states on its own
 *                       ("flash_lab.py", section 4 `split_kv_decode` combine, the
 *                       lse form of section 1 `merge_states`).
 *   fa_qk_norm_rope     a layer's query, key and value projections to fa_fwd's operands: norm of
 *                       each query and key head, position rotation and head-major layout;
 *   fa_qk_norm_rope_bwd its gradient from fa_bwd's outputs;
 *   fa_qk_norm_rope_append  the same for new tokens, keys and values written into a cache.
 *   fa_decode_tree      decode for a tree of drafted tokens over a cache (several queries for each
 *                       sequence, each seeing the cached tokens and its ancestors).
 *   fa_cache_compact    the accepted path of such a tree moved up behind the cached tokens.
 *   fa_fwd_rules        fa_fwd with rules for its scores (a cap by tanh, a bias that falls with the
 *                       distance) and for what a query sees (documents packed into a sequence, a
 *                       prefix that all see), and with shared key/value heads;
 *   fa_bwd_rules        its gradient.
 *   fa_decode_prefix    decode, one query a sequence, behind a prefix that the whole batch shares and that is
 *                       read once for it, under the same rules for the scores.
 *
 * Conventions shared by every entry point:
 *   - All tensors are dense, row-major, last dimension contiguous, in the layouts
 *     stated per argument ([B,H,rows,cols]); the projections that the fa_qk_norm_rope calls
 *     read, and the gradients written for them, have a token stride besides.  Device pointers
 *     must be 16-byte aligned.
 *   - q, k, v and the caches are bf16.  Arithmetic is fp32 (tensor-core accumulation in
 *     fp32; softmax statistics in fp32), but what a first product gives a second one on the
 *     tensor core is rounded to bf16 between them, by at most 2^-8 of each number: the softmax
 *     weights for the product with V (fa_fwd, fa_fwd_splitkv, fa_fwd_rules, fa_decode_tree,
 *     fa_decode_prefix, and fa_decode_splitkv_gqa but for groups of 1, 2 and, below d = 128, 4
 *     heads), and P and scale * dS in fa_bwd and fa_bwd_rules, whatever the output's type.  O is written as bf16 (FA_BF16) or fp32 (FA_F32);
 *     LSE is always fp32, natural log, scale included:
 *       LSE[i] = log sum_{visible j} exp(scale * q_i . k_j).
 *   - Causal masking places query i at position Nk - N + i and key j at position j
 *     ("02_flash_forward.py -- FlashAttention forward", demo 1; "flash_lab.py"
 *     `_causal_mask`).  A query row with no visible key (only when causal and N > Nk)
 *     gets O = 0 and LSE = -inf.
 *   - Ownership: the caller allocates and owns every buffer; the library allocates
 *     nothing.  Calls are asynchronous on `stream` (a cudaStream_t passed as void*;
 *     NULL = the legacy default stream) and never synchronise, except
 *     fa_get_device_error.
 *   - Stream order is kept: every kernel is launched with programmatic stream
 *     serialization, so it may start its setup (barriers, tensor memory) while the kernel
 *     before it on `stream` finishes, but it reads and writes global memory only after that
 *     kernel has completed and its writes are visible.  A caller's kernel launched after a
 *     call without that attribute starts once the call's kernels have completed, as usual.
 *   - CUDA graphs: after the first call on a device (which caches kernel attributes and
 *     device addresses), a call launches kernels on `stream` and does nothing else on the
 *     device, so every entry point but fa_get_device_error may be captured into a CUDA
 *     graph and replayed; the tensor maps are encoded at capture time from the pointers
 *     and sizes given, so a replay reads and writes the same buffers.
 *   - Errors: every argument is checked on the host before any launch; a bad argument
 *     returns a status and launches nothing.  A launch failure returns FA_ERR_CUDA.
 *     Failures the device detects (a bounded wait that ran out, a sequence length out
 *     of range) are recorded in a device status word read by fa_get_device_error.
 *   - Supported head sizes: d = dv, d in {32, 64, 128}.  Other sizes return
 *     FA_ERR_UNSUPPORTED.  Heads are independent; the number of key/value heads equals
 *     the number of query heads except in fa_decode_splitkv_gqa, fa_decode_tree, fa_decode_prefix,
 *     fa_fwd_rules, fa_bwd_rules and the fa_qk_norm_rope calls.
 */
#ifndef FA_H
#define FA_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1, /* null pointer, non-positive size, misaligned pointer, bad enum */
    FA_ERR_UNSUPPORTED = 2, /* valid arguments this build has no kernel for (head size) */
    FA_ERR_CUDA = 3,        /* a CUDA runtime call or kernel launch failed */
    FA_ERR_WORKSPACE = 4,   /* caller-provided workspace smaller than required */
    FA_ERR_TIMEOUT = 5      /* a device-side bounded wait ran out (kernel returned early) */
} fa_status;

typedef enum { FA_BF16 = 0, FA_F32 = 1 } fa_dtype;

/*
 * Exact attention forward ("flash_lab.py" section 3, FlashAttention-2 order): for each
 * (b, h) and query row i,
 *   O[b,h,i,:] = sum_j softmax_j(scale * Q[b,h,i,:] . K[b,h,j,:]) V[b,h,j,:]
 * over the visible keys j (all Nk keys, or j <= Nk - N + i when causal), and
 *   lse[b,h,i] = log sum_j exp(scale * Q[b,h,i,:] . K[b,h,j,:]).
 * The N x Nk score matrix never reaches memory.
 *
 *   q    bf16 [B, H, N,  d]        (device)
 *   k    bf16 [B, H, Nk, d]        (device)
 *   v    bf16 [B, H, Nk, dv]       (device)
 *   o    o_dtype [B, H, N, dv]     (device, written)
 *   lse  fp32 [B, H, N]            (device, written; may be NULL to skip it)
 *   B, H, N, Nk >= 1; d = dv in {32, 64, 128}; causal 0 or 1; scale > 0 and finite
 *   (1/sqrt(d) is the usual value); B*H*ceil(N/256) < 2^30 (else FA_ERR_INVALID_ARG).
 * Returns FA_OK after enqueueing the kernel on `stream`.
 */
fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                 int N, int Nk, int d, int dv, int causal, float scale, fa_dtype o_dtype,
                 void* stream);

/*
 * Bytes of workspace fa_bwd needs: with Tr = ceil(N / 128), an fp32 dQ accumulator of
 * B*H*Tr*128*d values, then fp32 base-2 log-sum-exps and fp32 scaled row terms of
 * B*H*Tr*128 values each, every region 256-byte aligned.  Returns 0 on invalid arguments.
 */
size_t fa_bwd_workspace_size(int B, int H, int N, int d);

/*
 * Exact attention backward ("flash_lab.py" section 3 `flash_bwd`).  For the upstream
 * gradient dO of the forward's output O, with P the attention weights of fa_fwd (same
 * mask and scale) and D_i = sum_c dO[i,c] O[i,c]:
 *   dV = P^T dO,  dP = dO V^T,  dS = P o (dP - D),  dQ = dS K scale,  dK = dS^T Q scale
 * for every (b, h).  P is recomputed tile by tile as exp(scale q.k - lse); it never reaches
 * memory.  Rows with no visible key (lse = -inf) contribute nothing.
 *
 *   q, k, v      bf16 [B, H, N, d], [B, H, Nk, d], [B, H, Nk, dv]  (device; the forward inputs)
 *   o            o_dtype [B, H, N, dv]   (device; the forward output, used only for D)
 *   lse          fp32 [B, H, N]          (device; the forward's log-sum-exp)
 *   grad_o       bf16 [B, H, N, dv]      (device; dO)
 *   grad_q, grad_k, grad_v   grad_dtype [B, H, N, d], [B, H, Nk, d], [B, H, Nk, dv]
 *                (device, written; every element is written)
 *   workspace    device scratch of ws_bytes >= fa_bwd_workspace_size(B, H, N, d) bytes,
 *                256-byte aligned; its contents on entry do not matter.
 *   B, H, N, Nk >= 1; d = dv in {32, 64, 128}; causal 0 or 1; scale > 0 and finite, the
 *   value the forward used; B*H*ceil(Nk/128) < 2^30 (else FA_ERR_INVALID_ARG).
 * Three kernels are enqueued on `stream`: a preparation pass (D, lse in base 2, zeroing the
 * dQ accumulator), the tensor-core pass (a persistent grid, one CTA per SM, walking the
 * (b, h, 128-key tile) items; each item's dK and dV written when its walk ends, dQ added into
 * the accumulator) and the dQ conversion.
 * The key tiles' shares of dQ are added into the fp32 accumulator by the memory system in
 * whatever order the CTAs reach it, so grad_q can differ in its last bits from run to run;
 * grad_k and grad_v are summed on chip in a fixed order and are reproducible.
 * Returns FA_ERR_WORKSPACE if ws_bytes is too small (nothing launched).
 */
fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                 const void* grad_o, void* grad_q, void* grad_k, void* grad_v, void* workspace,
                 size_t ws_bytes, int B, int H, int N, int Nk, int d, int dv, int causal,
                 float scale, fa_dtype o_dtype, fa_dtype grad_dtype, void* stream);

/*
 * Split count fa_decode_splitkv uses when asked for n_splits = 0, for a device with
 * `num_sms` streaming multiprocessors: enough splits of the longest sequence that the
 * non-empty (b, h, split) work items fill the device several times over, each split at
 * least one key block long.  Pure host function.  Returns 0 on invalid arguments.
 */
int fa_decode_default_splits(int B, int H, int Nk_max, int num_sms);

/*
 * Bytes of workspace fa_decode_splitkv needs for `n_splits` splits (n_splits >= 1):
 * fp32 partial outputs [B, H, n_splits, dv] followed by fp32 partial log-sum-exps
 * [B, H, n_splits], each region 256-byte aligned.  Returns 0 on invalid arguments.
 */
size_t fa_decode_workspace_size(int B, int H, int dv, int n_splits);

/*
 * Split-KV single-query decode ("flash_lab.py" section 4 `split_kv_decode`).  For each
 * (b, h), the first seqlens_k[b] cached keys are cut into n_splits consecutive chunks of
 * c = ceil(Nk_max / n_splits) keys (rounded up to the kernel's key block); split s covers
 * keys [s*c, min((s+1)*c, seqlens_k[b])) and is empty when that range is.  Each non-empty
 * split writes its normalised output o_s and lse_s to the workspace; a second kernel merges
 *   lse = log sum_s exp(lse_s),  o = sum_s exp(lse_s - lse) o_s.
 * The single query sits at position seqlens_k[b] - 1 and sees every cached key.
 *
 *   q          bf16 [B, H, 1, d]          (device)
 *   k_cache    bf16 [B, H, Nk_max, d]     (device; rows past seqlens_k[b] are never read)
 *   v_cache    bf16 [B, H, Nk_max, dv]    (device; idem)
 *   seqlens_k  int32 [B]                  (device; 0 <= seqlens_k[b] <= Nk_max.  Values
 *              outside that range are clamped into it and recorded as FA_ERR_INVALID_ARG in
 *              the device status word.  A length of 0 gives O = 0, LSE = -inf.)
 *   o          o_dtype [B, H, 1, dv]      (device, written)
 *   lse        fp32 [B, H, 1]             (device, written; may be NULL)
 *   workspace  device scratch of ws_bytes >= fa_decode_workspace_size(B, H, dv, n) bytes,
 *              256-byte aligned, where n is n_splits or, for n_splits = 0, the automatic
 *              count fa_decode_default_splits(B, H, Nk_max, <SMs of the current device>).
 *   n_splits   >= 0; 0 picks the automatic count.  Values above Nk_max are reduced to it.
 * Returns FA_ERR_WORKSPACE if ws_bytes is too small (nothing launched).
 */
fa_status fa_decode_splitkv(const void* q, const void* k_cache, const void* v_cache,
                            const int* seqlens_k, void* o, float* lse, void* workspace,
                            size_t ws_bytes, int B, int H, int Nk_max, int d, int dv, float scale,
                            int n_splits, fa_dtype o_dtype, void* stream);

/*
 * Split count fa_decode_splitkv_gqa uses when asked for n_splits = 0, for Hq query heads over Hkv
 * key/value heads of head size d on a device with `num_sms` multiprocessors.  Groups of
 * R = Hq / Hkv = 1 or 2 heads, and of 4 heads at d != 128, run on CUDA cores and take
 * fa_decode_default_splits(B, Hq, Nk_max, num_sms).  Other groups (tensor core) take
 * floor(1.7 * c * num_sms / (B * Hkv)) splits, where c = 2 for 3 to 8 heads at d = 128 (two CTAs
 * per multiprocessor) and 1 otherwise; raised to 2 while B * Hkv < 2 * num_sms, then to
 * ceil(ceil(Nk_max / 128) / T) with T = 64 key tiles for R <= 4 and 32 otherwise (no split
 * longer than T tiles), then clamped to [1, ceil(Nk_max / 128)].  Pure host function.  Returns 0
 * on invalid arguments (a non-positive size, or Hkv not dividing Hq).
 */
int fa_decode_gqa_default_splits(int B, int Hq, int Hkv, int Nk_max, int d, int num_sms);

/*
 * Split-KV decode with grouped key/value heads (GQA): Hq query heads share Hkv key/value heads,
 * query head h reading key/value head h / R with R = Hq / Hkv.  The R query heads of a group are
 * packed together ("flash_lab.py" section 4 `split_kv_decode`, q of shape [R, d]; section 4
 * `decode_attention_time`, method "fd": one work item per (b, key/value head, split), K and V read
 * once per group), so each cached key and value is read from memory once for all R heads.  The
 * split, merge, arguments and errors are those of fa_decode_splitkv, with:
 *
 *   q          bf16 [B, Hq, 1, d]          (device)
 *   k_cache    bf16 [B, Hkv, Nk_max, d]    (device)
 *   v_cache    bf16 [B, Hkv, Nk_max, dv]   (device)
 *   o          o_dtype [B, Hq, 1, dv]      (device, written)
 *   lse        fp32 [B, Hq, 1]             (device, written; may be NULL)
 *   workspace  ws_bytes >= fa_decode_workspace_size(B, Hq, dv, n) bytes, where n is n_splits or,
 *              for n_splits = 0, fa_decode_gqa_default_splits(B, Hq, Hkv, Nk_max, d, <SMs of the
 *              device>).
 *   Hkv >= 1 dividing Hq, R = Hq / Hkv <= 128 (larger groups return FA_ERR_UNSUPPORTED).
 *   Hkv = Hq is fa_decode_splitkv.  Groups of 1 or 2 heads, and of 4 heads at d != 128, run on
 *   CUDA cores; other group sizes on the tensor core (3 to 32 heads at d = 128 with the product
 *   transposed, keys on the tensor-memory lanes; otherwise the R query rows are the rows of a
 *   128-row tile), where splits are whole 128-key tiles (the chunk is rounded up to a multiple of
 *   128 instead of the key block) and cache rows past a sequence's length are never used,
 *   whatever they hold.
 */
fa_status fa_decode_splitkv_gqa(const void* q, const void* k_cache, const void* v_cache,
                                const int* seqlens_k, void* o, float* lse, void* workspace,
                                size_t ws_bytes, int B, int Hq, int Hkv, int Nk_max, int d, int dv,
                                float scale, int n_splits, fa_dtype o_dtype, void* stream);

/*
 * Bytes of workspace fa_decode_splitkv_fused needs: fa_decode_workspace_size(B, H, dv, n_splits)
 * followed by B*H 32-bit arrival counters (256-byte aligned).  0 on invalid arguments.
 */
size_t fa_decode_fused_workspace_size(int B, int H, int dv, int n_splits);

/*
 * fa_decode_splitkv with the combine fused into the split kernel: every non-empty split of a
 * (b, h) writes its o_s, lse_s and then counts itself on a per-(b, h) counter; the split that
 * arrives last merges the row ("flash_lab.py" section 4 combine), so one kernel is launched
 * instead of two (the launch gap is a decode cost the pages single out, section 5).  Same
 * arguments, checks and result as fa_decode_splitkv, except:
 *   workspace  ws_bytes >= fa_decode_fused_workspace_size(B, H, dv, n) bytes.  Its counter region
 *              (the last B*H*4 bytes of that size) must be zero before the first call that uses
 *              this workspace; every call that completes leaves it zero again.  After a call that
 *              failed on the device (fa_get_device_error != FA_OK) zero it again.  Calls sharing a
 *              workspace must not overlap on the GPU.
 */
fa_status fa_decode_splitkv_fused(const void* q, const void* k_cache, const void* v_cache,
                                  const int* seqlens_k, void* o, float* lse, void* workspace,
                                  size_t ws_bytes, int B, int H, int Nk_max, int d, int dv, float scale,
                                  int n_splits, fa_dtype o_dtype, void* stream);

/*
 * Split count fa_fwd_splitkv uses for n_splits = 0 on a device with `num_sms` multiprocessors:
 * the largest count for which the B*H*ceil(N/256) pairs of query tiles times the splits fit one
 * persistent CTA per multiprocessor (one round), at least 1 and at most ceil(Nk/128) (each split
 * at least one 128-key tile).  Pure host function; 0 on invalid arguments.
 */
int fa_fwd_splitkv_default_splits(int B, int H, int N, int Nk, int num_sms);

/*
 * Bytes of workspace fa_fwd_splitkv needs for n_splits splits: fp32 partial outputs
 * [B, H, N, n_splits, dv] then fp32 partial log-sum-exps [B, H, N, n_splits], each region
 * 256-byte aligned.  0 on invalid arguments.
 */
size_t fa_fwd_splitkv_workspace_size(int B, int H, int N, int dv, int n_splits);

/*
 * Exact attention forward with the keys split ("flash_lab.py" section 4 `split_kv_decode`
 * applied to a query tile): for workloads with few 128-row query tiles (B*H*ceil(N/256) pairs
 * of them below the number of multiprocessors) the keys are cut into chunks of whole 128-key
 * tiles (ceil(ceil(Nk/128) / n_splits) tiles each; chunks past the keys are dropped); the
 * forward kernel computes each (head, query tile pair, chunk)'s normalised output and
 * log-sum-exp, and a second kernel merges them.  Same arguments, masks, result and output
 * conventions as fa_fwd, plus:
 *   workspace  ws_bytes >= fa_fwd_splitkv_workspace_size(B, H, N, dv, n) bytes, 256-byte aligned,
 *              where n is n_splits or, for 0, fa_fwd_splitkv_default_splits(B, H, N, Nk, <SMs>);
 *   n_splits   >= 0; values above Nk are reduced to it.
 * B*H*N must be below 2^31 and B*H*ceil(N/256)*chunks below 2^30.  Returns FA_ERR_WORKSPACE if
 * ws_bytes is too small (nothing launched).
 */
fa_status fa_fwd_splitkv(const void* q, const void* k, const void* v, void* o, float* lse,
                         void* workspace, size_t ws_bytes, int B, int H, int N, int Nk, int d, int dv,
                         int causal, float scale, int n_splits, fa_dtype o_dtype, void* stream);

/*
 * Bytes of device scratch that fa_decode_splitkv_noalloc owns (8 MiB): room for the split
 * partials of B*H*n_splits*(dv+1) fp32 values, e.g. B=16, H=32, dv=128 with up to 30 splits.
 */
#define FA_DECODE_NOALLOC_SCRATCH_BYTES (8u << 20)

/*
 * fa_decode_splitkv without a workspace argument: the same computation, arguments, checks and
 * result, but the split partials go to a fixed scratch array of FA_DECODE_NOALLOC_SCRATCH_BYTES
 * that the library keeps in device memory (every GPU that loads the library holds it until the
 * process exits).  The pages have no counterpart; it exists for callers that cannot allocate
 * device memory: code whose memory belongs to another allocator (a framework's caching allocator,
 * a serving engine's fixed pool) and may not call cudaMalloc behind its back, code under a hard
 * per-process memory budget, and code that must not risk the device-wide synchronisation that
 * cudaMalloc and cudaFree can cause.  It allocates nothing and calls no allocating routine.
 *
 *   - Size limit: returns FA_ERR_WORKSPACE, launching nothing, when
 *     fa_decode_workspace_size(B, H, dv, n) exceeds FA_DECODE_NOALLOC_SCRATCH_BYTES, where n is
 *     n_splits or, for n_splits = 0, the automatic count.  Use fewer splits, or
 *     fa_decode_splitkv with a workspace of your own, for larger problems.
 *   - Set-up: the first call on each device looks up the scratch array's device address
 *     (cudaGetSymbolAddress, with that device current) and caches it; make that first call
 *     before any stream capture.  A failed look-up returns FA_ERR_CUDA.
 *   - Sharing: every call on a device uses the same array, which keeps the last call's contents.
 *     Nothing in it needs to start at zero (each non-empty split writes its slot before the
 *     combine reads it, and empty splits are never read).  Calls whose kernels overlap on the GPU
 *     (concurrent streams, or several host threads) race on the array: order them on one stream.
 */
fa_status fa_decode_splitkv_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                    const int* seqlens_k, void* o, float* lse, int B, int H,
                                    int Nk_max, int d, int dv, float scale, int n_splits,
                                    fa_dtype o_dtype, void* stream);

/*
 * Log-sum-exp combine of n_parts partial attention states per row ("flash_lab.py"
 * section 4 combine; section 1 `merge_states`, where a state with lse = -inf is empty and
 * gets weight 0):
 *   lse[r] = log sum_p exp(lse_parts[p, r]),  o[r, :] = sum_p exp(lse_parts[p, r] - lse[r]) o_parts[p, r, :]
 * A row whose every part is empty gets o = 0, lse = -inf.
 *
 *   o_parts    fp32 [n_parts, rows, dv]   (device)
 *   lse_parts  fp32 [n_parts, rows]       (device)
 *   o          o_dtype [rows, dv]         (device, written)
 *   lse        fp32 [rows]                (device, written; may be NULL)
 *   n_parts >= 1, rows >= 1, 1 <= dv <= 512.
 */
fa_status fa_merge_states(const float* o_parts, const float* lse_parts, int n_parts, int rows,
                          int dv, void* o, float* lse, fa_dtype o_dtype, void* stream);

/*
 * Operands of exact attention from a layer's projections.  For every token and head, with x the
 * head's d elements, w the weights and pos the token's position:
 *   y = x w / sqrt(mean(x^2) + eps)                          (query and key heads)
 *   (y_a, y_b) -> (y_a c - y_b s, y_a s + y_b c),  c = cos_table[pos][i], s = sin_table[pos][i]
 * for the pairs i < rot/2 of the first rot elements: (a, b) = (i, i + rot/2), or (2i, 2i + 1) with
 * interleaved = 1; the elements from rot on stay.  Value heads are copied.  Arithmetic is fp32, each
 * output element rounded once to bf16.
 *
 *   q, k, v    bf16 [B, N, heads, d]   (device; token (b, n) at (b N + n) * stride elements, its heads
 *              d apart: slices of one projection's output will do.  Strides >= heads * d, multiples
 *              of 8.  v may be NULL, with v_out.)
 *   q_weight, k_weight   w_dtype [d]   (device; 4-byte aligned)
 *   cos_table, sin_table fp32 [max_pos, rot/2]  (device)
 *   positions  int32 [B, N]            (device; NULL: n.  Values outside [0, max_pos) are clamped and
 *              recorded as FA_ERR_INVALID_ARG in the device status word.)
 *   q_out      bf16 [B, Hq, N, d]      (device, written)
 *   k_out, v_out  bf16 [B, Hkv, N, d], or with expand = 1 [B, Hq, N, d]: head h is key/value head
 *              h / (Hq / Hkv), as fa_fwd takes them  (device, written)
 *   d in {32, 64, 128}; Hkv dividing Hq; rot a multiple of 16, at most d; B * N < 2^31; eps >= 0.
 * Outputs must not overlap inputs.  mean(x^2) is an fp32 sum: where it overflows (elements of about 1e18
 * and more) the row is written as 0, and its gradient is 0.  With eps = 0 a row whose squares are 0 in fp32
 * (zeros, or elements below about 1e-23) has no norm: it becomes NaN or infinite, here and in the gradients.
 */
fa_status fa_qk_norm_rope(const void* q, const void* k, const void* v, const void* q_weight,
                          const void* k_weight, const float* cos_table, const float* sin_table,
                          const int* positions, void* q_out, void* k_out, void* v_out,
                          long long q_stride, long long k_stride, long long v_stride, int B, int N,
                          int Hq, int Hkv, int d, int rot, int max_pos, int interleaved, int expand,
                          float eps, fa_dtype w_dtype, void* stream);

/* Bytes of workspace fa_qk_norm_rope_bwd needs (8192 * d).  0 on invalid arguments. */
size_t fa_qk_norm_rope_bwd_workspace_size(int d);

/*
 * Gradient of fa_qk_norm_rope.  With g the gradient of a rotated head, h = g rotated back, x^ =
 * x / sqrt(mean(x^2) + eps):
 *   grad_w = sum over tokens and heads of h x^,
 *   grad_x = (w h - x^ mean(x^ w h)) / sqrt(mean(x^2) + eps),
 * and with expand = 1 the gradients of a key/value head's copies are added up first (fp32).
 *
 *   grad_q_out, grad_k_out, grad_v_out  grad_out_dtype, shaped as q_out, k_out, v_out (fa_bwd's
 *              outputs; grad_v_out may be NULL, with grad_v)
 *   q, k, weights, tables, positions    as given to the forward
 *   grad_q, grad_k, grad_v  grad_dtype [B, N, heads, d] with token strides  (device, written)
 *   grad_q_weight, grad_k_weight  fp32 [d]  (device, written)
 *   workspace  ws_bytes >= fa_qk_norm_rope_bwd_workspace_size(d), 256-byte aligned; its contents on
 *              entry do not matter.  Calls sharing a workspace must not overlap on the GPU.
 * Every sum is in a fixed order: results are the same from run to run.  grad_w is an fp32 sum, in which a
 * warp adds its rows one after the other (a token in 2432 on 152 SMs) before the warps' sums are joined.
 * Outputs must not overlap inputs.
 * Returns FA_ERR_WORKSPACE if ws_bytes is too small (nothing launched).
 */
fa_status fa_qk_norm_rope_bwd(const void* grad_q_out, const void* grad_k_out, const void* grad_v_out,
                              const void* q, const void* k, const void* q_weight,
                              const void* k_weight, const float* cos_table, const float* sin_table,
                              const int* positions, void* grad_q, void* grad_k, void* grad_v,
                              float* grad_q_weight, float* grad_k_weight, void* workspace,
                              size_t ws_bytes, long long q_stride, long long k_stride,
                              long long grad_q_stride, long long grad_k_stride,
                              long long grad_v_stride, int B, int N, int Hq, int Hkv, int d, int rot,
                              int max_pos, int interleaved, int expand, float eps, fa_dtype w_dtype,
                              fa_dtype grad_out_dtype, fa_dtype grad_dtype, void* stream);

/* Nodes of a tree of drafted tokens, at most. */
#define FA_TREE_MAX_NODES 128

/*
 * Trees of drafted tokens (fa_qk_norm_rope_append, fa_decode_tree, fa_cache_compact): sequence b
 * has p = seqlens[b] cached tokens in cache rows 0 .. p - 1 and n = n_nodes[b] <= T drafted ones in
 * rows p .. p + n - 1.  parents[b][t] < t is the node that node t continues, -1 the last cached
 * token.  n_nodes = NULL: T for every sequence; parents = NULL: a chain (node t continues t - 1).
 * A length or node count out of range (p + n above Nk_max too) is clamped, a parent that is not an
 * earlier node is taken as -1; both are recorded as FA_ERR_INVALID_ARG in the device status word.
 *
 * fa_qk_norm_rope_append: fa_qk_norm_rope for the n nodes of each sequence, node t at position
 * p + (number of its ancestors), its key and value heads written to cache row p + t.
 *
 *   q, k, v    bf16 [B, T, heads, d] with token strides
 *   seqlens    int32 [B], parents int32 [B, T] or NULL, n_nodes int32 [B] or NULL  (device)
 *   q_out      bf16 [B, Hq, T, d]           (device, written; 0 for nodes from n on)
 *   k_cache, v_cache  bf16 [B, Hkv, Nk_max, d]  (device; rows p .. p + n - 1 written, no other; they must
 *              not overlap)
 *   T <= FA_TREE_MAX_NODES (else FA_ERR_UNSUPPORTED); positions past max_pos as in fa_qk_norm_rope.
 */
fa_status fa_qk_norm_rope_append(const void* q, const void* k, const void* v, const void* q_weight,
                                 const void* k_weight, const float* cos_table,
                                 const float* sin_table, const int* seqlens, const int* parents,
                                 const int* n_nodes, void* q_out, void* k_cache, void* v_cache,
                                 long long q_stride, long long k_stride, long long v_stride, int B,
                                 int T, int Hq, int Hkv, int Nk_max, int d, int rot, int max_pos,
                                 int interleaved, float eps, fa_dtype w_dtype, void* stream);

/*
 * Bytes of workspace fa_decode_tree needs on a device with `num_sms` multiprocessors: with rows =
 * Hq / Hkv * T, and s = 2 num_sms and r = rows, or s = num_sms and r = 256 above 128 rows, fp32
 * partial outputs [2 s, r, d], fp32 log-sum-exps [2 s, r] and 16 s bytes of records, each 256-byte
 * aligned, whatever the batch and the lengths.  Pure host function.  0 on invalid arguments.
 */
size_t fa_decode_tree_workspace_size(int Hq, int Hkv, int T, int d, int num_sms);

/*
 * Decode attention for a tree of drafted tokens (above): node t of sequence b attends to the p cached
 * tokens, to itself and to its ancestors,
 *   o[b,h,t,:] = sum_j softmax_j(scale q[b,h,t,:] . K[b,g,j,:]) V[b,g,j,:],  g = h / (Hq / Hkv),
 * over the visible rows j of the cache, lse the log of the sum.  With T = 1 it is
 * fa_decode_splitkv_gqa over p + 1 cached tokens.  The weights that multiply V are rounded to bf16, their
 * sum is not: o is off by up to 2^-8 of sum_j weight_j |V_j|, also where it is written in fp32 (on normally
 * distributed inputs 0.0014 of o, in the root mean square; writing o in bf16 is off by 0.0017).  lse does not
 * depend on it.
 *
 *   q          bf16 [B, Hq, T, d]          (device; fa_qk_norm_rope_append's q_out)
 *   k_cache, v_cache  bf16 [B, Hkv, Nk_max, d]  (device; rows from p + n on are never used, whatever
 *              they hold.  A non-finite key reaches only the rows that see it; a non-finite value of
 *              a visible node may reach every row of its sequence.)
 *   seqlens_k  int32 [B], parents int32 [B, T] or NULL, n_nodes int32 [B] or NULL  (device)
 *   o          o_dtype [B, Hq, T, dv]      (device, written; 0 for nodes from n on)
 *   lse        fp32 [B, Hq, T]             (device, written, -inf for nodes from n on; may be NULL)
 *   workspace  ws_bytes >= fa_decode_tree_workspace_size(Hq, Hkv, T, d, <SMs of the current device>),
 *              256-byte aligned; its contents on entry do not matter.  Calls sharing a workspace must
 *              not overlap on the GPU.
 *   T <= FA_TREE_MAX_NODES (else FA_ERR_UNSUPPORTED), Hq / Hkv * T <= 2^20.
 * The result does not depend on other calls, and is the same from run to run.
 */
fa_status fa_decode_tree(const void* q, const void* k_cache, const void* v_cache,
                         const int* seqlens_k, const int* parents, const int* n_nodes, void* o,
                         float* lse, void* workspace, size_t ws_bytes, int B, int Hq, int Hkv, int T,
                         int Nk_max, int d, int dv, float scale, fa_dtype o_dtype, void* stream);

/*
 * Moves the accepted nodes of each sequence up behind its cached tokens: for every layer, key/value
 * head, and for keys and values, row p + accepted[b][i] goes to row p + i for i < n_accepted[b]; the
 * rows are read before any is written, so any order (and a node named twice) is fine.  Other rows
 * stay as they were.  seqlens_out[b] = p + n_accepted[b].
 *
 *   k_cache, v_cache  bf16 [L, B, Hkv, Nk_max, d]  (device; L layers' caches behind one another; they must
 *              not overlap)
 *   seqlens, n_accepted  int32 [B], accepted int32 [B, T]  (device; 0 <= accepted < T, 0 <= n_accepted
 *              <= T, rows below Nk_max.  An accepted node out of range is not moved, lengths and counts
 *              are clamped; both are recorded as FA_ERR_INVALID_ARG in the device status word.)
 *   seqlens_out  int32 [B]  (device, written; may be NULL; must not overlap the other int32 arrays)
 *   T <= FA_TREE_MAX_NODES (else FA_ERR_UNSUPPORTED), L * B * Hkv < 2^31.
 */
fa_status fa_cache_compact(void* k_cache, void* v_cache, const int* seqlens, const int* accepted,
                           const int* n_accepted, int* seqlens_out, int L, int B, int Hkv,
                           int Nk_max, int d, int dv, int T, void* stream);

/*
 * Attention under score rules (fa_fwd_rules, fa_bwd_rules).  Query i of a sequence sits at position
 * Nk - N + i, key j at position j, query head h reads key/value head g = h / (Hq / Hkv).
 *   Scores:  x = scale * q_i . k_j;  softcap > 0: s = softcap * tanh(x / softcap), softcap = 0: s = x;
 *            then, with slopes, s -= slopes[h] * |Nk - N + i - j|.
 *   Masks:   with causal = 1, key j is hidden from query i if j > Nk - N + i, but for the keys j <
 *            prefix_lens[b], which all queries of sequence b see.  With documents, query i and key j
 *            see each other only in one document: a run of equal numbers documents[b][j] >= 0 along the
 *            keys (a query is where its position is).  A number below 0 is padding, in no document; a
 *            query there, or before position 0, sees nothing.  Two runs of the same number are two
 *            documents.
 *
 *   scale > 0 and softcap >= 0, both finite; scale, 1 / scale, softcap, 1 / softcap and scale / softcap must be
 *   within fp32's normal numbers where they come in (else FA_ERR_INVALID_ARG).
 *   slopes       fp32 [Hq]      (device; slopes and slopes / scale, with a cap slopes / softcap, finite; NULL: no
 *                bias.  Distances are exact up to 2^24.)
 *   documents    int32 [B, Nk]  (device; NULL: one document)
 *   prefix_lens  int32 [B]      (device; NULL: 0.  Without causal it has no effect.  Values outside
 *                [0, Nk] are clamped and recorded as FA_ERR_INVALID_ARG in the device status word.)
 *
 * The cap's tanh is off by up to 1.2e-6 of its value; with a cap of up to 128 it may instead be off by 2e-7, so that a score
 * is off by 2e-7 caps (1e-5 at a cap of 50).
 *
 * A non-finite score of a hidden pair reaches nothing; a finite one of up to 10 caps may decide in which form a cap is taken,
 * within the errors above.  A non-finite q, v or grad_o, or k in the gradient, may reach every row whose 128-row tile
 * meets its own (its weight there is 0, and 0 times NaN is NaN), so rows of padding must be finite too.
 */

/* Bytes of workspace fa_fwd_rules needs with documents, 0 on invalid arguments.  Without documents it needs none. */
size_t fa_fwd_rules_workspace_size(int B, int N);

/*
 * Exact attention forward under score rules:
 *   O[b,h,i,:] = sum_j softmax_j(s_ij) V[b,g,j,:],  lse[b,h,i] = log sum_j exp(s_ij)
 * over the keys j that query i sees; O = 0 and lse = -inf where there are none.  Without rules it is
 * fa_fwd.  Weights are rounded to bf16 for the product with V, also where O is fp32; lse sums them unrounded.
 *
 *   q          bf16 [B, Hq, N, d]        (device)
 *   k, v       bf16 [B, Hkv, Nk, d]      (device)
 *   o          o_dtype [B, Hq, N, d]     (device, written)
 *   lse        fp32 [B, Hq, N]           (device, written; may be NULL)
 *   workspace  with documents: ws_bytes >= fa_fwd_rules_workspace_size(B, N), 256-byte aligned; its
 *              contents on entry do not matter.  Calls sharing a workspace must not overlap on the GPU.
 *              Without documents it may be NULL.
 *   Hkv dividing Hq; d = dv in {32, 64, 128}.
 * The result is the same from run to run.
 */
fa_status fa_fwd_rules(const void* q, const void* k, const void* v, const float* slopes,
                       const int* documents, const int* prefix_lens, void* o, float* lse,
                       void* workspace, size_t ws_bytes, int B, int Hq, int Hkv, int N, int Nk, int d,
                       int dv, int causal, float scale, float softcap, fa_dtype o_dtype, void* stream);

/*
 * Bytes of workspace fa_bwd_rules needs on a device with `num_sms` multiprocessors: fa_bwd's, room for
 * the documents' intervals, and, where key/value heads are few, fp32 sums of dK and dV for parts of
 * their query heads.  Pure host function.  0 on invalid arguments.
 */
size_t fa_bwd_rules_workspace_size(int B, int Hq, int Hkv, int N, int Nk, int d, int num_sms);

/*
 * Gradient of fa_fwd_rules.  With P_ij = exp(s_ij - lse_i) for pairs that see each other and D_i =
 * dO_i . O_i:
 *   dV = P^T dO,  dX_ij = P_ij (dO_i . V_j - D_i) scale (1 - tanh^2(x_ij / softcap)),
 *   dQ = dX K,  dK = dX^T Q,
 * dK and dV added up over the query heads of a key/value head.  The slopes are constants.
 *
 *   q, k, v, o, lse, rules  as given to and returned by the forward, with the same scale and softcap
 *   grad_o     bf16 [B, Hq, N, d]        (device)
 *   grad_q     grad_dtype [B, Hq, N, d], grad_k, grad_v grad_dtype [B, Hkv, Nk, d]  (device, every
 *              element written)
 *   workspace  ws_bytes >= fa_bwd_rules_workspace_size(B, Hq, Hkv, N, Nk, d, <SMs of the current
 *              device>), 256-byte aligned; its contents on entry do not matter.  Calls sharing a
 *              workspace must not overlap on the GPU.
 * P and dX are rounded to bf16 for the products, as in fa_bwd.  grad_q's sums run in whatever order
 * the key tiles come to it, so that it can differ in its last bits from run to run; grad_k and grad_v are
 * summed in a fixed order.  Returns FA_ERR_WORKSPACE if ws_bytes is too small (nothing launched).
 */
fa_status fa_bwd_rules(const void* q, const void* k, const void* v, const void* o, const float* lse,
                       const void* grad_o, const float* slopes, const int* documents,
                       const int* prefix_lens, void* grad_q, void* grad_k, void* grad_v, void* workspace,
                       size_t ws_bytes, int B, int Hq, int Hkv, int N, int Nk, int d, int dv, int causal,
                       float scale, float softcap, fa_dtype o_dtype, fa_dtype grad_dtype, void* stream);

/*
 * Bytes of workspace fa_decode_prefix needs on a device with `num_sms` multiprocessors, whatever the
 * lengths.  Pure host function.  0 on invalid arguments.
 */
size_t fa_decode_prefix_workspace_size(int B, int Hq, int Hkv, int d, int num_sms);

/*
 * Decode attention, one query a sequence, for a batch whose sequences begin with the same P tokens.  With
 * n = seqlens_k[b] tokens of its own, sequence b's query sits at position P + n - 1 and sees the prefix's
 * keys (positions 0 .. P - 1) and its own (P .. P + n - 1):
 *   o[b,h,:] = sum_j softmax_j(s_j) V_j,  lse[b,h] = log sum_j exp(s_j),
 * the scores as under score rules (above).  The prefix's keys and values are read once for the whole batch.
 * The weights that multiply V are rounded to bf16, as in fa_decode_tree.
 *
 *   q          bf16 [B, Hq, 1, d]          (device)
 *   k_prefix, v_prefix  bf16 [Hkv, P_max, d]  (device; both NULL with P_max = 0: no prefix)
 *   prefix_len int32 [1]                   (device; P; NULL: P_max)
 *   k_cache, v_cache  bf16 [B, Hkv, Nk_max, d]  (device)
 *   seqlens_k  int32 [B]                   (device; lengths out of range, P too, are clamped and recorded as
 *              FA_ERR_INVALID_ARG in the device status word.  With no key at all o = 0 and lse = -inf.)
 *   slopes     fp32 [Hq] or NULL           (device)
 *   o          o_dtype [B, Hq, 1, d]       (device, written)
 *   lse        fp32 [B, Hq, 1]             (device, written; may be NULL)
 *   workspace  ws_bytes >= fa_decode_prefix_workspace_size(B, Hq, Hkv, d, <SMs of the current device>),
 *              256-byte aligned; its contents on entry do not matter.  Calls sharing a workspace must not
 *              overlap on the GPU.
 *   Hkv dividing Hq, Hq / Hkv <= 128 (else FA_ERR_UNSUPPORTED).
 * Rows behind P or n are never used, whatever they hold.  The result is the same from run to run.
 */
fa_status fa_decode_prefix(const void* q, const void* k_prefix, const void* v_prefix,
                           const int* prefix_len, const void* k_cache, const void* v_cache,
                           const int* seqlens_k, const float* slopes, void* o, float* lse, void* workspace,
                           size_t ws_bytes, int B, int Hq, int Hkv, int P_max, int Nk_max, int d, int dv,
                           float scale, float softcap, fa_dtype o_dtype, void* stream);

/*
 * Synchronises `stream`, then returns and clears the device status word of the current
 * device: FA_OK if no kernel recorded a failure since the last call, else the first
 * recorded status (FA_ERR_TIMEOUT, FA_ERR_INVALID_ARG).  FA_ERR_CUDA if the synchronisation
 * itself failed.
 */
fa_status fa_get_device_error(void* stream);

/*
 * Upper bound, in nanoseconds of the GPU global timer, on every wait for a barrier inside
 * the forward and backward tensor-core kernels (default 2e9).  When a wait runs out the kernel records FA_ERR_TIMEOUT,
 * drains its own copies in flight, frees its tensor memory and returns.  0 restores the
 * default.  Applies to launches made after the call.
 */
void fa_set_wait_timeout_ns(unsigned long long ns);

/* Static description of a status code. */
const char* fa_status_string(fa_status s);

#ifdef __cplusplus
}
#endif

#endif /* FA_H */

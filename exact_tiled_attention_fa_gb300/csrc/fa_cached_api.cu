// fa_cached_api.cu -- the C ABI of the operators around cached attention (include/fa.h): query/key
// norm with rotation and its gradient, the same written into a cache, decode for a tree of drafted
// tokens, cache compaction.  Argument checks and dispatch, host code only.
#include <cmath>
#include <cstdint>

#include "fa_internal.h"

namespace {

constexpr size_t kAlign = 256;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool head_ok(int d) { return d == 32 || d == 64 || d == 128; }
bool dtype_ok(fa_dtype t) { return t == FA_BF16 || t == FA_F32; }
bool flag_ok(int f) { return f == 0 || f == 1; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Whether two buffers of a and b bytes overlap.
bool overlap(const void* p, size_t a, const void* q, size_t b)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    return x < y + b && y < x + a;
}

// Token stride of `heads` heads of d elements: heads do not overlap the next token's, rows stay on
// 16 bytes (a multiple of 8 elements of either type).
bool stride_ok(long long s, long long heads, int d) { return s >= heads * d && s % 8 == 0; }

// The checks that the norm's forward, backward and cache forms share.
fa_status check_rope(const void* q, const void* k, const void* wq, const void* wk, const float* cos_t, const float* sin_t,
                     const int* positions, long long q_stride, long long k_stride, int B, int N, int Hq, int Hkv, int d,
                     int rot, int max_pos, int interleaved, float eps, fa_dtype w_dtype)
{
    if (q == nullptr || k == nullptr || wq == nullptr || wk == nullptr || cos_t == nullptr || sin_t == nullptr)
        return FA_ERR_INVALID_ARG;
    if (B <= 0 || N <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || rot <= 0 || max_pos <= 0) return FA_ERR_INVALID_ARG;
    if (Hq % Hkv != 0 || rot > d || !flag_ok(interleaved) || !dtype_ok(w_dtype)) return FA_ERR_INVALID_ARG;
    if (!(std::isfinite(eps) && eps >= 0.f)) return FA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(wq, 4) || !aligned(wk, 4) || !aligned(cos_t, 16) ||
        !aligned(sin_t, 16) || !aligned(positions, 4))
        return FA_ERR_INVALID_ARG;
    if (!stride_ok(q_stride, Hq, d) || !stride_ok(k_stride, Hkv, d)) return FA_ERR_INVALID_ARG;
    // tokens index a grid, heads are counted in 32 bits
    if (static_cast<long long>(B) * N > 0x7fffffffLL || Hq > (1 << 20) || Hkv > (1 << 20)) return FA_ERR_INVALID_ARG;
    if (!head_ok(d) || rot % 16 != 0) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

}  // namespace

extern "C" {

fa_status fa_qk_norm_rope(const void* q, const void* k, const void* v, const void* q_weight, const void* k_weight,
                          const float* cos_table, const float* sin_table, const int* positions, void* q_out, void* k_out,
                          void* v_out, long long q_stride, long long k_stride, long long v_stride, int B, int N, int Hq,
                          int Hkv, int d, int rot, int max_pos, int interleaved, int expand, float eps, fa_dtype w_dtype,
                          void* stream)
{
    if (q_out == nullptr || k_out == nullptr || (v == nullptr) != (v_out == nullptr) || !flag_ok(expand))
        return FA_ERR_INVALID_ARG;
    const fa_status bad = check_rope(q, k, q_weight, k_weight, cos_table, sin_table, positions, q_stride, k_stride, B, N, Hq,
                                     Hkv, d, rot, max_pos, interleaved, eps, w_dtype);
    if (bad == FA_ERR_INVALID_ARG) return bad;
    if (!aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(v_out, 16) ||
        (v != nullptr && !stride_ok(v_stride, Hkv, d)))
        return FA_ERR_INVALID_ARG;
    if (bad != FA_OK) return bad;
    fa::RopeParams p{};
    if (fa::device_status_word(&p.status) != cudaSuccess) return FA_ERR_CUDA;
    int sms = 0;
    if (fa::device_sm_count(&sms) != cudaSuccess) return FA_ERR_CUDA;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.wq = q_weight;
    p.wk = k_weight;
    p.cos_t = cos_table;
    p.sin_t = sin_table;
    p.positions = positions;
    p.q_out = q_out;
    p.k_out = k_out;
    p.v_out = v_out;
    p.B = B;
    p.N = N;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.rot = rot;
    p.max_pos = max_pos;
    p.copies = expand ? Hq / Hkv : 1;
    p.eps = eps;
    p.w_dtype = w_dtype;
    return fa::launch_qk_rope(p, d, interleaved != 0, false, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FA_OK
               : FA_ERR_CUDA;
}

size_t fa_qk_norm_rope_bwd_workspace_size(int d)
{
    return d <= 0 ? 0 : round_up(static_cast<size_t>(fa::kRopeBwdCtas) * 2 * d * sizeof(float), kAlign);
}

fa_status fa_qk_norm_rope_bwd(const void* grad_q_out, const void* grad_k_out, const void* grad_v_out, const void* q,
                              const void* k, const void* q_weight, const void* k_weight, const float* cos_table,
                              const float* sin_table, const int* positions, void* grad_q, void* grad_k, void* grad_v,
                              float* grad_q_weight, float* grad_k_weight, void* workspace, size_t ws_bytes,
                              long long q_stride, long long k_stride, long long grad_q_stride, long long grad_k_stride,
                              long long grad_v_stride, int B, int N, int Hq, int Hkv, int d, int rot, int max_pos,
                              int interleaved, int expand, float eps, fa_dtype w_dtype, fa_dtype grad_out_dtype,
                              fa_dtype grad_dtype, void* stream)
{
    if (grad_q_out == nullptr || grad_k_out == nullptr || grad_q == nullptr || grad_k == nullptr ||
        grad_q_weight == nullptr || grad_k_weight == nullptr || workspace == nullptr ||
        (grad_v_out == nullptr) != (grad_v == nullptr))
        return FA_ERR_INVALID_ARG;
    if (!flag_ok(expand) || !dtype_ok(grad_out_dtype) || !dtype_ok(grad_dtype)) return FA_ERR_INVALID_ARG;
    const fa_status bad = check_rope(q, k, q_weight, k_weight, cos_table, sin_table, positions, q_stride, k_stride, B, N, Hq,
                                     Hkv, d, rot, max_pos, interleaved, eps, w_dtype);
    if (bad == FA_ERR_INVALID_ARG) return bad;
    if (!aligned(grad_q_out, 16) || !aligned(grad_k_out, 16) || !aligned(grad_v_out, 16) || !aligned(grad_q, 16) ||
        !aligned(grad_k, 16) || !aligned(grad_v, 16) || !aligned(grad_q_weight, 4) || !aligned(grad_k_weight, 4) ||
        !aligned(workspace, kAlign))
        return FA_ERR_INVALID_ARG;
    if (!stride_ok(grad_q_stride, Hq, d) || !stride_ok(grad_k_stride, Hkv, d) ||
        (grad_v != nullptr && !stride_ok(grad_v_stride, Hkv, d)))
        return FA_ERR_INVALID_ARG;
    if (bad != FA_OK) return bad;
    if (ws_bytes < fa_qk_norm_rope_bwd_workspace_size(d)) return FA_ERR_WORKSPACE;
    fa::RopeBwdParams p{};
    if (fa::device_status_word(&p.status) != cudaSuccess) return FA_ERR_CUDA;
    int sms = 0;
    if (fa::device_sm_count(&sms) != cudaSuccess) return FA_ERR_CUDA;
    p.dq = grad_q_out;
    p.dk = grad_k_out;
    p.dv = grad_v_out;
    p.q = q;
    p.k = k;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.wq = q_weight;
    p.wk = k_weight;
    p.cos_t = cos_table;
    p.sin_t = sin_table;
    p.positions = positions;
    p.gq = grad_q;
    p.gk = grad_k;
    p.gv = grad_v;
    p.gq_stride = grad_q_stride;
    p.gk_stride = grad_k_stride;
    p.gv_stride = grad_v_stride;
    p.gwq = grad_q_weight;
    p.gwk = grad_k_weight;
    p.part = static_cast<float*>(workspace);
    p.B = B;
    p.N = N;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.rot = rot;
    p.max_pos = max_pos;
    p.copies = expand ? Hq / Hkv : 1;
    p.eps = eps;
    p.w_dtype = w_dtype;
    p.g_dtype = grad_out_dtype;
    p.out_dtype = grad_dtype;
    return fa::launch_qk_rope_bwd(p, d, interleaved != 0, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FA_OK
               : FA_ERR_CUDA;
}

fa_status fa_qk_norm_rope_append(const void* q, const void* k, const void* v, const void* q_weight, const void* k_weight,
                                 const float* cos_table, const float* sin_table, const int* seqlens, const int* parents,
                                 const int* n_nodes, void* q_out, void* k_cache, void* v_cache, long long q_stride,
                                 long long k_stride, long long v_stride, int B, int T, int Hq, int Hkv, int Nk_max, int d,
                                 int rot, int max_pos, int interleaved, float eps, fa_dtype w_dtype, void* stream)
{
    if (v == nullptr || seqlens == nullptr || q_out == nullptr || k_cache == nullptr || v_cache == nullptr || Nk_max <= 0)
        return FA_ERR_INVALID_ARG;
    const fa_status bad = check_rope(q, k, q_weight, k_weight, cos_table, sin_table, nullptr, q_stride, k_stride, B, T, Hq,
                                     Hkv, d, rot, max_pos, interleaved, eps, w_dtype);
    if (bad == FA_ERR_INVALID_ARG) return bad;
    if (!aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(seqlens, 4) ||
        !aligned(parents, 4) || !aligned(n_nodes, 4) || !stride_ok(v_stride, Hkv, d))
        return FA_ERR_INVALID_ARG;
    const size_t cache = static_cast<size_t>(B) * Hkv * static_cast<size_t>(Nk_max) * d * 2;
    if (overlap(k_cache, cache, v_cache, cache)) return FA_ERR_INVALID_ARG;
    if (bad != FA_OK) return bad;
    if (T > FA_TREE_MAX_NODES) return FA_ERR_UNSUPPORTED;
    fa::RopeParams p{};
    if (fa::device_status_word(&p.status) != cudaSuccess) return FA_ERR_CUDA;
    int sms = 0;
    if (fa::device_sm_count(&sms) != cudaSuccess) return FA_ERR_CUDA;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.wq = q_weight;
    p.wk = k_weight;
    p.cos_t = cos_table;
    p.sin_t = sin_table;
    p.q_out = q_out;
    p.k_out = k_cache;
    p.v_out = v_cache;
    p.seqlens = seqlens;
    p.parents = parents;
    p.n_nodes = n_nodes;
    p.B = B;
    p.N = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.rot = rot;
    p.max_pos = max_pos;
    p.Nk_max = Nk_max;
    p.copies = 1;
    p.eps = eps;
    p.w_dtype = w_dtype;
    return fa::launch_qk_rope(p, d, interleaved != 0, true, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FA_OK
               : FA_ERR_CUDA;
}

size_t fa_decode_tree_workspace_size(int Hq, int Hkv, int T, int d, int num_sms)
{
    if (Hq <= 0 || Hkv <= 0 || T <= 0 || d <= 0 || num_sms <= 0 || Hq % Hkv != 0) return 0;
    const long long rows = static_cast<long long>(Hq / Hkv) * T;
    const bool pair = rows > fa::kBlockM;  // up to 128 rows: room for either form
    const size_t shares = (pair ? 1 : 2) * static_cast<size_t>(num_sms);
    const size_t slots = 2 * shares * (pair ? 2 * fa::kBlockM : static_cast<size_t>(rows));  // rows of them
    return round_up(slots * d * sizeof(float), kAlign) + round_up(slots * sizeof(float), kAlign) +
           round_up(shares * sizeof(fa::TreeJoin), kAlign);
}

fa_status fa_decode_tree(const void* q, const void* k_cache, const void* v_cache, const int* seqlens_k, const int* parents,
                         const int* n_nodes, void* o, float* lse, void* workspace, size_t ws_bytes, int B, int Hq, int Hkv,
                         int T, int Nk_max, int d, int dv, float scale, fa_dtype o_dtype, void* stream)
{
    if (q == nullptr || k_cache == nullptr || v_cache == nullptr || seqlens_k == nullptr || o == nullptr ||
        workspace == nullptr)
        return FA_ERR_INVALID_ARG;
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || T <= 0 || Nk_max <= 0 || d <= 0 || dv <= 0 || Hq % Hkv != 0)
        return FA_ERR_INVALID_ARG;
    if (!dtype_ok(o_dtype) || !(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
        !aligned(seqlens_k, 4) || !aligned(parents, 4) || !aligned(n_nodes, 4) || !aligned(workspace, kAlign))
        return FA_ERR_INVALID_ARG;
    const long long groups = static_cast<long long>(B) * Hkv;
    const long long rows = static_cast<long long>(Hq / Hkv) * T;
    if (!head_ok(d) || dv != d || T > FA_TREE_MAX_NODES) return FA_ERR_UNSUPPORTED;
    if (rows > (1 << 20) || Nk_max > 0x7fffff00) return FA_ERR_INVALID_ARG;
    const int part = rows > fa::kBlockM ? 2 * fa::kBlockM : static_cast<int>(rows);
    const long long n_qp = (rows + part - 1) / part;
    if (groups * n_qp > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
    int sms = 0;
    if (fa::device_sm_count(&sms) != cudaSuccess) return FA_ERR_CUDA;
    if (ws_bytes < fa_decode_tree_workspace_size(Hq, Hkv, T, d, sms)) return FA_ERR_WORKSPACE;
    fa::TreeParams p{};
    if (!fa::bf16_tile_map(&p.tm_q, q, static_cast<int>(groups), static_cast<int>(rows), d) ||
        !fa::bf16_tile_map(&p.tm_k, k_cache, static_cast<int>(groups), Nk_max, d) ||
        !fa::bf16_tile_map(&p.tm_v, v_cache, static_cast<int>(groups), Nk_max, dv))
        return FA_ERR_CUDA;
    if (fa::device_status_word(&p.status) != cudaSuccess) return FA_ERR_CUDA;
    p.seqlens = seqlens_k;
    p.parents = parents;
    p.n_nodes = n_nodes;
    p.o = o;
    p.lse = lse;
    p.o_part = static_cast<float*>(workspace);
    const bool pair = rows > fa::kBlockM;
    p.num_ctas = sms < fa::kTreeMaxShares / 2 ? sms : fa::kTreeMaxShares / 2;
    // Which form (fa_tree_kernel.cuh).  Measured on GB300, 4 query heads per key/value head, 8 nodes (ALT /
    // SOLO, us).  d = 128, where K and V bound both: 2048 units of at most 400 tokens 113 / 86, 1500 tokens
    // 213 / 202, 4500 tokens 519 / 531; 512 units 37 / 32, 63 / 61, 139 / 144; 384 units 31 / 28, 51 / 49; 256
    // units 23 / 22, 37 / 38; 128 units of 16K 123 / 128.  The lengths are only known on the device: many
    // units are taken to be short ones (at most 4 % lost), fewer only if none can be long.
    // d = 64, where a tile is less to wait for: 2048 units of 1500 tokens 132 / 103, 4500 278 / 263; 128
    // units of 1500 18.3 / 16.4, 16K 67.6 / 66.3 (32 nodes 71.2 / 72.2); 64 units 14.0 / 13.4, but with 32
    // nodes 16.5 / 18.1; 32 units 12.2 / 12.8.  d = 32, 128 units of 16K: 61 / 53; 32 units 11.1 / 12.1.
    const long long units = groups * n_qp;
    const bool solo = !pair && (d < 128 ? 4 * units >= 3LL * p.num_ctas
                                        : units >= 6LL * p.num_ctas || (units >= 2LL * p.num_ctas && Nk_max <= 1536));
    p.num_shares = solo ? 2 * p.num_ctas : p.num_ctas;
    // a unit's start and end took a CTA about three tiles' time (one share's last units of 9 tiles each: the
    // CTA ended 30 us after the others without it), two under the other warpgroup's tiles
    p.unit_cost = solo ? 2 : 3;
    const size_t slots = 2 * static_cast<size_t>(p.num_shares) * part;
    char* at = static_cast<char*>(workspace) + round_up(slots * d * sizeof(float), kAlign);
    p.lse_part = reinterpret_cast<float*>(at);
    p.joins = reinterpret_cast<fa::TreeJoin*>(at + round_up(slots * sizeof(float), kAlign));
    p.B = B;
    p.Hkv = Hkv;
    p.rows = static_cast<int>(rows);
    p.T = T;
    p.Nk_max = Nk_max;
    p.part_rows = part;
    p.n_qp = static_cast<int>(n_qp);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.o_dtype = o_dtype;
    p.wait_limit_ns = fa::wait_limit_ns();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = d == 32 ? fa::launch_tree_32(p, st) : d == 64 ? fa::launch_tree_64(p, st) : fa::launch_tree_128(p, st);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_cache_compact(void* k_cache, void* v_cache, const int* seqlens, const int* accepted, const int* n_accepted,
                           int* seqlens_out, int L, int B, int Hkv, int Nk_max, int d, int dv, int T, void* stream)
{
    if (k_cache == nullptr || v_cache == nullptr || seqlens == nullptr || accepted == nullptr || n_accepted == nullptr)
        return FA_ERR_INVALID_ARG;
    if (L <= 0 || B <= 0 || Hkv <= 0 || Nk_max <= 0 || d <= 0 || dv <= 0 || T <= 0) return FA_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(seqlens, 4) || !aligned(accepted, 4) ||
        !aligned(n_accepted, 4) || !aligned(seqlens_out, 4))
        return FA_ERR_INVALID_ARG;
    if (static_cast<long long>(L) * B > 0x7fffffffLL / Hkv) return FA_ERR_INVALID_ARG;
    // lengths and counts are read by every CTA and written by one: not in place
    const size_t b4 = static_cast<size_t>(B) * sizeof(int);
    if (seqlens_out != nullptr && (overlap(seqlens_out, b4, seqlens, b4) || overlap(seqlens_out, b4, n_accepted, b4) ||
                                   overlap(seqlens_out, b4, accepted, b4 * static_cast<size_t>(T))))
        return FA_ERR_INVALID_ARG;
    const size_t cache = static_cast<size_t>(L) * B * Hkv * static_cast<size_t>(Nk_max) * d * 2;
    if (overlap(k_cache, cache, v_cache, cache)) return FA_ERR_INVALID_ARG;
    if (!head_ok(d) || dv != d || T > FA_TREE_MAX_NODES) return FA_ERR_UNSUPPORTED;
    fa::CompactParams p{};
    if (fa::device_status_word(&p.status) != cudaSuccess) return FA_ERR_CUDA;
    p.k = k_cache;
    p.v = v_cache;
    p.seqlens = seqlens;
    p.accepted = accepted;
    p.n_accepted = n_accepted;
    p.seqlens_out = seqlens_out;
    p.L = L;
    p.B = B;
    p.Hkv = Hkv;
    p.Nk_max = Nk_max;
    p.d = d;
    p.T = T;
    return fa::launch_cache_compact(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"

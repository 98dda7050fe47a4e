// fa_rules_api.cu -- the C ABI of attention under score rules (include/fa.h): forward, backward, decode behind
// a shared prefix.  Argument checks, workspace layout and dispatch, host code only.
#include <cmath>
#include <cstdint>
#include <limits>
#include <type_traits>

#include "fa_internal.h"
#include "fa_rules_common.cuh"

namespace {

constexpr size_t kAlign = 256;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool head_ok(int d) { return d == 32 || d == 64 || d == 128; }
bool dtype_ok(fa_dtype t) { return t == FA_BF16 || t == FA_F32; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int tiles_of(int n) { return static_cast<int>((static_cast<long long>(n) + fa::kBlockM - 1) / fa::kBlockM); }

// Documents' part of a workspace: a counter of work items, an interval for each of B * n rows and for each tile of them.
size_t ranges_size(int B, int n)
{
    return kAlign + round_up(static_cast<size_t>(B) * n * sizeof(int2), kAlign) +
           round_up(static_cast<size_t>(B) * tiles_of(n) * sizeof(int2), kAlign);
}

struct Ranges {
    int* counter;
    int2 *each, *tile;
    Ranges(char* at, int B, int n)
        : counter(reinterpret_cast<int*>(at)),
          each(reinterpret_cast<int2*>(at + kAlign)),
          tile(reinterpret_cast<int2*>(at + kAlign + round_up(static_cast<size_t>(B) * n * sizeof(int2), kAlign)))
    {
    }
};

// Scale and cap as the kernels take them (`forward`: the polynomials with mult in them, unless there is a bias); false
// for a cap or scale that fp32 cannot hold so.
bool make_rules(fa::ScoreRules* r, float scale, float softcap, const float* slopes, bool forward)
{
    if (!(std::isfinite(scale) && scale > 0.f) || !(std::isfinite(softcap) && softcap >= 0.f)) return false;
    r->cap_in = softcap > 0.f ? scale / softcap : 0.f;
    r->mult = (softcap > 0.f ? softcap : scale) * fa::kLog2e;
    r->slopes = slopes;
    r->bias_in = fa::kLog2e / r->mult;
    auto normal = [](float x) { return std::isfinite(x) && x >= std::numeric_limits<float>::min(); };
    if (!normal(r->mult) || (softcap > 0.f && !normal(r->cap_in)) || (slopes != nullptr && !normal(r->bias_in))) return false;
    r->far = softcap > fa::kFarCap;
    r->near_in = r->mid_in = r->wide_in = INFINITY;
    const double near[] = {FA_TANH_NEAR}, mid[] = {FA_TANH_MID}, wide[] = {FA_TANH_WIDE}, k = r->cap_in;
    if (softcap == 0.f || k > 1e2) return true;  // (above, powers of cap_in up to the eleventh leave fp32)
    // Below 1e-5 and 8e-4 the seventh and the eleventh power come near fp32's least.  The near polynomial is then taken
    // alone: where its own higher terms vanish they are below 1e-7 of scores up to 10^6.
    const bool low = k < 1e-5;
    double at = k * (forward && slopes == nullptr ? r->mult : 1.0);
    for (int i = 0; i < 6; ++i, at *= k * k) {
        auto twice = [&](double c) { return make_float2(static_cast<float>(c * at), static_cast<float>(c * at)); };
        if (i < 3) r->near[i] = twice(near[i]);
        if (i < 4) r->mid[i] = twice(!low ? mid[i] : i < 3 ? near[i] : 0.0);
        r->wide[i] = twice(wide[i]);
    }
    r->near_in = r->cap_in / fa::kNearRange;
    if (!low) r->mid_in = r->cap_in / fa::kMidRange;
    if (k >= 8e-4) r->wide_in = r->cap_in / fa::kWideRange;
    return true;
}

// f with the head size and the kind of rules as constants.
template <typename F>
cudaError_t by_kind(int d, const fa::ScoreRules& r, F f)
{
    auto kinds = [&](auto D) {
        using std::integral_constant;
        switch (fa::rule_kind(r)) {
        case 0: return f(D, integral_constant<int, 0>());
        case 1: return f(D, integral_constant<int, 1>());
        case 2: return f(D, integral_constant<int, 2>());
        default: return f(D, integral_constant<int, 3>());
        }
    };
    return d == 32 ? kinds(std::integral_constant<int, 32>()) : d == 64 ? kinds(std::integral_constant<int, 64>())
                                                                        : kinds(std::integral_constant<int, 128>());
}

// The checks that forward and backward share.
fa_status check_rules(const void* q, const void* k, const void* v, const float* slopes, const int* documents, const int* prefix_lens,
                      int B, int Hq, int Hkv, int N, int Nk, int d, int dv, int causal, float scale, float softcap)
{
    if (q == nullptr || k == nullptr || v == nullptr) return FA_ERR_INVALID_ARG;
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || Nk <= 0 || d <= 0 || dv <= 0) return FA_ERR_INVALID_ARG;
    if (Hq % Hkv != 0 || (causal != 0 && causal != 1)) return FA_ERR_INVALID_ARG;
    fa::ScoreRules r;
    if (!make_rules(&r, scale, softcap, slopes, true)) return FA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(slopes, 4) || !aligned(documents, 4) || !aligned(prefix_lens, 4))
        return FA_ERR_INVALID_ARG;
    // positions and tile indices are 32-bit, with room for a tile and for a look ahead (fa_rules_ranges.cuh) past the end
    if (N > 0x7fff0000 || Nk > 0x7fff0000) return FA_ERR_INVALID_ARG;
    const long long tiles = static_cast<long long>(B) * Hq * (tiles_of(N) > tiles_of(Nk) ? tiles_of(N) : tiles_of(Nk));
    if (static_cast<long long>(B) * Hq > 0x3fffffffLL || tiles > 0x3fffffffLL) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

// As many of `heads` at a time as the L2 (129 MB) holds the data of, `bytes` each, but at least kAtOnce: with fewer
// heads than CTAs some share what they read all the same.  In chunks of one size.  (4 sequences of 4097 tokens, 16 heads,
// causal: forward d = 64 all 64 heads at once 155 us, 44 181; d = 128 285, 32 heads 303; backward d = 128 799, 15 heads
// 844.  64 sequences of 1024, d = 64: 128, 183 and single heads within 2 %.)
constexpr long long kAtOnce = 100;
int chunk_of(long long heads, long long bytes)
{
    long long n = (96LL << 20) / bytes;
    if (n < kAtOnce) n = kAtOnce;
    const long long chunks = (heads + n - 1) / n;
    return static_cast<int>((heads + chunks - 1) / chunks);
}

// Items of the backward that share a key tile's R query heads: the number for which an estimate of the longest CTA's
// time is least, counted in steps of one query tile with one key tile (about 0.008 d us).  Equal items (`uniform`: no
// causal mask and no documents) come in rounds of one for each CTA; others are handed out one by one, and the
// last to end is up to the longest item behind the mean.  An item's start and end take 3 steps; the
// parts' sums go out and in again, half of it past the L2.  Measured, us for 1 / 2 / 4 parts, causal but the last: 32/4
// heads of 128, 8192 tokens 2575 / 1931 / 1631; 16/4, 4097 tokens 443 / 431 / 339; 8 sequences of 1024, 32/8 heads
// 349 / 377 / -; without a mask 2048 tokens, 32/8 heads 218 / - / 238.
int bwd_parts(int B, int Hkv, int R, int N, int Nk, bool uniform, int sms)
{
    const double groups = static_cast<double>(B) * Hkv, Tr = tiles_of(N), Tc = tiles_of(Nk);
    int best = 1;
    double least = INFINITY;
    for (int heads = R; heads >= 1; heads = heads > 8 ? heads / 2 : heads - 1) {
        const int parts = (R + heads - 1) / heads;
        const double items = groups * parts * Tc, item = heads * Tr + 3;
        const double sums = parts > 1 ? parts * groups * Nk * 1.5e-4 : 0;
        const double steps = uniform ? std::ceil(items / sms) * item : (groups * R * Tr * Tc / 2 + 3 * items) / sms + item;
        if (steps + sums < least) least = steps + sums, best = parts;
    }
    return best;
}

}  // namespace

extern "C" {

size_t fa_fwd_rules_workspace_size(int B, int N)
{
    return B <= 0 || N <= 0 ? 0 : ranges_size(B, N);
}

fa_status fa_fwd_rules(const void* q, const void* k, const void* v, const float* slopes, const int* documents,
                       const int* prefix_lens, void* o, float* lse, void* workspace, size_t ws_bytes, int B, int Hq, int Hkv,
                       int N, int Nk, int d, int dv, int causal, float scale, float softcap, fa_dtype o_dtype, void* stream)
{
    const fa_status bad = check_rules(q, k, v, slopes, documents, prefix_lens, B, Hq, Hkv, N, Nk, d, dv, causal, scale, softcap);
    if (bad != FA_OK) return bad;
    if (o == nullptr || !dtype_ok(o_dtype) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, kAlign))
        return FA_ERR_INVALID_ARG;
    if (documents != nullptr && workspace == nullptr) return FA_ERR_INVALID_ARG;
    if (!head_ok(d) || dv != d) return FA_ERR_UNSUPPORTED;
    if (documents != nullptr && ws_bytes < fa_fwd_rules_workspace_size(B, N)) return FA_ERR_WORKSPACE;
    fa::FwdRulesParams p{};
    make_rules(&p.rules, scale, softcap, slopes, true);
    fa::FwdParams& f = p.f;
    if (!fa::bf16_tile_map(&f.tm_q, q, B * Hq, N, d) || !fa::bf16_tile_map(&f.tm_k, k, B * Hkv, Nk, d) ||
        !fa::bf16_tile_map(&f.tm_v, v, B * Hkv, Nk, dv) || !fa::out_tile_map(&f.tm_o, o, B * Hq, N, dv, o_dtype, 32))
        return FA_ERR_CUDA;
    if (fa::device_status_word(&f.status) != cudaSuccess || fa::device_sm_count(&f.num_ctas) != cudaSuccess) return FA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    f.o = o;
    f.lse = lse;
    f.BH = B * Hq;
    f.N = N;
    f.Nk = Nk;
    f.n_qp = (tiles_of(N) + 1) / 2;
    f.n_items = f.BH * f.n_qp;
    f.wait_limit_ns = fa::wait_limit_ns();
    f.n_splits = 1;
    p.prefix = prefix_lens;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.causal = causal;
    p.chunk = chunk_of(B * Hkv, 4LL * Nk * d) * (Hq / Hkv);
    if (documents != nullptr) {
        const Ranges r(static_cast<char*>(workspace), B, N);
        const fa::RangesParams rp{documents, prefix_lens, r.each, r.tile, r.counter, f.status, B, N, Nk, tiles_of(N), causal};
        if (fa::launch_rules_ranges(rp, st) != cudaSuccess) return FA_ERR_CUDA;
        p.each = r.each;
        p.tile = r.tile;
        p.counter = r.counter;
    }
    const cudaError_t e = by_kind(d, p.rules, [&](auto D, auto kind) { return fa::launch_fwd_rules<D(), kind()>(p, o_dtype, st); });
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_bwd_rules_workspace_size(int B, int Hq, int Hkv, int N, int Nk, int d, int num_sms)
{
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || Nk <= 0 || d <= 0 || num_sms <= 0 || Hq % Hkv != 0) return 0;
    const int even = bwd_parts(B, Hkv, Hq / Hkv, N, Nk, true, num_sms), other = bwd_parts(B, Hkv, Hq / Hkv, N, Nk, false, num_sms);
    const int parts = even > other ? even : other;  // whatever the masks
    const size_t sums = parts > 1 ? 2 * round_up(static_cast<size_t>(parts) * B * Hkv * Nk * d * sizeof(float), kAlign) : 0;
    return fa_bwd_workspace_size(B, Hq, N, d) + ranges_size(B, Nk) + sums;
}

fa_status fa_bwd_rules(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* grad_o,
                       const float* slopes, const int* documents, const int* prefix_lens, void* grad_q, void* grad_k,
                       void* grad_v, void* workspace, size_t ws_bytes, int B, int Hq, int Hkv, int N, int Nk, int d, int dv,
                       int causal, float scale, float softcap, fa_dtype o_dtype, fa_dtype grad_dtype, void* stream)
{
    const fa_status bad = check_rules(q, k, v, slopes, documents, prefix_lens, B, Hq, Hkv, N, Nk, d, dv, causal, scale, softcap);
    if (bad != FA_OK) return bad;
    if (o == nullptr || lse == nullptr || grad_o == nullptr || grad_q == nullptr || grad_k == nullptr || grad_v == nullptr ||
        workspace == nullptr || !dtype_ok(o_dtype) || !dtype_ok(grad_dtype))
        return FA_ERR_INVALID_ARG;
    if (!aligned(o, 16) || !aligned(lse, 4) || !aligned(grad_o, 16) || !aligned(grad_q, 16) || !aligned(grad_k, 16) ||
        !aligned(grad_v, 16) || !aligned(workspace, kAlign))
        return FA_ERR_INVALID_ARG;
    if (!head_ok(d) || dv != d) return FA_ERR_UNSUPPORTED;
    fa::BwdRulesParams p{};
    make_rules(&p.rules, scale, softcap, slopes, false);
    fa::BwdParams& b = p.b;
    if (fa::device_status_word(&b.status) != cudaSuccess || fa::device_sm_count(&b.num_ctas) != cudaSuccess) return FA_ERR_CUDA;
    if (ws_bytes < fa_bwd_rules_workspace_size(B, Hq, Hkv, N, Nk, d, b.num_ctas)) return FA_ERR_WORKSPACE;
    const int R = Hq / Hkv, Tr = tiles_of(N), Tc = tiles_of(Nk);
    const int parts = bwd_parts(B, Hkv, R, N, Nk, causal == 0 && documents == nullptr, b.num_ctas);
    // workspace: fa_bwd's (dQ accumulator, log-sum-exps, row terms), the documents' ranges, the parts' sums
    char* ws = static_cast<char*>(workspace);
    const size_t rows = static_cast<size_t>(B) * Hq * Tr * fa::kBlockM;
    float* dq_acc = reinterpret_cast<float*>(ws);
    float* lse2 = reinterpret_cast<float*>(ws + round_up(rows * d * sizeof(float), kAlign));
    float* dsc = reinterpret_cast<float*>(reinterpret_cast<char*>(lse2) + round_up(rows * sizeof(float), kAlign));
    ws += fa_bwd_workspace_size(B, Hq, N, d);
    const Ranges r(ws, B, Nk);
    ws += ranges_size(B, Nk);
    const size_t n_sum = static_cast<size_t>(B) * Hkv * Nk * d;
    float* dk_part = reinterpret_cast<float*>(ws);
    float* dv_part = reinterpret_cast<float*>(ws + round_up(parts * n_sum * sizeof(float), kAlign));
    void* dk = parts > 1 ? static_cast<void*>(dk_part) : grad_k;
    void* dv_ = parts > 1 ? static_cast<void*>(dv_part) : grad_v;
    const fa_dtype kv_type = parts > 1 ? FA_F32 : grad_dtype;
    if (static_cast<long long>(B) * Hkv * parts * Tc > 0x3fffffffLL) return FA_ERR_INVALID_ARG;
    if (!fa::bf16_tile_map(&b.tm_q, q, B * Hq, N, d) || !fa::bf16_tile_map(&b.tm_k, k, B * Hkv, Nk, d) ||
        !fa::bf16_tile_map(&b.tm_v, v, B * Hkv, Nk, dv) || !fa::bf16_tile_map(&b.tm_do, grad_o, B * Hq, N, dv) ||
        !fa::out_tile_map(&b.tm_dk, dk, B * Hkv * parts, Nk, d, kv_type, fa::kBlockM) ||
        !fa::out_tile_map(&b.tm_dv, dv_, B * Hkv * parts, Nk, dv, kv_type, fa::kBlockM))
        return FA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const fa::BwdPrepParams pp{o, grad_o, lse, lse2, dsc, dq_acc, B * Hq, N, Tr, d, scale, r.counter};
    if (documents != nullptr) {
        const fa::RangesParams rp{documents, prefix_lens, r.each, r.tile, nullptr, b.status, B, N, Nk, Tc, causal};
        if (fa::launch_bwd_prep_ranges(pp, rp, o_dtype, st) != cudaSuccess) return FA_ERR_CUDA;
        p.each = r.each;
        p.tile = r.tile;
    } else if (fa::launch_bwd_prep(pp, o_dtype, st) != cudaSuccess) {
        return FA_ERR_CUDA;
    }
    b.lse2 = lse2;
    b.dsc = dsc;
    b.dq_acc = dq_acc;
    b.dk = dk;
    b.dv = dv_;
    b.BH = B * Hq;
    b.N = N;
    b.Nk = Nk;
    b.Tr = Tr;
    b.Tc = Tc;
    b.scale = scale;
    b.wait_limit_ns = fa::wait_limit_ns();
    p.prefix = prefix_lens;
    p.counter = r.counter;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.causal = causal;
    p.parts = parts;
    p.part_heads = (R + parts - 1) / parts;  // (at most the heads that this number of parts was made from)
    p.n_items = B * Hkv * parts * Tc;
    p.chunk = causal != 0 || documents != nullptr ? chunk_of(B * Hkv * parts, 8LL * N * d * p.part_heads) : 1;
    const cudaError_t e = by_kind(d, p.rules, [&](auto D, auto kind) { return fa::launch_bwd_rules<D(), kind()>(p, kv_type, st); });
    if (e != cudaSuccess) return FA_ERR_CUDA;
    fa::BwdDqParams dp{dq_acc, grad_q, B * Hq, N, Tr, d};
    if (parts > 1) {
        dp.dk_part = dk_part;
        dp.dv_part = dv_part;
        dp.dk = grad_k;
        dp.dv = grad_v;
        dp.n_sum = static_cast<long long>(n_sum);
        dp.parts = parts;
    }
    return fa::launch_bwd_dq(dp, grad_dtype, st) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"

namespace {

// How a call of fa_decode_prefix is divided and where its workspace holds what.
struct PrefixPlan {
    int R, seqs, n_qp;  // rows of a group, sequences of a query tile of the prefix, such tiles
    int ctas, part_rows, units_pre, units_own;
    size_t o_part, lse_part, whole, whole_lse, joins, total;  // offsets; whole: of both sides
    PrefixPlan(int B, int Hq, int Hkv, int d, int sms)
    {
        R = Hq / Hkv;
        seqs = fa::kBlockM / R < B ? fa::kBlockM / R : B;
        n_qp = (B + seqs - 1) / seqs;
        ctas = sms < fa::kTreeMaxShares / 2 ? sms : fa::kTreeMaxShares / 2;
        part_rows = seqs * R;
        units_pre = Hkv * n_qp;
        units_own = B * Hkv;
        // two slots a share, up to two shares a CTA
        const size_t slots = 4 * static_cast<size_t>(ctas) * part_rows, rows = static_cast<size_t>(B) * Hq;
        const size_t row = static_cast<size_t>(d) * sizeof(float);
        size_t at = 0;
        auto take = [&](size_t bytes) {
            const size_t x = at;
            at += round_up(bytes, kAlign);
            return x;
        };
        o_part = take(slots * row);
        lse_part = take(slots * sizeof(float));
        whole = take(2 * rows * row);
        whole_lse = take(2 * rows * sizeof(float));
        joins = take((static_cast<size_t>(units_pre) + units_own) * sizeof(fa::TreeJoin));
        total = at;
    }
};

bool prefix_sizes_ok(int B, int Hq, int Hkv, int d)
{
    return B > 0 && Hq > 0 && Hkv > 0 && d > 0 && Hq % Hkv == 0 && static_cast<long long>(B) * Hq <= 0x3fffffffLL;
}

}  // namespace

extern "C" {

size_t fa_decode_prefix_workspace_size(int B, int Hq, int Hkv, int d, int num_sms)
{
    if (!prefix_sizes_ok(B, Hq, Hkv, d) || num_sms <= 0 || Hq / Hkv > fa::kBlockM) return 0;
    return PrefixPlan(B, Hq, Hkv, d, num_sms).total;
}

fa_status fa_decode_prefix(const void* q, const void* k_prefix, const void* v_prefix, const int* prefix_len, const void* k_cache,
                           const void* v_cache, const int* seqlens_k, const float* slopes, void* o, float* lse, void* workspace,
                           size_t ws_bytes, int B, int Hq, int Hkv, int P_max, int Nk_max, int d, int dv, float scale, float softcap,
                           fa_dtype o_dtype, void* stream)
{
    if (q == nullptr || k_cache == nullptr || v_cache == nullptr || seqlens_k == nullptr || o == nullptr || workspace == nullptr)
        return FA_ERR_INVALID_ARG;
    // a prefix, or none
    const bool pre = k_prefix != nullptr;
    if (pre != (v_prefix != nullptr) || (pre ? P_max <= 0 : P_max != 0 || prefix_len != nullptr)) return FA_ERR_INVALID_ARG;
    if (!prefix_sizes_ok(B, Hq, Hkv, d) || dv <= 0 || Nk_max <= 0 || !dtype_ok(o_dtype)) return FA_ERR_INVALID_ARG;
    fa::ScoreRules rules;
    if (!make_rules(&rules, scale, softcap, slopes, true)) return FA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_prefix, 16) || !aligned(v_prefix, 16) || !aligned(prefix_len, 4) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(seqlens_k, 4) || !aligned(slopes, 4) || !aligned(o, 16) || !aligned(lse, 4) ||
        !aligned(workspace, kAlign))
        return FA_ERR_INVALID_ARG;
    if (P_max > 0x3fffff00 || Nk_max > 0x3fffff00) return FA_ERR_INVALID_ARG;  // positions behind both are 32-bit
    if (!head_ok(d) || dv != d || Hq / Hkv > fa::kBlockM) return FA_ERR_UNSUPPORTED;
    // the kernel counts tiles, and a few more for each unit, in 32 bits
    const double units_most = static_cast<double>(B) * Hkv, tiles_most = units_most * (tiles_of(Nk_max) + tiles_of(P_max) + 8.0);
    if (tiles_most > 0x3fffffff) return FA_ERR_INVALID_ARG;
    int sms = 0;
    if (fa::device_sm_count(&sms) != cudaSuccess) return FA_ERR_CUDA;
    const PrefixPlan plan(B, Hq, Hkv, d, sms);
    if (ws_bytes < plan.total) return FA_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    auto at = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
    const size_t rows = static_cast<size_t>(B) * Hq;
    fa::PrefixParams p{};
    const int n_pre = pre ? plan.units_pre : 0;
    const long long units = static_cast<long long>(n_pre) + plan.units_own;
    // Which form (ALT / SOLO, us).  d = 128, where SOLO's K and V come in halves: 2 sequences behind 512 tokens 12.8 / 11.1,
    // 16 behind 8192 38.6 / 31.8, 64 behind 32K 114 / 103 (SharedWalk: 88), 64 without a prefix 63.8 / 50.9.  d = 64, 5 heads, 37 sequences
    // behind 3000 tokens 19.7 / 21.7, without a prefix 19.0 / 15.5; 8 heads, 64 sequences behind 32K 68 / 53.
    const bool solo = d == 128 || (pre ? units >= 2LL * plan.ctas : 4 * units >= 3LL * plan.ctas);
    const int box = solo && d == 128 ? fa::kBlockN / 2 : fa::kBlockN;  // TrCfg::kHalves
    if (!fa::bf16_group_map(&p.tm_q1, q, B, Hkv, plan.R, d, 1) || !fa::bf16_tile_map(&p.tm_k, k_cache, B * Hkv, Nk_max, d, box) ||
        !fa::bf16_tile_map(&p.tm_v, v_cache, B * Hkv, Nk_max, dv, box))
        return FA_ERR_CUDA;
    if (pre && (!fa::bf16_group_map(&p.tm_q, q, B, Hkv, plan.R, d, plan.seqs) || !fa::bf16_tile_map(&p.tm_kp, k_prefix, Hkv, P_max, d, box) ||
                !fa::bf16_tile_map(&p.tm_vp, v_prefix, Hkv, P_max, dv, box)))
        return FA_ERR_CUDA;
    if (fa::device_status_word(&p.status) != cudaSuccess) return FA_ERR_CUDA;
    p.seqlens = seqlens_k;
    p.o = o;
    p.lse = lse;
    p.B = B;
    p.Hkv = Hkv;
    p.rows = plan.R;
    p.T = 1;
    p.Nk_max = Nk_max;
    p.num_ctas = plan.ctas;
    p.o_dtype = o_dtype;
    p.wait_limit_ns = fa::wait_limit_ns();
    p.prefix_len = prefix_len;
    p.rules = rules;
    p.P_max = P_max;
    p.R = plan.R;
    p.seqs = plan.seqs;
    p.rows_all = B * plan.R;
    p.scale_log2 = rules.mult;
    p.o_pre = at(plan.whole);
    p.lse_pre = at(plan.whole_lse);
    p.o_own = pre ? p.o_pre + rows * d : nullptr;
    p.lse_own = pre ? p.lse_pre + rows : nullptr;
    fa::TreeJoin* joins = reinterpret_cast<fa::TreeJoin*>(ws + plan.joins);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    p.joins = joins;
    p.o_part = at(plan.o_part);
    p.lse_part = at(plan.lse_part);
    p.part_rows = plan.part_rows;
    p.n_qp = plan.n_qp;
    p.n_pre = n_pre;
    p.num_shares = solo ? 2 * plan.ctas : plan.ctas;
    p.unit_cost = solo ? 2 : 3;  // as fa_decode_tree
    if (by_kind(d, rules, [&](auto D, auto kind) { return fa::launch_prefix<D(), kind()>(p, st); }) != cudaSuccess) return FA_ERR_CUDA;
    fa::PrefixMergeParams m{};
    m.own = fa::PrefixSide{joins + n_pre, p.o_own, p.lse_own};
    if (pre) m.pre = fa::PrefixSide{joins, p.o_pre, p.lse_pre};
    m.o_part = p.o_part;
    m.lse_part = p.lse_part;
    m.part_rows = p.part_rows;
    m.num_shares = p.num_shares;
    m.o = o;
    m.lse = lse;
    m.B = B;
    m.Hkv = Hkv;
    m.R = plan.R;
    m.seqs = plan.seqs;
    m.n_qp = plan.n_qp;
    m.o_dtype = o_dtype;
    return fa::launch_prefix_merge(m, d, st) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"

// fa_rules_bwd_kernel.cuh -- exact attention backward under score rules, for sm_103a.
//
// Mathematics.  Scores are those of fa_rules_fwd_kernel.cuh, s = cap tanh(x / cap) - slope_h |distance|, x = scale q.k;
// the slopes are constants.  With P = exp(s - LSE) for a pair that sees each other, else 0, and D_i = dO_i . O_i:
//   dV_j = sum_i P dO_i,  dP = dO_i . V_j,  dS = P (dP - D_i),  dX = dS (1 - tanh^2(x / cap)) scale,
//   dQ_i = sum_j dX K_j,  dK_j = sum_i dX Q_i,
// the sums of dK and dV over all query heads of the key/value head.  What sees a key is one interval of queries
// (fa_rules_ranges.cuh): a key tile visits one run of query tiles and only its first and last ones are masked.
//
// The tiles, roles, tensor memory, pipeline and bounded waits are those of fa_bwd_kernel.cuh (a work item is a
// 128-key tile whose dK and dV stay in tensor memory while Q and dO tiles pass by).  What differs:
//  - An item is a key tile of a key/value head and walks the query tiles of several of its query heads, one head
//    after the other, so that their dK and dV are added up in tensor memory.  With few items (long sequences with few
//    key/value heads) a group's query heads are divided over `parts` items, whose fp32 dK and dV the last kernel adds
//    up in order.
//  - Items' lengths depend on masks and documents: each CTA asks a counter for its next one.  Where they differ, they
//    go out key tile by key tile (with a causal mask the longest first) over as many heads at a time as the L2 holds
//    the Q, dO and dQ of, so that short ones fill the end: causal, 4097 tokens, 16 heads of 64 and 128 head by head 151
//    and 287 us, so 111 and 212.  (64 sequences of 1024 tokens, whose 268 MB of Q and dO the L2 does not hold, all at
//    once 740 us, head by head 613; chunk_of in fa_rules_api.cu.)  The producer hands items to the other roles by
//    records in shared memory.
//  - P's recomputation has the cap and the bias, and dS the cap's slope, made beside P from the same tanh.
//
// What bounds it, by the times of a CTA's steps (cycles, no rules).  d = 64: 2700 a step, of which the compute warps are
// busy 2350 (P 1200, about 500 more where pairs are hidden, dS 1150), and some 4500 more an item from its last dS to its
// successor's first P (last products, dK and dV on their way out).  d = 128: 5180 a step, 2900 of them products; P and dS
// take 1800, but dQ lies in dP's columns: dP 870, dS 880, dK 650, dQ 710, its reductions 1390 (64 KB at 64 bytes a cycle
// to the L2), the next dP 580 later.  4 sequences of 4097 tokens, 16 heads, causal, none / bias / cap of 50 / both: d = 64
// 410 / 454 / 519 / 639 us, d = 128 788 / 820 / 834 / 954.  Capped so for scores of deviation 3; deviation 10, beyond the middle
// range (the wide polynomial is not used here): d = 64 660, both rules 751, d = 128 935 and 1048.
// Bytes stored and loaded that spill: d = 128 48/48 (no rules), 56/52 (bias, cap), 32/32 - 52/68 (both); d <= 64 up to 8/32 with a
// cap, 36/44 with both rules.
#pragma once

#include "fa_bwd_kernel.cuh"
#include "fa_rules_common.cuh"

namespace fa {

// A work item as the producer hands it to the other roles; kv < 0: no more items.
struct RulesBwdItem {
    int kv, b, out;       // key/value head, sequence, head of the output (kv, or in a part's partial sums)
    int bh0, heads;       // first query head, query heads
    int j0, i_first, n;   // first key; query tiles i_first .. i_first + n - 1 of each of the heads
    int prefix;           // of the sequence
};
enum : int { kBbItemFull = kBbCount, kBbItemEmpty = kBbItemFull + kRulesItems, kRulesBbCount = kBbItemEmpty + kRulesItems };

// Registers after the split (fa_bwd_kernel.cuh): with its 184 / 80 / 64 the control and dQ warps spill up to 290 bytes.
constexpr int kRulesBwdComputeRegs = 168;
constexpr int kRulesBwdControlRegs = 104;
constexpr int kRulesBwdDqRegs = 72;

template <int D>
struct RulesBwdCfg : BwdCfg<D> {
    using Base = BwdCfg<D>;
    // the barriers are Base's and then these records' (kOffBar is the last thing in Base's layout but 16 bytes)
    static constexpr int kNumBars = kRulesBbCount;
    static constexpr int kOffItems = (Base::kOffBar + kNumBars * 8 + 16 + 15) / 16 * 16;
    static constexpr int kUsed = kOffItems + kRulesItems * static_cast<int>(sizeof(RulesBwdItem));
    static constexpr int kSmem = kUsed + 1024 <= Base::kMaxSmem ? kUsed + 1024 : Base::kMaxSmem;  // slack as in BwdCfg
    static_assert(kUsed <= Base::kMaxSmem, "shared memory");
};

__device__ __forceinline__ RulesBwdItem rules_bwd_item(const BwdRulesParams& rp, int item)
{
    const BwdParams& p = rp.b;
    RulesBwdItem it;
    const int first = item / (rp.chunk * p.Tc) * rp.chunk;              // of the chunk of (key/value head, part)s
    const int many = min(rp.chunk, rp.n_items / p.Tc - first);
    const int at = item - first * p.Tc;
    const int j = at / many, group = first + at - j * many;
    const int part = group % rp.parts;
    const int R = rp.Hq / rp.Hkv;
    it.kv = group / rp.parts;
    it.b = it.kv / rp.Hkv;
    it.out = part * (rp.B * rp.Hkv) + it.kv;
    it.bh0 = it.kv * R + part * rp.part_heads;
    it.heads = min(rp.part_heads, R - part * rp.part_heads);
    it.j0 = j * kBlockN;
    it.prefix = rp.causal ? rules_prefix(rp.prefix, it.b, p.Nk, p.status) : 0;
    if (rp.tile != nullptr) {
        const int2 x = rp.tile[static_cast<size_t>(it.b) * p.Tc + j];
        it.i_first = x.x;
        it.n = x.y - x.x;
    } else {
        it.i_first = 0;
        if (rp.causal && it.j0 >= it.prefix) {
            const int a = it.j0 - (p.Nk - p.N);  // first query that sees the tile's first key
            it.i_first = a <= 0 ? 0 : a / kBlockM;
        }
        it.n = p.Tr > it.i_first ? p.Tr - it.i_first : 0;
    }
    return it;
}

// P and P times the cap's slope for 64 scores of one key (columns: queries).  CAP: -1 none, 3 the near and 2 the
// middle range (cap_range), 0 any.  BIAS: -slope2 |dist + c|; sign 1 where dist + c >= 0 in every column that counts, -1 where <= 0, 0 either.
template <int CAP, bool BIAS>
__device__ __forceinline__ void rules_weights(const uint32_t (&u)[64], float (&pf)[64], uint32_t (&pk)[32], uint32_t l_addr,
                                              const ScoreRules& r, float slope2, float dist, int sign)
{
    const float2 m2 = two(r.mult);
    const float2 sg = two(sign < 0 ? slope2 : -slope2), eight = two(8.f);
    float2 away[4];  // distances, exact and counted on by eights
    if constexpr (BIAS) {
#pragma unroll
        for (int h = 0; h < 4; ++h) away[h] = make_float2(dist + static_cast<float>(2 * h), dist + static_cast<float>(2 * h + 1));
    }
#pragma unroll
    for (int c0 = 0; c0 < 64; c0 += 32) {
        float t[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) t[c] = __uint_as_float(u[c0 + c]);
        if constexpr (CAP == 0) tanh_any<32>(t, r.cap_in, r.far);
#pragma unroll
        for (int c = 0; c < 32; c += 8) {
#pragma unroll
            for (int h = 0; h < 4; h += 2) {
                const float4 l4 = ld_shared_f4(l_addr + (c0 + c + 2 * h) * 4);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = c + 2 * (h + e);
                    float2 y = make_float2(t[i], t[i + 1]);
                    if constexpr (CAP == 3) y = __fmul2_rn(y, cap_factor(y, r.near));
                    if constexpr (CAP == 2) y = __fmul2_rn(y, cap_factor(y, r.mid));
                    float2 x = __ffma2_rn(y, m2, e == 0 ? make_float2(-l4.x, -l4.y) : make_float2(-l4.z, -l4.w));
                    if constexpr (BIAS) {
                        if (sign != 0) {
                            x = __ffma2_rn(sg, away[h + e], x);
                            if (c0 + c + 8 < 64) away[h + e] = __fadd2_rn(away[h + e], eight);
                        } else {
                            x.x = fmaf(-slope2, fabsf(dist + static_cast<float>(c0 + i)), x.x);
                            x.y = fmaf(-slope2, fabsf(dist + static_cast<float>(c0 + i + 1)), x.y);
                        }
                    }
                    const float2 w = make_float2(ex2(x.x), ex2(x.y));
                    pk[(c0 + i) / 2] = pack_bf16x2(w.x, w.y);
                    float2 g = w;
                    if constexpr (CAP >= 0) g = __fmul2_rn(w, __ffma2_rn(make_float2(-y.x, -y.y), y, make_float2(1.f, 1.f)));
                    pf[c0 + i] = g.x;
                    pf[c0 + i + 1] = g.y;
                }
            }
        }
    }
}

template <int D, int RULES, typename GradT>
__global__ void __launch_bounds__(kBwdThreads, 1) fa_rules_bwd_kernel(const __grid_constant__ BwdRulesParams rp)
{
    using C = RulesBwdCfg<D>;
    constexpr bool kWithCap = (RULES & kCap) != 0, kWithBias = (RULES & kBias) != 0;
    const BwdParams& p = rp.b;
    // No grid_launch_dependents here: letting the dQ conversion that follows launch early made
    // the backward 6 % slower (B=64 H=16 N=1024 d=64); it starts once this grid's CTAs have exited.
    extern __shared__ __align__(1024) uint8_t bwd_smem_raw[];
    const uint32_t raw = smem_u32(bwd_smem_raw);
    const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
    if (pad + C::kUsed > static_cast<uint32_t>(C::kSmem)) {  // cannot align the swizzled tiles
        grid_dependency_wait();
        if (threadIdx.x == 0) atomicCAS(p.status, 0, FA_ERR_UNSUPPORTED);
        return;
    }
    uint8_t* smem = bwd_smem_raw + pad;
    const uint32_t sbase = raw + pad;
    auto bar = [&](int i) -> uint32_t { return sbase + C::kOffBar + 8u * static_cast<uint32_t>(i); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + C::kNumBars * 8);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const unsigned long long limit = p.wait_limit_ns;

    const int off = p.Nk - p.N;
    RulesBwdItem* items = reinterpret_cast<RulesBwdItem*>(smem + C::kOffItems);
    // Item i of the CTA, by every role but the producer, and its record's release (one arrival a warp).
    auto take = [&](int i, RulesBwdItem& it) -> bool {
        const int at = i % kRulesItems;
        if (!mbar_wait(bar(kBbItemFull + at), static_cast<uint32_t>(i / kRulesItems) & 1, limit, abort_flag)) return false;
        it = items[at];
        return true;
    };
    auto release = [&](int i) { mbar_arrive(bar(kBbItemEmpty + i % kRulesItems)); };
    // the next query tile of an item: its query heads one after the other
    auto step = [](const RulesBwdItem& it, int& bh, int& tile) {
        if (++tile < it.i_first + it.n) return;
        tile = it.i_first;
        ++bh;
    };
    constexpr int QS = C::kQStages;
    constexpr int KVB = C::kKVBufs;
    // dK_j and dV_j leave through shared memory and bulk tensor stores when both tiles fit in
    // the dS buffer, which no tensor-core operation reads once the item's last dQ is done
    // (bf16 gradients with d <= 64, fp32 with d = 32); otherwise each thread stores its row.
    constexpr int kGRow = D * static_cast<int>(sizeof(GradT));  // bytes of a gradient row
    constexpr bool kStageGrad = C::kDSOwn && kGRow <= 128;
    constexpr int kGTile = kBlockN * kGRow;                      // one staged 128-row tile
    static_assert(!kStageGrad || 2 * kGTile <= 2 * C::kDSBlk, "staging tiles exceed the dS buffer");

    if (threadIdx.x == 0) {
        for (int i = 0; i < KVB; ++i) {
            mbar_init(bar(kBbKVFull + i), 1);
            mbar_init(bar(kBbKVEmpty + i), 2);  // one commit from each issuer
        }
        for (int s = 0; s < QS; ++s) {
            mbar_init(bar(kBbQFull + s), 1);
            mbar_init(bar(kBbQEmpty + s), 2);
        }
        mbar_init(bar(kBbDrain), 1);
        mbar_init(bar(kBbDrain + 1), 1);
        mbar_init(bar(kBbSFull), 1);
        mbar_init(bar(kBbDPFull), 1);
        mbar_init(bar(kBbPReady), 256);
        mbar_init(bar(kBbDSReady), 256);
        mbar_init(bar(kBbDQFull), 1);
        mbar_init(bar(kBbDQFree), 128);
        mbar_init(bar(kBbDPFree), 256);
        // Only warp 10 (dV, dK) commits Done: with two K/V buffers warp 9 may finish the next
        // item before warp 10 finishes this one, and a second arrival of its own would complete
        // the phase early.
        mbar_init(bar(kBbDone), 1);
        mbar_init(bar(kBbDVDone), 1);
        mbar_init(bar(kBbSFree), 256);
        mbar_init(bar(kBbStageFull), 256);
        mbar_init(bar(kBbStageFree), 1);
        for (int i = 0; i < kRulesItems; ++i) {
            mbar_init(bar(kBbItemFull + i), 1);
            mbar_init(bar(kBbItemEmpty + i), 14);  // the issuers, the compute and the dQ warps
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kBwdWarpMma) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    // Launched with programmatic stream serialization: the setup above may overlap the preparation
    // kernel; every global read and write comes after it has completed.
    grid_dependency_wait();

    if (warp >= 8 && warp < 12) {
        regs_decrease<kRulesBwdControlRegs>();
        if (warp == kBwdWarpProducer && lane == 0) {
            // ============================================================ producer
            prefetch_tensormap(&p.tm_q);
            prefetch_tensormap(&p.tm_k);
            prefetch_tensormap(&p.tm_v);
            prefetch_tensormap(&p.tm_do);
            if (kStageGrad) {
                prefetch_tensormap(&p.tm_dk);
                prefetch_tensormap(&p.tm_dv);
            }
            const uint64_t pol_keep = policy_evict_last();  // Q_i, dO_i: read by every key tile of the head
            const uint64_t pol_once = policy_evict_first(); // K_j, V_j: read by one CTA only
            int g = 0;        // query tiles loaded (Q ring position)
            int kv = 0;       // items whose K/V were loaded
            bool ok = true;
            int asked = atomicAdd(rp.counter, 1);  // the next item, asked for one ahead
            for (int i = 0;; ++i) {
                RulesBwdItem it;
                it.kv = -1;
                if (asked < rp.n_items) {
                    it = rules_bwd_item(rp, asked);
                    asked = atomicAdd(rp.counter, 1);
                }
                const int at = i % kRulesItems;
                if (i >= kRulesItems &&
                    !mbar_wait(bar(kBbItemEmpty + at), static_cast<uint32_t>(i / kRulesItems - 1) & 1, limit, abort_flag)) {
                    ok = false;
                    break;
                }
                items[at] = it;
                mbar_arrive(bar(kBbItemFull + at));
                if (it.kv < 0) break;
                if (it.n == 0) continue;  // no query tile sees this key tile (every role skips it)
                const int kb = kv % KVB;
                if (kv >= KVB && !mbar_wait(bar(kBbKVEmpty + kb), static_cast<uint32_t>(kv / KVB - 1) & 1, limit, abort_flag)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(bar(kBbKVFull + kb), 2 * C::kTileBytes);
#pragma unroll
                for (int cb = 0; cb < C::kNumCB; ++cb) {
                    tma_load_3d(sbase + C::kOffK + kb * C::kTileBytes + cb * C::kBlkBytes, &p.tm_k, bar(kBbKVFull + kb),
                                cb * C::kCB, it.j0, it.kv, pol_once);
                    tma_load_3d(sbase + C::kOffV + kb * C::kTileBytes + cb * C::kBlkBytes, &p.tm_v, bar(kBbKVFull + kb),
                                cb * C::kCB, it.j0, it.kv, pol_once);
                }
                ++kv;
                for (int h = 0; ok && h < it.heads; ++h) {
                    const int bh = it.bh0 + h;
                    for (int t = 0; t < it.n; ++t, ++g) {
                        const int s = g % QS;
                        if (g >= QS && !mbar_wait(bar(kBbQEmpty + s), static_cast<uint32_t>(g / QS - 1) & 1, limit, abort_flag)) {
                            ok = false;
                            break;
                        }
                        const int i0 = (it.i_first + t) * kBlockM;
                        mbar_arrive_expect_tx(bar(kBbQFull + s), 2 * C::kTileBytes + 2 * 512);
#pragma unroll
                        for (int cb = 0; cb < C::kNumCB; ++cb) {
                            tma_load_3d(sbase + C::kOffQ + s * C::kTileBytes + cb * C::kBlkBytes, &p.tm_q, bar(kBbQFull + s),
                                        cb * C::kCB, i0, bh, pol_keep);
                            tma_load_3d(sbase + C::kOffDO + s * C::kTileBytes + cb * C::kBlkBytes, &p.tm_do,
                                        bar(kBbQFull + s), cb * C::kCB, i0, bh, pol_keep);
                        }
                        const size_t row = static_cast<size_t>(bh) * p.Tr * kBlockM + i0;
                        bulk_load(sbase + C::kOffL + s * 512, p.lse2 + row, 512, bar(kBbQFull + s));
                        bulk_load(sbase + C::kOffDsc + s * 512, p.dsc + row, 512, bar(kBbQFull + s));
                    }
                }
                if (!ok) break;
            }
            if (!ok && !*abort_flag) record_failure(p.status, abort_flag, FA_ERR_TIMEOUT);
            // every issued copy lands before the CTA may exit
            for (int t = kv - KVB < 0 ? 0 : kv - KVB; t < kv; ++t)
                mbar_wait(bar(kBbKVFull + t % KVB), static_cast<uint32_t>(t / KVB) & 1, kDrainLimitNs, nullptr);
            for (int t = g - QS < 0 ? 0 : g - QS; t < g; ++t)
                mbar_wait(bar(kBbQFull + t % QS), static_cast<uint32_t>(t / QS) & 1, kDrainLimitNs, nullptr);
        } else if ((warp == kBwdWarpMma || warp == kBwdWarpMma + 1) && lane == 0) {
            // ============================================================ MMA issuers
            // Barrier operations stall the issuing thread for a few hundred cycles, and the
            // tensor core holds only a short queue of these small MMAs: one issuer that also
            // waits and commits leaves the tensor core idle much of the time.  Warp 9 issues
            // the transposed products S^T, dP^T; warp 10 the accumulations dV, dK and dQ.
            const bool issuer_t = warp == kBwdWarpMma;
            bool ok = true;
            auto wait = [&](int b, int parity) -> bool {
                ok = ok && mbar_wait(bar(b), static_cast<uint32_t>(parity) & 1, limit, abort_flag);
                return ok;
            };
            // S^T = K_j Q_i^T or dP^T = V_j dO_i^T: both operands K-major in shared memory.
            auto issue_t = [&](uint32_t d_col, int a_off, int b_off) {
                const uint64_t a0 = smem_desc(sbase + a_off, 16, C::kAtomBytes, C::kLayout);
                const uint64_t b0 = smem_desc(sbase + b_off, 16, C::kAtomBytes, C::kLayout);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = ((kk * 16) / C::kCB * C::kBlkBytes + ((kk * 16) % C::kCB) * 2) >> 4;
                    umma_ss(tmem + d_col, a0 + o, b0 + o, C::kIdescT, kk > 0 ? 1u : 0u);
                }
            };
            // dV += P^T dO_i or dK += dS^T Q_i: A (bf16, packed two per column) from TMEM, the two
            // query halves half_stride columns apart (64 when each half sits over its own 64
            // source columns, 32 when packed back to back); B MN-major in shared memory.
            auto issue_acc = [&](uint32_t d_col, uint32_t a_col, uint32_t half_stride, int b_off, bool accumulate) {
                const uint64_t b0 = smem_desc(sbase + b_off, C::kBlkBytes, C::kAtomBytes, C::kLayout);
#pragma unroll
                for (int kk = 0; kk < kBlockM / 16; ++kk)
                    umma_ts(tmem + d_col, tmem + a_col + half_stride * (kk >> 2) + 8u * (kk & 3),
                            b0 + ((kk * 16 * C::kRowBytes) >> 4), C::kIdescAcc, (accumulate || kk > 0) ? 1u : 0u);
            };
            // d <= 64: dK += dS^T Q_i with A = dS^T read from the shared-memory dS buffer, whose key
            // rows hold their 128 queries as two swizzled 64-query blocks (K-major for this product).
            auto issue_dk_smem = [&](int q_off, bool accumulate) {
                const uint64_t a0 = smem_desc(sbase + C::kOffDS, 16, 1024, kSwizzle128B);
                const uint64_t b0 = smem_desc(sbase + q_off, C::kBlkBytes, C::kAtomBytes, C::kLayout);
#pragma unroll
                for (int kk = 0; kk < kBlockM / 16; ++kk) {
                    const uint32_t ao = ((kk * 16) / 64 * C::kDSBlk + ((kk * 16) % 64) * 2) >> 4;
                    umma_ss(tmem + C::kColDK, a0 + ao, b0 + ((kk * 16 * C::kRowBytes) >> 4), C::kIdescAcc,
                            (accumulate || kk > 0) ? 1u : 0u);
                }
            };
            // dQ = dS K_j: A = dS (MN-major, two 64-query blocks), B = K_j (MN-major).
            auto issue_dq = [&](int k_off) {
                const uint64_t a0 = smem_desc(sbase + C::kOffDS, C::kDSBlk, 1024, kSwizzle128B);
                const uint64_t b0 = smem_desc(sbase + k_off, C::kBlkBytes, C::kAtomBytes, C::kLayout);
#pragma unroll
                for (int kk = 0; kk < kBlockN / 16; ++kk)
                    umma_ss(tmem + C::kColDQ, a0 + ((kk * 16 * 128) >> 4), b0 + ((kk * 16 * C::kRowBytes) >> 4),
                            C::kIdescDQ, kk > 0 ? 1u : 0u);
            };
            int g = 0;  // query tiles processed (all items)
            int k = 0;  // items processed
            for (int i = 0; ok; ++i) {
                RulesBwdItem it;
                ok = take(i, it);
                if (!ok || it.kv < 0) break;
                release(i);
                if (it.n == 0) continue;
                const int n = it.n * it.heads;  // query tiles of all its heads
                const int kb = k % KVB;
                const int k_off = C::kOffK + kb * C::kTileBytes;
                const int v_off = C::kOffV + kb * C::kTileBytes;
                if (!wait(kBbKVFull + kb, k / KVB)) break;
                if (issuer_t) {
                    // S^T and dP^T of every query tile; a Q stage is released (one of two arrivals)
                    // once dP^T has been issued, this issuer's last read of it.
                    for (int t = 0; t < n; ++t, ++g) {
                        const int s = g % QS;
                        // S^T(g) overwrites S^T(g-1), loaded by the compute warps (d <= 64), or
                        // P^T(g-1) (d = 128), which dV(g-1) must have read
                        if ((g > 0 && !wait(C::kDSOwn ? kBbSFree : kBbDVDone, g - 1)) || !wait(kBbQFull + s, g / QS)) break;
                        tc_fence_after_sync();
                        issue_t(C::kColS, k_off, C::kOffQ + s * C::kTileBytes);
                        umma_commit(bar(kBbSFull));
                        // dP^T(g) overwrites dP^T(g-1): loaded by the compute warps (d <= 64), or, with
                        // dS^T and dQ in those columns (d = 128), dK and dQ done and dQ read out
                        if (g > 0 && !wait(C::kDSOwn ? kBbDPFree : kBbDQFree, g - 1)) break;
                        tc_fence_after_sync();
                        issue_t(C::kColDP, v_off, C::kOffDO + s * C::kTileBytes);
                        umma_commit(bar(kBbDPFull));
                        umma_commit(bar(kBbQEmpty + s));
                    }
                } else {
                    for (int t = 0; t < n; ++t, ++g) {
                        const int s = g % QS;
                        if (!wait(kBbPReady, g)) break;
                        tc_fence_after_sync();
                        issue_acc(C::kColDV, C::kColP, C::kPHalf, C::kOffDO + s * C::kTileBytes, t > 0);
                        umma_commit(bar(kBbDVDone));
                        if (!wait(kBbDSReady, g)) break;
                        tc_fence_after_sync();
                        if constexpr (C::kDSOwn)
                            issue_dk_smem(C::kOffQ + s * C::kTileBytes, t > 0);
                        else
                            issue_acc(C::kColDK, C::kColDS, C::kPHalf, C::kOffQ + s * C::kTileBytes, t > 0);
                        umma_commit(bar(kBbQEmpty + s));
                        if (!C::kDQAlias && g > 0 && !wait(kBbDQFree, g - 1)) break;
                        tc_fence_after_sync();
                        issue_dq(k_off);
                        umma_commit(bar(kBbDQFull));
                    }
                }
                if (!ok) break;
                umma_commit(bar(kBbKVEmpty + kb));  // this issuer's reads of K_j, V_j are done
                if (!issuer_t) umma_commit(bar(kBbDone));
                ++k;
            }
            if (!ok && !*abort_flag) record_failure(p.status, abort_flag, FA_ERR_TIMEOUT);
            const int me = issuer_t ? 0 : 1;
            umma_commit(bar(kBbDrain + me));
            mbar_wait(bar(kBbDrain + me), 0, kDrainLimitNs, nullptr);
        }
    } else if (warp >= kBwdWarpDq) {
        regs_decrease<kRulesBwdDqRegs>();
        // ============================================================ dQ reduction
        const int r = threadIdx.x & 127;  // query row of the tile == TMEM lane
        const uint32_t t_dq = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + C::kColDQ;
        bool ok = true;
        int g = 0;
        auto dq_item = [&](int i, RulesBwdItem& it) -> bool {
            ok = __all_sync(0xffffffffu, take(i, it));
            if (!ok || it.kv < 0) return false;
            __syncwarp();  // every lane has its copy
            if ((threadIdx.x & 31) == 0) release(i);
            return true;
        };
        if constexpr (C::kDQBulk) {
            // Each warp stages its 32 rows 16 columns at a time (column groups of 4: lane l writes 16
            // bytes at (group * 32 + l) * 16, so a warp's stores hit distinct banks) and lane 0 adds the
            // 2 KB block into the accumulator with one bulk reduction; two blocks alternate, and before
            // refilling one, lane 0 waits until the reduction issued from it has read it.
            const int wq = warp & 3;
            const int lane = threadIdx.x & 31;
            const uint32_t stg = sbase + C::kOffDQS + static_cast<uint32_t>(wq) * 4096u;
            int chunks = 0;
            for (int i = 0; ok; ++i) {
                RulesBwdItem it;
                if (!dq_item(i, it)) break;
                for (int t = 0, bh = it.bh0, tile = it.i_first; t < it.n * it.heads; ++t, ++g, step(it, bh, tile)) {
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(kBbDQFull), g & 1, limit, abort_flag));
                    if (!ok) break;
                    tc_fence_after_sync();
                    // this warp's [d/4][32][4] block of the (head, query tile) accumulator
                    float* acc = p.dq_acc + (static_cast<size_t>(bh) * p.Tr + tile) * (D * kBlockM) +
                                 static_cast<size_t>(wq) * (D * 32);
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t v[32];
                        tmem_ld32(t_dq + 32u * c, v);
                        tmem_ld_wait();
                        if (c == D / 32 - 1) {  // the whole dQ row is in registers: release the columns
                            tc_fence_before_sync();
                            mbar_arrive(bar(kBbDQFree));
                        }
#pragma unroll
                        for (int k2 = 0; k2 < 2; ++k2, ++chunks) {
                            const uint32_t blk = stg + static_cast<uint32_t>(chunks & 1) * 2048u;
                            if (lane == 0) bulk_wait_read<1>();  // the reduction from this block two chunks ago read it
                            __syncwarp();
#pragma unroll
                            for (int q4 = 0; q4 < 4; ++q4)
                                st_shared_v4(blk + static_cast<uint32_t>(q4 * 32 + lane) * 16u, v[16 * k2 + 4 * q4],
                                             v[16 * k2 + 4 * q4 + 1], v[16 * k2 + 4 * q4 + 2], v[16 * k2 + 4 * q4 + 3]);
                            fence_proxy_async_shared();
                            __syncwarp();
                            if (lane == 0) {
                                bulk_reduce_add_f32(acc + (2 * c + k2) * (4 * 32 * 4), blk, 2048u);
                                bulk_commit_group();
                            }
                        }
                    }
                }
            }
            if (lane == 0 && chunks > 0) bulk_wait_all();  // reductions complete before the CTA exits
        }
        for (int i = 0; !C::kDQBulk && ok; ++i) {
            RulesBwdItem it;
            if (!dq_item(i, it)) break;
            for (int t = 0, bh = it.bh0, tile = it.i_first; t < it.n * it.heads; ++t, ++g, step(it, bh, tile)) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar(kBbDQFull), g & 1, limit, abort_flag));
                if (!ok) break;
                tc_fence_after_sync();
                float* acc = p.dq_acc + (static_cast<size_t>(bh) * p.Tr + tile) * (D / 4) * (kBlockM * 4) +
                             r * 4;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t v[32];
                    tmem_ld32(t_dq + 32u * c, v);
                    tmem_ld_wait();
                    if (c == D / 32 - 1) {  // the whole dQ row is in registers: release the columns
                        tc_fence_before_sync();
                        mbar_arrive(bar(kBbDQFree));
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        red_add_v4(acc + static_cast<size_t>(c * 8 + e / 4) * (kBlockM * 4), __uint_as_float(v[e]),
                                   __uint_as_float(v[e + 1]), __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
                }
            }
        }
        if (!ok && !*abort_flag) record_failure(p.status, abort_flag, FA_ERR_TIMEOUT);
    } else {
        regs_increase<kRulesBwdComputeRegs>();
        // ============================================================ compute
        const int h = warp >> 2;                 // query half of the tile
        const int kr = threadIdx.x & 127;        // key row of the tile == TMEM lane
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lane_base + C::kColS + 64u * h;
        const uint32_t t_dp = tmem + lane_base + C::kColDP + 64u * h;
        const uint32_t t_ds = tmem + lane_base + C::kColDS + C::kPHalf * h;
        const uint32_t t_p = tmem + lane_base + C::kColP + C::kPHalf * h;
        const uint32_t ds_row = sbase + C::kOffDS + h * C::kDSBlk + kr * 128;  // this thread's dS^T row
        const float2 sc2 = make_float2(p.scale, p.scale);
        bool ok = true;
        int g = 0;
        int k = 0;
        int staged = 0;            // items whose dK, dV went out through the staging tiles
        float slope2 = 0.f;
        bool stage_busy = false;   // the last of those stores may still be reading the dS buffer
        for (int i = 0; ok; ++i) {
            RulesBwdItem it;
            ok = __all_sync(0xffffffffu, take(i, it));
            if (!ok || it.kv < 0) break;
            __syncwarp();  // every lane has its copy
            if ((threadIdx.x & 31) == 0) release(i);
            const int key = it.j0 + kr;
            const bool valid = key < p.Nk;
            const size_t row = (static_cast<size_t>(it.out) * p.Nk + (valid ? key : 0)) * D + h * (D / 2);
            // the queries [qa, qe) that see the key; none see a key past Nk (its score 0 can be far above the row's)
            int qa = 0, qe = 0;
            if (valid) {
                if (rp.each != nullptr) {
                    const int2 x = rp.each[static_cast<size_t>(it.b) * p.Nk + key];
                    qa = x.x;
                    qe = x.y;
                } else {
                    qa = rp.causal && key >= it.prefix ? max(key - off, 0) : 0;
                    qe = p.N;
                }
            }
            GradT* dk = reinterpret_cast<GradT*>(p.dk) + row;
            GradT* dv = reinterpret_cast<GradT*>(p.dv) + row;
            if (it.n == 0) {  // no query sees these keys: zero gradients, no tensor-core work
                float z[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) z[e] = 0.f;
                if (valid)
                    for (int c = 0; c < D / 2; c += 16) {
                        store_row16<GradT>(dv + c, z);
                        store_row16<GradT>(dk + c, z);
                    }
                continue;
            }
            const int n = it.n * it.heads;
            for (int t = 0, bh = it.bh0, tile = it.i_first; t < n; ++t, ++g, step(it, bh, tile)) {
                const int s = g % QS;
                const int i0 = tile * kBlockM;
                if (kWithBias && tile == it.i_first) slope2 = rp.rules.slopes[bh - it.b * rp.Hq] * kLog2e;
                ok = __all_sync(0xffffffffu, mbar_wait(bar(kBbSFull), g & 1, limit, abort_flag));
                if (!ok) break;
                tc_fence_after_sync();
                uint32_t u[64];
                float mx[2];  // under a cap the largest absolute scores of both halves
                if constexpr (kWithCap) {
                    tmem_ld32_absmax(t_s, *reinterpret_cast<uint32_t(*)[32]>(&u[0]), mx[0]);
                    tmem_ld32_absmax(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(&u[32]), mx[1]);
                    tmem_ld_wait();
                } else {
                    tmem_ld32(t_s, *reinterpret_cast<uint32_t(*)[32]>(&u[0]));
                    tmem_ld32(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(&u[32]));
                    tmem_ld_wait();
                }
                if constexpr (C::kDSOwn) {  // the S^T columns may now be overwritten by the next S^T
                    tc_fence_before_sync();
                    mbar_arrive(bar(kBbSFree));
                }
                // Hidden pairs: P = 0.  Without a cap by their scores, one selection each, with one, which makes a number of
                // any score, by P in both its forms: 16 sequences of 1024 tokens in documents, 16 heads of 64, forward and
                // backward, 182 us by P, 169 by the scores.  (Masked inside rules_weights under a cap too: registers spill,
                // d = 128 840 -> 885 us.)
                const int q0 = i0 + 64 * h;  // this thread's first query
                const bool hides = !__all_sync(0xffffffffu, qa <= q0 && qe >= q0 + 64);
                int range = 0;
                if constexpr (kWithCap) {
                    float t[64];
#pragma unroll
                    for (int c = 0; c < 64; ++c) t[c] = __uint_as_float(u[c]);
                    const float m = fmaxf(mx[0], mx[1]);
                    range = cap_range(rp.rules, m);
                    if (range == 0 && hides) range = cap_range_seen<64>(rp.rules, t, m, qa - q0, qe - q0);
                }
                if (!kWithCap && hides) {
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const uint32_t see = low_bits(qe - q0 - 32 * w) & ~low_bits(qa - q0 - 32 * w);
#pragma unroll
                        for (int c = 0; c < 32; ++c) u[32 * w + c] = (see >> c) & 1u ? u[32 * w + c] : 0xff800000u;  // -inf
                    }
                }
                // P = exp2(s - L log2(e)), s the score in base 2; L = +inf gives 0 (row past N or with no key).  pf
                // is P times the cap's slope, pk P in bf16 (rounded for the product with dO, half a step of 2^-8).
                const uint32_t l_addr = sbase + C::kOffL + s * 512 + h * 256;
                float pf[64];
                uint32_t pk[32];
                int sign = 0;
                if constexpr (kWithBias)
                    sign = __all_sync(0xffffffffu, off + q0 >= key || (rp.causal && key >= it.prefix)) ? 1
                           : __all_sync(0xffffffffu, off + q0 + 63 <= key)                             ? -1
                                                                                                       : 0;
                const float dist = static_cast<float>(off + q0 - key);
                if (kWithCap && range == 3) rules_weights<3, kWithBias>(u, pf, pk, l_addr, rp.rules, slope2, dist, sign);
                else if (kWithCap && range == 2) rules_weights<2, kWithBias>(u, pf, pk, l_addr, rp.rules, slope2, dist, sign);
                else rules_weights<kWithCap ? 0 : -1, kWithBias>(u, pf, pk, l_addr, rp.rules, slope2, dist, sign);
                if (kWithCap && hides) {
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const uint32_t see = low_bits(qe - q0 - 32 * w) & ~low_bits(qa - q0 - 32 * w);
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            const bool a = (see >> c) & 1u, b = (see >> (c + 1)) & 1u;
                            pf[32 * w + c] = a ? pf[32 * w + c] : 0.f;
                            pf[32 * w + c + 1] = b ? pf[32 * w + c + 1] : 0.f;
                            pk[16 * w + c / 2] &= (a ? 0x0000ffffu : 0u) | (b ? 0xffff0000u : 0u);
                        }
                    }
                }
                if (C::kDSOwn && g > 0) {  // dV must have read the previous P^T from these columns
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(kBbDVDone), (g - 1) & 1, limit, abort_flag));
                    if (!ok) break;
                    tc_fence_after_sync();
                }
                tmem_st32(t_p, pk);
                tmem_st_wait();
                tc_fence_before_sync();
                mbar_arrive(bar(kBbPReady));

                ok = __all_sync(0xffffffffu, mbar_wait(bar(kBbDPFull), g & 1, limit, abort_flag));
                if (!ok) break;
                tc_fence_after_sync();
                tmem_ld32(t_dp, *reinterpret_cast<uint32_t(*)[32]>(&u[0]));
                tmem_ld32(t_dp + 32, *reinterpret_cast<uint32_t(*)[32]>(&u[32]));
                tmem_ld_wait();
                if constexpr (C::kDSOwn) {  // the dP^T columns may now be overwritten by the next dP^T
                    tc_fence_before_sync();
                    mbar_arrive(bar(kBbDPFree));
                }
                // dS' = scale dS = pf o (dP scale - scale D), rounded to bf16 for the products with K and Q (half a step, 2^-8 of
                // each, as P for dV: one type for both operands of a tensor-core product)
                const uint32_t d_addr = sbase + C::kOffDsc + s * 512 + h * 256;
#pragma unroll
                for (int c = 0; c < 64; c += 4) {
                    const float4 d4 = ld_shared_f4(d_addr + c * 4);
                    const float2 y01 = __ffma2_rn(make_float2(__uint_as_float(u[c]), __uint_as_float(u[c + 1])), sc2,
                                                  make_float2(-d4.x, -d4.y));
                    const float2 y23 = __ffma2_rn(make_float2(__uint_as_float(u[c + 2]), __uint_as_float(u[c + 3])), sc2,
                                                  make_float2(-d4.z, -d4.w));
                    const float2 g01 = __fmul2_rn(y01, make_float2(pf[c], pf[c + 1]));
                    const float2 g23 = __fmul2_rn(y23, make_float2(pf[c + 2], pf[c + 3]));
                    pk[c / 2] = pack_bf16x2(g01.x, g01.y);
                    pk[c / 2 + 1] = pack_bf16x2(g23.x, g23.y);
                }
                if constexpr (C::kDSOwn) {
                    // the previous dK and dQ must have read the previous dS from shared memory (dQ is
                    // issued after dK by the same thread, so its completion covers both)
                    ok = __all_sync(0xffffffffu, g == 0 || mbar_wait(bar(kBbDQFull), (g - 1) & 1, limit, abort_flag));
                    if (!ok) break;
                    tc_fence_after_sync();
                }
                if (kStageGrad && stage_busy) {  // the previous item's bulk stores read the dS buffer
                    if (threadIdx.x == 0) {
                        bulk_wait_read_all();
                        mbar_arrive(bar(kBbStageFree));
                    }
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(kBbStageFree), (staged - 1) & 1, limit, abort_flag));
                    if (!ok) break;
                    stage_busy = false;
                }
                if constexpr (!C::kDSOwn) tmem_st32(t_ds, pk);  // d = 128: dK reads dS^T from tensor memory
                // dS^T row kr into the MN-major dS operand: 16-byte chunk q8 of the 128-byte row goes
                // to chunk q8 ^ (kr mod 8) (128-byte swizzle).
#pragma unroll
                for (int q8 = 0; q8 < 8; ++q8)
                    st_shared_v4(ds_row + ((q8 ^ (kr & 7)) << 4), pk[4 * q8], pk[4 * q8 + 1], pk[4 * q8 + 2],
                                 pk[4 * q8 + 3]);
                fence_proxy_async_shared();
                if constexpr (!C::kDSOwn) tmem_st_wait();
                tc_fence_before_sync();
                mbar_arrive(bar(kBbDSReady));
            }
            if (!ok) break;
            // dK_j and dV_j of this item: this thread writes key row j0 + kr, columns of its half.
            // The next item's first dV and dK (which overwrite these columns) are issued only after
            // this warpgroup's next P^T arrival, i.e. after these loads.
            ok = __all_sync(0xffffffffu, mbar_wait(bar(kBbDone), k & 1, limit, abort_flag));
            if (!ok) break;
            ++k;
            tc_fence_after_sync();
            if constexpr (kStageGrad) {
                // Row kr of each tile, this thread's half of the columns, into the staging tiles
                // (dV at the start of the dS buffer, dK after it), 16-byte chunks swizzled like
                // the tensor maps (chunk index XOR kr mod 8 for 128-byte rows, XOR (kr / 2) mod 4
                // for 64-byte rows); one thread then stores both tiles, rows past Nk clipped.
                constexpr int kEpc = 16 / static_cast<int>(sizeof(GradT));  // elements per chunk
                constexpr int kHalfChunks = kGRow / 32;                     // chunks of a half row
                const uint32_t sw = kGRow == 128 ? static_cast<uint32_t>(kr & 7) : static_cast<uint32_t>((kr >> 1) & 3);
                const uint32_t stg = sbase + C::kOffDS + static_cast<uint32_t>(kr) * kGRow;
                uint32_t a[D / 2], b[D / 2];
#pragma unroll
                for (int c = 0; c < D / 2; c += 16) {
                    tmem_ld16(tmem + lane_base + C::kColDV + h * (D / 2) + c, *reinterpret_cast<uint32_t(*)[16]>(&a[c]));
                    tmem_ld16(tmem + lane_base + C::kColDK + h * (D / 2) + c, *reinterpret_cast<uint32_t(*)[16]>(&b[c]));
                }
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < kHalfChunks; ++q) {
                    const uint32_t off = ((static_cast<uint32_t>(h * kHalfChunks + q) ^ sw) << 4);
                    const int e = q * kEpc;
                    if constexpr (sizeof(GradT) == 2) {
                        st_shared_v4(stg + off, pack_bf16x2(__uint_as_float(a[e]), __uint_as_float(a[e + 1])),
                                     pack_bf16x2(__uint_as_float(a[e + 2]), __uint_as_float(a[e + 3])),
                                     pack_bf16x2(__uint_as_float(a[e + 4]), __uint_as_float(a[e + 5])),
                                     pack_bf16x2(__uint_as_float(a[e + 6]), __uint_as_float(a[e + 7])));
                        st_shared_v4(stg + kGTile + off, pack_bf16x2(__uint_as_float(b[e]), __uint_as_float(b[e + 1])),
                                     pack_bf16x2(__uint_as_float(b[e + 2]), __uint_as_float(b[e + 3])),
                                     pack_bf16x2(__uint_as_float(b[e + 4]), __uint_as_float(b[e + 5])),
                                     pack_bf16x2(__uint_as_float(b[e + 6]), __uint_as_float(b[e + 7])));
                    } else {
                        st_shared_v4(stg + off, a[e], a[e + 1], a[e + 2], a[e + 3]);
                        st_shared_v4(stg + kGTile + off, b[e], b[e + 1], b[e + 2], b[e + 3]);
                    }
                }
                fence_proxy_async_shared();
                mbar_arrive(bar(kBbStageFull));
                bool stored = true;
                if (threadIdx.x == 0) {
                    stored = mbar_wait(bar(kBbStageFull), staged & 1, limit, abort_flag);
                    if (stored) {
                        tma_store_3d(&p.tm_dv, sbase + C::kOffDS, 0, it.j0, it.out);
                        tma_store_3d(&p.tm_dk, sbase + C::kOffDS + kGTile, 0, it.j0, it.out);
                        bulk_commit_group();
                    }
                }
                ok = __all_sync(0xffffffffu, stored);
                if (!ok) break;
                ++staged;
                stage_busy = true;
            } else {
#pragma unroll
                for (int c = 0; c < D / 2; c += 16) {
                    uint32_t a[16], b[16];
                    tmem_ld16(tmem + lane_base + C::kColDV + h * (D / 2) + c, a);
                    tmem_ld16(tmem + lane_base + C::kColDK + h * (D / 2) + c, b);
                    tmem_ld_wait();
                    float fa[16], fb[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        fa[e] = __uint_as_float(a[e]);
                        fb[e] = __uint_as_float(b[e]);
                    }
                    if (valid) {
                        store_row16<GradT>(dv + c, fa);
                        store_row16<GradT>(dk + c, fb);
                    }
                }
            }
        }
        if (kStageGrad && threadIdx.x == 0 && staged > 0) bulk_wait_all();  // stores done before exit
        if (!ok && !*abort_flag) record_failure(p.status, abort_flag, FA_ERR_TIMEOUT);
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == kBwdWarpMma) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

template <int D, int RULES, typename GradT>
cudaError_t launch_bwd_rules_t(const BwdRulesParams& p, cudaStream_t st)
{
    using C = RulesBwdCfg<D>;
    auto kern = fa_rules_bwd_kernel<D, RULES, GradT>;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        cudaFuncAttributes attr;
        e = cudaFuncGetAttributes(&attr, kern);
        if (e != cudaSuccess) return e;
        if (attr.numRegs * kBwdThreads < 256 * kRulesBwdComputeRegs + 128 * (kRulesBwdControlRegs + kRulesBwdDqRegs))
            return cudaErrorLaunchOutOfResources;  // the register split would not fit
        configured[dev] = true;
    }
    const int grid = p.n_items < p.b.num_ctas ? p.n_items : p.b.num_ctas;
    return launch_pdl(kern, static_cast<unsigned>(grid), kBwdThreads, C::kSmem, st, p);
}

template <int D, int RULES>
cudaError_t launch_bwd_rules_d(const BwdRulesParams& p, fa_dtype grad_dtype, cudaStream_t st)
{
    return grad_dtype == FA_F32 ? launch_bwd_rules_t<D, RULES, float>(p, st) : launch_bwd_rules_t<D, RULES, __nv_bfloat16>(p, st);
}

}  // namespace fa

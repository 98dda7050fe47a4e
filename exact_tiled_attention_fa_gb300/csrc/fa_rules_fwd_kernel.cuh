// fa_rules_fwd_kernel.cuh -- exact attention forward under score rules, for sm_103a.
//
// Mathematics.  For query i of head h (position Nk - N + i) and key j of key/value head h / (Hq / Hkv):
//   x = scale q_i . k_j;  s = cap tanh(x / cap) with a cap, else x;  s -= slope_h |position - j|
//   O_i = sum_j softmax_j(s) V_j over the keys that i sees,  LSE_i = log sum_j exp(s)
// i sees j unless a causal mask hides it (j after i's position and not in the sequence's prefix) or the two are in
// different documents.  What a query sees is one interval of keys [lo, hi) whose ends never fall from a row to the
// next (fa_rules_ranges.cuh), so a query tile visits one run of key tiles, and only its first and last ones are masked.
//
// The tiles, roles, tensor memory, pipeline and bounded waits are those of fa_fwd_kernel.cuh (two query tiles of 128
// rows share a ring of K and V tiles; two softmax warpgroups, a producer, an issuer for each query tile).  What
// differs:
//  - The producer alone knows the work items; the others take them from a ring of records in shared memory.  With
//    documents their lengths depend on data, and each CTA asks a counter for its next one (an item's result does not
//    depend on who computes it).  Under a causal mask alone they go round by round to the CTAs, longest first over as
//    many heads at a time as may be (chunk_of), one round forward and one back: 4 sequences of 4097 tokens, 16 heads,
//    d = 64 155 us and d = 128 285, in heavy and light pairs head by head (fa_fwd) 181 and 318.
//  - An item's two query tiles may begin and end at different key tiles: K and V run over both, and the issuer of a
//    tile passes on the stages that it does not visit.
//  - Between a row's scores and its exponentials stand the cap and the bias, in registers.  Both can change which score
//    is the largest, so the row's maximum is taken after them (without them the loads from tensor memory bring it, and
//    under a cap whose tile lies in the near range the largest raw score gives it).  What was chosen for tanh, and why,
//    stands in fa_rules_common.cuh.
//  - A correction warpgroup (kRulesCorr).
//
// What bounds it: the softmax's chain between two products, as in fa_fwd_kernel.cuh, lengthened by the FMA units' work on
// the rules: at the shape above d = 64 152 us, with a bias 199, a cap of 50 220, both 296; d = 128 285, 314, 360, 393.  The
// capped times are those of scores of deviation 3, nearly all in the cheapest range; deviation 10 / 30: d = 64 331 / 398, both
// rules 410; d = 128 456 / 562, both 528.  In documents (64 sequences of 1024 tokens, 16 heads of 64) 144 us: 3.7 TB/s of the
// 541 MB that have to move; by the counters tensor cores 22 % busy, the ALUs (masks by bits, packing) 47 %, issue slots 49 %.
// Bytes stored and loaded that spill: cap d = 32 80/136, d = 128 84/104; bias d = 32 24/56, d = 64 12/32; both d <= 64 20/44.
#pragma once

#include "fa_fwd_kernel.cuh"
#include "fa_rules_common.cuh"

namespace fa {

// A work item as the producer hands it to the other roles.  Tiles a[i] .. n[i] - 1 of the item's n_kv are those that
// query tile i visits; n_kv < 0: no more items.
struct RulesItem {
    int bh, b, kv;  // query head, sequence, key/value head
    int prefix;     // of the sequence
    int r0[2], rows[2];
    int a[2], n[2];
    int j0, n_kv;   // first key tile, key tiles
};
enum : int { kBarItemFull = kBarCount, kBarItemEmpty = kBarItemFull + kRulesItems, kRulesBarCount = kBarItemEmpty + kRulesItems };

// Whether calls without a causal mask take a kernel with a correction warpgroup (16 warps).  us, d = 128, without / with it:
// 64 sequences of 1024 tokens, 16 heads 571 / 465, biased 639 / 551, both rules 787 / 747; 4 of 4097, 32/8 heads 1080 /
// 1021; 16 of 1024 in documents of 100 - 300 94.5 / 88.2.  With a cap alone its softmax warps spill: 632 / 634, scores of
// deviation 10 under a cap of 50 903 / 864, but in documents 138 / 141, 16384 tokens 802 / 818.  With a causal mask (4 x 4097,
// 16 heads) 286 / 288, capped (before hidden scores were looked at) 348 / 365.  At d = 64, where the softmax
// warps need the registers, 64 x 1024 took 279 against 278, in documents, causal 155 (with O read whole and released
// at once 164) against 144.
template <int D, int RULES>
constexpr bool kRulesCorr = D == 128 && RULES != kCap;

template <int D, int OutBytes>
struct RulesCfg : FwdCfg<D, OutBytes> {
    using Base = FwdCfg<D, OutBytes>;
    static_assert(kRulesBarCount <= Base::kNumBars, "barrier slots");
    static constexpr int kOffItems = Base::kOffBar + Base::kNumBars * 8 + 16;
    static constexpr int kOffInv = kOffItems + kRulesItems * static_cast<int>(sizeof(RulesItem));  // 1 / l of both tiles' rows
    static constexpr int kUsed = kOffInv + 2 * kBlockM * 4 + 1024;  // 1 KB to align
    static_assert(kUsed <= 227 * 1024, "shared memory per CTA");
    static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;  // one CTA on an SM, as FwdCfg
    static constexpr int kSoftRegs = 216;
    static constexpr int kCtrlRegs = 72;
};

// Query pair qp of head bh.  `swap`: the tiles change places (as in decode_item, where it evens out which of them walks
// further under a causal mask).
__device__ __forceinline__ RulesItem rules_item(const FwdRulesParams& p, int bh, int qp, int swap)
{
    const FwdParams& f = p.f;
    RulesItem it;
    it.bh = bh;
    it.b = bh / p.Hq;
    it.kv = bh / (p.Hq / p.Hkv);
    it.prefix = p.causal ? rules_prefix(p.prefix, it.b, f.Nk, f.status) : 0;
    const int off = f.Nk - f.N;
    const int n_all = (f.Nk + kBlockN - 1) / kBlockN;
    const int q_tiles = (f.N + kBlockM - 1) / kBlockM;
    int from[2], to[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r0 = qp * 2 * kBlockM + (i ^ swap) * kBlockM;
        it.r0[i] = r0;
        it.rows[i] = r0 < f.N ? min(kBlockM, f.N - r0) : 0;
        from[i] = to[i] = 0;
        if (it.rows[i] == 0) continue;
        if (p.tile != nullptr) {
            const int2 x = p.tile[static_cast<size_t>(it.b) * q_tiles + r0 / kBlockM];
            from[i] = x.x;
            to[i] = x.y;
        } else if (p.causal) {
            const int end = max(off + r0 + it.rows[i], it.prefix);  // keys the last row sees
            to[i] = end <= 0 ? 0 : min(n_all, (end + kBlockN - 1) / kBlockN);
        } else {
            to[i] = n_all;
        }
    }
    const bool has0 = to[0] > from[0], has1 = to[1] > from[1];
    it.j0 = has0 && has1 ? min(from[0], from[1]) : has0 ? from[0] : has1 ? from[1] : 0;
    it.a[0] = has0 ? from[0] - it.j0 : 0;
    it.a[1] = has1 ? from[1] - it.j0 : 0;
    it.n[0] = has0 ? to[0] - it.j0 : 0;
    it.n[1] = has1 ? to[1] - it.j0 : 0;
    it.n_kv = max(it.n[0], it.n[1]);
    return it;
}

// Sets the scores s of a tile that the row's keys [lo, hi) (counted from the tile's first) do not hold to -infinity.  (By
// selection: a non-finite score of a hidden key does not reach the row.)  Bits of four words and no branches: 64
// sequences of 1024 tokens in documents of 60 - 320, 16 heads of 64, 144 us; telling apart pieces of 32 columns that
// all rows of the warp see, some or none 160; passing over the exponentials of the latter too 206.
__device__ __forceinline__ void rules_mask(float* s, int lo, int hi)
{
#pragma unroll
    for (int q = 0; q < kBlockN / 32; ++q) {
        float* t = s + 32 * q;
        const uint32_t see = low_bits(hi - 32 * q) & ~low_bits(lo - 32 * q);
#pragma unroll
        for (int c = 0; c < 32; ++c) t[c] = (see >> c) & 1u ? t[c] : -INFINITY;
    }
}

// Correction warpgroup: the epilogue of both query tiles, so that the softmax warpgroups go on to the next item's
// scores at once.  The tile that ends first goes first (16384 tokens in documents of 1800 and 2500, 32/8 heads 624 us in
// fixed order, 606 - 618 so).  Warp w takes rows 32 (w mod 4) .. + 31 of each.  Once an item's last P V has completed (OReady)
// and the softmax has written the rows' 1 / l (LFull; 0 for a row that saw no key) it writes the rows out; when it has
// read them it releases O_i and 1 / l (OFree).
template <int D, typename OutT>
__device__ __forceinline__ void rules_correction(const FwdRulesParams& p, const uint8_t* smem, uint32_t bar0, uint32_t tmem,
                                                 volatile int* abort_flag)
{
    using C = RulesCfg<D, static_cast<int>(sizeof(OutT))>;
    auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
    const FwdParams& f = p.f;
    const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const int r = 32 * wq + lane;  // row within a query tile == TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>(32 * wq) << 16;
    const float* inv_l = reinterpret_cast<const float*>(smem + C::kOffInv);
    const unsigned long long limit = f.wait_limit_ns;
    int done[2] = {0, 0};  // items whose O_i has been read, of each query tile
    bool ok = true;
    for (int k = 0; ok; ++k) {
        const int at = k % kRulesItems;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarItemFull + at), static_cast<uint32_t>(k / kRulesItems) & 1, limit, abort_flag));
        if (!ok) break;
        const RulesItem it = reinterpret_cast<const RulesItem*>(smem + C::kOffItems)[at];
        if (it.n_kv < 0) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarItemEmpty + at));
        const int order = it.n[1] < it.n[0] ? 1 : 0;
#pragma unroll 1
        for (int ii = 0; ii < 2; ++ii) {
            const int i = ii ^ order;
            const int rows = i ? it.rows[1] : it.rows[0], n = i ? it.n[1] : it.n[0], r0 = i ? it.r0[1] : it.r0[0];
            int& dn = i ? done[1] : done[0];
            if (rows == 0) continue;  // tile lies past N
            const bool any = n > 0;
            float inv = 0.f;
            if (any) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarOReady + i), dn & 1, limit, abort_flag) &&
                                                 mbar_wait(bar(kBarLFull + i), dn & 1, limit, abort_flag));
                if (!ok) break;
                tc_fence_after_sync();
                inv = inv_l[i * kBlockM + r];
            }
            const uint32_t t_o = tmem + lane_base + C::col_o(i);
            OutT* orow = reinterpret_cast<OutT*>(f.o) + (static_cast<size_t>(it.bh) * f.N + static_cast<size_t>(r0 + r)) * D;
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                if (any) {
                    tmem_ld32(t_o + static_cast<uint32_t>(c), o);
                    tmem_ld_wait();
                }
                if (any && c + 32 == D) {
                    tc_fence_before_sync();
                    mbar_arrive(bar(kBarOFree + i));
                    ++dn;
                }
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = inv == 0.f ? 0.f : __uint_as_float(o[e]) * inv;
                if (r < rows) store_row32<OutT>(orow + c, v);
            }
        }
    }
    if (!ok && !*abort_flag) record_failure(f.status, abort_flag, FA_ERR_TIMEOUT);
}

template <int D, int RULES, bool CORR, typename OutT>
__global__ void __launch_bounds__(CORR ? 512 : kFwdThreads, 1) fa_rules_fwd_kernel(const __grid_constant__ FwdRulesParams p)
{
    using C = RulesCfg<D, static_cast<int>(sizeof(OutT))>;
    constexpr int S = C::kStages;
    constexpr bool kWithCap = (RULES & kCap) != 0, kWithBias = (RULES & kBias) != 0;
    static_assert(!CORR || C::kAliasP, "an item's first P goes where the last item's P V may still read");
    extern __shared__ uint8_t rules_smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(rules_smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + C::kOffBar;
    auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + C::kNumBars * 8);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    RulesItem* items = reinterpret_cast<RulesItem*>(smem + C::kOffItems);
    const FwdParams& f = p.f;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const unsigned long long limit = f.wait_limit_ns;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(kBarQFull + i), 1);
            mbar_init(bar(kBarQEmpty + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kBarSFull + i), 1);
            mbar_init(bar(kBarPFull + i), kBlockM);
            mbar_init(bar(kBarPVDone + i), 1);
            mbar_init(bar(kBarOReady + i), 1);
            mbar_init(bar(kBarDrain + i), 1);
            mbar_init(bar(kBarSFree + i), kBlockM);
            if constexpr (CORR) {
                mbar_init(bar(kBarLFull + i), kBlockM);
                mbar_init(bar(kBarOFree + i), kBlockM);
            }
        }
        for (int s = 0; s < S; ++s) {
            mbar_init(bar(kBarKVFull + s), 1);
            mbar_init(bar(kBarKVEmpty + s), 2);  // one arrival from each MMA issuer
        }
        for (int i = 0; i < kRulesItems; ++i) {
            mbar_init(bar(kBarItemFull + i), 1);
            mbar_init(bar(kBarItemEmpty + i), CORR ? 14 : 10);  // the issuers, the softmax and the correction warps
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();  // every global read and write comes after the kernel before
    grid_launch_dependents();

    // Item k of the CTA, by every role but the producer; lane 0 of a warp releases the record.
    auto take = [&](int k, RulesItem& it) -> bool {
        const int at = k % kRulesItems;
        if (!mbar_wait(bar(kBarItemFull + at), static_cast<uint32_t>(k / kRulesItems) & 1, limit, abort_flag)) return false;
        it = items[at];
        return true;
    };

    if constexpr (CORR) {
        if (warp >= kWarpCorr) {
            regs_decrease<kCorrRegs>();
            rules_correction<D, OutT>(p, smem, bar0, tmem, abort_flag);
        }
    }
    if (warp >= kWarpProducer && !(CORR && warp >= kWarpCorr)) {
        regs_decrease<CORR ? kCorrControlRegs : C::kCtrlRegs>();
        if (warp == kWarpProducer) {
            // ======================================================== producer
            if (lane == 0) {
                prefetch_tensormap(&f.tm_q);
                prefetch_tensormap(&f.tm_k);
                prefetch_tensormap(&f.tm_v);
                if (C::kStoreO) prefetch_tensormap(&f.tm_o);
                const uint64_t pol_q = policy_evict_first();
                const uint64_t pol_kv = policy_evict_last();
                const bool ask = p.counter != nullptr;
                int q_loads[2] = {0, 0};  // loads issued into each Q buffer
                long long g = 0;          // K/V tiles issued so far (ring position)
                int k = 0;                // items published
                bool ok = true;
                const int G = static_cast<int>(gridDim.x);
                int next = ask ? atomicAdd(p.counter, 1) : static_cast<int>(blockIdx.x);  // (asked for one item ahead)
                while (true) {
                    RulesItem it;
                    it.n_kv = -1;
                    if (next < f.n_items) {
                        const int swap = C::kAlternate && p.causal ? k & 1 : 0;
                        if (ask || !p.causal) {  // head by head
                            const int bh = next / f.n_qp;
                            const int qp = next - bh * f.n_qp;
                            next = ask ? atomicAdd(p.counter, 1) : next + G;
                            it = rules_item(p, bh, qp, swap);
                        } else {
                            const int first = next / (p.chunk * f.n_qp) * p.chunk;  // head of the chunk
                            const int many = min(p.chunk, f.BH - first);
                            const int place = next - first * f.n_qp;
                            const int t = place / many;
                            // there and back: the CTA with the longest item of a round has the shortest of the next
                            next = (k + 1) * G + ((k & 1) ? static_cast<int>(blockIdx.x) : G - 1 - static_cast<int>(blockIdx.x));
                            it = rules_item(p, first + place - t * many, f.n_qp - 1 - t, swap);
                        }
                    }
                    const int at = k % kRulesItems;
                    if (k >= kRulesItems &&
                        !mbar_wait(bar(kBarItemEmpty + at), static_cast<uint32_t>(k / kRulesItems - 1) & 1, limit, abort_flag)) {
                        ok = false;
                        break;
                    }
                    items[at] = it;
                    mbar_arrive(bar(kBarItemFull + at));
                    ++k;
                    if (it.n_kv < 0) break;
                    for (int i = 0; i < 2 && ok; ++i) {
                        if (it.n[i] == 0) continue;
                        const int q_bar = 2 * (q_loads[i] % C::kQBuf) + i;
                        if (q_loads[i] >= C::kQBuf &&
                            !mbar_wait(bar(kBarQEmpty + q_bar), (q_loads[i] / C::kQBuf - 1) & 1, limit, abort_flag)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(bar(kBarQFull + q_bar), C::kTileBytes);
#pragma unroll
                        for (int cb = 0; cb < C::kNumCB; ++cb)
                            tma_load_3d(sbase + C::kOffQ + q_bar * C::kTileBytes + cb * C::kBlkBytes, &f.tm_q,
                                        bar(kBarQFull + q_bar), cb * C::kCB, it.r0[i], it.bh, pol_q);
                        ++q_loads[i];
                    }
                    for (int j = 0; ok && j < it.n_kv; ++j, ++g) {
                        const int s = static_cast<int>(g % S);
                        const uint32_t round = static_cast<uint32_t>(g / S);
                        if (g >= S && !mbar_wait(bar(kBarKVEmpty + s), (round - 1) & 1, limit, abort_flag)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(bar(kBarKVFull + s), 2 * C::kTileBytes);
#pragma unroll
                        for (int cb = 0; cb < C::kNumCB; ++cb)
                            tma_load_3d(sbase + C::kOffK + s * C::kTileBytes + cb * C::kBlkBytes, &f.tm_k,
                                        bar(kBarKVFull + s), cb * C::kCB, (it.j0 + j) * kBlockN, it.kv, pol_kv);
#pragma unroll
                        for (int cb = 0; cb < C::kNumCB; ++cb)
                            tma_load_3d(sbase + C::kOffV + s * C::kTileBytes + cb * C::kBlkBytes, &f.tm_v,
                                        bar(kBarKVFull + s), cb * C::kCB, (it.j0 + j) * kBlockN, it.kv, pol_kv);
                    }
                    if (!ok) break;
                }
                if (!ok && !*abort_flag) record_failure(f.status, abort_flag, FA_ERR_TIMEOUT);
                // Every issued copy must land before the CTA may exit (its last phase per barrier).
                for (int i = 0; i < 2; ++i)
                    for (int t = q_loads[i] - C::kQBuf < 0 ? 0 : q_loads[i] - C::kQBuf; t < q_loads[i]; ++t)
                        mbar_wait(bar(kBarQFull + 2 * (t % C::kQBuf) + i), (t / C::kQBuf) & 1, kDrainLimitNs, nullptr);
                for (long long t = g - S < 0 ? 0 : g - S; t < g; ++t)
                    mbar_wait(bar(kBarKVFull + static_cast<int>(t % S)), static_cast<uint32_t>(t / S) & 1, kDrainLimitNs, nullptr);
            }
        } else if (warp == kWarpMma || warp == kWarpMma + 1) {
            // ======================================================== MMA issuers
            if (lane == 0) {
                const int i = warp - kWarpMma;  // query tile of this issuer
                int q_uses = 0;                 // items in which this query tile had key tiles
                int tiles = 0;                  // (query tile, key tile) pairs processed
                int s_issued = 0;               // S_i tiles issued so far
                long long g = 0;                // K/V ring position
                bool ok = true;
                const uint32_t d_s = tmem + C::col_s(i);
                const uint32_t d_o = tmem + C::col_o(i);
                const uint32_t a_p = tmem + C::col_p(i);
                auto issue_s = [&](int q_bar, int stage) {
                    const uint64_t a0 = smem_desc(sbase + C::kOffQ + q_bar * C::kTileBytes, 16, C::kAtomBytes, C::kLayout);
                    const uint64_t b0 = smem_desc(sbase + C::kOffK + stage * C::kTileBytes, 16, C::kAtomBytes, C::kLayout);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk * 16) / C::kCB * C::kBlkBytes + ((kk * 16) % C::kCB) * 2) >> 4;
                        umma_ss(d_s, a0 + off, b0 + off, C::kIdescS, kk > 0 ? 1u : 0u);
                    }
                };
                auto issue_pv = [&](int stage, bool accumulate) {
                    const uint64_t b0 = smem_desc(sbase + C::kOffV + stage * C::kTileBytes, C::kBlkBytes, C::kAtomBytes, C::kLayout);
#pragma unroll
                    for (int kk = 0; kk < kBlockN / 16; ++kk)
                        umma_ts(d_o, a_p + 8u * kk, b0 + ((kk * 16 * C::kRowBytes) >> 4), C::kIdescO,
                                (accumulate || kk > 0) ? 1u : 0u);
                };
                auto kv_full = [&](long long t) -> bool {
                    return mbar_wait(bar(kBarKVFull + static_cast<int>(t % S)), static_cast<uint32_t>(t / S) & 1, limit, abort_flag);
                };
                // S_i of ring tile t: its columns must have been read by the softmax; with P aliased into them the
                // previous P_i V must also have completed.
                auto do_s = [&](int q_bar, long long t, bool last) -> bool {
                    if (!kv_full(t)) return false;
                    if (C::kAliasP) {
                        if (tiles > 0 && !mbar_wait(bar(kBarPVDone + i), (tiles - 1) & 1, limit, abort_flag)) return false;
                    } else {
                        if (s_issued > 0 && !mbar_wait(bar(kBarSFree + i), (s_issued - 1) & 1, limit, abort_flag)) return false;
                    }
                    ++s_issued;
                    tc_fence_after_sync();
                    issue_s(q_bar, static_cast<int>(t % S));
                    umma_commit(bar(kBarSFull + i));
                    if (last) umma_commit(bar(kBarQEmpty + q_bar));  // Q_i no longer read
                    return true;
                };
                for (int k = 0; ok; ++k) {
                    RulesItem it;
                    ok = take(k, it);
                    if (!ok || it.n_kv < 0) break;
                    mbar_arrive(bar(kBarItemEmpty + k % kRulesItems));
                    const int a = i ? it.a[1] : it.a[0];
                    const int n = i ? it.n[1] : it.n[0];
                    const int q_bar = 2 * (q_uses % C::kQBuf) + i;
                    if (n > 0 && !mbar_wait(bar(kBarQFull + q_bar), (q_uses / C::kQBuf) & 1, limit, abort_flag)) {
                        ok = false;
                        break;
                    }
                    for (int j = 0; ok && j < it.n_kv; ++j) {
                        const long long gj = g + j;
                        const int sj = static_cast<int>(gj % S);
                        if (j < a || j >= n) {
                            // key tile this query tile does not visit: release the stage once it is loaded
                            ok = kv_full(gj);
                            if (ok) mbar_arrive(bar(kBarKVEmpty + sj));
                            continue;
                        }
                        if (j == a) ok = do_s(q_bar, gj, n == a + 1);
                        // Without aliasing, S_i(j+1) only needs S_i(j) read: issue it before P_i(j) V_j,
                        // so that it runs while the softmax of tile j is still exponentiating.
                        if (!C::kAliasP && ok && j + 1 < n) ok = do_s(q_bar, gj + 1, j + 1 == n - 1);
                        if (!ok || !mbar_wait(bar(kBarPFull + i), tiles & 1, limit, abort_flag)) {
                            ok = false;
                            break;
                        }
                        // the columns of O_i have been read
                        if constexpr (CORR) {
                            ok = j != a || q_uses == 0 || mbar_wait(bar(kBarOFree + i), (q_uses - 1) & 1, limit, abort_flag);
                            if (!ok) break;
                        }
                        tc_fence_after_sync();
                        issue_pv(sj, j > a);
                        umma_commit(bar(kBarPVDone + i));
                        if (j == n - 1) umma_commit(bar(kBarOReady + i));
                        umma_commit(bar(kBarKVEmpty + sj));
                        ++tiles;
                        if (C::kAliasP && j + 1 < n) ok = do_s(q_bar, gj + 1, j + 1 == n - 1);
                    }
                    if (n > 0) ++q_uses;
                    g += it.n_kv;
                }
                if (!ok && !*abort_flag) record_failure(f.status, abort_flag, FA_ERR_TIMEOUT);
                // Wait for every tensor-core operation this thread issued.
                umma_commit(bar(kBarDrain + i));
                mbar_wait(bar(kBarDrain + i), 0, kDrainLimitNs, nullptr);
            }
        }
    } else if (!CORR || warp < kWarpProducer) {
        regs_increase<CORR ? kCorrSoftmaxRegs : C::kSoftRegs>();
        // ============================================================ softmax + epilogue
        const int wg = warp >> 2;         // query tile of this warpgroup
        const int r = threadIdx.x & 127;  // row within the tile == TMEM lane
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lane_base + C::col_s(wg);
        const uint32_t t_o = tmem + lane_base + C::col_o(wg);
        const uint32_t t_p = tmem + lane_base + C::col_p(wg);
        const int off = f.Nk - f.N;
        int tiles = 0;   // (query tile, key tile) pairs processed by this warpgroup
        int uses = 0;    // items in which this warpgroup had key tiles
        bool ok = true;

        for (int k = 0; ok; ++k) {
            // (read field by field where it is used, so that the tiles' loop does not hold it in registers)
            const volatile RulesItem& it = items[k % kRulesItems];
            ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarItemFull + k % kRulesItems), static_cast<uint32_t>(k / kRulesItems) & 1, limit, abort_flag));
            if (!ok || it.n_kv < 0) break;
            auto release = [&] {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarItemEmpty + k % kRulesItems));
            };
            if (it.rows[wg] == 0) {  // tile lies past N
                release();
                continue;
            }
            const int a = it.a[wg];
            const int n = it.n[wg];
            const int qpos = off + it.r0[wg] + r;
            // the row's keys [lo, hi); rows past N take the last row's
            int lo = 0, hi = f.Nk;
            {
                const int row = it.r0[wg] + min(r, it.rows[wg] - 1);
                if (p.each != nullptr) {
                    const int2 x = p.each[static_cast<size_t>(it.b) * f.N + row];
                    lo = x.x;
                    hi = x.y;
                } else if (p.causal) {
                    hi = min(f.Nk, max(off + row + 1, it.prefix));
                }
            }
            const float slope = kWithBias ? p.rules.slopes[it.bh - it.b * p.Hq] * p.rules.bias_in : 0.f;
            float m_run = -INFINITY;  // running max of the scores in base 2 over visible keys
            float l = 0.f;
            int k0 = (it.j0 + a) * kBlockN;  // first key of the tile
            for (int j = a; j < n; ++j, k0 += kBlockN) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarSFull + wg), tiles & 1, limit, abort_flag));
                if (!ok) break;
                tc_fence_after_sync();
                uint32_t u[kBlockN];
                float mrow;  // the row's largest score, or under a cap the largest absolute one
                if constexpr (D == 128) {
                    float mh[2];
                    if constexpr (kWithCap) {
                        tmem_ld64_absmax(t_s + 0, *reinterpret_cast<uint32_t(*)[64]>(&u[0]), mh[0]);
                        tmem_ld64_absmax(t_s + 64, *reinterpret_cast<uint32_t(*)[64]>(&u[64]), mh[1]);
                    } else {
                        tmem_ld64_max(t_s + 0, *reinterpret_cast<uint32_t(*)[64]>(&u[0]), mh[0]);
                        tmem_ld64_max(t_s + 64, *reinterpret_cast<uint32_t(*)[64]>(&u[64]), mh[1]);
                    }
                    tmem_ld_wait();
                    mrow = fmaxf(mh[0], mh[1]);
                } else {
                    float mq[4];
                    if constexpr (kWithCap) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            tmem_ld32_absmax(t_s + 32u * q, *reinterpret_cast<uint32_t(*)[32]>(&u[32 * q]), mq[q]);
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            tmem_ld32_max(t_s + 32u * q, *reinterpret_cast<uint32_t(*)[32]>(&u[32 * q]), mq[q]);
                    }
                    tmem_ld_wait();
                    mrow = max3(mq[0], mq[1], fmaxf(mq[2], mq[3]));
                }
                if constexpr (!C::kAliasP) {  // S_i is in registers: its columns may be overwritten
                    tc_fence_before_sync();
                    mbar_arrive(bar(kBarSFree + wg));
                }
                float s[kBlockN];
#pragma unroll
                for (int c = 0; c < kBlockN; ++c) s[c] = __uint_as_float(u[c]);
                const bool mask = !__all_sync(0xffffffffu, lo <= k0 && hi >= k0 + kBlockN);
                // Raises the running max to mt; the weights are then 2^(score - m_use).
                bool grow;
                float alpha = 1.f, m_use;
                auto raise = [&](float mt) {
                    grow = mt > m_run;
                    if (grow) {
                        alpha = ex2(m_run - mt);  // 0 when m_run = -inf
                        m_run = mt;
                    }
                    m_use = m_run == -INFINITY ? 0.f : m_run;
                };
                float2 rs[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                uint32_t pk[kBlockN / 2];  // weights, rounded to bf16 for the product with V (half a step, 2^-8 of each)
                // Weights of scores g(s, -max), their sums in four running pairs.
                auto weigh = [&](auto g) {
                    const float2 negm = two(-m_use);
#pragma unroll
                    for (int c = 0; c < kBlockN; c += 8) {
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const float2 x = g(make_float2(s[c + 2 * h], s[c + 2 * h + 1]), negm);
                            const float2 e = make_float2(ex2(x.x), ex2(x.y));
                            rs[h] = __fadd2_rn(rs[h], e);
                            pk[c / 2 + h] = pack_bf16x2(e.x, e.y);
                        }
                    }
                };
                // Test whether P_i(j-1) V_{j-1} has completed before the exponentials; the answer is needed after them.
                bool pv_ready = true;
                auto test_pv = [&] {
                    if (!C::kAliasP && j > a) pv_ready = mbar_test(bar(kBarPVDone + wg), (tiles - 1) & 1);
                };
                int range = 0;
                // What hidden scores hold is looked at here, the range asked for on both sides, or, for a cap alone at d = 128, under
                // the scores that are not in the near range.  (Whichever spills less: d = 128 64 x 1024 tokens cap and bias 746
                // and 810 us, 4 x 4097 cap 368 and 360; d = 64 64 x 1024 in documents, cap 30 220 and 225.)
                constexpr bool kCutHere = kWithBias || D < 128;
                if constexpr (kWithCap && kCutHere) {
                    if (mask) {
                        range = cap_range(p.rules, mrow);
                        if (range == 0) range = cap_range_seen<kBlockN>(p.rules, s, mrow, lo - k0, hi - k0);
                    } else {
                        range = cap_range(p.rules, mrow);
                    }
                } else if constexpr (kWithCap) {
                    range = cap_range(p.rules, mrow);
                }
                bool done = false;
                if (kWithCap && !kWithBias && range == 3 && !mask) {
                    // tanh rises with its argument: the largest raw score is the largest capped one
                    const float2 top = two(max_of<kBlockN>(s));
                    raise(__fmul2_rn(top, cap_factor(top, p.rules.near)).x);
                    test_pv();
                    weigh([&](float2 x, float2 m) { return __ffma2_rn(x, cap_factor(x, p.rules.near), m); });
                    done = true;
                }
                bool before = false, behind = false;  // every key that counts lies at or before, behind every row's position
                if constexpr (kWithBias) {
                    // (keys behind a causal row's position are hidden, whatever bias they get)
                    before = __all_sync(0xffffffffu, k0 + kBlockN - 1 <= qpos || (p.causal && hi <= qpos + 1));
                    behind = __all_sync(0xffffffffu, k0 >= qpos);
                }
                if (!done) {
                    if (kWithCap && !kCutHere && range == 0 && mask) range = cap_range_seen<kBlockN>(p.rules, s, mrow, lo - k0, hi - k0);
                    if constexpr (kWithBias) {
                        biased_scores<kBlockN, kWithCap>(s, p.rules, range, p.rules.far, slope, static_cast<float>(qpos - k0), before ? 1 : behind ? -1 : 0);
                    } else if constexpr (kWithCap) {
                        capped_scores<kBlockN>(s, p.rules, range, p.rules.far);
                    }
                    if (mask) rules_mask(s, lo - k0, hi - k0);
                    if (RULES != kNoRules || mask) mrow = max_of<kBlockN>(s);
                    if constexpr (RULES == kCap) {
                        raise(mrow);
                        test_pv();
                        weigh([&](float2 x, float2 m) { return __fadd2_rn(x, m); });
                    } else {
                        raise(mrow * p.rules.mult);
                        test_pv();
                        weigh([&](float2 x, float2 m) { return __ffma2_rn(x, two(p.rules.mult), m); });
                    }
                }
                // O_i and the P_i columns are free once P_i(j-1) V_{j-1} has completed.  With P aliased into S_i this is
                // implied by the arrival of S_i(j); otherwise wait for it.
                if (!C::kAliasP && j > a) {
                    ok = __all_sync(0xffffffffu, pv_ready || mbar_wait(bar(kBarPVDone + wg), (tiles - 1) & 1, limit, abort_flag));
                    if (!ok) break;
                    tc_fence_after_sync();
                }
                if (j > a && __any_sync(0xffffffffu, grow)) {
                    constexpr int kRescale = D <= 64 ? D : 32;  // columns at a time (registers)
                    const float2 a2 = make_float2(alpha, alpha);
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += kRescale) {
                        uint32_t oc[kRescale];
#pragma unroll
                        for (int c = 0; c < kRescale; c += 32)
                            tmem_ld32(t_o + static_cast<uint32_t>(c0 + c), *reinterpret_cast<uint32_t(*)[32]>(&oc[c]));
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < kRescale; e += 2) {
                            const float2 v = __fmul2_rn(make_float2(__uint_as_float(oc[e]), __uint_as_float(oc[e + 1])), a2);
                            oc[e] = __float_as_uint(v.x);
                            oc[e + 1] = __float_as_uint(v.y);
                        }
#pragma unroll
                        for (int c = 0; c < kRescale; c += 32)
                            tmem_st32(t_o + static_cast<uint32_t>(c0 + c), *reinterpret_cast<uint32_t(*)[32]>(&oc[c]));
                    }
                }
                tmem_st32(t_p + 0, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
                tmem_st32(t_p + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
                tmem_st_wait();
                tc_fence_before_sync();
                mbar_arrive(bar(kBarPFull + wg));
                l = l * alpha + (((rs[0].x + rs[0].y) + (rs[1].x + rs[1].y)) + ((rs[2].x + rs[2].y) + (rs[3].x + rs[3].y)));
                ++tiles;
            }
            if (!ok) break;
            if constexpr (CORR) {
                const bool none = l == 0.f;
                if (n > 0) {  // 1 / l to the correction warpgroup, once it has read the last item's
                    if (uses > 0) {
                        ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarOFree + wg), (uses - 1) & 1, limit, abort_flag));
                        if (!ok) break;
                    }
                    reinterpret_cast<float*>(smem + C::kOffInv)[wg * kBlockM + r] = none ? 0.f : 1.f / l;
                    mbar_arrive(bar(kBarLFull + wg));
                    ++uses;
                }
                const size_t row = static_cast<size_t>(it.bh) * f.N + static_cast<size_t>(it.r0[wg] + r);
                const bool valid = r < it.rows[wg];
                release();
                if (valid && f.lse != nullptr) f.lse[row] = none ? -INFINITY : (m_run + lg2_approx(l)) * kLn2;
                continue;
            }
            if (n > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarOReady + wg), uses & 1, limit, abort_flag));
                if (!ok) break;
                ++uses;
                tc_fence_after_sync();
            }
            const bool none = l == 0.f;  // a row that sees no key: O = 0, LSE = -inf
            const bool hide = __any_sync(0xffffffffu, none);
            const float inv = none ? 0.f : 1.f / l;
            const int bh = it.bh, row0 = it.r0[wg];
            const size_t row = static_cast<size_t>(bh) * f.N + static_cast<size_t>(row0 + r);
            const bool valid = r < it.rows[wg];
            release();
            if constexpr (C::kStoreO) {
                using OS = OStage<OutT, D>;
                const uint32_t stg = sbase + C::kOffStage + static_cast<uint32_t>(wg) * C::kStageTileBytes;
                // Each warp stages its 32 rows and stores them itself (a 32-row box): lane 0 first waits until the
                // warp's previous store has read its rows (issued one item ago, long done).
                const int wq = warp & 3;
                if (lane == 0) bulk_wait_read_all();
                __syncwarp();
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    if (n > 0) {
                        tmem_ld32(t_o + static_cast<uint32_t>(c), o);
                        tmem_ld_wait();
                    }
                    if (n == 0 || hide) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = n == 0 || none ? 0u : o[e];
                    }
                    stage_cols<OutT, D>(stg, r, c, o, inv);
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0 && row0 + 32 * wq < f.N) {  // rows past N lie outside the map and are skipped
#pragma unroll
                    for (int cb = 0; cb < OS::kNumCB; ++cb)
                        tma_store_3d(&f.tm_o, stg + cb * OS::kBlkBytes + wq * 32 * OS::kRowBytes, cb * OS::kElems,
                                     row0 + 32 * wq, bh);
                    bulk_commit_group();
                }
            } else {
                OutT* orow = reinterpret_cast<OutT*>(f.o) + row * D;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    float v[32];
                    uint32_t o[32];
                    if (n > 0) {
                        tmem_ld32(t_o + 32u * c, o);
                        tmem_ld_wait();
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = n == 0 || none ? 0.f : __uint_as_float(o[e]) * inv;
                    if (valid) store_row32<OutT>(orow + 32 * c, v);
                }
            }
            if (valid && f.lse != nullptr) f.lse[row] = none ? -INFINITY : (m_run + lg2_approx(l)) * kLn2;
        }
        // Bulk stores must finish before the CTA's shared memory goes away.
        if (C::kStoreO && lane == 0) bulk_wait_all();
        if (!ok && !*abort_flag) record_failure(f.status, abort_flag, FA_ERR_TIMEOUT);
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == kWarpMma) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

template <int D, int RULES, bool CORR, typename OutT>
cudaError_t launch_fwd_rules_t(const FwdRulesParams& p, cudaStream_t st)
{
    using C = RulesCfg<D, static_cast<int>(sizeof(OutT))>;
    constexpr int kThreads = CORR ? 512 : kFwdThreads;
    auto kern = fa_rules_fwd_kernel<D, RULES, CORR, OutT>;
    static bool configured[64] = {};  // attributes set and registers checked, per device
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
        // a register increase that the launch's pool cannot satisfy would wait forever
        constexpr int kNeed = CORR ? 256 * kCorrSoftmaxRegs + 128 * (kCorrRegs + kCorrControlRegs)
                                                   : 256 * C::kSoftRegs + 128 * C::kCtrlRegs;
        if (attr.numRegs * kThreads < kNeed) return cudaErrorLaunchOutOfResources;
        configured[dev] = true;
    }
    const int grid = p.f.n_items < p.f.num_ctas ? p.f.n_items : p.f.num_ctas;
    return launch_pdl(kern, static_cast<unsigned>(grid), kThreads, C::kSmem, st, p);
}

template <int D, int RULES>
cudaError_t launch_fwd_rules_d(const FwdRulesParams& p, fa_dtype o_dtype, cudaStream_t st)
{
    if constexpr (kRulesCorr<D, RULES>) {
        if (p.causal == 0)
            return o_dtype == FA_F32 ? launch_fwd_rules_t<D, RULES, true, float>(p, st)
                                     : launch_fwd_rules_t<D, RULES, true, __nv_bfloat16>(p, st);
    }
    return o_dtype == FA_F32 ? launch_fwd_rules_t<D, RULES, false, float>(p, st)
                             : launch_fwd_rules_t<D, RULES, false, __nv_bfloat16>(p, st);
}

}  // namespace fa

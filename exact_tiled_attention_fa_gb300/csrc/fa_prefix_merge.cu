// fa_prefix_merge.cu -- joins what the shared prefix and its own keys gave each row of fa_decode_prefix.
//
// Either side of a row is one result of its unit, or the parts of a unit that several shares hold (fa_tree_kernel.cuh):
//   lse = log sum_s exp(lse_s),  o = sum_s exp(lse_s - lse) o_s
// over all of them ("flash_lab.py", section 4).  A warp a row.  The time is that of three loads one behind the other
// (the units' records, the log-sum-exps, the outputs) and of the launch; up to FEW results are loaded beside their
// log-sum-exps.  More of them take registers, which counts where there are many rows.  Whole calls at FEW = 8, 12 and 16, us,
// 32/8 heads of 128: 16 sequences behind 8192 tokens, 13 parts a row 32.2, 32.1 and 28.6; 64 behind 32K, 10 parts 89.9, 87.1 and
// 89.7; 256 behind 8192 86.5, 88.5 and 92.  By rows, as the lengths are known on the device alone; few rows that also have
// few parts would do with 8: 2 behind 512 11.6, 11.8 and 13.0, 37 behind 3001, 15/5 heads of 64, 19.3, 20.3 and 21.3.
#include <cuda_bf16.h>

#include <type_traits>

#include "fa_rules_common.cuh"

namespace fa {

template <int D, int FEW>
__global__ void __launch_bounds__(256) fa_prefix_merge_kernel(const __grid_constant__ PrefixMergeParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int V = D / 32;  // columns of a lane
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);  // (b, key/value head, r)
    if (row >= static_cast<long long>(p.B) * p.Hkv * p.R) return;
    const int group = static_cast<int>(row / p.R);
    const int r = static_cast<int>(row - static_cast<long long>(group) * p.R);
    const int b = group / p.Hkv, kvh = group - b * p.Hkv;
    // the row's place in its prefix unit
    const int qp = b / p.seqs;  // query tile
    const int row_pre = (b - qp * p.seqs) * p.R + r;
    // A unit's record, or none: where a wait ran out it may not have been written, and what stands there is not to be
    // followed out of the slots.
    auto record = [&](const TreeJoin* at) -> TreeJoin {
        TreeJoin j = *at;
        if (j.rows < 0 || j.rows >= p.num_shares || j.parts < 0 || j.parts > p.num_shares - j.rows) j = TreeJoin{0, 0, 0};
        return j;
    };
    TreeJoin jp{0, 0, 0};
    const TreeJoin jo = record(p.own.units + group);
    if (p.pre.units != nullptr) jp = record(p.pre.units + (kvh * p.n_qp + qp));
    else if (jo.parts == 1) return;  // written where it was made
    const int n1 = jp.parts, n = n1 + jo.parts;
    // row of result s among its side's, and that side's arrays
    auto place = [&](int s, const float*& o, const float*& lse) -> size_t {
        const bool pre = s < n1;
        const PrefixSide& side = pre ? p.pre : p.own;
        const TreeJoin& j = pre ? jp : jo;
        const int k = pre ? s : s - n1;
        if (j.parts == 1) {
            o = side.o_whole;
            lse = side.lse_whole;
            return pre ? (static_cast<size_t>(kvh) * p.B + b) * p.R + r : static_cast<size_t>(row);
        }
        o = p.o_part;
        lse = p.lse_part;
        return static_cast<size_t>(2 * (j.rows + k) + (k == 0 ? 1 : 0)) * p.part_rows + static_cast<size_t>(pre ? row_pre : r);
    };
    auto load = [&](int s, float (&v)[V]) {
        const float *o, *lse;
        const float* src = nullptr;
        const size_t at = place(s, o, lse);
        src = o + at * D + lane * V;
        if constexpr (V == 4) *reinterpret_cast<float4*>(v) = __ldcg(reinterpret_cast<const float4*>(src));
        else if constexpr (V == 2) *reinterpret_cast<float2*>(v) = __ldcg(reinterpret_cast<const float2*>(src));
        else v[0] = __ldcg(src);
    };
    auto load_lse = [&](int s) -> float {
        if (s >= n) return -INFINITY;
        const float *o, *lse;
        const size_t at = place(s, o, lse);
        return __ldcg(lse + at);
    };
    float acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
    float M = -INFINITY, sum = 0.f;
    bool live = false;
    if (n <= FEW) {
        float x[FEW], v[FEW][V];
#pragma unroll
        for (int s = 0; s < FEW; ++s) {
            x[s] = load_lse(s);
            if (s < n) load(s, v[s]);
        }
#pragma unroll
        for (int s = 0; s < FEW; ++s) {
            live = live || x[s] != -INFINITY;
            M = fmaxf(M, x[s]);
        }
#pragma unroll
        for (int s = 0; s < FEW; ++s) {
            x[s] = x[s] == -INFINITY ? 0.f : ex2((x[s] - M) * kLog2e);
            sum += x[s];
        }
        const float inv = live ? 1.f / sum : 0.f;
#pragma unroll
        for (int s = 0; s < FEW; ++s) {
            if (s >= n) continue;
            const float f = x[s] * inv;  // an empty result is 0
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = fmaf(f, v[s][e], acc[e]);
        }
    } else {
        constexpr int kHeld = 2 * kTreeMaxShares / 32;  // log-sum-exps a lane holds: at most a part for each share and side
        float x[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            x[i] = 32 * i < n ? load_lse(32 * i + lane) : -INFINITY;
            live = live || x[i] != -INFINITY;
            M = fmaxf(M, x[i]);
        }
        live = __any_sync(0xffffffffu, live);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            x[i] = x[i] == -INFINITY ? 0.f : ex2((x[i] - M) * kLog2e);
            sum += x[i];
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = live ? 1.f / sum : 0.f;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int m = min(32, n - 32 * i);
#pragma unroll 8
            for (int j = 0; j < m; ++j) {
                const float f = __shfl_sync(0xffffffffu, x[i], j) * inv;
                float v[V];
                load(32 * i + j, v);
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] = fmaf(f, v[e], acc[e]);
            }
        }
    }
    const size_t out = static_cast<size_t>(row) * D + lane * V;
    if (p.o_dtype == FA_F32) {
        float* o = static_cast<float*>(p.o) + out;
        if constexpr (V == 4) *reinterpret_cast<float4*>(o) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        else if constexpr (V == 2) *reinterpret_cast<float2*>(o) = make_float2(acc[0], acc[1]);
        else o[0] = acc[0];
    } else {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + out;
        if constexpr (V == 4) *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
        else if constexpr (V == 2) *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(acc[0], acc[1]);
        else o[0] = __float2bfloat16_rn(acc[0]);
    }
    if (lane == 0 && p.lse != nullptr) p.lse[row] = live ? M + log2f(sum) * kLn2 : -INFINITY;
}

cudaError_t launch_prefix_merge(const PrefixMergeParams& p, int d, cudaStream_t st)
{
    const long long rows = static_cast<long long>(p.B) * p.Hkv * p.R;
    const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
    auto with = [&](auto few) {
        switch (d) {
        case 32: return launch_pdl(fa_prefix_merge_kernel<32, few()>, grid, 256, 0, st, p);
        case 64: return launch_pdl(fa_prefix_merge_kernel<64, few()>, grid, 256, 0, st, p);
        case 128: return launch_pdl(fa_prefix_merge_kernel<128, few()>, grid, 256, 0, st, p);
        default: return cudaErrorInvalidValue;
        }
    };
    if (rows <= 1024) return with(std::integral_constant<int, 16>());
    return rows <= 4096 ? with(std::integral_constant<int, 12>()) : with(std::integral_constant<int, 8>());
}

}  // namespace fa

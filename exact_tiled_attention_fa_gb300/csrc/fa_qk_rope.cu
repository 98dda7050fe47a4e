// fa_qk_rope.cu -- norm of queries and keys for each head with the position rotation in the same
// pass, its gradient, and the form that writes a key/value cache.
//
// Mathematics.  For a row x (one head of one token, d elements) with weights w and the angles of
// its position, r = 1 / sqrt(mean x^2 + eps), y = x r w, and each pair (y_a, y_b) of the first `rot`
// elements becomes (y_a c - y_b s, y_a s + y_b c), c and s read from tables.  Pairs are (i, i + rot/2)
// or, interleaved, (2i, 2i + 1).  Values pass through unchanged.
// Backward, for the gradient g of the rotated row: h = the rotation by the opposite angle applied to
// g (its transpose), dw = sum over rows of h x r, and with z = w h
//   dx = r (z - x r^2 mean(x z)).
// Where key/value heads were written once per query head, g is first summed over the copies.
// All of it is fp32; each output element is rounded once.
//
// What bounds it: bytes.  A row is read and written once, 16 bytes a lane; D / 8 lanes share a row,
// so the sums are a few shuffles.  A warp takes one token and walks its heads, holding the token's
// cosines and sines in registers, with U rows' loads in flight; neighbouring warps take neighbouring
// tokens, whose rows are neighbours in the head-major output.
#include <cuda_bf16.h>

#include <cstdint>

#include "fa_internal.h"
#include "fa_kernel_common.cuh"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kRopeWarps = 8;

__device__ __forceinline__ void unpack_bf16(const uint4 u, float (&f)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack_bf16(const float (&f)[8])
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// Eight weights at element c.
__device__ __forceinline__ void load_weights(const void* w, fa_dtype t, int c, float (&f)[8])
{
    if (t == FA_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __ldg(reinterpret_cast<const float*>(w) + c + i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[c + i]);
    }
}

// The rotation of a lane's eight elements.  Halves: out = x c + partner s, the partner's elements
// held by another lane of the row and s carrying the sign (-sin in the first half, +sin in the
// second; 0, with c = 1, past rot).  Interleaved: four pairs within the lane.
template <bool INTERLEAVED>
struct Turn {
    float c[INTERLEAVED ? 4 : 8], s[INTERLEAVED ? 4 : 8];
    int partner;  // lane of the partner elements

    __device__ __forceinline__ void load(const float* cos_t, const float* sin_t, int pos, int rot, int sub, int lane, float sign)
    {
        const int half = rot >> 1;
        const int e = sub * 8;
        partner = lane;
        if constexpr (INTERLEAVED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = 1.f;
                s[i] = 0.f;
            }
            if (e < rot) {
                const size_t at = static_cast<size_t>(pos) * half + (e >> 1);
                const float4 x = __ldg(reinterpret_cast<const float4*>(cos_t + at));
                const float4 y = __ldg(reinterpret_cast<const float4*>(sin_t + at));
                c[0] = x.x, c[1] = x.y, c[2] = x.z, c[3] = x.w;
                s[0] = sign * y.x, s[1] = sign * y.y, s[2] = sign * y.z, s[3] = sign * y.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = 1.f;
                s[i] = 0.f;
            }
            if (e < rot) {
                const bool second = e >= half;
                const size_t at = static_cast<size_t>(pos) * half + (second ? e - half : e);
                const float sg = second ? sign : -sign;
                partner = second ? lane - (half >> 3) : lane + (half >> 3);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float4 x = __ldg(reinterpret_cast<const float4*>(cos_t + at) + q);
                    const float4 y = __ldg(reinterpret_cast<const float4*>(sin_t + at) + q);
                    c[4 * q] = x.x, c[4 * q + 1] = x.y, c[4 * q + 2] = x.z, c[4 * q + 3] = x.w;
                    s[4 * q] = sg * y.x, s[4 * q + 1] = sg * y.y, s[4 * q + 2] = sg * y.z, s[4 * q + 3] = sg * y.w;
                }
            }
        }
    }
    // Whole warp.
    __device__ __forceinline__ void apply(float (&y)[8]) const
    {
        if constexpr (INTERLEAVED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = y[2 * i], b = y[2 * i + 1];
                y[2 * i] = fmaf(a, c[i], -b * s[i]);
                y[2 * i + 1] = fmaf(a, s[i], b * c[i]);
            }
        } else {
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, y[i], partner);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = s[i] == 0.f ? y[i] * c[i] : fmaf(y[i], c[i], o[i] * s[i]);
        }
    }
};

template <int LANES>
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int o = LANES / 2; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ int checked_position(int pos, int max_pos, int* status)
{
    if (pos < 0 || pos >= max_pos) {
        atomicCAS(status, 0, FA_ERR_INVALID_ARG);
        pos = pos < 0 ? 0 : max_pos - 1;
    }
    return pos;
}

// Depth of node t: the number of its ancestors.  Whole warp, t < 128: the warp holds the parents,
// so a step up is a shuffle instead of a load that waits for the one before it.
__device__ __forceinline__ int tree_depth(const int* parents, int t, int lane, int* status)
{
    int par[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) par[i] = 32 * i + lane <= t ? __ldg(parents + 32 * i + lane) : -1;
    int depth = 0;
    for (int cur = t;;) {  // strictly decreasing
        const int sel = (cur >> 5) == 0 ? par[0] : (cur >> 5) == 1 ? par[1] : (cur >> 5) == 2 ? par[2] : par[3];
        int up = __shfl_sync(0xffffffffu, sel, cur & 31);
        if (up >= cur || up < -1) {
            if (lane == 0) atomicCAS(status, 0, FA_ERR_INVALID_ARG);
            up = -1;
        }
        if (up < 0) return depth;
        ++depth;
        cur = up;
    }
}

// Grid (tokens / kRopeWarps, head chunks).  A warp: one token, heads blockIdx.y * chunk .. + chunk of
// the Hq query heads, Hkv key heads and Hkv value heads in this order.
// APPEND: token t of sequence b is node t of its tree, at position seqlens[b] + depth, and its key
// and value go to cache row seqlens[b] + t.  Nodes past n_nodes[b] have zero query rows and no cache
// row.
template <int D, bool INTERLEAVED, bool APPEND>
__global__ void __launch_bounds__(kRopeWarps * 32) fa_qk_rope_kernel(const RopeParams p, int heads, int chunk)
{
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int LPR = D / 8;    // lanes of a row
    constexpr int RPW = 32 / LPR; // rows of a warp's step
    constexpr int U = 4;          // steps in flight
    const int lane = threadIdx.x & 31;
    const int sub = lane % LPR;
    const int grp = lane / LPR;
    const long long token = static_cast<long long>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
    if (token >= static_cast<long long>(p.B) * p.N) return;
    const int b = static_cast<int>(token / p.N);
    const int t = static_cast<int>(token - static_cast<long long>(b) * p.N);

    bool live = true;  // APPEND: the node is part of the tree
    int row = t;       // row of the key and value in their head
    int pos;
    if constexpr (APPEND) {
        const int len = p.seqlens[b];
        const int nodes = p.n_nodes != nullptr ? p.n_nodes[b] : p.N;
        const bool bad = len < 0 || len > p.Nk_max || nodes < 0 || nodes > p.N || len > p.Nk_max - nodes;
        const int from = min(max(len, 0), p.Nk_max);
        const int n = min(min(max(nodes, 0), p.N), p.Nk_max - from);
        if (bad && lane == 0) atomicCAS(p.status, 0, FA_ERR_INVALID_ARG);
        live = t < n;
        row = from + t;
        pos = 0;
        if (live) {
            pos = from + (p.parents != nullptr ? tree_depth(p.parents + static_cast<size_t>(b) * p.N, t, lane, p.status) : t);
            pos = checked_position(pos, p.max_pos, p.status);
        }
    } else {
        pos = checked_position(p.positions != nullptr ? p.positions[token] : t, p.max_pos, p.status);
    }
    Turn<INTERLEAVED> turn;
    turn.load(p.cos_t, p.sin_t, pos, p.rot, sub, lane, 1.f);
    float wq[8], wk[8];
    load_weights(p.wq, p.w_dtype, sub * 8, wq);
    load_weights(p.wk, p.w_dtype, sub * 8, wk);
    const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(p.q) + token * p.q_stride + sub * 8;
    const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(p.k) + token * p.k_stride + sub * 8;
    const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(p.v) + token * p.v_stride + sub * 8;
    const size_t kv_rows = APPEND ? p.Nk_max : p.N;
    const int h_end = min(heads, (static_cast<int>(blockIdx.y) + 1) * chunk);

    for (int h0 = static_cast<int>(blockIdx.y) * chunk; h0 < h_end; h0 += U * RPW) {
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * RPW + grp;
            const __nv_bfloat16* src = h < p.Hq ? q + static_cast<size_t>(h) * D
                                     : h < p.Hq + p.Hkv ? k + static_cast<size_t>(h - p.Hq) * D
                                                        : v + static_cast<size_t>(h - p.Hq - p.Hkv) * D;
            raw[u] = h < h_end ? ld_stream_v4(src) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * RPW + grp;
            if (h0 + u * RPW >= h_end) break;  // uniform
            float x[8];
            unpack_bf16(raw[u], x);
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
            const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
            const bool is_q = h < p.Hq;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (is_q ? wq[i] : wk[i]);
            turn.apply(x);
            if (h < h_end && is_q) {
                const uint4 y = APPEND && !live ? make_uint4(0, 0, 0, 0) : pack_bf16(x);
                __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.q_out) +
                                     ((static_cast<size_t>(b) * p.Hq + h) * p.N + t) * D + sub * 8;
                *reinterpret_cast<uint4*>(dst) = y;
            } else if (h < h_end && (!APPEND || live)) {
                const bool is_k = h < p.Hq + p.Hkv;
                const int hk = is_k ? h - p.Hq : h - p.Hq - p.Hkv;
                const uint4 y = is_k ? pack_bf16(x) : raw[u];
                __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(is_k ? p.k_out : p.v_out) +
                                     ((static_cast<size_t>(b) * p.Hkv + hk) * p.copies * kv_rows + row) * D + sub * 8;
                for (int c = 0; c < p.copies; ++c) *reinterpret_cast<uint4*>(dst + static_cast<size_t>(c) * kv_rows * D) = y;
            }
        }
    }
}

template <int D, bool INTERLEAVED>
cudaError_t launch_rope_t(const RopeParams& p, bool append, int sms, cudaStream_t st)
{
    constexpr int RPW = 32 / (D / 8);
    const long long tokens = static_cast<long long>(p.B) * p.N;
    const long long blocks = (tokens + kRopeWarps - 1) / kRopeWarps;
    const int heads = p.Hq + p.Hkv + (p.v != nullptr ? p.Hkv : 0);
    // With few tokens the heads of one are shared out among warps, a step of RPW heads at least
    const int steps = (heads + RPW - 1) / RPW;
    long long chunks = (4LL * sms + blocks - 1) / blocks;
    if (chunks > steps) chunks = steps;
    const int chunk = static_cast<int>((steps + chunks - 1) / chunks) * RPW;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((heads + chunk - 1) / chunk));
    return append ? launch_pdl(fa_qk_rope_kernel<D, INTERLEAVED, true>, grid, kRopeWarps * 32, 0, st, p, heads, chunk)
                  : launch_pdl(fa_qk_rope_kernel<D, INTERLEAVED, false>, grid, kRopeWarps * 32, 0, st, p, heads, chunk);
}

// ---- backward ----------------------------------------------------------------------------------

// Eight gradient elements at g.
__device__ __forceinline__ void load_grad(const void* g, bool f32, size_t at, float (&f)[8])
{
    if (f32) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(g) + at));
        const float4 c = __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(g) + at) + 1);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = c.x, f[5] = c.y, f[6] = c.z, f[7] = c.w;
    } else {
        unpack_bf16(ld_stream_v4(reinterpret_cast<const __nv_bfloat16*>(g) + at), f);
    }
}

__device__ __forceinline__ void store_grad(void* o, bool f32, size_t at, const float (&f)[8])
{
    if (f32) {
        float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(o) + at);
        dst[0] = make_float4(f[0], f[1], f[2], f[3]);
        dst[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(o) + at) = pack_bf16(f);
    }
}

// A fixed number of CTAs walk the tokens, a warp a token at a time; the weights' gradients stay in
// registers (eight columns of each a lane) until the CTA adds its warps' up in a fixed order and
// writes one partial row of each, which fa_rope_weight_kernel adds up, also in a fixed order: the
// result does not change from run to run.
template <int D, bool INTERLEAVED, bool GF32>
__global__ void __launch_bounds__(kRopeWarps * 32) fa_qk_rope_bwd_kernel(const RopeBwdParams p, int heads)
{
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int LPR = D / 8;
    constexpr int RPW = 32 / LPR;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int sub = lane % LPR;
    const int grp = lane / LPR;
    const bool of32 = p.out_dtype == FA_F32;
    float wq[8], wk[8], aq[8], ak[8];
    load_weights(p.wq, p.w_dtype, sub * 8, wq);
    load_weights(p.wk, p.w_dtype, sub * 8, wk);
#pragma unroll
    for (int i = 0; i < 8; ++i) aq[i] = ak[i] = 0.f;
    const long long tokens = static_cast<long long>(p.B) * p.N;
    for (long long token = static_cast<long long>(blockIdx.x) * kRopeWarps + warp; token < tokens;
         token += static_cast<long long>(gridDim.x) * kRopeWarps) {
        const int b = static_cast<int>(token / p.N);
        const int t = static_cast<int>(token - static_cast<long long>(b) * p.N);
        const int pos = checked_position(p.positions != nullptr ? p.positions[token] : t, p.max_pos, p.status);
        Turn<INTERLEAVED> turn;
        turn.load(p.cos_t, p.sin_t, pos, p.rot, sub, lane, -1.f);
        const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(p.q) + token * p.q_stride + sub * 8;
        const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(p.k) + token * p.k_stride + sub * 8;
        for (int h0 = 0; h0 < heads; h0 += RPW) {
            const int h = h0 + grp;
            const bool in = h < heads;
            const bool is_q = h < p.Hq;
            const bool is_v = h >= p.Hq + p.Hkv;
            const int hk = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
            float x[8], g[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = g[i] = 0.f;
            if (in) {
                if (!is_v) unpack_bf16(ld_stream_v4(is_q ? q + static_cast<size_t>(h) * D : k + static_cast<size_t>(hk) * D), x);
                const void* src = is_q ? p.dq : is_v ? p.dv : p.dk;
                const int n = is_q ? 1 : p.copies;
                const size_t head0 = is_q ? static_cast<size_t>(b) * p.Hq + h : (static_cast<size_t>(b) * p.Hkv + hk) * p.copies;
                for (int c = 0; c < n; ++c) {
                    float y[8];
                    load_grad(src, GF32, ((head0 + c) * p.N + t) * D + sub * 8, y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[i] += y[i];
                }
            }
            float plain[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) plain[i] = g[i];
            turn.apply(g);
            float ss = 0.f, sz = 0.f, z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                z[i] = (is_q ? wq[i] : wk[i]) * g[i];
                ss = fmaf(x[i], x[i], ss);
                sz = fmaf(x[i], z[i], sz);
            }
            ss = row_sum<LPR>(ss);
            sz = row_sum<LPR>(sz);
            const float r = rsqrtf(ss * (1.f / D) + p.eps);
            const float f = r * r * sz * (1.f / D);
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float dw = g[i] * x[i] * r;  // 0 for value rows and lanes without a row (x = 0)
                aq[i] += is_q ? dw : 0.f;
                ak[i] += is_q ? 0.f : dw;
                o[i] = is_v ? plain[i] : r * (z[i] - x[i] * f);
            }
            if (in) {
                void* dst = is_q ? p.gq : is_v ? p.gv : p.gk;
                const long long stride = is_q ? p.gq_stride : is_v ? p.gv_stride : p.gk_stride;
                store_grad(dst, of32, static_cast<size_t>(token * stride) + static_cast<size_t>(is_q ? h : hk) * D + sub * 8, o);
            }
        }
    }
    __shared__ float sm[kRopeWarps][2][D];
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            aq[i] += __shfl_xor_sync(0xffffffffu, aq[i], o);
            ak[i] += __shfl_xor_sync(0xffffffffu, ak[i], o);
        }
    if (grp == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sm[warp][0][sub * 8 + i] = aq[i];
            sm[warp][1][sub * 8 + i] = ak[i];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kRopeWarps * 32) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kRopeWarps; ++w) s += sm[w][i / D][i % D];
        p.part[static_cast<size_t>(blockIdx.x) * 2 * D + i] = s;
    }
}

// Sums the partial rows: block y (0 query, 1 key weights) x 32 columns, 32 slices of the rows each.
__global__ void __launch_bounds__(1024) fa_rope_weight_kernel(const float* part, int n, int d, float* gwq, float* gwk)
{
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ float sm[32][33];
    const int col = static_cast<int>(blockIdx.x) * 32 + static_cast<int>(threadIdx.x & 31);
    const int slice = threadIdx.x >> 5;
    float s = 0.f;
#pragma unroll 8
    for (int c = slice; c < n; c += 32) s += __ldg(part + (static_cast<size_t>(c) * 2 + blockIdx.y) * d + col);
    sm[slice][threadIdx.x & 31] = s;
    __syncthreads();
    if (slice == 0) {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) a += sm[i][threadIdx.x];
        (blockIdx.y == 0 ? gwq : gwk)[col] = a;
    }
}

template <int D, bool INTERLEAVED>
cudaError_t launch_rope_bwd_t(const RopeBwdParams& p, int sms, cudaStream_t st)
{
    const long long tokens = static_cast<long long>(p.B) * p.N;
    const int heads = p.Hq + p.Hkv + (p.dv != nullptr ? p.Hkv : 0);
    long long grid = (tokens + kRopeWarps - 1) / kRopeWarps;
    const long long most = 4LL * sms < kRopeBwdCtas ? 4LL * sms : kRopeBwdCtas;
    if (grid > most) grid = most;
    const unsigned g = static_cast<unsigned>(grid);
    cudaError_t e = p.g_dtype == FA_F32
                        ? launch_pdl(fa_qk_rope_bwd_kernel<D, INTERLEAVED, true>, g, kRopeWarps * 32, 0, st, p, heads)
                        : launch_pdl(fa_qk_rope_bwd_kernel<D, INTERLEAVED, false>, g, kRopeWarps * 32, 0, st, p, heads);
    if (e != cudaSuccess) return e;
    return launch_pdl(fa_rope_weight_kernel, dim3(D / 32, 2), 1024, 0, st, static_cast<const float*>(p.part),
                      static_cast<int>(grid), D, p.gwq, p.gwk);
}

}  // namespace

cudaError_t launch_qk_rope(const RopeParams& p, int d, bool interleaved, bool append, int sms, cudaStream_t st)
{
    switch (d) {
    case 32: return interleaved ? launch_rope_t<32, true>(p, append, sms, st) : launch_rope_t<32, false>(p, append, sms, st);
    case 64: return interleaved ? launch_rope_t<64, true>(p, append, sms, st) : launch_rope_t<64, false>(p, append, sms, st);
    case 128: return interleaved ? launch_rope_t<128, true>(p, append, sms, st) : launch_rope_t<128, false>(p, append, sms, st);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_qk_rope_bwd(const RopeBwdParams& p, int d, bool interleaved, int sms, cudaStream_t st)
{
    switch (d) {
    case 32: return interleaved ? launch_rope_bwd_t<32, true>(p, sms, st) : launch_rope_bwd_t<32, false>(p, sms, st);
    case 64: return interleaved ? launch_rope_bwd_t<64, true>(p, sms, st) : launch_rope_bwd_t<64, false>(p, sms, st);
    case 128: return interleaved ? launch_rope_bwd_t<128, true>(p, sms, st) : launch_rope_bwd_t<128, false>(p, sms, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace fa

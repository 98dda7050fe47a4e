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
// What bounds it: bytes.  D / 8 lanes share a row, each with four of its pairs, so the rotation stays
// within a lane and a row's sums are a few shuffles; the arithmetic is done two elements at a time.
// A warp takes one token and walks its heads, the token's cosines and sines, times the weights, in
// registers, with the loads of U steps in flight; neighbouring warps take neighbouring tokens, whose
// rows are neighbours in the head-major output.
#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "fa_internal.h"
#include "fa_kernel_common.cuh"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kRopeWarps = 8;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A lane's four pairs of a row, a in x[0], x[1] and b in x[2], x[3].
struct Pairs {
    float2 x[4];
};

// Which elements of a row a lane holds.  Interleaved: elements 8 sub .. 8 sub + 7, the pairs side by
// side.  Halves: elements at .. at + 3 (a) and bt .. bt + 3 (b): the lane's share of the two halves, or
// past rot two neighbouring pieces that stay as they are.
template <bool INTERLEAVED>
struct Share {
    int at, bt;
    int pair;    // first pair, an index into the tables; -1 past rot
    __device__ __forceinline__ Share(int sub, int rot)
    {
        if (INTERLEAVED) {
            at = 8 * sub;
            bt = at + 4;
            pair = at < rot ? 4 * sub : -1;
        } else if (8 * sub < rot) {
            at = 4 * sub;
            bt = at + (rot >> 1);
            pair = at;
        } else {
            at = 8 * sub;
            bt = at + 4;
            pair = -1;
        }
    }
    // Eight elements of a row of bf16, raw: two words from at, two from bt.
    __device__ __forceinline__ uint4 load(const __nv_bfloat16* row) const
    {
        if (INTERLEAVED) return ld_stream_v4(row + at);
        const uint2 a = ld_stream_v2(row + at), b = ld_stream_v2(row + bt);
        return make_uint4(a.x, a.y, b.x, b.y);
    }
    // The same from shared memory.
    __device__ __forceinline__ uint4 read(const __nv_bfloat16* row) const
    {
        if (INTERLEAVED) return *reinterpret_cast<const uint4*>(row + at);
        const uint2 a = *reinterpret_cast<const uint2*>(row + at), b = *reinterpret_cast<const uint2*>(row + bt);
        return make_uint4(a.x, a.y, b.x, b.y);
    }
    __device__ __forceinline__ void store(__nv_bfloat16* row, uint4 u) const
    {
        if (INTERLEAVED) {
            *reinterpret_cast<uint4*>(row + at) = u;
        } else {
            *reinterpret_cast<uint2*>(row + at) = make_uint2(u.x, u.y);
            *reinterpret_cast<uint2*>(row + bt) = make_uint2(u.z, u.w);
        }
    }
    __device__ __forceinline__ Pairs unpack(uint4 u) const
    {
        Pairs p;
        if (INTERLEAVED) {
            p.x[0] = make_float2(bf16_lo(u.x), bf16_lo(u.y)), p.x[1] = make_float2(bf16_lo(u.z), bf16_lo(u.w));
            p.x[2] = make_float2(bf16_hi(u.x), bf16_hi(u.y)), p.x[3] = make_float2(bf16_hi(u.z), bf16_hi(u.w));
        } else {
            p.x[0] = make_float2(bf16_lo(u.x), bf16_hi(u.x)), p.x[1] = make_float2(bf16_lo(u.y), bf16_hi(u.y));
            p.x[2] = make_float2(bf16_lo(u.z), bf16_hi(u.z)), p.x[3] = make_float2(bf16_lo(u.w), bf16_hi(u.w));
        }
        return p;
    }
    __device__ __forceinline__ uint4 pack(const Pairs& p) const
    {
        if (INTERLEAVED)
            return make_uint4(pack_bf16x2(p.x[0].x, p.x[2].x), pack_bf16x2(p.x[0].y, p.x[2].y),
                              pack_bf16x2(p.x[1].x, p.x[3].x), pack_bf16x2(p.x[1].y, p.x[3].y));
        return make_uint4(pack_bf16x2(p.x[0].x, p.x[0].y), pack_bf16x2(p.x[1].x, p.x[1].y),
                          pack_bf16x2(p.x[2].x, p.x[2].y), pack_bf16x2(p.x[3].x, p.x[3].y));
    }
    // The same eight elements in fp32: four from at, four from bt.
    __device__ __forceinline__ Pairs unpack32(float4 a, float4 b) const
    {
        Pairs p;
        if (INTERLEAVED) {
            p.x[0] = make_float2(a.x, a.z), p.x[1] = make_float2(b.x, b.z);
            p.x[2] = make_float2(a.y, a.w), p.x[3] = make_float2(b.y, b.w);
        } else {
            p.x[0] = make_float2(a.x, a.y), p.x[1] = make_float2(a.z, a.w);
            p.x[2] = make_float2(b.x, b.y), p.x[3] = make_float2(b.z, b.w);
        }
        return p;
    }
    __device__ __forceinline__ void store32(float* row, const Pairs& p) const
    {
        if (INTERLEAVED) {
            *reinterpret_cast<float4*>(row + at) = make_float4(p.x[0].x, p.x[2].x, p.x[0].y, p.x[2].y);
            *reinterpret_cast<float4*>(row + bt) = make_float4(p.x[1].x, p.x[3].x, p.x[1].y, p.x[3].y);
        } else {
            *reinterpret_cast<float4*>(row + at) = make_float4(p.x[0].x, p.x[0].y, p.x[1].x, p.x[1].y);
            *reinterpret_cast<float4*>(row + bt) = make_float4(p.x[2].x, p.x[2].y, p.x[3].x, p.x[3].y);
        }
    }
    __device__ __forceinline__ Pairs weights(const void* w, fa_dtype t) const
    {
        if (t == FA_F32) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // a weight vector need only be aligned to its elements
                f[i] = __ldg(reinterpret_cast<const float*>(w) + at + i);
                f[4 + i] = __ldg(reinterpret_cast<const float*>(w) + bt + i);
            }
            return unpack32(make_float4(f[0], f[1], f[2], f[3]), make_float4(f[4], f[5], f[6], f[7]));
        }
        const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
        return unpack(make_uint4(__ldg(u + at / 2), __ldg(u + at / 2 + 1), __ldg(u + bt / 2), __ldg(u + bt / 2 + 1)));
    }
    // Cosines and sines of the lane's pairs from a token's cosines and, 64 values on, sines.
    __device__ __forceinline__ Pairs angles_at(const float* t) const
    {
        Pairs p;
        p.x[0] = p.x[1] = make_float2(1.f, 1.f);
        p.x[2] = p.x[3] = make_float2(0.f, 0.f);
        if (pair >= 0) {
            const float4 c = *reinterpret_cast<const float4*>(t + pair), s = *reinterpret_cast<const float4*>(t + 64 + pair);
            p.x[0] = make_float2(c.x, c.y), p.x[1] = make_float2(c.z, c.w);
            p.x[2] = make_float2(s.x, s.y), p.x[3] = make_float2(s.z, s.w);
        }
        return p;
    }
    // Cosines and sines of the lane's pairs at position pos: c[0], c[1] and s in c[2], c[3].
    __device__ __forceinline__ Pairs angles(const float* cos_t, const float* sin_t, int pos, int rot) const
    {
        Pairs p;
        p.x[0] = p.x[1] = make_float2(1.f, 1.f);
        p.x[2] = p.x[3] = make_float2(0.f, 0.f);
        if (pair >= 0) {
            const size_t i = static_cast<size_t>(pos) * (rot >> 1) + pair;
            const float4 c = __ldg(reinterpret_cast<const float4*>(cos_t + i));
            const float4 s = __ldg(reinterpret_cast<const float4*>(sin_t + i));
            p.x[0] = make_float2(c.x, c.y), p.x[1] = make_float2(c.z, c.w);
            p.x[2] = make_float2(s.x, s.y), p.x[3] = make_float2(s.z, s.w);
        }
        return p;
    }
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

// Norm weights and rotation of a lane in one: a' = (r a) aa + (r b) ab, b' = (r a) ba + (r b) bb.  (r first:
// where the sum of squares overflows r is 0, and the row times its weights may be past fp32.)
struct Turn {
    float2 aa[2], ab[2], ba[2], bb[2];
    __device__ __forceinline__ Turn(const Pairs& w, const Pairs& cs)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            aa[i] = mul2(w.x[i], cs.x[i]);
            ab[i] = neg2(mul2(w.x[2 + i], cs.x[2 + i]));
            ba[i] = mul2(w.x[i], cs.x[2 + i]);
            bb[i] = mul2(w.x[2 + i], cs.x[i]);
        }
    }
    __device__ __forceinline__ Pairs apply(const Pairs& p, float r) const
    {
        const float2 rr = make_float2(r, r);
        Pairs o;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 a = mul2(rr, p.x[i]), b = mul2(rr, p.x[2 + i]);
            o.x[i] = fma2(a, aa[i], mul2(b, ab[i]));
            o.x[2 + i] = fma2(a, ba[i], mul2(b, bb[i]));
        }
        return o;
    }
};

// Sum of products of a lane's elements.
__device__ __forceinline__ float dot(const Pairs& p, const Pairs& q)
{
    const float2 t = __fadd2_rn(fma2(p.x[0], q.x[0], mul2(p.x[1], q.x[1])), fma2(p.x[2], q.x[2], mul2(p.x[3], q.x[3])));
    return t.x + t.y;
}

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

// The steps of a token: RPW query heads each, then key heads, then value heads.
template <int RPW>
struct Steps {
    int nq, nk, n;
    __host__ __device__ Steps(int Hq, int Hkv, bool values)
    {
        nq = (Hq + RPW - 1) / RPW;
        nk = (Hkv + RPW - 1) / RPW;
        n = nq + nk + (values ? nk : 0);
    }
};

// Grid (tokens / kRopeWarps, step chunks).  A warp: one token, steps blockIdx.y * chunk .. + chunk.
// Four rows in flight and four CTAs an SM (64 registers): B=64 N=1024 H=16 d=64 120 us, 6.7 TB/s of
// reads and writes; three CTAs 136, two with eight rows 168, five (48 registers, which spill) 145 (at 123 for
// four).  Rows through a ring of asynchronous copies, as in the backward kernel: 128 us there, 6-10 % slower at
// d = 128.
// APPEND: token t of sequence b is node t of its tree, at position seqlens[b] + depth, and its key
// and value go to cache row seqlens[b] + t.  Nodes past n_nodes[b] have zero query rows and no cache
// row.
template <int D, bool INTERLEAVED, bool APPEND>
__global__ void __launch_bounds__(kRopeWarps * 32, 4) fa_qk_rope_kernel(const RopeParams p, int chunk)
{
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int LPR = D / 8;    // lanes of a row
    constexpr int RPW = 32 / LPR; // rows of a warp's step
    constexpr int U = 4;          // steps in flight
    // The first values are copied while the position and the angles are on their way: a token may have few steps
    // to hide that under (share of the copy's rate with and without, d = 64: 16 heads 98 / 95 %, 12 heads 93 / 86,
    // 8 heads 84 / 76; d = 32: 16 heads 84 / 77, 12 heads 70 / 64; d = 128: 32/8 heads 95 / 94).  Not for a cache,
    // whose rows are known with the length only.
    constexpr bool EARLY = !APPEND;
    using bf16 = __nv_bfloat16;
    const int lane = threadIdx.x & 31;
    const int sub = lane % LPR;
    const int grp = lane / LPR;
    // (tokens are below 2^31: a 64-bit division here was a tenth of a small token's instructions)
    const unsigned token = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    if (token >= static_cast<unsigned>(p.B) * static_cast<unsigned>(p.N)) return;
    const unsigned b = token / static_cast<unsigned>(p.N);
    const int t = static_cast<int>(token - b * static_cast<unsigned>(p.N));
    const Share<INTERLEAVED> share(sub, p.rot);
    const Steps<RPW> steps(p.Hq, p.Hkv, p.v != nullptr);
    const int begin = static_cast<int>(blockIdx.y) * chunk;
    const int end = min(steps.n, begin + chunk);

    // U steps' rows at once, from step i of a kind's heads; zeros where there is no head.
    auto load = [&](uint4 (&raw)[U], const bf16* rows, int i, int to, int heads) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (i + u) * RPW + grp;
            raw[u] = i + u < to && h < heads ? share.load(rows + h * D) : make_uint4(0, 0, 0, 0);
        }
    };
    // Values pass through: 16 bytes a lane.
    const int vb = max(begin, steps.nq + steps.nk) - steps.nq - steps.nk, ve = end - steps.nq - steps.nk;
    auto load_v = [&](uint4 (&x)[U], int i) {
        const bf16* v = reinterpret_cast<const bf16*>(p.v) + static_cast<long long>(token) * p.v_stride + sub * 8;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (i + u) * RPW + grp;
            x[u] = i + u < ve && h < p.Hkv ? ld_stream_v4(v + h * D) : make_uint4(0, 0, 0, 0);
        }
    };
    // The first rows are on their way while the position is found.  Nodes that are not there are not read:
    // where there may be some, whether this one is comes first.
    const bf16* q = reinterpret_cast<const bf16*>(p.q) + static_cast<long long>(token) * p.q_stride;
    uint4 raw[U], first_v[U];
    auto first_rows = [&] {
        if (EARLY && vb < ve) load_v(first_v, vb);
        if (begin < steps.nq) load(raw, q, begin, min(end, steps.nq), p.Hq);
    };
    const bool ragged = APPEND && p.n_nodes != nullptr;
    if (!ragged) first_rows();
    int row = t;  // row of the key and value in their head
    if constexpr (APPEND) {
        const int len = p.seqlens[b];
        const int nodes = p.n_nodes != nullptr ? p.n_nodes[b] : p.N;
        const bool bad = len < 0 || len > p.Nk_max || nodes < 0 || nodes > p.N || len > p.Nk_max - nodes;
        const int from = min(max(len, 0), p.Nk_max);
        const int n = min(min(max(nodes, 0), p.N), p.Nk_max - from);
        if (bad && lane == 0) atomicCAS(p.status, 0, FA_ERR_INVALID_ARG);
        if (t >= n) {  // the whole warp: zero query rows, nothing else
            bf16* out = reinterpret_cast<bf16*>(p.q_out) + (static_cast<size_t>(b) * p.Hq * p.N + t) * D;
            for (int i = begin; i < min(end, steps.nq); ++i)
                if (i * RPW + grp < p.Hq)
                    *reinterpret_cast<uint4*>(out + static_cast<size_t>(i * RPW + grp) * p.N * D + sub * 8) = make_uint4(0, 0, 0, 0);
            return;
        }
        row = from + t;
    }
    if (ragged) first_rows();
    int pos;
    if constexpr (APPEND)
        pos = p.parents != nullptr ? row - t + tree_depth(p.parents + static_cast<size_t>(b) * p.N, t, lane, p.status) : row;
    else
        pos = p.positions != nullptr ? p.positions[token] : t;
    pos = checked_position(pos, p.max_pos, p.status);
    const size_t kv_rows = APPEND ? p.Nk_max : p.N;
    const size_t head = static_cast<size_t>(p.copies) * kv_rows * D;
    // Elements into the keys or values of the warp's token, first head.  The first values ask for it early; kept
    // across the query heads it would take registers that are short there, so the later kinds of heads work it out
    // anew (the empty statement hides that it is the same).  In the APPEND form the key heads' angles are read
    // again for the same reason.  With both kept the forms spilled: B=64 N=1024 H=16 d=64 123.5 us against 120,
    // 12 heads 98 against 95; 64 full trees of 64 nodes into a cache 18.9 against 17.9, d=32 5.9 against 5.8.
    auto kv_at = [&]() -> size_t {
        unsigned i = b;
        if (EARLY) asm volatile("" : "+r"(i));
        return static_cast<size_t>(i) * p.Hkv * head + static_cast<size_t>(row) * D;
    };
    auto store_v = [&](const uint4 (&x)[U], int i, size_t at) {
        bf16* out = reinterpret_cast<bf16*>(p.v_out) + at + sub * 8;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u >= ve) break;  // uniform
            const int h = (i + u) * RPW + grp;
            if (h < p.Hkv) {
                bf16* to = out + h * head;
                for (int c = 0; c < p.copies; ++c, to += kv_rows * D) *reinterpret_cast<uint4*>(to) = x[u];
            }
        }
    };
    const Pairs cs = share.angles(p.cos_t, p.sin_t, pos, p.rot);
    if (EARLY && vb < ve) store_v(first_v, vb, kv_at());
    auto turned = [&](const Turn& turn, uint4 u) -> uint4 {
        const Pairs x = share.unpack(u);
        return share.pack(turn.apply(x, rsqrtf(row_sum<LPR>(dot(x, x)) * (1.f / D) + p.eps)));
    };
    if (begin < steps.nq) {
        const Turn turn(share.weights(p.wq, p.w_dtype), cs);
        bf16* out = reinterpret_cast<bf16*>(p.q_out) + (static_cast<size_t>(b) * p.Hq * p.N + t) * D;
        const size_t q_head = static_cast<size_t>(p.N) * D;
        const int to = min(end, steps.nq);
        for (int i = begin; i < to; i += U) {
            if (i != begin) load(raw, q, i, to, p.Hq);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i + u >= to) break;  // uniform
                const uint4 y = turned(turn, raw[u]);
                const int h = (i + u) * RPW + grp;
                if (h < p.Hq) share.store(out + h * q_head, y);
            }
        }
    }
    auto store = [&](bf16* out, int i, uint4 y) {
        const int h = i * RPW + grp;
        if (h < p.Hkv) {
            bf16* to = out + h * head;
            share.store(to, y);
            for (int c = 1; c < p.copies; ++c) share.store(to + static_cast<size_t>(c) * kv_rows * D, y);
        }
    };
    const int kb = max(begin, steps.nq) - steps.nq, ke = min(end, steps.nq + steps.nk) - steps.nq;
    if (kb < ke) {
        int again = pos;  // (see kv_at)
        if (APPEND) asm volatile("" : "+r"(again));
        const Turn turn(share.weights(p.wk, p.w_dtype), APPEND ? share.angles(p.cos_t, p.sin_t, again, p.rot) : cs);
        const bf16* k = reinterpret_cast<const bf16*>(p.k) + static_cast<long long>(token) * p.k_stride;
        bf16* out = reinterpret_cast<bf16*>(p.k_out) + kv_at();
        for (int i = kb; i < ke; i += U) {
            load(raw, k, i, ke, p.Hkv);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i + u >= ke) break;
                store(out, i + u, turned(turn, raw[u]));
            }
        }
    }
    for (int i = EARLY ? vb + U : vb; i < ve; i += U) {
        load_v(raw, i);
        store_v(raw, i, kv_at());
    }
}

template <int D, bool INTERLEAVED>
cudaError_t launch_rope_t(const RopeParams& p, bool append, int sms, cudaStream_t st)
{
    constexpr int RPW = 32 / (D / 8);
    const long long tokens = static_cast<long long>(p.B) * p.N;
    const long long blocks = (tokens + kRopeWarps - 1) / kRopeWarps;
    // With few tokens the steps of one are shared out among warps, as far as two rounds of CTAs go
    const int steps = Steps<RPW>(p.Hq, p.Hkv, p.v != nullptr).n;
    long long chunks = 8LL * sms / blocks;
    if (chunks > steps) chunks = steps;
    if (chunks < 1) chunks = 1;
    const int chunk = static_cast<int>((steps + chunks - 1) / chunks);
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((steps + chunk - 1) / chunk));
    return append ? launch_pdl(fa_qk_rope_kernel<D, INTERLEAVED, true>, grid, kRopeWarps * 32, 0, st, p, chunk)
                  : launch_pdl(fa_qk_rope_kernel<D, INTERLEAVED, false>, grid, kRopeWarps * 32, 0, st, p, chunk);
}

// ---- backward ----------------------------------------------------------------------------------

// Two CTAs for each SM; a warp walks its tokens, of each the query, key and value heads, in batches of U
// row sets (RPW heads' rows, or RPW heads' copies of one number).  Batches go through a ring of kStages
// in shared memory, filled by asynchronous copies kStages - 1 batches ahead (a token's angles too), so that
// the bytes in flight do not depend on registers.  Measured with bf16 gradients on B=64 N=1024 H=16 d=64:
// 165 us a call, 6.5 TB/s; with the rows loaded into registers it was bound by latency whatever the split
// (four rows in flight, 16 warps an SM 214 us; two rows, 24 warps 227).  fp32 gradients of 4 copies,
// B=2 N=4097 32/8 heads d=128: 112 us, 6.2 TB/s.  The weights' gradients stay in registers (a lane's
// eight columns of each) until the CTA adds its warps' up in a fixed order and writes one partial row of
// each, which fa_rope_weight_kernel adds up, also in a fixed order: the result does not change from run
// to run.
// Batches: 64 to 96 KB in flight an SM do best; three stages of four sets (128 KB) took 193 us on the first
// case, two of two 172.  In share of the copy's rate, two stages of four sets / three of two, bf16
// gradients: d = 64 16 heads 94 / 93 %, 12 heads 91 / 82, 25 heads 89 / 80, 8 heads 77 / 88; d = 128 32
// heads 87 / 94, 32/8 90 / 90; d = 32 16 heads 78 / 90, 12 heads 61 / 67.  (Three CTAs an SM spill: 250 us.)
template <int D, bool GF32, bool MULTI>
struct RopeBwdCfg {
    static constexpr bool kThin = !GF32 && !MULTI && D != 64;
    static constexpr int kStages = kThin ? 3 : 2;
    static constexpr int U = kThin ? 2 : 4;
    static constexpr int kSet = GF32 ? 1536 : 1024;        // a row set: x (512 bytes), then the gradient's
    static constexpr int kAngles = U * kSet * kStages;     // cosines (256 bytes) and sines of a token, a ring too
    static constexpr int kWarp = kAngles + 512 * kStages;  // bytes of a warp
    static constexpr int kSmem = kRopeWarps * kWarp;
};

// MULTI: key and value heads have several copies; a row set is then one copy's.
template <int D, bool INTERLEAVED, bool GF32, bool MULTI>
__global__ void __launch_bounds__(kRopeWarps * 32, 2) fa_qk_rope_bwd_kernel(const RopeBwdParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    using C = RopeBwdCfg<D, GF32, MULTI>;
    using G = typename std::conditional<GF32, float, __nv_bfloat16>::type;
    using bf16 = __nv_bfloat16;
    constexpr int LPR = D / 8;
    constexpr int RPW = 32 / LPR;
    constexpr int U = C::U;
    extern __shared__ __align__(16) uint8_t rb_smem[];
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int sub = lane % LPR;
    const int grp = lane / LPR;
    uint8_t* mine = rb_smem + warp * C::kWarp;
    const uint32_t ring = smem_u32(mine);
    const Share<INTERLEAVED> share(sub, p.rot);
    const bool of32 = p.out_dtype == FA_F32;
    const size_t head = static_cast<size_t>(p.N) * D;  // elements of a head of the gradients
    const int nq = (p.Hq + RPW - 1) / RPW, nk = (p.Hkv + RPW - 1) / RPW;
    const int kinds = p.dv != nullptr ? 3 : 2;
    const Pairs wq = share.weights(p.wq, p.w_dtype), wk = share.weights(p.wk, p.w_dtype);
    Pairs aq, ak;
#pragma unroll
    for (int i = 0; i < 4; ++i) aq.x[i] = ak.x[i] = make_float2(0.f, 0.f);

    // Tokens are below 2^31, and unsigned holds a stride or two more.
    const unsigned tokens = static_cast<unsigned>(p.B) * static_cast<unsigned>(p.N);
    const unsigned stride = gridDim.x * kRopeWarps;
    // A place in the walk: token, kind of heads (0 query, 1 key, 2 value), step of RPW heads, copy.
    struct Place {
        unsigned token;
        int kind, step, copy;
    };
    const int copies = MULTI ? p.copies : 1;
    // `sets` row sets on, within the kind; true at its end (and then at the next kind's, or token's, start).
    auto advance = [&](Place& x, int sets) {
        if (MULTI && x.kind > 0) {
            if (++x.copy < copies) return false;
            x.copy = 0;
        }
        x.step += sets;
        if (x.step < (x.kind == 0 ? nq : nk)) return false;
        x.step = 0;
        if (++x.kind == kinds) {
            x.kind = 0;
            x.token += stride;
        }
        return true;
    };
    Place ahead{blockIdx.x * kRopeWarps + warp, 0, 0, 0}, at = ahead;
    auto position = [&](unsigned i) -> int {
        return p.positions != nullptr ? __ldg(p.positions + i) : static_cast<int>(i % static_cast<unsigned>(p.N));
    };
    int pos = ahead.token < tokens ? position(ahead.token) : 0;  // of the next token to be copied
    int token_slot = 0;                                          // of its angles
    const int half = p.rot >> 1;

    const G* copy_row = nullptr;  // MULTI: of the row set being copied
    size_t token_b = 0, token_t = 0;  // sequence of the token being copied, and its elements into a head
    // The copies of one batch into a stage: at most U row sets of one kind.
    auto copy_batch = [&](int stage) {
        if (ahead.token < tokens) {
            const int kind = ahead.kind;
            if (kind == 0 && ahead.step == 0) {  // a new token: its angles
                token_b = ahead.token / static_cast<unsigned>(p.N);
                token_t = (ahead.token - token_b * static_cast<unsigned>(p.N)) * D;
                const size_t i = static_cast<size_t>(checked_position(pos, p.max_pos, p.status)) * half;
                const int piece = lane & 15;
                if (4 * piece < half)
                    cp_async16(ring + C::kAngles + token_slot * 512 + (lane >> 4) * 256 + piece * 16,
                               (lane < 16 ? p.cos_t : p.sin_t) + i + 4 * piece, 16);
                token_slot = token_slot == C::kStages - 1 ? 0 : token_slot + 1;
                if (ahead.token + stride < tokens) pos = position(ahead.token + stride);
            }
            const int heads = kind == 0 ? p.Hq : p.Hkv;
            const size_t each = MULTI && kind > 0 ? copies * head : head;  // elements of a head's copies
            const bf16* x = (kind == 0 ? reinterpret_cast<const bf16*>(p.q) + static_cast<long long>(ahead.token) * p.q_stride
                                       : reinterpret_cast<const bf16*>(p.k) + static_cast<long long>(ahead.token) * p.k_stride) +
                            lane * 8;  // a step's rows are 256 elements, whatever the head size
            const G* g = reinterpret_cast<const G*>(kind == 0 ? p.dq : kind == 1 ? p.dk : p.dv) + token_b * (heads * each) + token_t;
            const uint32_t to = ring + stage * (U * C::kSet);
            // one row set; zeros where there is no head
            auto copy_set = [&](int u, const bf16* xs, const G* row, int h) {
                const int bytes = h < heads ? 16 : 0;
                if (kind < 2 && (!MULTI || ahead.copy == 0)) cp_async16(to + u * C::kSet + lane * 16, h < heads ? xs : x, bytes);
                if constexpr (GF32) {
                    cp_async16(to + u * C::kSet + 512 + grp * (D * 4) + sub * 16, row + sub * 4, bytes);
                    cp_async16(to + u * C::kSet + 512 + grp * (D * 4) + (LPR + sub) * 16, row + (LPR + sub) * 4, bytes);
                } else {
                    cp_async16(to + u * C::kSet + 512 + lane * 16, row + sub * 8, bytes);
                }
            };
            if (MULTI && kind > 0) {  // (step, copy) in order; a head's copies lie behind one another
                if (ahead.step == 0 && ahead.copy == 0) copy_row = g + (grp < heads ? grp * each : 0);
                bool end = false;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (end) continue;  // uniform
                    const int h = ahead.step * RPW + grp;
                    copy_set(u, x + ahead.step * 256, h < heads ? copy_row : g, h);
                    copy_row += head;
                    if (ahead.copy == copies - 1) copy_row += (RPW - 1) * each;
                    end = advance(ahead, 1);
                }
            } else {
                const int n = (kind == 0 ? nq : nk) - ahead.step;
                const G* row = g + static_cast<size_t>(ahead.step * RPW + grp) * each;
                const bf16* xs = x + ahead.step * 256;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (u < n) {
                        const int h = (ahead.step + u) * RPW + grp;
                        copy_set(u, xs + u * 256, h < heads ? row : g, h);
                        row += RPW * each;
                    }
                }
                advance(ahead, U);
            }
        }
        cp_async_commit();
    };
    for (int i = 0; i < C::kStages - 1; ++i) copy_batch(i);

    Pairs cs, g;
    uint4 xr = make_uint4(0, 0, 0, 0);
    int cs_slot = 0;
    // one row: its gradient g to the projection's.  A lane without a row (not `live`) has zeros, whose
    // norm is infinite at eps = 0: it takes r = 0, so that it adds 0 to acc.
    auto finish = [&](const Pairs& w, Pairs& acc, bool live) {
        const Pairs x = share.unpack(xr);
        Pairs hb, z;  // the gradient turned back, and times the weights
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            hb.x[e] = fma2(g.x[e], cs.x[e], mul2(g.x[2 + e], cs.x[2 + e]));
            hb.x[2 + e] = fma2(g.x[2 + e], cs.x[e], neg2(mul2(g.x[e], cs.x[2 + e])));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) z.x[e] = mul2(w.x[e], hb.x[e]);
        const float ss = row_sum<LPR>(dot(x, x));
        const float sz = row_sum<LPR>(dot(x, z));
        const float r = live ? rsqrtf(ss * (1.f / D) + p.eps) : 0.f;
        const float f = r == 0.f ? 0.f : -(r * r) * sz * (1.f / D);  // (then sz may have overflowed too)
        const float2 rr = make_float2(r, r), ff = make_float2(f, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            acc.x[e] = fma2(hb.x[e], mul2(x.x[e], rr), acc.x[e]);
            g.x[e] = mul2(rr, fma2(x.x[e], ff, z.x[e]));
        }
    };
    int stage = 0;
    while (at.token < tokens) {
        copy_batch(stage == 0 ? C::kStages - 1 : stage - 1);
        cp_async_wait<C::kStages - 1>();
        __syncwarp();
        const int kind = at.kind;
        if (kind == 0 && at.step == 0) {
            cs = share.angles_at(reinterpret_cast<const float*>(mine + C::kAngles + cs_slot * 512));
            cs_slot = cs_slot == C::kStages - 1 ? 0 : cs_slot + 1;
        }
        const uint8_t* from = mine + stage * (U * C::kSet) + grp * (D * 2);
        char* out = static_cast<char*>(kind == 0 ? p.gq : kind == 1 ? p.gk : p.gv);
        const long long row = static_cast<long long>(at.token) * (kind == 0 ? p.gq_stride : kind == 1 ? p.gk_stride : p.gv_stride);
        const int heads = kind == 0 ? p.Hq : p.Hkv;
        auto gradient = [&](int u) -> Pairs {
            if constexpr (GF32) {
                const float* sg = reinterpret_cast<const float*>(from + u * C::kSet + 512 + grp * (D * 2));
                return share.unpack32(*reinterpret_cast<const float4*>(sg + share.at), *reinterpret_cast<const float4*>(sg + share.bt));
            } else {
                return share.unpack(share.read(reinterpret_cast<const bf16*>(from + u * C::kSet + 512)));
            }
        };
        auto write = [&](int step) {
            const int h = step * RPW + grp;
            if (h < heads) {
                if (of32) share.store32(reinterpret_cast<float*>(out) + row + h * D, g);
                else share.store(reinterpret_cast<bf16*>(out) + row + h * D, share.pack(g));
            }
        };
        if (MULTI && kind > 0) {
            bool end = false;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (end) continue;  // uniform
                const Pairs y = gradient(u);
                if (at.copy == 0) {
                    g = y;
                    if (kind == 1) xr = share.read(reinterpret_cast<const bf16*>(from + u * C::kSet));
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) g.x[e] = __fadd2_rn(g.x[e], y.x[e]);
                }
                if (at.copy == copies - 1) {
                    if (kind == 1) finish(wk, ak, at.step * RPW + grp < heads);
                    write(at.step);
                }
                end = advance(at, 1);
            }
        } else {
            const int n = (kind == 0 ? nq : nk) - at.step;
            auto sets = [&](auto turn) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (u < n) {
                        g = gradient(u);
                        turn(u);
                        write(at.step + u);
                    }
                }
            };
            auto read_x = [&](int u) { xr = share.read(reinterpret_cast<const bf16*>(from + u * C::kSet)); };
            auto live = [&](int u) { return (at.step + u) * RPW + grp < heads; };
            if (kind == 0) sets([&](int u) { read_x(u), finish(wq, aq, live(u)); });
            else if (kind == 1) sets([&](int u) { read_x(u), finish(wk, ak, live(u)); });  // (not MULTI)
            else sets([](int) {});
            advance(at, U);
        }
        __syncwarp();  // the stage may be filled again
        stage = stage == C::kStages - 1 ? 0 : stage + 1;
    }
    __syncthreads();  // (no copy is in flight: the batches ahead of the last were empty)
    float(*sm)[2][D] = reinterpret_cast<float(*)[2][D]>(rb_smem);
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            aq.x[i].x += __shfl_xor_sync(0xffffffffu, aq.x[i].x, o);
            aq.x[i].y += __shfl_xor_sync(0xffffffffu, aq.x[i].y, o);
            ak.x[i].x += __shfl_xor_sync(0xffffffffu, ak.x[i].x, o);
            ak.x[i].y += __shfl_xor_sync(0xffffffffu, ak.x[i].y, o);
        }
    if (grp == 0) {
        share.store32(sm[warp][0], aq);
        share.store32(sm[warp][1], ak);
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
    for (int c = slice; c < n; c += 32) s += __ldcg(part + (static_cast<size_t>(c) * 2 + blockIdx.y) * d + col);
    sm[slice][threadIdx.x & 31] = s;
    __syncthreads();
    if (slice == 0) {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) a += sm[i][threadIdx.x];
        (blockIdx.y == 0 ? gwq : gwk)[col] = a;
    }
}

template <int D, bool INTERLEAVED, bool GF32, bool MULTI>
cudaError_t launch_rope_bwd_g(const RopeBwdParams& p, int grid, cudaStream_t st)
{
    auto kern = fa_qk_rope_bwd_kernel<D, INTERLEAVED, GF32, MULTI>;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, RopeBwdCfg<D, GF32, MULTI>::kSmem);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    return launch_pdl(kern, static_cast<unsigned>(grid), kRopeWarps * 32, RopeBwdCfg<D, GF32, MULTI>::kSmem, st, p);
}

template <int D, bool INTERLEAVED>
cudaError_t launch_rope_bwd_t(const RopeBwdParams& p, int sms, cudaStream_t st)
{
    const long long tokens = static_cast<long long>(p.B) * p.N;
    long long n = (tokens + kRopeWarps - 1) / kRopeWarps;
    if (n > 2LL * sms) n = 2LL * sms;
    if (n > kRopeBwdCtas) n = kRopeBwdCtas;
    const int grid = static_cast<int>(n);
    const bool f32 = p.g_dtype == FA_F32;
    const cudaError_t e = p.copies > 1 ? (f32 ? launch_rope_bwd_g<D, INTERLEAVED, true, true>(p, grid, st)
                                              : launch_rope_bwd_g<D, INTERLEAVED, false, true>(p, grid, st))
                                       : (f32 ? launch_rope_bwd_g<D, INTERLEAVED, true, false>(p, grid, st)
                                              : launch_rope_bwd_g<D, INTERLEAVED, false, false>(p, grid, st));
    if (e != cudaSuccess) return e;
    return launch_pdl(fa_rope_weight_kernel, dim3(D / 32, 2), 1024, 0, st, static_cast<const float*>(p.part), grid, D, p.gwq, p.gwk);
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

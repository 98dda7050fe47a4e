// fa_cache.cu -- compaction of a cache onto the accepted path of a tree of drafted tokens.
//
// The drafted nodes of sequence b lie in cache rows p .. p + T - 1 (p = seqlens[b]); verification
// keeps a path accepted[b][0 .. n - 1] of them.  Row p + accepted[b][i] moves to row p + i for every
// layer, key/value head, and for keys and values, and the sequence then has p + n cached tokens.
//
// One CTA per (layer, sequence, head, keys or values) reads all its rows into registers before it
// writes any, so any order of the nodes, and a node named twice, gives the rows as they were before
// the call.  A few rows of 64 to 256 bytes each: the time is the launch and two dependent loads.
#include <cstdint>

#include "fa_internal.h"
#include "fa_kernel_common.cuh"

namespace fa {

namespace {

constexpr int kCompactThreads = 128;
constexpr int kCompactItems = 16;  // 16-byte pieces a thread may hold: 128 rows of 256 bytes

__global__ void __launch_bounds__(kCompactThreads) fa_cache_compact_kernel(const CompactParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int h = blockIdx.x % p.Hkv;
    const long long lb = blockIdx.x / p.Hkv;  // layer * B + sequence
    const int b = static_cast<int>(lb % p.B);
    const int len_in = p.seqlens[b];
    const int n_in = p.n_accepted[b];
    const int len = min(max(len_in, 0), p.Nk_max);
    const int n = min(min(max(n_in, 0), p.T), p.Nk_max - len);
    if (threadIdx.x == 0) {
        if (len != len_in || n != n_in) atomicCAS(p.status, 0, FA_ERR_INVALID_ARG);
        if (p.seqlens_out != nullptr && blockIdx.y == 0 && h == 0 && lb < p.B) p.seqlens_out[b] = len + n;
    }
    const int pieces = p.d / 8;  // of 16 bytes in a row
    const int total = n * pieces;
    uint4* base = reinterpret_cast<uint4*>(blockIdx.y == 0 ? p.k : p.v) +
                  (static_cast<size_t>(lb) * p.Hkv + h) * static_cast<size_t>(p.Nk_max) * pieces;
    uint4 x[kCompactItems];
    unsigned move = 0u;
#pragma unroll
    for (int i = 0; i < kCompactItems; ++i) {
        const int at = i * kCompactThreads + threadIdx.x;
        if (at < total) {
            const int r = at / pieces;
            const int node = p.accepted[static_cast<size_t>(b) * p.T + r];
            if (node < 0 || node >= p.T || node >= p.Nk_max - len) {
                atomicCAS(p.status, 0, FA_ERR_INVALID_ARG);  // the row stays as it was
            } else if (node != r) {
                x[i] = base[static_cast<size_t>(len + node) * pieces + (at - r * pieces)];
                move |= 1u << i;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kCompactItems; ++i) {
        const int at = i * kCompactThreads + threadIdx.x;
        if ((move >> i) & 1u) base[static_cast<size_t>(len) * pieces + at] = x[i];
    }
}

}  // namespace

cudaError_t launch_cache_compact(const CompactParams& p, cudaStream_t st)
{
    const dim3 grid(static_cast<unsigned>(static_cast<long long>(p.L) * p.B * p.Hkv), 2);
    return launch_pdl(fa_cache_compact_kernel, grid, kCompactThreads, 0, st, p);
}

}  // namespace fa

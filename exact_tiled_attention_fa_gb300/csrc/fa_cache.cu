// fa_cache.cu -- compaction of a cache onto the accepted path of a tree of drafted tokens.
//
// The drafted nodes of sequence b lie in cache rows p .. p + T - 1 (p = seqlens[b]); verification
// keeps a path accepted[b][0 .. n - 1] of them.  Row p + accepted[b][i] moves to row p + i for every
// layer, key/value head, and for keys and values, and the sequence then has p + n cached tokens.
//
// One CTA per (layer, sequence) reads all rows of a number of heads into registers before it writes
// any of them, so any order of the nodes, and a node named twice, gives the rows as they were before
// the call.  A few rows of 64 to 256 bytes a head: the time is the launch and three dependent loads
// (length, nodes, rows), which is why a CTA takes the keys and values of all heads at once where they
// fit (16 layers x 32 sequences x 8 heads, 4 rows each: 5.9 us, with one CTA per head, keys and values
// 12.7; one layer of 2 sequences 2.1).
#include <cstdint>

#include "fa_internal.h"
#include "fa_kernel_common.cuh"

namespace fa {

namespace {

constexpr int kCompactThreads = 256;
constexpr int kCompactItems = 8;  // 16-byte pieces a thread holds: a head's 128 rows of 256 bytes fit a CTA

__global__ void __launch_bounds__(kCompactThreads) fa_cache_compact_kernel(const CompactParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ int sm_node[FA_TREE_MAX_NODES];
    const int lb = blockIdx.x;  // layer * B + sequence
    const int b = lb % p.B;
    const int len_in = p.seqlens[b];
    const int n_in = p.n_accepted[b];
    // (read for all T, together with the length and the count)
    const int node = threadIdx.x < p.T ? p.accepted[static_cast<size_t>(b) * p.T + threadIdx.x] : 0;
    const int len = min(max(len_in, 0), p.Nk_max);
    const int n = min(min(max(n_in, 0), p.T), p.Nk_max - len);
    if (threadIdx.x < n) {
        const bool bad = node < 0 || node >= p.T || node >= p.Nk_max - len;
        if (bad) atomicCAS(p.status, 0, FA_ERR_INVALID_ARG);
        sm_node[threadIdx.x] = bad ? threadIdx.x : node;  // out of range: the row stays as it was
    }
    if (threadIdx.x == 0) {
        if (len != len_in || n != n_in) atomicCAS(p.status, 0, FA_ERR_INVALID_ARG);
        if (p.seqlens_out != nullptr && lb < p.B) p.seqlens_out[b] = len + n;
    }
    __syncthreads();
    if (n == 0) return;
    const int pieces = p.d / 8;   // of 16 bytes in a row
    const int each = n * pieces;  // of a head's keys or values
    const int together = kCompactThreads * kCompactItems / each;  // at least one
    const size_t head = static_cast<size_t>(p.Nk_max) * pieces;
    // head x: keys for x < Hkv, then values
    for (int x0 = 0; x0 < 2 * p.Hkv; x0 += together) {
        const int total = min(together, 2 * p.Hkv - x0) * each;
        uint4 v[kCompactItems];
        uint4* dst[kCompactItems];
#pragma unroll
        for (int i = 0; i < kCompactItems; ++i) {
            const int at = i * kCompactThreads + threadIdx.x;
            dst[i] = nullptr;
            if (at < total) {
                const int x = at / each;
                const int in = at - x * each;
                const int r = in / pieces;
                const int c = in - r * pieces;
                const int from = sm_node[r];
                if (from != r) {
                    const int h = x0 + x;
                    uint4* base = reinterpret_cast<uint4*>(h < p.Hkv ? p.k : p.v) +
                                  (static_cast<size_t>(lb) * p.Hkv + (h < p.Hkv ? h : h - p.Hkv)) * head +
                                  static_cast<size_t>(len) * pieces + c;
                    v[i] = base[static_cast<size_t>(from) * pieces];
                    dst[i] = base + static_cast<size_t>(r) * pieces;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kCompactItems; ++i)
            if (dst[i] != nullptr) *dst[i] = v[i];
    }
}

}  // namespace

cudaError_t launch_cache_compact(const CompactParams& p, cudaStream_t st)
{
    const dim3 grid(static_cast<unsigned>(static_cast<long long>(p.L) * p.B));
    return launch_pdl(fa_cache_compact_kernel, grid, kCompactThreads, 0, st, p);
}

}  // namespace fa

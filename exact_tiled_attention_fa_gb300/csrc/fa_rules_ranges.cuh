// fa_rules_ranges.cuh -- what documents let each query see, and which queries see each key.
//
// A document is a run of equal numbers >= 0 along the keys; a number below 0 is padding, in no document.  Query i
// sits at position Nk - N + i and sees the keys of its position's document, cut off behind its own position by a
// causal mask, but for a prefix.  Both a query's keys and a key's queries are then intervals whose ends never fall
// from one row to the next, so a tile of 128 rows has to do with one interval of tiles of the other side.
//
// One CTA for 128 positions.  Runs that begin and end in them are found by a scan; for the first and the last run the
// CTA looks back and ahead, 2048 numbers at a time, to the first other number.  It takes 2 - 3 us for documents
// of a few thousand tokens and about 1 us more for every 2048 tokens a document is longer.
#pragma once

#include "fa_rules_common.cuh"

namespace fa {

constexpr int kRangeThreads = 256;
constexpr int kRangeLook = 8 * kRangeThreads;

__device__ __forceinline__ int block_max(int x, int* slot)
{
    __syncthreads();
    if (threadIdx.x == 0) *slot = INT32_MIN;
    __syncthreads();
    x = __reduce_max_sync(0xffffffffu, x);
    if ((threadIdx.x & 31) == 0) atomicMax(slot, x);
    __syncthreads();
    return *slot;
}

// The CTA's part `block` of B * tiles.
template <bool KEYS>
__device__ __forceinline__ void rules_ranges(const RangesParams& p, int block)
{
    __shared__ int slot, begins[4], ends[4];
    const int b = block / p.tiles;
    const int t = block - b * p.tiles;
    const int off = p.Nk - p.N;
    const int n = KEYS ? p.Nk : p.N;                // rows
    const int p0 = 128 * t + (KEYS ? 0 : off);      // position of the tile's first row
    const int* docs = p.docs + static_cast<size_t>(b) * p.Nk;
    const int i = threadIdx.x;                      // threads 0 .. 127: a row each
    const int lane = i & 31, warp = i >> 5;
    const int row = 128 * t + i;
    const int pos = p0 + i;
    const bool here = i < 128 && row < n && pos >= 0;  // (pos < Nk follows)
    const int first = max(p0, 0);                      // the tile's first and last position
    const int last = min(p0 + 127, p.Nk - 1);          // (the last row's: rows end where positions do)
    const int id = here ? docs[pos] : -1;
    // where this row's run begins and ends, as far as the tile goes
    int begin = here && (pos == first || docs[pos - 1] != id) ? pos : -1;
    int end = here && (pos == last || docs[pos + 1] != id) ? pos + 1 : INT32_MAX;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, begin, o);
        const int y = __shfl_down_sync(0xffffffffu, end, o);
        if (lane >= o) begin = max(begin, x);
        if (lane + o < 32) end = min(end, y);
    }
    if (warp < 4) {
        if (lane == 31) begins[warp] = begin;
        if (lane == 0) ends[warp] = end;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < warp) begin = max(begin, begins[w]);
        if (w > warp) end = min(end, ends[w]);
    }
    // the first run's beginning and the last one's end may lie outside the tile
    int run0 = first, run1 = last + 1;
    if (first <= last) {  // (the same for the whole CTA; a tile of rows before position 0 has none)
        const int id0 = docs[first], id1 = docs[last];
        if (id0 >= 0) {
            for (int e = first; e > 0; e -= kRangeLook) {  // positions [e - kRangeLook, e)
                int other = -1;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int x = e - 1 - i - kRangeThreads * k;
                    if (x >= 0 && docs[x] != id0) other = max(other, x);
                }
                other = block_max(other, &slot);
                run0 = other >= 0 ? other + 1 : max(e - kRangeLook, 0);
                if (other >= 0) break;
            }
        }
        if (id1 >= 0) {
            for (int e = last + 1; e < p.Nk; e += kRangeLook) {  // positions [e, e + kRangeLook)
                int other = INT32_MIN;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int x = e + i + kRangeThreads * k;
                    if (x < p.Nk && docs[x] != id1) other = max(other, -x);
                }
                other = block_max(other, &slot);
                run1 = other != INT32_MIN ? -other : min(e + kRangeLook, p.Nk);
                if (other != INT32_MIN) break;
            }
        }
    }
    if (begin == first) begin = run0;
    if (end == last + 1) end = run1;
    const int prefix = p.causal ? rules_prefix(p.prefix, b, p.Nk, p.status) : 0;
    int lo = 0, hi = 0;
    if (here && id >= 0) {
        if (KEYS) {  // queries, by their index
            lo = max(p.causal && pos >= prefix ? pos : begin, begin) - off;
            hi = end - off;
            lo = max(lo, 0);
        } else {
            lo = begin;
            hi = p.causal ? min(end, max(pos + 1, prefix)) : end;
        }
        if (hi <= lo) lo = hi = 0;
    }
    if (i < 128 && row < n) p.each[static_cast<size_t>(b) * n + row] = make_int2(lo, hi);
    // the tile's: the smallest and the largest of its rows
    const int most = block_max(hi > lo ? hi : 0, &slot);
    const int least = -block_max(hi > lo ? -lo : INT32_MIN + 1, &slot);
    if (i == 0) p.tile[block] = most > 0 ? make_int2(least / 128, (most + 127) / 128) : make_int2(0, 0);
}

}  // namespace fa

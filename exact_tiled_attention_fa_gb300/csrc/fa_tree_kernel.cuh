// fa_tree_kernel.cuh -- decode attention for a tree of drafted tokens over a cache, for sm_103a.
//
// Mathematics.  Sequence b has p cached tokens (cache rows 0 .. p - 1) and n <= T drafted tokens
// whose keys and values were written to cache rows p .. p + n - 1.  parents[t] < t is the node that
// node t continues (-1: the last cached token).  With A(t) the set of t and its ancestors, query
// row (h, t) attends to
//   { rows j < p }  and  { rows p + a, a in A(t) },
// O = softmax(scale q K^T) V over those rows.  The Hq / Hkv query heads of a key/value head and
// their T nodes are the rows of one group ("flash_lab.py -- FlashAttention, flash-decoding and
// megakernel in numpy", section 4 `split_kv_decode`: a group's query heads are packed as the rows
// of q), the walk over 128-key tiles keeps the running max and sum of section 1 `softmax_online`,
// and key ranges are joined by section 4's log-sum-exp combine.
//
// Work division.  A unit is a group's block of up to 128 query rows (256 in PAIR form); it has
// ceil((p + n) / 128) key tiles, and counts for unit_cost more, about what its start and end cost.
// The tiles of all units, in order, are cut into equal shares, from lengths that only the device
// knows: each CTA scans the lengths once.  A share crosses unit borders, and the rings of K and V
// tiles run on across them, so a CTA pays its start-up once, however short the caches are.  A unit
// that lies in one share is finished there; the parts of the others go to at most two slots a share
// (its first and its last unit) and fa_tree_merge_kernel joins them.  The slots are thus bounded by the
// number of shares, not by the number of units.
//
// Roles of a CTA, one per SM (12 warps):
//   warps 0-3 / 4-7  softmax warpgroups 0 / 1: thread t owns row t of a 128-row tile (TMEM lane t).
//   warps 8, 11      TMA producers: query tiles, K and V tiles into rings of their own (11: SOLO only).
//   warps 9, 10      tcgen05 issuers of warpgroup 0 / 1: S = Q K^T, O += P V (P from tensor memory).
// A single query tile would leave the tensor core idle under its exponentials and the exponentials
// under its products, so the two warpgroups work on different keys (or different rows):
// ALT form (groups of at most 128 rows, few units): both hold the same 128 query rows and take the key
// tiles of the CTA's share in turn (tile k goes to warpgroup k mod 2), each with its own running max,
// sum and O accumulator.  At the end of a unit the two exchange max and sum through shared memory and
// each reads half of the columns of both accumulators out of tensor memory (warps w and w + 4 reach
// the same lanes).
// SOLO form (at most 128 rows, many units): each warpgroup has a share, a producer and rings of its own,
// so the start and end of one's units run under the other's tiles; but there are twice as many shares,
// and so parts to write and join.
// PAIR form (more than 128 rows): warpgroup i takes query rows 128 i .. 128 i + 127 of the unit and
// both walk every key tile of the CTA's share, so that K and V are read once for 256 rows.
// (fa_cached_api.cu chooses, with what the forms measured.)
//
// What bounds it, and what it takes with the merge (16 sequences of 1 - 32K tokens, 32/8 heads, d = 128):
// with 16 nodes K and V, 168-173 us, 6.5 TB/s; with 64 nodes the softmax's chain between two products (scores
// out of tensor memory, exponentials, weights back, two barriers), 258 us, 1100 TFLOP/s in a short series and
// 275 us, 1030 TFLOP/s in a long one at the power limit's clock, tensor cores 47 % busy.  One sequence of 2000
// tokens, 8 nodes: 12.1 us, latency: two launches, lengths, the first tiles, one tile's softmax, its rows out
// and in again.  Many short caches (256 sequences of 150 - 300 tokens, 4 nodes) 73 us, half the copy's rate: a
// unit's end, its rows out by the warps that are to take the next one's scores, comes once in two or three
// tiles, and at d = 128 a SOLO stream has one stage each of K and V, so a tile is asked for only when the
// product before it is done.
//
// Masks.  Only the tiles that hold drafted rows are masked, by four 32-bit words per query row (its
// ancestors), shifted to the tile; hidden scores become -inf by selection, so a non-finite key
// never reaches a row that does not see it.  V rows past the tree are zeroed in shared memory (0
// times NaN would be NaN).
//
// Tensor memory, P's aliasing of S at d = 128, the bounded waits and the drain after a failure are
// those of fa_fwd_kernel.cuh.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "fa_internal.h"
#include "fa_kernel_common.cuh"
#include "ptx.cuh"

namespace fa {

constexpr int kTrThreads = 384;  // 12 warps = 3 warpgroups
constexpr int kTrWarpProducer = 8;
constexpr int kTrWarpMma = 9;  // and 10
enum : int {
    kTbQFull = 0,     // + query buffer
    kTbQEmpty = 2,    // + query buffer: its issuers are done with it
    kTbSFull = 4,     // + 2 * warpgroup + step: scores of a step's keys
    kTbPFull = 8,     // + 2 * warpgroup + step: their weights
    kTbPVDone = 12,   // + 2 * warpgroup + step: the product with them has completed
    kTbOReady = 16,   // + warpgroup: the last product of a unit has completed
    kTbOFree = 18,    // + warpgroup, ALT: O_i has been read out of TMEM by both
    kTbMLFull = 20,   // ALT: both warpgroups' max and sum are in shared memory
    kTbDrain = 21,    // + warpgroup
    kTbSFree = 48,    // + warpgroup, d <= 64: S_i has been read out of TMEM
    kTbKFull = 24,    // + K stage (up to 4)
    kTbKEmpty = 28,
    kTbVFull = 32,    // + V stage (up to 4)
    kTbVEmpty = 36,
    kTbSegFull = 40,  // + place in the ring of records: the segment's is in shared memory
    kTbCount = 50
};

// A segment as the producer hands it to the other roles: a run of key tiles of one unit.
struct TreeSeg {
    int n;              // tiles; 0: the share is done
    int tile;           // the first one
    int prefix, nodes;  // of the sequence
    int b, group, qp;
    int slot;           // of its part; -1: the unit is whole
};
// Records in the ring, 8 for the one stream of tiles (ALT, PAIR) or 4 for each of two (SOLO).  The producer
// is at most two segments ahead of the scores (ALT; one otherwise: the query buffers), those at most two
// ahead of a softmax warpgroup (ALT; one otherwise), which copies a record when it comes to it: a record
// is never overwritten before it has been read.
constexpr int kTrSegs = 8;

enum TreeForm { kAlt, kSolo, kPair };

template <int D, TreeForm FORM>
struct TrCfg {
    static_assert(D == 32 || D == 64 || D == 128, "head size");
    // Steps of a tile.  At d = 128 tensor memory has no room for P beside S and O: P overwrites S, and a
    // tile's scores wait for the product of the tile before.  In PAIR form, where the tensor core is what
    // counts, a tile therefore goes in two steps of 64 keys whose columns are used in turn: one's product
    // and its next scores run under the other's exponentials (16 sequences of 1 - 32K tokens, 64 nodes,
    // 32/8 heads: 288 us in one step, 259 in two; 64 of 1000 tokens: 101 and 94).  The other forms wait for
    // memory, and a tile in two steps reads the queries from shared memory twice: one step (16 nodes 170 us,
    // in two steps 177; d = 64, 64 nodes 111 and 155).
    static constexpr int kSteps = D == 128 && FORM == kPair ? 2 : 1;
    static constexpr int kStep = kBlockN / kSteps;  // keys
    // Registers after the split: 256 * softmax + 128 * control = 64512 = 384 * 168, checked by the launcher.
    // A softmax thread holds the scores of a step.  (With 224 and 56 at d = 128 the producers and issuers
    // spilled more: 256 sequences of 300 tokens 77.7 us, with 216 and 72 they take 72.9.  Bytes stored and
    // loaded that still spill: d = 128 ALT 136/164, SOLO 56/72, PAIR 24/128; d <= 64 ALT 60/80, others none.)
    static constexpr int kSoftmaxRegs = kSteps == 2 ? 192 : D == 128 ? 216 : 208;
    static constexpr int kControlRegs = kSteps == 2 ? 120 : D == 128 ? 72 : 88;
    static constexpr int kCB = D < 64 ? D : 64;
    static constexpr int kNumCB = D / kCB;
    static constexpr int kRowBytes = kCB * 2;
    static constexpr uint32_t kLayout = kRowBytes == 128 ? kSwizzle128B : kSwizzle64B;
    static constexpr int kAtomBytes = 8 * kRowBytes;
    static constexpr int kBlkBytes = kBlockM * kRowBytes;
    static constexpr int kTileBytes = kNumCB * kBlkBytes;  // 128 x D bf16
    // Stages of K and of V, all streams' together.  Even: in ALT form a stage then always serves the same
    // warpgroup, so its tile before was consumed by the very thread that waits for the next one, which the
    // phase parity of the wait relies on.
    static constexpr int kStages = D == 128 ? 2 : 4;
    static_assert(kStages % 2 == 0 && kStages <= 4, "ring stages");
    static constexpr int kOffQ = 0;  // two query tiles: two units' (ALT), a warpgroup's each (SOLO, PAIR)
    static constexpr int kOffK = 2 * kTileBytes;
    static constexpr int kOffV = kOffK + kStages * kTileBytes;
    static constexpr int kOffML = kOffV + kStages * kTileBytes;  // ALT: [2 warpgroups][128] (max, sum)
    static constexpr int kOffStage = kOffML + 2 * kBlockM * 8;  // [8 warps][32 rows of 64 bytes]: rows on their way out
    static constexpr int kOffSeg = kOffStage + 8 * 2048;
    static constexpr int kOffBar = kOffSeg + kTrSegs * static_cast<int>(sizeof(TreeSeg));
    static constexpr int kOffStart = kOffBar + kTbCount * 8;
    static constexpr int kUsedBytes = kOffStart + 2 * 64 + 16;
    // At least 120 KB, so that no second CTA (which would wait for the 512 TMEM columns) shares the SM.
    static constexpr int kSmemBytes = kUsedBytes + 1024 > 120 * 1024 ? kUsedBytes + 1024 : 120 * 1024;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
    static constexpr int kTmemCols = 512;
    static constexpr bool kAliasP = D == 128;
    __host__ __device__ static constexpr uint32_t col_s(int i) { return 128u * i; }  // a step's columns: + kStep * step
    __host__ __device__ static constexpr uint32_t col_o(int i) { return 256u + static_cast<uint32_t>(D) * i; }
    __host__ __device__ static constexpr uint32_t col_p(int i) { return kAliasP ? col_s(i) : 256u + 2u * D + 64u * i; }
    static constexpr uint32_t kIdescS = idesc_bf16(kBlockM, kStep, false);
    static constexpr uint32_t kIdescO = idesc_bf16(kBlockM, D, true);
};

// ---- work division -----------------------------------------------------------------------------

// Cached tokens and drafted nodes of sequence b, clamped into the cache.
struct TreeLen {
    int prefix, nodes;
    __device__ __forceinline__ int tiles() const
    {
        const int n = (prefix + nodes + kBlockN - 1) / kBlockN;
        return n > 0 ? n : 1;  // a sequence without keys still has its rows written (O = 0)
    }
};

__device__ __forceinline__ TreeLen tree_clamp(int prefix, int nodes, int T, int Nk_max, int* status)
{
    TreeLen x{prefix, nodes};
    const bool bad = x.prefix < 0 || x.prefix > Nk_max || x.nodes < 0 || x.nodes > T || x.prefix > Nk_max - x.nodes;
    if (bad) {
        atomicCAS(status, 0, FA_ERR_INVALID_ARG);
        x.prefix = min(max(x.prefix, 0), Nk_max);
        x.nodes = min(min(max(x.nodes, 0), T), Nk_max - x.prefix);
    }
    return x;
}

__device__ __forceinline__ TreeLen tree_len(const int* seqlens, const int* n_nodes, int b, int T, int Nk_max, int* status)
{
    return tree_clamp(seqlens[b], n_nodes != nullptr ? n_nodes[b] : T, T, Nk_max, status);
}

// Share c: places [w0, w1) of all units in order (a unit's unit_cost places come before its tiles), and
// the unit and place it starts in.
struct TreeStart {
    long long w0, w1;
    long long total, shares;
    int b, unit, at;    // sequence, unit within the sequence, place within the unit
    int prefix, nodes;  // of the sequence
};

__device__ __forceinline__ long long share_begin(long long c, long long total, long long shares) { return c * total / shares; }

__device__ __forceinline__ TreeLen tree_at(const TreeParams& p, int b)
{
    return tree_len(p.seqlens, p.n_nodes, b, p.T, p.Nk_max, p.status);
}
__device__ __forceinline__ int tree_places(const TreeParams& p, int b) { return tree_at(p, b).tiles() + p.unit_cost; }

// By one warp; every lane returns the same.  Empty (w0 = w1) for shares past the number of places.
__device__ __forceinline__ TreeStart tree_locate(const TreeParams& p, int c, int lane)
{
    const long long upb = static_cast<long long>(p.Hkv) * p.n_qp;
    TreeLen len{0, 0};  // the first 32 sequences'
    if (lane < p.B) len = tree_at(p, lane);
    long long total = lane < p.B ? len.tiles() + p.unit_cost : 0;
    for (int b = 32 + lane; b < p.B; b += 32) total += tree_places(p, b);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    total *= upb;
    const long long shares = p.num_shares < total ? p.num_shares : total;
    TreeStart s{0, 0, total, shares, 0, 0, 0, 0, 0};
    if (c >= shares) return s;
    s.w0 = share_begin(c, total, shares);
    s.w1 = share_begin(c + 1, total, shares);
    long long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        if (b0 > 0 && b < p.B) len = tree_at(p, b);
        const int places = b < p.B ? len.tiles() + p.unit_cost : 0;
        long long incl = places * upb;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const unsigned past = __ballot_sync(0xffffffffu, base + incl > s.w0);
        if (past != 0u) {
            const int j = __ffs(past) - 1;  // the first sequence that ends after w0
            const int pj = __shfl_sync(0xffffffffu, places, j);
            const long long in = s.w0 - (base + __shfl_sync(0xffffffffu, incl, j) - pj * upb);
            s.b = b0 + j;
            s.unit = static_cast<int>(in / pj);
            s.at = static_cast<int>(in - static_cast<long long>(s.unit) * pj);
            s.prefix = __shfl_sync(0xffffffffu, len.prefix, j);
            s.nodes = __shfl_sync(0xffffffffu, len.nodes, j);
            return s;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    s.w1 = s.w0;
    return s;
}

// A share, segment by segment (the producer's).
struct TreeWalk {
    int left;            // places of the share from this segment on
    int used;            // places of this segment
    int b, kvh, qp;      // sequence, key/value head, query block
    int tile, tiles, n;  // first tile of the segment, tiles of the unit, tiles of the segment
    TreeLen len;
    int next_len, next_nodes;  // of sequence b + 1, read one sequence ahead

    __device__ __forceinline__ void begin(const TreeParams& p, const TreeStart& s)
    {
        left = static_cast<int>(s.w1 - s.w0);
        b = kvh = qp = tile = tiles = n = 0;
        len = TreeLen{0, 0};
        if (left == 0) return;
        b = s.b;
        kvh = s.unit / p.n_qp;
        qp = s.unit - kvh * p.n_qp;
        len = TreeLen{s.prefix, s.nodes};
        tiles = len.tiles();
        ahead(p);
        take(p, s.at);
    }
    __device__ __forceinline__ bool live() const { return left > 0; }
    __device__ __forceinline__ void next(const TreeParams& p)
    {
        left -= used;
        if (left == 0) return;
        step(p);
        take(p, 0);
    }
    // the segment at place `at` of the current unit; left = 0 if nothing but a unit's first places is left
    __device__ __forceinline__ void take(const TreeParams& p, int at)
    {
        used = min(tiles + p.unit_cost - at, left);
        tile = max(at - p.unit_cost, 0);
        n = at + used - p.unit_cost - tile;
        if (n <= 0) left = 0;  // the share ends in the unit's first places: its tiles are the next share's
    }
    __device__ __forceinline__ void step(const TreeParams& p)
    {
        if (++qp < p.n_qp) return;
        qp = 0;
        if (++kvh < p.Hkv) return;
        kvh = 0;
        ++b;
        len = tree_clamp(next_len, next_nodes, p.T, p.Nk_max, p.status);
        tiles = len.tiles();
        ahead(p);
    }
    __device__ __forceinline__ void ahead(const TreeParams& p)
    {
        const int i = min(b + 1, p.B - 1);
        next_len = p.seqlens[i];
        next_nodes = p.n_nodes != nullptr ? p.n_nodes[i] : p.T;
    }
    __device__ __forceinline__ int group(const TreeParams& p) const { return b * p.Hkv + kvh; }
    // Slot of a part: of the units that a share holds without finishing them alone, one was begun in the
    // share before (it is the share's first) and one is begun here (its last).
    __device__ __forceinline__ int slot(int share) const { return n == tiles ? -1 : 2 * share + (tile == 0 ? 1 : 0); }
};

// Ancestors of each lane's node t (and t itself) as 128 bits; t < 0: none.  Whole warp: it holds the
// parents, so that a step up is a shuffle instead of a load that waits for the one before it (with
// loads a unit's start took about 3 us).
__device__ __forceinline__ void tree_ancestors(const int* parents, int T, int t, int lane, int* status, uint32_t (&vis)[4])
{
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int bits = min(max(t + 1 - 32 * w, 0), 32);
        vis[w] = parents != nullptr ? 0u : bits == 32 ? 0xffffffffu : (1u << bits) - 1u;  // a chain: nodes 0 .. t
    }
    if (parents == nullptr) return;
    int par[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) par[i] = 32 * i + lane < T ? __ldg(parents + 32 * i + lane) : -1;
    int cur = t;
    while (__any_sync(0xffffffffu, cur >= 0)) {  // strictly decreasing: at most T steps
        int up = -1;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int x = __shfl_sync(0xffffffffu, par[w], cur & 31);
            if (cur >> 5 == w) {
                vis[w] |= 1u << (cur & 31);
                up = x;
            }
        }
        if (cur >= 0 && (up >= cur || up < -1)) {  // not a node before it: taken as a child of the last cached token
            atomicCAS(status, 0, FA_ERR_INVALID_ARG);
            up = -1;
        }
        cur = up;
    }
}

// ---- kernel ------------------------------------------------------------------------------------

// A warp's 32 consecutive rows on their way out, 16 columns at a time through shared memory: a thread's
// row written by itself would be 16-byte pieces of 32 lines an instruction.  A row's 64 bytes are read
// back by four lanes, the 16-byte pieces exchanged by bits of the row, so that neither side has bank
// conflicts.  (The end of a unit is latency: addresses and row tests are made once.)
template <int D>
struct RowsOut {
    char* at;             // this lane's piece of row lane / 4
    uint32_t put, get;    // its places in the warp's 2 KB of shared memory
    int rows;             // of the warp
    bool f32;
    __device__ __forceinline__ RowsOut(uint32_t stage, void* o, bool f32_, size_t first_row, int rows_, int lane)
    {
        const int r = lane >> 2, j = lane & 3;
        f32 = f32_;
        rows = rows_ - r;
        at = static_cast<char*>(o) + (first_row + r) * (D * (f32 ? 4 : 2)) + j * (f32 ? 16 : 8);
        put = stage + lane * 64 + (((lane >> 1) & 3) << 4);
        get = stage + r * 64 + ((j ^ ((r >> 1) & 3)) << 4);
    }
    // columns c .. c + 15 of the lane's row (as 2 x 8)
    __device__ __forceinline__ void store(int c, const float2 (&x)[8]) const
    {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            st_shared_v4(put ^ (j << 4), __float_as_uint(x[2 * j].x), __float_as_uint(x[2 * j].y), __float_as_uint(x[2 * j + 1].x),
                         __float_as_uint(x[2 * j + 1].y));
        __syncwarp();
        float4 v[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) v[it] = ld_shared_f4(get + it * 512);  // rows r, r + 8, ..: the same exchange
        if (f32) {
            char* dst = at + c * 4;
#pragma unroll
            for (int it = 0; it < 4; ++it)
                if (8 * it < rows) *reinterpret_cast<float4*>(dst + it * 8 * D * 4) = v[it];
        } else {
            char* dst = at + c * 2;
#pragma unroll
            for (int it = 0; it < 4; ++it)
                if (8 * it < rows)
                    *reinterpret_cast<uint2*>(dst + it * 8 * D * 2) = make_uint2(pack_bf16x2(v[it].x, v[it].y), pack_bf16x2(v[it].z, v[it].w));
        }
    }
};

__device__ __forceinline__ float2 as_float2(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }

// Masks scores s of the N keys from node index `shift` on (keys before node 0 are cached tokens, seen by
// all) by the row's ancestors; their max.
template <int N>
__device__ __forceinline__ float tree_mask(float (&s)[N], int shift, const uint32_t (&vis)[4])
{
    auto word = [&](int q) -> uint32_t {
        return q == 0 ? vis[0] : q == 1 ? vis[1] : q == 2 ? vis[2] : q == 3 ? vis[3] : 0u;
    };
    float a[N / 32];
#pragma unroll
    for (int q = 0; q < N / 32; ++q) {
        const int bit = shift + 32 * q;
        const int cached = min(max(-bit, 0), 32);  // columns that are cached tokens
        const uint32_t seen = __funnelshift_r(word(bit >> 5), word((bit >> 5) + 1), bit & 31) |
                              (cached == 32 ? 0xffffffffu : (1u << cached) - 1u);
        a[q] = -INFINITY;
#pragma unroll
        for (int c = 0; c < 32; ++c) {
            s[32 * q + c] = (seen >> c) & 1u ? s[32 * q + c] : -INFINITY;
            a[q] = fmaxf(a[q], s[32 * q + c]);
        }
    }
    if constexpr (N == 64) return fmaxf(a[0], a[1]);
    else return fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
}

// A row's running max (of scale * log2(e) * S over visible keys) and sum, for scores with max `mrow`.
struct TreeRow {
    float m = -INFINITY, l = 0.f;
    float alpha;  // what a grown max scales the sum and O by
    __device__ __forceinline__ bool grow(float mrow, float sl2)
    {
        const float mt = mrow * sl2;
        alpha = 1.f;
        if (!(mt > m)) return false;
        alpha = ex2(m - mt);  // 0 when m = -inf
        m = mt;
        return true;
    }
    __device__ __forceinline__ void add(const float2 (&rs)[4])
    {
        l = l * alpha + (((rs[0].x + rs[0].y) + (rs[1].x + rs[1].y)) + ((rs[2].x + rs[2].y) + (rs[3].x + rs[3].y)));
    }
};

// Weights 2^(sl2 s - m) of columns c0 .. c0 + N - 1 into pk, rounded to bf16 for the product (half a step,
// 2^-8 of each weight); their fp32 values are added to the four partial sums rs.
template <int N, int KS>
__device__ __forceinline__ void tree_exps(int c0, const float (&s)[KS], float sl2, float m, float2 (&rs)[4], uint32_t (&pk)[KS / 2])
{
    const float m_use = m == -INFINITY ? 0.f : m;
    const float2 sl2x2 = make_float2(sl2, sl2), negm = make_float2(-m_use, -m_use);
#pragma unroll
    for (int cc = 0; cc < N; cc += 8) {
        const int c = c0 + cc;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 x = __ffma2_rn(make_float2(s[c + 2 * q], s[c + 2 * q + 1]), sl2x2, negm);
            const float2 e = make_float2(ex2(x.x), ex2(x.y));
            rs[q] = __fadd2_rn(rs[q], e);
            pk[c / 2 + q] = pack_bf16x2(e.x, e.y);
        }
    }
}

template <int N>
__device__ __forceinline__ void tree_scale(uint32_t (&o)[N], float alpha)
{
    const float2 a2 = make_float2(alpha, alpha);
#pragma unroll
    for (int e = 0; e < N; e += 2) {
        const float2 x = __fmul2_rn(as_float2(o[e], o[e + 1]), a2);
        o[e] = __float_as_uint(x.x);
        o[e + 1] = __float_as_uint(x.y);
    }
}

template <int D, TreeForm FORM>
__global__ void __launch_bounds__(kTrThreads, 1) fa_tree_kernel(const __grid_constant__ TreeParams p)
{
    using C = TrCfg<D, FORM>;
    constexpr bool ALT = FORM == kAlt, SOLO = FORM == kSolo, PAIR = FORM == kPair;
    constexpr int kStreams = SOLO ? 2 : 1;         // shares, producers, rings
    constexpr int S = C::kStages / kStreams;       // stages of a stream's ring
    constexpr int kSegs = kTrSegs / kStreams;      // records of a stream
    constexpr int H = C::kSteps, KS = C::kStep;    // steps of a tile, keys of a step
    extern __shared__ uint8_t tr_smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tr_smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + C::kOffBar;
    auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
    TreeStart* start_slot = reinterpret_cast<TreeStart*>(smem + C::kOffStart);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffStart + 2 * 64);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert(sizeof(TreeStart) <= 64, "start record");

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const unsigned long long limit = p.wait_limit_ns;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kTbQFull + i), 1);
            mbar_init(bar(kTbQEmpty + i), SOLO ? 1 : 2);
            for (int h = 0; h < 2; ++h) {
                mbar_init(bar(kTbSFull + 2 * i + h), 1);
                mbar_init(bar(kTbPFull + 2 * i + h), kBlockM);
                mbar_init(bar(kTbPVDone + 2 * i + h), 1);
            }
            mbar_init(bar(kTbSFree + i), kBlockM);
            mbar_init(bar(kTbOReady + i), 1);
            mbar_init(bar(kTbOFree + i), 2 * kBlockM);
            mbar_init(bar(kTbDrain + i), 1);
        }
        mbar_init(bar(kTbMLFull), 2 * kBlockM);
        for (int i = 0; i < kTrSegs; ++i) mbar_init(bar(kTbSegFull + i), 1);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(bar(kTbKFull + s), 1);
            mbar_init(bar(kTbKEmpty + s), PAIR ? 2 : 1);
            mbar_init(bar(kTbVFull + s), 1);
            mbar_init(bar(kTbVEmpty + s), PAIR ? 2 : 1);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kTrWarpMma) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    grid_dependency_wait();    // launched as a programmatic dependent of the previous kernel
    grid_launch_dependents();  // the merge may begin launching (it waits for this grid)
    if (warp % 4 == 0 && warp / 4 < kStreams) {  // share `stream * CTAs + CTA`: few shares go to different SMs
        const int stream = warp / 4;
        const TreeStart s = tree_locate(p, stream * static_cast<int>(gridDim.x) + blockIdx.x, lane);
        if (lane == 0) *reinterpret_cast<TreeStart*>(reinterpret_cast<uint8_t*>(start_slot) + 64 * stream) = s;
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    TreeSeg* seg_ring = reinterpret_cast<TreeSeg*>(smem + C::kOffSeg);
    // Record of segment i of a stream (of any role but the producer); n = 0 past the last, and when a wait
    // ran out.
    auto segment = [&](int stream, int i, bool& ok) -> TreeSeg {
        const int at = stream * kSegs + i % kSegs;
        TreeSeg x;
        x.n = 0;
        ok = mbar_wait(bar(kTbSegFull + at), static_cast<uint32_t>(i / kSegs) & 1, limit, abort_flag);
        if (ok) x = seg_ring[at];
        return x;
    };

    if (warp >= kTrWarpProducer) {
        regs_decrease<C::kControlRegs>();
        const int stream = warp == kTrWarpProducer ? 0 : warp == kTrWarpProducer + 3 ? 1 : kStreams;
        if (stream < kStreams) {
            // ======================================================== producer
            if (lane == 0) {
                prefetch_tensormap(&p.tm_q);
                prefetch_tensormap(&p.tm_k);
                prefetch_tensormap(&p.tm_v);
                // K and V are read again only by a group's further query blocks
                const uint64_t pol_kv = p.n_qp > 1 ? policy_evict_last() : policy_evict_first();
                const uint64_t pol_q = policy_evict_first();
                const TreeStart start = *reinterpret_cast<TreeStart*>(reinterpret_cast<uint8_t*>(start_slot) + 64 * stream);
                const int share = stream * static_cast<int>(gridDim.x) + blockIdx.x;
                const int stage0 = stream * S;
                TreeWalk kw, vw;  // K runs one tile ahead of V
                kw.begin(p, start);
                vw.begin(p, start);
                int kj = 0, vj = 0;  // tile within the segment
                int segs = 0;        // records written
                int k_issued = 0, v_issued = 0;
                TreeJoin join{0, 0, 0};
                auto publish = [&](int n) {  // the walk's segment to the other roles
                    TreeSeg x;
                    x.n = n;
                    x.tile = kw.tile;
                    x.prefix = kw.len.prefix;
                    x.nodes = kw.len.nodes;
                    x.b = kw.b;
                    x.group = kw.group(p);
                    x.qp = kw.qp;
                    x.slot = kw.slot(share);
                    if (n > 0 && x.slot >= 0 && kw.tile == 0) {
                        // begun here, finished in the share of its last place
                        const long long last = start.w1 + (kw.tiles - kw.n);
                        join.first_row = static_cast<long long>(x.group) * p.rows + static_cast<long long>(kw.qp) * p.part_rows;
                        join.rows = min(p.part_rows, p.rows - kw.qp * p.part_rows);
                        join.parts = static_cast<int>((last * start.shares - 1) / start.total) - share + 1;
                    }
                    const int at = stream * kSegs + segs % kSegs;
                    seg_ring[at] = x;
                    mbar_arrive(bar(kTbSegFull + at));
                    ++segs;
                };
                auto load_k = [&]() -> bool {
                    const int g = kw.group(p);
                    if (kj == 0) {  // the segment's query rows
                        const int buf = ALT ? segs & 1 : stream;
                        const int use = ALT ? segs >> 1 : segs;
                        if (use > 0 && !mbar_wait(bar(kTbQEmpty + buf), static_cast<uint32_t>(use - 1) & 1, limit, abort_flag))
                            return false;
                        const int row0 = kw.qp * (PAIR ? 2 : 1) * kBlockM;
                        const int q_tiles = PAIR && p.rows - row0 > kBlockM ? 2 : 1;
                        mbar_arrive_expect_tx(bar(kTbQFull + buf), q_tiles * C::kTileBytes);
                        for (int i = 0; i < q_tiles; ++i)
                            for (int cb = 0; cb < C::kNumCB; ++cb)
                                tma_load_3d(sbase + C::kOffQ + (buf + i) * C::kTileBytes + cb * C::kBlkBytes, &p.tm_q,
                                            bar(kTbQFull + buf), cb * C::kCB, row0 + i * kBlockM, g, pol_q);
                        publish(kw.n);
                    }
                    const int s = stage0 + k_issued % S;
                    if (k_issued >= S &&
                        !mbar_wait(bar(kTbKEmpty + s), static_cast<uint32_t>(k_issued / S - 1) & 1, limit, abort_flag))
                        return false;
                    mbar_arrive_expect_tx(bar(kTbKFull + s), C::kTileBytes);
                    for (int cb = 0; cb < C::kNumCB; ++cb)
                        tma_load_3d(sbase + C::kOffK + s * C::kTileBytes + cb * C::kBlkBytes, &p.tm_k, bar(kTbKFull + s),
                                    cb * C::kCB, (kw.tile + kj) * kBlockN, g, pol_kv);
                    ++k_issued;
                    if (++kj == kw.n) {
                        kj = 0;
                        kw.next(p);
                    }
                    return true;
                };
                auto load_v = [&]() -> bool {
                    const int s = stage0 + v_issued % S;
                    if (v_issued >= S &&
                        !mbar_wait(bar(kTbVEmpty + s), static_cast<uint32_t>(v_issued / S - 1) & 1, limit, abort_flag))
                        return false;
                    mbar_arrive_expect_tx(bar(kTbVFull + s), C::kTileBytes);
                    for (int cb = 0; cb < C::kNumCB; ++cb)
                        tma_load_3d(sbase + C::kOffV + s * C::kTileBytes + cb * C::kBlkBytes, &p.tm_v, bar(kTbVFull + s),
                                    cb * C::kCB, (vw.tile + vj) * kBlockN, vw.group(p), pol_kv);
                    ++v_issued;
                    if (++vj == vw.n) {
                        vj = 0;
                        vw.next(p);
                    }
                    return true;
                };
                bool ok = !kw.live() || load_k();
                while (ok && vw.live()) ok = (!kw.live() || load_k()) && load_v();
                const int loads = segs;  // query loads issued
                if (ok) publish(0);
                p.joins[share] = join;
                if (!ok && !*abort_flag) record_failure(p.status, abort_flag, FA_ERR_TIMEOUT);
                // Every issued copy must land before the CTA may exit (its last phase per barrier).
                if constexpr (ALT) {
                    for (int t = loads - 2 < 0 ? 0 : loads - 2; t < loads; ++t)
                        mbar_wait(bar(kTbQFull + (t & 1)), static_cast<uint32_t>(t >> 1) & 1, kDrainLimitNs, nullptr);
                } else if (loads > 0) {
                    mbar_wait(bar(kTbQFull + stream), static_cast<uint32_t>(loads - 1) & 1, kDrainLimitNs, nullptr);
                }
                for (int t = k_issued - S < 0 ? 0 : k_issued - S; t < k_issued; ++t)
                    mbar_wait(bar(kTbKFull + stage0 + t % S), static_cast<uint32_t>(t / S) & 1, kDrainLimitNs, nullptr);
                for (int t = v_issued - S < 0 ? 0 : v_issued - S; t < v_issued; ++t)
                    mbar_wait(bar(kTbVFull + stage0 + t % S), static_cast<uint32_t>(t / S) & 1, kDrainLimitNs, nullptr);
            }
        } else if (warp == kTrWarpMma || warp == kTrWarpMma + 1) {
            // ======================================================== MMA issuers
            if (lane == 0) {
                const int i = warp - kTrWarpMma;  // warpgroup of this issuer
                const uint32_t d_s = tmem + C::col_s(i);
                const uint32_t d_o = tmem + C::col_o(i);
                const uint32_t a_p = tmem + C::col_p(i);
                int tiles = 0;   // tiles whose products have been issued
                int s_done = 0;  // tiles whose scores have been issued
                int k = 0;       // tile of the share
                int segs = 0;    // segments walked
                int o_uses = 0;  // ALT: OFree phases that precede the next first product
                const int my = SOLO ? i : 0;  // stream
                const int stage0 = my * S;
                bool ok = true;
                auto issue_s = [&](int q_tile, int stage, int h) {
                    const uint64_t a0 = smem_desc(sbase + C::kOffQ + q_tile * C::kTileBytes, 16, C::kAtomBytes, C::kLayout);
                    const uint64_t b0 = smem_desc(sbase + C::kOffK + stage * C::kTileBytes + h * KS * C::kRowBytes, 16,
                                                  C::kAtomBytes, C::kLayout);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk * 16) / C::kCB * C::kBlkBytes + ((kk * 16) % C::kCB) * 2) >> 4;
                        umma_ss(d_s + KS * h, a0 + off, b0 + off, C::kIdescS, kk > 0 ? 1u : 0u);
                    }
                };
                auto issue_pv = [&](int stage, int h, bool accumulate) {
                    const uint64_t b0 = smem_desc(sbase + C::kOffV + stage * C::kTileBytes + h * KS * C::kRowBytes, C::kBlkBytes,
                                                  C::kAtomBytes, C::kLayout);
#pragma unroll
                    for (int kk = 0; kk < KS / 16; ++kk)
                        umma_ts(d_o, a_p + KS * h + 8u * kk, b0 + ((kk * 16 * C::kRowBytes) >> 4), C::kIdescO,
                                (accumulate || kk > 0) ? 1u : 0u);
                };
                // Step h of S_i of share tile kk: its columns must have been read (and, where the weights
                // overwrite them, the product with those must have completed).
                auto do_s = [&](int q_tile, int q_buf, int kk, int h, bool last) -> bool {
                    const int s = stage0 + kk % S;
                    if (h == 0 && !mbar_wait(bar(kTbKFull + s), static_cast<uint32_t>(kk / S) & 1, limit, abort_flag)) return false;
                    if (s_done > 0 && !mbar_wait(bar(C::kAliasP ? kTbPVDone + 2 * i + h : kTbSFree + i),
                                                 static_cast<uint32_t>(s_done - 1) & 1, limit, abort_flag))
                        return false;
                    tc_fence_after_sync();
                    issue_s(q_tile, s, h);
                    umma_commit(bar(kTbSFull + 2 * i + h));
                    if (h == H - 1) {
                        ++s_done;
                        umma_commit(bar(kTbKEmpty + s));
                        if (last) umma_commit(bar(kTbQEmpty + q_buf));
                    }
                    return true;
                };
                constexpr int step = ALT ? 2 : 1;
                while (ok) {
                    const TreeSeg w = segment(my, segs, ok);
                    if (w.n == 0) break;
                    const int q_buf = ALT ? segs & 1 : my;
                    const int q_tile = ALT ? q_buf : i;
                    const int j0 = ALT ? (k + i) & 1 : 0;  // first tile of the segment for this warpgroup
                    // Also without tiles of its own in the segment: an issuer that skipped a phase of the
                    // query barrier could take the phase before it for the one it needs.
                    ok = mbar_wait(bar(kTbQFull + q_buf), static_cast<uint32_t>(ALT ? segs >> 1 : segs) & 1, limit, abort_flag);
                    if (!ok) break;
                    const bool rows = !PAIR || i == 0 || p.rows - w.qp * 2 * kBlockM > kBlockM;
                    if (!rows || j0 >= w.n) {
                        // (The queries first: the producer may be waiting to load the next unit's ahead of
                        // this unit's last V.)
                        mbar_arrive(bar(kTbQEmpty + q_buf));
                        if (PAIR) {  // no rows: pass every tile on
                            for (int j = 0; ok && j < w.n; ++j) {
                                const int s = (k + j) % S;
                                const uint32_t ph = static_cast<uint32_t>((k + j) / S) & 1;
                                ok = mbar_wait(bar(kTbKFull + s), ph, limit, abort_flag) &&
                                     mbar_wait(bar(kTbVFull + s), ph, limit, abort_flag);
                                if (!ok) break;
                                mbar_arrive(bar(kTbKEmpty + s));
                                mbar_arrive(bar(kTbVEmpty + s));
                            }
                        }
                    } else {
                        const int j_last = j0 + (w.n - 1 - j0) / step * step;
                        for (int h = 0; ok && h < H; ++h) ok = do_s(q_tile, q_buf, k + j0, h, j0 == j_last);
                        for (int j = j0; ok && j < w.n; j += step) {
                            const int kk = k + j;
                            const int s = stage0 + kk % S;
                            const uint32_t ph = static_cast<uint32_t>(tiles) & 1;
                            if constexpr (H == 1) {
                                // Without aliasing the next scores need only the current ones read: they run
                                // while this tile is still being exponentiated.
                                if (!C::kAliasP && j + step < w.n) ok = do_s(q_tile, q_buf, kk + step, 0, j + step == j_last);
                                ok = ok && mbar_wait(bar(kTbPFull + 2 * i), ph, limit, abort_flag) &&
                                     mbar_wait(bar(kTbVFull + s), static_cast<uint32_t>(kk / S) & 1, limit, abort_flag);
                                // The first product of a segment overwrites O_i: the last segment's must have been
                                // read.  P's arrival means that for this warpgroup; in ALT form the other reads O_i
                                // too.  (Waited for after P: this warpgroup has then been through every earlier
                                // segment's exchange, so the barrier is at most one phase behind.)
                                if (ALT && ok && j == j0 && o_uses > 0)
                                    ok = mbar_wait(bar(kTbOFree + i), static_cast<uint32_t>(o_uses - 1) & 1, limit, abort_flag);
                                if (!ok) break;
                                tc_fence_after_sync();
                                issue_pv(s, 0, j > j0);
                                umma_commit(bar(kTbPVDone + 2 * i));
                                if (j == j_last) umma_commit(bar(kTbOReady + i));
                                umma_commit(bar(kTbVEmpty + s));
                                ++tiles;
                                if (C::kAliasP && j + step < w.n) ok = do_s(q_tile, q_buf, kk + step, 0, j + step == j_last);
                            } else {
                                static_assert(H == 1 || (PAIR && C::kAliasP), "two steps");
                                // Scores run a step or more ahead of the weights: while the softmax works on one
                                // step, the other's product and its next scores are under way.
                                bool early = false;
                                for (int h = 0; ok && h < 2; ++h) {
                                    ok = mbar_wait(bar(kTbPFull + 2 * i + h), ph, limit, abort_flag);
                                    if (h == 0) ok = ok && mbar_wait(bar(kTbVFull + s), static_cast<uint32_t>(kk / S) & 1, limit, abort_flag);
                                    if (!ok) break;
                                    tc_fence_after_sync();
                                    issue_pv(s, h, j > j0 || h > 0);
                                    umma_commit(bar(kTbPVDone + 2 * i + h));
                                    if (h == 1) {
                                        if (j == j_last) umma_commit(bar(kTbOReady + i));
                                        umma_commit(bar(kTbVEmpty + s));
                                    }
                                    // The next tile's scores in the columns that this product frees; its first step's
                                    // now only if its keys are there already: the second step's product must not wait
                                    // for them (V's stage, and with it the next V, would wait too).
                                    if (j + step < w.n) {
                                        const int nx = stage0 + (kk + step) % S;
                                        if (h == 0) early = mbar_test(bar(kTbKFull + nx), static_cast<uint32_t>((kk + step) / S) & 1);
                                        if (h == 0 ? early : !early) ok = do_s(q_tile, q_buf, kk + step, 0, j + step == j_last);
                                        if (h == 1) ok = ok && do_s(q_tile, q_buf, kk + step, 1, j + step == j_last);
                                    }
                                }
                                ++tiles;
                            }
                        }
                    }
                    ++o_uses;
                    k += w.n;
                    ++segs;
                }
                if (!ok && !*abort_flag) record_failure(p.status, abort_flag, FA_ERR_TIMEOUT);
                umma_commit(bar(kTbDrain + i));
                mbar_wait(bar(kTbDrain + i), 0, kDrainLimitNs, nullptr);
            }
        }
    } else {
        regs_increase<C::kSoftmaxRegs>();
        // ============================================================ softmax + epilogue
        const int wg = warp >> 2;
        const int r = threadIdx.x & 127;  // row of the tile == TMEM lane
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lane_base + C::col_s(wg);
        const uint32_t t_o = tmem + lane_base + C::col_o(wg);
        const uint32_t t_p = tmem + lane_base + C::col_p(wg);
        const float sl2 = p.scale_log2;
        int tiles = 0;                 // key tiles processed by this warpgroup
        int ready[2] = {0, 0};         // segments with tiles of warpgroup 0, 1 (ALT); this warpgroup's (else, [0])
        int segs = 0, k = 0;
        const int my = SOLO ? wg : 0;  // stream
        float2* ml = reinterpret_cast<float2*>(smem + C::kOffML);
        constexpr int step = ALT ? 2 : 1;
        uint32_t vis[4] = {0u, 0u, 0u, 0u};
        int vis_b = -1, vis_qp = -1;
        bool ok = true;
        const uint32_t stage = sbase + C::kOffStage + warp * 2048;
        while (ok) {
            const TreeSeg w = segment(my, segs, ok);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || w.n == 0) break;
            const int row0 = PAIR ? w.qp * 2 * kBlockM + wg * kBlockM : 0;
            const int rows = min(p.rows - row0, kBlockM);  // rows of this warpgroup's tile (<= 0: none)
            if (PAIR && rows <= 0) {
                k += w.n;
                ++segs;
                continue;
            }
            const int rows_warp = rows - 32 * (warp & 3);  // of this warp (<= 0: none)
            const bool warp_live = rows_warp > 0;
            const int j0 = ALT ? (k + wg) & 1 : 0;  // first tile of the segment for this warpgroup
            const int end = w.prefix + w.nodes;     // keys of the sequence
            // the row's ancestors, kept while the sequence and the row stay the same
            if ((w.tile + w.n) * kBlockN > w.prefix && (w.b != vis_b || (PAIR && w.qp != vis_qp))) {
                vis_b = w.b;
                vis_qp = w.qp;
                const int node = (row0 + r) % p.T;
                tree_ancestors(p.parents != nullptr ? p.parents + static_cast<size_t>(w.b) * p.T : nullptr, p.T,
                               r < rows && node < w.nodes ? node : -1, lane, p.status, vis);
            }
            TreeRow row;
            // V rows past the tree may hold anything: zero them before the product reads them.  (The stage's
            // tile before has been consumed, by the issuer that then issued this tile's scores, so the phase
            // parity cannot mean that one.)
            auto zero_tail = [&](int j, int k0) {
                const int vs = my * S + (k + j) % S;  // V stage
                ok = __all_sync(0xffffffffu, mbar_wait(bar(kTbVFull + vs), static_cast<uint32_t>((k + j) / S) & 1, limit, abort_flag));
                if (!ok) return;
                if (k0 + r >= end) {
                    const uint32_t vrow = sbase + C::kOffV + vs * C::kTileBytes + r * C::kRowBytes;
#pragma unroll
                    for (int cb = 0; cb < C::kNumCB; ++cb)
#pragma unroll
                        for (int c16 = 0; c16 < C::kRowBytes; c16 += 16)
                            st_shared_v4(vrow + cb * C::kBlkBytes + c16, 0u, 0u, 0u, 0u);
                }
                fence_proxy_async_shared();
            };
            for (int j = j0; ok && j < w.n; j += step) {
                const int k0 = (w.tile + j) * kBlockN;
                if constexpr (H == 1) {
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(kTbSFull + 2 * wg), tiles & 1, limit, abort_flag));
                    if (!ok) break;
                    tc_fence_after_sync();
                    if (warp_live) {
                        uint32_t u[kBlockN];
                        float mrow;
                        if constexpr (D == 128) {
                            float mh[2];
                            tmem_ld64_max(t_s + 0, *reinterpret_cast<uint32_t(*)[64]>(&u[0]), mh[0]);
                            tmem_ld64_max(t_s + 64, *reinterpret_cast<uint32_t(*)[64]>(&u[64]), mh[1]);
                            tmem_ld_wait();
                            mrow = fmaxf(mh[0], mh[1]);
                        } else {
                            float mq[4];
                            tmem_ld32_max(t_s + 0, *reinterpret_cast<uint32_t(*)[32]>(&u[0]), mq[0]);
                            tmem_ld32_max(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(&u[32]), mq[1]);
                            tmem_ld32_max(t_s + 64, *reinterpret_cast<uint32_t(*)[32]>(&u[64]), mq[2]);
                            tmem_ld32_max(t_s + 96, *reinterpret_cast<uint32_t(*)[32]>(&u[96]), mq[3]);
                            tmem_ld_wait();
                            mrow = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
                        }
                        if constexpr (!C::kAliasP) {
                            tc_fence_before_sync();
                            mbar_arrive(bar(kTbSFree + wg));
                        }
                        float s[kBlockN];
#pragma unroll
                        for (int c = 0; c < kBlockN; ++c) s[c] = __uint_as_float(u[c]);
                        if (k0 + kBlockN > w.prefix) mrow = tree_mask(s, k0 - w.prefix, vis);  // drafted rows, or rows past them
                        const bool rescale = __any_sync(0xffffffffu, row.grow(mrow, sl2)) && j > j0;
                        float2 rs[4] = {};
                        uint32_t pk[kBlockN / 2];
                        if constexpr (C::kAliasP) {
                            // The previous product has completed (the arrival of S_i implies it): where the
                            // max grew, O_i is rescaled 32 columns at a time under the exponentials of 32.
#pragma unroll
                            for (int c = 0; c < kBlockN; c += 32) {
                                uint32_t oc[32];
                                if (rescale) tmem_ld32(t_o + static_cast<uint32_t>(c), oc);
                                tree_exps<32>(c, s, sl2, row.m, rs, pk);
                                if (rescale) {
                                    tmem_ld_wait();
                                    tree_scale(oc, row.alpha);
                                    tmem_st32(t_o + static_cast<uint32_t>(c), oc);
                                }
                            }
                        } else {
#pragma unroll
                            for (int c = 0; c < kBlockN; c += 32) tree_exps<32>(c, s, sl2, row.m, rs, pk);
                            // O_i and P_i are free once the previous product has completed
                            if (j > j0) {
                                ok = __all_sync(0xffffffffu, mbar_wait(bar(kTbPVDone + 2 * wg), (tiles - 1) & 1, limit, abort_flag));
                                if (!ok) break;
                                tc_fence_after_sync();
                            }
                            if (rescale) {
                                uint32_t oc[D / 32][32];
#pragma unroll
                                for (int c = 0; c < D / 32; ++c) tmem_ld32(t_o + 32u * c, oc[c]);
                                tmem_ld_wait();
#pragma unroll
                                for (int c = 0; c < D / 32; ++c) {
                                    tree_scale(oc[c], row.alpha);
                                    tmem_st32(t_o + 32u * c, oc[c]);
                                }
                            }
                        }
                        tmem_st32(t_p + 0, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
                        tmem_st32(t_p + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
                        tmem_st_wait();
                        row.add(rs);
                    } else if (!C::kAliasP) {
                        mbar_arrive(bar(kTbSFree + wg));
                        // A warp without rows waits for the previous product too: with the next scores
                        // already there, it could otherwise arrive twice in one phase of PFull.
                        if (j > j0) {
                            ok = __all_sync(0xffffffffu, mbar_wait(bar(kTbPVDone + 2 * wg), (tiles - 1) & 1, limit, abort_flag));
                            if (!ok) break;
                        }
                    }
                    if (k0 + kBlockN > end) {
                        zero_tail(j, k0);
                        if (!ok) break;
                    }
                    tc_fence_before_sync();
                    mbar_arrive(bar(kTbPFull + 2 * wg));
                } else {
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        ok = __all_sync(0xffffffffu, mbar_wait(bar(kTbSFull + 2 * wg + h), tiles & 1, limit, abort_flag));
                        if (!ok) break;
                        tc_fence_after_sync();
                        if (warp_live) {
                            uint32_t u[KS];
                            float mrow;
                            tmem_ld64_max(t_s + KS * h, u, mrow);
                            tmem_ld_wait();
                            float s[KS];
#pragma unroll
                            for (int c = 0; c < KS; ++c) s[c] = __uint_as_float(u[c]);
                            const int shift = k0 + KS * h - w.prefix;
                            if (shift > -KS) mrow = tree_mask(s, shift, vis);  // drafted rows, or rows past them
                            const bool grow = row.grow(mrow, sl2);
                            float2 rs[4] = {};
                            uint32_t pk[KS / 2];
                            tree_exps<KS>(0, s, sl2, row.m, rs, pk);
                            row.add(rs);
                            // the columns of these scores are free: each thread has read its own
                            tmem_st32(t_p + KS * h, pk);
                            if (__any_sync(0xffffffffu, grow) && (j > j0 || h > 0)) {
                                // O_i can be rescaled once the product before (the other step's) has completed.  (The
                                // one before that has: the arrival of these scores means it, so the parity is clear.)
                                const uint32_t ph = static_cast<uint32_t>(h == 1 ? tiles : tiles - 1) & 1;
                                ok = __all_sync(0xffffffffu, mbar_wait(bar(kTbPVDone + 2 * wg + 1 - h), ph, limit, abort_flag));
                                if (!ok) break;
                                tc_fence_after_sync();
#pragma unroll
                                for (int c0 = 0; c0 < D; c0 += 64) {
                                    uint32_t oc[64];
#pragma unroll
                                    for (int c = 0; c < 64; c += 32) tmem_ld32(t_o + static_cast<uint32_t>(c0 + c), *reinterpret_cast<uint32_t(*)[32]>(&oc[c]));
                                    tmem_ld_wait();
                                    tree_scale(oc, row.alpha);
#pragma unroll
                                    for (int c = 0; c < 64; c += 32) tmem_st32(t_o + static_cast<uint32_t>(c0 + c), *reinterpret_cast<uint32_t(*)[32]>(&oc[c]));
                                }
                            }
                            tmem_st_wait();
                        }
                        if (k0 + kBlockN > end && h == 0) {
                            zero_tail(j, k0);
                            if (!ok) break;
                        }
                        tc_fence_before_sync();
                        mbar_arrive(bar(kTbPFull + 2 * wg + h));
                    }
                }
                ++tiles;
            }
            if (!ok) break;
            // ---- end of the segment: its rows' output and log-sum-exp, final or to a slot
            const bool part = w.slot >= 0;
            const bool shown = (row0 + r) % p.T < w.nodes;  // rows of nodes past the tree: O = 0, LSE = -inf
            // first row of the warp in the output (or the slots)
            const size_t first = part ? static_cast<size_t>(w.slot) * p.part_rows + (PAIR ? wg * kBlockM : 0) + 32 * (warp & 3)
                                      : static_cast<size_t>(w.group) * p.rows + row0 + 32 * (warp & 3);
            const RowsOut<D> out(stage, part ? static_cast<void*>(p.o_part) : p.o, part || p.o_dtype == FA_F32, first, rows_warp, lane);
            auto store_lse = [&](float lse) {
                if (lane < rows_warp) {
                    if (part) p.lse_part[first + lane] = lse;
                    else if (p.lse != nullptr) p.lse[first + lane] = lse;
                }
            };
            if constexpr (!ALT) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar(kTbOReady + wg), ready[0] & 1, limit, abort_flag));
                if (!ok) break;
                ++ready[0];
                tc_fence_after_sync();
                if (warp_live) {
                    const bool none = row.l == 0.f || !shown;
                    const bool hide = __any_sync(0xffffffffu, none);
                    const float inv = none ? 0.f : 1.f / row.l;
                    const float2 inv2 = make_float2(inv, inv);
                    uint32_t o[16];
                    tmem_ld16(t_o, o);
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float2 x[8];
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = __fmul2_rn(as_float2(o[2 * e], o[2 * e + 1]), inv2);
                        if (c + 16 < D) tmem_ld16(t_o + static_cast<uint32_t>(c + 16), o);  // on its way while these are stored
                        if (hide) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = none ? make_float2(0.f, 0.f) : x[e];
                        }
                        out.store(c, x);
                    }
                    store_lse(none ? -INFINITY : (row.m + lg2_approx(row.l)) * 0.69314718055994531f);
                }
            } else {
                const int jw[2] = {k & 1, (k + 1) & 1};  // first tile of the segment for warpgroups 0 and 1
                const bool has0 = jw[0] < w.n, has1 = jw[1] < w.n;
                // the other warpgroup must have read the previous segment's max and sum
                if (segs > 0) ok = mbar_wait(bar(kTbOFree + wg), static_cast<uint32_t>(segs - 1) & 1, limit, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ml[wg * kBlockM + r] = make_float2(row.m, row.l);
                mbar_arrive(bar(kTbMLFull));
                ok = mbar_wait(bar(kTbMLFull), static_cast<uint32_t>(segs) & 1, limit, abort_flag);
                if (ok && has0) ok = mbar_wait(bar(kTbOReady + 0), ready[0] & 1, limit, abort_flag);
                if (ok && has1) ok = mbar_wait(bar(kTbOReady + 1), ready[1] & 1, limit, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ready[0] += has0 ? 1 : 0;
                ready[1] += has1 ? 1 : 0;
                tc_fence_after_sync();
                if (warp_live) {
                    const float2 x0 = ml[r], x1 = ml[kBlockM + r];
                    const float M = fmaxf(x0.x, x1.x);
                    const float f0 = x0.x == -INFINITY ? 0.f : ex2(x0.x - M);
                    const float f1 = x1.x == -INFINITY ? 0.f : ex2(x1.x - M);
                    const float L = x0.y * f0 + x1.y * f1;
                    const bool none = L == 0.f || !shown;
                    const float inv = none ? 0.f : 1.f / L;
                    const float g0 = f0 * inv, g1 = f1 * inv;
                    // this warpgroup's half of the columns
                    const uint32_t col0 = static_cast<uint32_t>(wg * (D / 2));
                    const uint32_t t_o0 = tmem + lane_base + C::col_o(0) + col0;
                    const uint32_t t_o1 = tmem + lane_base + C::col_o(1) + col0;
                    const bool hide = __any_sync(0xffffffffu, none);
                    const float2 w0 = make_float2(g0, g0), w1 = make_float2(g1, g1);
                    uint32_t a[16], b[16];
                    auto load = [&](uint32_t c) {  // a warpgroup without tiles has nothing in its columns
                        if (has0) tmem_ld16(t_o0 + c, a);
                        if (has1) tmem_ld16(t_o1 + c, b);
                    };
                    load(0u);
#pragma unroll 1
                    for (int c = 0; c < D / 2; c += 16) {
                        float2 x[8];
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = make_float2(0.f, 0.f);
                        if (has0) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = __fmul2_rn(as_float2(a[2 * e], a[2 * e + 1]), w0);
                        }
                        if (has1) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = __ffma2_rn(as_float2(b[2 * e], b[2 * e + 1]), w1, x[e]);
                        }
                        if (c + 16 < D / 2) load(static_cast<uint32_t>(c + 16));  // on their way while these are stored
                        if (hide) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = none ? make_float2(0.f, 0.f) : x[e];
                        }
                        out.store(static_cast<int>(col0) + c, x);
                    }
                    if (wg == 0) store_lse(none ? -INFINITY : (M + lg2_approx(L)) * 0.69314718055994531f);
                }
                tc_fence_before_sync();
                mbar_arrive(bar(kTbOFree + 0));
                mbar_arrive(bar(kTbOFree + 1));
            }
            k += w.n;
            ++segs;
        }
        if (!ok && !*abort_flag) record_failure(p.status, abort_flag, FA_ERR_TIMEOUT);
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == kTrWarpMma) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// Joins the parts of the units that several CTAs share: lse = log sum_s exp(lse_s),
// o = sum_s exp(lse_s - lse) o_s ("flash_lab.py" section 4).  Blocks (c, y) serve the unit that share
// c began and did not finish, if there is one (joins[c]): its part is in that share's second slot, the
// others in the following shares' first (slot()).  The time is the latency of the parts' loads, so all of
// them are in flight at once, or in two goes, where they are few (up to 8: eight lanes to a row, 32 rows a
// block), and eight at a time otherwise (a warp a row, 8 rows a block).
constexpr int kFew = 8;

template <int D>
__global__ void __launch_bounds__(256) fa_tree_merge_kernel(const __grid_constant__ TreeParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int c0 = blockIdx.x;
    const TreeJoin join = p.joins[c0];
    const int n = join.parts;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
    auto at = [&](int s, int r) -> size_t {  // row of part s in the slots
        return static_cast<size_t>(2 * (c0 + s) + (s == 0 ? 1 : 0)) * p.part_rows + static_cast<size_t>(r);
    };
    auto write = [&](size_t i, float4 v) {
        if (p.o_dtype == FA_F32) reinterpret_cast<float4*>(p.o)[i / 4] = v;
        else *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.o) + i) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    };
    if (n <= kFew) {
        if (blockIdx.y % 4 != 0) return;
        const int r = static_cast<int>(blockIdx.y) * 8 + warp * 4 + (lane >> 3);
        if (r >= join.rows) return;  // (no warp-wide operation below)
        const int l8 = lane & 7;
        constexpr int Q = D / 32;  // float4 of a lane
        float4 v[4][Q];
        auto load = [&](int s0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (s0 + j >= n) continue;
                const float4* src = reinterpret_cast<const float4*>(p.o_part + at(s0 + j, r) * D) + l8;
#pragma unroll
                for (int i = 0; i < Q; ++i) v[j][i] = __ldcg(src + 8 * i);
            }
        };
        float x[kFew];
#pragma unroll
        for (int s = 0; s < kFew; ++s) x[s] = s < n ? __ldcg(p.lse_part + at(s, r)) : -INFINITY;
        load(0);  // with the log-sum-exps
        float M = -INFINITY;
        bool live = false;
#pragma unroll
        for (int s = 0; s < kFew; ++s) {
            live = live || x[s] != -INFINITY;
            M = fmaxf(M, x[s]);
        }
        float sum = 0.f;
#pragma unroll
        for (int s = 0; s < kFew; ++s) {
            x[s] = x[s] == -INFINITY ? 0.f : ex2((x[s] - M) * kLog2e);
            sum += x[s];
        }
        const float inv = live ? 1.f / sum : 0.f;
        float4 a[Q];
#pragma unroll
        for (int i = 0; i < Q; ++i) a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int s0 = 0; s0 < kFew; s0 += 4) {
            if (s0 >= n) continue;
            if (s0 > 0) load(s0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float f = x[s0 + j] * inv;  // an empty part's output is 0
                if (s0 + j >= n) continue;
#pragma unroll
                for (int i = 0; i < Q; ++i)
                    a[i] = make_float4(fmaf(f, v[j][i].x, a[i].x), fmaf(f, v[j][i].y, a[i].y), fmaf(f, v[j][i].z, a[i].z),
                                       fmaf(f, v[j][i].w, a[i].w));
            }
        }
        const size_t row = static_cast<size_t>(join.first_row) + r;
#pragma unroll
        for (int i = 0; i < Q; ++i) write(row * D + 4 * (l8 + 8 * i), a[i]);
        if (l8 == 0 && p.lse != nullptr) p.lse[row] = live ? M + log2f(sum) * kLn2 : -INFINITY;
        return;
    }
    const int r = static_cast<int>(blockIdx.y) * 8 + warp;
    if (r >= join.rows) return;
    constexpr int kHeld = kTreeMaxShares / 32;  // log-sum-exps a lane holds: at most a part for each share
    constexpr int V = D / 32;                 // columns of a lane
    float x[kHeld];
    float M = -INFINITY;
    bool live = false;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int s = 32 * i + lane;
        x[i] = s < n ? __ldcg(p.lse_part + at(s, r)) : -INFINITY;
        live = live || x[i] != -INFINITY;
        M = fmaxf(M, x[i]);
    }
    live = __any_sync(0xffffffffu, live);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        x[i] = x[i] == -INFINITY ? 0.f : ex2((x[i] - M) * kLog2e);
        sum += x[i];
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = live ? 1.f / sum : 0.f;
    float acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int m = min(32, n - 32 * i);
#pragma unroll 8
        for (int j = 0; j < m; ++j) {
            const float f = __shfl_sync(0xffffffffu, x[i], j) * inv;
            const float* src = p.o_part + at(32 * i + j, r) * D + lane * V;
            float v[V];
            if constexpr (V == 4) *reinterpret_cast<float4*>(v) = __ldcg(reinterpret_cast<const float4*>(src));
            else if constexpr (V == 2) *reinterpret_cast<float2*>(v) = __ldcg(reinterpret_cast<const float2*>(src));
            else v[0] = __ldcg(src);
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = fmaf(f, v[e], acc[e]);
        }
    }
    const size_t row = static_cast<size_t>(join.first_row) + r;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if (p.o_dtype == FA_F32)
            reinterpret_cast<float*>(p.o)[row * D + lane * V + e] = acc[e];
        else
            reinterpret_cast<__nv_bfloat16*>(p.o)[row * D + lane * V + e] = __float2bfloat16_rn(acc[e]);
    }
    if (lane == 0 && p.lse != nullptr) p.lse[row] = live ? M + log2f(sum) * kLn2 : -INFINITY;
}

template <int D, TreeForm FORM>
cudaError_t launch_tree_t(const TreeParams& p, cudaStream_t st)
{
    using C = TrCfg<D, FORM>;
    auto kern = fa_tree_kernel<D, FORM>;
    static bool configured[64] = {};  // attributes set and registers checked, per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess) return e;
        cudaFuncAttributes attr;
        e = cudaFuncGetAttributes(&attr, kern);
        if (e != cudaSuccess) return e;
        // a register increase that the launch's pool cannot satisfy would wait forever
        if (attr.numRegs * kTrThreads < 256 * C::kSoftmaxRegs + 128 * C::kControlRegs)
            return cudaErrorLaunchOutOfResources;
        configured[dev] = true;
    }
    e = launch_pdl(kern, dim3(static_cast<unsigned>(p.num_ctas)), kTrThreads, C::kSmemBytes, st, p);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(p.num_shares), static_cast<unsigned>((p.part_rows + 7) / 8));
    return launch_pdl(fa_tree_merge_kernel<D>, grid, 256, 0, st, p);
}

template <int D>
cudaError_t launch_tree_d(const TreeParams& p, cudaStream_t st)
{
    if (p.part_rows > kBlockM) return launch_tree_t<D, kPair>(p, st);
    return p.num_shares > p.num_ctas ? launch_tree_t<D, kSolo>(p, st) : launch_tree_t<D, kAlt>(p, st);
}

}  // namespace fa

// tree_attn.cuh -- schedule shared by the draft-tree / latent attention kernels.
//
// Work.  A (batch, KV head) pair holds R = n_draft * G query rows (row r is drafted token r / G of
// query head r % G of the group) that all read the same cache slots, cut into RT row tiles of RP
// rows.  The slots of a pair are cut into tiles of TS; the drafted tokens are one more tile at
// the end, the only one with a mask per row.  The tiles of all pairs form one sequence, split
// into equal contiguous ranges over `groups` groups of RT blocks; block (g, rt) of a group
// walks range g for row tile rt, so the RT blocks that read the same slots run side by side
// and all but the first find them in L2.
//
// The lengths live on the device, so every warp finds its block's range by itself: it scans the
// pairs' tile counts (one read of the lengths, no block barrier), which makes the ranges equal
// however ragged the batch is, without a host round trip.
//
// A pair that lies inside one range is finished by its block.  A pair that crosses ranges leaves
// one partial state (max, sum, unnormalised output) per range: workspace slot 2*block for the
// first pair of a block's range, 2*block + 1 for its last; tree_merge_kernel, launched next,
// joins them in range order (no atomics: results do not depend on timing).
//
// Short pairs are not split: the ranges are whole pairs then, and the merge is not launched.  The
// tensor-core kernel does so where the most tiles that a pair can have (by the cache's capacity, which
// the host knows) are kWholeTiles at most and the fullest range has no more than kWholeWait tiles above
// the mean.  Measured with 8 rows and 128 dims, split and whole: 128 pairs of 4 tiles 15.5 and 11.1 us,
// of 12 tiles 25.6 and 20.0; 512 pairs of 4 tiles 39.8 and 34.7.  With more tiles above the mean
// splitting wins: 8 pairs of 9 tiles 11.1 and 15.0, 192 pairs of 12 tiles 36.0 and 41.3.  Latent tiles
// take longer: 1 sequence of 3 tiles 9.8 and 9.9, of 4 tiles 10.0 and 11.6.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace kvc {

constexpr int kWholeTiles = 12, kWholeWait = 4, kWholeWaitLatent = 3;
constexpr int kPairEnd = 2;
// A running maximum that has seen nothing: no finite logit (in log2 units) lies below it, and it is
// finite, so that differences with it are no NaN.
constexpr float kNoMax = -3.402823466e38f;
constexpr int kDevBadLengthCode = 5;         // KVC_DEV_BAD_LENGTH
constexpr int kDevBadBlockCode = 9;          // KVC_DEV_BAD_BLOCK

// Cached slots and drafted tokens of a pair, clamped to their ranges.
__device__ __forceinline__ int tree_len(const TreeParams &p, int pair)
{
    int n = p.n_valid;
    if (p.len != nullptr) n = p.len[p.len_per_pair ? pair : pair / p.Hkv];
    return n < 0 ? 0 : (n > p.cap ? p.cap : n);
}
__device__ __forceinline__ int tree_count(const TreeParams &p, int b)
{
    if (p.count == nullptr) return p.T;
    const int n = p.count[b];
    return n < 0 ? 0 : (n > p.T ? p.T : n);
}
// Tiles of a pair: its slots, then the drafted tokens; at least one when it has rows to write.
__device__ __forceinline__ int tree_tiles(const TreeParams &p, int len, int cnt, int TS)
{
    if (cnt == 0) return 0;
    const int n = (len + TS - 1) / TS + (p.kd != nullptr ? 1 : 0);
    return n > 0 ? n : 1;
}

// The same with what the end of a pair costs a block (its outputs, then the next pair's first S and
// softmax with nothing before them), so that ranges with such an end get fewer tiles.
// Counted as none, one and two tiles: 32 pairs of 5243 slots 29.9, 29.1 and 28.3 us, 8 pairs of up to
// 13107 slots of 256 dims 29.4, 28.1 and 27.6, 32 latent sequences 45.4, 44.6 and 44.4.
__device__ __forceinline__ int tree_cost(const TreeParams &p, int len, int cnt, int TS)
{
    const int n = tree_tiles(p, len, cnt, TS);
    return n > 0 ? n + kPairEnd : 0;
}

// Range g holds the units [g*q + min(g, r), ...): q units, one more in the first r ranges.
struct TreeRange {
    int pair, off;               // first pair of the range and the unit inside it
    int len, cnt;                // that pair's slots and drafted tokens
    int n;                       // units in the range
    long long t0;                // the range's first unit
    long long q;
    int r;
    __device__ __forceinline__ int group_of(long long t) const
    {
        const long long big = r * (q + 1);
        return (int)(t < big ? t / (q + 1) : r + (t - big) / q);
    }
};

// Called by a converged warp; every warp of a block gets the same range.
__device__ __forceinline__ TreeRange tree_range(const TreeParams &p, int g, int TS)
{
    const int lane = threadIdx.x & 31;
    // items: pairs, or whole sequences (Hkv equal pairs) where the heads share a length
    const int items = p.len_per_pair ? p.P : p.B, heads = p.len_per_pair ? 1 : p.Hkv;
    const int per = (items + 31) >> 5;
    const int q0 = min(items, lane * per), q1 = min(items, q0 + per);
    const bool check = blockIdx.x == 0 && threadIdx.x < 32;
    if (p.whole) {
        if (check) {
            for (int q = lane; q < items; q += 32) {
                const int n = p.len != nullptr ? p.len[q] : p.n_valid;
                const int c = p.count == nullptr ? p.T : p.count[p.len_per_pair ? q / p.Hkv : q];
                if (n < 0 || n > p.cap || c < 0 || c > p.T) record_code(p.dev_code, kDevBadLengthCode);
            }
            __syncwarp();
        }
        TreeRange r{};
        const int end = (int)((long long)p.P * (g + 1) / p.groups);
        unsigned at = p.P;                       // the first pair with tiles
        for (int q = (int)((long long)p.P * g / p.groups) + lane; q < end; q += 32) {
            const int n = tree_cost(p, tree_len(p, q), tree_count(p, q / p.Hkv), TS);
            r.n += n;
            if (n > 0) at = min(at, (unsigned)q);
        }
        r.n = __reduce_add_sync(0xffffffffu, r.n);
        r.pair = (int)__reduce_min_sync(0xffffffffu, at);
        if (r.n > 0) {
            r.len = tree_len(p, r.pair);
            r.cnt = tree_count(p, r.pair / p.Hkv);
        }
        r.q = 1;
        return r;
    }
    auto count_of = [&](int q) {
        return p.count == nullptr ? p.T : p.count[p.len_per_pair ? q / p.Hkv : q];
    };
    long long sum = 0;
#pragma unroll 4
    for (int q = q0; q < q1; ++q) {
        int n = p.len != nullptr ? p.len[q] : p.n_valid, c = count_of(q);
        if (check && (n < 0 || n > p.cap || c < 0 || c > p.T)) record_code(p.dev_code, kDevBadLengthCode);
        n = n < 0 ? 0 : (n > p.cap ? p.cap : n);
        c = c < 0 ? 0 : (c > p.T ? p.T : c);
        sum += (long long)tree_cost(p, n, c, TS) * heads;
    }
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    const long long T = __shfl_sync(0xffffffffu, incl, 31);
    TreeRange r;
    if (T <= 0x7fffffff) {                       // (64-bit division is a long subroutine)
        const unsigned c = (unsigned)p.groups, t = (unsigned)T;
        r.q = t / c;
        r.r = (int)(t - (unsigned)r.q * c);
    } else {
        r.q = T / p.groups;
        r.r = (int)(T % p.groups);
    }
    r.t0 = g * r.q + min(g, r.r);
    r.n = (int)(r.q + (g < r.r ? 1 : 0));
    const long long before = incl - sum;
    const bool here = r.n > 0 && before <= r.t0 && r.t0 < incl;
    int q = q0, off = 0, len = 0, cnt = 0;
    if (here) {
        long long t = before;
        int nt = 0;
        for (;; ++q) {
            len = p.len != nullptr ? p.len[q] : p.n_valid;
            len = len < 0 ? 0 : (len > p.cap ? p.cap : len);
            cnt = count_of(q);
            cnt = cnt < 0 ? 0 : (cnt > p.T ? p.T : cnt);
            nt = tree_cost(p, len, cnt, TS);
            const long long end = t + (long long)nt * heads;
            if (r.t0 < end || q == q1 - 1) break;
            t = end;
        }
        off = (int)(r.t0 - t);
        if (heads > 1) {
            const int kh = nt > 0 ? off / nt : 0;
            off -= kh * nt;
            q = q * heads + kh;
        }
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    if (src < 0) r.n = 0;
    r.pair = __shfl_sync(0xffffffffu, q, src & 31);
    r.off = __shfl_sync(0xffffffffu, off, src & 31);
    r.len = __shfl_sync(0xffffffffu, len, src & 31);
    r.cnt = __shfl_sync(0xffffffffu, cnt, src & 31);
    return r;
}

// One pair's part of a block's range.
struct TreeSeg {
    int pair, b, kh;
    int len, cnt;                // cached slots, drafted tokens
    int nt;                      // tiles of the whole pair
    int lo, hi;                  // this part: tiles [lo, hi)
    int rows;                    // valid rows of the block's row tile (may be <= 0)
    bool first;                  // first pair of the range
    __device__ __forceinline__ bool whole() const { return lo == 0 && hi == nt; }
    // slots (or drafted tokens) of tile i, and whether it is the drafted tokens' tile
    __device__ __forceinline__ bool is_draft(const TreeParams &p, int i) const
    {
        return p.kd != nullptr && i == nt - 1;
    }
    __device__ __forceinline__ int valid(const TreeParams &p, int i, int TS) const
    {
        if (is_draft(p, i)) return cnt;
        const int v = len - i * TS;
        return v < 0 ? 0 : (v > TS ? TS : v);
    }
};

// Walks the pairs of a range in order.
struct TreeWalk {
    int pair, b, kh, off, left, len, cnt;
    bool first;
    __device__ __forceinline__ TreeWalk(const TreeParams &p, const TreeRange &r)
        : pair(r.pair), b(r.pair / p.Hkv), kh(r.pair - r.pair / p.Hkv * p.Hkv), off(r.off), left(r.n),
          len(r.len), cnt(r.cnt), first(true)
    {
    }
    __device__ __forceinline__ bool next(const TreeParams &p, int rt, int TS, TreeSeg &s)
    {
        while (left > 0 && pair < p.P) {
            if (!first || len < 0) {             // (the range knows its first pair's)
                len = tree_len(p, pair);
                cnt = tree_count(p, b);
            }
            s.pair = pair;
            s.b = b;
            s.kh = kh;
            s.len = len;
            s.cnt = cnt;
            s.nt = tree_tiles(p, len, cnt, TS);
            const int cost = s.nt > 0 ? min(left, s.nt + kPairEnd - off) : 0;
            s.lo = off;
            s.hi = min(s.nt, off + cost);
            s.rows = min(p.RP, cnt * p.G - rt * p.RP);
            s.first = first;
            ++pair;
            if (++kh == p.Hkv) {
                kh = 0;
                ++b;
            }
            off = 0;
            left -= cost;
            if (s.hi <= s.lo) {                  // (no tiles, or none in this range)
                len = -1;
                continue;
            }
            first = false;
            return true;
        }
        return false;
    }
};

// Where the merge finds a split pair: written by the block that holds its first part.
//   info[g] = {sequence or -1, KV head, last group, drafted tokens * 2 + workspace slot (0 or 1) of
//   the first part}
// (The division that finds the last group is left for the end: in 64 bits it costs some 500 clocks.)
struct TreeNote {
    int b = -1, kh = 0, how = 0;
    long long last = 0;                          // the pair's last tile (its unit)
    __device__ __forceinline__ void see(const TreeRange &r, const TreeSeg &s)
    {
        if (s.lo != 0 || s.hi == s.nt) return;
        b = s.b;
        kh = s.kh;
        how = s.cnt * 2 + (s.first ? 0 : 1);
        last = r.t0 + r.n - s.hi + s.nt - 1;
    }
    __device__ __forceinline__ int4 get(const TreeRange &r) const
    {
        return make_int4(b, kh, b < 0 ? 0 : r.group_of(last), how);
    }
};

__device__ __forceinline__ uint64_t tree_mask_word(const TreeParams &p, int b, int t, int cnt)
{
    const uint64_t live = cnt >= 64 ? ~0ull : ((1ull << cnt) - 1ull);
    const uint64_t w = p.mask != nullptr ? p.mask[(size_t)b * p.T + t]
                                         : (t >= 63 ? ~0ull : ((2ull << t) - 1ull));
    return w & live;
}

}  // namespace kvc

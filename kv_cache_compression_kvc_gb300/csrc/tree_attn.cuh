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
// The lengths live on the device, so every block finds its own range: the block scans the
// pairs' tile counts (one read of the lengths), which makes the ranges equal however ragged the
// batch is, without a host round trip.
//
// A pair that lies inside one range is finished by its block.  A pair that crosses ranges leaves
// one partial state (max, sum, unnormalised output) per range: workspace slot 2*block for the
// first pair of a block's range, 2*block + 1 for its last; tree_merge_kernel, launched next,
// joins them in range order (no atomics: results do not depend on timing).
#pragma once

#include "common.cuh"
#include "internal.h"

namespace kvc {

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

struct TreeRange {
    int pair, off;               // first pair of the range and the tile inside it
    int n;                       // tiles in the range
    long long t0, T;             // the range's first tile, all tiles
    int Ce;                      // ranges in use: min(groups, T)
};

// Called by all NT threads of a block; scratch: NT / 32 + 4 long longs of shared memory.
template <int NT>
__device__ __forceinline__ TreeRange tree_range(const TreeParams &p, int g, int TS,
                                                long long *scratch)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (p.P + NT - 1) / NT;
    const int q0 = threadIdx.x * per, q1 = min(p.P, q0 + per);
    const bool check = g == 0 && blockIdx.x == 0;
    long long sum = 0;
    for (int q = q0; q < q1; ++q) {
        const int b = q / p.Hkv;
        sum += tree_tiles(p, tree_len(p, q), tree_count(p, b), TS);
        if (check) {
            if (p.len != nullptr) {
                const int n = p.len[p.len_per_pair ? q : b];
                if (n < 0 || n > p.cap) record_code(p.dev_code, kDevBadLengthCode);
            }
            if (p.count != nullptr && (p.count[b] < 0 || p.count[b] > p.T))
                record_code(p.dev_code, kDevBadLengthCode);
        }
    }
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    long long before = incl - sum, T = 0;
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += scratch[w];
        T += scratch[w];
    }
    TreeRange r;
    r.T = T;
    r.Ce = T < p.groups ? (int)T : p.groups;
    r.t0 = g < r.Ce ? (long long)g * T / r.Ce : 0;
    const long long t1 = g < r.Ce ? (long long)(g + 1) * T / r.Ce : 0;
    r.n = (int)(t1 - r.t0);
    long long *res = scratch + NT / 32;
    if (r.n > 0 && before <= r.t0 && r.t0 < before + sum) {
        long long t = before;
        for (int q = q0; q < q1; ++q) {
            const int nt = tree_tiles(p, tree_len(p, q), tree_count(p, q / p.Hkv), TS);
            if (r.t0 < t + nt) {
                res[0] = q;
                res[1] = r.t0 - t;
                break;
            }
            t += nt;
        }
    }
    __syncthreads();
    r.pair = r.n > 0 ? (int)res[0] : 0;
    r.off = r.n > 0 ? (int)res[1] : 0;
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
    int pair, off, left;
    bool first;
    __device__ __forceinline__ explicit TreeWalk(const TreeRange &r)
        : pair(r.pair), off(r.off), left(r.n), first(true)
    {
    }
    __device__ __forceinline__ bool next(const TreeParams &p, int rt, int TS, TreeSeg &s)
    {
        while (left > 0 && pair < p.P) {
            s.pair = pair;
            s.b = pair / p.Hkv;
            s.kh = pair - s.b * p.Hkv;
            s.len = tree_len(p, pair);
            s.cnt = tree_count(p, s.b);
            s.nt = tree_tiles(p, s.len, s.cnt, TS);
            if (s.nt == 0) {
                ++pair;
                off = 0;
                continue;
            }
            s.lo = off;
            s.hi = min(s.nt, off + left);
            left -= s.hi - s.lo;
            s.rows = min(p.RP, s.cnt * p.G - rt * p.RP);
            s.first = first;
            first = false;
            ++pair;
            off = 0;
            return true;
        }
        return false;
    }
};

// Where the merge finds a split pair: written by the block that holds its first part.
//   info[g] = {pair or -1, last group, workspace slot (0 or 1) of the first part, 0}
__device__ __forceinline__ void tree_note_split(const TreeParams &p, const TreeRange &r, int g,
                                                const TreeSeg &s, int4 &note)
{
    if (s.lo != 0 || s.hi == s.nt) return;
    const long long last = r.t0 + r.n - s.hi + s.nt - 1;     // the pair's last tile
    note = make_int4(s.pair, (int)(((last + 1) * r.Ce - 1) / r.T), s.first ? 0 : 1, 0);
}

__device__ __forceinline__ uint64_t tree_mask_word(const TreeParams &p, int b, int t, int cnt)
{
    const uint64_t live = cnt >= 64 ? ~0ull : ((1ull << cnt) - 1ull);
    const uint64_t w = p.mask != nullptr ? p.mask[(size_t)b * p.T + t]
                                         : (t >= 63 ? ~0ull : ((2ull << t) - 1ull));
    return w & live;
}

}  // namespace kvc

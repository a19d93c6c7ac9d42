// pages.cu -- pages held by several sequences, and pools made dense.
//
// Full pages are never written again, so sequences may share them: shares[x] counts the sequences
// that hold page x beyond the first (0 for a page that one sequence holds, and for a free one).  Partly
// filled pages belong to one sequence each; that is all that appends need to know, so those that pop
// pages and write rows work on forked sequences as they are.
//
// pages_reorder_kernel: sequence b becomes a copy of what sequence parent[b] was, or is freed.  A
// page that s sequences held is held afterwards by the sum of their children: every table entry adds
// (children - 1) to its page's count, and a page that ends at -1 is free.  All entries are counted, those
// of sequences that stay too: a page listed more often than its count says would be freed under a holder
// that goes on.  A partly filled page stays with the sequence itself or its first child; the other
// children get a page of their own, copied by pages_copy_kernel.  Free pages go on the stack in ascending
// order, copies take theirs from its top in sequence order: results do not depend on timing.
//
// pages_compact_kernel: the k-th live page beyond the number of live pages moves to the k-th free page
// below it; tables, counts and the stack follow.  No page is both read and written.
//
// The tables' kernels are a cluster of 8 blocks with a few barriers (a launch per step would cost more than the
// steps); what blocks tell each other goes through the workspace.  Bound by latency: every step is a trip or two
// to memory.  Reorders whose tables and counts fit the shared memory of one block need two trips and no barrier
// of the cluster (pages_reorder_one_kernel: 128 sequences of 26 pages with 20 MB of copies 17.2 -> 14.1 us).
// For compaction each block keeps the free pages as bits in shared memory and works out by itself where
// everything goes, which left one barrier of the cluster of six (16384 pages, tables and copies: 111 -> 105 us).
// The copies are bound by HBM: a page's keys or values of a head are one run, which a warp copies with 128
// bytes a lane in flight and the next copy's ids read ahead: 515 MB of 4 KB runs, read and written, in 77 us,
// 6.7 TB/s (a block a page with 64 bytes a thread: 84 us).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace kvc {

namespace {

constexpr int kCl = 8;                       // blocks of the cluster
constexpr int kThreads = 1024;
constexpr int kAll = kCl * kThreads;
constexpr int kCopyThreads_ = 256, kCopyBlocks = 8;      // of the copies: threads of a block, blocks per SM
// Copies of so many bytes at most are made by the tables' kernel itself.  Reorders, by it and by a second kernel:
// 64 KB 5.3 and 5.7 us, 256 KB 11.6 and 12.3, 512 KB 8.9 and 7.9.  Compaction, 256 KB: 10.9 and 9.8 on the
// device, but a call from Python, which the host bounds, 24 and 27.
constexpr long long kFusedBytes = 1 << 18;
// Reorders that one block takes: bytes of shared memory, runs of 32 table entries.  Device times by one block and by
// the cluster: 4 runs 5.8 and 10.0 us, 128 runs 14.1 and 17.2, 256 runs 13.1 and 14.5, 512 runs 21.7 to 22.0 and
// 17.4, 1024 runs 33.0 and 21.0; 4 runs and a pool of 32000 pages 10.3 and 12.5.
constexpr int kOneBytes = 200 * 1024, kOneRuns = 256;
constexpr int kBadIndex = 3, kBadLength = 5, kBadBlock = 9, kPoolEmpty = 10, kPoolOverflow = 11, kSharedPage = 12;

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Also orders the cluster's global memory accesses.
__device__ __forceinline__ void cluster_barrier()
{
    __threadfence();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Threads before this one (in order) whose flag is set, and how many are set in the block.
__device__ __forceinline__ int block_rank(bool flag, int *s_warp, int *all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t votes = __ballot_sync(0xffffffffu, flag);
    __syncthreads();                         // (s_warp is free)
    if (lane == 0) s_warp[warp] = __popc(votes);
    __syncthreads();
    int x = s_warp[lane];
    const int own = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    *all = __shfl_sync(0xffffffffu, x, 31);
    return __shfl_sync(0xffffffffu, x - own, warp) + __popc(votes & ((1u << lane) - 1u));
}

// Calls f(b, i) for the entries i < n(b) of every sequence's table, 32 of one sequence a warp.
template <int CL, typename N, typename F>
__device__ __forceinline__ void each_entry(int B, int max_blocks, int rank, N n, F f)
{
    const int lane = threadIdx.x & 31, first = rank * (kThreads / 32) + (threadIdx.x >> 5);
    const int per = (max_blocks + 31) / 32;
    int b = first / per, c = first - b * per;
    constexpr int kStride = CL * kThreads / 32;
    const int db = kStride / per, dc = kStride - db * per;
    while (b < B) {
        const int i = c * 32 + lane;
        if (i < n(b)) f(b, i);
        b += db;
        c += dc;
        if (c >= per) {
            c -= per;
            ++b;
        }
    }
}

// Task (copy, head, keys or values), a warp each: the rows of a page of a head are one run, with the page's
// scale; head 0's keys take the tokens' positions along.  Warps first, first + stride, ... take them in
// turn and read the next one's copy ahead.
__device__ __forceinline__ void copy_pages(const PagesParams &p, int n_copies, long long first, long long stride)
{
    const int lane = threadIdx.x & 31;
    const unsigned per = 2u * (unsigned)p.H;
    const long long tasks = (long long)n_copies * per;
    if (first >= tasks) return;
    const size_t page_bytes = (size_t)p.bs * p.row_bytes;
    int4 what = __ldcg(p.ws_copies + (unsigned)(first / per));
    for (long long j = first; j < tasks; j += stride) {
        const int rest = (int)(j - j / per * per), h = rest >> 1;
        const int4 now = what;
        if (j + stride < tasks) what = __ldcg(p.ws_copies + (unsigned)((j + stride) / per));
        const size_t from = (size_t)h * p.n_pool + now.x, to = (size_t)h * p.n_pool + now.y;
        char *pool = rest & 1 ? p.v : p.k;
        const char *src = pool + from * page_bytes;
        char *dst = pool + to * page_bytes;
        const int n = now.z * p.row_bytes;
        constexpr int U = 8;
        for (int i0 = lane * 16; i0 < n; i0 += 512 * U) {
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u * 512 < n) x[u] = ld_stream_16(src + i0 + u * 512);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u * 512 < n) *reinterpret_cast<uint4 *>(dst + i0 + u * 512) = x[u];
        }
        float *scale = rest & 1 ? p.vs : p.ks;
        if (lane == 0 && scale != nullptr) scale[to] = scale[from];
        if (rest == 0 && p.pos != nullptr)
            for (int i = lane; i < now.z; i += 32) p.pos[(size_t)now.y * p.bs + i] = p.pos[(size_t)now.x * p.bs + i];
    }
}

__global__ void __cluster_dims__(kCl, 1, 1) __launch_bounds__(kThreads) pages_reorder_kernel(const PagesParams p)
{
    extern __shared__ int s_seq[];           // per sequence: children, keeper, parent, blocks, length, copy
    __shared__ int s_warp[32];
    int *s_kids = s_seq, *s_keep = s_kids + p.B, *s_par = s_keep + p.B, *s_nb = s_par + p.B, *s_len = s_nb + p.B,
        *s_copy = s_len + p.B;
    const int tid = threadIdx.x, rank = (int)cluster_rank();
    pdl_trigger();
    pdl_wait();
    // ---- the sequences, in every block alike ----
    int code = 0;
    const int top = *p.free_top;
    if (top < 0 || top > p.free_cap) code = kPoolEmpty;
    if (rank == 0 && tid == 0) {
        p.ws_n[0] = 0;                       // copies
        p.ws_n[1] = 0;                       // what is wrong
    }
    // of every page: how often the tables list it, and how many holders more (or less) it is to have
    int32_t *lists = reinterpret_cast<int32_t *>(p.ws_copies), *more = lists + p.n_pool;
    const int x0 = (int)((long long)p.n_pool * rank / kCl), x1 = (int)((long long)p.n_pool * (rank + 1) / kCl);
    for (int x = x0 + tid; x < x1; x += kThreads) lists[x] = more[x] = 0;
    for (int b = tid; b < p.B; b += kThreads) {
        const int par = p.parent[b], len = p.len[b], nb = p.n_blocks[b];
        if (par < -1 || par >= p.B) code = kBadIndex;
        if (len < 0 || len > p.max_blocks * p.bs || nb != (len + p.bs - 1) / p.bs) code = kBadLength;
        s_kids[b] = 0;
        s_keep[b] = 0x7fffffff;
        s_par[b] = par;
        s_nb[b] = nb;
        s_len[b] = len;
    }
    const bool bad = __syncthreads_or(code != 0);
    cluster_barrier();                       // (ws_n and the counts are there; no block has left)
    if (bad) {
        if (rank == 0 && code != 0) record_code(p.dev_code, code);
        return;
    }
    for (int b = tid; b < p.B; b += kThreads) {
        const int par = s_par[b];
        if (par >= 0) {
            atomicAdd(&s_kids[par], 1);
            atomicMin(&s_keep[par], b);
        }
    }
    __syncthreads();
    for (int b = tid; b < p.B; b += kThreads)
        if (s_par[b] == b) s_keep[b] = b;
    __syncthreads();
    int n_copies = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + tid;
        bool own = false;
        if (b < p.B) {
            const int par = s_par[b];
            own = par >= 0 && s_len[par] % p.bs != 0 && s_keep[par] != b;
        }
        int all;
        const int r = block_rank(own, s_warp, &all);
        if (b < p.B) s_copy[b] = own ? n_copies + r : -1;
        n_copies += all;
    }
    __syncthreads();
    auto partial = [&](int b, int i) { return s_len[b] % p.bs != 0 && i == s_nb[b] - 1; };
    // ---- the tables' ids, and what the call makes of their holders ----
    each_entry<kCl>(p.B, p.max_blocks, rank, [&](int b) { return s_nb[b]; }, [&](int b, int i) {
        const int id = p.table[(size_t)b * p.max_blocks + i], kids = s_kids[b];
        if (id < 0 || id >= p.n_pool) {
            atomicCAS(&p.ws_n[1], 0, kBadBlock);
            return;
        }
        atomicAdd(&lists[id], 1);
        if (partial(b, i)) {
            if (p.shares[id] != 0 && !(kids == 1 && s_par[b] == b)) atomicCAS(&p.ws_n[1], 0, kSharedPage);
            if (kids == 0) atomicAdd(&more[id], -1);
        } else if (kids != 1) {
            atomicAdd(&more[id], kids - 1);
        }
    });
    cluster_barrier();
    int gone = 0;
    for (int x = x0 + tid; x < x1; x += kThreads) {
        const int s = p.shares[x];
        gone += s + __ldcg(&more[x]) < 0 ? 1 : 0;
        if (s < 0 || __ldcg(&lists[x]) - 1 > s) atomicCAS(&p.ws_n[1], 0, kBadBlock);   // listed more often than counted
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) gone += __shfl_xor_sync(0xffffffffu, gone, o);
    __syncthreads();
    if ((tid & 31) == 0) s_warp[tid >> 5] = gone;
    __syncthreads();
    if (tid < 32) {
        int x = s_warp[tid];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (tid == 0) p.ws_n[2 + rank] = x;
    }
    cluster_barrier();
    int before = 0, n_gone = 0;
#pragma unroll
    for (int r = 0; r < kCl; ++r) {
        const int x = __ldcg(&p.ws_n[2 + r]);
        if (r < rank) before += x;
        n_gone += x;
    }
    const int new_top = top + n_gone - n_copies;
    code = __ldcg(&p.ws_n[1]);
    if (code == 0 && new_top < 0) code = kPoolEmpty;
    if (code == 0 && new_top > p.free_cap) code = kPoolOverflow;
    if (code == 0)
        for (int i = max(new_top, 0) + tid; i < top; i += kThreads) {
            const int id = p.free_ids[i];
            if (id < 0 || id >= p.n_pool) code = kBadBlock;
        }
    if (__syncthreads_or(code != 0)) {       // (the same in every block) nothing has changed
        if (rank == 0 && code != 0) record_code(p.dev_code, code);
        return;
    }
    // ---- freed pages in ascending order; the tables as the children will have them ----
    for (int c = x0; c < x1; c += kThreads) {
        const int x = c + tid;
        const int s = x < x1 ? p.shares[x] : 0, add = x < x1 ? __ldcg(&more[x]) : 0;
        const bool free_now = s + add < 0;
        int all;
        const int r = before + block_rank(free_now, s_warp, &all);
        if (add != 0) p.shares[x] = max(s + add, 0);
        if (free_now) {
            p.ws_ids[r] = x;
            if (top + r < new_top) p.free_ids[top + r] = x;
        }
        before += all;
    }
    auto moved = [&](int b) { return s_par[b] < 0 || s_par[b] == b ? 0 : s_nb[s_par[b]]; };
    each_entry<kCl>(p.B, p.max_blocks, rank, moved, [&](int b, int i) {
        const size_t from = (size_t)s_par[b] * p.max_blocks + i, to = (size_t)b * p.max_blocks + i;
        p.ws_table[to] = p.table[from];
        p.ws_score[to] = p.score[from];
    });
    cluster_barrier();
    each_entry<kCl>(p.B, p.max_blocks, rank, moved, [&](int b, int i) {
        const size_t at = (size_t)b * p.max_blocks + i;
        int id = __ldcg(&p.ws_table[at]);
        const int copy = s_copy[b];
        if (copy >= 0 && i == s_nb[s_par[b]] - 1) {
            const int place = top + n_gone - 1 - copy;
            const int to = place >= top ? __ldcg(&p.ws_ids[place - top]) : p.free_ids[place];
            p.ws_copies[copy] = make_int4(id, to, s_len[s_par[b]] % p.bs, 0);
            id = to;
        }
        p.table[at] = id;
        p.score[at] = __ldcg(&p.ws_score[at]);
    });
    if (rank == 0) {
        for (int b = tid; b < p.B; b += kThreads) {
            const int par = s_par[b];
            if (par == b) continue;
            p.n_blocks[b] = par < 0 ? 0 : s_nb[par];
            p.len[b] = par < 0 ? 0 : s_len[par];
        }
        if (tid == 0) {
            p.ws_n[0] = n_copies;
            *p.free_top = new_top;
        }
    }
    if (p.fused) {
        cluster_barrier();
        copy_pages(p, n_copies, rank * (kThreads / 32) + (tid >> 5), kAll / 32);
    }
}

// The same by one block that holds everything in shared memory: tables, scores, counts and sequences come
// in one trip to memory, the rest is steps between barriers of the block, and results go out once.
__host__ __device__ inline size_t one_block_bytes(const PagesParams &p)
{
    return ((size_t)p.B * (7 + 2 * (size_t)p.max_blocks) + (size_t)p.n_pool) * 4 + ((size_t)p.n_pool + 1) / 2 * 4;
}
__device__ __forceinline__ void take_4(void *dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}

__global__ void __launch_bounds__(kThreads) pages_reorder_one_kernel(const PagesParams p)
{
    extern __shared__ int s_seq[];           // per sequence as above and an id of the stack; tables, scores, counts, freed
    __shared__ int s_warp[32];
    int *s_kids = s_seq, *s_keep = s_kids + p.B, *s_par = s_keep + p.B, *s_nb = s_par + p.B, *s_len = s_nb + p.B,
        *s_copy = s_len + p.B, *s_stack = s_copy + p.B, *s_table = s_stack + p.B;
    const int entries = p.B * p.max_blocks;
    int *s_score = s_table + entries, *s_count = s_score + entries;
    uint16_t *s_freed = reinterpret_cast<uint16_t *>(s_count + p.n_pool);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    pdl_wait();
    if (tid == 0) p.ws_n[0] = 0;             // copies
    const int top = *p.free_top;
    for (int j = tid; j < entries; j += kThreads) {
        take_4(s_table + j, p.table + j);
        take_4(s_score + j, p.score + j);
    }
    for (int x = tid; x < p.n_pool; x += kThreads) take_4(s_count + x, p.shares + x);
    int code = top < 0 || top > p.free_cap ? kPoolEmpty : 0;
    for (int b = tid; b < p.B; b += kThreads) {
        const int par = p.parent[b], len = p.len[b], nb = p.n_blocks[b];
        if (par < -1 || par >= p.B) code = kBadIndex;
        if (len < 0 || len > p.max_blocks * p.bs || nb != (len + p.bs - 1) / p.bs) code = kBadLength;
        s_kids[b] = 0;
        s_keep[b] = 0x7fffffff;
        s_par[b] = par;
        s_nb[b] = nb;
        s_len[b] = len;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    for (int x = tid; x < p.n_pool; x += kThreads)             // (what this thread copied)
        if (s_count[x] < 0) code = kBadBlock;
    if (__syncthreads_or(code != 0)) {
        if (code != 0) record_code(p.dev_code, code);
        return;
    }
    for (int b = tid; b < p.B; b += kThreads) {
        const int par = s_par[b];
        if (par >= 0) {
            atomicAdd(&s_kids[par], 1);
            atomicMin(&s_keep[par], b);
        }
    }
    __syncthreads();
    int n_copies = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + tid;
        bool own = false;
        if (b < p.B) {
            const int par = s_par[b];
            own = par >= 0 && par != b && s_len[par] % p.bs != 0 && (s_par[par] == par || s_keep[par] != b);
        }
        int all;
        const int r = block_rank(own, s_warp, &all);
        if (b < p.B) s_copy[b] = own ? n_copies + r : -1;
        n_copies += all;
    }
    // ids that copies may need, from the top of the stack
    for (int e = tid; e < min(n_copies, top); e += kThreads) take_4(s_stack + e, p.free_ids + top - 1 - e);
    auto partial = [&](int b, int i) { return s_len[b] % p.bs != 0 && i == s_nb[b] - 1; };
    auto stays = [&](int b) { return s_kids[b] == 1 && s_par[b] == b; };
    // ---- partly filled pages of the sequences that change have one holder ----
    for (int b = tid; b < p.B; b += kThreads)
        if (!stays(b) && s_len[b] % p.bs != 0) {
            const int id = s_table[b * p.max_blocks + s_nb[b] - 1];
            if (id >= 0 && id < p.n_pool && s_count[id] != 0) code = kSharedPage;
        }
    __syncthreads();
    // ---- holders of every page: no more listings than counted ones, then what the call makes of them ----
    each_entry<1>(p.B, p.max_blocks, 0, [&](int b) { return s_nb[b]; }, [&](int b, int i) {
        const int id = s_table[b * p.max_blocks + i];
        if (id < 0 || id >= p.n_pool) code = kBadBlock;
        else if (atomicSub(&s_count[id], 1) < 0) code = kBadBlock;
    });
    if (__syncthreads_or(code != 0)) {
        if (code != 0) record_code(p.dev_code, code);
        return;
    }
    each_entry<1>(p.B, p.max_blocks, 0, [&](int b) { return s_kids[b] > 0 ? s_nb[b] : 0; }, [&](int b, int i) {
        atomicAdd(&s_count[s_table[b * p.max_blocks + i]], partial(b, i) ? 1 : s_kids[b]);
    });
    __syncthreads();
    // a warp looks at `per` runs of 32 pages
    const int per = (p.n_pool + kThreads - 1) / kThreads, x0 = warp * per * 32 + lane;
    int gone = 0;
    for (int r = 0, x = x0; r < per; ++r, x += 32) {
        const int s = x < p.n_pool ? s_count[x] : 0;
        gone += __popc(__ballot_sync(0xffffffffu, s < 0));
    }
    if (lane == 0) s_warp[warp] = gone;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    int x = s_warp[lane];
    const int own = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    const int n_gone = __shfl_sync(0xffffffffu, x, 31);
    int before = __shfl_sync(0xffffffffu, x - own, warp);
    const int new_top = top + n_gone - n_copies;
    if (code == 0 && new_top < 0) code = kPoolEmpty;
    if (code == 0 && new_top > p.free_cap) code = kPoolOverflow;
    for (int e = tid; e < min(n_copies - n_gone, top); e += kThreads)
        if (code == 0 && (s_stack[e] < 0 || s_stack[e] >= p.n_pool)) code = kBadBlock;
    if (__syncthreads_or(code != 0)) {       // nothing has changed
        if (code != 0) record_code(p.dev_code, code);
        return;
    }
    // ---- freed pages in ascending order; the tables as the children have them ----
    for (int r = 0, x = x0; r < per; ++r, x += 32) {
        const int s = x < p.n_pool ? s_count[x] : 0;
        const uint32_t votes = __ballot_sync(0xffffffffu, s < 0);
        if (s < 0) {
            const int k = before + __popc(votes & ((1u << lane) - 1u));
            s_freed[k] = (uint16_t)x;
            if (top + k < new_top) p.free_ids[top + k] = x;
        }
        if (x < p.n_pool) p.shares[x] = max(s, 0);
        before += __popc(votes);
    }
    __syncthreads();
    each_entry<1>(p.B, p.max_blocks, 0, [&](int b) { return s_par[b] < 0 || s_par[b] == b ? 0 : s_nb[s_par[b]]; },
                  [&](int b, int i) {
        const int par = s_par[b], from = par * p.max_blocks + i, copy = s_copy[b];
        int id = s_table[from];
        if (copy >= 0 && i == s_nb[par] - 1) {
            const int place = n_gone - 1 - copy;
            const int to = place >= 0 ? s_freed[place] : s_stack[-1 - place];
            p.ws_copies[copy] = make_int4(id, to, s_len[par] % p.bs, 0);
            id = to;
        }
        p.table[b * p.max_blocks + i] = id;
        p.score[b * p.max_blocks + i] = __int_as_float(s_score[from]);
    });
    for (int b = tid; b < p.B; b += kThreads) {
        const int par = s_par[b];
        if (par == b) continue;
        p.n_blocks[b] = par < 0 ? 0 : s_nb[par];
        p.len[b] = par < 0 ? 0 : s_len[par];
    }
    if (tid == 0) {
        p.ws_n[0] = n_copies;
        *p.free_top = new_top;
    }
    if (p.fused) {
        __syncthreads();
        copy_pages(p, n_copies, warp, kThreads / 32);
    }
}

// Free pages as bits of shared memory, which every block of the cluster sets for itself from the whole
// stack, and how many of them lie below a page: thread t keeps the count before its `per` words in s_before.
struct FreeBits {
    const uint32_t *bits;
    const int *before;
    int per, n_live;
    __device__ __forceinline__ bool get(int x) const { return bits[x >> 5] >> (x & 31) & 1u; }
    __device__ __forceinline__ int below(int x) const
    {
        const int word = x >> 5, t = word / per;
        int n = before[t] + __popc(bits[word] & ((1u << (x & 31)) - 1u));
        for (int w = t * per; w < word; ++w) n += __popc(bits[w]);
        return n;
    }
    // the number of a live page with an id >= n_live among those
    __device__ __forceinline__ int rank_high(int x, int holes) const { return x - n_live - (below(x) - holes); }
};

__global__ void __cluster_dims__(kCl, 1, 1) __launch_bounds__(kThreads) pages_compact_kernel(const PagesParams p)
{
    extern __shared__ int s_seq[];           // the bits
    __shared__ int s_warp[32], s_before[kThreads], s_holes;
    const int tid = threadIdx.x, lane = tid & 31, rank = (int)cluster_rank(), all_tid = rank * kThreads + tid;
    uint32_t *bits = reinterpret_cast<uint32_t *>(s_seq);
    const int words = (p.n_pool + 31) / 32, per = (words + kThreads - 1) / kThreads;
    for (int w = tid; w < words; w += kThreads) bits[w] = 0u;
    pdl_trigger();
    pdl_wait();
    const int top = *p.free_top;
    int code = top < 0 || top > p.free_cap || top > p.n_pool ? kPoolEmpty : 0;
    const int n_live = p.n_pool - top;
    __syncthreads();
    if (code == 0) {
        bool bad = false;
        constexpr int U = 8;                 // ids on their way at once
        for (int i0 = tid; i0 < top; i0 += kThreads * U) {
            int id[U];
#pragma unroll
            for (int u = 0; u < U; ++u) id[u] = i0 + u * kThreads < top ? p.free_ids[i0 + u * kThreads] : 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i0 + u * kThreads >= top) break;
                const bool in = id[u] >= 0 && id[u] < p.n_pool;
                bad |= !in || (atomicOr(&bits[in ? id[u] >> 5 : 0], in ? 1u << (id[u] & 31) : 0u) >> (id[u] & 31) & 1u);
            }
        }
        if (__syncthreads_or(bad)) code = kBadBlock;
    }
    // ---- the tables, each block its part ----
    auto entries = [&](int b) {
        const int n = p.n_blocks[b];
        return n < 0 || n > p.max_blocks ? 0 : n;
    };
    if (code == 0) {
        int c = 0;
        each_entry<kCl>(p.B, p.max_blocks, rank, entries, [&](int b, int i) {
            const int id = p.table[(size_t)b * p.max_blocks + i];
            if (id < 0 || id >= p.n_pool || (bits[id >> 5] >> (id & 31) & 1u)) c = max(c, kBadBlock);
        });
        for (int b = all_tid; b < p.B; b += kAll) {
            const int n = p.n_blocks[b];
            if (n < 0 || n > p.max_blocks) c = max(c, kBadLength);
        }
        c = __reduce_max_sync(0xffffffffu, c);
        __syncthreads();                     // (s_warp is free)
        if (lane == 0) s_warp[tid >> 5] = c;
        __syncthreads();
        code = __reduce_max_sync(0xffffffffu, s_warp[lane]);
        __syncthreads();
    }
    if (tid == 0) p.ws_n[2 + rank] = code;
    // ---- free pages before every thread's words, and below the number of live pages: the holes ----
    int own = 0;
    for (int w = tid * per; w < min(words, (tid + 1) * per); ++w) own += __popc(bits[w]);
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[tid >> 5] = incl;
    __syncthreads();
    int warps = s_warp[lane];
    const int mine = warps;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, warps, o);
        if (lane >= o) warps += y;
    }
    const int first = __shfl_sync(0xffffffffu, warps - mine, tid >> 5) + incl - own;
    s_before[tid] = first;
    if (tid == 0) s_holes = top;             // (with no page from n_live on: none is free either)
    __syncthreads();
    const FreeBits f{bits, s_before, per, n_live};
    if (tid == 0 && code == 0 && n_live < p.n_pool) s_holes = f.below(n_live);
    // the holes in order, each block the words of its threads' share
    if (code == 0 && tid % kCl == rank) {
        int r = first;
        for (int w = tid * per; w < min(words, (tid + 1) * per); ++w)
            for (uint32_t m = bits[w]; m != 0; m &= m - 1) {
                const int x = w * 32 + __ffs(m) - 1;
                if (x < n_live) p.ws_ids[r] = x;
                ++r;
            }
    }
    cluster_barrier();
#pragma unroll
    for (int r = 0; r < kCl; ++r) code = max(code, __ldcg(&p.ws_n[2 + r]));
    const int holes = s_holes;
    if (all_tid == 0) p.ws_n[0] = code == 0 ? holes : 0;       // moves
    if (code != 0) {                         // nothing has changed
        if (all_tid == 0) record_code(p.dev_code, code);
        return;
    }
    for (int x = all_tid; x < p.n_pool; x += kAll) {
        const bool free_page = f.get(x);
        int to = free_page ? -1 : x;
        if (!free_page && x >= n_live) {
            const int k = f.rank_high(x, holes);
            to = __ldcg(&p.ws_ids[k]);
            p.ws_copies[k] = make_int4(x, to, p.bs, 0);
            if (p.shares != nullptr) {
                p.shares[to] = p.shares[x];
                p.shares[x] = 0;
            }
        }
        p.remap[x] = to;
    }
    // the stack hands out the lowest free page first
    for (int i = all_tid; i < top; i += kAll) p.free_ids[i] = p.n_pool - 1 - i;
    each_entry<kCl>(p.B, p.max_blocks, rank, entries, [&](int b, int i) {
        int32_t *e = p.table + (size_t)b * p.max_blocks + i;
        const int x = *e;
        if (x >= n_live) *e = __ldcg(&p.ws_ids[f.rank_high(x, holes)]);
    });
    if (p.fused) {
        cluster_barrier();
        copy_pages(p, holes, rank * (kThreads / 32) + (tid >> 5), kAll / 32);
    }
}

__global__ void __launch_bounds__(kCopyThreads_) pages_copy_kernel(const PagesParams p)
{
    pdl_trigger();
    pdl_wait();
    constexpr int kWarps = kCopyThreads_ / 32;
    copy_pages(p, *p.ws_n, (long long)blockIdx.x * kWarps + (threadIdx.x >> 5), (long long)gridDim.x * kWarps);
}

// `copies`: the most that there can be.
cudaError_t launch_copies(const PagesParams &p, long long copies, int n_sm, cudaStream_t stream)
{
    const long long most = (long long)n_sm * kCopyBlocks, need = (copies * p.H * 2 + kCopyThreads_ / 32 - 1) / (kCopyThreads_ / 32);
    const long long blocks = std::max(1LL, std::min(need, most));
    return launch_pdl(pages_copy_kernel, dim3((unsigned)blocks), dim3(kCopyThreads_), 0, stream, p);
}
bool copies_fit(const PagesParams &p, long long copies)
{
    return copies * p.H * p.bs * p.row_bytes * 2 <= kFusedBytes;
}

cudaError_t configure(const void *kernel, int bytes, bool *configured)
{
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || configured[dev]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) configured[dev] = true;
    return e;
}

}  // namespace

cudaError_t launch_pages_reorder(PagesParams p, int n_sm, cudaStream_t stream)
{
    static bool configured[64] = {}, configured_one[64] = {};
    const bool one = one_block_bytes(p) <= (size_t)kOneBytes && (long long)p.B * ((p.max_blocks + 31) / 32) <= kOneRuns;
    auto kernel = one ? pages_reorder_one_kernel : pages_reorder_kernel;
    cudaError_t e = one ? configure(reinterpret_cast<const void *>(kernel), kOneBytes, configured_one)
                        : configure(reinterpret_cast<const void *>(kernel), kPagesMaxBatch * 6 * (int)sizeof(int), configured);
    if (e != cudaSuccess) return e;
    p.fused = copies_fit(p, p.B);
    e = launch_pdl(kernel, dim3(one ? 1 : kCl), dim3(kThreads), one ? one_block_bytes(p) : (size_t)p.B * 6 * sizeof(int),
                   stream, p);
    if (e != cudaSuccess || p.fused) return e;
    return launch_copies(p, p.B, n_sm, stream);
}

cudaError_t launch_pages_compact(PagesParams p, int n_sm, cudaStream_t stream)
{
    static bool configured[64] = {};
    cudaError_t e = configure(reinterpret_cast<const void *>(pages_compact_kernel), kPagesMaxPool / 8, configured);
    if (e != cudaSuccess) return e;
    p.fused = copies_fit(p, p.n_pool / 2);
    e = launch_pdl(pages_compact_kernel, dim3(kCl), dim3(kThreads), (size_t)((p.n_pool + 31) / 32) * 4, stream, p);
    if (e != cudaSuccess || p.fused) return e;
    return launch_copies(p, p.n_pool / 2, n_sm, stream);
}

}  // namespace kvc

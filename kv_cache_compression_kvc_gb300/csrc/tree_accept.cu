// tree_accept.cu -- appending the accepted path of a draft tree to a cache.
//
// A gather of at most 64 rows per (sequence, head) from the drafted rows to consecutive tail
// slots, bit exact, in 16-byte vectors.  Bound by latency for small batches and by HBM for large
// ones (each row read once, written once): one block per (sequence, head), every thread with
// four independent copies in flight.
//
// Paged caches first need blocks.  tree_accept_pages_kernel, one block for the whole batch, checks
// every sequence (its path, its lengths, its partly filled page), numbers the blocks they need in
// sequence order (a block-wide scan) and takes them from the top of the free stack, so that ids do
// not depend on timing; the copy kernel follows.
#include "common.cuh"
#include "internal.h"

namespace kvc {

namespace {

constexpr int kCopyThreads = 128;
constexpr int kPageThreads = 1024;
constexpr int kDevTailFull = 1;
constexpr int kDevBadIndex = 3;
constexpr int kDevBadLen = 5;
constexpr int kDevBadBlk = 9;
constexpr int kDevPoolEmpty_ = 10;

// Accepted tokens of sequence b if its path is sound, else -1 and the code to record.
__device__ __forceinline__ int path_tokens(const AcceptParams &p, int b, int lane, int lanes,
                                           int *code)
{
    const int n = p.n_accept[b];
    if (n < 0 || n > p.T) {
        *code = kDevBadLen;
        return -1;
    }
    int cnt = p.count != nullptr ? p.count[b] : p.T;
    if (cnt < 0 || cnt > p.T) {              // recorded and clamped, as the attention does
        if (lane == 0) record_code(p.dev_code, kDevBadLen);
        cnt = cnt < 0 ? 0 : p.T;
    }
    bool bad = false;
    for (int i = lane; i < n; i += lanes) {
        const int t = p.path[(size_t)b * p.T + i];
        bad |= t < 0 || t >= cnt;
    }
    if (bad) {
        *code = kDevBadIndex;
        return -1;
    }
    return n;
}

// Copies rows i < n: drafted token path[i] of (b, h) to dst(i).  vpr: 16-byte vectors per row.
template <typename Dst>
__device__ __forceinline__ void copy_rows(const AcceptParams &p, int b, int h, int n, Dst dst)
{
    const int vpr = p.row_bytes / 16;
    const int per = p.v != nullptr ? 2 * vpr : vpr;      // K then V
    const int total = n * per;
    const char *kd = static_cast<const char *>(p.kd), *vd = static_cast<const char *>(p.vd);
    constexpr int U = 4;
    for (int i0 = threadIdx.x; i0 < total; i0 += kCopyThreads * U) {
        uint4 x[U];
        char *to[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kCopyThreads;
            to[u] = nullptr;
            if (i < total) {
                const int row = i / per, c = i - row * per;
                const int t = __ldg(p.path + (size_t)b * p.T + row);
                const bool isv = c >= vpr;
                const size_t off = (((size_t)b * p.T + t) * p.H + h) * p.row_bytes +
                                   (size_t)(isv ? c - vpr : c) * 16;
                x[u] = __ldg(reinterpret_cast<const uint4 *>((isv ? vd : kd) + off));
                to[u] = dst(row, isv) + (size_t)(isv ? c - vpr : c) * 16;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (to[u] != nullptr) *reinterpret_cast<uint4 *>(to[u]) = x[u];
    }
}

__global__ void __launch_bounds__(kCopyThreads) tree_accept_kernel(const AcceptParams p)
{
    pdl_trigger();
    pdl_wait();
    const int pair = blockIdx.x, b = pair / p.H, h = pair - b * p.H;
    int code = 0;
    int n = path_tokens(p, b, threadIdx.x, kCopyThreads, &code);
    const int len = p.len[pair];
    const bool bad_path = __syncthreads_or(n < 0);       // also: every thread has read len
    if (bad_path) {
        if (h == 0 && code != 0) record_code(p.dev_code, code);
        return;
    }
    if (n == 0) return;
    if (len < 0 || len > p.cap || n > p.cap - len) {
        if (threadIdx.x == 0)
            record_code(p.dev_code, len < 0 || len > p.cap ? kDevBadLen : kDevTailFull);
        return;
    }
    copy_rows(p, b, h, n, [&](int row, bool isv) -> char * {
        const int64_t at = b * p.sb + h * p.sh + (int64_t)(len + row) * p.ss;
        return static_cast<char *>(isv ? p.v : p.k) + at * p.eb;
    });
    if (threadIdx.x == 0) p.len[pair] = len + n;
}

__global__ void __launch_bounds__(kPageThreads) tree_accept_pages_kernel(const AcceptParams p)
{
    __shared__ int s_warp[kPageThreads / 32];
    __shared__ int s_top;                    // ids left on the stack
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int top0 = 0;                            // (of thread 0)
    if (threadIdx.x == 0) {
        int top = *p.free_top;
        if (top < 0 || top > p.free_cap) {
            record_code(p.dev_code, kDevPoolEmpty_);
            top = 0;
        }
        s_top = top0 = top;
    }
    __syncthreads();
    for (int b0 = 0; b0 < p.B; b0 += kPageThreads) {
        const int b = b0 + threadIdx.x;
        int n = 0, need = 0, len = 0, nb = 0, code = 0;
        if (b < p.B) {
            n = path_tokens(p, b, 0, 1, &code);
            len = p.len[b];
            nb = p.n_blocks[b];
            if (n >= 0 && (len < 0 || len > p.max_blocks * p.bs || nb != (len + p.bs - 1) / p.bs ||
                           n > p.max_blocks * p.bs - len)) {
                code = kDevBadLen;
                n = -1;
            }
            if (n > 0 && len % p.bs != 0) {  // the page that takes the first token is there already
                const int id = p.table[(size_t)b * p.max_blocks + len / p.bs];
                if (id < 0 || id >= p.n_pool) {
                    code = kDevBadBlk;
                    n = -1;
                }
            }
            if (n < 0) {
                record_code(p.dev_code, code);
                n = 0;
            }
            need = n > 0 ? (len + n + p.bs - 1) / p.bs - nb : 0;
        }
        // the blocks taken before this sequence: a scan, or -- when the stack cannot serve
        // everyone or holds an id that is no block, and sequences must be skipped -- one by one
        // in order
        int incl = need;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        int before = incl - need, all = 0;
        for (int w = 0; w < kPageThreads / 32; ++w) {
            if (w < warp) before += s_warp[w];
            all += s_warp[w];
        }
        const int top = s_top;
        int first = top - before;            // this sequence's ids: first - 1, first - 2, ...
        bool skip = all > top;
        if (!skip)
            for (int i = 0; i < need; ++i) {
                const int id = p.free_ids[first - 1 - i];
                skip |= id < 0 || id >= p.n_pool;
            }
        if (__syncthreads_or(skip)) {
            for (int i = 0; i < min(kPageThreads, p.B - b0); ++i) {
                if (threadIdx.x == i && need > 0) {
                    first = s_top;
                    if (need > first) {
                        record_code(p.dev_code, kDevPoolEmpty_);
                        n = need = 0;
                    } else {
                        // a bad id leaves the stack; the good ones with it stay for the sequences
                        // behind
                        int keep = first - need;
                        for (int j = first - need; j < first; ++j) {
                            const int id = p.free_ids[j];
                            if (id < 0 || id >= p.n_pool) continue;
                            if (keep != j) p.free_ids[keep] = id;
                            ++keep;
                        }
                        if (keep < first) {
                            record_code(p.dev_code, kDevBadBlk);
                            n = need = 0;
                            s_top = keep;
                        } else {
                            s_top = first - need;
                        }
                    }
                }
                __syncthreads();
            }
        } else if (threadIdx.x == 0) {
            s_top = top - all;
        }
        if (b < p.B) {
            if (n > 0) {
                for (int i = 0; i < need; ++i) {
                    p.table[(size_t)b * p.max_blocks + nb + i] = p.free_ids[first - 1 - i];
                    p.score[(size_t)b * p.max_blocks + nb + i] = 0.f;
                }
                p.n_blocks[b] = nb + need;
                p.len[b] = len + n;
            }
            p.accepted[b] = n;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0 && s_top != top0) *p.free_top = s_top;
}

__global__ void __launch_bounds__(kCopyThreads) tree_accept_paged_kernel(const AcceptParams p)
{
    pdl_trigger();
    pdl_wait();
    const int pair = blockIdx.x, b = pair / p.H, h = pair - b * p.H;
    const int n = p.accepted[b];
    if (n == 0) return;
    const int first = p.len[b] - n;
    const int32_t *tab = p.table + (size_t)b * p.max_blocks;
    copy_rows(p, b, h, n, [&](int row, bool isv) -> char * {
        const int slot = first + row;
        const size_t blk = (size_t)tab[slot / p.bs];     // (every id was looked at before)
        char *base = static_cast<char *>(isv ? p.v : p.k);
        return base + (((size_t)h * p.n_pool + blk) * p.bs + slot % p.bs) * p.row_bytes;
    });
}

}  // namespace

cudaError_t launch_tree_accept(const AcceptParams &p, cudaStream_t stream)
{
    return launch_pdl(tree_accept_kernel, dim3((unsigned)(p.B * p.H)), dim3(kCopyThreads), 0, stream,
                      p);
}

cudaError_t launch_tree_accept_paged(const AcceptParams &p, cudaStream_t stream)
{
    const cudaError_t e =
        launch_pdl(tree_accept_pages_kernel, dim3(1), dim3(kPageThreads), 0, stream, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(tree_accept_paged_kernel, dim3((unsigned)(p.B * p.H)), dim3(kCopyThreads), 0,
                      stream, p);
}

}  // namespace kvc

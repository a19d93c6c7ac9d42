// append_q8.cu -- new rows into pages of e4m3 numbers with a scale for each page and head.
//
//   s = 2^e, the smallest power of two with max|x| / s <= 448 over the page's rows of a head,
//   stored x8 = e4m3(x / s), rounded to nearest even: 4 significant bits down to 2^-6 s.
//
// Scales are powers of two so that a growing one only moves exponents: rows that a partly filled
// page held already are brought to the new scale (x8 * s_old / s_new, exact unless it falls below
// 2^-6 s_new, where the steps are 2^-9 s_new), and a page filled token by token holds what the same
// rows quantised at once hold, but for such small values.  A page whose scale is no power of two
// (written by someone else) is read and continued just as well, with a division.
//
// append_plan, by one block: checks every sequence, numbers the pages they need in sequence order
// (block-wide scans) and takes them from the top of the free stack, so that ids do not depend on
// timing; it writes one job per page that gets rows.  Then persistent warps, as many for a (job, head, K or
// V) as hold its rows in registers between the maximum and the rounding.  Small steps do both in one cluster.
// Bound by HBM for prompts (2 or 4 bytes in, 1 out an element): 16 prompts of 2048 to 4096 tokens, 32 heads of
// 128, bf16, 192 us (6.3 TB/s), of which the plan is 7.  Rows fetched into L2 while the plan is made, or one task
// ahead: 1 us at most.  Bound by latency for single tokens, a group of lanes a row: 16 x 32 heads 8.8 us (a warp a
// row: 11.2); ids and pages that the plan would read before it knows them save nothing.
#include <algorithm>

#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace kvc {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kRowWarps = 4;
// Warps of a block whose TEAM warps share a page, and blocks per SM, as registers allow.  In blocks of 4 warps: the
// smallest pages 6 58.7 us, 7 55.5, 8 54.8; the prompts above 6 194, 7 197.
constexpr int warps_of(int team) { return team > 1 ? team : kRowWarps; }
template <typename T>
constexpr int blocks_of(int NV, int team)
{
    return (NV * (int)sizeof(T) > 16 ? 5 : NV * (int)sizeof(T) > 8 ? 6 : 8) * kRowWarps / warps_of(team);
}
constexpr int kCl = 8;                       // blocks of the cluster that takes a small decode step
// (page, head, K or V) of it, at most.  256: 7.6 us by the cluster and 7.7 by two kernels, 1024: 8.8 and 8.5, but a
// call from Python, which the host bounds, 16.4 and 19; 2048: 11.4 and 9.4; 4096: 15.9 and 12.2.
constexpr int kStepTasks = 1024;
constexpr int kDevBadLen_ = 5;               // KVC_DEV_BAD_LENGTH
constexpr int kDevBadBlk_ = 9;               // KVC_DEV_BAD_BLOCK
constexpr int kDevPoolEmpty_ = 10;           // KVC_DEV_POOL_EMPTY

// Inclusive scan of two counters over the block (threads in order); s_warp: 2 * 32 words.
__device__ __forceinline__ int2 block_scan(int2 x, int *s_warp, int2 *all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o);
        if (lane >= o) {
            x.x += a;
            x.y += b;
        }
    }
    __syncthreads();                         // (s_warp is free)
    if (lane == 31) {
        s_warp[warp] = x.x;
        s_warp[32 + warp] = x.y;
    }
    __syncthreads();
    const int2 own = make_int2(s_warp[lane], s_warp[32 + lane]);
    int2 w = own;                            // (kPlanThreads / 32 warps are a warp's lanes)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, w.x, o), b = __shfl_up_sync(0xffffffffu, w.y, o);
        if (lane >= o) {
            w.x += a;
            w.y += b;
        }
    }
    *all = make_int2(__shfl_sync(0xffffffffu, w.x, 31), __shfl_sync(0xffffffffu, w.y, 31));
    return make_int2(x.x + __shfl_sync(0xffffffffu, w.x - own.x, warp), x.y + __shfl_sync(0xffffffffu, w.y - own.y, warp));
}

// The first of n ascending numbers above x.
__device__ __forceinline__ int find_above(const int *a, int n, int x)
{
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ void append_plan(const AppendQ8Params &p)
{
    __shared__ int s_warp[64];
    __shared__ int s_need[kPlanThreads];     // pages to pop
    __shared__ int s_jobs[kPlanThreads];     // inclusive scan of the pages that get rows
    __shared__ int s_first[kPlanThreads];    // a sequence's ids are ids[first - 1], ids[first - 2], ...
    __shared__ int s_n[kPlanThreads];        // rows to append
    __shared__ int s_len[kPlanThreads], s_row[kPlanThreads];
    __shared__ int s_top;
    const int tid = threadIdx.x;
    bool bad = false;
    if (p.cu != nullptr)
        for (int b = tid; b < p.B; b += kPlanThreads) {
            const int lo = p.cu[b], hi = p.cu[b + 1];
            bad |= lo < 0 || hi < lo || hi > p.n_tokens;
        }
    int top0 = 0;
    if (tid == 0) {
        top0 = *p.free_top;
        if (top0 < 0 || top0 > p.free_cap) {
            record_code(p.dev_code, kDevPoolEmpty_);
            top0 = 0;
        }
        s_top = top0;
    }
    if (__syncthreads_or(bad)) {             // offsets that are none: nothing is appended at all
        if (tid == 0) {
            record_code(p.dev_code, kDevBadLen_);
            *p.n_jobs = 0;
        }
        if (p.appended != nullptr)
            for (int b = tid; b < p.B; b += kPlanThreads) p.appended[b] = 0;
        return;
    }
    int jobs0 = 0;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int n = 0, need = 0, jobs = 0, len = 0, nb = 0, row = 0;
        if (b < p.B) {
            row = p.cu != nullptr ? p.cu[b] : b;
            n = p.cu != nullptr ? p.cu[b + 1] - row : 1;
            len = p.len[b];
            nb = p.n_blocks[b];
            int code = 0;
            if (len < 0 || len > p.max_blocks * p.bs || nb != (len + p.bs - 1) / p.bs ||
                n > p.max_blocks * p.bs - len) {
                code = kDevBadLen_;
            } else if (n > 0 && len % p.bs != 0) {   // the page that takes the first row is there already
                const int id = p.table[(size_t)b * p.max_blocks + len / p.bs];
                if (id < 0 || id >= p.n_pool) code = kDevBadBlk_;
            }
            if (code != 0) {
                record_code(p.dev_code, code);
                n = 0;
            }
            if (n > 0) {
                need = (len + n + p.bs - 1) / p.bs - nb;
                jobs = need + (len % p.bs != 0 ? 1 : 0);
            }
        }
        int2 all;
        int2 incl = block_scan(make_int2(need, jobs), s_warp, &all);
        const int top = s_top;
        int first = top - (incl.x - need);
        bool skip = all.x > top;
        if (!skip)
            for (int i = tid; i < all.x; i += kPlanThreads) {
                const int id = p.free_ids[top - 1 - i];
                skip |= id < 0 || id >= p.n_pool;
            }
        s_need[tid] = need;
        s_n[tid] = n;
        if (__syncthreads_or(skip)) {
            // too few ids, or one that is no page: the sequences one by one in order
            if (tid == 0) {
                int t = top;
                for (int i = 0; i < min(kPlanThreads, p.B - b0); ++i) {
                    const int want = s_need[i];
                    s_first[i] = t;
                    if (want == 0) continue;
                    if (want > t) {
                        record_code(p.dev_code, kDevPoolEmpty_);
                        s_n[i] = 0;
                        continue;
                    }
                    int keep = t - want;     // a bad id leaves the stack, the good ones stay for the others
                    for (int j = t - want; j < t; ++j) {
                        const int id = p.free_ids[j];
                        if (id < 0 || id >= p.n_pool) continue;
                        if (keep != j) p.free_ids[keep] = id;
                        ++keep;
                    }
                    if (keep < t) {
                        record_code(p.dev_code, kDevBadBlk_);
                        s_n[i] = 0;
                        t = keep;
                    } else {
                        t -= want;
                    }
                }
                s_top = t;
            }
            __syncthreads();
            n = s_n[tid];
            first = s_first[tid];
            if (n == 0) need = jobs = 0;
            incl = block_scan(make_int2(need, jobs), s_warp, &all);
        } else if (tid == 0) {
            s_top = top - all.x;
        }
        __syncthreads();
        s_jobs[tid] = incl.y;
        s_first[tid] = first;
        s_n[tid] = n;
        s_len[tid] = len;
        s_row[tid] = row;
        __syncthreads();
        // a job for every page that gets rows, and a table entry for the popped ones
        for (int e = tid; e < all.y; e += kPlanThreads) {
            const int i = find_above(s_jobs, min(kPlanThreads, p.B - b0), e);
            const int j = e - (i > 0 ? s_jobs[i - 1] : 0);
            const int l = s_len[i], lb = l / p.bs + j, held = j == 0 ? l % p.bs : 0;
            const int at = lb * p.bs + held;                   // the first new row's slot
            const size_t entry = (size_t)(b0 + i) * p.max_blocks + lb;
            int id;
            if (held > 0) {
                id = p.table[entry];
            } else {
                id = p.free_ids[s_first[i] - 1 - (lb - (l + p.bs - 1) / p.bs)];
                p.table[entry] = id;
                p.score[entry] = 0.f;
            }
            p.jobs[jobs0 + e] = make_int4(id, held, s_row[i] + at - l, min(p.bs - held, l + s_n[i] - at));
        }
        jobs0 += all.y;
        if (b < p.B) {
            if (n > 0) {
                p.n_blocks[b] = nb + need;
                p.len[b] = len + n;
            }
            if (p.appended != nullptr) p.appended[b] = n;
        }
        __syncthreads();
    }
    if (tid == 0) {
        *p.n_jobs = jobs0;
        if (s_top != top0) *p.free_top = s_top;
    }
}

__global__ void __launch_bounds__(kPlanThreads) append_q8_plan_kernel(const AppendQ8Params p)
{
    pdl_trigger();
    pdl_wait();
    append_plan(p);
}

// 8 elements of a row, and the largest size among them and `a` (NaN counts as nothing).
template <typename T>
struct Row8;
template <>
struct Row8<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const void *p) { w = ld_stream_16(p); }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float *f) const
    {
        f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
        f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z); f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
    }
    using Max = __nv_bfloat162;              // of the even and of the odd elements
    static __device__ __forceinline__ Max none() { return __floats2bfloat162_rn(0.f, 0.f); }
    __device__ __forceinline__ void widen(Max &m) const
    {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = x[i] & 0x7fff7fffu;
            m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162 *>(&a));
        }
    }
    static __device__ __forceinline__ float size(Max m) { return fmaxf(__low2float(m), __high2float(m)); }
};
template <>
struct Row8<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const void *p)
    {
        a = ld_stream_16(p);
        b = ld_stream_16(static_cast<const char *>(p) + 16);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float *f) const
    {
        f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
        f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
        f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
        f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
    }
    using Max = float;
    static __device__ __forceinline__ Max none() { return 0.f; }
    __device__ __forceinline__ void widen(Max &m) const
    {
        float f[8];
        get(f);
#pragma unroll
        for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(f[k]));
    }
    static __device__ __forceinline__ float size(Max m) { return m; }
};

// The smallest power of two s >= 2^-120 with amax / s <= 448 = 1.75 * 2^8 (2^119 at most: beyond
// 448 * 2^119 = 2.98e38 values saturate).
__device__ __forceinline__ float scale_for(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < -120 ? -120 : (e > 119 ? 119 : e);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// The lanes of this thread's group of LANES in its warp.
template <int LANES>
__device__ __forceinline__ uint32_t group_mask()
{
    return LANES >= 32 ? 0xffffffffu : ((1u << (LANES & 31)) - 1u) << (threadIdx.x & 31 & ~(LANES - 1));
}
// The largest x of LANES threads: some lanes of a warp, a warp, or a block.  s_max: two sets of words, one a warp, used
// in turn, so that one barrier a call is enough.
template <int LANES>
__device__ __forceinline__ float team_max(float x, float *s_max, int &turn)
{
#pragma unroll
    for (int o = (LANES < 32 ? LANES : 32) / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(group_mask<LANES>(), x, o));
    if (LANES <= 32) return x;
    float *s = s_max + turn * (LANES / 32);
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < LANES / 32; ++w) x = fmaxf(x, s[w]);
    return x;
}

// One task: a page's new rows of a head, keys or values, by LANES threads.  NV: vectors of 8 elements that a
// lane holds at once.
template <typename T, int D, int NV, int LANES>
__device__ __forceinline__ void quantise(const AppendQ8Params &p, const int4 j, int rest, float *s_max, int &turn)
{
    constexpr int VPR = D / 8;               // vectors per row
    const int lane = LANES <= 32 ? threadIdx.x & (LANES - 1) : threadIdx.x;
    const int h = rest >> 1, held = j.y, n_vec = j.w * VPR;
    const bool is_v = rest & 1;
    const int64_t st = p.new_st;
    const T *src = static_cast<const T *>(is_v ? p.v_new : p.k_new) + h * p.new_sh + j.z * st;
    const size_t page = (size_t)h * p.n_pool + j.x;
    uint8_t *dst = (is_v ? p.v : p.k) + page * p.bs * D;
    float *scale = (is_v ? p.vs : p.ks) + page;
    const float s_old = held > 0 ? *scale : 0.f;

    Row8<T> x[NV];
    auto fetch = [&](int v0) {
        if (n_vec - v0 >= LANES * NV) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = v0 + i * LANES + lane;
                x[i].load(src + v / VPR * st + v % VPR * 8);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = v0 + i * LANES + lane;
            if (v < n_vec) x[i].load(src + v / VPR * st + v % VPR * 8);
            else x[i].zero();
        }
    };
    typename Row8<T>::Max big = Row8<T>::none();
    for (int v0 = 0; v0 < n_vec; v0 += LANES * NV) {
        fetch(v0);
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i].widen(big);
    }
    float amax = team_max<LANES>(Row8<T>::size(big), s_max, turn);
    const bool inf = amax == INFINITY;       // then the largest finite one counts
    if (inf) {
        amax = 0.f;
        for (int v0 = 0; v0 < n_vec; v0 += LANES * NV) {
            fetch(v0);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float f[8];
                x[i].get(f);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (fabsf(f[k]) < INFINITY) amax = fmaxf(amax, fabsf(f[k]));
            }
        }
        amax = team_max<LANES>(amax, s_max, turn);
    }
    const float s = fmaxf(s_old, scale_for(amax));
    if (LANES <= 32) __syncwarp(group_mask<LANES>());          // every lane has read the scale
    if (lane == 0 && (held == 0 || s != s_old)) *scale = s;
    if (held > 0 && s != s_old) {            // the rows held before go over to the new scale
        const float ratio = s_old / s;
        for (int i = lane; i < held * (D / 16); i += LANES) {
            uint4 w = *reinterpret_cast<uint4 *>(dst + i * 16);
            uint32_t *q = &w.x;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 a = __half22float2(
                    __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(q[k] & 0xffffu), __NV_E4M3)));
                const float2 b = __half22float2(
                    __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(q[k] >> 16), __NV_E4M3)));
                q[k] = pack4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
            }
            *reinterpret_cast<uint4 *>(dst + i * 16) = w;
        }
    }
    const float inv = 1.f / s;
    const bool power = (__float_as_uint(s) & 0x7fffffu) == 0u;   // then x * inv is x / s
    for (int v0 = 0; v0 < n_vec; v0 += LANES * NV) {
        if (n_vec > LANES * NV || inf) fetch(v0);
        uint8_t *to = dst + (size_t)held * D + (size_t)(v0 + lane) * 8;
        const int in = n_vec - v0 - lane;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[8];
            x[i].get(f);
            if (power && !inf) {
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] *= inv;
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = fabsf(f[k]) == INFINITY ? __uint_as_float(0x7fc00000u) : f[k] / s;
            }
            if (i * LANES < in)
                *reinterpret_cast<uint2 *>(to + i * LANES * 8) =
                    make_uint2(pack4(f[0], f[1], f[2], f[3]), pack4(f[4], f[5], f[6], f[7]));
        }
    }
}

// Tasks (job, head, K or V) w, w + n_w, ... of team w; the next task's job is read ahead.
template <typename T, int D, int NV, int LANES>
__device__ __forceinline__ void quantise_all(const AppendQ8Params &p, long long w, long long n_w, float *s_max = nullptr)
{
    int turn = 0;
    const unsigned per = 2u * (unsigned)p.H;
    const long long tasks = (long long)__ldcg(p.n_jobs) * per;
    if (w >= tasks) return;
    unsigned job = (unsigned)(w / per);
    int4 j = __ldcg(p.jobs + job);
    for (; w < tasks; w += n_w) {
        const int rest = (int)(w - (long long)job * per);
        const unsigned job1 = (unsigned)((unsigned long long)(w + n_w) / per);
        int4 j1 = j;
        if (job1 != job && w + n_w < tasks) j1 = __ldcg(p.jobs + job1);
        quantise<T, D, NV, LANES>(p, j, rest, s_max, turn);
        job = job1;
        j = j1;
    }
}

template <typename T, int D, int NV, int TEAM>
__global__ void __launch_bounds__(warps_of(TEAM) * 32, blocks_of<T>(NV, TEAM)) append_q8_rows_kernel(const AppendQ8Params p)
{
    __shared__ float s_max[2 * TEAM];
    pdl_trigger();
    pdl_wait();
    if constexpr (TEAM > 1) {
        quantise_all<T, D, NV, 32 * TEAM>(p, blockIdx.x, gridDim.x, s_max);
    } else {
        // (a single row is less than a warp's lanes hold)
        constexpr int LANES = NV == 1 ? D / 8 : 32, TEAMS = kRowWarps * 32 / LANES;
        quantise_all<T, D, NV, LANES>(p, (long long)blockIdx.x * TEAMS + threadIdx.x / LANES, (long long)gridDim.x * TEAMS);
    }
}

// Both steps in one cluster, for few rows.
template <typename T, int D>
__global__ void __cluster_dims__(kCl, 1, 1) __launch_bounds__(kPlanThreads) append_q8_step_kernel(const AppendQ8Params p)
{
    pdl_trigger();
    pdl_wait();
    if (blockIdx.x == 0) append_plan(p);
    __threadfence();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
    // a group of lanes a row; warps of a block take tasks of different jobs: its share is no smaller where jobs are few
    constexpr int LANES = D / 8, PER = 32 / LANES;
    quantise_all<T, D, 1, LANES>(p, ((threadIdx.x >> 5) * kCl + blockIdx.x) * PER + (threadIdx.x & 31) / LANES,
                                 kCl * kPlanThreads / LANES);
}

template <typename T, int D>
cudaError_t append_typed(const AppendQ8Params &p, int n_sm, cudaStream_t stream)
{
    const long long tasks = (long long)p.max_jobs * 2 * p.H;
    if (p.n_tokens <= 4 * p.B && tasks <= kStepTasks)
        return launch_pdl(append_q8_step_kernel<T, D>, dim3(kCl), dim3(kPlanThreads), 0, stream, p);
    const cudaError_t e = launch_pdl(append_q8_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p);
    if (e != cudaSuccess) return e;
    auto rows = [&](auto kernel, int NV, int team) {
        const int at_once = team > 1 ? 1 : NV == 1 ? kRowWarps * 256 / D : kRowWarps;          // tasks of a block
        const long long blocks = (tasks + at_once - 1) / at_once, most = (long long)n_sm * blocks_of<T>(NV, team);
        return launch_pdl(kernel, dim3((unsigned)std::max(1LL, std::min(blocks, most))), dim3(warps_of(team) * 32), 0,
                          stream, p);
    };
    if (p.cu == nullptr) return rows(append_q8_rows_kernel<T, D, 1, 1>, 1, 1);
    // A lane holds NV vectors, 128 bytes of rows of either type, which leaves 24 warps an SM, and as many warps share
    // a page as that takes.  Measured (us), 16 prompts of 2048 to 4096 rows of 32 heads of 128, bf16, pages of 32:
    // one warp with 2 NV 201, two with NV 194, four with NV / 2 211; 41 x 1000 to 2000 rows of 4 heads of 256 in pages
    // of 32: one warp in two passes 110, four with 2 NV 114, four with NV 69, eight with NV / 2 78; 20 x the same in
    // pages of 64: one warp 61, four with 2 NV 42, eight with NV 39; 40 x 1000 rows of 8 heads of 128 in pages of
    // 16: one warp with 2 NV 80, with NV 50; of 16 heads of 64: one warp with 2 NV 127, NV 71, NV / 2 55 (their bytes
    // at the copy rate: 36; the plan, 7 us or more in which no row is read, is the largest part of the rest).
    constexpr int NV = 16 / (int)sizeof(T);
    const int page = p.bs * D / 256;         // vectors a lane of one warp
    if constexpr (NV == 8)                   // (the smallest fp32 page takes more)
        if (page <= NV / 2) return rows(append_q8_rows_kernel<T, D, NV / 2, 1>, NV / 2, 1);
    if (page <= NV) return rows(append_q8_rows_kernel<T, D, NV, 1>, NV, 1);
    if (page <= NV * 2) return rows(append_q8_rows_kernel<T, D, NV, 2>, NV, 2);
    if (page <= NV * 4) return rows(append_q8_rows_kernel<T, D, NV, 4>, NV, 4);
    if (page <= NV * 8) return rows(append_q8_rows_kernel<T, D, NV, 8>, NV, 8);
    return rows(append_q8_rows_kernel<T, D, 2 * NV, 8>, 2 * NV, 8);
}
template <typename T>
cudaError_t append_dims(const AppendQ8Params &p, int n_sm, cudaStream_t stream)
{
    switch (p.D) {
    case 64: return append_typed<T, 64>(p, n_sm, stream);
    case 128: return append_typed<T, 128>(p, n_sm, stream);
    default: return append_typed<T, 256>(p, n_sm, stream);
    }
}

}  // namespace

cudaError_t launch_paged_append_q8(const AppendQ8Params &p, bool bf16, int n_sm, cudaStream_t stream)
{
    return bf16 ? append_dims<__nv_bfloat16>(p, n_sm, stream) : append_dims<float>(p, n_sm, stream);
}

}  // namespace kvc

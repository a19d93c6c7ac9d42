// latent_expand_tc.cu -- the expanded form of a bf16 latent cache on the 5th-generation tensor
// cores: K[b,h,s] = [W_k[h] c | c_rope], V[b,h,s] = W_v[h] c, one product of 128 slots by the
// rows of a head's matrices, over d_latent.
//
// Bound: the products (2 * d_latent * (2 d_head - d_rope) FLOP a slot and head) and the writes of K
// and V (4 d_head bytes), of the same order.
//
// Tiling.  A block keeps a tile of 128 slots resident in shared memory (all d_latent columns: 128
// KB at 512) and streams the matrices of head after head past it, 64 columns of W_k[h] and W_v[h]
// (up to 256 rows) a stage: the latent rows are read once per block, the matrices (a few MB)
// from L2.  A head's K and V rows form one accumulator of up to 256 columns (K then V, K's width
// rounded up to 16; d_head 256: K and V one after the other), double-buffered in tensor memory, so
// the writes of one head overlap the products of the next.
//
// Work: (slot tile, head) units in one sequence, split evenly over the blocks; tiles are counted
// from the lengths on the device.  Clusters of two or four blocks that share the matrices' stages
// by multicast were measured and dropped (52.9 and 59.9 us against 53.0 alone: L2 is not what
// bounds it).
//
// Roles (320 threads): warp 0 copies (TMA), warp 1 issues the products, warps 2-9 (two sets, one
// for either accumulator) take a slot per thread from tensor memory, round once, and pass 32
// columns at a time through shared memory so that a store instruction writes contiguous pieces of
// 8 slots (32-byte pieces of 32 slots straight from registers: 57 us against 35 for the
// products alone); the shared rope part goes from the latent rows to the keys in the same
// stores.  Warp 1 looks at the next stage's barrier before it issues a stage's products and waits
// only if it had not arrived: a satisfied wait between two stages costs it about 200 clocks, in
// which the tensor cores run dry.  (A warp of its own that waited and passed the stages on: through
// a named barrier 1.6 us faster, 52.6, but a wait without a limit; through a counted word 55.8 us.)
//
// Every wait is bounded (p.spin_limit polls).  One that gives up records KVC_DEV_TIMEOUT and raises
// s_abort, which ends the others.  The warp that copies then stops, warp 1 issues no more products,
// the others walk to their ends, and the block exits once its copies and products in flight are
// done.  No warp waits for another in any other way, but for the barriers over the whole block.
#include "tc_ops.cuh"
#include "internal.h"

namespace kvc {

namespace {

constexpr int kThreads = 320;
constexpr int kStaging = 8 * 2048;           // a writing warp's [32 slots][32 columns]
constexpr int kTile = 128;                   // slots
constexpr int kSub = kTile * 128;            // bytes of [128 slots][64]
constexpr int kSmemMax = 227 * 1024;
constexpr int kMaxStages = 8;
constexpr int kDevBadLen = 5;

struct ExpandMaps {
    CUtensorMap c, wk, wv;
};

struct ExpandPlan {
    int32_t jobs;                // per head: 1 (K and V together) or 2
    int32_t nk, nk16;            // K rows, rounded up to 16
    int32_t stage, stages;       // bytes of a stage, stages
    int32_t smem;
};

// Slots of sequence b to expand.
__device__ __forceinline__ int expand_len(const ExpandParams &p, int b)
{
    const int n = p.len != nullptr ? p.len[b] : p.n_valid;
    const int most = p.cap < p.dst_cap ? p.cap : p.dst_cap;
    return n < 0 ? 0 : (n > most ? most : n);
}

// A block's units: jobs [lo, hi) of the first tile, all jobs of the tiles between, ...
struct ExpandRange {
    int b, tile;                 // first slot tile
    long long first, last;       // units, from the first job of that tile
};

__device__ __forceinline__ ExpandRange expand_range(const ExpandParams &p, int per_tile)
{
    const int lane = threadIdx.x & 31;
    const int per = (p.B + 31) >> 5;
    const int b0 = min(p.B, lane * per), b1 = min(p.B, b0 + per);
    const int most = p.cap < p.dst_cap ? p.cap : p.dst_cap;
    long long sum = 0;
    for (int b = b0; b < b1; ++b) {
        const int raw = p.len != nullptr ? p.len[b] : p.n_valid;
        if (blockIdx.x == 0 && threadIdx.x < 32 && (raw < 0 || raw > most))
            record_code(p.dev_code, kDevBadLen);
        sum += (expand_len(p, b) + kTile - 1) / kTile;
    }
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    const long long units = __shfl_sync(0xffffffffu, incl, 31) * per_tile;
    const long long u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
    const long long t0 = u0 / per_tile, before = incl - sum;
    const bool here = u1 > u0 && before <= t0 && t0 < incl;
    int b = b0, tile = 0;
    if (here) {
        long long t = before;
        for (;; ++b) {
            const int nt = (expand_len(p, b) + kTile - 1) / kTile;
            if (t0 < t + nt || b == b1 - 1) break;
            t += nt;
        }
        tile = (int)(t0 - t);
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    ExpandRange r;
    r.b = __shfl_sync(0xffffffffu, b, src & 31);
    r.tile = __shfl_sync(0xffffffffu, tile, src & 31);
    r.first = u0 - t0 * per_tile;
    r.last = src < 0 ? r.first : r.first + (u1 - u0);
    return r;
}

// Walks the slot tiles of a range.
struct ExpandWalk {
    int b, tile, n, per_tile;
    long long first, last;
    bool begun;
    __device__ __forceinline__ ExpandWalk(const ExpandRange &r, int per)
        : b(r.b), tile(r.tile), n(0), per_tile(per), first(r.first), last(r.last), begun(false)
    {
    }
    // next tile with its jobs [lo, hi)
    __device__ __forceinline__ bool next(const ExpandParams &p, int &lo, int &hi)
    {
        if (begun) {
            ++tile;
            last -= per_tile;
            first = 0;
        }
        if (last <= first) return false;
        for (; b < p.B; ++b, tile = 0, begun = false) {
            if (!begun) n = expand_len(p, b);
            begun = true;
            if (tile * kTile < n) {
                lo = (int)first;
                hi = (int)(last < per_tile ? last : per_tile);
                return true;
            }
        }
        return false;
    }
};

__global__ void __launch_bounds__(kThreads, 1)
latent_expand_tc_kernel(const __grid_constant__ ExpandMaps maps, const ExpandParams p,
                        const ExpandPlan pl)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t sA = (raw + 1023u) & ~1023u;
    const int subs = p.R / 64;
    const uint32_t sW = sA + subs * kSub;
    const uint32_t sE = sW + pl.stages * pl.stage;
    const uint32_t bars = sE + kStaging;
    const uint32_t b_full = bars, b_empty = b_full + 8 * kMaxStages;
    const uint32_t b_a_full = b_empty + 8 * kMaxStages, b_a_empty = b_a_full + 8;
    const uint32_t b_acc_full = b_a_empty + 8, b_acc_empty = b_acc_full + 16;
    const uint32_t b_done = b_acc_empty + 16, tmem_slot = b_done + 8;
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem_raw + (tmem_slot + 8 - raw));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 2 && lane < 3) tc::prefetch_map(&maps.c + lane);
    if (threadIdx.x == 0) {
        for (int i = 0; i < pl.stages; ++i) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, 1);
        }
        mbar_init(b_a_full, 1);
        mbar_init(b_a_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_acc_full + 8 * i, 1);
            mbar_init(b_acc_empty + 8 * i, 4);
        }
        mbar_init(b_done, 1);
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tc::alloc(tmem_slot, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot));
    pdl_trigger();
    pdl_wait();
    const int per_tile = p.H * pl.jobs;
    const ExpandRange range = expand_range(p, per_tile);
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {             // whether the phase completed
        if (mbar_wait_abortable(bar, parity, p.spin_limit, s_abort)) return true;
        *s_abort = 1;
        record_code(p.dev_code, kDevCodeTimeout);
        return false;
    };
    ExpandWalk walk(range, per_tile);
    int lo = 0, hi = 0;
    unsigned n_w = 0, n_a = 0;                   // the producer's counts (for the drain)
    if (warp == 0) {
        uint32_t slot = 0, ph = 1;
        bool go = p.starve == 0;                 // (test hook: no copies, so the first waits run out)
        while (walk.next(p, lo, hi)) {
            if (n_a > 0 && go) go = __all_sync(0xffffffffu, wait(b_a_empty, (n_a - 1) & 1));
            if (!go) break;
            if (tc::elect()) {
                mbar_arrive_expect_tx(b_a_full, (uint32_t)subs * kSub);
                for (int i = 0; i < subs; i += 2)
                    tc::tma_5d(sA + i * kSub, &maps.c, 0, walk.tile * kTile, i, walk.b, 0, b_a_full);
            }
            __syncwarp();
            ++n_a;
            int h = lo / pl.jobs, job = lo - h * pl.jobs;
            for (int j = lo; j < hi; ++j) {
                const bool dok = pl.jobs == 1 || job == 0, dov = pl.jobs == 1 || job == 1;
                const uint32_t bytes = (uint32_t)((dok ? pl.nk : 0) + (dov ? p.D : 0)) * 128u;
                const uint32_t v_off = dok ? (uint32_t)pl.nk16 * 128u : 0u;
                for (int k = 0; k < subs; ++k, ++n_w) {
                    if (n_w >= (unsigned)pl.stages) go = __all_sync(0xffffffffu, wait(b_empty + 8 * slot, ph));
                    if (!go) break;
                    if (tc::elect()) {
                        const uint32_t dst = sW + slot * pl.stage, bar = b_full + 8 * slot;
                        mbar_arrive_expect_tx(bar, bytes);
                        if (dok) tc::tma_5d(dst, &maps.wk, 0, h * pl.nk, k, 0, 0, bar);
                        if (dov) tc::tma_5d(dst + v_off, &maps.wv, 0, h * p.D, k, 0, 0, bar);
                    }
                    __syncwarp();
                    if (++slot == (uint32_t)pl.stages) {
                        slot = 0;
                        ph ^= 1;
                    }
                }
                if (!go) break;
                if (++job == pl.jobs) {
                    job = 0;
                    ++h;
                }
            }
        }
    } else if (warp == 1) {
        uint32_t slot = 0, ph = 0;
        unsigned n = 0;                          // accumulators so far
        bool in = false;                         // the next stage was seen to have arrived
        bool go = true;                          // no wait of this lane has given up
        while (walk.next(p, lo, hi)) {
            go &= wait(b_a_full, n_a & 1);
            ++n_a;
            int job = lo - lo / pl.jobs * pl.jobs;
            for (int j = lo; j < hi; ++j, ++n) {
                const int cols = (pl.jobs == 1 || job == 0 ? pl.nk16 : 0) + (pl.jobs == 1 || job == 1 ? p.D : 0);
                const uint32_t id = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(cols >> 3) << 17) |
                                    ((uint32_t)(kTile >> 4) << 24);
                const uint32_t buf = n & 1, d = tmem + buf * 256;
                if (n >= 2) go &= wait(b_acc_empty + 8 * buf, ((n >> 1) - 1) & 1);
                for (int k = 0; k < subs; ++k) {
                    if (!__all_sync(0xffffffffu, in)) go &= wait(b_full + 8 * slot, ph);
                    const uint32_t at = slot;
                    if (++slot == (uint32_t)pl.stages) {
                        slot = 0;
                        ph ^= 1;
                    }
                    in = tc::test(b_full + 8 * slot, ph);    // answered while the products are issued
                    tc::fence_after();
                    if (tc::elect() && go) {
                        const uint32_t a = sA + k * kSub, w = sW + at * pl.stage;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc::mma(d, tc::desc_k(a + kk * 32), tc::desc_k(w + kk * 32), id, k > 0 || kk > 0);
                        tc::commit(b_empty + 8 * at);
                        if (k == subs - 1) {
                            tc::commit(b_acc_full + 8 * buf);
                            if (j == hi - 1) tc::commit(b_a_empty);
                        }
                    }
                    __syncwarp();
                }
                if (++job == pl.jobs) job = 0;
            }
        }
    } else {
        const int q4 = warp & 3, set = (warp - 2) >> 2;
        const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
        const uint32_t mem = sE + (warp - 2) * 2048;
        const int row4 = lane >> 2, piece = lane & 3;        // store phase: rows 8 i + row4, 8 columns
        unsigned n = 0;
        while (walk.next(p, lo, hi)) {
            const int s0 = walk.tile * kTile + q4 * 32;
            const int live = walk.n - s0;                    // slots of this warp to write
            const __nv_bfloat16 *rope = static_cast<const __nv_bfloat16 *>(p.c) + walk.b * p.c_sb +
                                        (int64_t)s0 * p.c_ss + p.R - pl.nk;   // indexed by K column
            int h = lo / pl.jobs, job = lo - h * pl.jobs;
            for (int j = lo; j < hi; ++j, ++n) {
                const bool dok = pl.jobs == 1 || job == 0, dov = pl.jobs == 1 || job == 1;
                const int64_t at = walk.b * p.sb + h * p.sh + (int64_t)s0 * p.ss;
                if (++job == pl.jobs) {
                    job = 0;
                    ++h;
                }
                const uint32_t buf = n & 1, acc = tmem + buf * 256 + lanes;
                if ((int)buf != set) continue;
                const int kcols = dok ? pl.nk16 : 0;
                wait(b_acc_full + 8 * buf, (n >> 1) & 1);
                tc::fence_after();
#pragma unroll 1
                for (int c = dok ? 0 : p.D; c < (dov ? 2 * p.D : p.D); c += 32) {
                    const bool isv = c >= p.D;
                    const int col0 = isv ? c - p.D : c;
                    const int width = isv ? p.D : pl.nk;     // columns that are products
                    __syncwarp();                            // the last piece is stored
                    if (col0 < width) {                      // (else all rope)
                        float x[32];
                        tc::ld32(acc + (isv ? kcols : 0) + col0, x);
                        tc::wait_ld();
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            tc::st_shared_16(mem + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4),
                                             tc::pack_bf16(x[8 * i], x[8 * i + 1]),
                                             tc::pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                                             tc::pack_bf16(x[8 * i + 4], x[8 * i + 5]),
                                             tc::pack_bf16(x[8 * i + 6], x[8 * i + 7]));
                    }
                    __syncwarp();
                    const int col = col0 + 8 * piece;
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(isv ? p.v : p.k) + at + col;
                    uint4 w[4];
                    if (col < width) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 8 * i + row4;
                            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                                         : "r"(mem + r * 64 + ((piece ^ ((r >> 1) & 3)) << 4)));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 8 * i + row4;
                            if (r < live)
                                w[i] = __ldg(reinterpret_cast<const uint4 *>(rope + (int64_t)r * p.c_ss + col));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 8 * i + row4;
                        if (r < live) *reinterpret_cast<uint4 *>(dst + (int64_t)r * p.ss) = w[i];
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_acc_empty + 8 * buf);
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (*s_abort) {                              // copies and products in flight end before the block
        if (threadIdx.x == 0) {
            for (unsigned i = n_w > (unsigned)pl.stages ? n_w - pl.stages : 0; i < n_w; ++i)
                mbar_wait_ok(b_full + 8 * (i % pl.stages), (i / pl.stages) & 1, kMbarSpinLimit >> 4);
            if (n_a > 0) mbar_wait_ok(b_a_full, (n_a - 1) & 1, kMbarSpinLimit >> 4);
        } else if (warp == 1) {
            if (tc::elect()) tc::commit(b_done);
            __syncwarp();
            mbar_wait_ok(b_done, 0, kMbarSpinLimit);
        }
        __syncthreads();
    }
    tc::fence_after();
    if (warp == 1) tc::dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_latent_expand_tc(const ExpandParams &params, cudaStream_t stream, bool *used)
{
    *used = false;
    ExpandParams p = params;
    if (p.spin_limit == 0) p.spin_limit = kMbarSpinLimit;
    ExpandPlan pl{};
    pl.nk = p.D - p.E;
    pl.nk16 = (pl.nk + 15) / 16 * 16;
    pl.jobs = pl.nk16 + p.D <= 256 ? 1 : 2;
    const int rows = pl.jobs == 1 ? pl.nk16 + p.D : 256;
    const int subs = p.R / 64;
    pl.stage = rows * 128;
    const int room = kSmemMax - 1024 - subs * kSub - kStaging - 512;
    pl.stages = room / pl.stage;
    if (pl.stages > kMaxStages) pl.stages = kMaxStages;
    pl.smem = 1024 + subs * kSub + pl.stages * pl.stage + kStaging + 512;
    ExpandMaps maps;
    const uint64_t R = p.R, B = p.B, H = p.H, S = subs;
    const uint64_t ss = (uint64_t)p.c_ss * 2, sb = (uint64_t)p.c_sb * 2, row = R * 2;
    const bool ok = pl.stages >= 2 &&
        tc::encode_5d(&maps.c, p.c, {64, (uint64_t)p.cap, S, B, 1}, {ss, 128, sb, sb * B}, kTile, 2, 1) &&
        tc::encode_5d(&maps.wk, p.wk, {64, H * pl.nk, S, 1, 1}, {row, 128, row * H * pl.nk, row * H * pl.nk},
                      pl.nk, 1, 1) &&
        tc::encode_5d(&maps.wv, p.wv, {64, H * p.D, S, 1, 1}, {row, 128, row * H * p.D, row * H * p.D}, p.D,
                      1, 1);
    if (!ok) return cudaSuccess;
    *used = true;
    static bool configured[64] = {};
    static int sms[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        cudaError_t e = cudaFuncSetAttribute(latent_expand_tc_kernel,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
        if (e != cudaSuccess) return e;
        e = cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    // no more blocks than units there can be
    const long long most = (long long)p.B * (((p.cap < p.dst_cap ? p.cap : p.dst_cap) + kTile - 1) / kTile) *
                           p.H * pl.jobs;
    const unsigned grid = (unsigned)(most < sms[dev] ? (most > 0 ? most : 1) : sms[dev]);
    return launch_pdl(latent_expand_tc_kernel, dim3(grid), dim3(kThreads), (size_t)pl.smem, stream, maps, p, pl);
}

}  // namespace kvc

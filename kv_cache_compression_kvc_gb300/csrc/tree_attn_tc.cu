// tree_attn_tc.cu -- attention of a tree of drafted tokens over a bf16 cache (contiguous, paged or
// latent) on the 5th-generation tensor cores.
//
// R = n_draft * G query rows share every cached slot, so both products are dense: per tile of TS
// slots   S[rows x slots] = Q K^T   and   O^T[dims x rows] += V^T P^T,   with a running softmax
// between them.  What bounds it is the stream of the cache (a row tile of 64 or 128 rows costs
// the tensor cores less than its bytes cost HBM), up to about 128 rows a pair; beyond that each
// further row tile reads the slots again from L2.
//
// Layout choices.
//   S has a query row per tensor-memory lane: a thread owns a row, so its maximum and sum need no
//   exchange between threads.  M = RN rows (64 or 128).
//   O is kept transposed, a value dimension per lane and a row per column: a 512-wide latent
//   value of 64 rows takes 256 columns of tensor memory (rows x dims would take all 512 and leave
//   none for S), and the value rows are used as they lie in memory (V^T is the MN-major A
//   operand).  P goes through shared memory as the K-major B operand, rounded to bf16: the weights
//   are off by at most 2^-8 each, as is the bf16 output.
//   A latent cache's tile is loaded once and serves as K (all of it) and V (its first d_latent
//   columns).
//   The running maximum is lazy: a tile whose logits stay below max + 8 (log2 units) keeps the old
//   reference, so P stays below 2^8 and O is rescaled only when the maximum really rises.
//
// Roles (192 threads): warp 0 issues TMA loads into a ring of units (128 dims x TS slots), warp 1
// owns tensor memory and issues the products, one tile ahead for S so that the softmax of a tile
// overlaps the next tile's Q K^T, warps 2-5 (one per 32 lanes) run the softmax, rescale and write
// the outputs.  Hand-over by mbarriers; every wait is bounded (see common.cuh): when one gives up
// the block records KVC_DEV_TIMEOUT, stops issuing and walks to its end, waits for its loads and
// products in flight and frees its tensor memory.
//
// Slots past the valid ones hold anything, so their value rows are zeroed in shared memory before
// the product (0 * inf would not be 0); so are a drafted token's non-finite values, which are then
// added to the rows that do see the token when the output is written.
#include <mutex>

#include "tc_ops.cuh"
#include "tree_attn.cuh"

namespace kvc {

namespace tc {
PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        else
            cudaGetLastError();
    });
    return fn;
}
}  // namespace tc

namespace {

constexpr int kThreads = 192;
constexpr int kSoftmax = 128;                // softmax threads
constexpr int kBar = 1;                      // their named barrier
constexpr float kSlack = 8.f;                // lazy maximum, log2 units
constexpr int kSmemMax = 227 * 1024;

// DKP: key width padded to 64; DV: value width; RN: rows of a row tile.
template <int DKP, int DV, bool LATENT, int RN>
struct Plan {
    static constexpr int UD = DV < 128 ? 64 : 128;           // dims per ring unit
    static constexpr int TS = LATENT || DV == 256 ? 64 : 128;   // slots per tile
    static constexpr int SUB = TS * 128;                     // [TS slots][64 dims]
    static constexpr int SUBS = UD / 64;
    static constexpr int UNIT = SUBS * SUB;
    static constexpr int KU = DV / UD;                       // key units of a tile (besides rope)
    static constexpr int VU = LATENT ? 0 : KU;               // value units of their own
    static constexpr int PER = KU + VU;
    static constexpr int MB = DV / UD;                       // blocks of O^T
    static constexpr int QSUBS = DKP / 64;
    static constexpr int Q_BYTES = QSUBS * RN * 128;
    static constexpr int P_BYTES = TS / 64 * RN * 128;
    static constexpr int ROPE = LATENT ? SUB : 0;
    static constexpr int SMALL = 1024 + RN * 4;              // barriers, flags, factors
    static constexpr int FIT = (kSmemMax - 1024 - Q_BYTES - P_BYTES - ROPE - SMALL) / UNIT;
    static constexpr int NU = FIT > 16 ? 16 : FIT;           // ring units
    // S of tile t + 1 is issued before the values of tile t are used
    static_assert(NU >= 2 * KU, "ring too small");
    static constexpr int SMEM = 1024 + Q_BYTES + P_BYTES + ROPE + NU * UNIT + SMALL;
    static constexpr int O_COLS = MB * RN;
    static constexpr int USED = O_COLS + 2 * TS;
    static constexpr uint32_t COLS = USED > 256 ? 512 : 256;
    static_assert(USED <= 512, "tensor memory");
};

struct Maps {
    CUtensorMap q, k, v, kd, vd;
};

template <int DKP, int DV, bool LATENT, int RN>
__global__ void __launch_bounds__(kThreads, 1)
tree_tc_kernel(const __grid_constant__ Maps maps, const TreeParams p)
{
    using PL = Plan<DKP, DV, LATENT, RN>;
    constexpr int TS = PL::TS, NU = PL::NU, KU = PL::KU, PER = PL::PER, MB = PL::MB, UD = PL::UD;
    constexpr int SUB = PL::SUB, SUBS = PL::SUBS, UNIT = PL::UNIT;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t sQ = (raw + 1023u) & ~1023u;
    const uint32_t sP = sQ + PL::Q_BYTES;
    const uint32_t sR = sP + PL::P_BYTES;                    // rope part of the keys
    const uint32_t ring = sR + PL::ROPE;
    const uint32_t bars = ring + NU * UNIT;
    const uint32_t b_full = bars, b_empty = b_full + 8 * NU;
    const uint32_t b_rope_full = b_empty + 8 * NU, b_rope_empty = b_rope_full + 8;
    const uint32_t b_q_full = b_rope_empty + 8, b_q_empty = b_q_full + 8;
    const uint32_t b_s_full = b_q_empty + 8, b_s_empty = b_s_full + 16;
    const uint32_t b_p_full = b_s_empty + 16, b_pv = b_p_full + 8, b_done = b_pv + 8;
    const uint32_t tmem_slot = b_done + 8;
    unsigned char *small = smem_raw + (bars - raw) + 512;
    long long *s_scan = reinterpret_cast<long long *>(small);             // 10
    unsigned long long *s_nf2 = reinterpret_cast<unsigned long long *>(small + 96);
    volatile int *s_abort = reinterpret_cast<volatile int *>(small + 112);
    float *s_fac = reinterpret_cast<float *>(small + 128);                // RN
    static_assert(8 * (2 * 16 + 12) + 8 <= 512, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rt = blockIdx.x % p.RT, g = blockIdx.x / p.RT;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NU; ++i) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, 1);
        }
        mbar_init(b_rope_full, 1);
        mbar_init(b_rope_empty, 1);
        mbar_init(b_q_full, 1);
        mbar_init(b_q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_s_full + 8 * i, 1);
            mbar_init(b_s_empty + 8 * i, 4);
        }
        mbar_init(b_p_full, 4);
        mbar_init(b_pv, 1);
        mbar_init(b_done, 1);
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tc::alloc(tmem_slot, PL::COLS);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot));
    const uint32_t tO = tmem, tS = tmem + PL::O_COLS;

    pdl_trigger();
    pdl_wait();
    const TreeRange range = tree_range<kThreads>(p, g, TS, s_scan);

    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!mbar_wait_abortable(bar, parity, kMbarSpinLimit, s_abort)) {
            *s_abort = 1;
            record_code(p.dev_code, kDevCodeTimeout);
        }
    };
    // slots of tile i rounded up to the product's depth of 16 (at least one step)
    auto steps_of = [&](const TreeSeg &s, int i) {
        const int v = s.valid(p, i, TS);
        return v > 16 ? (v + 15) / 16 : 1;
    };

    unsigned n_units = 0, n_tiles = 0, n_segs = 0;           // the producer's counts (for the drain)
    if (warp == 0) {
        // ================================ loads ===================================================
        TreeWalk walk(range);
        TreeSeg s;
        const uint32_t q_bytes = (uint32_t)PL::QSUBS * (LATENT ? RN : p.RP) * 128;
        const int bx = p.table != nullptr ? min(p.bs, TS) : TS;      // rows of a cache box
        while (walk.next(p, rt, TS, s)) {
            if (s.rows <= 0) continue;
            if (lane == 0) {
                if (n_segs > 0) wait(b_q_empty, (n_segs - 1) & 1);
                if (!*s_abort) {
                    mbar_arrive_expect_tx(b_q_full, q_bytes);
                    const int y = LATENT ? s.b * p.T * p.Hq + rt * p.RP : s.kh * p.G;
                    const int z = LATENT ? 0 : s.b * p.T + rt * (p.RP / p.G);
                    for (int i = 0; i < PL::QSUBS; ++i)
                        tc::tma_4d(sQ + i * RN * 128, &maps.q, i * 64, y, z, 0, b_q_full);
                }
            }
            ++n_segs;
            for (int tile = s.lo; tile < s.hi; ++tile, ++n_tiles) {
                const bool draft = s.is_draft(p, tile);
                const int valid = s.valid(p, tile, TS);
                // page of this lane (paged caches): row of its first slot in the pool
                int page_row = 0, pages = 1;
                if (p.table != nullptr && !draft && valid > 0) {
                    pages = p.bs < TS ? (valid + p.bs - 1) / p.bs : 1;
                    if (lane < pages) {
                        const int lb = tile * TS / p.bs + lane;
                        int blk = __ldg(p.table + (size_t)s.b * p.max_blocks + lb);
                        if (blk < 0 || blk >= p.n_pool) {
                            record_code(p.dev_code, kDevBadBlockCode);
                            blk = 0;
                        }
                        page_row = (int)(((long long)s.kh * p.n_pool + blk) * p.bs) +
                                   (p.bs > TS ? tile * TS % p.bs : 0);
                    }
                }
                const int rows = draft ? 64 : bx * pages;
                if (LATENT && lane == 0) {
                    if (n_tiles > 0) wait(b_rope_empty, (n_tiles - 1) & 1);
                    if (valid == 0) mbar_arrive(b_rope_full);
                    else if (!*s_abort) {
                        mbar_arrive_expect_tx(b_rope_full, (uint32_t)rows * 128);
                        if (draft) tc::tma_4d(sR, &maps.kd, DV, 0, 0, s.b, b_rope_full);
                        else tc::tma_4d(sR, &maps.k, DV, tile * TS, 0, s.b, b_rope_full);
                    }
                }
                for (int u = 0; u < PER; ++u, ++n_units) {
                    const uint32_t slot = n_units % NU;
                    const uint32_t bar = b_full + 8 * slot, dst = ring + slot * UNIT;
                    if (lane == 0) {
                        if (n_units >= NU) wait(b_empty + 8 * slot, (n_units / NU - 1) & 1);
                        if (valid == 0) mbar_arrive(bar);
                        else if (!*s_abort) mbar_arrive_expect_tx(bar, (uint32_t)rows * 128 * SUBS);
                    }
                    __syncwarp();
                    if (valid == 0 || *s_abort) continue;
                    const bool isv = u >= KU;
                    const int x = (isv ? u - KU : u) * UD;
                    if (draft || p.table == nullptr) {
                        if (lane == 0) {
#pragma unroll
                            for (int i = 0; i < SUBS; ++i) {
                                if (draft)
                                    tc::tma_4d(dst + i * SUB, isv ? &maps.vd : &maps.kd, x + i * 64,
                                               s.kh, 0, s.b, bar);
                                else
                                    tc::tma_4d(dst + i * SUB, isv ? &maps.v : &maps.k, x + i * 64,
                                               tile * TS, s.kh, s.b, bar);
                            }
                        }
                    } else if (lane < pages) {
#pragma unroll
                        for (int i = 0; i < SUBS; ++i)
                            tc::tma_4d(dst + i * SUB + lane * bx * 128, isv ? &maps.v : &maps.k,
                                       x + i * 64, page_row, 0, 0, bar);
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp == 1) {
        // ================================ products ================================================
        if (lane == 0) {
            constexpr uint32_t id_s = tc::idesc(RN, TS, false);
            constexpr uint32_t id_o = tc::idesc(UD, RN, true);
            TreeWalk walk(range);
            TreeSeg s, nx;
            auto next_seg = [&](TreeSeg &x) {
                while (walk.next(p, rt, TS, x))
                    if (x.rows > 0) return true;
                return false;
            };
            unsigned seg_no = 0;                             // segments whose S has begun
            auto scores = [&](const TreeSeg &x, int tile, unsigned n) {
                const uint32_t buf = n & 1;
                if (n >= 2) wait(b_s_empty + 8 * buf, ((n >> 1) - 1) & 1);
                if (tile == x.lo) {
                    wait(b_q_full, seg_no & 1);
                    ++seg_no;
                }
                const uint32_t d = tS + buf * TS;
                if constexpr (LATENT) {
                    wait(b_rope_full, n & 1);
                    tc::fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc::mma(d, tc::desc_k(sQ + KU * SUBS * RN * 128 + kk * 32),
                                tc::desc_k(sR + kk * 32), id_s, kk > 0);
                    tc::commit(b_rope_empty);
                }
#pragma unroll
                for (int u = 0; u < KU; ++u) {
                    const unsigned un = n * PER + u;
                    const uint32_t slot = un % NU, src = ring + slot * UNIT;
                    wait(b_full + 8 * slot, (un / NU) & 1);
                    tc::fence_after();
#pragma unroll
                    for (int i = 0; i < SUBS; ++i)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc::mma(d, tc::desc_k(sQ + (u * SUBS + i) * RN * 128 + kk * 32),
                                    tc::desc_k(src + i * SUB + kk * 32), id_s,
                                    LATENT || u > 0 || i > 0 || kk > 0);
                    if (!LATENT) tc::commit(b_empty + 8 * slot);
                }
                tc::commit(b_s_full + 8 * buf);
                if (tile == x.hi - 1) tc::commit(b_q_empty);
            };
            unsigned n = 0;
            bool have = next_seg(s);
            int tile = have ? s.lo : 0;
            if (have) scores(s, tile, 0);
            while (have) {
                const bool more_here = tile + 1 < s.hi;
                if (more_here) scores(s, tile + 1, n + 1);
                // O^T += V^T P^T
                const int steps = steps_of(s, tile);
                wait(b_p_full, n & 1);
                tc::fence_after();
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    const unsigned un = n * PER + (LATENT ? 0 : KU) + m;
                    const uint32_t slot = un % NU, src = ring + slot * UNIT;
                    wait(b_full + 8 * slot, (un / NU) & 1);
                    tc::fence_after();
                    for (int ks = 0; ks < steps; ++ks)
                        tc::mma(tO + m * RN, tc::desc(src + ks * 2048, SUB, 1024),
                                tc::desc_k(sP + (ks >> 2) * RN * 128 + (ks & 3) * 32), id_o,
                                tile > s.lo || ks > 0);
                    tc::commit(b_empty + 8 * slot);
                }
                tc::commit(b_pv);
                ++n;
                ++tile;
                if (!more_here) {
                    have = next_seg(nx);
                    if (have) {
                        s = nx;
                        tile = s.lo;
                        scores(s, tile, n);
                    }
                }
            }
        }
    } else {
        // ================================ softmax, outputs ========================================
        const int q4 = warp & 3;                             // lanes 32 q4 .. of tensor memory
        const int tw = q4 * 32 + lane;                       // 0..127
        const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
        // the row of S (M = RN) and the dimension of O^T (M = UD) this thread's lane holds
        const int row = RN == 128 ? tw : (lane < 16 ? q4 * 16 + lane : RN);
        const int dim = UD == 128 ? tw : (lane < 16 ? q4 * 16 + lane : UD);
        const int row_lo = RN == 128 ? q4 * 32 : q4 * 16;    // first row of this warp
        TreeWalk walk(range);
        TreeSeg s;
        int4 note = make_int4(-1, 0, 0, 0);
        unsigned n = 0, seg_no = 0;
        while (walk.next(p, rt, TS, s)) {
            tree_note_split(p, range, g, s, note);
            if (s.rows <= 0) continue;
            const bool mine = row < s.rows;
            const bool any = row_lo < s.rows;                // warp-uniform
            const int r0 = rt * p.RP;
            float m = kNegBig, l = 0.f;
            bool drafts = false;
            // drafted tokens with non-finite values: alternate words, since a thread may set up
            // the next pair's while another still reads this one's
            unsigned long long *s_nf = s_nf2 + (seg_no++ & 1);
            for (int tile = s.lo; tile < s.hi; ++tile, ++n) {
                const bool draft = s.is_draft(p, tile);
                const int valid = s.valid(p, tile, TS);
                const uint32_t buf = n & 1;
                float x[TS];
                float mx = -INFINITY;
                wait(b_s_full + 8 * buf, (n >> 1) & 1);
                tc::fence_after();
                if (any) {
#pragma unroll
                    for (int c = 0; c < TS; c += 32) tc::ld32(tS + buf * TS + lanes + c, x + c);
                    tc::wait_ld();
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_s_empty + 8 * buf);
                if (any) {
#pragma unroll
                    for (int c = 0; c < TS; ++c) x[c] *= p.scale_log2;
                    if (draft) {
                        const uint64_t see =
                            mine ? tree_mask_word(p, s.b, (r0 + row) / p.G, s.cnt) : 0ull;
#pragma unroll
                        for (int c = 0; c < TS; ++c)
                            if (c >= 64 || !((see >> (c & 63)) & 1ull)) x[c] = -INFINITY;
                    } else if (valid < TS) {
#pragma unroll
                        for (int c = 0; c < TS; ++c)
                            if (c >= valid) x[c] = -INFINITY;
                    }
                    float a0 = x[0], a1 = x[1], a2 = x[2], a3 = x[3];
#pragma unroll
                    for (int c = 4; c < TS; c += 4) {
                        a0 = fmaxf(a0, x[c]);
                        a1 = fmaxf(a1, x[c + 1]);
                        a2 = fmaxf(a2, x[c + 2]);
                        a3 = fmaxf(a3, x[c + 3]);
                    }
                    mx = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3));
                }
                if (draft && tw == 0) *s_nf = 0ull;          // ordered by the barrier below
                if (tc::bar_any(kBar, kSoftmax, mine && mx > m + kSlack)) {
                    const float m_new = fmaxf(m, mx);
                    const float f = ex2(m - m_new);
                    m = m_new;
                    l *= f;
                    if (tile > s.lo) {
                        if (row < RN) s_fac[row] = f;
                        wait(b_pv, (n - 1) & 1);
                        tc::fence_after();
                        tc::bar_sync(kBar, kSoftmax);
#pragma unroll 1
                        for (int c = 0; c < MB * RN; c += 32) {
                            if ((c & (RN - 1)) >= s.rows) continue;
                            float o[32];
                            tc::ld32(tO + lanes + c, o);
                            tc::wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] *= s_fac[(c & (RN - 1)) + j];
                            tc::st32(tO + lanes + c, o);
                        }
                        tc::wait_st();
                    }
                }
                if (any) {
#pragma unroll
                    for (int c = 0; c < TS; ++c) {
                        x[c] = ex2(x[c] - m);
                        l += x[c];
                    }
                }
                if (n > 0) wait(b_pv, (n - 1) & 1);          // P of the previous tile is used up
                if (any && row < RN) {
#pragma unroll
                    for (int c = 0; c < TS / 8; ++c) {       // 16-byte chunks of the row
                        const float *y = x + 8 * c;
                        tc::st_shared_16(sP + (c >> 3) * RN * 128 + row * 128 +
                                             (((c & 7) ^ (row & 7)) << 4),
                                         tc::pack_bf16(y[0], y[1]), tc::pack_bf16(y[2], y[3]),
                                         tc::pack_bf16(y[4], y[5]), tc::pack_bf16(y[6], y[7]));
                    }
                }
                // value rows past the valid ones, and a drafted token's non-finite values
                const int depth = steps_of(s, tile) * 16;
                if (valid < depth || draft) {
                    for (int u = 0; u < MB; ++u) {
                        const unsigned un = n * PER + (LATENT ? 0 : KU) + u;
                        const uint32_t slot = un % NU;
                        wait(b_full + 8 * slot, (un / NU) & 1);
                        unsigned char *base = smem_raw + (ring + slot * UNIT - raw);
                        for (int i = tw; i < SUBS * (depth - valid) * 8; i += kSoftmax) {
                            const int sub = i / ((depth - valid) * 8), k = i % ((depth - valid) * 8);
                            *reinterpret_cast<uint4 *>(base + sub * SUB + valid * 128 + k * 16) =
                                make_uint4(0, 0, 0, 0);
                        }
                        if (draft) {
                            for (int i = tw; i < SUBS * valid * 8; i += kSoftmax) {
                                const int sub = i / (valid * 8), k = i % (valid * 8);
                                uint4 *at = reinterpret_cast<uint4 *>(base + sub * SUB + k * 16);
                                uint4 w = *at;
                                uint32_t bad = 0;
                                auto fix = [&](uint32_t y) {
                                    if ((y & 0x7f80u) == 0x7f80u) y &= 0xffff0000u, bad = 1;
                                    if ((y & 0x7f800000u) == 0x7f800000u) y &= 0xffffu, bad = 1;
                                    return y;
                                };
                                w.x = fix(w.x); w.y = fix(w.y); w.z = fix(w.z); w.w = fix(w.w);
                                if (bad) {
                                    *at = w;
                                    atomicOr(s_nf, 1ull << (k >> 3));
                                }
                            }
                        }
                    }
                    drafts |= draft;
                }
                tc::fence_async();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_p_full);
            }
            // this part's outputs: O^T / l, or the partial state
            const bool whole = s.whole();
            const size_t part = (size_t)blockIdx.x * 2 + (s.first ? 0 : 1);
            if (mine) {
                const int t = (r0 + row) / p.G, h = s.kh * p.G + (r0 + row) % p.G;
                if (!whole) {
                    p.ws_ml[(part * RN + row) * 2] = m;
                    p.ws_ml[(part * RN + row) * 2 + 1] = l;
                } else if (p.lse != nullptr) {
                    p.lse[((size_t)s.b * p.T + t) * p.Hq + h] =
                        l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
                }
            }
            wait(b_pv, (n - 1) & 1);                         // every warp is past its last rescaling
            tc::fence_after();
            if (row < RN) s_fac[row] = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
            tc::bar_sync(kBar, kSoftmax);
            const unsigned long long nf = drafts ? *s_nf : 0ull;
#pragma unroll 1
            for (int c = 0; c < MB * RN; c += 32) {
                const int ra = c & (RN - 1);                 // first row of these columns
                if (ra >= s.rows) continue;
                const int d = c / RN * UD + dim;
                float o[32];
                tc::ld32(tO + lanes + c, o);
                tc::wait_ld();
                if (dim >= UD) continue;
                int t = (r0 + ra) / p.G, hg = (r0 + ra) % p.G;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (ra + j < s.rows) {
                        float y = o[j] * s_fac[ra + j];
                        if (nf) {
                            unsigned long long hit = nf & tree_mask_word(p, s.b, t, s.cnt);
                            while (hit) {
                                const int i = __ffsll((long long)hit) - 1;
                                hit &= hit - 1;
                                const float z = __bfloat162float(
                                    static_cast<const __nv_bfloat16 *>(
                                        p.vd)[(((size_t)s.b * p.T + i) * p.Hkv + s.kh) * p.DK + d]);
                                if (!(fabsf(z) <= 3.402823466e38f)) y += z;
                            }
                        }
                        if (whole) {
                            const size_t at = ((size_t)s.b * p.T + t) * p.Hq + s.kh * p.G + hg;
                            static_cast<__nv_bfloat16 *>(p.out)[at * DV + d] = __float2bfloat16(y);
                        } else {
                            p.ws_o[(part * RN + ra + j) * DV + d] = y;
                        }
                    }
                    if (++hg == p.G) {
                        hg = 0;
                        ++t;
                    }
                }
            }
            tc::fence_before();
        }
        if (rt == 0 && tw == 0) p.ws_info[g] = note;
    }

    tc::fence_before();
    __syncthreads();
    // after a wait ran out: the loads in flight have landed and the products issued have completed
    // before the block frees tensor memory and exits
    if (*s_abort) {
        if (threadIdx.x == 0) {
            auto drain = [&](uint32_t bar, uint32_t parity) {
                mbar_wait_ok(bar, parity, kMbarSpinLimit >> 4);
            };
            for (unsigned i = n_units > NU ? n_units - NU : 0; i < n_units; ++i)
                drain(b_full + 8 * (i % NU), (i / NU) & 1);
            if (LATENT && n_tiles > 0) drain(b_rope_full, (n_tiles - 1) & 1);
            if (n_segs > 0) drain(b_q_full, (n_segs - 1) & 1);
        } else if (threadIdx.x == 32) {
            tc::commit(b_done);
            mbar_wait_ok(b_done, 0, kMbarSpinLimit);
        }
        __syncthreads();
    }
    tc::fence_after();
    if (warp == 1) tc::dealloc(tmem, PL::COLS);
}

template <int DKP, int DV, bool LATENT, int RN>
cudaError_t launch_typed(const TreeParams &p, const Maps &maps, cudaStream_t stream)
{
    using PL = Plan<DKP, DV, LATENT, RN>;
    static bool configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !configured[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(tree_tc_kernel<DKP, DV, LATENT, RN>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, PL::SMEM);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    return launch_pdl(tree_tc_kernel<DKP, DV, LATENT, RN>, dim3((unsigned)(p.groups * p.RT)),
                      dim3(kThreads), PL::SMEM, stream, maps, p);
}

int tile_slots(int D) { return D == 256 ? 64 : 128; }

}  // namespace

bool tree_tc_pages(int bs, int D)
{
    const int TS = tile_slots(D);
    return bs % 8 == 0 && (TS % bs == 0 || bs % TS == 0);
}

cudaError_t launch_tree_attn_tc(const TreeParams &p, cudaStream_t stream, bool *used)
{
    *used = false;
    Maps maps;
    const uint64_t dk = (uint64_t)p.DK, row = dk * 2;
    const uint64_t B = p.B, T = p.T, Hq = p.Hq, Hkv = p.Hkv;
    const int TS = p.latent ? 64 : tile_slots(p.DV);
    if (B * T * Hq > 0x7fffffffull) return cudaSuccess;
    bool ok = p.latent ? tc::encode_4d(&maps.q, p.q, {dk, B * T * Hq, 1, 1},
                                       {row, row * B * T * Hq, row * B * T * Hq}, p.RN, 1)
                       : tc::encode_4d(&maps.q, p.q, {dk, Hq, B * T, 1},
                                       {row, row * Hq, row * Hq * B * T}, p.G, p.RP / p.G);
    auto cache = [&](CUtensorMap *m, const void *ptr) {
        if (p.table != nullptr) {
            const uint64_t rows = Hkv * (uint64_t)p.n_pool * p.bs;
            if (rows > 0x7fffffffull) return false;
            return tc::encode_4d(m, ptr, {dk, rows, 1, 1}, {row, row * rows, row * rows},
                                 p.bs < TS ? p.bs : TS, 1);
        }
        const uint64_t sh = p.latent ? row : (uint64_t)p.sh * 2;
        return tc::encode_4d(m, ptr, {dk, (uint64_t)p.cap, Hkv, B},
                             {(uint64_t)p.ss * 2, sh, (uint64_t)p.sb * 2}, TS, 1);
    };
    auto drafted = [&](CUtensorMap *m, const void *ptr) {
        return tc::encode_4d(m, ptr, {dk, Hkv, T, B}, {row, row * Hkv, row * Hkv * T}, 1, 64);
    };
    ok = ok && cache(&maps.k, p.k);
    maps.v = maps.kd = maps.vd = maps.k;
    if (ok && !p.latent) ok = cache(&maps.v, p.v);
    if (ok && p.kd != nullptr) {
        ok = drafted(&maps.kd, p.kd);
        if (ok && !p.latent) ok = drafted(&maps.vd, p.vd);
    }
    if (!ok) return cudaSuccess;
    *used = true;
    if (p.latent) {
        switch (p.DV) {
        case 128: return launch_typed<192, 128, true, 64>(p, maps, stream);
        case 256: return launch_typed<320, 256, true, 64>(p, maps, stream);
        default: return launch_typed<576, 512, true, 64>(p, maps, stream);
        }
    }
    const bool wide = p.RN == 128;
    switch (p.DV) {
    case 64:
        return wide ? launch_typed<64, 64, false, 128>(p, maps, stream)
                    : launch_typed<64, 64, false, 64>(p, maps, stream);
    case 128:
        return wide ? launch_typed<128, 128, false, 128>(p, maps, stream)
                    : launch_typed<128, 128, false, 64>(p, maps, stream);
    default:
        return wide ? launch_typed<256, 256, false, 128>(p, maps, stream)
                    : launch_typed<256, 256, false, 64>(p, maps, stream);
    }
}

}  // namespace kvc

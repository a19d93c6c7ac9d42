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
//   are off by at most 2^-8 each, as is the bf16 output, and errors against 64 bits are 0.0018 to
//   0.0023 of the outputs' norm where rounding the output alone makes 0.0017.  Carrying the rest of a
//   weight as a second bf16 term, as the single-token decode does, would double the values' products
//   and P's room: with 128 rows tensor memory is full as it is, and latent rows are bound by what
//   shared memory delivers.  The sum l is taken of the unrounded weights, so lse has no part in it.
//   With 128 rows of an ordinary cache of up to 128 dims (PT below) O is kept by row instead and P
//   goes through tensor memory as the A operand (O += P V): that leaves shared memory for a third
//   tile in flight, a row's O is in its own thread's lane, and two P buffers let the softmax of two
//   tiles run side by side.  16 pairs of 131072 slots, 256 rows each, 128 dims: 258 us, without
//   it 265.  With 256 dims (64-slot tiles, short budgets) it was the slower one, 36 us for 31 when it
//   was tried.
//   A latent cache's tile is loaded once and serves as K (all of it) and V (its first d_latent
//   columns).
//   The running maximum is lazy: a tile whose logits stay below max + 8 (log2 units) keeps the old
//   reference, so P stays below 2^8 and O is rescaled only when the maximum really rises.
//
// Roles: warp 0 (and 3, for latent rows) issues TMA loads into a ring of units (up to 128 dims x TS
// slots); warp 1 issues S = Q K^T, two S buffers ahead of the softmax, and owns tensor memory; warp 2
// issues the values' products; the others (sets of four, one warp per 32 lanes and 32 of a tile's
// slots each, or one tile in two with PT) run the softmax, rescale and write the outputs.  Hand-over
// by mbarriers; every wait is bounded (see common.cuh).  When one gives up the block records
// KVC_DEV_TIMEOUT and loads no further tile.  No wait holds a warp any more then: all of them walk to
// their ends on whatever memory holds (the products go on; what the softmax warps do between their
// named barriers is decided by all of them together, so they stay in step), and the block waits for
// its loads and products in flight and frees its tensor memory.
//
// Measured, device time: 32 pairs of 5243 slots, 64 rows, 128 dims 29 us (HBM alone 13; a block has
// nine tiles, so the start, 5 us until its first keys, and the merge, 5 us, count as much as the
// stream); 512 paged pairs of 817 slots, 8 rows 57 us (33); 16 pairs of 131072 slots, 256 rows 258 us
// (161; 8.5 TB/s from L2 to the SMs); 32 latent sequences of 4608 slots, 32 rows 45 us (26); 8 of
// 6144 slots, 512 rows in eight row tiles 80 us (28 by the products' operations; shared memory moves
// 320 KB for a tile of 64 slots by 64 rows, which at 128 B a clock is 56 us alone).
//
// Slots past the valid ones hold anything, so their value rows are zeroed in shared memory before
// the product (0 * inf would not be 0); so are a drafted token's non-finite values, which are then
// added to the rows that do see the token when the output is written.
#include <mutex>
#include <type_traits>

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

constexpr int kBar = 1;                      // their named barrier
constexpr float kSlack = 8.f;                // lazy maximum, log2 units
// Weights are exp2(fma(s, scale, -m)).  m is a rounded product and s * scale in the fma is not, so they
// differ by up to half of m's last place even at the maximum: with m = 2^32 a weight could be 2^128.
// From here on (half a unit) the products are rounded first, which leaves 0 at the maximum.  That takes
// the way of the masked tiles, so that other tiles have no further branch (one: 260 -> 272 us for 16
// pairs of 131072 slots, 256 rows).
constexpr float kBigMax = 16777216.f;
constexpr int kSmemMax = 227 * 1024;

// DKP: key width padded to 64; DV: value width; RN: rows of a row tile.
template <int DKP, int DV, bool LATENT, int RN>
struct Plan {
    static constexpr int SM = RN < 64 ? 64 : RN;             // M of S (rows past RN: not used)
    static constexpr int UD = DV < 128 ? 64 : 128;           // dims per ring unit
    static constexpr int TS = LATENT || DV == 256 ? 64 : 128;   // slots per tile
    static constexpr bool PT = RN == 128 && DV <= 128 && !LATENT;   // P in tensor memory, O by row
    static constexpr int SETS = PT ? 2 : TS / 32;            // softmax sets of four warps
    static constexpr int SOFTMAX = 128 * SETS;               // softmax threads
    static constexpr int CONTROL = LATENT ? 4 : 3;           // loading and issuing warps come first
    static constexpr int THREADS = 32 * CONTROL + SOFTMAX;
    static constexpr int SUB = TS * 128;                     // [TS slots][64 dims]
    static constexpr int SUBS = UD / 64;
    static constexpr int UNIT = SUBS * SUB;
    static constexpr int KU = DV / UD;                       // key units of a tile (besides rope)
    static constexpr int VU = LATENT ? 0 : KU;               // value units of their own
    static constexpr int PER = KU + VU;
    static constexpr int MB = DV / UD;                       // blocks of O^T
    static constexpr int QSUBS = DKP / 64;
    static constexpr int Q_BYTES = QSUBS * RN * 128;
    static constexpr int P_BYTES = PT ? 0 : TS / 64 * RN * 128;
    static constexpr int ROPE = LATENT ? 2 * SUB : 0;        // two tiles' rope parts
    static constexpr int SMALL = 640 + (PT ? 2 : 1 + SETS) * RN * 4;         // barriers, flags, row values
    static constexpr int FIT = (kSmemMax - 1024 - Q_BYTES - P_BYTES - ROPE - SMALL) / UNIT;
    static constexpr int NU = FIT > 16 ? 16 : FIT;           // ring units
    // A latent tile's copies complete on one barrier (its units are keys and values at once), ring
    // of NTB; other caches' units have a barrier each.
    static constexpr int NTB = LATENT ? (NU + KU - 1) / KU + 1 : NU;
    // the next tile's keys arrive while a tile's values are still needed
    static_assert(NU >= 2 * KU, "ring too small");
    static constexpr int SMEM = 1024 + Q_BYTES + P_BYTES + ROPE + NU * UNIT + SMALL;
    static constexpr int O_COLS = PT ? DV : MB * RN;
    static constexpr int USED = O_COLS + 2 * TS + (PT ? TS : 0);
    static constexpr uint32_t COLS = USED > 256 ? 512 : 256;
    static_assert(USED <= 512, "tensor memory");
};

// Rows are seen as [sub][64]: dimensions {64, slot, sub, head, sequence} for the caches and the
// drafted rows, {64, head, token, sub} for tree queries and {64, row, sub} for latent ones, so one
// copy brings all 64-element pieces of a unit.  r*: the rope parts of a latent cache's rows
// (q, cache, drafts), widths below 64 filled with zeros.
struct Maps {
    CUtensorMap q, k, v, kd, vd, rq, rk, rd;
};

// The values that are not finite among the drafted tokens that row r of the row tile sees (nf: the
// tokens that have some), added as they are to what this thread wrote of dimension d of the row: such
// a value leaves nothing else of it.  Hardly ever called, so kept out of the loop that writes.
template <int RN, int DV>
__device__ __forceinline__ void add_stray(const TreeParams &p, const TreeSeg &s, size_t part, int r0, int r,
                                          int d, unsigned long long nf)
{
    const int tok = (r0 + r) / p.G, h = s.kh * p.G + (r0 + r) - tok * p.G;
    const long long stride = (long long)p.Hkv * p.DK;
    const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.vd) + (size_t)s.b * p.T * stride +
                             (size_t)s.kh * p.DK + d;
    float y = 0.f;
    for (unsigned long long hit = nf & tree_mask_word(p, s.b, tok, s.cnt); hit; hit &= hit - 1) {
        const float z = __bfloat162float(v[(__ffsll((long long)hit) - 1) * stride]);
        if (!(fabsf(z) <= 3.402823466e38f)) y += z;
    }
    if (y == 0.f) return;
    if (s.whole()) {
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + (((size_t)s.b * p.T + tok) * p.Hq + h) * DV + d;
        *o = __float2bfloat16(__bfloat162float(*o) + y);
    } else {
        p.ws_o[(part * RN + r) * DV + d] += y;
    }
}

// Zeroes the value rows [valid, depth) of a unit and, in the drafted tokens' tile, every value that
// is not finite (its row goes into *nf).  Called by `warps` warps, w the caller's number: a warp
// takes a row, eight lanes per 64 dims.
template <int SUBS, int SUB>
__device__ __forceinline__ void clean_unit(unsigned char *base, int w, int warps, int valid, int depth,
                                           bool draft, unsigned long long *nf)
{
    const int lane = threadIdx.x & 31, sub = lane >> 3;
    if (sub >= SUBS) return;
    uint4 *at = reinterpret_cast<uint4 *>(base + sub * SUB + (lane & 7) * 16);
    for (int r = valid + w; r < depth; r += warps) at[r * 8] = make_uint4(0, 0, 0, 0);
    if (!draft) return;
    for (int r = w; r < valid; r += warps) {
        uint4 x = at[r * 8];
        uint32_t bad = 0;
        auto fix = [&](uint32_t y) {
            if ((y & 0x7f80u) == 0x7f80u) y &= 0xffff0000u, bad = 1;
            if ((y & 0x7f800000u) == 0x7f800000u) y &= 0xffffu, bad = 1;
            return y;
        };
        x.x = fix(x.x); x.y = fix(x.y); x.z = fix(x.z); x.w = fix(x.w);
        if (bad) {
            at[r * 8] = x;
            atomicOr(nf, 1ull << r);
        }
    }
}

template <int DKP, int DV, bool LATENT, int RN>
__global__ void __launch_bounds__(Plan<DKP, DV, LATENT, RN>::THREADS, 1)
tree_tc_kernel(const __grid_constant__ Maps maps, const TreeParams p)
{
    using PL = Plan<DKP, DV, LATENT, RN>;
    constexpr int TS = PL::TS, NU = PL::NU, KU = PL::KU, PER = PL::PER, MB = PL::MB, UD = PL::UD;
    constexpr int kSets = PL::SETS, kSoftmax = PL::SOFTMAX;
    constexpr int SUB = PL::SUB, SUBS = PL::SUBS, UNIT = PL::UNIT;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t sQ = (raw + 1023u) & ~1023u;
    const uint32_t sP = sQ + PL::Q_BYTES;
    const uint32_t sR = sP + PL::P_BYTES;                    // rope part of the keys
    const uint32_t ring = sR + PL::ROPE;
    const uint32_t bars = ring + NU * UNIT;
    constexpr int NTB = PL::NTB;
    const uint32_t b_full = bars, b_empty = b_full + 8 * NTB;
    const uint32_t b_rope_empty = b_empty + 8 * NU;
    const uint32_t b_q_full = b_rope_empty + 16, b_q_empty = b_q_full + 8;
    const uint32_t b_s_full = b_q_empty + 8;
    const uint32_t b_p_full = b_s_full + 16, b_pv = b_p_full + 16, b_done = b_pv + 16;
    const uint32_t tmem_slot = b_done + 8;
    unsigned char *small = smem_raw + (bars - raw) + 512;
    unsigned long long *s_nf2 = reinterpret_cast<unsigned long long *>(small);
    volatile int *s_abort = reinterpret_cast<volatile int *>(small + 16);
    float *s_fac = reinterpret_cast<float *>(small + 128);                // RN
    float *s_row = s_fac + RN;                                            // [kSets][RN]
    static_assert(8 * (NTB + NU + 11) + 8 <= 512, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rt = blockIdx.x % p.RT, g = blockIdx.x / p.RT;
    if (warp == 2 && lane < 8) tc::prefetch_map(&maps.q + lane);
    if (threadIdx.x == 0) {
        for (int i = 0; i < NTB; ++i) mbar_init(b_full + 8 * i, 1);
        for (int i = 0; i < NU; ++i) mbar_init(b_empty + 8 * i, 1);
        mbar_init(b_q_full, 1);
        mbar_init(b_q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_rope_empty + 8 * i, 1);
            mbar_init(b_s_full + 8 * i, 1);
            mbar_init(b_p_full + 8 * i, PL::PT ? 4 : 4 * kSets);
            mbar_init(b_pv + 8 * i, 1);
        }
        mbar_init(b_done, 2);
        *s_abort = p.starve;                     // (test hook: as if a wait had given up already)
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tc::alloc(tmem_slot, PL::COLS);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot));
    const uint32_t tO = tmem, tS = tmem + PL::O_COLS, tP = tS + 2 * TS;

    pdl_trigger();
    pdl_wait();
    const TreeRange range = tree_range(p, g, TS);

    const bool rope = LATENT && p.DK > DV;                   // the keys have a rope part
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!mbar_wait_abortable(bar, parity, kMbarSpinLimit, s_abort)) {
            *s_abort = 1;
            record_code(p.dev_code, kDevCodeTimeout);
        }
    };
    // slots of tile i rounded up to the product's depth of 16 (at least one step); all of them with
    // PT, where the issuing warp's instructions count for more than a last tile's products
    auto steps_of = [&](const TreeSeg &s, int i) {
        if constexpr (PL::PT) return TS / 16;
        const int v = s.valid(p, i, TS);
        return v > 16 ? (v + 15) / 16 : 1;
    };

    // Warp 0 loads, and the second half of a latent tile's units warp 3 (a unit takes a warp some 400
    // clocks: 128 heads 84 -> 80 us; the keys and values of other caches from two warps came out slower,
    // 260 us for 254 and 60 for 57).
    constexpr int FIRST = LATENT ? (PER + 1) / 2 : PER;      // warp 0's
    const int u_lo = warp == 0 ? 0 : FIRST, u_hi = warp == 0 ? FIRST : PER;
    unsigned n_tiles = 0, n_segs = 0;                        // their counts (for the drain)
    if (warp == 0 || (LATENT && warp == 3)) {
        // ================================ loads ===================================================
        TreeWalk walk(p, range);
        TreeSeg s;
        const bool paged = p.table != nullptr;
        const int bx = paged ? min(p.bs, TS) : TS;           // slots of a cache copy
        uint32_t slot = u_lo, ph = 1, t_slot = 0;            // ring positions
        auto step = [&](uint32_t by) {
            slot += by;
            if (slot >= NU) {
                slot -= NU;
                ph ^= 1;
            }
        };
        // A pair's queries replace the last pair's once its last S is complete.  Their load is held
        // back until then while the pair's tiles go on filling the ring: waiting for the queries'
        // place first left HBM idle at each change of pair (a block that changed pairs took 27 us
        // where the others took 22).
        bool queries = false;                                // this pair's are still to be loaded
        TreeNote note;
        auto load_q = [&] {
            queries = false;
            ++n_segs;
            if (!*s_abort && tc::elect()) {
                if constexpr (LATENT) {
                    const int y = s.b * p.T * p.Hq + rt * RN;
                    mbar_arrive_expect_tx(b_q_full, (uint32_t)(KU * SUBS + (rope ? 1 : 0)) * RN * 128);
                    tc::tma_5d(sQ, &maps.q, 0, y, 0, 0, 0, b_q_full);
                    if (rope) tc::tma_5d(sQ + KU * SUBS * RN * 128, &maps.rq, 0, y, 0, 0, 0, b_q_full);
                } else {
                    const int t0 = s.b * p.T + rt * (p.RP / p.G);
                    mbar_arrive_expect_tx(b_q_full, (uint32_t)PL::QSUBS * p.RP * 128);
#pragma unroll
                    for (int i = 0; i < PL::QSUBS; ++i)
                        tc::tma_5d(sQ + i * RN * 128, &maps.q, 0, s.kh * p.G, t0, i, 0, b_q_full);
                }
            }
            __syncwarp();
        };
        auto seen = [&](uint32_t bar, uint32_t parity) {
            return __shfl_sync(0xffffffffu, (int)tc::test(bar, parity), 0) != 0;
        };
        // the place of a ring unit, loading the queries meanwhile if theirs comes first
        auto wait_unit = [&](uint32_t bar, uint32_t parity) {
            for (uint32_t it = 0; queries && it < kMbarSpinLimit; ++it) {
                if (seen(b_q_empty, (n_segs - 1) & 1)) load_q();
                else if (seen(bar, parity) || __shfl_sync(0xffffffffu, *s_abort, 0)) return;
            }
            wait(bar, parity);
        };
        while (walk.next(p, rt, TS, s)) {
            if (s.rows <= 0) continue;
            queries = warp == 0;
            if (queries && n_segs == 0) load_q();
            note.see(range, s);
            for (int tile = s.lo; tile < s.hi; ++tile, ++n_tiles) {
                const bool draft = s.is_draft(p, tile);
                const int valid = s.valid(p, tile, TS);
                const int y = draft ? 0 : tile * TS;
                // page of this lane (paged caches): row of its first slot in the pool
                int page_row = 0, pages = 1;
                const bool by_page = paged && !draft;
                if (by_page) {
                    pages = p.bs < TS ? (valid + p.bs - 1) / p.bs : 1;
                    if (lane < pages && valid > 0) {
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
                const bool go = !*s_abort;
                const uint32_t bytes = (draft ? TS : bx * pages) * 128u;   // of a 64-wide piece
                uint32_t bar = b_full + 8 * t_slot;          // latent: one barrier for the tile
                if constexpr (LATENT) {
                    const uint32_t r = n_tiles & 1;
                    if (warp == 0) {
                        if (rope && n_tiles >= 2) wait_unit(b_rope_empty + 8 * r, ((n_tiles >> 1) - 1) & 1);
                        if (go && tc::elect()) {
                            if (valid == 0) mbar_arrive(bar);
                            else {
                                mbar_arrive_expect_tx(bar, bytes * (KU * SUBS + (rope ? 1 : 0)));
                                if (rope)
                                    tc::tma_5d(sR + r * SUB, draft ? &maps.rd : &maps.rk, 0, y, 0, 0, s.b, bar);
                            }
                        }
                        __syncwarp();
                    }
                    if (++t_slot == NTB) t_slot = 0;
                }
#pragma unroll 1
                for (int u = u_lo; u < u_hi; ++u) {
                    const uint32_t dst = ring + slot * UNIT;
                    if (!LATENT) bar = b_full + 8 * slot;
                    const bool isv = u >= KU;
                    const int sub = (isv ? u - KU : u) * SUBS;
                    if (n_tiles * PER + u >= NU) wait_unit(b_empty + 8 * slot, ph);
                    if (go && tc::elect()) {
                        if (!LATENT) {
                            if (valid == 0) mbar_arrive(bar);
                            else mbar_arrive_expect_tx(bar, bytes * SUBS);
                        }
                        if (valid > 0 && !by_page)
                            tc::tma_5d(dst, draft ? (isv ? &maps.vd : &maps.kd) : (isv ? &maps.v : &maps.k),
                                       0, y, sub, s.kh, s.b, bar);
                    }
                    __syncwarp();
                    if (by_page && go && valid > 0) {
                        for (int i = 0; i < pages; ++i) {
                            const int row = __shfl_sync(0xffffffffu, page_row, i);
                            if (tc::elect()) {
#pragma unroll
                                for (int c = 0; c < SUBS; ++c)
                                    tc::tma_5d(dst + c * SUB + i * bx * 128, isv ? &maps.v : &maps.k, 0,
                                               row, sub + c, 0, 0, bar);
                            }
                            __syncwarp();
                        }
                    }
                    step(1);
                }
                step(PER - (u_hi - u_lo));
            }
            if (queries) {
                wait(b_q_empty, (n_segs - 1) & 1);
                load_q();
            }
        }
        if (warp == 0 && rt == 0 && lane == 0) p.ws_info[g] = note.get(range);
    } else if (warp < 3) {
        // ================================ products ================================================
        // Warp 1 issues S = Q K^T, warp 2 the values' products; what orders them are the barriers
        // between each and the softmax.  (One warp for both left the tensor cores waiting for it: a
        // step takes an issuing warp some 600 clocks besides the products themselves.)
        TreeWalk walk(p, range);
        TreeSeg s, nx;
        auto next_seg = [&] {
            while (walk.next(p, rt, TS, nx))
                if (nx.rows > 0) return true;
            return false;
        };
        auto step = [&](uint32_t &slot, uint32_t &ph, uint32_t by, uint32_t size) {
            slot += by;
            if (slot >= size) {
                slot -= size;
                ph ^= 1;
            }
        };
        unsigned n = 0;
        uint32_t slot = LATENT || warp == 1 ? 0 : KU, ph = 0;         // ring position
        uint32_t t_slot = 0, t_ph = 0;                                // latent: tile barriers
        uint32_t src[KU], bar[KU];                                    // (a tile has KU value units too)
        // The next COUNT units have arrived, and one more barrier has completed.  Looks at all of them
        // at once first, since a wait for one that has long completed takes some 200 clocks.  A latent
        // tile has one barrier, which its values need not look at: the weights came after its S.
        auto take = [&](auto COUNT, uint32_t more, uint32_t more_ph) {
            bool in = tc::test(more, more_ph);
            uint32_t at = slot, at_ph = ph;
            if (LATENT && warp == 1) in &= tc::test(b_full + 8 * t_slot, t_ph);
#pragma unroll
            for (int u = 0; u < COUNT; ++u) {
                if (!LATENT) in &= tc::test(b_full + 8 * at, at_ph);
                src[u] = ring + at * UNIT;
                bar[u] = b_empty + 8 * at;
                step(at, at_ph, 1, NU);
            }
            if (!__all_sync(0xffffffffu, in)) {
                if constexpr (LATENT) {
                    if (warp == 1) wait(b_full + 8 * t_slot, t_ph);
                } else {
#pragma unroll 1
                    for (int u = 0; u < COUNT; ++u) {
                        wait(b_full + 8 * slot, ph);
                        step(slot, ph, 1, NU);
                    }
                }
                wait(more, more_ph);
                __syncwarp();
            }
            slot = at;
            ph = at_ph;
            if (LATENT && warp == 1) step(t_slot, t_ph, 1, NTB);
            tc::fence_after();
        };
        bool any = next_seg();
        if (warp == 1) {
            constexpr uint32_t id_s = tc::idesc(PL::SM, TS, false);
            const tc::Desc dq = tc::desc_k(sQ);
            unsigned seg_no = 0;
            while (any) {
                s = nx;
                wait(b_q_full, seg_no & 1);
                ++seg_no;
                for (int tile = s.lo; tile < s.hi; ++tile, ++n) {
                    const uint32_t buf = n & 1, d = tS + buf * TS;
                    // As each unit arrives, or a latent tile's together (a row tile of 128 heads 84 us,
                    // by units 87).  The S buffer has been read: the weights of the tile before last
                    // came from it.
                    constexpr int AT_ONCE = LATENT ? KU : 1;
#pragma unroll
                    for (int u0 = 0; u0 < KU; u0 += AT_ONCE) {
                        using Count = std::integral_constant<int, AT_ONCE>;
                        if (n >= 2) take(Count{}, b_p_full + 8 * buf, ((n >> 1) - 1) & 1);
                        else take(Count{}, b_q_full, (seg_no - 1) & 1);
                        if (tc::elect()) {
                            if (rope && u0 == 0) {
                                const tc::Desc dr = tc::desc_k(sR + buf * SUB);
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    tc::mma(d, dq + (KU * SUBS * RN * 128 + kk * 32), dr + kk * 32, id_s, kk > 0);
                                tc::commit(b_rope_empty + 8 * buf);
                            }
#pragma unroll
                            for (int u = u0; u < u0 + AT_ONCE; ++u) {
                                const tc::Desc dk = tc::desc_k(src[u - u0]);
#pragma unroll
                                for (int i = 0; i < SUBS; ++i)
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk)
                                        tc::mma(d, dq + ((u * SUBS + i) * RN * 128 + kk * 32),
                                                dk + (i * SUB + kk * 32), id_s,
                                                rope || u > 0 || i > 0 || kk > 0);
                                if (!LATENT) tc::commit(bar[u - u0]);
                            }
                            if (u0 + AT_ONCE == KU) {
                                tc::commit(b_s_full + 8 * buf);
                                if (tile == s.hi - 1) tc::commit(b_q_empty);
                            }
                        }
                        __syncwarp();
                    }
                    if (!LATENT) step(slot, ph, KU, NU);                  // past the values
                    if (tile == s.lo) any = next_seg();               // (its lengths arrive meanwhile)
                }
            }
        } else {
            // O^T += V^T P^T, or O += P V
            constexpr uint32_t id_o = PL::PT ? tc::idesc_b_mn(RN, UD) : tc::idesc(UD, RN, true);
            const tc::Desc dp = tc::desc_k(sP);
            while (any) {
                s = nx;
                for (int tile = s.lo; tile < s.hi; ++tile, ++n) {
                    const int steps = steps_of(s, tile);
                    take(std::integral_constant<int, KU>{}, b_p_full + 8 * (n & 1), (n >> 1) & 1);
                    if (!LATENT) step(slot, ph, KU, NU);              // past the next tile's keys
                    if (tc::elect()) {
#pragma unroll
                        for (int m = 0; m < MB; ++m) {
                            const tc::Desc dv = tc::desc(src[m], SUB, 1024);
#pragma unroll
                            for (int ks = 0; ks < TS / 16; ++ks)
                                if (ks < steps) {
                                    if constexpr (PL::PT)
                                        tc::mma_ta(tO + m * UD, tP + (n & 1) * (TS / 2) + ks * 8, dv + ks * 2048,
                                                   id_o, tile > s.lo || ks > 0);
                                    else
                                        tc::mma(tO + m * RN, dv + ks * 2048,
                                                dp + ((ks >> 2) * RN * 128 + (ks & 3) * 32), id_o,
                                                tile > s.lo || ks > 0);
                                }
                            tc::commit(bar[m]);
                        }
                        tc::commit(b_pv + (PL::PT ? 8 * (n & 1) : 0));
                    }
                    __syncwarp();
                    if (tile == s.lo) any = next_seg();
                }
            }
        }
    } else if constexpr (PL::PT) {
        // ================================ softmax, outputs: P in tensor memory ====================
        // Set 0 takes the even tiles, set 1 the odd ones; a row is one thread's in either set, and
        // its row of O in the same lane, so only the two warps of the same 32 rows have to agree.
        // The rows' running maxima (shared memory) move in tile order: the warp of tile n passes
        // its partner a token (named barrier) once tile n's are final; a warp whose weights refer
        // to an older maximum by then computes them again.
        const int set = (warp - PL::CONTROL) / 4;
        const int q4 = warp & 3;                             // lanes 32 q4 .. of tensor memory
        const int row = q4 * 32 + lane;
        const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
        const int token = kBar + 1 + q4;                     // + 4 * set
        volatile float *v_max = s_fac + RN;
        if (set == 0) v_max[row] = kNoMax;
        tc::bar_sync(kBar, kSoftmax);
        TreeWalk walk(p, range);
        TreeSeg s, nx;
        unsigned n = 0, seg_no = 0;
        uint32_t v_unit = KU;                                // this tile's first value unit
        const int r0 = rt * p.RP;
        const int tok = (r0 + row) / p.G, hg_row = (r0 + row) - tok * p.G;
        auto next_seg = [&]() {                              // (row tile 0 has rows in every pair)
            while (walk.next(p, rt, TS, nx))
                if (nx.rows > 0) return true;
            return false;
        };
        bool more = next_seg();
        while (more) {
            s = nx;
            more = next_seg();
            const bool mine = row < s.rows;
            const bool any = q4 * 32 < s.rows;               // warp-uniform
            float l = 0.f, l_ref = kNoMax;                   // sum over this set's tiles, its reference
            const uint64_t word = mine && s.hi == s.nt ? tree_mask_word(p, s.b, tok, s.cnt) : 0ull;
            unsigned long long *s_nf = s_nf2 + (seg_no++ & 1);
            for (int tile = s.lo; tile < s.hi; ++tile, ++n, v_unit += PER) {
                if ((int)(n & 1) != set) continue;
                const bool draft = s.is_draft(p, tile);
                const int valid = s.valid(p, tile, TS);
                bool scaled = draft || valid < TS;           // logits are masked and scaled as they are read
                float mx = -INFINITY, m = kNoMax, z = 0.f;
                uint32_t w[TS / 2];                          // the row's weights, bf16 pairs
                // 64 logits of the row, masked ones -inf (and then scaled: returns the scale to use)
                auto logits = [&](int half, float *x) -> float {
                    tc::ld32(tS + set * TS + lanes + 64 * half, x);
                    tc::ld32(tS + set * TS + lanes + 64 * half + 32, x + 32);
                    tc::wait_ld();
                    if (!scaled) return p.scale_log2;
                    const int v = valid - 64 * half;
                    const uint64_t see = draft ? (half == 0 ? word : 0ull)
                                               : v >= 64 ? ~0ull : v <= 0 ? 0ull : (1ull << v) - 1ull;
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        x[c] = (see >> c) & 1ull ? x[c] * p.scale_log2 : -INFINITY;
                    return 1.f;
                };
                wait(b_s_full + 8 * set, (n >> 1) & 1);
                tc::fence_after();
                if (any) {
#pragma unroll
                    for (int half = 0; half < TS / 64; ++half) {
                        float x[64];
                        const float scale = logits(half, x);
                        // the largest scaled logit: of the smallest value when the scale is negative
                        float a[4] = {x[0], x[1], x[2], x[3]};
                        if (scale >= 0.f) {
#pragma unroll
                            for (int c = 4; c < 64; ++c) a[c & 3] = fmaxf(a[c & 3], x[c]);
                            mx = fmaxf(mx, fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) * scale);
                        } else {
#pragma unroll
                            for (int c = 4; c < 64; ++c) a[c & 3] = fminf(a[c & 3], x[c]);
                            mx = fmaxf(mx, fminf(fminf(a[0], a[1]), fminf(a[2], a[3])) * scale);
                        }
                    }
                    // weights against the maximum as it stands, or this tile's where it rises
                    m = v_max[row];
                    if (mx > m + kSlack) m = mx;
                }
                float m_cur = kNoMax, m_fin = kNoMax;
                bool rise = false;
#pragma unroll 1
                for (int pass = 0; pass < 2; ++pass) {
                    scaled |= mine && fabsf(m) >= kBigMax;
                    if (any) {
                        z = 0.f;
#pragma unroll
                        for (int half = 0; half < TS / 64; ++half) {
                            float x[64];
                            const float scale = logits(half, x);
                            const float2 sc = make_float2(scale, scale), mm = make_float2(-m, -m);
                            float2 z0 = make_float2(0.f, 0.f), z1 = z0;
#pragma unroll
                            for (int c = 0; c < 64; c += 4) {
                                float2 y0 = __ffma2_rn(make_float2(x[c], x[c + 1]), sc, mm);
                                float2 y1 = __ffma2_rn(make_float2(x[c + 2], x[c + 3]), sc, mm);
                                y0.x = ex2(y0.x);
                                y0.y = ex2(y0.y);
                                y1.x = ex2(y1.x);
                                y1.y = ex2(y1.y);
                                z0 = __fadd2_rn(z0, y0);
                                z1 = __fadd2_rn(z1, y1);
                                w[32 * half + c / 2] = tc::pack_bf16(y0.x, y0.y);
                                w[32 * half + c / 2 + 1] = tc::pack_bf16(y1.x, y1.y);
                            }
                            z0 = __fadd2_rn(z0, z1);
                            z += z0.x + z0.y;
                        }
                    }
                    if (pass == 1) break;
                    // the maxima up to the tile before are final
                    if (n > 0) tc::bar_sync(token + 4 * (set ^ 1), 64);
                    m_cur = v_max[row];
                    rise = mine && mx > m_cur + kSlack;
                    m_fin = rise ? m : m_cur;
                    if (!__any_sync(0xffffffffu, mine && m != m_fin)) break;
                    m = m_fin;
                }
                if (rise) v_max[row] = m_fin;
                __threadfence_block();
                __syncwarp();
                if (more || tile + 1 < s.hi) tc::bar_arrive(token + 4 * set, 64);
                if (tile > s.lo && __any_sync(0xffffffffu, rise)) {
                    wait(b_pv + 8 * ((n - 1) & 1), ((n - 1) >> 1) & 1);
                    tc::fence_after();
                    const float f = rise ? ex2(m_cur - m_fin) : 1.f;
#pragma unroll 1
                    for (int c = 0; c < DV; c += 16) {
                        float o[16];
                        tc::ld16(tO + lanes + c, o);
                        tc::wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] *= f;
                        tc::st16(tO + lanes + c, o);
                    }
                }
                l = l * ex2(l_ref - m_fin) + z;
                l_ref = m_fin;
                if (n >= 2) wait(b_pv + 8 * (n & 1), ((n - 2) >> 1) & 1);   // this P buffer is used up
                tc::fence_after();
                if (any) {
#pragma unroll
                    for (int half = 0; half < TS / 64; ++half)
                        tc::st32(tP + set * (TS / 2) + lanes + 32 * half, w + 32 * half);
                }
                tc::wait_st();
                // value rows past the valid ones, and a drafted token's non-finite values
                const int depth = steps_of(s, tile) * 16;
                if (valid < depth || draft) {
                    if (draft) {
                        if (q4 == 0 && lane == 0) *s_nf = 0ull;
                        tc::bar_sync(kBar + 9 + set, 128);
                    }
                    for (int u = 0; u < MB; ++u) {
                        const unsigned un = v_unit + u;
                        const uint32_t slot = un % NU;
                        wait(b_full + 8 * slot, (un / NU) & 1);
                        clean_unit<SUBS, SUB>(smem_raw + (ring + slot * UNIT - raw), q4, 4, valid, depth, draft, s_nf);
                    }
                }
                tc::fence_async();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_p_full + 8 * set);
            }
            // this part's outputs: O / l, or the partial state
            const bool whole = s.whole();
            const size_t part = (size_t)blockIdx.x * 2 + (s.first ? 0 : 1);
            wait(b_pv + 8 * ((n - 1) & 1), ((n - 1) >> 1) & 1);
            tc::fence_after();
            const float m = v_max[row];
            l *= ex2(l_ref - m);
            if (set == 1) s_fac[row] = l;
            tc::bar_sync(kBar, kSoftmax);
            if (set == 0) {
                l += s_fac[row];
                v_max[row] = kNoMax;                         // for the next pair
                s_fac[row] = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                if (mine) {
                    if (!whole) {
                        p.ws_ml[(part * RN + row) * 2] = m;
                        p.ws_ml[(part * RN + row) * 2 + 1] = l;
                    } else if (p.lse != nullptr) {
                        p.lse[((size_t)s.b * p.T + tok) * p.Hq + s.kh * p.G + hg_row] =
                            l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
                    }
                }
            }
            tc::bar_sync(kBar, kSoftmax);
            const unsigned long long nf = p.kd != nullptr && s.hi == s.nt ? *s_nf : 0ull;
            const float f = s_fac[row];
            if (any) {
#pragma unroll 1
                for (int c = set * (DV / 2); c < (set + 1) * (DV / 2); c += 16) {
                    float o[16];
                    __syncwarp();
                    tc::ld16(tO + lanes + c, o);
                    tc::wait_ld();
                    if (!mine) continue;
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] *= f;
                    if (whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(
                            static_cast<__nv_bfloat16 *>(p.out) +
                            (((size_t)s.b * p.T + tok) * p.Hq + s.kh * p.G + hg_row) * DV + c);
                        dst[0] = make_uint4(tc::pack_bf16(o[0], o[1]), tc::pack_bf16(o[2], o[3]),
                                            tc::pack_bf16(o[4], o[5]), tc::pack_bf16(o[6], o[7]));
                        dst[1] = make_uint4(tc::pack_bf16(o[8], o[9]), tc::pack_bf16(o[10], o[11]),
                                            tc::pack_bf16(o[12], o[13]), tc::pack_bf16(o[14], o[15]));
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>(p.ws_o + (part * RN + row) * DV + c);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    }
                }
                if (nf && mine)
#pragma unroll 1
                    for (int d = set * (DV / 2); d < (set + 1) * (DV / 2); ++d)
                        add_stray<RN, DV>(p, s, part, r0, row, d, nf);
            }
            __syncwarp();
            tc::fence_before();
            tc::bar_sync(kBar, kSoftmax);                    // O is free for the next pair
        }
    } else {
        // ================================ softmax, outputs ========================================
        // Set i takes slots 32 i .. 32 i + 31 of a tile: a row has a thread in each set, which keep
        // the same maximum and their own part of the sum.
        constexpr int HC = 32;
        const int set = (warp - PL::CONTROL) / 4;
        const int q4 = warp & 3;                             // lanes 32 q4 .. of tensor memory
        const int ln = q4 * 32 + lane;                       // 0..127
        const int tw = set * 128 + ln;
        const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
        // the row of S (M = RN) and the dimension of O^T (M = UD) this thread's lane holds
        const int row = RN == 128 ? ln : (lane < 16 ? q4 * 16 + lane : 64);
        const int dim = UD == 128 ? ln : (lane < 16 ? q4 * 16 + lane : UD);
        const int row_lo = RN == 128 ? q4 * 32 : q4 * 16;    // first row of this warp
        const int c0 = set * HC;                             // first slot
        TreeWalk walk(p, range);
        TreeSeg s;
        unsigned n = 0, seg_no = 0;
        uint32_t v_unit = LATENT ? 0 : KU;                   // this tile's first value unit
        const int r0 = rt * p.RP;
        const int tok = (r0 + row) / p.G, hg_row = (r0 + row) - tok * p.G;   // of this thread's row
        auto token_of = [&](int r) { return (int)(((float)r + 0.5f) * p.inv_G); };
        TreeSeg nx;
        bool more = walk.next(p, rt, TS, nx);
        while (more) {
            s = nx;
            more = walk.next(p, rt, TS, nx);                 // its lengths arrive meanwhile
            if (s.rows <= 0) continue;
            const bool mine = row < s.rows;
            const bool any = row_lo < s.rows;                // warp-uniform
            float m = kNoMax, l = 0.f;
            bool big = false;                                // some row of the warp has kBigMax
            bool drafts = false;
            const uint64_t word = mine && s.hi == s.nt ? tree_mask_word(p, s.b, tok, s.cnt) : 0ull;
            // drafted tokens with non-finite values: alternate words, since a thread may set up
            // the next pair's while another still reads this one's
            unsigned long long *s_nf = s_nf2 + (seg_no++ & 1);
            for (int tile = s.lo; tile < s.hi; ++tile, ++n, v_unit += PER) {
                const bool draft = s.is_draft(p, tile);
                const int valid = s.valid(p, tile, TS);
                const uint32_t buf = n & 1;
                float x[HC];
                float mx = -INFINITY, scale = p.scale_log2;
                wait(b_s_full + 8 * buf, (n >> 1) & 1);
                tc::fence_after();
                if (any) {
#pragma unroll
                    for (int c = 0; c < HC; c += 32) tc::ld32(tS + buf * TS + lanes + c0 + c, x + c);
                    tc::wait_ld();
                }
                if (any) {
                    if (draft || valid < TS || big) {        // masked: scaled here, once
                        uint32_t see;                        // slots c0 .. c0 + 31
                        if (draft) see = set == 0 ? (uint32_t)word : set == 1 ? (uint32_t)(word >> 32) : 0u;
                        else see = valid - c0 >= 32 ? ~0u : valid > c0 ? (1u << (valid - c0)) - 1u : 0u;
#pragma unroll
                        for (int c = 0; c < HC; ++c)
                            x[c] = (see >> c) & 1u ? x[c] * scale : -INFINITY;
                        scale = 1.f;
                    }
                    // the largest scaled logit: of the smallest value when the scale is negative
                    float a[4] = {x[0], x[1], x[2], x[3]};
                    if (scale >= 0.f) {
#pragma unroll
                        for (int c = 4; c < HC; ++c) a[c & 3] = fmaxf(a[c & 3], x[c]);
                        mx = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) * scale;
                    } else {
#pragma unroll
                        for (int c = 4; c < HC; ++c) a[c & 3] = fminf(a[c & 3], x[c]);
                        mx = fminf(fminf(a[0], a[1]), fminf(a[2], a[3])) * scale;
                    }
                }
                if (draft && tw == 0) *s_nf = 0ull;          // ordered by the barrier below
                if (tc::bar_any(kBar, kSoftmax, mine && mx > m + kSlack)) {
                    // the maximum rises: agree on it, then bring l and O to it
                    if (row < RN) s_row[set * RN + row] = mx;
                    tc::bar_sync(kBar, kSoftmax);
                    float m_new = m;
                    if (row < RN) {
#pragma unroll
                        for (int i = 0; i < kSets; ++i) m_new = fmaxf(m_new, s_row[i * RN + row]);
                    }
                    const float f = ex2(m - m_new);
                    m = m_new;
                    big = __any_sync(0xffffffffu, mine && fabsf(m) >= kBigMax);
                    if (big) {
#pragma unroll
                        for (int c = 0; c < HC; ++c) x[c] *= scale;
                        scale = 1.f;
                    }
                    l *= f;
                    if (tile > s.lo) {
                        if (set == 0 && row < RN) s_fac[row] = f;
                        wait(b_pv, (n - 1) & 1);
                        tc::fence_after();
                        tc::bar_sync(kBar, kSoftmax);
#pragma unroll 1
                        for (int c = set * 16; c < MB * RN; c += 16 * kSets) {
                            if ((c & (RN - 1)) >= s.rows) continue;
                            float o[16];
                            tc::ld16(tO + lanes + c, o);
                            tc::wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] *= s_fac[(c & (RN - 1)) + j];
                            tc::st16(tO + lanes + c, o);
                        }
                        tc::wait_st();
                    }
                }
                if (any) {
                    const float2 sc = make_float2(scale, scale), mm = make_float2(-m, -m);
                    float2 z0 = make_float2(0.f, 0.f), z1 = z0;
#pragma unroll
                    for (int c = 0; c < HC; c += 4) {
                        float2 y0 = __ffma2_rn(make_float2(x[c], x[c + 1]), sc, mm);
                        float2 y1 = __ffma2_rn(make_float2(x[c + 2], x[c + 3]), sc, mm);
                        x[c] = y0.x = ex2(y0.x);
                        x[c + 1] = y0.y = ex2(y0.y);
                        x[c + 2] = y1.x = ex2(y1.x);
                        x[c + 3] = y1.y = ex2(y1.y);
                        z0 = __fadd2_rn(z0, y0);
                        z1 = __fadd2_rn(z1, y1);
                    }
                    z0 = __fadd2_rn(z0, z1);
                    l += z0.x + z0.y;
                }
                if (n > 0) wait(b_pv, (n - 1) & 1);          // P of the previous tile is used up
                if (any && row < RN) {
#pragma unroll
                    for (int c = 0; c < HC / 8; ++c) {       // 16-byte chunks of the row
                        const float *y = x + 8 * c;
                        const int k = c0 / 8 + c;
                        tc::st_shared_16(sP + (k >> 3) * RN * 128 + row * 128 +
                                             (((k & 7) ^ (row & 7)) << 4),
                                         tc::pack_bf16(y[0], y[1]), tc::pack_bf16(y[2], y[3]),
                                         tc::pack_bf16(y[4], y[5]), tc::pack_bf16(y[6], y[7]));
                    }
                }
                // value rows past the valid ones, and a drafted token's non-finite values
                const int depth = steps_of(s, tile) * 16;
                if (valid < depth || draft) {
                    for (int u = 0; u < MB; ++u) {
                        const unsigned un = v_unit + u;
                        const uint32_t slot = un % NU;
                        if (!LATENT) wait(b_full + 8 * slot, (un / NU) & 1);   // (S implies a latent tile)
                        unsigned char *base = smem_raw + (ring + slot * UNIT - raw);
                        clean_unit<SUBS, SUB>(base, warp - PL::CONTROL, kSoftmax / 32, valid, depth, draft, s_nf);
                    }
                    drafts |= draft;
                }
                tc::fence_async();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_p_full + 8 * buf);
            }
            // this part's outputs: O^T / l, or the partial state
            const bool whole = s.whole();
            const size_t part = (size_t)blockIdx.x * 2 + (s.first ? 0 : 1);
            wait(b_pv, (n - 1) & 1);                         // every warp is past its last rescaling
            tc::fence_after();
            if (set > 0 && row < RN) s_row[set * RN + row] = l;
            tc::bar_sync(kBar, kSoftmax);
            if (set == 0 && row < RN) {
#pragma unroll
                for (int i = 1; i < kSets; ++i) l += s_row[i * RN + row];
                s_fac[row] = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                if (mine) {
                    const int h = s.kh * p.G + hg_row;
                    if (!whole) {
                        p.ws_ml[(part * RN + row) * 2] = m;
                        p.ws_ml[(part * RN + row) * 2 + 1] = l;
                    } else if (p.lse != nullptr) {
                        p.lse[((size_t)s.b * p.T + tok) * p.Hq + h] =
                            l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
                    }
                }
            }
            tc::bar_sync(kBar, kSoftmax);
            const unsigned long long nf = drafts ? *s_nf : 0ull;
#pragma unroll 1
            for (int c = set * 16; c < MB * RN; c += 16 * kSets) {
                const int ra = c & (RN - 1);                 // first row of these columns
                if (ra >= s.rows) continue;
                const int d = c / RN * UD + dim;
                const int here = min(16, s.rows - ra);
                float o[16];
                __syncwarp();
                tc::ld16(tO + lanes + c, o);
                tc::wait_ld();
                if (dim >= UD) continue;
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(s_fac + ra + j);
                    o[j] *= f.x; o[j + 1] *= f.y; o[j + 2] *= f.z; o[j + 3] *= f.w;
                }
                const int t = token_of(r0 + ra);
                int hg = (r0 + ra) - t * p.G;
                if (whole) {
                    __nv_bfloat16 *dst =
                        static_cast<__nv_bfloat16 *>(p.out) +
                        (((size_t)s.b * p.T + t) * p.Hq + s.kh * p.G + hg) * DV + d;
                    const int wrap = (p.Hq - p.G + 1) * DV;  // to the next token's first head
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        if (j < here) *dst = __float2bfloat16(o[j]);
                        ++hg;
                        dst += hg == p.G ? wrap : DV;
                        hg = hg == p.G ? 0 : hg;
                    }
                } else {
                    float *dst = p.ws_o + (part * RN + ra) * DV + d;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (j < here) dst[j * DV] = o[j];
                }
            }
            if (nf && dim < UD)
#pragma unroll 1
                for (int c = set * 16; c < MB * RN; c += kSets * 16)
#pragma unroll 1
                    for (int ra = c & (RN - 1); ra < min((c & (RN - 1)) + 16, s.rows); ++ra)
                        add_stray<RN, DV>(p, s, part, r0, ra, c / RN * UD + dim, nf);
            __syncwarp();
            tc::fence_before();
        }
    }

    tc::fence_before();
    __syncthreads();
    // after a wait ran out: the loads in flight have landed and the products issued have completed
    // before the block frees tensor memory and exits
    if (*s_abort) {
        if (threadIdx.x == 0 || (LATENT && threadIdx.x == 96)) {   // each its own loads
            auto drain = [&](uint32_t bar, uint32_t parity) {
                mbar_wait_ok(bar, parity, kMbarSpinLimit >> 4);
            };
            if constexpr (LATENT) {
                for (unsigned i = n_tiles > NTB ? n_tiles - NTB : 0; i < n_tiles; ++i)
                    drain(b_full + 8 * (i % NTB), (i / NTB) & 1);
            } else {
                const unsigned units = n_tiles * PER;
                for (unsigned i = units > NU ? units - NU : 0; i < units; ++i)
                    if ((int)(i % PER) >= u_lo && (int)(i % PER) < u_hi) drain(b_full + 8 * (i % NU), (i / NU) & 1);
            }
            if (n_segs > 0) drain(b_q_full, (n_segs - 1) & 1);
        } else if (warp == 1 || warp == 2) {                 // each its own products
            if (tc::elect()) tc::commit(b_done);
            __syncwarp();
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
                      dim3(PL::THREADS), PL::SMEM, stream, maps, p);
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
    const uint64_t row = (uint64_t)p.DK * 2;
    const uint64_t B = p.B, T = p.T, Hq = p.Hq, Hkv = p.Hkv, subs = p.DV / 64;
    const int TS = p.latent ? 64 : tile_slots(p.DV);
    const int units = p.DV < 128 ? 1 : 2;                    // 64-wide pieces of a ring unit
    const uint64_t ss = (uint64_t)p.ss * 2, sb = (uint64_t)p.sb * 2;
    auto cache = [&](CUtensorMap *m, const void *ptr) {
        if (p.table != nullptr) {
            const uint64_t rows = Hkv * (uint64_t)p.n_pool * p.bs;
            return tc::encode_5d(m, ptr, {64, rows, subs, 1, 1}, {row, 128, row * rows, row * rows},
                                 p.bs < TS ? p.bs : TS, 1, 1);
        }
        const uint64_t sh = p.latent ? row : (uint64_t)p.sh * 2;
        return tc::encode_5d(m, ptr, {64, (uint64_t)p.cap, subs, Hkv, B}, {ss, 128, sh, sb}, TS, units, 1);
    };
    auto drafted = [&](CUtensorMap *m, const void *ptr) {
        return tc::encode_5d(m, ptr, {64, T, subs, Hkv, B}, {row * Hkv, 128, row, row * Hkv * T}, TS,
                             units, 1);
    };
    bool ok = cache(&maps.k, p.k);
    if (ok && p.latent) {
        const uint64_t rows = B * T * Hq, all = row * rows, E = p.DK - p.DV;
        ok = tc::encode_5d(&maps.q, p.q, {64, rows, subs, 1, 1}, {row, 128, all, all}, p.RN, (uint32_t)subs, 1);
        const auto part = [&](const void *ptr) { return static_cast<const char *>(ptr) + p.DV * 2; };
        if (ok && E > 0)
            ok = tc::encode_5d(&maps.rq, part(p.q), {E, rows, 1, 1, 1}, {row, all, all, all}, p.RN, 1, 1) &&
                 tc::encode_5d(&maps.rk, part(p.k), {E, (uint64_t)p.cap, 1, 1, B}, {ss, row, row, sb}, TS, 1, 1);
        else if (ok)
            maps.rq = maps.q, maps.rk = maps.k;
        maps.kd = maps.vd = maps.v = maps.rd = maps.k;
        if (ok && p.kd != nullptr) {
            ok = drafted(&maps.kd, p.kd);
            if (ok && E > 0)
                ok = tc::encode_5d(&maps.rd, part(p.kd), {E, T, 1, 1, B}, {row, row, row, row * T}, TS, 1, 1);
        }
    } else if (ok) {
        ok = tc::encode_5d(&maps.q, p.q, {64, Hq, B * T, subs, 1}, {row, row * Hq, 128, row * Hq * B * T},
                           p.G, p.RP / p.G, 1) &&
             cache(&maps.v, p.v);
        maps.kd = maps.vd = maps.rq = maps.rk = maps.rd = maps.k;
        if (ok && p.kd != nullptr) ok = drafted(&maps.kd, p.kd) && drafted(&maps.vd, p.vd);
    }
    if (!ok) return cudaSuccess;
    *used = true;
    if (p.latent) {
        switch (p.DV) {
        case 128:
            return p.RN == 32 ? launch_typed<192, 128, true, 32>(p, maps, stream)
                              : launch_typed<192, 128, true, 64>(p, maps, stream);
        case 256:
            return p.RN == 32 ? launch_typed<320, 256, true, 32>(p, maps, stream)
                              : launch_typed<320, 256, true, 64>(p, maps, stream);
        default:
            return p.RN == 32 ? launch_typed<576, 512, true, 32>(p, maps, stream)
                              : launch_typed<576, 512, true, 64>(p, maps, stream);
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

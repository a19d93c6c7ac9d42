// decode_q8.cu -- attention of one new token per sequence over pages of e4m3 numbers with a scale for
// each page and head.
//
//   x_j = scale * ks(j) * (q . k8_j),   out = sum_j softmax(x)_j vs(j) v8_j,
//   ks(j), vs(j): the key and value scales of token j's page for this head.
//
// What bounds it is the stream of the cache: one byte an element, 4 G operations for the G query heads
// that share it, far below the ridge.  So everything is arranged around bytes in flight:
//   A warp works alone.  The steps (16 slots of one (sequence, KV head, row tile), 32 with 64 dims) of the
//   whole batch are dealt out evenly, in order, to the blocks and again to a block's warps, and a warp
//   keeps two to five steps in flight in its own ring in shared memory (cp.async, 16 bytes a lane; rows
//   behind the length are filled with zeros, whatever the page holds there).  No barrier between warps
//   while they stream, and no wait that could fail to end: a warp waits for its own copies only.
//   Both products run on mma.m16n8k16 with the cache as the 16-row operand and the query heads as the 8
//   columns, so that up to 8 heads waste nothing: S^T = K Q^T, O^T = V^T P^T.  (5th-generation
//   products want 64 or 128 rows of one operand and, of 8-bit operands, both in 8 bits; the stream
//   leaves the legacy pipe four fifths idle.)  e4m3 numbers are exact in fp16, so K and V enter
//   the products as they are stored; a fragment's 16 bytes of one row are 4 steps of the
//   product's inner dimension, which may be dealt out in any order as long as Q is dealt out alike.
//   Queries are brought to [2^14, 2^15) by a power of two per row: bf16 then is exact in fp16 down to
//   2^-31 of the row's largest element.  fp32 queries become two fp16 terms (22 bits), and so do the
//   weights, whatever the queries: bf16 outputs then are those of fp32 weights but for one in some thousands, while
//   weights of 11 bits would turn the rounding of one in fifty (relative difference 6e-4 for 512 rows of 832
//   slots, 7e-5 with two terms; 24.6 and 25.3 us, groups of 12 4 to 6 % more, long rows of few heads nothing).
//   Weights carry the value scale: w_j = 2^(x_j - m + log2 vs(j) - ref), with the softmax's running maximum m, whose
//   sum l is kept beside it, and a whole number ref of its own that follows the weights up and down: pages whose
//   values differ by any factor meet on equal terms, and the light weights behind a heavy one, fp16 in the products,
//   are held to as many bits as that one was.  Exponents are formed from the difference x_j - m, which is exact where it
//   counts however large the logits are.  All sums are fp32.
//
// The range of a warp is found on the device (a scan of the lengths), even however ragged the batch
// is.  A row tile that crosses warps leaves partial states (m, l, ref, O): those of a block are joined in
// shared memory at its end, those of several blocks by decode_q8_merge_kernel, both in order of
// the slots, so results do not depend on timing.
//
// Measured: 2 x 131072 slots of 8 heads of 128, 4 query heads each (537 MB) 94.7 us, 5.7 TB/s.  Copies
// alone in this pattern take 78 us.  3 us pass until the first copies leave (lengths, page ids, cold
// instructions), 3 us after the last (parts), and equal shares take some SMs 61 us and others 85: whole
// groups of neighbours are slower.  Variants, when the weights had one term and this took 92.5: more blocks than fit
// at once, so that the fast ones take more, 115 us; four blocks of 4 warps an SM 111; 6 warps a block with four
// stages 94.7; one block of 8 warps with six stages 99.5; two products side by side with 128 dims 93.4; one warp that
// finds the block's range for all 95.2; L2 prefetch hints no change; parts joined per warp instead of per block 110.
#include <algorithm>
#include <type_traits>

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace kvc {

namespace {

constexpr int kSub = 16;                     // slots of one product; a step is one or two of them
constexpr int kEnd = 2;                      // steps that the end of a row tile counts as (0: 35.3 us for 8 fp32
                                             // sequences of 3277 to 13107 slots, 1: 34.3, 2: 33.7, 4: 33.3)
// Warps of a block: what registers allow (one block an SM with 16 heads or fp32 queries, two otherwise).  fp32
// queries over 2 x 32768 slots of 8 heads of 128: 8 warps 36.1 us, 10 35.9, 12 32.1.
constexpr int warps_of(int D, int NT, bool split)
{
    return D > 128 || (NT == 2 && split) || (NT == 1 && !split) ? 8 : 12;
}
constexpr int kMergeThreads = 256;
constexpr int kWholeSteps = 16;              // row tiles of so many steps stay in one block, however many there are (2000 x
                                             // 100 to 256 slots of 8 heads: 149 us, split 161; 250 to 256: 192 and 214)
constexpr int kWholeWait = 20;               // and longer ones where the fullest block has so many above the mean
constexpr int kMinUnits = 16;                // units that a block is worth at least (1 x 1000 slots of 8 heads of 128:
                                             // 8 9.1 us, 16 10.1, 32 12.0)
constexpr float kSlack = 8.f;                // a maximum or reference moves when it is passed by 2^8 either way
constexpr float kBoost = 6.f;                // weights are held times 2^6: at most 2^15, and the largest of a step
                                             // that lies low but moves nothing, 2^-2, is 22 bits above the last place
                                             // (slack 4 and boost 10: groups of 12 2 % slower)
constexpr int kLook = 16;                    // a reference may go down every so many steps (8: groups of 12, fp32, 43.3 us,
                                             // 16 42.8; a vote on it in every step 50.6)
constexpr int kTop = 100;                    // and as far as the sums stay below 2^101
constexpr float kNone = -3.402823466e38f;    // a maximum of nothing
constexpr int kDevBadLen_ = 5;
constexpr int kDevBadBlk_ = 9;

// Products of 16 slots that a step takes side by side: with 64 dims one alone is half bookkeeping (8 x 16384
// slots of 4 heads of 64, 4 query heads each: one 23.9 us, two 22.6; fp32 queries 26.1 and 24.0).
constexpr int subs_of(int D) { return D == 64 ? 2 : 1; }

template <int D, int NT, bool SPLIT>
struct Q8Plan {
    static constexpr int SUB = subs_of(D), STEP = kSub * SUB;
    static constexpr int WARPS = warps_of(D, NT, SPLIT);
    static constexpr int BLOCKS = D <= 128 && NT == 1 && !SPLIT ? 2 : 1;    // per SM (registers)
    static constexpr int STAGE = 2 * STEP * D + 32;      // keys and values, their scales, what they are of
    static constexpr int ROOM = (BLOCKS == 2 ? 112 : 224) * 1024 / WARPS;
    static constexpr int FIT = ROOM / STAGE;
    static constexpr int STAGES = FIT > 6 ? 6 : FIT;
    static constexpr int SMEM = WARPS * STAGES * STAGE;
};

// Four e4m3 numbers to two pairs of fp16.
__device__ __forceinline__ void cvt_e4m3x4(uint32_t four, uint32_t &lo, uint32_t &hi)
{
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}
__device__ __forceinline__ void mma_16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same onto zero.
__device__ __forceinline__ void mma_16816_new(float *c, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_h2(uint32_t x)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&x));
}
__device__ __forceinline__ void cp_16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_16(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds_16(uint32_t a)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds_8(uint32_t a)
{
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}

// 2^(ref - kBoost) as two factors, since it may pass the range where the outputs do not.  The second one is 1 for values
// of ordinary size.
__device__ __forceinline__ float ex2_near(float ref) { return ex2(fminf(fmaxf(ref - kBoost, -60.f), 60.f)); }
__device__ __forceinline__ float ex2_far(float ref)
{
    return ex2(ref - kBoost - fminf(fmaxf(ref - kBoost, -60.f), 60.f));
}

// The largest x of a row's lanes.
__device__ __forceinline__ float row_max(float x)
{
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// Slots of sequence b, clamped to the table, and its steps (one for an empty one, which has rows to write).
__device__ __forceinline__ int len_of(const DecodeQ8Params &p, int b)
{
    const int n = p.len[b];
    return n < 0 ? 0 : (n > p.cap ? p.cap : n);
}
template <int STEP>
__device__ __forceinline__ int steps_of(int len)
{
    return len > 0 ? (len + STEP - 1) / STEP : 1;
}

// A warp's share of the units: every row tile counts its steps and kEnd.  Called by a whole warp.
struct Range {
    int b, hr, off, len;         // the first row tile: sequence, head * RT + tile, first unit in it, slots
    int left;                    // units of this warp
};
// U: 32 bits where they hold all units (a 64-bit division is a long subroutine).
template <typename U, int W, int STEP>
__device__ __forceinline__ Range split_range(const DecodeQ8Params &p)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool check = blockIdx.x == 0 && warp == 0;
    const int per = (p.B + 31) >> 5;
    const int b0 = min(p.B, lane * per), b1 = min(p.B, b0 + per);
    U sum = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = p.len[b];
        if (check && (n < 0 || n > p.cap)) record_code(p.dev_code, kDevBadLen_);
        sum += (U)(steps_of<STEP>(n < 0 ? 0 : min(n, p.cap)) + kEnd) * (U)p.HR;
    }
    U incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const U y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    const U T = __shfl_sync(0xffffffffu, incl, 31);
    U blocks = T / kMinUnits;                // a block is worth a few steps
    blocks = blocks < 1 ? 1 : (blocks > gridDim.x ? gridDim.x : blocks);
    const U q = T / blocks, r = T - q * blocks, bl = blockIdx.x;
    const U first = bl * q + (bl < r ? bl : r);
    const unsigned mine = bl < blocks ? (unsigned)(q + (bl < r ? 1 : 0)) : 0u;
    const unsigned w0 = (unsigned)((unsigned long long)mine * warp / W);
    const U t0 = first + w0;
    Range g;
    g.left = (int)((unsigned)((unsigned long long)mine * (warp + 1) / W) - w0);
    const U before = incl - sum;
    const bool here = g.left > 0 && before <= t0 && t0 < incl;
    int b = b0, hr = 0, off = 0, len = 0;
    if (here) {
        U t = before;
        U cost = 0;
        for (;; ++b) {
            len = len_of(p, b);
            cost = (U)(steps_of<STEP>(len) + kEnd);
            if (t0 < t + cost * (U)p.HR || b == b1 - 1) break;
            t += cost * (U)p.HR;
        }
        hr = (int)((t0 - t) / cost);
        off = (int)(t0 - t - (U)hr * cost);
    }
    const int src = (__ffs(__ballot_sync(0xffffffffu, here)) - 1) & 31;
    g.b = __shfl_sync(0xffffffffu, b, src);
    g.hr = __shfl_sync(0xffffffffu, hr, src);
    g.off = __shfl_sync(0xffffffffu, off, src);
    g.len = __shfl_sync(0xffffffffu, len, src);
    return g;
}
template <int W, int STEP>
__device__ __noinline__ Range split_range_64(const DecodeQ8Params &p)
{
    return split_range<unsigned long long, W, STEP>(p);
}

template <int W, int STEP>
__device__ __forceinline__ Range find_range(const DecodeQ8Params &p)
{
    if (!p.whole) return p.small ? split_range<unsigned, W, STEP>(p) : split_range_64<W, STEP>(p);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool check = blockIdx.x == 0 && warp == 0;
    Range g;
    g.b = g.hr = g.off = g.len = 0;
    {                            // whole row tiles, equally many a block
        if (check)
            for (int b = lane; b < p.B; b += 32)
                if (p.len[b] < 0 || p.len[b] > p.cap) record_code(p.dev_code, kDevBadLen_);
        const unsigned tiles = (unsigned)(p.B * p.HR), n = gridDim.x;
        const unsigned i0 = (unsigned)((unsigned long long)tiles * blockIdx.x / n);
        const unsigned i1 = (unsigned)((unsigned long long)tiles * (blockIdx.x + 1) / n);
        int units = 0;
        for (unsigned i = i0 + lane; i < i1; i += 32) units += steps_of<STEP>(len_of(p, (int)(i / p.HR)));
        units = __reduce_add_sync(0xffffffffu, units);
        int at = units * warp / W;
        g.left = units * (warp + 1) / W - at;
        if (g.left > 0) {                    // (a sequence's row tiles are alike)
            g.b = (int)(i0 / p.HR);
            g.hr = (int)(i0 - (unsigned)g.b * p.HR);
            for (;;) {
                g.len = len_of(p, g.b);
                const int n = steps_of<STEP>(g.len), k = at / n;
                if (k < p.HR - g.hr) {
                    g.hr += k;
                    g.off = at - k * n;
                    break;
                }
                at -= (p.HR - g.hr) * n;
                g.hr = 0;
                ++g.b;
            }
        }
        return g;
    }
}

// The steps of a range in order.
template <int STEP>
struct Walk {
    int b, hr, step, len, n;     // the step: row tile (b, hr), its number, the tile's slots and steps
    int left;                    // units of the range left, this step's among them
    __device__ __forceinline__ Walk(const DecodeQ8Params &p, const Range &g)
        : b(g.b), hr(g.hr), step(g.off), len(g.len), n(steps_of<STEP>(g.len)), left(g.left)
    {
        settle(p);
    }
    // Moves past a tile's end units to a step, if one is left.
    __device__ __forceinline__ void settle(const DecodeQ8Params &p)
    {
        while (left > 0 && step >= n) {
            left -= n + (p.whole ? 0 : kEnd) - step;
            step = 0;
            if (++hr == p.HR) {
                hr = 0;
                if (++b == p.B) {
                    left = 0;
                    return;
                }
                len = len_of(p, b);
                n = steps_of<STEP>(len);
            }
        }
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ void next(const DecodeQ8Params &p)
    {
        ++step;
        --left;
        settle(p);
    }
};

// 4 columns of an output row from its joined state.
template <typename T>
__device__ __forceinline__ void store_row(const DecodeQ8Params &p, size_t row, int D, int col, float m, float l,
                                          float ref, float4 o)
{
    const float f = l == 0.f ? 0.f : ex2_near(ref) / l, f2 = ex2_far(ref);
    o.x *= f2; o.y *= f2; o.z *= f2; o.w *= f2;
    if (col == 0 && p.lse != nullptr) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    T *dst = static_cast<T *>(p.out) + row * D + col;
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(dst) = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * f, o.y * f), c = __floats2bfloat162_rn(o.z * f, o.w * f);
        *reinterpret_cast<uint2 *>(dst) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&c));
    }
}

template <int D, int NT, bool SPLIT>
__global__ void __launch_bounds__(Q8Plan<D, NT, SPLIT>::WARPS * 32, Q8Plan<D, NT, SPLIT>::BLOCKS)
    decode_q8_kernel(const DecodeQ8Params p)
{
    using PL = Q8Plan<D, NT, SPLIT>;
    using T = typename std::conditional<SPLIT, float, __nv_bfloat16>::type;
    constexpr int CPR = D / 16;              // 16-byte chunks of a row
    constexpr int KC = D / 64;               // chunks of a key row that a lane takes
    constexpr int KS = D / 16;               // steps of the first product's inner dimension
    constexpr int DT = D / 16;               // 16-dim tiles of the output
    constexpr int VB = D == 64 ? 8 : 16;     // bytes of a value row that a lane takes at once
    constexpr int VC = D == 256 ? 2 : 1;     // how often
    constexpr int S = PL::STAGES, W = PL::WARPS, SUB = PL::SUB, STEP = PL::STEP;
    constexpr int SCALES = 2 * STEP * D;     // where a stage keeps its scales; 16 bytes on, what it holds
    extern __shared__ __align__(128) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_addr(smem) + warp * (S * PL::STAGE);
    // parts of row tiles that this block's warps leave: a warp's first one (if others follow) in the
    // workspace, its last one in its ring: {row tile or -1, first step, behind the last, steps of the tile}
    __shared__ int4 s_part[2 * W];
    if (threadIdx.x < 2 * W) s_part[threadIdx.x] = make_int4(-1, 0, 0, 0);
    pdl_trigger();
    pdl_wait();
    const Range range = find_range<W, STEP>(p);
    __syncthreads();                         // (s_part)

    // ---- copies: one step ahead by step into the ring ----
    Walk<STEP> ld(p, range);
    const Walk<STEP> first = ld;
    int page_at = -1, pages = 0;             // the 32 table entries in this warp's lanes: first one's number
    int ld_b = -1, ld_hr = -1;
    long long head = 0;                      // the loaded row tile's head's first page
    // where this lane's chunk i * 32 + lane of a step's rows goes: chunk c of row r lies at c ^ 4 (r & 1) for
    // keys and at c ^ 2 (r / 2 & 3) for values (64 dims: c and c ^ 2 (r / 2 & 1)), which keeps the
    // fragments' reads free of bank conflicts (the values of 64 dims: two ways).  A copy's rows are
    // 32 / CPR further on than the last one's, which turns the values' swizzle but not the keys'.
    const int row0 = lane / CPR, c0 = lane % CPR;
    const uint32_t k_to = row0 * D + (D == 64 ? c0 : c0 ^ ((row0 & 1) << 2)) * 16;
    const uint32_t v_to = row0 * D + (D == 64 ? c0 ^ ((row0 >> 1 & 1) << 1) : c0 ^ ((row0 >> 1 & 3) << 1)) * 16;
    auto v_turn = [](int i) -> uint32_t { return D == 64 ? 0u : (uint32_t)(i * (32 / CPR) >> 1 & 3) << 5; };
    auto fetch = [&](int slot) {
        const uint32_t st = ring + slot * PL::STAGE;
        if (ld.more()) {
            if (ld.hr != ld_hr) {            // (a division, once a row tile)
                ld_hr = ld.hr;
                head = (long long)(p.RT == 1 ? ld.hr : ld.hr / p.RT) * p.n_pool;
            }
#pragma unroll
            for (int sub = 0; sub < SUB; ++sub) {
                const int pos = ld.step * STEP + sub * kSub, n = ld.step * SUB + sub;
                const int lb = p.magic != 0 ? (int)__umulhi((unsigned)n, p.magic) : n;
                const int valid = min(kSub, ld.len - pos);   // none behind the last slot, and in an empty sequence
                if (ld.b != ld_b || lb < page_at || lb >= page_at + 32) {
                    ld_b = ld.b;
                    page_at = lb & ~31;
                    pages = page_at + lane < p.max_blocks
                                ? __ldg(p.table + (size_t)ld.b * p.max_blocks + page_at + lane) : 0;
                }
                int id = __shfl_sync(0xffffffffu, pages, lb - page_at);
                if (id < 0 || id >= p.n_pool) {
                    if (valid > 0 && lane == 0) record_code(p.dev_code, kDevBadBlk_);
                    id = 0;
                }
                const long long page = head + id;
                const long long at = (page * p.bs + (pos - lb * p.bs)) * D + lane * 16;
                const uint8_t *k = p.k + at, *v = p.v + at;
                const uint32_t to = st + sub * 2 * kSub * D;
                if (valid == kSub) {
#pragma unroll
                    for (int i = 0; i < CPR / 2; ++i) {
                        cp_16(to + k_to + i * 512, k + i * 512);
                        cp_16(to + kSub * D + (v_to ^ v_turn(i)) + i * 512, v + i * 512);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < CPR / 2; ++i) {
                        const bool ok = (i * 32 + lane) / CPR < valid;
                        cp_16(to + k_to + i * 512, k + i * 512, ok);
                        cp_16(to + kSub * D + (v_to ^ v_turn(i)) + i * 512, v + i * 512, ok);
                    }
                }
                if (lane < 2) cp_4(st + SCALES + sub * 8 + lane * 4, (lane == 0 ? p.ks : p.vs) + page);
            }
            if (lane == 0) {
                const uint32_t m = st + SCALES + 16;
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(m), "r"(ld.b), "r"(ld.hr), "r"(ld.step),
                             "r"(ld.len)
                             : "memory");
            }
            ld.next(p);
        } else if (lane == 0) {
            const uint32_t m = st + SCALES + 16;
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(m), "r"(-1), "r"(0), "r"(0), "r"(0)
                         : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < S - 1; ++i) fetch(i);

    // ---- the row tile being worked on ----
    uint32_t bq[NT][KS][2], bl[SPLIT ? NT : 1][SPLIT ? KS : 1][2];
    float fq[NT][2];                         // row 2t, 2t + 1: the query's power of two times scale
    float o[DT][NT][4];
    float m[NT][2], ref[NT][2], l[NT][2];    // of the logits; of the weights, relative to m
    int cur_b = -1, cur_hr = -1, cur_len = 0, cur_n = 0, first_step = 0;

    auto begin = [&](int b, int hr) {
        const int h = hr / p.RT, r0 = (hr - h * p.RT) * NT * 8;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = r0 + nt * 8 + g;
            const T *q = static_cast<const T *>(p.q) + ((size_t)b * p.Hq + h * p.G + row) * D;
            float x[KC][16];
            float big = 0.f;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                if (row < p.G) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(q + (t + 4 * c) * 16);
#pragma unroll
                    for (int j = 0; j < (SPLIT ? 4 : 2); ++j) {
                        const uint4 y = __ldg(src + j);
                        if constexpr (SPLIT) {
                            x[c][4 * j] = __uint_as_float(y.x); x[c][4 * j + 1] = __uint_as_float(y.y);
                            x[c][4 * j + 2] = __uint_as_float(y.z); x[c][4 * j + 3] = __uint_as_float(y.w);
                        } else {
                            x[c][8 * j] = bf16_lo(y.x); x[c][8 * j + 1] = bf16_hi(y.x);
                            x[c][8 * j + 2] = bf16_lo(y.y); x[c][8 * j + 3] = bf16_hi(y.y);
                            x[c][8 * j + 4] = bf16_lo(y.z); x[c][8 * j + 5] = bf16_hi(y.z);
                            x[c][8 * j + 6] = bf16_lo(y.w); x[c][8 * j + 7] = bf16_hi(y.w);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[c][j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) big = fmaxf(big, fabsf(x[c][j]));
            }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            int e = (int)(__float_as_uint(big) >> 23) - 127;
            e = big == 0.f ? 14 : (e < -112 ? -112 : e);
            const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
            const float down = __uint_as_float((uint32_t)(e - 14 + 127) << 23);
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float a = x[c][4 * j + 2 * u] * up, d = x[c][4 * j + 2 * u + 1] * up;
                        const uint32_t hi = pack_h2(a, d);
                        bq[nt][c * 4 + j][u] = hi;
                        if constexpr (SPLIT) {
                            const float2 y = unpack_h2(hi);
                            bl[nt][c * 4 + j][u] = pack_h2(a - y.x, d - y.y);
                        }
                    }
            fq[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t) * p.scale;
            fq[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4) * p.scale;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                m[nt][r] = kNone;
                ref[nt][r] = l[nt][r] = 0.f;
            }
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int r = 0; r < 4; ++r) o[d][nt][r] = 0.f;
        }
    };
    // Outputs of the row tile, or the state of its part.
    auto finish = [&](int b, int hr, int lo, int hi, int n, bool last) {
        const int h = hr / p.RT, r0 = (hr - h * p.RT) * NT * 8;
        const bool whole = lo == 0 && hi == n;
        float *po = nullptr, *pm = nullptr;
        if (!whole) {
            const size_t at = (size_t)blockIdx.x * W + warp;
            po = last ? reinterpret_cast<float *>(smem + warp * (S * PL::STAGE)) : p.ws_wo + at * p.RP * D;
            pm = last ? po + p.RP * D : p.ws_wml + at * p.RP * 4;
            if (lane == 0) s_part[2 * warp + (last ? 1 : 0)] = make_int4(b * p.HR + hr, lo, hi, n);
        } else if (p.by_tile && !p.whole && lane == 0) {
            p.ws_first[b * p.HR + hr] = -1;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float sum = l[nt][r];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int row = nt * 8 + 2 * t + r;
                if (r0 + row >= p.G) continue;
                const size_t out_row = (size_t)b * p.Hq + h * p.G + r0 + row;
                float f = 1.f, f2 = 1.f;
                if (whole) {
                    f = sum == 0.f ? 0.f : ex2_near(ref[nt][r]) / sum;
                    f2 = ex2_far(ref[nt][r]);
                    if (g == 0 && p.lse != nullptr)
                        p.lse[out_row] = sum == 0.f ? -INFINITY : (m[nt][r] + log2f(sum)) * kLn2;
                } else if (g == 0) {
                    reinterpret_cast<float4 *>(pm)[row] = make_float4(m[nt][r], sum, ref[nt][r], 0.f);
                }
#pragma unroll
                for (int c = 0; c < VC; ++c) {
                    // VB consecutive dims of this row: tiles c * 8 .., a pair of dims each
                    const int d0 = (g + 8 * c) * VB;
                    float y[VB];
#pragma unroll
                    for (int i = 0; i < VB / 2; ++i) {
                        y[2 * i] = o[c * 8 + i][nt][r] * f2 * f;
                        y[2 * i + 1] = o[c * 8 + i][nt][2 + r] * f2 * f;
                    }
                    if (!whole || SPLIT) {
                        float *dst = whole ? static_cast<float *>(p.out) + out_row * D + d0 : po + row * D + d0;
#pragma unroll
                        for (int i = 0; i < VB; i += 4)
                            *reinterpret_cast<float4 *>(dst + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
                    } else {
                        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + out_row * D + d0;
#pragma unroll
                        for (int i = 0; i < VB; i += 8) {
                            uint32_t z[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const __nv_bfloat162 two = __floats2bfloat162_rn(y[i + 2 * j], y[i + 2 * j + 1]);
                                z[j] = *reinterpret_cast<const uint32_t *>(&two);
                            }
                            *reinterpret_cast<uint4 *>(dst + i) = make_uint4(z[0], z[1], z[2], z[3]);
                        }
                    }
                }
            }
    };

    if (first.more()) {                      // (while the first steps are on their way)
        cur_b = first.b;
        cur_hr = first.hr;
        cur_len = first.len;
        first_step = first.step;
        begin(cur_b, cur_hr);
    }
    int slot = 0, put = S - 1;
#pragma unroll 1
    for (;;) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        __syncwarp();                        // the step is there for every lane, and the one before is used up
        fetch(put);
        put = put + 1 == S ? 0 : put + 1;
        const uint32_t st = ring + slot * PL::STAGE;
        const uint4 what = lds_16(st + SCALES + 16);
        const int b = (int)what.x, hr = (int)what.y, step = (int)what.z, len = (int)what.w;
        if (b != cur_b || hr != cur_hr) {
            if (cur_b >= 0) finish(cur_b, cur_hr, first_step, first_step + cur_n, steps_of<STEP>(cur_len), b < 0);
            if (b < 0) break;
            cur_b = b;
            cur_hr = hr;
            cur_len = len;
            cur_n = 0;
            first_step = step;
            begin(b, hr);
        }
        ++cur_n;
        const int pos = step * STEP, valid = len - pos;      // (STEP or more of a full step)
        // ---- S^T = K Q^T: slots g and g + 8 of a product, rows 2t and 2t + 1 of the tile ----
        float c[SUB][NT][2][4];
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub) {
            const uint32_t sk_base = st + sub * 2 * kSub * D;
#pragma unroll
            for (int h = 0; h < KC; ++h) {
                const int ch = t + 4 * h, sw = D == 64 ? ch : ch ^ ((g & 1) << 2);
                const uint4 ka = lds_16(sk_base + g * D + sw * 16), kb = lds_16(sk_base + (g + 8) * D + sw * 16);
                const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t a[4];
                    cvt_e4m3x4(wa[j], a[0], a[2]);
                    cvt_e4m3x4(wb[j], a[1], a[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float(&cc)[2][4] = c[sub][nt];
                        if (h == 0 && j < 2) mma_16816_new(cc[j], a, bq[nt][j][0], bq[nt][j][1]);
                        else mma_16816(cc[j & 1], a, bq[nt][h * 4 + j][0], bq[nt][h * 4 + j][1]);
                        if constexpr (SPLIT) mma_16816(cc[j & 1], a, bl[nt][h * 4 + j][0], bl[nt][h * 4 + j][1]);
                    }
                }
            }
        }
        // ---- softmax ----
        float evf[SUB], fv[SUB];             // the value scale as 2^ev * fv, fv in [1, 2)
        float x[SUB][NT][4];                 // log2 units: (slot g, row 2t), (g, 2t+1), (g+8, 2t), (g+8, 2t+1)
        bool rise = false;
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub) {
            const uint2 scales = lds_8(st + SCALES + sub * 8);
            // (a product behind the last slot has no page of its own, and any scale)
            const float sk = __uint_as_float(scales.x), sv = valid > sub * kSub ? __uint_as_float(scales.y) : 1.f;
            int ev = (int)((__float_as_uint(sv) >> 23) & 255u) - 127;
            ev = ev < -126 ? -126 : (ev > 126 ? 126 : ev);
            fv[sub] = sv * __uint_as_float((uint32_t)(127 - ev) << 23);
            evf[sub] = (float)ev;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float f0 = fq[nt][0] * sk, f1 = fq[nt][1] * sk;
                float *xs = x[sub][nt];
#pragma unroll
                for (int i = 0; i < 4; ++i) xs[i] = c[sub][nt][0][i] + c[sub][nt][1][i];
                if (p.logits != nullptr) {
                    const int h = hr / p.RT, r0 = (hr - h * p.RT) * NT * 8 + nt * 8 + 2 * t, at = sub * kSub + g;
                    float *dst = p.logits + ((size_t)b * p.Hq + h * p.G + r0) * p.logits_stride + pos + at;
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (r0 + r < p.G) {
                            if (at < valid) dst[r * p.logits_stride] = xs[r] * (r ? f1 : f0);
                            if (at + 8 < valid) dst[r * p.logits_stride + 8] = xs[2 + r] * (r ? f1 : f0);
                        }
                }
                const float e0 = f0 * kLog2e, e1 = f1 * kLog2e;
#pragma unroll
                for (int i = 0; i < 4; ++i) xs[i] *= i & 1 ? e1 : e0;
                if (valid < (sub + 1) * kSub) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (sub * kSub + g + (i >> 1) * 8 >= valid) xs[i] = -INFINITY;
                }
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    rise |= fmaxf(xs[r], xs[2 + r]) - m[nt][r] > fminf(0.f, ref[nt][r] - evf[sub]) + kSlack;
            }
        }
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float y[SUB], xm = -INFINITY, want = -INFINITY;
#pragma unroll
                    for (int sub = 0; sub < SUB; ++sub) {
                        y[sub] = row_max(fmaxf(x[sub][nt][r], x[sub][nt][2 + r]));
                        xm = fmaxf(xm, y[sub]);
                    }
                    const float m1 = xm - m[nt][r] > kSlack ? xm : m[nt][r];
#pragma unroll
                    for (int sub = 0; sub < SUB; ++sub) want = fmaxf(want, y[sub] - m1 + evf[sub]);
                    const float dm = m[nt][r] - m1, now = ref[nt][r] + dm;      // the reference from m1 on
                    const float r1 = want > now + kSlack ? ceilf(want) : rintf(now);
                    const float f = ex2(dm + (ref[nt][r] - r1));
                    l[nt][r] *= ex2(dm);
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        o[d][nt][r] *= f;
                        o[d][nt][2 + r] *= f;
                    }
                    m[nt][r] = m1;
                    ref[nt][r] = r1;
                }
        }
        if (step % kLook == kLook - 1) {     // do all slots of a row lie low?  4 bits of the vote for each t
            float top[NT][2];
            uint32_t low = ~(15u << (4 * t));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float y = -INFINITY;
#pragma unroll
                    for (int sub = 0; sub < SUB; ++sub)
                        y = fmaxf(y, fmaxf(x[sub][nt][r], x[sub][nt][2 + r]) - m[nt][r] + evf[sub]);
                    top[nt][r] = y;
                    low |= y < ref[nt][r] - kSlack ? 1u << (4 * t + 2 * nt + r) : 0u;
                }
            if ((__reduce_and_sync(0xffffffffu, low) & 0xffffu) != 0u) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float want = row_max(top[nt][r]);
                        float big = 0.f;
#pragma unroll
                        for (int d = 0; d < DT; ++d) big = fmaxf(big, fmaxf(fabsf(o[d][nt][r]), fabsf(o[d][nt][2 + r])));
                        // as far as the sums stay in their range, and not for -inf alone
                        const int room = kTop + 127 - (int)(__float_as_uint(row_max(big)) >> 23);
                        float r1 = ref[nt][r];
                        if (want < r1 - kSlack && want > -INFINITY)
                            r1 = ceilf(fmaxf(want, r1 - (float)max(0, min(126, room))));
                        const float f = ex2(ref[nt][r] - r1);
#pragma unroll
                        for (int d = 0; d < DT; ++d) {
                            o[d][nt][r] *= f;
                            o[d][nt][2 + r] *= f;
                        }
                        ref[nt][r] = r1;
                    }
            }
        }
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub) {
            uint32_t pw[NT][2], pl[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float y[4];
                const float to[2] = {evf[sub] + kBoost - ref[nt][0], evf[sub] + kBoost - ref[nt][1]};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float u = x[sub][nt][i] - m[nt][i & 1];
                    l[nt][i & 1] += ex2(u);
                    y[i] = ex2(u + to[i & 1]) * fv[sub];
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t hi = pack_h2(y[2 * i], y[2 * i + 1]);
                    pw[nt][i] = transpose_8x8(hi);
                    const float2 z = unpack_h2(hi);
                    pl[nt][i] = transpose_8x8(pack_h2(y[2 * i] - z.x, y[2 * i + 1] - z.y));
                }
            }
            // ---- O^T += V^T P^T: slots 2t, 2t + 1, 2t + 8, 2t + 9 of VB dims ----
            const uint32_t sv_base = st + (sub * 2 + 1) * kSub * D;
#pragma unroll
            for (int vc = 0; vc < VC; ++vc) {
                uint32_t r[4][VB / 4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 2 * t + (i & 1) + (i >> 1) * 8;
                    if constexpr (VB == 16) {
                        const int ch = (g + 8 * vc) ^ (t << 1);
                        const uint4 y = lds_16(sv_base + row * D + ch * 16);
                        r[i][0] = y.x; r[i][1] = y.y; r[i][2] = y.z; r[i][3] = y.w;
                    } else {
                        const int ch = (g >> 1) ^ ((t & 1) << 1);
                        const uint2 y = lds_8(sv_base + row * D + ch * 16 + (g & 1) * 8);
                        r[i][0] = y.x; r[i][1] = y.y;
                    }
                }
#pragma unroll
                for (int q = 0; q < VB / 4; ++q)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t lo = __byte_perm(r[0][q], r[1][q], u ? 0x7362 : 0x5140);
                        const uint32_t hi = __byte_perm(r[2][q], r[3][q], u ? 0x7362 : 0x5140);
                        uint32_t a[4];
                        cvt_e4m3x4(lo, a[0], a[1]);
                        cvt_e4m3x4(hi, a[2], a[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_16816(o[vc * 8 + q * 2 + u][nt], a, pw[nt][0], pw[nt][1]);
                            mma_16816(o[vc * 8 + q * 2 + u][nt], a, pl[nt][0], pl[nt][1]);
                        }
                    }
            }
        }
        slot = slot + 1 == S ? 0 : slot + 1;
    }
    // ---- the block's parts, in order: those of one row tile are joined, a row a warp ----
    __syncthreads();
    const int4 mine = lane < 2 * W ? s_part[lane] : make_int4(-1, 0, 0, 0);
    const uint32_t parts = __ballot_sync(0xffffffffu, mine.x >= 0);
    const uint32_t below = parts & ((1u << lane) - 1u);
    const int tile_below = __shfl_sync(0xffffffffu, mine.x, below != 0 ? 31 - __clz(below) : 0);
    uint32_t firsts = __ballot_sync(0xffffffffu, mine.x >= 0 && (below == 0 || tile_below != mine.x));
    bool begun = false;                      // a row tile begins here and ends in a later block
    int turn = warp;                         // rows are dealt out to the warps in turn
#pragma unroll 1
    while (firsts != 0) {
        const int i = __ffs(firsts) - 1;
        firsts &= firsts - 1;
        const uint32_t members = parts & ~((1u << i) - 1u) & (firsts != 0 ? (1u << (__ffs(firsts) - 1)) - 1u : ~0u);
        const int tile = __shfl_sync(0xffffffffu, mine.x, i), lo = __shfl_sync(0xffffffffu, mine.y, i);
        const int n = __shfl_sync(0xffffffffu, mine.w, i), hi = __shfl_sync(0xffffffffu, mine.z, 31 - __clz(members));
        const bool whole = lo == 0 && hi == n;
        const int b = tile / p.HR, hr = tile - b * p.HR, h = hr / p.RT, r0 = (hr - h * p.RT) * NT * 8;
        const int rows = min(p.RP, p.G - r0);
        // part x: odd ones in the ring of warp x / 2, even ones in the workspace
        const float *ring_o = reinterpret_cast<const float *>(smem);
        const size_t ws_at = (size_t)blockIdx.x * W * p.RP;
        constexpr int RING = S * PL::STAGE / 4;
        int row = turn;
        for (; row < rows; row += W) {
            // lane x has part x's state, and then its factor
            float4 y = make_float4(kNone, 0.f, kNone, 0.f);
            if (members >> lane & 1u)
                y = lane & 1 ? reinterpret_cast<const float4 *>(ring_o + (lane >> 1) * RING + p.RP * D)[row]
                             : reinterpret_cast<const float4 *>(p.ws_wml)[ws_at + (lane >> 1) * p.RP + row];
            float m1 = 0.f, r1 = 0.f, sum = 0.f, f = 0.f;
#pragma unroll
            for (int c = 0; c < (D + 127) / 128; ++c) {
                const int col = c * 128 + lane * 4;
                const bool in = col < D;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f), z[2 * W];
#pragma unroll
                for (int x = 0; x < 2 * W; ++x) {
                    z[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (in && (members >> x & 1u))
                        z[x] = *reinterpret_cast<const float4 *>(
                            x & 1 ? ring_o + (x >> 1) * RING + row * D + col
                                  : p.ws_wo + (ws_at + (x >> 1) * p.RP + row) * D + col);
                }
                if (c == 0) {                // (while those are on their way)
                    m1 = warp_max(y.x);
                    const float dm = y.x - m1;
                    r1 = ceilf(warp_max(y.z + dm));
                    sum = warp_sum(y.y * ex2(dm));
                    f = ex2(dm + (y.z - r1));
                }
#pragma unroll
                for (int x = 0; x < 2 * W; ++x) {
                    const float fx = __shfl_sync(0xffffffffu, f, x);
                    acc.x = fmaf(fx, z[x].x, acc.x);
                    acc.y = fmaf(fx, z[x].y, acc.y);
                    acc.z = fmaf(fx, z[x].z, acc.z);
                    acc.w = fmaf(fx, z[x].w, acc.w);
                }
                if (!in) continue;
                // (of a row tile that began before this block the state is the block's first)
                const size_t part = ((size_t)blockIdx.x * 2 + (lo == 0 ? 1 : 0)) * p.RP + row;
                if (whole) store_row<T>(p, (size_t)b * p.Hq + h * p.G + r0 + row, D, col, m1, sum, r1, acc);
                else *reinterpret_cast<float4 *>(p.ws_o + part * D + col) = acc;
                if (!whole && col == 0) reinterpret_cast<float4 *>(p.ws_ml)[part] = make_float4(m1, sum, r1, 0.f);
            }
        }
        turn = row - rows;
        if (threadIdx.x == 0 && !p.whole) {
            if (lo == 0 && p.by_tile) p.ws_first[tile] = whole ? -1 : (int)blockIdx.x;
            if (lo == 0 && !whole && !p.by_tile) p.ws_first[blockIdx.x] = tile;
            if (lo > 0 && hi == n) p.ws_last[tile] = (int)blockIdx.x;
        }
        begun |= lo == 0 && !whole;
    }
    if (threadIdx.x == 0 && !p.whole && !p.by_tile && !begun) p.ws_first[blockIdx.x] = -1;
}

// Joins the parts that several blocks left of a row tile: a row a block, 4 columns a thread, the parts in
// turn over sets of threads that each keep a state of their own, so that states and outputs are read at
// once (two trips to memory in all: where the parts are, and the parts).
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) decode_q8_merge_kernel(const DecodeQ8Params p)
{
    constexpr int LPR = D / 4;               // threads of a row
    constexpr int SETS = kMergeThreads / LPR;
    __shared__ float4 s_o[kMergeThreads], s_m[SETS];
    const int row = blockIdx.y, tid = threadIdx.x, set = tid / LPR, col = tid % LPR * 4;
    pdl_trigger();
    pdl_wait();
    const int first = p.ws_first[blockIdx.x], tile = p.by_tile ? (int)blockIdx.x : first;
    int last = p.by_tile ? p.ws_last[tile] : 0;      // (no matter what where the tile is whole)
    if (first < 0) return;
    if (!p.by_tile) last = p.ws_last[tile];
    const int w0 = p.by_tile ? first : (int)blockIdx.x, nseg = last - w0 + 1;
    const int b = tile / p.HR, hr = tile - b * p.HR, h = hr / p.RT, r0 = (hr - h * p.RT) * p.RP;
    if (row >= min(p.RP, p.G - r0)) return;
    const float4 *ml = reinterpret_cast<const float4 *>(p.ws_ml);
    float m = kNone, ref = 0.f, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 4;
    for (int i0 = set; i0 < nseg; i0 += SETS * U) {
        float4 y[U], z[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * SETS;
            y[u] = make_float4(kNone, 0.f, kNone, 0.f);
            z[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < nseg) {
                const size_t part = ((size_t)(w0 + i) * 2 + (i == 0 ? 1 : 0)) * p.RP + row;
                y[u] = __ldcg(ml + part);
                z[u] = __ldcg(reinterpret_cast<const float4 *>(p.ws_o + part * D + col));
            }
        }
        float m1 = m;
#pragma unroll
        for (int u = 0; u < U; ++u) m1 = fmaxf(m1, y[u].x);
        const float dm = m - m1;
        float r1 = ref + dm;
#pragma unroll
        for (int u = 0; u < U; ++u) r1 = fmaxf(r1, y[u].z + (y[u].x - m1));
        r1 = ceilf(r1);
        const float f = ex2(dm + (ref - r1));
        l *= ex2(dm);
        o.x *= f; o.y *= f; o.z *= f; o.w *= f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float du = y[u].x - m1, g = ex2(du + (y[u].z - r1));
            l = fmaf(y[u].y, ex2(du), l);
            o.x = fmaf(g, z[u].x, o.x);
            o.y = fmaf(g, z[u].y, o.y);
            o.z = fmaf(g, z[u].z, o.z);
            o.w = fmaf(g, z[u].w, o.w);
        }
        m = m1;
        ref = r1;
    }
    s_o[tid] = o;
    if (tid % LPR == 0) s_m[set] = make_float4(m, l, ref, 0.f);
    __syncthreads();
    if (set != 0) return;
#pragma unroll
    for (int s = 1; s < SETS; ++s) m = fmaxf(m, s_m[s].x);
    ref = -INFINITY;
#pragma unroll
    for (int s = 0; s < SETS; ++s) ref = fmaxf(ref, s_m[s].z + (s_m[s].x - m));
    ref = ceilf(ref);
    l = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < SETS; ++s) {
        const float4 y = s_m[s], z = s_o[s * LPR + tid];
        const float dm = y.x - m, g = ex2(dm + (y.z - ref));
        l = fmaf(y.y, ex2(dm), l);
        o.x = fmaf(g, z.x, o.x);
        o.y = fmaf(g, z.y, o.y);
        o.z = fmaf(g, z.z, o.z);
        o.w = fmaf(g, z.w, o.w);
    }
    store_row<T>(p, (size_t)b * p.Hq + h * p.G + r0 + row, D, col, m, l, ref, o);
}

template <int D, int NT, bool SPLIT>
cudaError_t launch_typed(DecodeQ8Params p, cudaStream_t stream)
{
    using PL = Q8Plan<D, NT, SPLIT>;
    using T = typename std::conditional<SPLIT, float, __nv_bfloat16>::type;
    static_assert(PL::STAGES >= 3, "two steps in flight at least");
    static_assert(8 * NT * (D + 4) * 4 <= PL::STAGES * PL::STAGE, "a part fits its warp's ring");
    static bool configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !configured[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(decode_q8_kernel<D, NT, SPLIT>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, PL::SMEM);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    // no more blocks than the capacity can give work
    const long long tiles = (long long)p.B * p.HR, steps = (p.cap + PL::STEP - 1) / PL::STEP;
    const long long units = tiles * (steps + kEnd);
    const int grid = (int)std::min<long long>(p.blocks, p.whole ? tiles : units / kMinUnits + 1);
    p.small = units <= 0x7fffffffLL;
    cudaError_t e = launch_pdl(decode_q8_kernel<D, NT, SPLIT>, dim3((unsigned)grid), dim3(PL::WARPS * 32), PL::SMEM,
                               stream, p);
    if (e != cudaSuccess || p.whole) return e;
    return launch_pdl(decode_q8_merge_kernel<T, D>, dim3((unsigned)(p.by_tile ? tiles : grid), (unsigned)p.RP),
                      dim3(kMergeThreads), 0, stream, p);
}

}  // namespace

// Row tiles of 8 heads, of 16 where a group has more and that pays.  fp32 queries of 128 dims, tiles of 8 and of 16:
// 28 x 3963 to 6241 slots of 3 heads, groups of 12 47.0 and 42.6 us, 2 x 32768 of 8 heads, groups of 9 51.3 and 46.1, but
// groups of 24, which are three tiles or two, 36.7 and 39.5.  No gain with 64 dims (groups of 16 32.4 and 32.1), nor with
// bf16 queries of 256 (groups of 12 61.5 and 67.2).
static int tiles_of_8(int G, int D, bool bf16)
{
    if (bf16) return G > 8 && D <= 128 ? 2 : 1;
    return D == 128 && (G - 1) % 16 >= 8 ? 2 : 1;
}

DecodeQ8Plan decode_q8_plan(int B, int Hkv, int G, int D, bool bf16, int n_sm)
{
    DecodeQ8Plan pl{};
    const int NT = tiles_of_8(G, D, bf16);
    pl.RT = (G + 8 * NT - 1) / (8 * NT);
    pl.RP = G < 8 * NT ? G : 8 * NT;
    const bool two = D <= 128 && NT == 1 && bf16;        // blocks per SM, as Q8Plan says
    pl.blocks = n_sm * (two ? 2 : 1);
    const long long tiles = (long long)B * Hkv * pl.RT;
    const int most = pl.blocks;
    pl.by_tile = tiles <= most;
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    const size_t rows = (size_t)most * 2 * pl.RP, warp_rows = (size_t)most * warps_of(D, NT, !bf16) * pl.RP;
    pl.off_first = 0;
    pl.off_last = up((size_t)most * sizeof(int32_t));
    pl.off_ml = up(pl.off_last + (size_t)tiles * sizeof(int32_t));
    pl.off_o = up(pl.off_ml + rows * sizeof(float4));
    pl.off_wml = up(pl.off_o + rows * D * sizeof(float));
    pl.off_wo = up(pl.off_wml + warp_rows * sizeof(float4));
    pl.bytes = up(pl.off_wo + warp_rows * D * sizeof(float));
    return pl;
}

cudaError_t launch_decode_q8(DecodeQ8Params p, int D, bool bf16, cudaStream_t stream)
{
    // Row tiles stay in one block each, and no second kernel is needed, where that leaves the fullest block
    // little more than the mean: by the capacity (which the host knows), and with few steps a block, since the
    // lengths behind it may differ.  Measured with 52 steps of 128 dims, whole and split: 512 row tiles on 304
    // blocks (16 steps above the mean) 25.4 and 27.6 us.  Lengths well below the capacity lose by it: 400 to 832 slots
    // 24.4 and 23.3 us, 100 to 832 24.1 and 20.9, 1 to 832 23.9 and 19.7.
    const int step = kSub * subs_of(D);
    const long long tiles = (long long)p.B * p.HR, steps = (p.cap + step - 1) / step;
    const long long fullest = (tiles + p.blocks - 1) / p.blocks * steps;
    p.whole = steps <= kWholeSteps || (fullest * step * D <= 128 * 16 * 128 &&
                                       (fullest - tiles * steps / p.blocks) * step * D <= kWholeWait * 16 * 128);
    const bool wide = tiles_of_8(p.G, D, bf16) == 2;
    if (bf16) {
        switch (D) {
        case 64: return wide ? launch_typed<64, 2, false>(p, stream) : launch_typed<64, 1, false>(p, stream);
        case 128: return wide ? launch_typed<128, 2, false>(p, stream) : launch_typed<128, 1, false>(p, stream);
        default: return launch_typed<256, 1, false>(p, stream);
        }
    }
    switch (D) {
    case 64: return launch_typed<64, 1, true>(p, stream);
    case 128: return wide ? launch_typed<128, 2, true>(p, stream) : launch_typed<128, 1, true>(p, stream);
    default: return launch_typed<256, 1, true>(p, stream);
    }
}

}  // namespace kvc

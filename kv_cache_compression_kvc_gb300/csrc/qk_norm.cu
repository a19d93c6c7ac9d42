// qk_norm.cu -- RMS norm of every query and key head and the rotation to the token's position, in
// one pass over the rows.
//
//   y = x * rsqrt(mean(x^2) + eps) * w          (fp32; over the d_head elements of a row)
//   first d_rot elements, pairs (i, i + d_rot/2):  (a c - b s, b c + a s)
//   with c, s = row pos of the table; one rounding, to the rows' type.
//
// Bound by HBM (an element is read once and written once) as long as the instructions are few.  A row
// lies in D/8 lanes, and a lane holds 4 elements and their 4 partners, so that the rotation needs no
// exchange (with 8 neighbours a lane it took 8 shuffles a row: 151 us for 32768 tokens of 32 + 8 heads of
// 128, bf16); where only a part is rotated, the lanes behind it hold 8 neighbours.  Weights and angles
// are multiplied once for the rows of a unit (some rows per lane group, of one kind), which leaves three
// products an element:
//   out_a = r (a (w_a c) - b (w_b s)),  out_b = r (b (w_b c) + a (w_a s)),  r = rsqrt(mean + eps).
// The rows side by side in a warp are neighbouring heads of a token; where that leaves lanes without rows
// (few heads), those of neighbouring tokens: 100000 tokens of 8 + 1 heads of 64, bf16, 81.6 -> 44.6 us, 20000 of
// 4 + 1, fp32, 12.7 -> 8.6, but the prompt above 108.8 -> 111.6.
// Persistent warps take whole tokens in turn, so that all read from one stretch of memory, and share the
// units of the last ones; a token's angles are read once for its units.  Measured on that prompt: 108.8 us
// (6.3 TB/s, 93 % of the copy rate) with 24 warps an SM and the next unit on its way into L2; 114 without the
// latter, 108.2 with a ring in shared memory instead (which costs 2 us of 17 at 5000 tokens), 113.5 with neighbouring
// tokens a warp, 127 with the next unit's rows in registers (spills), 159 with a warp per unit.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace kvc {

namespace {

constexpr int kWarps = 8;
constexpr int kBlocks = 3;                   // per SM
// Rows per lane group and unit.
template <typename T>
constexpr int kIterOf = sizeof(T) == 2 ? 4 : 2;
// Rows of 16 bits, read and written, from which on the next unit is fetched into L2: 168 MB 31.9 us without and
// 30.0 with it, 671 MB 114.7 and 108.8; where L2 holds them, 102 MB, 17.4 and 18.3.  fp32 rows, whose loads are twice
// as wide, lose: 478 MB 76.2 and 81.0.
constexpr long long kAheadBytes = 128 << 20;
constexpr int kDevBadPos = 4;                // KVC_DEV_BAD_POSITION

// 4 neighbouring elements as they lie in memory.
template <typename T>
struct Four;
template <>
struct Four<__nv_bfloat16> {
    uint2 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = ld_stream_8(p); }
    __device__ __forceinline__ void load_cached(const __nv_bfloat16 *p) { w = __ldg(reinterpret_cast<const uint2 *>(p)); }
    __device__ __forceinline__ void zero() { w = make_uint2(0, 0); }
    __device__ __forceinline__ void get(float2 *f) const
    {
        f[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x));
        f[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
    }
    static __device__ __forceinline__ uint32_t pack(float2 x)
    {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x.y), "f"(x.x));
        return r;
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float2 *f)
    {
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack(f[0]), pack(f[1]));
    }
};
template <>
struct Four<float> {
    uint4 w;
    __device__ __forceinline__ void load(const float *p) { w = ld_stream_16(p); }
    __device__ __forceinline__ void load_cached(const float *p) { w = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float2 *f) const
    {
        f[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
        f[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
    }
    static __device__ __forceinline__ void store(float *p, const float2 *f)
    {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    }
};

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

// The cosines and sines of a lane's 4 pairs.
struct Turn {
    float4 c, s;
    bool ok;                                 // the position lies in the table
    __device__ __forceinline__ void load(const QkNormParams &p, int pos, int j, bool first)
    {
        ok = pos >= 0 && pos < p.n_pos;
        if (!ok) {
            if (first) record_code(p.dev_code, kDevBadPos);
            return;
        }
        if (j >= p.rot / 2) return;          // (a lane that rotates nothing)
        const float *row = p.cos_sin + (size_t)pos * p.rot + j;
        c = __ldg(reinterpret_cast<const float4 *>(row));
        s = __ldg(reinterpret_cast<const float4 *>(row + p.rot / 2));
    }
};

// A warp's units: `rounds` whole groups of tokens, n_w apart, then `left` units in a row.
struct Units {
    int group, part, rounds, left, group1, part1, n_w, tasks;
    __device__ __forceinline__ Units(const QkNormParams &p, int tokens)
        : n_w((int)gridDim.x * kWarps), tasks(p.tasks)
    {
        const int n_groups = (p.n_tokens + tokens - 1) / tokens;
        const int w = (int)blockIdx.x * kWarps + (threadIdx.x >> 5);
        rounds = n_groups / n_w;
        const int first = rounds * n_w;
        const long long units = (long long)(n_groups - first) * tasks, u0 = units * w / n_w;
        left = (int)(units * (w + 1) / n_w - u0);
        group1 = first + (int)(u0 / tasks);
        part1 = (int)(u0 - u0 / tasks * tasks);
        group = rounds > 0 ? w : group1;
        part = rounds > 0 ? 0 : part1;
    }
    __device__ __forceinline__ bool any() const { return rounds > 0 || left > 0; }
    __device__ __forceinline__ void next()
    {
        if (rounds == 0) --left;
        if (++part < tasks) return;
        part = 0;
        if (rounds == 0) {
            ++group;
            return;
        }
        group += n_w;
        if (--rounds == 0) {
            group = group1;
            part = part1;
        }
    }
};

// TOKENS: the rows side by side in a warp are those of neighbouring tokens, else of neighbouring heads.
template <typename T, int D, bool TOKENS>
__global__ void __launch_bounds__(kWarps * 32, kBlocks) qk_norm_rope_kernel(const QkNormParams p)
{
    constexpr int kIter = kIterOf<T>;
    constexpr int LPR = D / 8;               // lanes per row
    constexpr int TOK = TOKENS ? 32 / LPR : 1;                 // tokens of a group
    constexpr int SIDE = TOKENS ? 1 : 32 / LPR;                // heads side by side
    constexpr int HEADS = SIDE * kIter;                        // of a unit
    const int lane = threadIdx.x & 31;
    Units u(p, TOK);
    pdl_trigger();
    pdl_wait();
    if (!u.any()) return;
    // this lane's elements: 4 at `at` and 4 at `at2`, its partners or its next ones
    const int l = lane & (LPR - 1), mine = TOKENS ? lane / LPR : 0, row0 = TOKENS ? 0 : lane / LPR;
    const bool turns = l * 8 < p.rot;
    const int at = turns ? l * 4 : l * 8, at2 = at + (turns ? p.rot / 2 : 4);
    const bool part_turns = p.rot < D;       // some lanes do not

    Turn turn;
    turn.c = make_float4(1.f, 1.f, 1.f, 1.f);
    turn.s = make_float4(0.f, 0.f, 0.f, 0.f);
    turn.ok = true;
    int tok = u.group * TOK + mine;
    int pos = p.rot > 0 && (!TOKENS || tok < p.n_tokens) ? p.pos[tok] : 0;
    constexpr int kLines = D * (int)sizeof(T) / 128;           // of a row
    bool fresh = p.rot > 0;                  // tokens whose angles are not there yet
#pragma unroll 1
    for (;;) {
        Four<T> raw[kIter][2];
        const bool is_k = u.part >= p.q_tasks;
        const int h0 = (is_k ? u.part - p.q_tasks : u.part) * HEADS + row0;
        const int all = is_k ? p.Hkv : p.Hq, heads = !TOKENS || tok < p.n_tokens ? all : 0;
        {
            const int64_t sh = is_k ? p.k_sh : p.q_sh;
            const T *src = static_cast<const T *>(is_k ? p.k : p.q) + tok * (is_k ? p.k_st : p.q_st) + h0 * sh;
#pragma unroll
            for (int i = 0; i < kIter; ++i)
                if (h0 + i * SIDE < heads) {
                    raw[i][0].load(src + i * SIDE * sh + at);
                    raw[i][1].load(src + i * SIDE * sh + at2);
                } else {
                    raw[i][0].zero();
                    raw[i][1].zero();
                }
        }
        const int group = u.group;
        u.next();
        const bool more = u.any();
        if (p.ahead && more) {               // the next unit into L2, a line of 128 bytes a lane
            const bool is_k = u.part >= p.q_tasks;
            const int t = u.group * TOK + lane / (kLines * HEADS);
            const int h = (is_k ? u.part - p.q_tasks : u.part) * HEADS + lane / kLines % HEADS;
            if (lane < kLines * HEADS * TOK && t < p.n_tokens && h < (is_k ? p.Hkv : p.Hq))
                prefetch_l2(static_cast<const T *>(is_k ? p.k : p.q) + t * (is_k ? p.k_st : p.q_st) +
                            h * (is_k ? p.k_sh : p.q_sh) + lane % kLines * (128 / (int)sizeof(T)));
        }
        if (fresh && (!TOKENS || tok < p.n_tokens)) turn.load(p, pos, at, l == 0);
        const int64_t sh = is_k ? p.ko_sh : p.qo_sh;
        const int next = u.group * TOK + mine;
        fresh = p.rot > 0 && more && u.group != group;
        if (fresh && (!TOKENS || next < p.n_tokens)) pos = p.pos[next];
        T *dst = static_cast<T *>(is_k ? p.k_out : p.q_out) + tok * (is_k ? p.ko_st : p.qo_st) + h0 * sh;
        const T *wt = static_cast<const T *>(is_k ? p.w_k : p.w_q);
        // a c, a s, b c, b s of the weights a, b of the two groups of elements
        float2 wa[2] = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)}, wb[2] = {wa[0], wa[1]};
        if (wt != nullptr) {
            Four<T> x;
            x.load_cached(wt + at);
            x.get(wa);
            x.load_cached(wt + at2);
            x.get(wb);
        }
        float2 ac[2], as[2], bc[2], bs[2];
        const float2 c[2] = {make_float2(turn.c.x, turn.c.y), make_float2(turn.c.z, turn.c.w)};
        const float2 s[2] = {make_float2(turn.s.x, turn.s.y), make_float2(turn.s.z, turn.s.w)};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            ac[k] = turns ? mul2(wa[k], c[k]) : wa[k];
            as[k] = mul2(wa[k], s[k]);
            bc[k] = turns ? mul2(wb[k], c[k]) : wb[k];
            bs[k] = neg2(mul2(wb[k], s[k]));
        }
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            if (h0 - row0 + i * SIDE >= all) break;       // (the same for the whole warp)
            float2 a[2], b[2];
            raw[i][0].get(a);
            raw[i][1].get(b);
            float r = 1.f;
            if (wt != nullptr) {
                float2 ss = mul2(a[0], a[0]);
                ss = __ffma2_rn(a[1], a[1], ss);
                ss = __ffma2_rn(b[0], b[0], ss);
                ss = __ffma2_rn(b[1], b[1], ss);
                float sum = ss.x + ss.y;
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                r = rsqrtf(sum * (1.f / D) + p.eps);
            }
            const float2 rr = make_float2(r, r);
            float2 ya[2], yb[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                ya[k] = mul2(a[k], ac[k]);
                yb[k] = mul2(b[k], bc[k]);
                if (p.rot > 0) {
                    const float2 ta = __ffma2_rn(b[k], bs[k], ya[k]), tb = __ffma2_rn(a[k], as[k], yb[k]);
                    // (an infinity in an element that does not turn stays there)
                    ya[k] = part_turns && !turns ? ya[k] : ta;
                    yb[k] = part_turns && !turns ? yb[k] : tb;
                }
                ya[k] = mul2(ya[k], rr);
                yb[k] = mul2(yb[k], rr);
            }
            if (h0 + i * SIDE < heads && turn.ok) {
                Four<T>::store(dst + i * SIDE * sh + at, ya);
                Four<T>::store(dst + i * SIDE * sh + at2, yb);
            }
        }
        if (!more) return;
        tok = next;
    }
}

template <typename T>
cudaError_t launch_typed(QkNormParams p, int D, int n_sm, cudaStream_t stream)
{
    // units of `side` tokens with their heads side by side, or with the tokens side by side
    const int side = 256 / D, n = kIterOf<T>;
    const auto parts = [](int heads, int per) { return (heads + per - 1) / per; };
    const bool by_tokens = side > 1 && parts(p.Hq, n) + parts(p.Hkv, n) < side * (parts(p.Hq, side * n) + parts(p.Hkv, side * n));
    const int tokens = by_tokens ? side : 1, heads = by_tokens ? n : side * n;         // of a unit
    p.q_tasks = parts(p.Hq, heads);
    p.tasks = p.q_tasks + parts(p.Hkv, heads);
    const long long units = ((long long)p.n_tokens + tokens - 1) / tokens * p.tasks, most = (long long)n_sm * kBlocks;
    const long long blocks = std::min((units + kWarps - 1) / kWarps, most);
    p.ahead = sizeof(T) == 2 && (long long)p.n_tokens * (p.Hq + p.Hkv) * D * 4 > kAheadBytes;
    const dim3 grid((unsigned)blocks), block(kWarps * 32);
    auto kernel = D == 64    ? by_tokens ? qk_norm_rope_kernel<T, 64, true> : qk_norm_rope_kernel<T, 64, false>
                  : D == 128 ? by_tokens ? qk_norm_rope_kernel<T, 128, true> : qk_norm_rope_kernel<T, 128, false>
                             : qk_norm_rope_kernel<T, 256, false>;
    return launch_pdl(kernel, grid, block, 0, stream, p);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormParams &p, int D, bool bf16, int n_sm, cudaStream_t stream)
{
    return bf16 ? launch_typed<__nv_bfloat16>(p, D, n_sm, stream) : launch_typed<float>(p, D, n_sm, stream);
}

}  // namespace kvc

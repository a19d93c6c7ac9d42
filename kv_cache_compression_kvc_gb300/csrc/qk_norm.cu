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
// are multiplied once for the rows of a unit (some rows per lane group, of one token and kind), which
// leaves three products an element:
//   out_a = r (a (w_a c) - b (w_b s)),  out_b = r (b (w_b c) + a (w_a s)),  r = rsqrt(mean + eps).
// Persistent warps take units in order, and a token's angles are read once for them.  Measured on that
// prompt: 114 us (6.0 TB/s, 89 % of the copy rate) with 24 warps an SM; 116 with 32 (64 registers), 127
// with the next unit's rows loaded ahead in registers (spills), 159 with a warp per unit.
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

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

// The cosines and sines of a lane's 4 pairs.
struct Turn {
    float4 c, s;
    bool ok;                                 // the position lies in the table
    __device__ __forceinline__ void load(const QkNormParams &p, int pos, int j)
    {
        ok = pos >= 0 && pos < p.n_pos;
        if (!ok) {
            if ((threadIdx.x & 31) == 0) record_code(p.dev_code, kDevBadPos);
            return;
        }
        if (j >= p.rot / 2) return;          // (a lane that rotates nothing)
        const float *row = p.cos_sin + (size_t)pos * p.rot + j;
        c = __ldg(reinterpret_cast<const float4 *>(row));
        s = __ldg(reinterpret_cast<const float4 *>(row + p.rot / 2));
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, kBlocks) qk_norm_rope_kernel(const QkNormParams p)
{
    constexpr int kIter = kIterOf<T>;
    constexpr int LPR = D / 8;               // lanes per row
    constexpr int RPW = 32 / LPR;            // rows side by side in a warp
    constexpr int ROWS = RPW * kIter;        // rows of a unit
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5), n_w = (long long)gridDim.x * kWarps;
    const long long units = (long long)p.n_tokens * p.tasks;
    const long long u0 = units * w / n_w;
    int left = (int)(units * (w + 1) / n_w - u0);
    pdl_trigger();
    pdl_wait();
    if (left == 0) return;
    // this lane's elements: 4 at `at` and 4 at `at2`, its partners or its next ones
    const int l = lane & (LPR - 1), row0 = lane / LPR;
    const bool turns = l * 8 < p.rot;
    const int at = turns ? l * 4 : l * 8, at2 = at + (turns ? p.rot / 2 : 4);
    const bool part_turns = p.rot < D;       // some lanes do not

    int tok = (int)(u0 / p.tasks), part = (int)(u0 - (long long)tok * p.tasks);
    Turn turn;
    turn.c = make_float4(1.f, 1.f, 1.f, 1.f);
    turn.s = make_float4(0.f, 0.f, 0.f, 0.f);
    turn.ok = true;
    int pos = p.rot > 0 ? p.pos[tok] : 0;
    bool fresh = p.rot > 0;                  // a token whose angles are not there yet
#pragma unroll 1
    for (;; --left) {
        Four<T> raw[kIter][2];
        {
            const bool is_k = part >= p.q_tasks;
            const int h0 = (is_k ? part - p.q_tasks : part) * ROWS + row0, heads = is_k ? p.Hkv : p.Hq;
            const int64_t sh = is_k ? p.k_sh : p.q_sh;
            const T *src = static_cast<const T *>(is_k ? p.k : p.q) + tok * (is_k ? p.k_st : p.q_st) + h0 * sh;
#pragma unroll
            for (int i = 0; i < kIter; ++i)
                if (h0 + i * RPW < heads) {
                    raw[i][0].load(src + i * RPW * sh + at);
                    raw[i][1].load(src + i * RPW * sh + at2);
                } else {
                    raw[i][0].zero();
                    raw[i][1].zero();
                }
        }
        if (fresh) {
            turn.load(p, pos, at);
            if (tok + 1 < p.n_tokens) pos = p.pos[tok + 1];
        }
        int tok1 = tok, part1 = part + 1;
        if (part1 == p.tasks) {
            part1 = 0;
            ++tok1;
        }
        const bool is_k = part >= p.q_tasks;
        const int h0 = (is_k ? part - p.q_tasks : part) * ROWS + row0, heads = is_k ? p.Hkv : p.Hq;
        const int64_t sh = is_k ? p.ko_sh : p.qo_sh;
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
            if (h0 + i * RPW < heads && turn.ok) {
                Four<T>::store(dst + i * RPW * sh + at, ya);
                Four<T>::store(dst + i * RPW * sh + at2, yb);
            }
        }
        if (left == 1) return;
        fresh = p.rot > 0 && part1 == 0;
        tok = tok1;
        part = part1;
    }
}

template <typename T>
cudaError_t launch_typed(QkNormParams p, int D, int n_sm, cudaStream_t stream)
{
    const int rows = 256 / D * kIterOf<T>;   // rows of a unit
    p.q_tasks = (p.Hq + rows - 1) / rows;
    p.tasks = p.q_tasks + (p.Hkv + rows - 1) / rows;
    const long long units = (long long)p.n_tokens * p.tasks, most = (long long)n_sm * kBlocks;
    const long long blocks = std::min((units + kWarps - 1) / kWarps, most);
    const dim3 grid((unsigned)blocks), block(kWarps * 32);
    switch (D) {
    case 64: return launch_pdl(qk_norm_rope_kernel<T, 64>, grid, block, 0, stream, p);
    case 128: return launch_pdl(qk_norm_rope_kernel<T, 128>, grid, block, 0, stream, p);
    default: return launch_pdl(qk_norm_rope_kernel<T, 256>, grid, block, 0, stream, p);
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormParams &p, int D, bool bf16, int n_sm, cudaStream_t stream)
{
    return bf16 ? launch_typed<__nv_bfloat16>(p, D, n_sm, stream) : launch_typed<float>(p, D, n_sm, stream);
}

}  // namespace kvc

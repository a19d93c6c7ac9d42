// qk_norm.cu -- RMS norm of every query and key head and the rotation to the token's position, in
// one pass over the rows.
//
//   y = x * rsqrt(mean(x^2) + eps) * w          (fp32; over the d_head elements of a row)
//   first d_rot elements, pairs (i, i + d_rot/2):  (a c - b s, b c + a s)
//   with c, s = row pos of the table; one rounding, to the rows' type.
//
// Bound by HBM: 8 operations an element that is read once and written once.  A row lies in D/8
// lanes, 8 elements each, so the mean takes log2(D/8) shuffles and an element's partner is 8 shuffles
// away.  A warp takes kIter rows per lane group of one token, all their loads in flight at once, and
// reads the token's cosines and sines once for them.
#include "common.cuh"
#include "internal.h"

namespace kvc {

namespace {

constexpr int kWarps = 8;
constexpr int kIter = 4;                     // rows per lane group and warp
constexpr int kDevBadPos = 4;                // KVC_DEV_BAD_POSITION

template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = ld_stream_16(p); }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float *f) const
    {
        f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
        f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z); f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *f)
    {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack(f[0], f[1]), pack(f[2], f[3]), pack(f[4], f[5]), pack(f[6], f[7]));
    }
};
template <>
struct Vec8<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = ld_stream_16(p);
        b = ld_stream_16(p + 4);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float *f) const
    {
        f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
        f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
        f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
        f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
    }
    static __device__ __forceinline__ void store(float *p, const float *f)
    {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) qk_norm_rope_kernel(const QkNormParams p)
{
    constexpr int LPR = D / 8;               // lanes per row
    constexpr int RPW = 32 / LPR;            // rows side by side in a warp
    constexpr int ROWS = RPW * kIter;        // rows of a warp
    const int lane = threadIdx.x & 31;
    const long long task = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    pdl_trigger();
    pdl_wait();
    if (task >= (long long)p.n_tokens * p.tasks) return;
    const int tok = (int)(task / p.tasks);
    int part = (int)(task - (long long)tok * p.tasks);
    const bool is_k = part >= p.q_tasks;
    if (is_k) part -= p.q_tasks;
    const int heads = is_k ? p.Hkv : p.Hq;
    const int64_t ht = is_k ? p.k_sh : p.q_sh, ho = is_k ? p.ko_sh : p.qo_sh;
    const T *src = static_cast<const T *>(is_k ? p.k : p.q) + tok * (is_k ? p.k_st : p.q_st);
    T *dst = static_cast<T *>(is_k ? p.k_out : p.q_out) + tok * (is_k ? p.ko_st : p.qo_st);
    const T *w = static_cast<const T *>(is_k ? p.w_k : p.w_q);
    const int l = lane & (LPR - 1), at = l * 8;
    const int h0 = part * ROWS + lane / LPR;

    Vec8<T> raw[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int h = h0 + i * RPW;
        if (h < heads) raw[i].load(src + h * ht + at);
        else raw[i].zero();
    }
    // this lane's cosines and sines, and the lane that holds the other elements of its pairs
    float c[8], s[8];
    int other = lane;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        c[j] = 1.f;
        s[j] = 0.f;
    }
    if (p.rot > 0) {
        const int pos = p.pos[tok];
        if (pos < 0 || pos >= p.n_pos) {     // the token's rows are left as they were
            if (lane == 0) record_code(p.dev_code, kDevBadPos);
            return;
        }
        const int half = p.rot / 2;
        if (at < p.rot) {
            const bool low = at < half;
            const float *row = p.cos_sin + (size_t)pos * p.rot + (low ? at : at - half);
            other = low ? lane + half / 8 : lane - half / 8;
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(row + j));
                const float4 y = __ldg(reinterpret_cast<const float4 *>(row + half + j));
                c[j] = x.x; c[j + 1] = x.y; c[j + 2] = x.z; c[j + 3] = x.w;
                s[j] = y.x; s[j + 1] = y.y; s[j + 2] = y.z; s[j + 3] = y.w;
            }
            if (low)
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = -s[j];
        }
    }
    float g[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = 1.f;
    if (w != nullptr) {
        Vec8<T> x;
        x.load(w + at);
        x.get(g);
    }
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int h = h0 + i * RPW;
        float y[8];
        raw[i].get(y);
        if (w != nullptr) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = y[j] * r * g[j];
        }
        if (p.rot > 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float z = __shfl_sync(0xffffffffu, y[j], other);
                y[j] = fmaf(z, s[j], y[j] * c[j]);
            }
        }
        if (h < heads) Vec8<T>::store(dst + h * ho + at, y);
    }
}

template <typename T>
cudaError_t launch_typed(QkNormParams p, int D, cudaStream_t stream)
{
    const int rows = 256 / D * kIter;        // rows of a warp
    p.q_tasks = (p.Hq + rows - 1) / rows;
    p.tasks = p.q_tasks + (p.Hkv + rows - 1) / rows;
    const long long blocks = ((long long)p.n_tokens * p.tasks + kWarps - 1) / kWarps;
    const dim3 grid((unsigned)blocks), block(kWarps * 32);
    switch (D) {
    case 64: return launch_pdl(qk_norm_rope_kernel<T, 64>, grid, block, 0, stream, p);
    case 128: return launch_pdl(qk_norm_rope_kernel<T, 128>, grid, block, 0, stream, p);
    default: return launch_pdl(qk_norm_rope_kernel<T, 256>, grid, block, 0, stream, p);
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormParams &p, int D, bool bf16, cudaStream_t stream)
{
    return bf16 ? launch_typed<__nv_bfloat16>(p, D, stream) : launch_typed<float>(p, D, stream);
}

}  // namespace kvc

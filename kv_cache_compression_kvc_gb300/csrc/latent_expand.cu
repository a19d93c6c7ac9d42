// latent_expand.cu -- the expanded form of a latent cache on the CUDA cores (fp32 caches, fp32
// arithmetic):
//   K[b,h,s,i] = sum_r W_k[h,i,r] c[b,s,r] (i < D - E),  K[b,h,s,D-E+e] = c[b,s,R+e],
//   V[b,h,s,i] = sum_r W_v[h,i,r] c[b,s,r].
// A block computes 64 slots x 64 outputs of one head (256 threads, 4 x 4 each) from 32-deep
// slices of both operands staged in shared memory.
#include "common.cuh"
#include "internal.h"

namespace kvc {

namespace {

constexpr int kThreads = 256;
constexpr int kTS = 64, kTO = 64, kTK = 32;
constexpr int kDevBadLengthC = 5;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16(x); }

template <typename T>
__global__ void __launch_bounds__(kThreads) latent_expand_kernel(const ExpandParams p)
{
    __shared__ float sA[kTK][kTS + 4];       // c, transposed: [r][slot]
    __shared__ float sB[kTK][kTO + 4];       // W, transposed: [r][output]
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.z, s0 = blockIdx.x * kTS;
    const int NK = p.D - p.E;
    const int kt = (NK + kTO - 1) / kTO, vt = p.D / kTO;
    const int h = blockIdx.y / (kt + vt), jt = blockIdx.y % (kt + vt);
    int n = p.len != nullptr ? p.len[b] : p.n_valid;
    const int most = p.cap < p.dst_cap ? p.cap : p.dst_cap;
    if (n < 0 || n > most) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0)
            record_code(p.dev_code, kDevBadLengthC);
        n = n < 0 ? 0 : most;
    }
    if (s0 >= n) return;
    const bool isv = jt >= kt;
    const int o0 = (isv ? jt - kt : jt) * kTO;
    const int n_out = isv ? p.D : NK;
    const T *c = static_cast<const T *>(p.c) + b * p.c_sb;
    const T *w = isv ? static_cast<const T *>(p.wv) + (size_t)h * p.D * p.R
                     : static_cast<const T *>(p.wk) + (size_t)h * NK * p.R;
    T *dst = static_cast<T *>(isv ? p.v : p.k) + b * p.sb + h * p.sh;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int r0 = 0; r0 < p.R; r0 += kTK) {
        __syncthreads();
        for (int i = threadIdx.x; i < kTS * kTK; i += kThreads) {
            const int j = i / kTK, r = i % kTK;
            sA[r][j] = s0 + j < n ? to_f(c[(int64_t)(s0 + j) * p.c_ss + r0 + r]) : 0.f;
            sB[r][j] = o0 + j < n_out ? to_f(w[(size_t)(o0 + j) * p.R + r0 + r]) : 0.f;
        }
        __syncthreads();
#pragma unroll 8
        for (int r = 0; r < kTK; ++r) {
            const float4 a = *reinterpret_cast<const float4 *>(&sA[r][4 * ty]);
            const float4 x = *reinterpret_cast<const float4 *>(&sB[r][4 * tx]);
            const float av[4] = {a.x, a.y, a.z, a.w}, xv[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], xv[j], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int s = s0 + 4 * ty + i;
        if (s >= n) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int o = o0 + 4 * tx + j;
            if (o < n_out) put(dst + (int64_t)s * p.ss + o, acc[i][j]);
        }
    }
    if (jt == 0)                             // the shared part of the keys
        for (int i = threadIdx.x; i < kTS * p.E; i += kThreads) {
            const int s = s0 + i / p.E, e = i % p.E;
            if (s < n) dst[(int64_t)s * p.ss + NK + e] = c[(int64_t)s * p.c_ss + p.R + e];
        }
}

}  // namespace

cudaError_t launch_latent_expand(const ExpandParams &p, int dtype, cudaStream_t stream)
{
    const int most = p.len != nullptr ? (p.cap < p.dst_cap ? p.cap : p.dst_cap) : p.n_valid;
    if (most <= 0) return cudaSuccess;
    if (dtype == 1) {
        bool used = false;
        const cudaError_t e = launch_latent_expand_tc(p, stream, &used);
        if (e != cudaSuccess || used) return e;
    }
    const int kt = (p.D - p.E + kTO - 1) / kTO, vt = p.D / kTO;
    const dim3 grid((unsigned)((most + kTS - 1) / kTS), (unsigned)(p.H * (kt + vt)), (unsigned)p.B);
    if (dtype == 1)
        return launch_pdl(latent_expand_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, p);
    return launch_pdl(latent_expand_kernel<float>, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace kvc

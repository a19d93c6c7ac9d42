// tree_attn.cu -- attention of a tree of drafted tokens over a cache on the CUDA cores (fp32
// arithmetic; fp32 caches, and bf16 pools whose block size the tensor-core kernel does not
// take), and the merge of split rows, which both kernels use.
//
// For row r (drafted token, query head) of a pair, over the visible slots j:
//   s_j = scale * q_r.k_j,  m = max s_j,  l = sum exp(s_j - m),  o = sum exp(s_j - m) v_j / l
// in one pass over the slots with a running (m, l) and a rescaled o (base-2 exponentials).
//
// Tiling.  256 threads take RN = 32 rows against tiles of 64 slots.  Q stays in shared memory in
// fp32; a tile's K and V rows are widened into shared memory once and read by all 32 rows.  Each
// thread computes 2 rows x 4 slots of the logits (K rows padded by 16 bytes: the 16 slots a
// quarter of the block reads at once fall into different banks) and 2..16 rows x 4 columns of
// the output, so every shared-memory word feeds 2 to 4 FMAs.
#include <algorithm>

#include "tree_attn.cuh"

namespace kvc {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 32;                    // RN
constexpr int kTile = 64;                    // TS

template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int VEC = 4;            // elements per 16 bytes
    static __device__ __forceinline__ void widen(uint4 w, float *f)
    {
        f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y);
        f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ float narrow(float x) { return x; }
    template <int W>
    static __device__ __forceinline__ void store(float *p, const float *x)
    {
        if constexpr (W == 4) *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        else *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
    }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int VEC = 8;
    static __device__ __forceinline__ void widen(uint4 w, float *f)
    {
        f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
        f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z); f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
    }
    static __device__ __forceinline__ __nv_bfloat16 narrow(float x) { return __float2bfloat16(x); }
    template <int W>
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *x)
    {
        __nv_bfloat162 y[W / 2];
#pragma unroll
        for (int i = 0; i < W / 2; ++i) y[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        if constexpr (W == 4) *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<uint2 *>(y);
        else *reinterpret_cast<uint32_t *>(p) = *reinterpret_cast<uint32_t *>(y);
    }
};

__device__ __forceinline__ bool finite_f(float x) { return fabsf(x) <= 3.402823466e38f; }

// K rows in shared memory are DK + 4 floats apart.
template <int DV>
constexpr int out_cols() { return DV / 4; }  // 4-float output columns

struct SimplePlan {
    static size_t smem(int DK, int DV, bool latent)
    {
        size_t f = (size_t)kRows * DK + (size_t)kTile * (DK + 4) + (size_t)kRows * (kTile + 4) +
                   3 * kRows;
        if (!latent) f += (size_t)kTile * DV;
        return f * sizeof(float) + 256;
    }
};

template <typename T, int DV, bool LATENT>
__global__ void __launch_bounds__(kThreads) tree_attn_kernel(const TreeParams p)
{
    using E = Elem<T>;
    constexpr int VEC = E::VEC;
    const int DK = LATENT ? p.DK : DV;
    const int KS = DK + 4;                   // K row stride, floats
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm;                          // [32][DK]
    float *sK = sQ + kRows * DK;             // [64][KS]
    float *sP = sK + kTile * KS;             // [32][68] logits, then probabilities
    float *sM = sP + kRows * (kTile + 4);    // running max (log2 units)
    float *sL = sM + kRows;
    float *sA = sL + kRows;                  // rescale factor of this tile
    float *sV = sA + kRows;                  // [64][DV]
    if (LATENT) sV = sK;
    const int VS = LATENT ? KS : DV;
    __shared__ unsigned long long s_nf;      // drafted tokens with non-finite values

    const int tid = threadIdx.x;
    const int rt = blockIdx.x % p.RT, g = blockIdx.x / p.RT;
    pdl_trigger();
    pdl_wait();
    const TreeRange range = tree_range(p, g, kTile);
    TreeNote note;
    TreeWalk walk(p, range);
    TreeSeg s;

    constexpr int NC = out_cols<DV>();       // column groups
    constexpr int RG = kThreads / NC;        // row groups
    constexpr int RPT = kRows / RG;          // rows per thread
    const int oc = tid % NC, orow = (tid / NC) * RPT;
    const int ty = tid / 16, tx = tid % 16;  // logits: rows 2ty, 2ty+1; slots tx + 16 i

    while (walk.next(p, rt, kTile, s)) {
        note.see(range, s);
        if (s.rows <= 0) continue;
        __syncthreads();                     // the previous pair's shared memory is done with
        const int r0 = rt * p.RP;
        for (int i = tid; i < kRows * (DK / VEC); i += kThreads) {
            const int r = i / (DK / VEC), c = i % (DK / VEC);
            float f[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = 0.f;
            if (r < s.rows) {
                const int t = (r0 + r) / p.G, h = s.kh * p.G + (r0 + r) % p.G;
                const T *src = static_cast<const T *>(p.q) +
                               (((size_t)s.b * p.T + t) * p.Hq + h) * DK + c * VEC;
                E::widen(__ldg(reinterpret_cast<const uint4 *>(src)), f);
            }
#pragma unroll
            for (int e = 0; e < VEC; e += 4)
                *reinterpret_cast<float4 *>(sQ + r * DK + c * VEC + e) =
                    make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
        }
        if (tid < kRows) {
            sM[tid] = kNoMax;
            sL[tid] = 0.f;
        }
        if (tid == 0) s_nf = 0ull;
        float4 o[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);

        for (int tile = s.lo; tile < s.hi; ++tile) {
            const bool draft = s.is_draft(p, tile);
            const int valid = s.valid(p, tile, kTile);
            __syncthreads();                 // the previous tile's reads are done
            // rows of the tile: K (and V), widened; rows past the valid ones are zero
            const int per_row = DK / VEC;
            for (int i = tid; i < kTile * per_row; i += kThreads) {
                const int j = i / per_row, c = i - j * per_row;
                float f[VEC], fv[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[e] = fv[e] = 0.f;
                if (j < valid) {
                    const T *kr, *vr;
                    if (draft) {
                        const size_t at = (((size_t)s.b * p.T + j) * p.Hkv + s.kh) * DK;
                        kr = static_cast<const T *>(p.kd) + at;
                        vr = static_cast<const T *>(p.vd) + at;
                    } else if (p.table != nullptr) {
                        const int slot = tile * kTile + j;
                        int blk = p.table[(size_t)s.b * p.max_blocks + slot / p.bs];
                        if (blk < 0 || blk >= p.n_pool) {
                            record_code(p.dev_code, kDevBadBlockCode);
                            blk = 0;
                        }
                        const size_t at = s.kh * p.sh + ((size_t)blk * p.bs + slot % p.bs) * DK;
                        kr = static_cast<const T *>(p.k) + at;
                        vr = static_cast<const T *>(p.v) + at;
                    } else {
                        const size_t at = s.b * p.sb + s.kh * p.sh +
                                          (int64_t)(tile * kTile + j) * p.ss;
                        kr = static_cast<const T *>(p.k) + at;
                        vr = static_cast<const T *>(p.v) + at;
                    }
                    E::widen(ld_stream_16(kr + c * VEC), f);
                    if (!LATENT) E::widen(ld_stream_16(vr + c * VEC), fv);
                }
#pragma unroll
                for (int e = 0; e < VEC; e += 4) {
                    *reinterpret_cast<float4 *>(sK + j * KS + c * VEC + e) =
                        make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
                    if (!LATENT)
                        *reinterpret_cast<float4 *>(sV + j * VS + c * VEC + e) =
                            make_float4(fv[e], fv[e + 1], fv[e + 2], fv[e + 3]);
                }
            }
            __syncthreads();
            // logits
            float acc[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
            if (2 * ty < s.rows) {
                const float *qa = sQ + 2 * ty * DK, *qb = qa + DK;
                const float *kk = sK + tx * KS;
                // sums of 32 dims, then of those: one sum over all of them loses twice as much
                for (int d0 = 0; d0 < DK; d0 += 32) {
                    const int d1 = min(DK, d0 + 32);
                    float part[2][4] = {};
#pragma unroll 4
                    for (int d = d0; d < d1; d += 4) {
                        const float4 a = *reinterpret_cast<const float4 *>(qa + d);
                        const float4 b = *reinterpret_cast<const float4 *>(qb + d);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 x = *reinterpret_cast<const float4 *>(kk + j * 16 * KS + d);
                            part[0][j] = fmaf(a.x, x.x, fmaf(a.y, x.y, fmaf(a.z, x.z, fmaf(a.w, x.w, part[0][j]))));
                            part[1][j] = fmaf(b.x, x.x, fmaf(b.y, x.y, fmaf(b.z, x.z, fmaf(b.w, x.w, part[1][j]))));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][j] += part[i][j];
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 2 * ty + i;
                uint64_t see = ~0ull;
                if (draft && r < s.rows) see = tree_mask_word(p, s.b, (r0 + r) / p.G, s.cnt);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = tx + 16 * j;
                    const bool ok = r < s.rows && c < valid && ((see >> c) & 1ull);
                    sP[r * (kTile + 4) + c] = ok ? acc[i][j] * p.scale_log2 : -INFINITY;
                }
            }
            __syncthreads();
            // running softmax: each warp takes four rows
            {
                const int w = tid >> 5, lane = tid & 31;
#pragma unroll
                for (int i = 0; i < kRows / 8; ++i) {
                    const int r = w * (kRows / 8) + i;
                    float *row = sP + r * (kTile + 4);
                    const float x0 = row[lane], x1 = row[lane + 32];
                    const float m_old = sM[r];
                    const float m = fmaxf(m_old, warp_max(fmaxf(x0, x1)));
                    const float p0 = ex2(x0 - m), p1 = ex2(x1 - m);
                    const float a = ex2(m_old - m);
                    const float z = warp_sum(p0 + p1);
                    row[lane] = p0;
                    row[lane + 32] = p1;
                    if (lane == 0) {
                        sM[r] = m;
                        sL[r] = sL[r] * a + z;
                        sA[r] = a;
                    }
                }
            }
            // a drafted token's non-finite values must not reach rows that do not see it
            // (0 * inf): they are taken out of the tile here and added to the rows that do at
            // the end
            if (draft) {
                for (int i = tid; i < valid * DV; i += kThreads) {
                    float *x = sV + (i / DV) * VS + i % DV;
                    if (!finite_f(*x)) {
                        *x = 0.f;
                        atomicOr(&s_nf, 1ull << (i / DV));
                    }
                }
            }
            __syncthreads();
            // output: rows orow .. orow + RPT - 1, columns 4 oc .. 4 oc + 3
            if (orow < s.rows) {
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const float a = sA[orow + i];
                    o[i].x *= a; o[i].y *= a; o[i].z *= a; o[i].w *= a;
                }
                for (int j = 0; j < valid; j += 4) {
                    float4 v[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        v[u] = *reinterpret_cast<const float4 *>(sV + (j + u) * VS + 4 * oc);
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        const float4 w =
                            *reinterpret_cast<const float4 *>(sP + (orow + i) * (kTile + 4) + j);
                        o[i].x += fmaf(w.x, v[0].x, fmaf(w.y, v[1].x, fmaf(w.z, v[2].x, w.w * v[3].x)));
                        o[i].y += fmaf(w.x, v[0].y, fmaf(w.y, v[1].y, fmaf(w.z, v[2].y, w.w * v[3].y)));
                        o[i].z += fmaf(w.x, v[0].z, fmaf(w.y, v[1].z, fmaf(w.z, v[2].z, w.w * v[3].z)));
                        o[i].w += fmaf(w.x, v[0].w, fmaf(w.y, v[1].w, fmaf(w.z, v[2].w, w.w * v[3].w)));
                    }
                }
            }
        }
        __syncthreads();
        const unsigned long long nf = s_nf;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int r = orow + i;
            if (r >= s.rows) break;
            const int t = (r0 + r) / p.G, h = s.kh * p.G + (r0 + r) % p.G;
            float f[4] = {o[i].x, o[i].y, o[i].z, o[i].w};
            unsigned long long hit = nf ? nf & tree_mask_word(p, s.b, t, s.cnt) : 0ull;
            while (hit) {
                const int j = __ffsll((long long)hit) - 1;
                hit &= hit - 1;
                const T *vr = static_cast<const T *>(p.vd) +
                              (((size_t)s.b * p.T + j) * p.Hkv + s.kh) * DK + 4 * oc;
                for (int e = 0; e < 4; ++e) {
                    const float x = (float)vr[e];
                    if (!finite_f(x)) f[e] += x;
                }
            }
            const float m = sM[r], l = sL[r];
            if (s.whole()) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const size_t row = ((size_t)s.b * p.T + t) * p.Hq + h;
                T *dst = static_cast<T *>(p.out) + row * DV + 4 * oc;
                for (int e = 0; e < 4; ++e) dst[e] = E::narrow(l == 0.f ? 0.f : f[e] * inv);
                if (oc == 0 && p.lse != nullptr)
                    p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            } else {
                const size_t slot = (size_t)blockIdx.x * 2 + (s.first ? 0 : 1);
                *reinterpret_cast<float4 *>(p.ws_o + (slot * p.RN + r) * DV + 4 * oc) =
                    make_float4(f[0], f[1], f[2], f[3]);
                if (oc == 0) {
                    p.ws_ml[(slot * p.RN + r) * 2] = m;
                    p.ws_ml[(slot * p.RN + r) * 2 + 1] = l;
                }
            }
        }
    }
    if (rt == 0 && tid == 0) p.ws_info[g] = note.get(range);
}

// Joins the partial states of split pairs.  Blocks (group g * row tile, row chunk) take the pair
// whose first part group g holds (if any): WPR of a block's eight warps per row, each every
// WPR-th part, DV / 32 columns a lane.  Bound by latency (a chain of three L2 reads), so a warp has
// several parts in flight and the grid is one wave: one warp per row where there are many rows
// (1216 blocks on the SnapKV cache instead of 9728 of a row each: 13 us to 4), eight where
// there are few rows of many parts.
constexpr int kMergeWarps = 8;
template <typename T, int DV, int WPR>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const TreeParams p)
{
    constexpr int CPL = DV / 32;             // columns per lane
    static_assert(CPL == 2 || CPL % 4 == 0, "vector columns");
    constexpr int W = CPL == 2 ? 2 : 4;      // floats per load
    constexpr int NV = CPL / W;
    constexpr int ROWS = kMergeWarps / WPR;  // rows per block
    __shared__ float s_o[WPR > 1 ? kMergeWarps : 1][WPR > 1 ? DV : 1];
    __shared__ float s_l[kMergeWarps];
    pdl_trigger();
    pdl_wait();
    const int rt = blockIdx.x % p.RT, g = blockIdx.x / p.RT;
    const int4 note = p.ws_info[g];
    if (note.x < 0) return;
    const int b = note.x, kh = note.y;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.y * ROWS + w / WPR, part0 = w % WPR;
    const int rows = min(p.RP, (note.w >> 1) * p.G - rt * p.RP);
    const bool live = r < rows;
    if (WPR == 1 && !live) return;
    const int nseg = live ? note.z - g + 1 : 0;
    auto slot_of = [&](int i) -> size_t {
        return ((size_t)((g + i) * p.RT + rt) * 2 + (i == 0 ? note.w & 1 : 0)) * p.RN + r;
    };
    float M = kNoMax;
    for (int i = lane; i < nseg; i += 32) M = fmaxf(M, __ldcg(p.ws_ml + slot_of(i) * 2));
    M = warp_max(M);
    float o[CPL], L = 0.f;
#pragma unroll
    for (int c = 0; c < CPL; ++c) o[c] = 0.f;
    constexpr int UNR = CPL >= 16 ? 4 : 8;
#pragma unroll 1
    for (int i0 = part0; i0 < nseg; i0 += WPR * UNR) {
        float x[UNR][CPL], ml[UNR][2];
#pragma unroll
        for (int u = 0; u < UNR; ++u) {
            const int i = i0 + u * WPR;
            ml[u][0] = kNoMax;
            ml[u][1] = 0.f;
#pragma unroll
            for (int c = 0; c < CPL; ++c) x[u][c] = 0.f;
            if (i < nseg) {
                const size_t st = slot_of(i);
                const float2 y2 = __ldcg(reinterpret_cast<const float2 *>(p.ws_ml + st * 2));
                ml[u][0] = y2.x;
                ml[u][1] = y2.y;
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    const float *src = p.ws_o + st * DV + (n * 32 + lane) * W;
                    if constexpr (W == 4) {
                        const float4 y = __ldcg(reinterpret_cast<const float4 *>(src));
                        x[u][n * 4] = y.x; x[u][n * 4 + 1] = y.y;
                        x[u][n * 4 + 2] = y.z; x[u][n * 4 + 3] = y.w;
                    } else {
                        const float2 y = __ldcg(reinterpret_cast<const float2 *>(src));
                        x[u][0] = y.x; x[u][1] = y.y;
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < UNR; ++u) {
            const float c = ex2(ml[u][0] - M);
            L += ml[u][1] * c;
            // a part that saw nothing holds zeros and has c = 0 or l = 0
#pragma unroll
            for (int k = 0; k < CPL; ++k) o[k] = fmaf(c, x[u][k], o[k]);
        }
    }
    if constexpr (WPR > 1) {                 // the row's warps meet, in order
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int e = 0; e < W; ++e) s_o[w][(n * 32 + lane) * W + e] = o[n * W + e];
        if (lane == 0) s_l[w] = L;
        __syncthreads();
        if (part0 != 0 || !live) return;
        L = 0.f;
#pragma unroll
        for (int c = 0; c < CPL; ++c) o[c] = 0.f;
#pragma unroll 1
        for (int i = 0; i < WPR; ++i) {
            L += s_l[w + i];
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int e = 0; e < W; ++e) o[n * W + e] += s_o[w + i][(n * 32 + lane) * W + e];
        }
    }
    const int row_g = rt * p.RP + r, t = row_g / p.G;
    const size_t row = ((size_t)b * p.T + t) * p.Hq + kh * p.G + (row_g - t * p.G);
    const float inv = 1.f / L;
    T *dst = static_cast<T *>(p.out) + row * DV;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        float y[W];
#pragma unroll
        for (int e = 0; e < W; ++e) y[e] = L == 0.f ? 0.f : o[n * W + e] * inv;
        Elem<T>::template store<W>(dst + (n * 32 + lane) * W, y);
    }
    if (lane == 0 && p.lse != nullptr)
        p.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

template <typename T, int DV, bool LATENT>
cudaError_t launch_typed(const TreeParams &p, cudaStream_t stream)
{
    const size_t smem = SimplePlan::smem(p.DK, DV, LATENT);
    static bool configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !configured[dev]) {
        const size_t most = SimplePlan::smem(LATENT ? DV + 64 : DV, DV, LATENT);
        const cudaError_t e = cudaFuncSetAttribute(
            tree_attn_kernel<T, DV, LATENT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    return launch_pdl(tree_attn_kernel<T, DV, LATENT>, dim3((unsigned)(p.groups * p.RT)),
                      dim3(kThreads), smem, stream, p);
}

template <typename T>
cudaError_t launch_dims(const TreeParams &p, cudaStream_t stream)
{
    if (p.latent) {
        switch (p.DV) {
        case 128: return launch_typed<T, 128, true>(p, stream);
        case 256: return launch_typed<T, 256, true>(p, stream);
        default: return launch_typed<T, 512, true>(p, stream);
        }
    }
    switch (p.DV) {
    case 64: return launch_typed<T, 64, false>(p, stream);
    case 128: return launch_typed<T, 128, false>(p, stream);
    default: return launch_typed<T, 256, false>(p, stream);
    }
}

template <typename T, int DV>
cudaError_t merge_typed(const TreeParams &p, cudaStream_t stream)
{
    const int rows = std::min(p.RP, p.T * p.G), gx = p.groups * p.RT;
    // eight warps a row while that makes at most four blocks an SM
    if ((long long)gx * rows <= 4 * 152)
        return launch_pdl(tree_merge_kernel<T, DV, 8>, dim3((unsigned)gx, (unsigned)rows),
                          dim3(kMergeWarps * 32), 0, stream, p);
    return launch_pdl(tree_merge_kernel<T, DV, 1>,
                      dim3((unsigned)gx, (unsigned)((rows + kMergeWarps - 1) / kMergeWarps)),
                      dim3(kMergeWarps * 32), 0, stream, p);
}
template <typename T>
cudaError_t merge_dims(const TreeParams &p, cudaStream_t stream)
{
    switch (p.DV) {
    case 64: return merge_typed<T, 64>(p, stream);
    case 128: return merge_typed<T, 128>(p, stream);
    case 256: return merge_typed<T, 256>(p, stream);
    default: return merge_typed<T, 512>(p, stream);
    }
}

}  // namespace

void tree_tc_rows(int G, int DV, int T, bool latent, int32_t *RN, int32_t *RP)
{
    (void)DV;
    if (latent) {
        *RN = *RP = T * G <= 32 ? 32 : 64;
    } else {
        *RN = T * G <= 64 ? 64 : 128;
        *RP = *RN / G * G;
    }
}

TreePlan tree_plan(int G, int DK, int DV, int T, bool latent, bool tc, int n_sm)
{
    TreePlan pl{};
    const int R = T * G;
    pl.tc = tc;
    long long blocks = n_sm;
    if (tc) {
        tree_tc_rows(G, DV, T, latent, &pl.RN, &pl.RP);
    } else {
        pl.RN = pl.RP = kRows;
        // blocks resident at once: shared memory allows one to five per SM
        const long long fit = (long long)(227 * 1024) / (long long)(SimplePlan::smem(DK, DV, latent) + 1024);
        blocks = n_sm * std::max(1LL, std::min(fit, 5LL));
    }
    pl.RT = (R + pl.RP - 1) / pl.RP;
    pl.groups = (int)std::max(1LL, blocks / pl.RT);
    const size_t parts = (size_t)pl.groups * pl.RT * 2;
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    pl.off_info = 0;
    pl.off_ml = up(pl.off_info + (size_t)pl.groups * sizeof(int4));
    pl.off_o = up(pl.off_ml + parts * pl.RN * 2 * sizeof(float));
    pl.bytes = up(pl.off_o + parts * pl.RN * DV * sizeof(float));
    return pl;
}

bool tree_whole(const TreeParams &p, bool tc)
{
    if (!tc) return false;
    const int TS = p.latent || p.DV == 256 ? 64 : 128;
    const long long slots = p.len == nullptr ? p.n_valid : p.cap;
    const long long tiles = (slots + TS - 1) / TS + (p.kd != nullptr);
    const long long spare = ((long long)p.P + p.groups - 1) / p.groups * p.groups - p.P;
    return tiles <= kWholeTiles && spare * tiles <= (long long)(p.latent ? kWholeWaitLatent : kWholeWait) * p.groups;
}

cudaError_t launch_tree_attn(const TreeParams &p, int dtype, cudaStream_t stream)
{
    return dtype == 1 ? launch_dims<__nv_bfloat16>(p, stream) : launch_dims<float>(p, stream);
}

cudaError_t launch_tree_merge(const TreeParams &p, int dtype, cudaStream_t stream)
{
    return dtype == 1 ? merge_dims<__nv_bfloat16>(p, stream) : merge_dims<float>(p, stream);
}

}  // namespace kvc

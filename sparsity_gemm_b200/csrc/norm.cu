// LayerNorm and RMSNorm with 16- or 32-bit outputs, and their backward pass.
//
// Forward, per row of k values:
//   mu = sum x / k (RMSNorm: 0), rstd = 1 / sqrt(sum (x - mu)^2 / k + eps),
//   y = (x - mu) rstd w + b.
// Backward, with xhat = (x - mu) rstd and g = dy w:
//   dx = rstd (g - mean(g) - xhat mean(g xhat))   (RMSNorm: no mean(g)),
//   dw = sum over rows of dy xhat, db = sum over rows of dy.
// Values are widened to binary32, all sums are binary32; the variance is
// taken around the mean in a second pass over registers, so a mean far above
// the spread costs no digits. Results are rounded once. Every sum has a fixed
// order: the same inputs give the same bits.
#include <cuda_runtime.h>
#include <string.h>

#include "sharq_dev.cuh"
#include "sq_internal.h"
#include "vec.cuh"

namespace sq {

// ---------------------------------------------------------------------------
// Sums over the threads of a row: one warp, or a CTA through `red` (one slot
// per warp; each call of a row uses its own array, so one barrier suffices).

template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = warp_sum(v);
    if (WARP) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    return warp_sum(lane < warps ? red[lane] : 0.0f);
}

// ---------------------------------------------------------------------------
// Forward

struct NormParams {
    const void *x, *w, *b;
    void *y;
    float *mean, *rstd;  // NULL: not wanted
    int64_t rows;
    int32_t k;
    float eps;
    int32_t rms;
};

// A row lives in the registers of its threads (NV vectors of VW elements
// each, vector i of a thread at i * threads + thread), so x is read once.
// WARP: one warp per row, kFwdWarps rows per CTA; else one CTA per row.
constexpr int kFwdWarps = 4;

template <typename T, int VW, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kFwdWarps : 1024) norm_fwd_kernel(const NormParams p) {
    using V = Vec<T, VW>;
    __shared__ float red[2][32];
    griddep_wait();
    griddep_launch();
    const int tid = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int threads = WARP ? 32 : blockDim.x;
    const int64_t row = WARP ? (int64_t)blockIdx.x * kFwdWarps + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    if (WARP && row >= p.rows) return;
    const int nvec = p.k / VW;
    const T *x = static_cast<const T *>(p.x) + row * p.k;
    T *y = static_cast<T *>(p.y) + row * p.k;
    const T *w = static_cast<const T *>(p.w), *b = static_cast<const T *>(p.b);

    typename V::P xv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * threads + tid;
        xv[i] = c < nvec ? V::load(x + (int64_t)c * VW) : V::zero();
    }
    const float inv_k = 1.0f / (float)p.k;
    float mu = 0.0f;
    if (!p.rms) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[VW];
            V::unpack(xv[i], f);
#pragma unroll
            for (int e = 0; e < VW; ++e) s += f[e];
        }
        mu = row_sum<WARP>(s, red[0]) * inv_k;
    }
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (i * threads + tid < nvec) {
            float f[VW];
            V::unpack(xv[i], f);
#pragma unroll
            for (int e = 0; e < VW; ++e) {
                const float d = f[e] - mu;
                q = fmaf(d, d, q);
            }
        }
    }
    const float rstd = 1.0f / sqrtf(row_sum<WARP>(q, red[1]) * inv_k + p.eps);
    if (tid == 0) {
        if (p.mean) p.mean[row] = mu;
        if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * threads + tid;
        if (c < nvec) {
            float f[VW], wf[VW], bf[VW];
            V::unpack(xv[i], f);
#pragma unroll
            for (int e = 0; e < VW; ++e) f[e] = (f[e] - mu) * rstd;
            if (w) {
                V::unpack(V::load(w + (int64_t)c * VW), wf);
#pragma unroll
                for (int e = 0; e < VW; ++e) f[e] *= wf[e];
            }
            if (b) {
                V::unpack(V::load(b + (int64_t)c * VW), bf);
#pragma unroll
                for (int e = 0; e < VW; ++e) f[e] += bf[e];
            }
            V::store(y + (int64_t)c * VW, V::pack(f));
        }
    }
}

// Rows too long for the registers: the same sums in three passes over the
// row, which stays in L2 (at most 256 KB).
constexpr int kLongThreads = 1024;

template <typename T, int VW>
__global__ void __launch_bounds__(kLongThreads) norm_fwd_long_kernel(const NormParams p) {
    using V = Vec<T, VW>;
    __shared__ float red[2][32];
    griddep_wait();
    griddep_launch();
    const int64_t row = blockIdx.x;
    const int nvec = p.k / VW;
    const T *x = static_cast<const T *>(p.x) + row * p.k;
    T *y = static_cast<T *>(p.y) + row * p.k;
    const T *w = static_cast<const T *>(p.w), *b = static_cast<const T *>(p.b);
    const float inv_k = 1.0f / (float)p.k;
    float mu = 0.0f, f[VW], wf[VW];
    if (!p.rms) {
        float s = 0.0f;
        for (int c = threadIdx.x; c < nvec; c += kLongThreads) {
            V::unpack(V::load(x + (int64_t)c * VW), f);
#pragma unroll
            for (int e = 0; e < VW; ++e) s += f[e];
        }
        mu = row_sum<false>(s, red[0]) * inv_k;
    }
    float q = 0.0f;
    for (int c = threadIdx.x; c < nvec; c += kLongThreads) {
        V::unpack(V::load(x + (int64_t)c * VW), f);
#pragma unroll
        for (int e = 0; e < VW; ++e) {
            const float d = f[e] - mu;
            q = fmaf(d, d, q);
        }
    }
    const float rstd = 1.0f / sqrtf(row_sum<false>(q, red[1]) * inv_k + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mu;
        if (p.rstd) p.rstd[row] = rstd;
    }
    for (int c = threadIdx.x; c < nvec; c += kLongThreads) {
        V::unpack(V::load(x + (int64_t)c * VW), f);
#pragma unroll
        for (int e = 0; e < VW; ++e) f[e] = (f[e] - mu) * rstd;
        if (w) {
            V::unpack(V::load(w + (int64_t)c * VW), wf);
#pragma unroll
            for (int e = 0; e < VW; ++e) f[e] *= wf[e];
        }
        if (b) {
            V::unpack(V::load(b + (int64_t)c * VW), wf);
#pragma unroll
            for (int e = 0; e < VW; ++e) f[e] += wf[e];
        }
        V::store(y + (int64_t)c * VW, V::pack(f));
    }
}

// ---------------------------------------------------------------------------
// Backward
//
// Persistent row groups (a warp, a CTA, or a cluster of CTAs for long rows)
// walk the rows; a thread always owns the same kBwdCols columns, so the
// weight gradients add up in its registers over all its rows and leave the
// SM once, as one partial row per CTA; a second kernel adds the partial rows
// in their order. The next row is loaded before the current one is reduced.
constexpr int kBwdCols = 16;          // columns per thread
constexpr int kBwdThreads = 512;      // most threads of a CTA
constexpr int kBwdCluster = 8;        // most CTAs of a row
constexpr int kBwdWarps = 8;          // rows at a time in a CTA of the warp form

struct NormBwdParams {
    const void *dy, *x, *w;
    const float *mean, *rstd;
    void *dx;
    float *part;  // [parts][2][k] (dw, then db), NULL: no weight gradients
    int64_t rows;
    int32_t k, parts, rms;
};

template <typename T, int VW, bool WARP>
__global__ void __launch_bounds__(kBwdThreads) norm_bwd_kernel(const NormBwdParams p) {
    using V = Vec<T, VW>;
    constexpr int NV = kBwdCols / VW;
    __shared__ float2 red[2][kBwdThreads / 32];
    __shared__ float2 peer[2][kBwdCluster];
    extern __shared__ float acc_sm[];  // WARP: [kBwdWarps][2][k]
    griddep_wait();
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const uint32_t crank = WARP ? 0 : cluster_ctarank();
    uint32_t csize = 1;
    if (!WARP) asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(csize));
    const int tid = WARP ? lane : (int)(crank * blockDim.x + threadIdx.x);
    const int threads = WARP ? 32 : (int)(csize * blockDim.x);
    const int part = (int)(blockIdx.x / csize);
    const int64_t first = WARP ? (int64_t)blockIdx.x * kBwdWarps + warp : (int64_t)part;
    const int64_t step = WARP ? (int64_t)gridDim.x * kBwdWarps : (int64_t)(gridDim.x / csize);
    const int nvec = p.k / VW;
    const T *xp = static_cast<const T *>(p.x), *dyp = static_cast<const T *>(p.dy), *wp = static_cast<const T *>(p.w);
    T *dxp = static_cast<T *>(p.dx);
    const float inv_k = 1.0f / (float)p.k;
    if (csize > 1) cluster_sync();  // every CTA of the row runs before another writes to its shared memory

    typename V::P wv[NV];
    float dw[kBwdCols], db[kBwdCols];
#pragma unroll
    for (int i = 0; i < kBwdCols; ++i) dw[i] = db[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * threads + tid;
        wv[i] = wp && c < nvec ? V::load(wp + (int64_t)c * VW) : V::zero();
    }
    typename V::P xn[NV], dn[NV];
    float mu_n = 0.0f, rs_n = 0.0f;
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * threads + tid;
            const bool in = c < nvec;
            xn[i] = in ? V::load(xp + row * p.k + (int64_t)c * VW) : V::zero();
            dn[i] = in ? V::load(dyp + row * p.k + (int64_t)c * VW) : V::zero();
        }
        mu_n = p.rms ? 0.0f : __ldg(p.mean + row);
        rs_n = __ldg(p.rstd + row);
    };
    if (first < p.rows) fetch(first);
    int parity = 0;
    for (int64_t row = first; row < p.rows; row += step, parity ^= 1) {
        typename V::P xv[NV], dv[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            xv[i] = xn[i];
            dv[i] = dn[i];
        }
        const float mu = mu_n, rs = rs_n;
        if (row + step < p.rows) fetch(row + step);
        float s1 = 0.0f, s2 = 0.0f;  // sum g, sum g xhat
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float xf[VW], df[VW], wf[VW];
            V::unpack(xv[i], xf);
            V::unpack(dv[i], df);
            V::unpack(wv[i], wf);
            // columns past the row: dy = 0, so they add nothing
#pragma unroll
            for (int e = 0; e < VW; ++e) {
                const float h = (xf[e] - mu) * rs;
                dw[i * VW + e] = fmaf(df[e], h, dw[i * VW + e]);
                db[i * VW + e] += df[e];
                const float g = wp ? df[e] * wf[e] : df[e];
                s1 += g;
                s2 = fmaf(g, h, s2);
            }
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (!WARP) {
            if (lane == 0) red[parity][warp] = make_float2(s1, s2);
            __syncthreads();
            const float2 r = lane < warps ? red[parity][lane] : make_float2(0.0f, 0.0f);
            s1 = warp_sum(r.x);
            s2 = warp_sum(r.y);
            if (csize > 1) {  // every CTA of the row gets every CTA's sums, added in rank order
                if (threadIdx.x < csize) {
                    const uint32_t at = mapa_shared(smem_u32(&peer[parity][crank]), threadIdx.x);
                    st_cluster_u32(at, __float_as_uint(s1));
                    st_cluster_u32(at + 4, __float_as_uint(s2));
                }
                cluster_sync();
                s1 = s2 = 0.0f;
                for (uint32_t c = 0; c < csize; ++c) {
                    s1 += peer[parity][c].x;
                    s2 += peer[parity][c].y;
                }
            }
        }
        const float m1 = p.rms ? 0.0f : s1 * inv_k, m2 = s2 * inv_k;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * threads + tid;
            if (c < nvec) {
                float xf[VW], df[VW], wf[VW];
                V::unpack(xv[i], xf);
                V::unpack(dv[i], df);
                V::unpack(wv[i], wf);
#pragma unroll
                for (int e = 0; e < VW; ++e) {
                    const float h = (xf[e] - mu) * rs;
                    const float g = wp ? df[e] * wf[e] : df[e];
                    df[e] = rs * (g - m1 - h * m2);
                }
                V::store(dxp + row * p.k + (int64_t)c * VW, V::pack(df));
            }
        }
    }
    if (!p.part) return;
    if (WARP) {
        float *mine = acc_sm + (int64_t)warp * 2 * p.k;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * threads + tid;
            if (c < nvec)
#pragma unroll
                for (int e = 0; e < VW; ++e) {
                    mine[c * VW + e] = dw[i * VW + e];
                    mine[p.k + c * VW + e] = db[i * VW + e];
                }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * p.k; c += blockDim.x) {
            float s = 0.0f;
            for (int g = 0; g < kBwdWarps; ++g) s += acc_sm[(int64_t)g * 2 * p.k + c];
            p.part[(int64_t)blockIdx.x * 2 * p.k + c] = s;
        }
    } else {
        float *mine = p.part + (int64_t)part * 2 * p.k;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * threads + tid;
            if (c < nvec)
#pragma unroll
                for (int e = 0; e < VW; ++e) {
                    mine[c * VW + e] = dw[i * VW + e];
                    mine[p.k + c * VW + e] = db[i * VW + e];
                }
        }
    }
}

// dw and db: column sums of the partial rows. A CTA takes 32 columns; its 32
// warps add every 32nd partial row, then the 32 sums are added in order.
__global__ void __launch_bounds__(1024) norm_bwd_reduce_kernel(const float *part, int parts, int k, float *dw, float *db) {
    __shared__ float sum[32][33];
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;  // column of [dw | db]
    float s = 0.0f;
    if (c < 2 * k)
        for (int r = warp; r < parts; r += 32) s += part[(int64_t)r * 2 * k + c];
    sum[warp][lane] = s;
    __syncthreads();
    const float t = warp_sum(sum[lane][warp]);  // column blockIdx.x * 32 + warp
    const int o = blockIdx.x * 32 + warp;
    if (lane == 0 && o < 2 * k) {
        if (o < k) {
            if (dw) dw[o] = t;
        } else if (db) {
            db[o - k] = t;
        }
    }
}

// ---------------------------------------------------------------------------
// Launches

static int threads_for(int nvec, int nv) { return (int)round_up((nvec + nv - 1) / nv, 32); }

template <typename T, int VW>
static sharq_status norm_fwd(LaunchCtx &ctx, const NormParams &p) {
    const int nvec = p.k / VW;
    const int64_t warp_grid = (p.rows + kFwdWarps - 1) / kFwdWarps;
    if (nvec <= 32) return launch_pdl(ctx, norm_fwd_kernel<T, VW, 1, true>, warp_grid, 32 * kFwdWarps, 0, 1, p);
    if (nvec <= 128) return launch_pdl(ctx, norm_fwd_kernel<T, VW, 4, true>, warp_grid, 32 * kFwdWarps, 0, 1, p);
    if (nvec <= 2048) return launch_pdl(ctx, norm_fwd_kernel<T, VW, 2, false>, p.rows, threads_for(nvec, 2), 0, 1, p);
    if (nvec <= 4096) return launch_pdl(ctx, norm_fwd_kernel<T, VW, 4, false>, p.rows, threads_for(nvec, 4), 0, 1, p);
    return launch_pdl(ctx, norm_fwd_long_kernel<T, VW>, p.rows, kLongThreads, 0, 1, p);
}

sharq_status launch_layer_norm(LaunchCtx &ctx, const void *x, int64_t rows, int64_t k, const void *w, const void *b,
                               float eps, int norm, int dtype, void *y, float *mean, float *rstd, bool vec16) {
    if (rows == 0) return SHARQ_OK;
    NormParams p{x, w, b, y, mean, rstd, rows, (int32_t)k, eps, norm};
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        return vec16 ? norm_fwd<T, 16 / (int)sizeof(T)>(ctx, p) : norm_fwd<T, 1>(ctx, p);
    });
}

// Partial rows of the weight gradients (a workspace size, so a function of
// the shape alone).
int64_t norm_bwd_parts(int64_t rows, int64_t k) {
    if (rows <= 0) return 0;
    const int64_t sms = 148;
    if (k <= 32 * kBwdCols) {
        const int64_t need = (rows + kBwdWarps - 1) / kBwdWarps;
        return need < 2 * sms ? need : 2 * sms;
    }
    const int64_t per_sm = k <= 4096 ? 3 : k <= 8192 ? 2 : 1;
    const int64_t most = k <= 8192 ? per_sm * sms : sms * 8192 / round_up(k, 8192);
    return rows < most ? rows : most;
}

template <typename T, int VW>
static sharq_status norm_bwd(LaunchCtx &ctx, const NormBwdParams &p) {
    if (p.k <= 32 * kBwdCols) {
        const size_t smem = (size_t)kBwdWarps * 2 * p.k * sizeof(float);  // at most 32 KB
        return launch_pdl(ctx, norm_bwd_kernel<T, VW, true>, p.parts, 32 * kBwdWarps, smem, 1, p);
    }
    int cluster = 1;
    while ((int64_t)cluster * kBwdThreads * kBwdCols < p.k) cluster *= 2;
    const int nvec = p.k / VW, nv = kBwdCols / VW;
    const int threads = (int)round_up(((nvec + nv - 1) / nv + cluster - 1) / cluster, 32);
    return launch_pdl(ctx, norm_bwd_kernel<T, VW, false>, (int64_t)p.parts * cluster, threads, 0, cluster, p);
}

sharq_status launch_layer_norm_backward(LaunchCtx &ctx, const void *dy, const void *x, int64_t rows, int64_t k,
                                        const void *w, const float *mean, const float *rstd, int norm, int dtype,
                                        void *dx, float *dw, float *db, float *part, bool vec16) {
    const int parts = (int)norm_bwd_parts(rows, k);
    const bool grads = dw || db;
    if (rows > 0) {
        NormBwdParams p{dy, x, w, mean, rstd, dx, grads ? part : nullptr, rows, (int32_t)k, parts, norm};
        const sharq_status st = with_dtype(dtype, [&](auto t) {
            using T = decltype(t);
            return vec16 ? norm_bwd<T, 16 / (int)sizeof(T)>(ctx, p) : norm_bwd<T, 1>(ctx, p);
        });
        if (st != SHARQ_OK) return st;
    }
    if (!grads) return SHARQ_OK;
    return launch_pdl(ctx, norm_bwd_reduce_kernel, (2 * k + 31) / 32, 1024, 0, 1, (const float *)part, parts, (int)k, dw, db);
}

}  // namespace sq

// LayerNorm and RMSNorm with 16- or 32-bit outputs, and their backward pass.
//
// Forward, per row of k values:
//   mu = sum x / k (RMSNorm: 0), rstd = 1 / sqrt(sum (x - mu)^2 / k + eps),
//   y = (x - mu) rstd w + b.
// Backward, with xhat = (x - mu) rstd and g = dy w:
//   dx = rstd (g - mean(g) - xhat mean(g xhat))   (RMSNorm: no mean(g)),
//   dw = sum over rows of dy xhat, db = sum over rows of dy.
// Values are widened to binary32, all sums are binary32; the variance is
// taken around the mean in a second pass over registers. That pass also sums
// x - mu, which is what the first sum's error left out of the mean: with it the
// mean is held as a binary32 number and a small rest, so a mean far above the
// spread costs no digits. Results are rounded once. Every sum has a fixed order:
// the same inputs give the same bits.
#include <cuda_runtime.h>
#include <string.h>

#include "sharq_dev.cuh"
#include "sq_internal.h"
#include "vec.cuh"

namespace sq {

// ---------------------------------------------------------------------------
// Sums over the threads of a row: `lanes` (a power of two) neighbouring lanes of
// a warp, or a CTA through `red` (one slot per warp; each call of a row uses
// its own array, so one barrier suffices).

template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float *red, int lanes = 32) {
    if (WARP) {
        for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        return v;
    }
    v = warp_sum(v);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    if (warps <= 8) {  // reading all of them takes fewer instructions than shuffles
        const float4 a = reinterpret_cast<const float4 *>(red)[0];
        float s = a.x;
        if (warps > 1) s += a.y;
        if (warps > 2) s += a.z;
        if (warps > 3) s += a.w;
        if (warps > 4) {
            const float4 b = reinterpret_cast<const float4 *>(red)[1];
            s += b.x;
            if (warps > 5) s += b.y;
            if (warps > 6) s += b.z;
            if (warps > 7) s += b.w;
        }
        return s;
    }
    return warp_sum(lane < warps ? red[lane] : 0.0f);
}

// The same for two sums at once; red: float2 slots.
template <bool WARP>
__device__ __forceinline__ float2 row_sum2(float2 v, float2 *red, int lanes = 32) {
    for (int o = (WARP ? lanes : 32) >> 1; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
        v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
    }
    if (WARP) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    if (warps <= 8) {
        float2 s = red[0];
#pragma unroll
        for (int i = 1; i < 8; ++i)
            if (i < warps) {
                s.x += red[i].x;
                s.y += red[i].y;
            }
        return s;
    }
    v = lane < warps ? red[lane] : make_float2(0.0f, 0.0f);
    return make_float2(warp_sum(v.x), warp_sum(v.y));
}

// sum / k, k an integer and inv_k = RN(1 / k): the product, corrected by its
// remainder (P. Markstein, IBM J. Res. Dev. 34(1), 1990), so that the mean of
// equal values with an exact sum is that value. Infinities pass.
__device__ __forceinline__ float divide_by(float sum, float k, float inv_k) {
    const float q = sum * inv_k, c = fmaf(fmaf(-q, k, sum), inv_k, q);
    return fabsf(c) <= 3.4e38f ? c : q;
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
    int32_t lanes;  // of a row, where a warp holds whole rows
    float inv_k;
};

// A row's statistics. The mean is mu + rest; rest is what mu as a binary32 number
// leaves of it.
struct RowStats {
    float mu, rest, rstd;
};

// From mu0 = the mean up to its sum's error and the sums around it of x - mu0
// and (x - mu0)^2.
__device__ __forceinline__ RowStats layer_stats(float mu0, float2 sums, const NormParams &p) {
    // where the values spread as far as the mean, the second sum is no better
    const float d = mu0 * mu0 > sums.y * p.inv_k ? divide_by(sums.x, (float)p.k, p.inv_k) : 0.0f;
    const float mu = mu0 + d;
    const float var = sums.y <= 3.4e38f ? fmaxf(sums.y * p.inv_k - d * d, 0.0f) : sums.y;
    const float rstd = rsqrtf(var + p.eps);
    if (!(fabsf(mu) <= 3.4e38f)) return {mu0, 0.0f, rstd};
    return {mu, d - (mu - mu0), rstd};
}
__device__ __forceinline__ RowStats rms_stats(float squares, const NormParams &p) {
    return {0.0f, 0.0f, rsqrtf(squares * p.inv_k + p.eps)};
}

// Steps on one vector of a row, on packed pairs of binary32 where it holds an
// even number of values (half the instructions; the pass is issue-bound
// otherwise).
template <typename T, int VW>
struct Row {
    using V = Vec<T, VW>;
    using P = typename V::P;
    static __device__ __forceinline__ float sum(P v) {
        if constexpr (VW > 1) {
            uint64_t f[VW / 2];
            V::unpack2(v, f);
            uint64_t s = f[0];
#pragma unroll
            for (int e = 1; e < VW / 2; ++e) s = add2(s, f[e]);
            const float2 t = up2(s);
            return t.x + t.y;
        } else {
            float f[VW];
            V::unpack(v, f);
            return f[0];
        }
    }
    // sum of x^2
    static __device__ __forceinline__ float sum_squares(P v) {
        if constexpr (VW > 1) {
            uint64_t f[VW / 2], q = pk2(0.0f, 0.0f);
            V::unpack2(v, f);
#pragma unroll
            for (int e = 0; e < VW / 2; ++e) q = fma2(f[e], f[e], q);
            const float2 t = up2(q);
            return t.x + t.y;
        } else {
            float f[VW];
            V::unpack(v, f);
            return f[0] * f[0];
        }
    }
    // sums of x - mu and (x - mu)^2
    static __device__ __forceinline__ float2 sums_around(P v, float mu) {
        if constexpr (VW > 1) {
            uint64_t f[VW / 2], s, q;
            const uint64_t m = pk2(-mu, -mu);
            V::unpack2(v, f);
#pragma unroll
            for (int e = 0; e < VW / 2; ++e) {
                const uint64_t d = add2(f[e], m);
                s = e == 0 ? d : add2(s, d);
                q = e == 0 ? mul2(d, d) : fma2(d, d, q);
            }
            const float2 t = up2(s), u = up2(q);
            return make_float2(t.x + t.y, u.x + u.y);
        } else {
            float f[VW];
            V::unpack(v, f);
            const float d = f[0] - mu;
            return make_float2(d, d * d);
        }
    }
    // (x - mean) rstd w + b; wv, bv: the vectors of w and b (not looked at where
    // there is none)
    static __device__ __forceinline__ P apply(P v, const RowStats &st, bool w, P wv, bool b, P bv) {
        const float shift = -st.rest * st.rstd;
        if constexpr (VW > 1) {
            uint64_t f[VW / 2], g[VW / 2];
            const uint64_t m = pk2(-st.mu, -st.mu), r = pk2(st.rstd, st.rstd), t = pk2(shift, shift);
            V::unpack2(v, f);
#pragma unroll
            for (int e = 0; e < VW / 2; ++e) f[e] = fma2(add2(f[e], m), r, t);
            if (w) {
                V::unpack2(wv, g);
#pragma unroll
                for (int e = 0; e < VW / 2; ++e) f[e] = mul2(f[e], g[e]);
            }
            if (b) {
                V::unpack2(bv, g);
#pragma unroll
                for (int e = 0; e < VW / 2; ++e) f[e] = add2(f[e], g[e]);
            }
            return V::pack2(f);
        } else {
            float f[VW], g[VW];
            V::unpack(v, f);
            f[0] = fmaf(f[0] - st.mu, st.rstd, shift);
            if (w) {
                V::unpack(wv, g);
                f[0] *= g[0];
            }
            if (b) {
                V::unpack(bv, g);
                f[0] += g[0];
            }
            return V::pack(f);
        }
    }
};

// A row lives in the registers of its threads (NV vectors of VW elements
// each, vector i of a thread at i * threads + thread), so x is read once.
// WARP: p.lanes lanes of a warp per row, kFwdWarps warps per CTA; else one CTA
// per row.
constexpr int kFwdWarps = 4;
constexpr int kFwdPair = 640;  // 16-bit rows of 513 to 640 threads: two CTAs on an SM, for a few spills (512 x 20000: 12.3 us from 13.3)

template <typename T, int VW, int NV, bool WARP, bool RMS, int MAXT = 1024>
__global__ void __launch_bounds__(WARP ? 32 * kFwdWarps : MAXT, MAXT == kFwdPair ? 2 : 1) norm_fwd_kernel(const NormParams p) {
    using V = Vec<T, VW>;
    using R = Row<T, VW>;
    __shared__ __align__(16) float red[32];
    __shared__ float2 red2[32];
    griddep_wait();
    griddep_launch();
    const int threads = WARP ? p.lanes : blockDim.x;
    const int tid = WARP ? (threadIdx.x & (p.lanes - 1)) : threadIdx.x;
    int64_t row = blockIdx.x;
    bool here = true;
    if (WARP) {
        row = ((int64_t)blockIdx.x * (32 * kFwdWarps) + threadIdx.x) / p.lanes;
        here = row < p.rows;
        if (!here) row = p.rows - 1;  // the warp's shuffles need every lane
    }
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
    auto fetch = [&](const T *from, int i) {
        const int c = i * threads + tid;
        return from && c < nvec ? V::load(from + (int64_t)c * VW) : V::zero();
    };
    // The first vectors of w and b set out before the row's sums, the others one
    // ahead: the compiler moves no load over a barrier or a store (8192 x 4096 in
    // fp16: 25.0 us from 27.0). In 32 bits that costs a CTA of registers (4096 x
    // 4096: 28.1 us against 25.5).
    constexpr int kAheadW = sizeof(T) == 4 && VW > 1 ? 0 : 1;
    typename V::P wv[NV], bv[NV];
#pragma unroll
    for (int i = 0; i < kAheadW; ++i) {
        wv[i] = fetch(w, i);
        bv[i] = fetch(b, i);
    }
    RowStats st;
    if (RMS) {
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) q += R::sum_squares(xv[i]);
        st = rms_stats(row_sum<WARP>(q, red, threads), p);
    } else {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) s += R::sum(xv[i]);
        const float mu0 = row_sum<WARP>(s, red, threads) * p.inv_k;
        float2 a = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float2 d = R::sums_around(xv[i], mu0);
            if (i * threads + tid < nvec) {
                a.x += d.x;
                a.y += d.y;
            }
        }
        st = layer_stats(mu0, row_sum2<WARP>(a, red2, threads), p);
    }
    if (tid == 0 && here) {
        if (p.mean) p.mean[row] = st.mu;
        if (p.rstd) p.rstd[row] = st.rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * threads + tid;
        if (i + kAheadW < NV) {
            wv[i + kAheadW] = fetch(w, i + kAheadW);
            bv[i + kAheadW] = fetch(b, i + kAheadW);
        }
        const typename V::P o = R::apply(xv[i], st, w != nullptr, wv[i], b != nullptr, bv[i]);
        if (c < nvec && here) V::store(y + (int64_t)c * VW, o);
    }
}

// Rows too long for the registers: the same sums in three passes over the
// row, which stays in L2 (at most 256 KB). Two sums of every kind per thread, so
// that none has more than 64 terms. Two CTAs of 512 threads on an SM leave room
// for two vectors in flight (8192 x 4097 in fp16, single values: 112 us with CTAs
// of 1024).
constexpr int kLongThreads = 512;

template <typename T, int VW, bool RMS>
__global__ void __launch_bounds__(kLongThreads, 2) norm_fwd_long_kernel(const NormParams p) {
    using V = Vec<T, VW>;
    __shared__ __align__(16) float red[32];
    __shared__ float2 red2[32];
    griddep_wait();
    griddep_launch();
    const int64_t row = blockIdx.x;
    const int nvec = p.k / VW;
    const T *x = static_cast<const T *>(p.x) + row * p.k;
    T *y = static_cast<T *>(p.y) + row * p.k;
    const T *w = static_cast<const T *>(p.w), *b = static_cast<const T *>(p.b);
    using R = Row<T, VW>;
    RowStats st;
    // f(u, vector c) for this thread's vectors, u = 0 and 1 in turn
    auto walk = [&](auto f) {
        for (int c = threadIdx.x; c < nvec; c += 2 * kLongThreads) {
            f(0, V::load(x + (int64_t)c * VW));
            if (c + kLongThreads < nvec) f(1, V::load(x + (int64_t)(c + kLongThreads) * VW));
        }
    };
    if (RMS) {
        float q[2] = {};
        walk([&](int u, typename V::P v) { q[u] += R::sum_squares(v); });
        st = rms_stats(row_sum<false>(q[0] + q[1], red), p);
    } else {
        float s[2] = {};
        walk([&](int u, typename V::P v) { s[u] += R::sum(v); });
        const float mu0 = row_sum<false>(s[0] + s[1], red) * p.inv_k;
        float2 a[2] = {};
        walk([&](int u, typename V::P v) {
            const float2 d = R::sums_around(v, mu0);
            a[u].x += d.x;
            a[u].y += d.y;
        });
        st = layer_stats(mu0, row_sum2<false>(make_float2(a[0].x + a[1].x, a[0].y + a[1].y), red2), p);
    }
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = st.mu;
        if (p.rstd) p.rstd[row] = st.rstd;
    }
    constexpr int U = VW > 1 ? 2 : 1;  // vectors in flight
    for (int c0 = threadIdx.x; c0 < nvec; c0 += U * kLongThreads) {
        typename V::P xv[U], wv[U], bv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = c0 + u * kLongThreads;
            const bool in = c < nvec;
            xv[u] = in ? V::load(x + c * VW) : V::zero();
            wv[u] = in && w ? V::load(w + c * VW) : V::zero();
            bv[u] = in && b ? V::load(b + c * VW) : V::zero();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = c0 + u * kLongThreads;
            const typename V::P o = R::apply(xv[u], st, w != nullptr, wv[u], b != nullptr, bv[u]);
            if (c < nvec) V::store(y + c * VW, o);
        }
    }
}

// ---------------------------------------------------------------------------
// Backward
//
// Persistent row groups (some lanes of a warp, or a CTA) walk the rows; a
// thread always owns the same kBwdCols columns, so the weight gradients add up
// in its registers over all its rows and leave the SM once, as one partial row
// per CTA; a second kernel adds the partial rows in their order. The next row
// is loaded before the current one is reduced. Rows longer than a CTA's
// registers take two passes, at the end of this section.
constexpr int kBwdCols = 16;          // columns per thread
constexpr int kBwdThreads = 512;      // most threads of a CTA
constexpr int kBwdSmall = 256;        // threads up to which an SM holds more than one
constexpr int kBwdRow = kBwdThreads * kBwdCols;  // longest row of one pass
constexpr int kBwdWarps = 8;          // warps of a CTA of the warp form

struct NormBwdParams {
    const void *dy, *x, *w;
    const float *mean, *rstd;
    void *dx;
    float *part;  // [parts][part_cols]: dw, then db (LayerNorm); NULL: no weight gradients
    int64_t rows, part_cols;
    int32_t k, parts, rms;
    int32_t lanes;  // of a row in the warp form
    float2 *sums;   // rows in two passes: each row's means of g and of g xhat
};

template <typename T, int VW, bool WARP>
__global__ void __launch_bounds__(kBwdThreads) norm_bwd_kernel(const NormBwdParams p) {
    using V = Vec<T, VW>;
    constexpr int NV = kBwdCols / VW;
    __shared__ float2 red[2][kBwdThreads / 32];
    extern __shared__ float acc_sm[];  // WARP: [row groups][2][k]
    griddep_wait();
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int threads = WARP ? p.lanes : (int)blockDim.x;
    const int tid = WARP ? (lane & (p.lanes - 1)) : (int)threadIdx.x;
    const int groups = WARP ? 32 * kBwdWarps / p.lanes : 1, group = WARP ? (int)threadIdx.x / p.lanes : 0;
    const int part = (int)blockIdx.x;
    const int64_t first = WARP ? (int64_t)blockIdx.x * groups + group : (int64_t)part;
    const int64_t step = WARP ? (int64_t)gridDim.x * groups : (int64_t)gridDim.x;
    // the warp form's shuffles need every lane: all groups take as many steps
    const int64_t last = WARP ? (int64_t)blockIdx.x * groups : first;
    const int nvec = p.k / VW;
    const T *xp = static_cast<const T *>(p.x), *dyp = static_cast<const T *>(p.dy), *wp = static_cast<const T *>(p.w);
    T *dxp = static_cast<T *>(p.dx);
    const float inv_k = 1.0f / (float)p.k;

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
    auto clear = [&]() {  // a row that adds nothing
#pragma unroll
        for (int i = 0; i < NV; ++i) xn[i] = dn[i] = V::zero();
    };
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * threads + tid;
            const bool in = c < nvec;
            xn[i] = in ? V::load(xp + row * p.k + (int64_t)c * VW) : V::zero();
            dn[i] = in ? V::load(dyp + row * p.k + (int64_t)c * VW) : V::zero();
        }
        mu_n = p.rms ? 0.0f : p.mean[row];
        rs_n = p.rstd[row];
    };
    if (first < p.rows) fetch(first);
    else clear();
    int parity = 0;
    for (int64_t row = first, lead = last; lead < p.rows; row += step, lead += step, parity ^= 1) {
        typename V::P xv[NV], dv[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            xv[i] = xn[i];
            dv[i] = dn[i];
        }
        const float mu = mu_n, rs = rs_n;
        if (row + step < p.rows) fetch(row + step);
        else clear();
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
        if (WARP) {
            for (int o = p.lanes >> 1; o > 0; o >>= 1) {
                s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, o);
                s2 += __shfl_xor_sync(0xFFFFFFFFu, s2, o);
            }
        } else {
            s1 = warp_sum(s1);
            s2 = warp_sum(s2);
            if (lane == 0) red[parity][warp] = make_float2(s1, s2);
            __syncthreads();
            const float2 r = lane < warps ? red[parity][lane] : make_float2(0.0f, 0.0f);
            s1 = warp_sum(r.x);
            s2 = warp_sum(r.y);
        }
        const float m1 = p.rms ? 0.0f : s1 * inv_k, m2 = s2 * inv_k;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * threads + tid;
            if (c < nvec && row < p.rows) {
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
        float *mine = acc_sm + (int64_t)group * 2 * p.k;
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
        for (int c = threadIdx.x; c < p.part_cols; c += blockDim.x) {
            float s = 0.0f;
            for (int g = 0; g < groups; ++g) s += acc_sm[(int64_t)g * 2 * p.k + c];
            p.part[(int64_t)blockIdx.x * p.part_cols + c] = s;
        }
    } else {
        float *mine = p.part + (int64_t)part * p.part_cols;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * threads + tid;
            if (c < nvec)
#pragma unroll
                for (int e = 0; e < VW; ++e) {
                    mine[c * VW + e] = dw[i * VW + e];
                    if (!p.rms) mine[p.k + c * VW + e] = db[i * VW + e];
                }
        }
    }
}

// The form for rows of whole 16-byte vectors: a CTA per row, kBwdCols columns
// per thread, and a ring of rows of x and dy filled by bulk copies several rows
// ahead. The barrier of a row's reduction also frees its ring slot. Bound by
// instructions and their latency (half the issue slots at 16 warps per SM;
// fewer columns per thread and more warps measured slower: 8192 x 4096 in bf16
// takes 36.5 us like this, 56 with 8 columns): 75% of the copy rate with the
// reduction of the partial rows.
constexpr int kRingMax = 8;            // most rows in a ring
constexpr int kRingBytes = 160 << 10;  // shared memory of an SM's rings
constexpr int kRingEnough = 3;         // rows of a ring where an SM has several (more measured no faster)

// FULL: every thread has all its columns.
template <typename T, int VW, int MAXT, bool FULL>
__global__ void __launch_bounds__(MAXT, MAXT <= kBwdSmall ? 2 : 1)
    norm_bwd_ring_kernel(const NormBwdParams p, int stages, uint64_t wait_ns, unsigned *status) {
    using V = Vec<T, VW>;
    constexpr int NV = kBwdCols / VW, H = VW / 2;
    extern __shared__ __align__(128) uint8_t ring[];  // [stages][x, dy][part of a row]
    __shared__ uint64_t full[kRingMax];
    __shared__ __align__(16) float2 red[2][MAXT / 32];
    __shared__ int gave_up[2];  // a wait of this row ran out (rows take turns, as in red)
    griddep_wait();
    griddep_launch();
    const int tid = threadIdx.x, threads = blockDim.x, warp = tid >> 5, lane = tid & 31;
    const int cnt = p.k / VW;  // vectors of a row
    const uint32_t bytes = (uint32_t)cnt * 16;
    const int64_t part = blockIdx.x, parts = gridDim.x;
    const int iters = (int)((p.rows - part + parts - 1) / parts);
    const T *xp = static_cast<const T *>(p.x), *dyp = static_cast<const T *>(p.dy);
    const T *wp = static_cast<const T *>(p.w);
    T *dxp = static_cast<T *>(p.dx);
    auto issue = [&](int it, int s) {
        const int64_t at = (part + it * parts) * p.k;
        const uint32_t dst = smem_u32(ring) + s * 2 * bytes, bar = smem_u32(&full[s]);
        mbar_arrive_expect_tx(bar, 2 * bytes);
        bulk_load(dst, xp + at, bytes, bar);
        bulk_load(dst + bytes, dyp + at, bytes, bar);
    };
    if (tid == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(smem_u32(&full[s]), 1);
        mbar_fence_init();
        gave_up[0] = gave_up[1] = 0;
    }
    if (tid < 2 * (MAXT / 32)) red[tid / (MAXT / 32)][tid % (MAXT / 32)] = make_float2(0.0f, 0.0f);  // warps not there
    __syncthreads();
    if (tid == 0)
        for (int it = 0; it < stages && it < iters; ++it) issue(it, it);
    const float inv_k = 1.0f / (float)p.k;
    uint64_t wf[NV][H], dw[NV][H], db[NV][H];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * threads + tid;
        V::unpack2(wp && (FULL || c < cnt) ? V::load(wp + (int64_t)c * VW) : V::ones(), wf[i]);
#pragma unroll
        for (int e = 0; e < H; ++e) dw[i][e] = db[i][e] = 0;
    }
    T *dx_row = dxp + part * p.k + tid * VW;
    const int64_t dx_step = parts * p.k;
    float mu_n = p.rms || iters <= 0 ? 0.0f : p.mean[part], rs_n = iters <= 0 ? 0.0f : p.rstd[part];
    int slot = 0;
    uint32_t phase = 0;
    for (int it = 0; it < iters; ++it) {
        const int64_t row = part + it * parts;
        const float mu = mu_n, rs = rs_n;
        if (it + 1 < iters) {
            if (!p.rms) mu_n = p.mean[row + parts];
            rs_n = p.rstd[row + parts];
        }
        const uint64_t mu2 = pk2(-mu, -mu), rs2 = pk2(rs, rs);
        const int parity = it & 1;
        if (!mbar_wait_own(smem_u32(&full[slot]), phase, status, kSiteNormRing, wait_ns)) gave_up[parity] = 1;
        uint64_t h[NV][H], g[NV][H], t1 = 0, t2 = 0;  // xhat and g = dy w; sums of g and g xhat
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * threads + tid;
            const uint8_t *at = ring + slot * 2 * bytes + c * 16;
            uint64_t df[H];
            // columns past the row: dy = 0, so they add nothing
            V::unpack2(FULL || c < cnt ? *reinterpret_cast<const typename V::P *>(at) : V::zero(), h[i]);
            V::unpack2(FULL || c < cnt ? *reinterpret_cast<const typename V::P *>(at + bytes) : V::zero(), df);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                h[i][e] = mul2(add2(h[i][e], mu2), rs2);
                dw[i][e] = fma2(df[e], h[i][e], dw[i][e]);
                db[i][e] = add2(db[i][e], df[e]);
                g[i][e] = mul2(df[e], wf[i][e]);
                t1 = add2(t1, g[i][e]);
                t2 = fma2(g[i][e], h[i][e], t2);
            }
        }
        const float2 f1 = up2(t1), f2 = up2(t2);
        // lanes 0-15 go on with the first sum, lanes 16-31 with the second
        float s1 = f1.x + f1.y, s2 = f2.x + f2.y;
        float v = (lane & 16 ? s2 : s1) + __shfl_xor_sync(0xFFFFFFFFu, lane & 16 ? s1 : s2, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        if (lane == 0) red[parity][warp].x = v;
        if (lane == 16) red[parity][warp].y = v;
        __syncthreads();
        if (gave_up[parity]) {  // the copies in flight land before the CTA's shared memory goes
            if (tid == 0)
                for (int f = it; f < iters && f < it + stages; ++f)
                    (void)mbar_wait_own(smem_u32(&full[f % stages]), (f / stages) & 1, nullptr, 0, kOwnDrainNs);
            return;
        }
        if (tid == 0 && it + stages < iters) issue(it + stages, slot);
        s1 = s2 = 0.0f;
        const float4 *rp = reinterpret_cast<const float4 *>(red[parity]);
#pragma unroll
        for (int i = 0; i < MAXT / 64; ++i) {
            const float4 r = rp[i];
            s1 += r.x + r.z;
            s2 += r.y + r.w;
        }
        const float m1 = p.rms ? 0.0f : s1 * inv_k, m2 = s2 * inv_k;
        const uint64_t m1n = pk2(-m1 * rs, -m1 * rs), m2n = pk2(-m2, -m2);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * threads + tid;
#pragma unroll
            for (int e = 0; e < H; ++e) g[i][e] = fma2(fma2(h[i][e], m2n, g[i][e]), rs2, m1n);
            if (FULL || c < cnt) V::store(dx_row + (int64_t)i * threads * VW, V::pack2(g[i]));
        }
        dx_row += dx_step;
        if (++slot == stages) {
            slot = 0;
            phase ^= 1;
        }
    }
    if (!p.part) return;
    float *mine = p.part + part * p.part_cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * threads + tid;
        if (c < cnt)
#pragma unroll
            for (int e = 0; e < H; ++e) {
                *reinterpret_cast<float2 *>(mine + c * VW + 2 * e) = up2(dw[i][e]);
                if (!p.rms) *reinterpret_cast<float2 *>(mine + p.k + c * VW + 2 * e) = up2(db[i][e]);
            }
    }
}

// Rows longer than kBwdRow: their sums first (a CTA per row), then dx and the
// weight gradients by columns (a CTA takes kColThreads x kColVecs vectors of
// some rows, and no thread waits for another). x and dy are read twice, the
// second time from L2 where they fit. (Clusters with a part of the columns per
// CTA read them once, but a cluster barrier per row costs more: 1024 x 14336 in
// bf16 took 43 us, 512 x 20000 62 us, against 35 and 26 like this, before plain
// loads added 0.7.)
constexpr int kColThreads = 256;
constexpr int kColRows = 4;  // rows in flight

template <typename T, int VW>
__global__ void __launch_bounds__(kBwdThreads) norm_bwd_sums_kernel(const NormBwdParams p) {
    using V = Vec<T, VW>;
    __shared__ __align__(16) float red[2][32];
    griddep_wait();
    griddep_launch();
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.k, *dy = static_cast<const T *>(p.dy) + row * p.k;
    const T *w = static_cast<const T *>(p.w);
    const float mu = p.rms ? 0.0f : p.mean[row], rs = p.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    const uint64_t mu2 = pk2(-mu, -mu), rs2 = pk2(rs, rs);
#pragma unroll 4
    for (int c = threadIdx.x; c < p.k / VW; c += kBwdThreads) {
        const typename V::P xv = V::load(x + (int64_t)c * VW), dv = V::load(dy + (int64_t)c * VW);
        const typename V::P wv = w ? V::load(w + (int64_t)c * VW) : V::ones();
        if constexpr (VW > 1) {
            uint64_t xf[VW / 2], df[VW / 2], wf[VW / 2], t1 = 0, t2 = 0;
            V::unpack2(xv, xf);
            V::unpack2(dv, df);
            V::unpack2(wv, wf);
#pragma unroll
            for (int e = 0; e < VW / 2; ++e) {
                const uint64_t g = mul2(df[e], wf[e]);
                t1 = add2(t1, g);
                t2 = fma2(g, mul2(add2(xf[e], mu2), rs2), t2);
            }
            const float2 a = up2(t1), b = up2(t2);
            s1 += a.x + a.y;
            s2 += b.x + b.y;
        } else {
            float xf[VW], df[VW], wf[VW];
            V::unpack(xv, xf);
            V::unpack(dv, df);
            V::unpack(wv, wf);
            const float g = df[0] * wf[0];
            s1 += g;
            s2 = fmaf(g, (xf[0] - mu) * rs, s2);
        }
    }
    s1 = row_sum<false>(s1, red[0]);
    s2 = row_sum<false>(s2, red[1]);
    const float inv_k = 1.0f / (float)p.k;
    if (threadIdx.x == 0) p.sums[row] = make_float2(p.rms ? 0.0f : s1 * inv_k, s2 * inv_k);
}

template <typename T, int VW, int NV>
__global__ void __launch_bounds__(kColThreads) norm_bwd_cols_kernel(const NormBwdParams p) {
    using V = Vec<T, VW>;
    griddep_wait();
    griddep_launch();
    const int nvec = p.k / VW, across = (nvec + kColThreads * NV - 1) / (kColThreads * NV);
    const int64_t part = blockIdx.x / across;
    const int v0 = (int)(blockIdx.x % across) * kColThreads * NV + (int)threadIdx.x;
    const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy), *w = static_cast<const T *>(p.w);
    T *dx = static_cast<T *>(p.dx);
    constexpr int H = (VW + 1) / 2;  // packed pairs (a single value: the pair's first)
    uint64_t wf[NV][H], dw[NV][H], db[NV][H];
    auto widen2 = [](typename V::P v, uint64_t (&f)[H]) {
        if constexpr (VW > 1) {
            V::unpack2(v, f);
        } else {
            float t[VW];
            V::unpack(v, t);
            f[0] = pk2(t[0], 0.0f);
        }
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = v0 + i * kColThreads;
        widen2(w && c < nvec ? V::load(w + (int64_t)c * VW) : V::ones(), wf[i]);
#pragma unroll
        for (int e = 0; e < H; ++e) dw[i][e] = db[i][e] = 0;
    }
    for (int64_t r0 = part; r0 < p.rows; r0 += (int64_t)kColRows * p.parts) {
        typename V::P xv[kColRows][NV], dv[kColRows][NV];
        float mu[kColRows], rs[kColRows];
        float2 m[kColRows];
#pragma unroll
        for (int j = 0; j < kColRows; ++j) {
            const int64_t row = r0 + (int64_t)j * p.parts;
            const bool in = row < p.rows;
            mu[j] = in && !p.rms ? p.mean[row] : 0.0f;
            rs[j] = in ? p.rstd[row] : 0.0f;
            m[j] = in ? p.sums[row] : make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = v0 + i * kColThreads;
                const bool here = in && c < nvec;
                xv[j][i] = here ? V::load(x + row * p.k + (int64_t)c * VW) : V::zero();
                dv[j][i] = here ? V::load(dy + row * p.k + (int64_t)c * VW) : V::zero();
            }
        }
#pragma unroll
        for (int j = 0; j < kColRows; ++j) {
            const int64_t row = r0 + (int64_t)j * p.parts;
            const uint64_t mu2 = pk2(-mu[j], -mu[j]), rs2 = pk2(rs[j], rs[j]), m2n = pk2(-m[j].y, -m[j].y);
            const uint64_t m1n = pk2(-m[j].x * rs[j], -m[j].x * rs[j]);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = v0 + i * kColThreads;
                uint64_t h[H], df[H];
                widen2(xv[j][i], h);
                widen2(dv[j][i], df);
#pragma unroll
                for (int e = 0; e < H; ++e) {  // rows past the end: dy = 0
                    h[e] = mul2(add2(h[e], mu2), rs2);
                    dw[i][e] = fma2(df[e], h[e], dw[i][e]);
                    db[i][e] = add2(db[i][e], df[e]);
                    df[e] = fma2(fma2(h[e], m2n, mul2(df[e], wf[i][e])), rs2, m1n);
                }
                if (row < p.rows && c < nvec) {
                    typename V::P o;
                    if constexpr (VW > 1) {
                        o = V::pack2(df);
                    } else {
                        const float t[VW] = {up2(df[0]).x};
                        o = V::pack(t);
                    }
                    V::store(dx + row * p.k + (int64_t)c * VW, o);
                }
            }
        }
    }
    if (!p.part) return;
    float *mine = p.part + part * p.part_cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = v0 + i * kColThreads;
        if (c < nvec)
#pragma unroll
            for (int e = 0; e < VW; ++e) {
                const float2 a = up2(dw[i][e / 2]), b = up2(db[i][e / 2]);
                mine[c * VW + e] = e & 1 ? a.y : a.x;
                if (!p.rms) mine[p.k + c * VW + e] = e & 1 ? b.y : b.x;
            }
    }
}

// dw and db: column sums of the partial rows. A CTA takes 32 columns; each of
// its W warps adds every W-th partial row, then the W sums are added in order.
template <int W>
__global__ void __launch_bounds__(32 * W) norm_bwd_reduce_kernel(const float *part, int parts, int64_t cols, int k, float *dw,
                                                                 float *db) {
    __shared__ float sum[W][32];
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;  // column of [dw | db]
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int r = warp; r < parts; r += W) s += part[r * cols + c];
    }
    sum[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || c >= cols) return;
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) t += sum[i][lane];
    if (c < k) {
        if (dw) dw[c] = t;
    } else if (db) {
        db[c - k] = t;
    }
}

// ---------------------------------------------------------------------------
// Launches

static int threads_for(int nvec, int nv) { return (int)round_up((nvec + nv - 1) / nv, 32); }

template <typename T, int VW, bool RMS>
static sharq_status norm_fwd(LaunchCtx &ctx, const NormParams &p) {
    const int nvec = p.k / VW;
    if (nvec <= 128) {
        NormParams q = p;
        const int nv = nvec <= 64 ? 2 : 4;
        for (q.lanes = 1; q.lanes * nv < nvec; q.lanes *= 2) {}
        const int64_t per = 32 * kFwdWarps / q.lanes, grid = (p.rows + per - 1) / per;
        return nv == 2 ? launch_pdl(ctx, norm_fwd_kernel<T, VW, 2, true, RMS>, grid, 32 * kFwdWarps, 0, 1, q)
                       : launch_pdl(ctx, norm_fwd_kernel<T, VW, 4, true, RMS>, grid, 32 * kFwdWarps, 0, 1, q);
    }
    if constexpr (VW == 8)
        if (nvec > 4 * 512 && nvec <= 4 * kFwdPair)
            return launch_pdl(ctx, norm_fwd_kernel<T, VW, 4, false, RMS, kFwdPair>, p.rows, threads_for(nvec, 4), 0, 1, p);
    if (nvec <= 4096) return launch_pdl(ctx, norm_fwd_kernel<T, VW, 4, false, RMS>, p.rows, threads_for(nvec, 4), 0, 1, p);
    return launch_pdl(ctx, norm_fwd_long_kernel<T, VW, RMS>, p.rows, kLongThreads, 0, 1, p);
}

sharq_status launch_layer_norm(LaunchCtx &ctx, const void *x, int64_t rows, int64_t k, const void *w, const void *b,
                               float eps, int norm, int dtype, void *y, float *mean, float *rstd, bool vec16) {
    if (rows == 0) return SHARQ_OK;
    NormParams p{x, w, b, y, mean, rstd, rows, (int32_t)k, eps, 32, 1.0f / (float)k};
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int VW = 16 / (int)sizeof(T);
        if (norm == 1) return vec16 ? norm_fwd<T, VW, true>(ctx, p) : norm_fwd<T, 1, true>(ctx, p);
        return vec16 ? norm_fwd<T, VW, false>(ctx, p) : norm_fwd<T, 1, false>(ctx, p);
    });
}

static int bwd_lanes(int64_t k) {  // of a row in the warp form
    int l = 1;
    while (l * kBwdCols < k) l *= 2;
    return l;
}
// Threads of a row's CTA, and how many such CTAs an SM holds.
static int bwd_threads(int64_t k) { return (int)round_up((k + kBwdCols - 1) / kBwdCols, 32); }
static int bwd_per_sm(int threads) {
    if (threads > kBwdSmall) return 1;
    const int n = 2 * kBwdSmall / threads;
    return n > 8 ? 8 : n;
}

// Row groups of the backward pass, each with a partial row of the weight
// gradients (a workspace size, so a function of the shape alone). A group has
// some rows to itself, or the partial rows outweigh the pass.
static int64_t norm_bwd_parts(int64_t rows, int64_t k) {
    if (rows <= 0) return 0;
    const int64_t sms = 148;
    if (k <= 32 * kBwdCols) {
        const int64_t per = 32 * kBwdWarps / bwd_lanes(k), need = (rows + per - 1) / per;
        return need < 2 * sms ? need : 2 * sms;
    }
    if (k > kBwdRow) {  // two CTAs per SM (as fit), each with at least kColRows rows
        const int64_t across = (k + 2047) / 2048, most = across < 2 * sms ? 2 * sms / across : 1;
        const int64_t need = (rows + kColRows - 1) / kColRows;
        return need < most ? need : most;
    }
    const int64_t most = bwd_per_sm(bwd_threads(k)) * sms;
    const int64_t few = rows <= 64 ? rows : rows / 4 < 64 ? 64 : rows / 4;
    return few < most ? few : most;
}

template <typename T, int VW>
static sharq_status norm_bwd(LaunchCtx &ctx, const NormBwdParams &p) {
    if (p.k <= 32 * kBwdCols) {
        NormBwdParams q = p;
        q.lanes = bwd_lanes(p.k);
        const size_t smem = (size_t)(32 * kBwdWarps / q.lanes) * 2 * p.k * sizeof(float);  // at most 32 KB
        return launch_pdl(ctx, norm_bwd_kernel<T, VW, true>, p.parts, 32 * kBwdWarps, smem, 1, q);
    }
    if (p.k > kBwdRow) {
        constexpr int NV = VW == 8 ? 1 : VW == 4 ? 2 : 4;
        const sharq_status st = launch_pdl(ctx, norm_bwd_sums_kernel<T, VW>, p.rows, kBwdThreads, 0, 1, p);
        if (st != SHARQ_OK) return st;
        const int64_t across = (p.k / VW + kColThreads * NV - 1) / (kColThreads * NV);
        return launch_pdl(ctx, norm_bwd_cols_kernel<T, VW, NV>, across * p.parts, kColThreads, 0, 1, p);
    }
    const int threads = bwd_threads(p.k);
    if constexpr (VW > 1) {
        const int64_t pair = 2 * 16 * (p.k / VW);
        const int per_sm = bwd_per_sm(threads), most = per_sm > 1 ? kRingEnough : kRingMax;
        const int64_t fit = kRingBytes / per_sm / pair;  // at least 2: a pair of rows has at most 64 KB
        const int stages = fit > most ? most : (int)fit;
        const bool full = p.k % ((int64_t)threads * kBwdCols) == 0;
        auto run = [&](auto kernel) {
            return launch_pdl(ctx, kernel, p.parts, threads, (size_t)(stages * pair), 1, p, stages, ctx.wait_ns, ctx.status);
        };
        SQ_SMEM_ONCE((norm_bwd_ring_kernel<T, VW, kBwdSmall, true>), kRingBytes);
        SQ_SMEM_ONCE((norm_bwd_ring_kernel<T, VW, kBwdSmall, false>), kRingBytes);
        SQ_SMEM_ONCE((norm_bwd_ring_kernel<T, VW, kBwdThreads, true>), kRingBytes);
        SQ_SMEM_ONCE((norm_bwd_ring_kernel<T, VW, kBwdThreads, false>), kRingBytes);
        if (threads <= kBwdSmall)
            return full ? run(norm_bwd_ring_kernel<T, VW, kBwdSmall, true>) : run(norm_bwd_ring_kernel<T, VW, kBwdSmall, false>);
        return full ? run(norm_bwd_ring_kernel<T, VW, kBwdThreads, true>) : run(norm_bwd_ring_kernel<T, VW, kBwdThreads, false>);
    } else {
        return launch_pdl(ctx, norm_bwd_kernel<T, VW, false>, p.parts, threads, 0, 1, p);
    }
}

int64_t norm_bwd_bytes(int64_t rows, int64_t k) {
    return round_up(norm_bwd_parts(rows, k) * 2 * k * (int64_t)sizeof(float), kAlign) + (k > kBwdRow ? rows * 8 : 0);
}

bool norm_bwd_one_pass(int64_t k) { return k <= kBwdRow; }

sharq_status launch_layer_norm_backward(LaunchCtx &ctx, const void *dy, const void *x, int64_t rows, int64_t k,
                                        const void *w, const float *mean, const float *rstd, int norm, int dtype,
                                        void *dx, float *dw, float *db, void *ws, bool vec16) {
    float *part = static_cast<float *>(ws);
    const int parts = (int)norm_bwd_parts(rows, k);
    const bool grads = dw || db;
    const int64_t cols = norm == 1 ? k : 2 * k;  // RMSNorm has no db
    if (rows > 0) {
        NormBwdParams p{dy, x, w, mean, rstd, dx, grads ? part : nullptr, rows, cols, (int32_t)k, parts, norm, 32, nullptr};
        if (k > kBwdRow)
            p.sums = reinterpret_cast<float2 *>(static_cast<uint8_t *>(ws) + round_up((int64_t)parts * 2 * k * (int64_t)sizeof(float), kAlign));
        const sharq_status st = with_dtype(dtype, [&](auto t) {
            using T = decltype(t);
            return vec16 ? norm_bwd<T, 16 / (int)sizeof(T)>(ctx, p) : norm_bwd<T, 1>(ctx, p);
        });
        if (st != SHARQ_OK) return st;
    }
    if (!grads) return SHARQ_OK;
    const int64_t grid = (cols + 31) / 32;
    return parts > 128 ? launch_pdl(ctx, norm_bwd_reduce_kernel<32>, grid, 1024, 0, 1, part, parts, cols, (int)k, dw, db)
                       : launch_pdl(ctx, norm_bwd_reduce_kernel<8>, grid, 256, 0, 1, part, parts, cols, (int)k, dw, db);
}

}  // namespace sq

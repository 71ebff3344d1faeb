// Token order of mixture-of-experts layers (and of adapters): entries sorted
// by group, rows moved into that order, and back with weights, with the
// gradient of the way back.
//
//   route     offsets, rows, slots of a stable counting sort of the entries
//             (token t, choice j), whose group is ids[t][j]
//   permute   out[slots[t][j]] = x[t]
//   combine   out[t] = residual[t] + sum_j weights[t][j] y[slots[t][j]]
//   gradient  dy[slots[t][j]] = weights[t][j] dout[t],
//             dweights[t][j] = <dout[t], y[slots[t][j]]>
//
// Sums are binary32 in a fixed order and rounded once. Entries without a
// group have slot -1 and are left out of every sum.
#include <cuda_runtime.h>

#include "sharq_dev.cuh"
#include "sq_internal.h"
#include "vec.cuh"

namespace sq {

// ---------------------------------------------------------------------------
// Route: one launch of one cluster. Every warp owns a contiguous run of
// entries, so the sort is stable if a warp's entries of a group follow those
// of the warps before it. Each warp counts its entries per group (lanes with
// the same group meet in a match, one lane adds), a scan over warps, CTAs
// (through distributed shared memory) and groups turns the counts into first
// slots, and a second walk over the entries hands the slots out.
constexpr int kRouteThreads = 1024;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteCluster = 8;
constexpr int kRouteKeep = 4;  // steps of 32 entries whose groups a lane keeps in registers

struct RouteParams {
    const void *ids;
    int64_t entries;
    int32_t top_k, groups;
    int32_t *offsets, *rows, *slots;
};

template <typename ID>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteParams p) {
    extern __shared__ int32_t sm[];
    int32_t *hist = sm;                               // [kRouteWarps][groups]
    int32_t *mine = sm + kRouteWarps * p.groups;      // [groups] entries of this CTA
    __shared__ int32_t scan[kRouteWarps];
    __shared__ int32_t total_s;
    griddep_wait();
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = threadIdx.x;
    const uint32_t rank = cluster_ctarank();
    const int64_t ctas = gridDim.x;
    const int64_t run = ((p.entries + ctas * kRouteWarps - 1) / (ctas * kRouteWarps) + 31) / 32 * 32;
    const int64_t e0 = ((int64_t)rank * kRouteWarps + warp) * run;
    const int64_t e1 = min(e0 + run, p.entries);
    const ID *ids = static_cast<const ID *>(p.ids);
    int32_t *wh = hist + warp * p.groups;

    for (int i = threadIdx.x; i < kRouteWarps * p.groups; i += kRouteThreads) hist[i] = 0;
    auto group_at = [&](int64_t e) -> int32_t {
        if (e >= e1) return -1;
        const ID v = ids[e];
        return v >= 0 && v < (ID)p.groups ? (int32_t)v : -1;
    };
    int32_t kept[kRouteKeep];
#pragma unroll
    for (int s = 0; s < kRouteKeep; ++s) kept[s] = group_at(e0 + s * 32 + lane);
    __syncthreads();

    // The lanes of my group before me in a step, and whether I add for them.
    auto count = [&](int32_t v) {
        const unsigned peers = __match_any_sync(0xFFFFFFFFu, v);
        if (v >= 0 && lane == __ffs((int)peers) - 1) wh[v] += __popc(peers);
        __syncwarp();
    };
#pragma unroll
    for (int s = 0; s < kRouteKeep; ++s)
        if (e0 + s * 32 < e1) count(kept[s]);
    for (int64_t e = e0 + kRouteKeep * 32; e < e1; e += 32) count(group_at(e + lane));
    __syncthreads();

    if (g < p.groups) {
        int32_t run_sum = 0;
#pragma unroll 8
        for (int w = 0; w < kRouteWarps; ++w) {
            const int32_t c = hist[w * p.groups + g];
            hist[w * p.groups + g] = run_sum;
            run_sum += c;
        }
        mine[g] = run_sum;
    }
    int32_t before = 0, all = 0;
    if (ctas > 1) {
        cluster_sync();
        if (g < p.groups)
            for (uint32_t c = 0; c < (uint32_t)ctas; ++c) {
                const int32_t v = (int32_t)ld_cluster_u32(mapa_shared(smem_u32(mine + g), c));
                if (c < rank) before += v;
                all += v;
            }
    } else if (g < p.groups) {
        all = mine[g];
    }
    // exclusive scan of the groups' totals over the CTA's threads
    int32_t inc = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int32_t v = scan[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
            if (lane >= o) v += u;
        }
        scan[lane] = v;
        if (lane == 31) total_s = v;
    }
    __syncthreads();
    const int32_t first = inc - all + (warp > 0 ? scan[warp - 1] : 0);
    const int32_t total = total_s;
    if (g < p.groups) {
        if (rank == 0) {
            p.offsets[g] = first;
            if (g == p.groups - 1) p.offsets[p.groups] = total;
        }
#pragma unroll 8
        for (int w = 0; w < kRouteWarps; ++w) hist[w * p.groups + g] += first + before;
    }
    __syncthreads();

    auto place = [&](int32_t v, int64_t e) {
        const unsigned peers = __match_any_sync(0xFFFFFFFFu, v);
        int32_t slot = -1;
        if (v >= 0) slot = wh[v] + __popc(peers & ((1u << lane) - 1u));
        __syncwarp();
        if (v >= 0 && lane == __ffs((int)peers) - 1) wh[v] += __popc(peers);
        __syncwarp();
        if (e < e1) {
            p.slots[e] = slot;
            if (slot >= 0) p.rows[slot] = (int32_t)(e / p.top_k);
        }
    };
#pragma unroll
    for (int s = 0; s < kRouteKeep; ++s)
        if (e0 + s * 32 < e1) place(kept[s], e0 + s * 32 + lane);
    for (int64_t e = e0 + kRouteKeep * 32; e < e1; e += 32) place(group_at(e + lane), e + lane);
    // rows behind the last group's
    for (int64_t i = total + (int64_t)rank * kRouteThreads + threadIdx.x; i < p.entries; i += ctas * kRouteThreads)
        p.rows[i] = -1;
    if (ctas > 1) cluster_sync();  // no CTA leaves while another reads its counts
}

template <typename ID>
static sharq_status route_run(LaunchCtx &ctx, const RouteParams &p) {
    const size_t smem = (size_t)(kRouteWarps + 1) * p.groups * sizeof(int32_t);
    SQ_SMEM_ONCE(route_kernel<ID>, (kRouteWarps + 1) * kGroupsMax * sizeof(int32_t));
    int ctas = 1;
    while (ctas < kRouteCluster && p.entries > (int64_t)ctas * kRouteThreads * 2) ctas *= 2;
    return launch_pdl(ctx, route_kernel<ID>, ctas, kRouteThreads, smem, ctas, p);
}

sharq_status launch_route(LaunchCtx &ctx, const void *ids, int id_bytes, int64_t tokens, int64_t top_k, int64_t groups,
                          int32_t *offsets, int32_t *rows, int32_t *slots) {
    RouteParams p{ids, tokens * top_k, (int32_t)top_k, (int32_t)groups, offsets, rows, slots};
    return id_bytes == 8 ? route_run<int64_t>(ctx, p) : route_run<int32_t>(ctx, p);
}

// ---------------------------------------------------------------------------
// Rows into grouped order and back. One CTA per token: the token's own row is
// read (or written) once, its top_k grouped rows are touched with all their
// loads in flight. Rows of the grouped matrix behind the last group's are
// zero in permute's and the gradient's outputs; they are spread over the
// CTAs.
constexpr int kMoveThreads = 256;
constexpr int kMoveJ = 8;  // choices of a token handled at once

struct MoveParams {
    const void *src;           // permute: x; combine and gradient: y
    const void *other;         // combine: residual or NULL; gradient: dout
    const float *weights;      // NULL: 1
    const int32_t *slots, *offsets;
    void *dst;                 // permute: grouped rows; combine: out; gradient: dy
    float *dweights;
    int64_t tokens, n_rows;    // n_rows: rows of the grouped matrix
    int32_t k, top_k, groups;
    unsigned *status;
};

__device__ __forceinline__ int32_t checked_slot(const MoveParams &p, int64_t token, int j) {
    const int32_t s = p.slots[token * p.top_k + j];
    if (s >= p.n_rows) {
        record_status(p.status, kSiteBadSlot);
        return -1;
    }
    return s;
}

template <typename T, int VW>
__device__ __forceinline__ void zero_tail(const MoveParams &p) {
    using V = Vec<T, VW>;
    const int64_t total = max(p.offsets[p.groups], 0);
    for (int64_t r = total + blockIdx.x; r < p.n_rows; r += gridDim.x)
        for (int c = threadIdx.x; c < p.k / VW; c += blockDim.x)
            V::store(static_cast<T *>(p.dst) + r * p.k + (int64_t)c * VW, V::zero());
}

template <typename T, int VW>
__global__ void __launch_bounds__(kMoveThreads) permute_kernel(const MoveParams p) {
    using V = Vec<T, VW>;
    griddep_wait();
    griddep_launch();
    const int64_t token = blockIdx.x;
    if (token < p.tokens) {
        const T *x = static_cast<const T *>(p.src) + token * p.k;
        for (int j0 = 0; j0 < p.top_k; j0 += kMoveJ) {
            int32_t slot[kMoveJ];
#pragma unroll
            for (int j = 0; j < kMoveJ; ++j) slot[j] = j0 + j < p.top_k ? checked_slot(p, token, j0 + j) : -1;
            for (int c = threadIdx.x; c < p.k / VW; c += blockDim.x) {
                const typename V::P v = V::load(x + (int64_t)c * VW);
#pragma unroll
                for (int j = 0; j < kMoveJ; ++j)
                    if (slot[j] >= 0) V::store(static_cast<T *>(p.dst) + (int64_t)slot[j] * p.k + (int64_t)c * VW, v);
            }
        }
    }
    zero_tail<T, VW>(p);
}

template <typename T, int VW>
__global__ void __launch_bounds__(kMoveThreads) combine_kernel(const MoveParams p) {
    using V = Vec<T, VW>;
    griddep_wait();
    griddep_launch();
    const int64_t token = blockIdx.x;
    const T *y = static_cast<const T *>(p.src), *res = static_cast<const T *>(p.other);
    T *out = static_cast<T *>(p.dst) + token * p.k;
    for (int c = threadIdx.x; c < p.k / VW; c += blockDim.x) {
        float acc[VW];
        if (res) {
            V::unpack(V::load(res + token * p.k + (int64_t)c * VW), acc);
        } else {
#pragma unroll
            for (int e = 0; e < VW; ++e) acc[e] = 0.0f;
        }
        for (int j0 = 0; j0 < p.top_k; j0 += kMoveJ) {
            typename V::P v[kMoveJ];
            float w[kMoveJ];
#pragma unroll
            for (int j = 0; j < kMoveJ; ++j) {
                const int32_t s = j0 + j < p.top_k ? checked_slot(p, token, j0 + j) : -1;
                v[j] = s >= 0 ? V::load(y + (int64_t)s * p.k + (int64_t)c * VW) : V::zero();
                w[j] = s >= 0 ? (p.weights ? p.weights[token * p.top_k + j0 + j] : 1.0f) : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < kMoveJ; ++j) {
                float f[VW];
                V::unpack(v[j], f);
#pragma unroll
                for (int e = 0; e < VW; ++e) acc[e] = fmaf(w[j], f[e], acc[e]);
            }
        }
        V::store(out + (int64_t)c * VW, V::pack(acc));
    }
}

template <typename T, int VW>
__global__ void __launch_bounds__(kMoveThreads) combine_bwd_kernel(const MoveParams p) {
    using V = Vec<T, VW>;
    __shared__ float red[kMoveJ][kMoveThreads / 32];
    griddep_wait();
    griddep_launch();
    const int64_t token = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (token < p.tokens) {
        const T *y = static_cast<const T *>(p.src), *dout = static_cast<const T *>(p.other) + token * p.k;
        T *dy = static_cast<T *>(p.dst);
        for (int j0 = 0; j0 < p.top_k; j0 += kMoveJ) {
            int32_t slot[kMoveJ];
            float w[kMoveJ], dot[kMoveJ];
#pragma unroll
            for (int j = 0; j < kMoveJ; ++j) {
                slot[j] = j0 + j < p.top_k ? checked_slot(p, token, j0 + j) : -1;
                w[j] = slot[j] >= 0 ? p.weights[token * p.top_k + j0 + j] : 0.0f;
                dot[j] = 0.0f;
            }
            for (int c = threadIdx.x; c < p.k / VW; c += blockDim.x) {
                const int64_t at = (int64_t)c * VW;
                typename V::P v[kMoveJ];
                float d[VW];
#pragma unroll
                for (int j = 0; j < kMoveJ; ++j)
                    v[j] = slot[j] >= 0 ? V::load(y + (int64_t)slot[j] * p.k + at) : V::zero();
                V::unpack(V::load(dout + at), d);
#pragma unroll
                for (int j = 0; j < kMoveJ; ++j) {
                    if (slot[j] < 0) continue;
                    float f[VW];
                    V::unpack(v[j], f);
#pragma unroll
                    for (int e = 0; e < VW; ++e) dot[j] = fmaf(d[e], f[e], dot[j]);
#pragma unroll
                    for (int e = 0; e < VW; ++e) f[e] = w[j] * d[e];
                    V::store(dy + (int64_t)slot[j] * p.k + at, V::pack(f));
                }
            }
#pragma unroll
            for (int j = 0; j < kMoveJ; ++j) {
                const float s = warp_sum(dot[j]);
                if (lane == 0) red[j][warp] = s;
            }
            __syncthreads();
            if (threadIdx.x < kMoveJ && j0 + (int)threadIdx.x < p.top_k) {
                float s = 0.0f;
                for (int i = 0; i < warps; ++i) s += red[threadIdx.x][i];
                p.dweights[token * p.top_k + j0 + threadIdx.x] = s;
            }
            __syncthreads();
        }
    }
    zero_tail<T, VW>(p);
}

enum class Move { kPermute, kCombine, kCombineBwd };

template <typename T, int VW>
static sharq_status move_run(LaunchCtx &ctx, Move what, const MoveParams &p) {
    int threads = (int)round_up(p.k / VW, 32);
    if (threads > kMoveThreads) threads = kMoveThreads;
    const int64_t grid = p.tokens > 0 ? p.tokens : 1;
    switch (what) {
        case Move::kPermute: return launch_pdl(ctx, permute_kernel<T, VW>, grid, threads, 0, 1, p);
        case Move::kCombine: return launch_pdl(ctx, combine_kernel<T, VW>, grid, threads, 0, 1, p);
        default: return launch_pdl(ctx, combine_bwd_kernel<T, VW>, grid, threads, 0, 1, p);
    }
}

static sharq_status move_any(LaunchCtx &ctx, Move what, int dtype, bool vec16, MoveParams p) {
    p.status = ctx.status;
    if (p.tokens == 0 && (what != Move::kCombineBwd || p.n_rows == 0)) return SHARQ_OK;
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        return vec16 ? move_run<T, 16 / (int)sizeof(T)>(ctx, what, p) : move_run<T, 1>(ctx, what, p);
    });
}

sharq_status launch_permute(LaunchCtx &ctx, const void *x, int64_t tokens, int64_t k, const int32_t *slots, int64_t top_k,
                            const int32_t *offsets, int64_t groups, int dtype, void *out, bool vec16) {
    MoveParams p{};
    p.src = x;
    p.slots = slots;
    p.offsets = offsets;
    p.dst = out;
    p.tokens = tokens;
    p.n_rows = tokens * top_k;
    p.k = (int32_t)k;
    p.top_k = (int32_t)top_k;
    p.groups = (int32_t)groups;
    return move_any(ctx, Move::kPermute, dtype, vec16, p);
}

sharq_status launch_combine(LaunchCtx &ctx, const void *y, int64_t n_rows, int64_t tokens, int64_t k,
                            const int32_t *slots, const float *weights, int64_t top_k, const void *residual, int dtype,
                            void *out, bool vec16) {
    MoveParams p{};
    p.src = y;
    p.other = residual;
    p.weights = weights;
    p.slots = slots;
    p.dst = out;
    p.tokens = tokens;
    p.n_rows = n_rows;
    p.k = (int32_t)k;
    p.top_k = (int32_t)top_k;
    return move_any(ctx, Move::kCombine, dtype, vec16, p);
}

sharq_status launch_combine_backward(LaunchCtx &ctx, const void *dout, const void *y, int64_t n_rows, int64_t tokens,
                                     int64_t k, const int32_t *slots, const float *weights, int64_t top_k,
                                     const int32_t *offsets, int64_t groups, int dtype, void *dy, float *dweights,
                                     bool vec16) {
    MoveParams p{};
    p.src = y;
    p.other = dout;
    p.weights = weights;
    p.slots = slots;
    p.offsets = offsets;
    p.dst = dy;
    p.dweights = dweights;
    p.tokens = tokens;
    p.n_rows = n_rows;
    p.k = (int32_t)k;
    p.top_k = (int32_t)top_k;
    p.groups = (int32_t)groups;
    return move_any(ctx, Move::kCombineBwd, dtype, vec16, p);
}

}  // namespace sq

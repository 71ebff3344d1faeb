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
// of the warps before it. Each warp counts its entries per group (the lanes
// with the same group find each other, one adds), which also gives each entry
// its place among its warp's entries of the group; a scan over warps, CTAs
// (through distributed shared memory) and groups gives the rest of its slot.
// Bound by latency (launch, cluster barriers, one load and one store): 32768
// entries of 128 groups move 0.4 MB.
constexpr int kRouteThreads = 1024;
constexpr int kRouteFew = 256;     // threads where entries and groups are few
constexpr int kRouteCluster = 8;
constexpr int kRouteKeep = 8;      // steps of 32 entries whose groups and places a lane keeps in registers

struct RouteParams {
    const void *ids;
    int64_t entries;
    int32_t top_k, groups;
    int32_t *offsets, *rows, *slots;
};

// Counts per group of a warp in shared memory: an odd row stride spreads the
// 8 x 4 reads of the scan over all banks.
__host__ __device__ __forceinline__ int route_stride(int groups) { return groups | 1; }

// The lanes with my value (below 2^bits): a ballot per bit. A match
// instruction does the same, but one SM gets through about one in 120 cycles
// (2 us more for 32768 entries, which take 8 like this).
__device__ __forceinline__ unsigned peers_of(int32_t v, int bits) {
    unsigned peers = 0xFFFFFFFFu;
    for (int b = 0; b < bits; ++b) {
        const bool one = (v >> b) & 1;
        const unsigned with = __ballot_sync(0xFFFFFFFFu, one);
        peers &= one ? with : ~with;
    }
    return peers;
}

// LONG: runs of more than kRouteKeep * 32 entries; a second walk over them
// then hands the slots out.
template <typename ID, bool LONG>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteParams p) {
    extern __shared__ int32_t sm[];
    __shared__ int32_t scan[32];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = threadIdx.x;
    const int stride = route_stride(p.groups), bits = 32 - __clz(p.groups);
    int32_t *hist = sm;                        // [warps][stride]
    int32_t *mine = sm + warps * stride;       // [groups] entries of this CTA
    int32_t *base = mine + p.groups;           // [groups] first slot of this CTA's entries
    for (int i = threadIdx.x; i < warps * stride; i += blockDim.x) hist[i] = 0;
    griddep_wait();
    griddep_launch();
    const uint32_t rank = cluster_ctarank();
    const int ctas = (int)gridDim.x;
    // at most 2^30 entries: 32-bit arithmetic
    const uint32_t run = (((uint32_t)p.entries + ctas * warps - 1) / (uint32_t)(ctas * warps) + 31) / 32 * 32;
    const int32_t e0 = (int32_t)min((int64_t)(rank * warps + warp) * run, p.entries);
    const int32_t e1 = (int32_t)min((int64_t)e0 + run, p.entries);
    const ID *ids = static_cast<const ID *>(p.ids);
    int32_t *wh = hist + warp * stride;

    auto group_at = [&](int32_t e) -> int32_t {
        if (e >= e1) return -1;
        const ID v = ids[e];
        return v >= 0 && v < (ID)p.groups ? (int32_t)v : -1;
    };
    // The entry's place among the warp's entries of its group so far; adds
    // the step's entries to the counts in wh.
    auto count = [&](int32_t v) -> int32_t {
        const unsigned peers = peers_of(v < 0 ? p.groups : v, bits);
        const int32_t before = v >= 0 ? wh[v] : 0;
        __syncwarp();
        if (v >= 0 && lane == __ffs((int)peers) - 1) wh[v] = before + __popc(peers);
        __syncwarp();
        return before + __popc(peers & ((1u << lane) - 1u));
    };
    int32_t kept[kRouteKeep], place[kRouteKeep];
#pragma unroll
    for (int s = 0; s < kRouteKeep; ++s) kept[s] = group_at(e0 + s * 32 + lane);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kRouteKeep; ++s) place[s] = e0 + s * 32 < e1 ? count(kept[s]) : 0;
    if (LONG)
        for (int32_t e = e0 + kRouteKeep * 32; e < e1; e += 32) count(group_at(e + lane));
    __syncthreads();

    // scan over the warps: 8 lanes per group, 4 warps each
    const int sub = threadIdx.x & 7;
    for (int h = threadIdx.x >> 3; h < (p.groups + 3) / 4 * 4; h += blockDim.x >> 3) {  // 4 groups of a warp together
        int32_t c[4], sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = h < p.groups && 4 * sub + i < warps ? hist[(4 * sub + i) * stride + h] : 0;
            sum += c[i];
        }
        int32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o, 8);
            if (sub >= o) inc += v;
        }
        int32_t at = inc - sum;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (h < p.groups && 4 * sub + i < warps) hist[(4 * sub + i) * stride + h] = at;
            at += c[i];
        }
        if (sub == 7 && h < p.groups) mine[h] = inc;
    }
    int32_t before = 0, all = 0;
    if (ctas > 1) {
        cluster_sync();
        if (g < p.groups) {
            const uint32_t at = smem_u32(mine + g);
#pragma unroll
            for (int c = 0; c < kRouteCluster; ++c) {
                const int32_t v = c < ctas ? (int32_t)ld_cluster_u32(mapa_shared(at, (uint32_t)c)) : 0;
                if (c < (int)rank) before += v;
                all += v;
            }
        }
    } else {
        __syncthreads();
        if (g < p.groups) all = mine[g];
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
    int32_t v = lane < warps ? scan[lane] : 0;  // every warp scans the warps' totals for itself
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
    }
    const int32_t total = __shfl_sync(0xFFFFFFFFu, v, 31);
    const int32_t ahead = __shfl_sync(0xFFFFFFFFu, v, warp > 0 ? warp - 1 : 0);
    const int32_t first = inc - all + (warp > 0 ? ahead : 0);
    if (g < p.groups) {
        if (rank == 0) {
            p.offsets[g] = first;
            if (g == p.groups - 1) p.offsets[p.groups] = total;
        }
        base[g] = first + before;
    }
    __syncthreads();
    if (ctas > 1) cluster_arrive_relaxed();  // this CTA has used what it read of the others' counts

    auto put = [&](int32_t v, int32_t e, int32_t slot) {
        if (e < e1) {
            p.slots[e] = v >= 0 ? slot : -1;
            if (v >= 0) p.rows[slot] = (int32_t)((uint32_t)e / (uint32_t)p.top_k);
        }
    };
#pragma unroll
    for (int s = 0; s < kRouteKeep; ++s)
        if (e0 + s * 32 < e1)
            put(kept[s], e0 + s * 32 + lane, kept[s] >= 0 ? base[kept[s]] + wh[kept[s]] + place[s] : 0);
    if (LONG && e0 < e1) {
        // the kept entries' part of the counts comes first
        __syncwarp();
#pragma unroll
        for (int s = 0; s < kRouteKeep; ++s)
            if (e0 + s * 32 < e1) count(kept[s]);
        for (int32_t e = e0 + kRouteKeep * 32; e < e1; e += 32) {
            const int32_t v = group_at(e + lane);
            const int32_t at = count(v);
            put(v, e + lane, v >= 0 ? base[v] + at : 0);
        }
    }
    // rows behind the last group's
    for (int64_t i = total + (int64_t)rank * blockDim.x + threadIdx.x; i < p.entries; i += (int64_t)ctas * blockDim.x)
        p.rows[i] = -1;
    if (ctas > 1) cluster_wait();  // no CTA leaves while another reads its counts
}

template <typename ID, bool LONG>
static sharq_status route_run(LaunchCtx &ctx, const RouteParams &p, int ctas, int threads) {
    auto bytes = [](int warps, int groups) { return (size_t)(warps * route_stride(groups) + 2 * groups) * sizeof(int32_t); };
    SQ_SMEM_ONCE((route_kernel<ID, LONG>), bytes(kRouteThreads / 32, (int)kGroupsMax));
    return launch_pdl(ctx, route_kernel<ID, LONG>, ctas, threads, bytes(threads / 32, p.groups), ctas, p);
}

template <typename ID>
static sharq_status route_any(LaunchCtx &ctx, const RouteParams &p) {
    const int threads = p.entries <= 4 * kRouteFew && p.groups <= kRouteFew ? kRouteFew : kRouteThreads;
    int ctas = 1;
    while (ctas < kRouteCluster && p.entries > (int64_t)ctas * threads * 2) ctas *= 2;
    return p.entries > (int64_t)ctas * threads * kRouteKeep ? route_run<ID, true>(ctx, p, ctas, threads)
                                                            : route_run<ID, false>(ctx, p, ctas, threads);
}

sharq_status launch_route(LaunchCtx &ctx, const void *ids, int id_bytes, int64_t tokens, int64_t top_k, int64_t groups,
                          int32_t *offsets, int32_t *rows, int32_t *slots) {
    RouteParams p{ids, tokens * top_k, (int32_t)top_k, (int32_t)groups, offsets, rows, slots};
    return id_bytes == 8 ? route_any<int64_t>(ctx, p) : route_any<int32_t>(ctx, p);
}

// ---------------------------------------------------------------------------
// Rows into grouped order and back. Some threads (whole warps) per token: the
// token's own row is read (or written) once, its top_k grouped rows are touched
// with several loads of a thread in flight (choices times vectors of the row).
// A CTA takes as many tokens as fit. Rows of the grouped matrix behind the last
// group's are zero in permute's and the gradient's outputs; they are spread
// over the CTAs.
constexpr int kMoveThreads = 256;

struct MoveParams {
    const void *src;           // permute: x; combine and gradient: y
    const void *other;         // combine: residual or NULL; gradient: dout
    const float *weights;      // NULL: 1
    const int32_t *slots, *offsets;
    void *dst;                 // permute: grouped rows; combine: out; gradient: dy
    float *dweights;
    int64_t tokens, n_rows;    // n_rows: rows of the grouped matrix
    int32_t k, top_k, groups;
    int32_t lanes;             // threads of a token
    unsigned *status;
};

// Slots of a token's choices j0 .. j0 + J - 1 and their weights (-1 and 0: none),
// all loads in flight at once. A slot past the grouped matrix counts as none;
// returns whether there was one (reported once the row's loads are under way:
// an atomic in between would hold them back).
template <int J>
__device__ __forceinline__ bool choices_of(const MoveParams &p, int64_t token, int j0, bool live, int32_t (&slot)[J],
                                           float (&w)[J]) {
    bool bad = false;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const bool in = live && j0 + j < p.top_k;
        slot[j] = in ? p.slots[token * p.top_k + j0 + j] : -1;
        w[j] = in ? (p.weights ? p.weights[token * p.top_k + j0 + j] : 1.0f) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const bool past = slot[j] >= (int32_t)p.n_rows;
        bad |= past;
        if (past) slot[j] = -1;
        if (slot[j] < 0) w[j] = 0.0f;
    }
    return bad;
}

template <typename T, int VW>
__device__ __forceinline__ void zero_tail(const MoveParams &p) {
    using V = Vec<T, VW>;
    const int64_t total = max(p.offsets[p.groups], 0);
    for (int64_t r = total + blockIdx.x; r < p.n_rows; r += gridDim.x)
        for (int c = threadIdx.x; c < p.k / VW; c += blockDim.x)
            V::store(static_cast<T *>(p.dst) + r * p.k + (int64_t)c * VW, V::zero());
}

// The row's vectors are walked U at a time; choices J at a time.
template <typename T, int VW, int U>
__global__ void __launch_bounds__(kMoveThreads) permute_kernel(const MoveParams p) {
    using V = Vec<T, VW>;
    constexpr int J = 8;
    griddep_wait();
    griddep_launch();
    const int64_t token = (int64_t)blockIdx.x * (blockDim.x / p.lanes) + threadIdx.x / p.lanes;
    const int sub = threadIdx.x % p.lanes, nvec = p.k / VW;
    if (token < p.tokens) {
        const T *x = static_cast<const T *>(p.src) + token * p.k;
        for (int j0 = 0; j0 < p.top_k; j0 += J) {
            int32_t slot[J];
            float w[J];
            const bool bad = choices_of<J>(p, token, j0, true, slot, w);
            for (int c0 = sub; c0 < nvec; c0 += U * p.lanes) {
                typename V::P v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + u * p.lanes;
                    v[u] = c < nvec ? V::load(x + (int64_t)c * VW) : V::zero();
                }
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    if (slot[j] < 0) continue;
                    T *dst = static_cast<T *>(p.dst) + (int64_t)slot[j] * p.k;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int c = c0 + u * p.lanes;
                        if (c < nvec) V::store(dst + (int64_t)c * VW, v[u]);
                    }
                }
            }
            if (bad) record_status(p.status, kSiteBadSlot);
        }
    }
    zero_tail<T, VW>(p);
}

// A vector as packed pairs of binary32 (VW even), or its value in the first of
// a pair; acc += w v on them.
template <typename T, int VW>
__device__ __forceinline__ void widen_pairs(typename Vec<T, VW>::P v, uint64_t (&f)[(VW + 1) / 2]) {
    if constexpr (VW > 1) {
        Vec<T, VW>::unpack2(v, f);
    } else {
        float t[VW];
        Vec<T, VW>::unpack(v, t);
        f[0] = pk2(t[0], 0.0f);
    }
}
template <typename T, int VW>
__device__ __forceinline__ void add_scaled(uint64_t (&acc)[(VW + 1) / 2], float w, typename Vec<T, VW>::P v) {
    uint64_t f[(VW + 1) / 2];
    widen_pairs<T, VW>(v, f);
    const uint64_t w2 = pk2(w, w);
#pragma unroll
    for (int e = 0; e < (VW + 1) / 2; ++e) acc[e] = fma2(w2, f[e], acc[e]);
}

// MORE: top_k > J, the choices in turns of J. Four CTAs per SM: left to itself the
// compiler takes fewer registers and waits for its loads one by one (35.7 us
// against 29.9 for 4096 x 8 rows of 2048 in fp16).
template <typename T, int VW, int J, int U, bool MORE>
__global__ void __launch_bounds__(kMoveThreads, 4) combine_kernel(const MoveParams p) {
    using V = Vec<T, VW>;
    griddep_wait();
    griddep_launch();
    const int64_t token = (int64_t)blockIdx.x * (blockDim.x / p.lanes) + threadIdx.x / p.lanes;
    const int sub = threadIdx.x % p.lanes, nvec = p.k / VW;
    if (token >= p.tokens) return;
    const T *y = static_cast<const T *>(p.src), *res = static_cast<const T *>(p.other);
    T *out = static_cast<T *>(p.dst) + token * p.k;
    bool bad = false;
    for (int c0 = sub; c0 < nvec; c0 += U * p.lanes) {
        uint64_t acc[U][(VW + 1) / 2];
        auto residual = [&](int u) {
            const int c = c0 + u * p.lanes;
            return res && c < nvec ? V::load(res + token * p.k + (int64_t)c * VW) : V::zero();
        };
        // 16 bits: the residual after the slots, or these wait for it (33.2 us against
        // 29.9 for the case above); 32 bits, where nothing is widened, the other way
        // round (17.7 against 15.5 for 2048 x 4096, one choice)
        constexpr bool kFirst = sizeof(T) == 4;
        if (kFirst)
#pragma unroll
            for (int u = 0; u < U; ++u) widen_pairs<T, VW>(residual(u), acc[u]);
        int j0 = 0;
        do {
            typename V::P v[U][J], rv[U];
            int32_t slot[J];
            float w[J];
            bad |= choices_of<J>(p, token, j0, true, slot, w);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!kFirst) rv[u] = j0 == 0 ? residual(u) : V::zero();
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int c = c0 + u * p.lanes;
                    v[u][j] = slot[j] >= 0 && c < nvec ? V::load(y + (int64_t)slot[j] * p.k + (int64_t)c * VW) : V::zero();
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!kFirst && j0 == 0) widen_pairs<T, VW>(rv[u], acc[u]);
#pragma unroll
                for (int j = 0; j < J; ++j) add_scaled<T, VW>(acc[u], w[j], v[u][j]);
            }
            j0 += J;
        } while (MORE && j0 < p.top_k);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * p.lanes;
            if (c >= nvec) continue;
            if constexpr (VW > 1) {
                V::store(out + (int64_t)c * VW, V::pack2(acc[u]));
            } else {
                const float f[VW] = {up2(acc[u][0]).x};
                V::store(out + (int64_t)c * VW, V::pack(f));
            }
        }
    }
    if (bad) record_status(p.status, kSiteBadSlot);
}

// At most four choices at a time keep a thread within 64 registers, so that
// four CTAs (32 warps) of an SM overlap their loads, sums and stores: 61 us with
// eight at a time and two CTAs, 48 us like this (32768 rows of 2048, bf16).
template <typename T, int VW, int J, int U>
__global__ void __launch_bounds__(kMoveThreads, 4) combine_bwd_kernel(const MoveParams p) {
    using V = Vec<T, VW>;
    __shared__ float red[2][J][kMoveThreads / 32];
    griddep_wait();
    griddep_launch();
    const int64_t token = (int64_t)blockIdx.x * (blockDim.x / p.lanes) + threadIdx.x / p.lanes;
    const int sub = threadIdx.x % p.lanes, nvec = p.k / VW;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int warps = p.lanes >> 5, warp0 = (int)threadIdx.x / p.lanes * warps;  // of this token
    const bool live = token < p.tokens;
    const T *y = static_cast<const T *>(p.src), *dout = static_cast<const T *>(p.other) + (live ? token : 0) * p.k;
    T *dy = static_cast<T *>(p.dst);
    for (int j0 = 0, parity = 0; p.tokens > 0 && j0 < p.top_k; j0 += J, parity ^= 1) {
        int32_t slot[J];
        float w[J], dot[J];
        const bool bad = choices_of<J>(p, token, j0, live, slot, w);
#pragma unroll
        for (int j = 0; j < J; ++j) dot[j] = 0.0f;
        for (int c0 = sub; c0 < nvec; c0 += U * p.lanes) {
            typename V::P v[U][J], dv[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * p.lanes;
#pragma unroll
                for (int j = 0; j < J; ++j)
                    v[u][j] = slot[j] >= 0 && c < nvec ? V::load(y + (int64_t)slot[j] * p.k + (int64_t)c * VW) : V::zero();
                dv[u] = c < nvec ? V::load(dout + (int64_t)c * VW) : V::zero();
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * p.lanes;
                if (c >= nvec) continue;
                const int64_t at = (int64_t)c * VW;
                if constexpr (VW > 1) {
                    uint64_t d[VW / 2];
                    V::unpack2(dv[u], d);
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        if (slot[j] < 0) continue;
                        uint64_t f[VW / 2], sum = 0;
                        V::unpack2(v[u][j], f);
#pragma unroll
                        for (int e = 0; e < VW / 2; ++e) sum = fma2(d[e], f[e], sum);
                        const float2 t = up2(sum);
                        dot[j] += t.x + t.y;
                        const uint64_t w2 = pk2(w[j], w[j]);
#pragma unroll
                        for (int e = 0; e < VW / 2; ++e) f[e] = mul2(w2, d[e]);
                        V::store(dy + (int64_t)slot[j] * p.k + at, V::pack2(f));
                    }
                } else {
                    float d[VW];
                    V::unpack(dv[u], d);
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        if (slot[j] < 0) continue;
                        float f[VW];
                        V::unpack(v[u][j], f);
                        dot[j] = fmaf(d[0], f[0], dot[j]);
                        f[0] = w[j] * d[0];
                        V::store(dy + (int64_t)slot[j] * p.k + at, V::pack(f));
                    }
                }
            }
        }
        // The warp's sums: lanes 32 / J * q and on go on with the q-th.
        float s;
        if constexpr (J == 4) {
            const bool hi = lane & 16, odd = lane & 8;
            const float a = (hi ? dot[2] : dot[0]) + __shfl_xor_sync(0xFFFFFFFFu, hi ? dot[0] : dot[2], 16);
            const float b = (hi ? dot[3] : dot[1]) + __shfl_xor_sync(0xFFFFFFFFu, hi ? dot[1] : dot[3], 16);
            s = (odd ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 8);
        } else if constexpr (J == 2) {
            const bool hi = lane & 16;
            s = (hi ? dot[1] : dot[0]) + __shfl_xor_sync(0xFFFFFFFFu, hi ? dot[0] : dot[1], 16);
        } else {
            s = dot[0];
        }
#pragma unroll
        for (int o = 16 / J; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (lane % (32 / J) == 0) red[parity][lane / (32 / J)][warp] = s;
        __syncthreads();
        if (live && sub < J && j0 + sub < p.top_k) {
            float t = 0.0f;
            for (int i = 0; i < warps; ++i) t += red[parity][sub][warp0 + i];
            p.dweights[token * p.top_k + j0 + sub] = t;
        }
        if (bad) record_status(p.status, kSiteBadSlot);
    }
    zero_tail<T, VW>(p);
}

enum class Move { kPermute, kCombine, kCombineBwd };

// Threads of a token so that each has about U vectors of its row: whole warps,
// a power of two of them, at most a CTA.
static int move_lanes(int nvec, int u) {
    int l = 32;
    while (l < kMoveThreads && l * u < nvec) l *= 2;
    return l;
}

template <typename T, int VW>
static sharq_status move_run(LaunchCtx &ctx, Move what, MoveParams p) {
    const int nvec = p.k / VW;
    auto run = [&](auto kernel, int u) {
        p.lanes = move_lanes(nvec, u);
        const int64_t per = kMoveThreads / p.lanes, grid = p.tokens > 0 ? (p.tokens + per - 1) / per : 1;
        return launch_pdl(ctx, kernel, grid, kMoveThreads, 0, 1, p);
    };
    switch (what) {
        case Move::kPermute: return p.top_k <= 2 ? run(permute_kernel<T, VW, 4>, 4) : run(permute_kernel<T, VW, 1>, 1);
        case Move::kCombine:
            return p.top_k == 1   ? run(combine_kernel<T, VW, 1, 2, false>, 2)
                   : p.top_k == 2 ? run(combine_kernel<T, VW, 2, 2, false>, 2)
                   : p.top_k <= 4 ? run(combine_kernel<T, VW, 4, 1, false>, 1)
                   : p.top_k <= 8 ? run(combine_kernel<T, VW, 8, 1, false>, 1) : run(combine_kernel<T, VW, 8, 1, true>, 1);
        default:
            return p.top_k == 1   ? run(combine_bwd_kernel<T, VW, 1, 4>, 4)
                   : p.top_k == 2 ? run(combine_bwd_kernel<T, VW, 2, 2>, 2) : run(combine_bwd_kernel<T, VW, 4, 1>, 1);
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

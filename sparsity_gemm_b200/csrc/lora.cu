// Low-rank adapters of many requests beside a shared projection.
//
//   out[row] = base[row] + scale[g] * (x[row] A[g]^T) B[g]^T,  g the row's group
//
// with A [groups][rank][k] and B [groups][n][rank]; rows come sorted by group
// (offsets, rows: the output of sharq_route), rows without a group keep base.
//
// One launch does both products. A cluster takes a tile of rows of one group:
// its CTAs split k for h = x A^T, add their parts through distributed shared
// memory, and then split the columns for out = base + scale h B^T. So x, base
// and out cross HBM once, h never leaves the SMs, and A and B are read once
// per tile (from L2 after the first).
//
// Both products are memory-bound (2 rank operations per 2-byte element of x),
// so the operands go from global memory straight into the registers of
// m16n8k16 tensor-core instructions. A dot product may take its terms in any
// order as long as both operands agree, so a lane loads 8 consecutive
// elements (16 bytes) of its row and uses them where the instruction expects
// elements 2q, 2q+1, 2q+8, 2q+9 of two steps; the columns of the second
// product are permuted the same way, so that a lane's results are 8
// consecutive columns.
//
// h is binary32. For the second product each row is scaled by a power of two
// and split into 16-bit terms, each the rounded rest of those before it. Three
// bf16 terms hold all 24 bits of a value. Two fp16 terms hold 23 (within 2^-23
// of the value; of values below 2^-16 of the row's largest, within 2^-39 of that
// largest): a third would add a half to the second product's instructions for
// one bit, far below what the sums of both products round away.
#include <cuda_runtime.h>

#include "sharq_dev.cuh"
#include "sq_internal.h"
#include "vec.cuh"

namespace sq {

constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;

struct LoraParams {
    const void *x, *a, *b, *base;
    const float *scales;
    void *out;
    const int32_t *offsets, *rows, *slots;
    int32_t ldx, ldbase, ldo;
    int64_t m;
    int32_t k, n, rank, groups;
    int32_t nsplit;     // one launch: clusters that share a tile, each with its part of the columns
    int32_t bare_ctas;  // CTAs, the grid's first, that copy rows without a group
    unsigned *status;
    uint64_t wait_ns;
    float *part;          // two-launch form: the parts of h, [part][128 rows][padded rank]
    int32_t shrink_ctas;  // and the CTAs that make them
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, __half) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, __nv_bfloat16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with nothing to add to.
template <typename T>
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    const float z = 0.0f;
    if constexpr (IsBf16<T>::v)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z));
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) { return __uint_as_float(ld_cluster_u32(addr)); }

// The terms of h, and the power of two that the row's largest value is brought
// to: near fp16's largest, so that the second terms of small values stay above
// its smallest (bf16 has binary32's range).
template <typename T>
constexpr int kTerms = IsBf16<T>::v ? 3 : 2;
template <typename T>
constexpr int kTopExponent = IsBf16<T>::v ? 0 : 14;

// The magnitude of a value as far as it counts for its row's scale.
__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a <= 3.4028235e38f ? a : 0.0f;
}

// The exponent of the power of two that a row is divided by; top: its largest
// finite magnitude.
template <typename T>
__device__ __forceinline__ int row_exponent(float top) {
    const int e = (int)(__float_as_uint(top) >> 23) - 127 - kTopExponent<T>;
    return e < -100 ? -100 : e > 126 ? 126 : e;
}

// An infinity or a NaN is its first term, with nothing left for the others.
template <typename T>
__device__ __forceinline__ void split_terms(float v, T (&t)[kTerms<T>]) {
#pragma unroll
    for (int z = 0; z < kTerms<T>; ++z) {
        t[z] = narrow<T>(v);
        v -= widen(t[z]);  // exact
        if (v != v) v = 0.0f;
    }
}

// The tile's group and rows, found by warp 0 in the offsets. tile_s: [0] group
// (-1: no such tile, -2: bad offsets), [1] first grouped row, [2] rows.
__device__ __forceinline__ void find_tile(const int32_t *off, int groups, int64_t m, int tile_rows, int tile,
                                          int32_t *tile_s) {
    const int lane = threadIdx.x & 31;
    bool ok = off[0] == 0 && off[groups] <= m;
    int32_t carry = 0, group = -1, first = 0;
    for (int base = 0; base < groups; base += 32) {
        const int g = base + lane;
        int32_t t = 0, a = 0;
        if (g < groups) {
            a = off[g];
            const int32_t b = off[g + 1];
            if (b < a || a < 0 || b > m) ok = false;
            else t = (b - a + tile_rows - 1) / tile_rows;
        }
        int32_t inc = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += v;
        }
        const int32_t at = tile - (carry + inc - t);  // the tile's place in my group
        const bool here = at >= 0 && at < t;
        const unsigned who = __ballot_sync(0xFFFFFFFFu, here);
        if (who) {
            const int src = __ffs((int)who) - 1;
            group = base + src;
            first = __shfl_sync(0xFFFFFFFFu, a + at * tile_rows, src);
        }
        carry += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (lane == 0) {
        tile_s[0] = ok ? group : -2;
        tile_s[1] = first;
        tile_s[2] = ok && group >= 0 ? min(tile_rows, off[group + 1] - first) : 0;
    }
}

// First tile of every group, tiles[groups] their number, by one warp from the
// offsets in shared memory. Returns, in every lane, whether these are valid.
__device__ __forceinline__ bool build_tiles(const int32_t *off, int groups, int64_t m, int tile_rows, int32_t *tiles) {
    const int lane = threadIdx.x & 31;
    bool ok = off[0] == 0 && off[groups] <= m;
    int32_t carry = 0;
    if (lane == 0) tiles[0] = 0;
    for (int base = 0; base < groups; base += 32) {
        const int g = base + lane;
        int32_t t = 0;
        if (g < groups) {
            const int32_t a = off[g], b = off[g + 1];
            if (b < a || a < 0 || b > m) ok = false;
            else t = (b - a + tile_rows - 1) / tile_rows;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xFFFFFFFFu, t, o);
            if (lane >= o) t += v;
        }
        if (g < groups) tiles[g + 1] = carry + t;
        carry += __shfl_sync(0xFFFFFFFFu, t, 31);
    }
    return __all_sync(0xFFFFFFFFu, ok);
}

// find_tile for the whole CTA. Up to 32 groups are read by their lanes; more go
// through shared memory (off), so that they are all in flight at once.
__device__ __forceinline__ void cta_find_tile(const LoraParams &p, int32_t *off, int tile_rows, int tile, int32_t *tile_s) {
    const int32_t *from = p.offsets;
    if (p.groups > 32) {
        for (int i = threadIdx.x; i <= p.groups; i += blockDim.x) off[i] = p.offsets[i];
        __syncthreads();
        from = off;
    }
    if (threadIdx.x < 32) find_tile(from, p.groups, p.m, tile_rows, tile, tile_s);
    __syncthreads();
}

// out = base + scale h B^T for the tile's rows, over the blocks c0 .. c1-1 of 32
// columns; warps take turns. terms: those of h, term_ld elements apart.
// A lane reads base for the very elements it writes, so the next blocks' are on
// their way into `ahead` (written and read by that thread alone) while a block
// is computed; B's part of the next block is on its way into registers. ready()
// runs after the first of these loads and before h is read.
constexpr int kAhead = 2;

// Row stride of a term of h: a lane of a quarter-warp reads 16 bytes of
// one of two rows, 64 bytes of each (rank up to 16: a half-warp 8 bytes of one of
// four rows), and these fill the 32 banks.
template <int NB>
constexpr int kHLd = NB == 2 ? 16 : NB == 4 ? 32 : 8 * NB + 32;

template <int MT>
constexpr int kAheadBytes = kAhead * 2 * MT * 16 * kLoraThreads;

template <typename T, int MT, int NB, typename F>
__device__ __forceinline__ void expand_tile(const LoraParams &p, int group, const int32_t *row_s, const float *scale_s,
                                            const uint16_t *terms, int term_ld, uint8_t *ahead, int c0, int c1,
                                            F ready) {
    constexpr int kLd = kHLd<NB>, kS = (NB + 3) / 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, q = lane & 3;
    const T *b = static_cast<const T *>(p.b) + (int64_t)group * p.n * p.rank;
    const T *base = static_cast<const T *>(p.base);
    T *out = static_cast<T *>(p.out);
    uint4 *mine = reinterpret_cast<uint4 *>(ahead) + threadIdx.x;
    int32_t row[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) row[i][h] = row_s[16 * i + 8 * h + g8];
    const uint32_t slots = smem_u32(mine);
    auto fetch = [&](int c, int s) {
        const int col = 32 * c + 8 * q;
        if (base && c < c1 && col < p.n) {
            const T *at = base + col;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (row[i][h] >= 0)
                        cp_async16(slots + (uint32_t)(((s * MT + i) * 2 + h) * kLoraThreads * 16),
                                   at + (int64_t)row[i][h] * p.ldbase);
        }
        cp_async_commit();
    };
    // this lane's rows of B in a block of 32: bl + 2 j; 8 of them end inside n or not at all
    const int bl = 8 * (g8 >> 1) + (g8 & 1);
    const T *b_lane = b + (int64_t)bl * p.rank + (NB == 2 ? 4 : 8) * q;
    auto fetch_b = [&](int c, uint4 (&v)[4][kS]) {
        const bool in = c < c1 && 32 * c + bl < p.n;
        const T *at = b_lane + (int64_t)c * (32 * p.rank);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int s = 0; s < kS; ++s) {
                v[j][s] = make_uint4(0, 0, 0, 0);
                if (NB == 2) {  // one step of 16
                    if (in && 4 * q < p.rank) {
                        const uint2 w = load_as<uint2>(at + 2 * j * p.rank);
                        v[j][s].x = w.x;
                        v[j][s].y = w.y;
                    }
                } else if (in && 32 * s + 8 * q < p.rank) {
                    v[j][s] = load_as<uint4>(at + 2 * j * p.rank + 32 * s);
                }
            }
        }
    };
#pragma unroll
    for (int s = 0; s < kAhead - 1; ++s) fetch(c0 + warp + s * kLoraWarps, s);
    constexpr bool kNextB = NB == 2 || (MT == 1 && NB <= 8);  // more does not fit in registers
    uint4 bv[4][kS], bn[4][kS];
    if (kNextB) fetch_b(c0 + warp, bn);
    ready();
    int slot = 0;
    for (int c = c0 + warp; c < c1; c += kLoraWarps) {
        const int col = 32 * c + 8 * q;
        if (kNextB) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int s = 0; s < kS; ++s) bv[j][s] = bn[j][s];
            fetch_b(c + kLoraWarps, bn);
        } else {
            fetch_b(c, bv);
        }
        fetch(c + (kAhead - 1) * kLoraWarps, slot == 0 ? kAhead - 1 : slot - 1);
        cp_async_wait<kAhead - 1>();
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            float d[4][4];
#pragma unroll
            for (int z = 0; z < kTerms<T>; ++z) {
                const uint16_t *hp = terms + z * term_ld + (16 * i + g8) * kLd;
#pragma unroll
                for (int s = 0; s < kS; ++s) {
                    if (NB == 2) {
                        const uint2 h0 = *reinterpret_cast<const uint2 *>(hp + 4 * q);
                        const uint2 h1 = *reinterpret_cast<const uint2 *>(hp + 8 * kLd + 4 * q);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (z == 0) mma16816_zero<T>(d[j], h0.x, h1.x, h0.y, h1.y, bv[j][s].x, bv[j][s].y);
                            else mma16816(d[j], h0.x, h1.x, h0.y, h1.y, bv[j][s].x, bv[j][s].y, T());
                        }
                    } else {
                        const uint4 h0 = *reinterpret_cast<const uint4 *>(hp + 32 * s + 8 * q);
                        const uint4 h1 = *reinterpret_cast<const uint4 *>(hp + 8 * kLd + 32 * s + 8 * q);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (z == 0 && s == 0) mma16816_zero<T>(d[j], h0.x, h1.x, h0.y, h1.y, bv[j][s].x, bv[j][s].y);
                            else mma16816(d[j], h0.x, h1.x, h0.y, h1.y, bv[j][s].x, bv[j][s].y, T());
                            mma16816(d[j], h0.z, h1.z, h0.w, h1.w, bv[j][s].z, bv[j][s].w, T());
                        }
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (row[i][h] >= 0 && col < p.n) {
                    const float sc = scale_s[16 * i + 8 * h + g8];
                    const uint64_t sc2 = pk2(sc, sc);
                    uint64_t f[4];
                    Vec<T, 8>::unpack2(base ? mine[((slot * MT + i) * 2 + h) * kLoraThreads] : make_uint4(0, 0, 0, 0), f);
#pragma unroll
                    for (int j = 0; j < 4; ++j) f[j] = fma2(sc2, pk2(d[j][2 * h], d[j][2 * h + 1]), f[j]);
                    *reinterpret_cast<uint4 *>(out + col + (int64_t)row[i][h] * p.ldo) = Vec<T, 8>::pack2(f);
                }
            }
        }
        slot = slot + 1 == kAhead ? 0 : slot + 1;
    }
    cp_async_wait<0>();
}

// Rows without a group: base (or zero), unless they are there already; the
// grid's first p.bare_ctas CTAs do it, a row per warp. Such rows come in runs (a
// request's rows), so the warps take rows in turn; a warp looks at 32 of its
// rows at a time.
template <typename T>
__device__ __forceinline__ void copy_bare_rows(const LoraParams &p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)p.bare_ctas * kLoraWarps, me = (int64_t)blockIdx.x * kLoraWarps + warp;
    for (int64_t i = 0; i * warps + me < p.m; i += 32) {
        const int64_t look = (i + lane) * warps + me;
        unsigned left = __ballot_sync(0xFFFFFFFFu, look < p.m && p.slots[look] < 0);
        for (; left; left &= left - 1) {
            const int64_t r = (i + __ffs((int)left) - 1) * warps + me;
            const T *src = static_cast<const T *>(p.base) + r * p.ldbase;
            T *dst = static_cast<T *>(p.out) + r * p.ldo;
            for (int c0 = 8 * lane; c0 < p.n; c0 += 8 * 256) {  // 8 loads in flight
                uint4 v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[j] = make_uint4(0, 0, 0, 0);
                    if (p.base && c0 + 256 * j < p.n) v[j] = load_as<uint4>(src + c0 + 256 * j);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c0 + 256 * j < p.n) *reinterpret_cast<uint4 *>(dst + c0 + 256 * j) = v[j];
            }
        }
    }
}

// CTAs for that: none where the rows are in place, else a warp per row up to
// one CTA per SM.
static int bare_ctas(const LaunchCtx &ctx, const LoraParams &p) {
    if (p.base == p.out) return 0;
    const int64_t n = (p.m + kLoraWarps - 1) / kLoraWarps;
    return (int)(n < ctx.num_sms ? n : ctx.num_sms);
}

// NB: 8-column blocks of the padded rank.
constexpr int kLoraCluster = 8;  // most CTAs of a tile
template <typename T, int NB>
struct LoraCfg {
    static constexpr int kRows = 16, kRank = 8 * NB;
    static constexpr int kLd = kRank + 8;   // row stride of the binary32 parts
    static constexpr int kTermLd = kRows * kHLd<NB>;
    static constexpr int kSmem = kLoraWarps * kRows * kLd * 4 + kTerms<T> * kTermLd * 2 + kAheadBytes<1>;
    static constexpr int kPerSm = NB == 2 ? 3 : NB <= 8 ? 2 : 1;  // CTAs on an SM, by registers
    static constexpr int kStep = NB >= 8 ? 1 : 2;  // steps of 32 elements of k in flight
};

template <typename T, int NB, int PER_SM>
__global__ void __launch_bounds__(kLoraThreads, PER_SM) lora_kernel(const LoraParams p) {
    using C = LoraCfg<T, NB>;
    extern __shared__ __align__(16) uint8_t smem[];
    float *part = reinterpret_cast<float *>(smem);  // [warps][rows][kLd]; [0]: the CTA's sum
    uint16_t *terms = reinterpret_cast<uint16_t *>(smem + kLoraWarps * C::kRows * C::kLd * 4);  // [terms][rows][kHLd]
    __shared__ int32_t off[kGroupsMax + 1];
    __shared__ int32_t tile_s[3];
    __shared__ int32_t row_s[C::kRows];
    __shared__ float scale_s[C::kRows];
    griddep_wait();
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, q = lane & 3;
    uint32_t csize;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(csize));
    const uint32_t crank = cluster_ctarank();
    if ((int)blockIdx.x < p.bare_ctas) {  // whole clusters
        copy_bare_rows<T>(p);
        return;
    }
    const int cluster_id = (int)((blockIdx.x - p.bare_ctas) / csize);
    const int tile = cluster_id / p.nsplit, part_n = cluster_id % p.nsplit;

    cta_find_tile(p, off, C::kRows, tile, tile_s);
    const int group = tile_s[0], first = tile_s[1], count = tile_s[2];
    if (group == -2) {
        if (threadIdx.x == 0) record_status(p.status, kSiteBadOffsets);
        return;
    }
    if (group >= 0) {
        if (threadIdx.x < C::kRows) {
            int32_t r = -1;
            if ((int)threadIdx.x < count) {
                r = p.rows[first + threadIdx.x];
                if (r < 0 || r >= p.m) {
                    record_status(p.status, kSiteBadRowIndex);
                    r = -1;
                }
            }
            row_s[threadIdx.x] = r;
        }
        __syncthreads();

        // The columns' part of B and base set out first; h is made meanwhile.
        const T *a = static_cast<const T *>(p.a) + (int64_t)group * p.rank * p.k;
        auto make_h = [&]() {
            // h = x A^T over this CTA's steps of k; warps take turns
            const T *xr[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int32_t r = row_s[8 * h + g8];
                xr[h] = r >= 0 ? static_cast<const T *>(p.x) + (int64_t)r * p.ldx : nullptr;
            }
            float acc[NB][4];
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
            const int steps = (p.k + 32 * C::kStep - 1) / (32 * C::kStep);
            const int s0 = (int)((int64_t)steps * crank / csize), s1 = (int)((int64_t)steps * (crank + 1) / csize);
            for (int s = s0 + warp; s < s1; s += kLoraWarps) {
                uint4 xv[C::kStep][2], av[C::kStep][NB];
#pragma unroll
                for (int u = 0; u < C::kStep; ++u) {
                    const int kk = (s * C::kStep + u) * 32 + q * 8;
                    const bool in = kk < p.k;
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        const int r = 8 * j + g8;
                        av[u][j] = in && r < p.rank ? load_as<uint4>(a + (int64_t)r * p.k + kk)
                                                    : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        xv[u][h] = in && xr[h] ? load_as<uint4>(xr[h] + kk) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int u = 0; u < C::kStep; ++u)
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        const uint4 &x0 = xv[u][0], &x1 = xv[u][1], &b = av[u][j];
                        mma16816(acc[j], x0.x, x1.x, x0.y, x1.y, b.x, b.y, T());
                        mma16816(acc[j], x0.z, x1.z, x0.w, x1.w, b.z, b.w, T());
                    }
            }
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                float *d = part + (warp * C::kRows + g8) * C::kLd + 8 * j + 2 * q;
                *reinterpret_cast<float2 *>(d) = make_float2(acc[j][0], acc[j][1]);
                *reinterpret_cast<float2 *>(d + 8 * C::kLd) = make_float2(acc[j][2], acc[j][3]);
            }
            __syncthreads();
            for (int i = threadIdx.x; i < count * C::kRank; i += kLoraThreads) {
                float *d = part + (i / C::kRank) * C::kLd + i % C::kRank;
                float sum = d[0];
#pragma unroll
                for (int w = 1; w < kLoraWarps; ++w) sum += d[w * C::kRows * C::kLd];
                d[0] = sum;
            }
            cluster_sync();
            // every CTA adds the parts in rank order, so all hold the same h
            const float scale = p.scales ? p.scales[group] : 1.0f;
            for (int r = warp; r < count; r += kLoraWarps) {
                constexpr int kPer = (C::kRank + 31) / 32;
                float h[kPer], top = 0.0f;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int c = i * 32 + lane;
                    const uint32_t at = smem_u32(part + r * C::kLd + (c < C::kRank ? c : 0));
                    float v[kLoraCluster];  // all in flight
#pragma unroll
                    for (uint32_t z = 0; z < kLoraCluster; ++z) v[z] = z < csize ? ld_cluster_f32(mapa_shared(at, z)) : 0.0f;
                    h[i] = 0.0f;
#pragma unroll
                    for (uint32_t z = 0; z < kLoraCluster; ++z) h[i] += v[z];
                    if (c >= p.rank) h[i] = 0.0f;  // an infinity in x makes NaN of the padding's zeros
                    top = fmaxf(top, finite_abs(h[i]));
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                const int e = row_exponent<T>(top);
                const float down = pow2f(-e), up = pow2f(e);
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int c = i * 32 + lane;
                    if (c < C::kRank) {
                        T t[kTerms<T>];
                        split_terms(h[i] * down, t);
#pragma unroll
                        for (int z = 0; z < kTerms<T>; ++z) memcpy(terms + z * C::kTermLd + r * kHLd<NB> + c, &t[z], 2);
                    }
                }
                if (lane == 0) scale_s[r] = scale * up;
            }
            __syncwarp();
            cluster_arrive_relaxed();  // this CTA reads no other CTA's part any more
            __syncthreads();
        };

        const int64_t piece = (int64_t)part_n * csize + crank, pieces = (int64_t)p.nsplit * csize;
        const int blocks = (p.n + 31) / 32;
        expand_tile<T, 1, NB>(p, group, row_s, scale_s, terms, C::kTermLd, smem + C::kSmem - kAheadBytes<1>,
                               (int)(blocks * piece / pieces), (int)(blocks * (piece + 1) / pieces), make_h);
        cluster_wait();  // no CTA leaves while another reads its part
    }
}

// ---------------------------------------------------------------------------
// Many rows per adapter: two launches, parts of h in the workspace.
//
// The first computes h = x A^T on the tensor cores of the fifth generation:
// 128 rows of a group per tile, gathered from x in 16-byte copies (a TMA gather
// of four rows per copy measured 34 us against 24 for 8192 x 4096, rank 16),
// A's rows beside them, k in steps of 64 through a ring of shared-memory
// stages, the accumulator in tensor memory. The tiles' steps, laid end to end,
// are divided evenly among the CTAs; what a CTA has of a tile is a part of h,
// which it leaves in the workspace while the next tile's copies are under way.
// It is bound by reading x and A. The second adds the parts in order and is the
// one-launch form's second half on tiles of 32 rows, bound by base and out. Two
// launches keep both streaming all the time; in one, a tile's reads of x and its
// writes alternate.
constexpr int kShRows = 128;
constexpr int kShK = 64;
constexpr int kShThreads = 320;  // warps 0-3: copies of x; 4: copies of A; 5: products; 6-9: parts out
constexpr int kShCopiers = 128, kShWriters = 128;
constexpr int kShX = kShRows * kShK * 2;
// CTAs per tile where there are more than that: with 4, 64 rows of rank 64 take
// 12.9 us, with 8 10.7, with 16 10.3, but 4096 rows of 8 adapters 44.8, 45.1 and 49.4.
constexpr int kShParts = 8;

template <int R>
struct ShrinkCfg {
    static constexpr int kStage = kShX + R * kShK * 2;
    static constexpr int kPerSm = R <= 64 ? 3 : 2;
    static constexpr int kStages = (R <= 64 ? 72 : 100) * 1024 / kStage;
    static constexpr int kSmem = 1024 + kStages * kStage;  // and the tables: two words per group, and one
    static constexpr int kTmem = 2 * R;  // two accumulators
};

// Padded rank of the two-launch form.
SQ_HD int shrink_rank(int64_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

// The division of the first launch: `total` tiles of `blocks` steps each among
// up to `ctas` CTAs, each with at least one step. CTA i has the steps work * i /
// ctas and on; its part of tile t is part number i + t of the workspace, so a
// tile's parts lie one after another.
struct Shares {
    int64_t work;
    int blocks, ctas;
    __device__ __forceinline__ Shares(int total, int blocks_, int most)
        : work((int64_t)total * blocks_), blocks(blocks_), ctas(min(most, total * min(blocks_, kShParts))) {}
    __device__ __forceinline__ int64_t start(int i) const { return work * i / ctas; }
    __device__ __forceinline__ int owner(int64_t step) const { return (int)(((step + 1) * ctas - 1) / work); }
};

template <typename T, int R>
__global__ void __launch_bounds__(kShThreads, ShrinkCfg<R>::kPerSm)
    lora_shrink_kernel(const __grid_constant__ CUtensorMap tm_a, const LoraParams p) {
    using C = ShrinkCfg<R>;
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t full[C::kStages], empty[C::kStages], made[2], taken[2], drained;
    __shared__ uint32_t tmem_s;
    __shared__ int table_ok, gave_up;  // gave_up: a role's wait ran out
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = (smem_u32(dyn) + 1023u) & ~1023u;
    int32_t *off = reinterpret_cast<int32_t *>(dyn + (ring - smem_u32(dyn)) + C::kStages * C::kStage);  // [groups + 1]
    int32_t *tiles = off + p.groups + 1;                                                               // [groups + 1]
    if (warp == 5) {
        tmem_alloc(smem_u32(&tmem_s), C::kTmem);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&full[s]), kShCopiers + 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&made[a]), 1);
            mbar_init(smem_u32(&taken[a]), kShWriters);
        }
        mbar_init(smem_u32(&drained), 1);
        gave_up = 0;
        mbar_fence_init();
    }
    tc_fence_before();
    griddep_wait();
    griddep_launch();
    for (int i = threadIdx.x; i <= p.groups; i += kShThreads) off[i] = p.offsets[i];
    __syncthreads();  // also publishes the set-up above
    tc_fence_after();
    if (warp == 0) {
        const bool ok = build_tiles(off, p.groups, p.m, kShRows, tiles);
        if (lane == 0) table_ok = ok;
    }
    __syncthreads();
    const uint32_t tmem = tmem_s;
    const int total = table_ok ? tiles[p.groups] : 0;
    if (!table_ok && blockIdx.x == 0 && threadIdx.x == 0) record_status(p.status, kSiteBadOffsets);
    const Shares share(total, (p.k + kShK - 1) / kShK, (int)gridDim.x);
    const int me = (int)blockIdx.x;
    const int64_t w0 = me < share.ctas ? share.start(me) : 0, w1 = me < share.ctas ? share.start(me + 1) : 0;

    // Every role walks the same parts: f(number of the part here, tile, its group, steps b0 .. b1-1)
    auto parts = [&](auto f) {
        int n = 0;
        for (int64_t w = w0; w < w1; ++n) {
            const int tile = (int)(w / share.blocks), b0 = (int)(w % share.blocks);
            const int b1 = (int)min((int64_t)share.blocks, b0 + w1 - w);
            if (!f(n, tile, group_of_tile(tiles, p.groups, tile), b0, b1)) {
                gave_up = 1;
                return;
            }
            w += b1 - b0;
        }
    };
    int fills = 0;  // stages that the thread of A's copies has set out
    if (warp < 4) {
        // 16-byte copies into the products' layout (128-byte rows, piece c of
        // row r at c ^ (r % 8)): 8 threads per row, every 16th row. Rows past
        // the tile's end are not copied: what their lanes of the accumulator
        // hold is not read.
        const int r0 = threadIdx.x >> 3, piece = threadIdx.x & 7;
        const uint32_t at = (uint32_t)(r0 * 128 + ((piece ^ (r0 & 7)) * 16));  // rows 16 apart: the same r % 8
        int i = 0;
        parts([&](int, int tile, int group, int b0, int b1) {
            const int first = off[group] + (tile - tiles[group]) * kShRows, count = min(kShRows, off[group + 1] - first);
            const T *src[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                src[j] = nullptr;
                if (r0 + 16 * j < count) {
                    const int32_t v = p.rows[first + r0 + 16 * j];
                    // an invalid row is reported, and left out, by the second launch
                    src[j] = static_cast<const T *>(p.x) + (int64_t)(v >= 0 && v < p.m ? v : 0) * p.ldx + piece * 8;
                }
            }
            for (int b = b0; b < b1; ++b, ++i) {
                const int s = i % C::kStages;
                const bool ok = mbar_wait_own(smem_u32(&empty[s]), ((i / C::kStages) & 1) ^ 1, p.status, kSiteLoraEmpty, p.wait_ns);
                if (!__all_sync(0xFFFFFFFFu, ok)) return false;
                const uint32_t dst = ring + s * C::kStage + at, in = b * kShK + piece * 8 < p.k ? 16u : 0u;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (src[j]) cp_async16_zfill(dst + j * 16 * 128, in ? src[j] + b * kShK : src[j], in);
                cp_async_arrive(smem_u32(&full[s]));
            }
            return true;
        });
        cp_async_wait<0>();
    } else if (warp == 4) {
        if (lane == 0) {
            parts([&](int, int, int group, int b0, int b1) {
                for (int b = b0; b < b1; ++b, ++fills) {
                    const int s = fills % C::kStages;
                    if (!mbar_wait_own(smem_u32(&empty[s]), ((fills / C::kStages) & 1) ^ 1, p.status, kSiteLoraEmpty, p.wait_ns))
                        return false;
                    const uint32_t bar = smem_u32(&full[s]);
                    mbar_arrive_expect_tx(bar, R * kShK * 2);
                    tma_load_2d(ring + s * C::kStage + kShX, &tm_a, b * kShK, group * p.rank, bar);
                }
                return true;
            });
        }
        __syncwarp();
    } else if (warp == 5) {
        if (lane == 0) {
            // D binary32; A and B of type T, both K-major; N = R, M = 128
            const uint32_t fmt = IsBf16<T>::v ? 1u : 0u;
            const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(R >> 3) << 17) | ((kShRows >> 4) << 24);
            int i = 0;
            parts([&](int n, int, int, int b0, int b1) {
                const uint32_t acc = tmem + (n & 1) * R;
                if (!mbar_wait_own(smem_u32(&taken[n & 1]), ((n >> 1) & 1) ^ 1, p.status, kSiteLoraTaken, p.wait_ns)) return false;
                tc_fence_after();
                for (int b = b0; b < b1; ++b, ++i) {
                    const int s = i % C::kStages;
                    if (!mbar_wait_own(smem_u32(&full[s]), (i / C::kStages) & 1, p.status, kSiteLoraFull, p.wait_ns)) return false;
                    fence_proxy_async();  // x came through the generic proxy
                    tc_fence_after();
                    const uint32_t st = ring + s * C::kStage;
                    const uint64_t dx = smem_desc(st, 16, 8 * kShK * 2, 2u), da = smem_desc(st + kShX, 16, 8 * kShK * 2, 2u);
#pragma unroll
                    for (int j = 0; j < kShK / 16; ++j) tc_mma_f16(acc, dx + 2 * j, da + 2 * j, idesc, b != b0 || j != 0);
                    tc_commit(smem_u32(&empty[s]));
                }
                tc_commit(smem_u32(&made[n & 1]));
                return true;
            });
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3, row = quarter * 32 + lane;  // a warp reads its quarter of tensor memory
        parts([&](int n, int tile, int group, int, int) {
            const int count = off[group + 1] - (off[group] + (tile - tiles[group]) * kShRows);
            const bool ok = mbar_wait_own(smem_u32(&made[n & 1]), (n >> 1) & 1, p.status, kSiteLoraDone, p.wait_ns);
            if (!__all_sync(0xFFFFFFFFu, ok)) return false;
            tc_fence_after();
            float *dst = p.part + ((int64_t)(me + tile) * kShRows + row) * R;
            const uint32_t from = tmem + (n & 1) * R + ((uint32_t)(quarter * 32) << 16);
#pragma unroll
            for (int c = 0; c < R; c += 16) {
                uint32_t v[16];
                tmem_ld16(from + c, v);
                tmem_ld_wait();
                if (row < count)
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<uint4 *>(dst + c + e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
            }
            tc_fence_before();
            mbar_arrive(smem_u32(&taken[n & 1]));
            return true;
        });
        tc_fence_before();
    }
    __syncthreads();
    if (gave_up) {
        // A's copies and the products in flight end before the CTA's shared and
        // tensor memory go (a copier waited for its own above)
        if (warp == 4 && lane == 0)
            for (int f = fills < C::kStages ? 0 : fills - C::kStages; f < fills; ++f)
                (void)mbar_wait_own(smem_u32(&full[f % C::kStages]), (f / C::kStages) & 1, nullptr, 0, kOwnDrainNs);
        if (warp == 5 && lane == 0) {
            tc_commit(smem_u32(&drained));
            (void)mbar_wait_own(smem_u32(&drained), 0, nullptr, 0, kOwnDrainNs);
        }
        __syncwarp();
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tmem, C::kTmem);
}

// Tiles of 32 rows: 64 rows halve what is read of B (from L2) but leave two
// CTAs of registers on an SM; 8192 x 4096, rank 16: 33.6 us against 30.0, 4099
// x 4096, rank 64, 64 adapters: 40.2 against 33.5. More CTAs than these take
// the L1 that B's lines need: with four, 32.5 and 35.8 us; so does fetching B ahead
// into shared memory (rank 64: 39 us against 33.6), and more of base in flight
// changes nothing. (Rank 64 in bf16, measured with two terms of h; the third
// takes 3.5 us more.)
constexpr int kExRows = 32;
template <int NB>
constexpr int kExPerSm = NB <= 4 ? 3 : 2;

// The tiles' blocks of 32 columns, laid end to end, are divided evenly among
// the CTAs, which stay for the whole launch: a CTA's share ends inside a tile.
template <typename T, int NB>
__global__ void __launch_bounds__(kLoraThreads, kExPerSm<NB>) lora_expand_kernel(const LoraParams p) {
    constexpr int R = 8 * NB, kLd = kHLd<NB>;
    extern __shared__ __align__(16) uint8_t ahead[];
    __shared__ __align__(16) uint16_t terms[kTerms<T>][kExRows * kLd];
    __shared__ int32_t off[kGroupsMax + 1], tiles[kGroupsMax + 1], sh_tiles[kGroupsMax + 1];
    __shared__ int32_t row_s[kExRows], part_s[2];
    __shared__ float scale_s[kExRows];
    // This launch starts when every CTA of the first has passed its own wait,
    // so all that came before the first (routing, base, weights) is there;
    // only the parts of h, the first launch's results, need the wait below.
    if (p.base != p.out) copy_bare_rows<T>(p);
    for (int i = threadIdx.x; i <= p.groups; i += kLoraThreads) off[i] = p.offsets[i];
    __syncthreads();
    __shared__ int table_ok;
    if (threadIdx.x < 32) {
        const bool ok = build_tiles(off, p.groups, p.m, kExRows, tiles);
        if (threadIdx.x == 0) table_ok = ok;
    } else if (threadIdx.x < 64) {
        (void)build_tiles(off, p.groups, p.m, kShRows, sh_tiles);
    }
    __syncthreads();
    if (!table_ok) {  // reported by the first launch
        griddep_wait();
        return;
    }
    const int blocks = (p.n + 31) / 32;
    const int64_t work = (int64_t)tiles[p.groups] * blocks, ctas = gridDim.x, me = blockIdx.x;
    const int64_t w1 = work * (me + 1) / ctas;
    bool waited = false;
    for (int64_t w = work * me / ctas; w < w1;) {
        const int tile = (int)(w / blocks), c0 = (int)(w % blocks), c1 = (int)min((int64_t)blocks, c0 + w1 - w);
        const int group = group_of_tile(tiles, p.groups, tile);
        const int first = off[group] + (tile - tiles[group]) * kExRows, count = min(kExRows, off[group + 1] - first);
        __syncthreads();  // the last tile's rows and h are no longer needed
        if (threadIdx.x < kExRows) {
            int32_t r = -1;
            if ((int)threadIdx.x < count) {
                r = p.rows[first + threadIdx.x];
                if (r < 0 || r >= p.m) {
                    record_status(p.status, kSiteBadRowIndex);
                    r = -1;
                }
            }
            row_s[threadIdx.x] = r;
        } else if (threadIdx.x == 64) {  // the tile's parts: first and number
            const Shares share(sh_tiles[p.groups], (p.k + kShK - 1) / kShK, p.shrink_ctas);
            const int sh_tile = sh_tiles[group] + (first - off[group]) / kShRows;
            const int64_t step0 = (int64_t)sh_tile * share.blocks;
            const int lo = share.owner(step0);
            part_s[0] = lo + sh_tile;
            part_s[1] = share.owner(step0 + share.blocks - 1) - lo + 1;
        }
        __syncthreads();
        expand_tile<T, kExRows / 16, NB>(p, group, row_s, scale_s, terms[0], kExRows * kLd, ahead, c0, c1, [&]() {
            if (!waited) griddep_wait();
            waited = true;
            // h: 4 columns of a row per thread and turn, the parts added in order
            const int n_parts = part_s[1];
            const float *from = p.part + ((int64_t)part_s[0] * kShRows + (first - off[group]) % kShRows) * R;
            constexpr int kLanes = R / 4, kTurns = (kExRows * kLanes + kLoraThreads - 1) / kLoraThreads;
            constexpr int kFlight = 8 / kTurns;  // parts in flight
            const int c = (int)threadIdx.x % kLanes, r0 = (int)threadIdx.x / kLanes;
            float4 a[kTurns];
#pragma unroll
            for (int u = 0; u < kTurns; ++u) a[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int z0 = 0; z0 < n_parts; z0 += kFlight) {
                float4 v[kFlight][kTurns];
#pragma unroll
                for (int z = 0; z < kFlight; ++z)
#pragma unroll
                    for (int u = 0; u < kTurns; ++u) {
                        const int r = r0 + u * (kLoraThreads / kLanes);
                        v[z][u] = z0 + z < n_parts && r < count
                                      ? __ldcg(reinterpret_cast<const float4 *>(from + ((int64_t)(z0 + z) * kShRows + r) * R) + c)
                                      : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    }
#pragma unroll
                for (int z = 0; z < kFlight; ++z)
#pragma unroll
                    for (int u = 0; u < kTurns; ++u) {
                        a[u].x += v[z][u].x;
                        a[u].y += v[z][u].y;
                        a[u].z += v[z][u].z;
                        a[u].w += v[z][u].w;
                    }
            }
            const float scale = p.scales ? p.scales[group] : 1.0f;
#pragma unroll
            for (int u = 0; u < kTurns; ++u) {
                const int r = r0 + u * (kLoraThreads / kLanes);
                // the columns behind the rank belong to another adapter
                if (4 * c >= p.rank) a[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                float top = fmaxf(fmaxf(finite_abs(a[u].x), finite_abs(a[u].y)), fmaxf(finite_abs(a[u].z), finite_abs(a[u].w)));
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                const int e = row_exponent<T>(top);
                const float down = pow2f(-e), f[4] = {a[u].x * down, a[u].y * down, a[u].z * down, a[u].w * down};
                T t[4][kTerms<T>];
#pragma unroll
                for (int j = 0; j < 4; ++j) split_terms(f[j], t[j]);
                if (r < kExRows) {
#pragma unroll
                    for (int z = 0; z < kTerms<T>; ++z) {
                        const T four[4] = {t[0][z], t[1][z], t[2][z], t[3][z]};
                        memcpy(terms[z] + r * kLd + 4 * c, four, 8);
                    }
                    if (c == 0) scale_s[r] = scale * pow2f(e);
                }
            }
            __syncthreads();
        });
        w += c1 - c0;
    }
    if (!waited) griddep_wait();
}

// Tiles of `rows` rows: a bound on sum ceil(rows of a group / rows).
static int64_t tiles_bound(int64_t m, int64_t groups, int64_t rows) {
    const int64_t t = m / rows + (groups < m ? groups : m);
    return t < m ? t : m;
}

// CTAs of the first launch: as many as stay on the GPU (a workspace size, so a
// function of the shape alone).
static int shrink_ctas(int64_t m, int64_t rank, int64_t groups) {
    // three CTAs on an SM have 75 KB each: 73 of ring, the rest for tables
    const int64_t stay = (rank <= 64 && groups <= 224 ? 3 : 2) * 148, most = tiles_bound(m, groups, kShRows) * kShParts;
    return (int)(most < stay ? most : stay);
}

template <typename T, int NB>
static sharq_status lora_two(LaunchCtx &ctx, LoraParams p) {
    constexpr int R = 8 * NB;
    using C = ShrinkCfg<R>;
    CUtensorMap tm_a;
    if (!make_row_map(&tm_a, p.a, (uint64_t)p.k, (uint64_t)p.groups * p.rank, (uint64_t)p.k * 2, R))
        return SHARQ_ERR_CUDA;
    constexpr int kTables = 2 * (int)sizeof(int32_t);
    SQ_SMEM_ONCE((lora_shrink_kernel<T, R>), C::kSmem + kTables * ((int)kGroupsMax + 1));
    p.shrink_ctas = shrink_ctas(p.m, p.rank, p.groups);
    sharq_status st = launch_pdl(ctx, lora_shrink_kernel<T, R>, p.shrink_ctas, kShThreads,
                                 C::kSmem + kTables * (p.groups + 1), 1, tm_a, p);
    if (st != SHARQ_OK) return st;
    // CTAs that stay, unless that leaves a warp less than a block
    const int64_t ex = tiles_bound(p.m, p.groups, kExRows) * ((p.n + 32 * kLoraWarps - 1) / (32 * kLoraWarps));
    const int64_t stay = (int64_t)kExPerSm<NB> * ctx.num_sms;
    const int64_t ctas = ex < stay ? ex : stay;
    p.bare_ctas = (int32_t)ctas;
    SQ_SMEM_ONCE((lora_expand_kernel<T, NB>), kAheadBytes<kExRows / 16>);
    return launch_pdl(ctx, lora_expand_kernel<T, NB>, ctas, kLoraThreads, kAheadBytes<kExRows / 16>, 1, p);
}

// Whether a call takes the two-launch form (and so needs a workspace), by what
// the host knows: rows, rank and adapters (not how many of them the batch
// uses). Measured at k = n = 4096 in fp16, one launch against two, in us, rows
// shared evenly among the adapters:
//   rank 16   1 adapter:           1024 rows 12 / 14, 3000 22 / 23, 4096 40 / 29
//             64 adapters:         1024 13 / 21, 3000 24 / 27, 4096 41 / 32
//   rank 32   1 adapter:           2048 18 / 21, 3000 34 / 26; 64: 2048 20 / 26, 3000 38 / 32
//   rank 64   1 adapter:           64 10 / 11, 1024 17 / 19, 1500 30 / 23, 4096 64 / 43
//             64 adapters:         64 17 / 26, 1024 23 / 31, 1500 38 / 33
//             64 used of 256:      64 19 / 28, 256 31 / 29, 1024 38 / 32
//   rank 128  1 adapter:           1024 27 / 27, 1500 55 / 33
//             100 used of 256:     128 74 / 65, 1024 80 / 70
// Shared at random, groups end in more tiles (64 adapters, rank 64, 1024 rows: 41
// / 32). The third term in bf16 costs both forms alike.
// One launch leads as long as its 16-row tiles fit on the GPU at once; their
// accumulators and reading A and B per 16 rows cost more the larger the rank is.
static bool lora_many(int64_t m, int64_t rank, int64_t groups) {
    if (rank <= 32) return m >= (rank <= 16 ? 3500 : 2500);
    return m > 1024 || (m >= 128 && groups > 148);
}

int64_t lora_ws_bytes(int64_t m, int64_t rank, int64_t groups) {
    if (!lora_many(m, rank, groups)) return 0;
    return (shrink_ctas(m, rank, groups) + tiles_bound(m, groups, kShRows)) * kShRows * shrink_rank(rank) * (int64_t)sizeof(float);
}

template <typename T, int NB>
static sharq_status lora_run(LaunchCtx &ctx, LoraParams p) {
    using C = LoraCfg<T, NB>;
    const int64_t tiles = tiles_bound(p.m, p.groups, C::kRows);
    // Split a tile as long as the CTAs fit on the GPU together (clusters of 8 leave
    // a part of it empty) and keep a few hundred elements of k and of the columns.
    // How many tiles there are is only known on the device: the guess is that every
    // group is used and most of them fill their last tile. A second wave costs the
    // most: 64 rows of 64 adapters, rank 64, take 17 us with 256 CTAs, 35 with 512
    // that do not fit. A tile split in two whatever the guess helps where few of
    // the adapters are used (256 rows, rank 16, one of 256: 12.7 us, 19.4 without).
    const int64_t guess = p.m >= 16 * p.groups ? p.m / 16 + p.groups / 8 : p.groups < p.m ? p.groups : p.m;
    const int64_t sms = ctx.num_sms, slots = C::kPerSm * sms, eights = slots * 3 / 4;
    int cluster = 1;
    while (cluster < kLoraCluster && p.k >= 512 * cluster &&
           (2 * guess * cluster <= (2 * cluster == 8 ? eights : slots) || (cluster == 1 && guess < 2 * sms)))
        cluster *= 2;
    p.nsplit = 1;
    const int64_t wide = eights < 2 * sms ? eights : 2 * sms;
    while (p.nsplit < 16 && 2 * guess * cluster * p.nsplit <= wide && p.n >= 256 * cluster * p.nsplit) p.nsplit *= 2;
    p.bare_ctas = (int32_t)round_up(bare_ctas(ctx, p), cluster);
    const int64_t ctas = p.bare_ctas + tiles * cluster * p.nsplit;
    // rank 33 to 64: two CTAs on an SM leave too few registers; where one per SM is
    // all there is they keep theirs (one row of rank 64: 6.1 us against 6.7)
    if constexpr (NB == 8) {
        if (ctas <= sms) {
            SQ_SMEM_ONCE((lora_kernel<T, NB, 1>), C::kSmem);
            return launch_pdl(ctx, lora_kernel<T, NB, 1>, ctas, kLoraThreads, C::kSmem, cluster, p);
        }
    }
    SQ_SMEM_ONCE((lora_kernel<T, NB, C::kPerSm>), C::kSmem);
    return launch_pdl(ctx, lora_kernel<T, NB, C::kPerSm>, ctas, kLoraThreads, C::kSmem, cluster, p);
}

template <typename T>
static sharq_status lora_any(LaunchCtx &ctx, const LoraParams &p) {
    if (lora_many(p.m, p.rank, p.groups)) {
        switch (shrink_rank(p.rank)) {
            case 16: return lora_two<T, 2>(ctx, p);
            case 32: return lora_two<T, 4>(ctx, p);
            case 64: return lora_two<T, 8>(ctx, p);
            default: return lora_two<T, 16>(ctx, p);
        }
    }
    if (p.rank <= 16) return lora_run<T, 2>(ctx, p);
    if (p.rank <= 32) return lora_run<T, 4>(ctx, p);
    if (p.rank <= 64) return lora_run<T, 8>(ctx, p);
    return lora_run<T, 16>(ctx, p);
}

sharq_status launch_lora(LaunchCtx &ctx, const void *x, int64_t ldx, int64_t m, int64_t k, const void *a, const void *b,
                         int64_t n, int64_t rank, int64_t groups, const float *scales, const int32_t *offsets,
                         const int32_t *rows, const int32_t *slots, int dtype, const void *base, int64_t ldbase, void *out,
                         int64_t ldo, void *ws) {
    if (m == 0) return SHARQ_OK;
    LoraParams p{x, a, b, base, scales, out, offsets, rows, slots, (int32_t)ldx, (int32_t)ldbase, (int32_t)ldo, m,
                 (int32_t)k, (int32_t)n, (int32_t)rank, (int32_t)groups, 1, 0, ctx.status, ctx.wait_ns,
                 static_cast<float *>(ws), 0};
    return dtype == SHARQ_F16 ? lora_any<__half>(ctx, p) : lora_any<__nv_bfloat16>(ctx, p);
}

}  // namespace sq

// Element types and 16-byte vectors of the operators that work in 16 or 32
// bits (normalization, adapters, token order): every value is widened to
// binary32 exactly on load and rounded once, to nearest even, on store.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <atomic>
#include <type_traits>

#include "sharq_dev.cuh"
#include "sq_internal.h"

namespace sq {

// Loads are plain ones. What they read the launch before may have written, and it
// still runs when these kernels start; and some of it is the call's own output (dy,
// residual, base). Loads marked read-only may be moved ahead of griddep_wait, or
// past the store to the same place.
template <typename P>
__device__ __forceinline__ P load_as(const void *p) { return *static_cast<const P *>(p); }

// Loads and stores of VW consecutive elements (VW * sizeof(T) bytes, that
// alignment), held packed until they are widened.
template <int BYTES>
struct Packed;
template <>
struct Packed<16> { using type = uint4; };
template <>
struct Packed<4> { using type = uint32_t; };
template <>
struct Packed<2> { using type = uint16_t; };

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T>
struct IsBf16 { static constexpr bool v = false; };
template <>
struct IsBf16<__nv_bfloat16> { static constexpr bool v = true; };

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}

template <typename T, int VW>
struct Vec {
    using P = typename Packed<VW * (int)sizeof(T)>::type;
    static __device__ __forceinline__ P zero() {
        P p;
        memset(&p, 0, sizeof(p));
        return p;
    }
    static __device__ __forceinline__ P ones() {
        float f[VW];
#pragma unroll
        for (int i = 0; i < VW; ++i) f[i] = 1.0f;
        return pack(f);
    }
    static __device__ __forceinline__ P load(const T *p) { return load_as<P>(p); }
    static __device__ __forceinline__ void store(T *p, P v) { *reinterpret_cast<P *>(p) = v; }
    static __device__ __forceinline__ void unpack(P v, float (&f)[VW]) {
        T t[VW];
        memcpy(t, &v, sizeof(v));
#pragma unroll
        for (int i = 0; i < VW; ++i) f[i] = widen(t[i]);
    }
    // The same as packed binary32 pairs (VW even).
    static __device__ __forceinline__ void unpack2(P v, uint64_t (&f)[(VW + 1) / 2]) {
        uint32_t w[sizeof(P) / 4 ? sizeof(P) / 4 : 1];
        memcpy(w, &v, sizeof(v));
#pragma unroll
        for (int i = 0; i < VW / 2; ++i) {
            if constexpr (sizeof(T) == 4) f[i] = (uint64_t)w[2 * i] | (uint64_t)w[2 * i + 1] << 32;
            else if constexpr (sizeof(T) == 2 && !IsBf16<T>::v) f[i] = h2_to_f2(w[i]);
            else f[i] = pk2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
        }
    }
    static __device__ __forceinline__ P pack2(const uint64_t (&f)[(VW + 1) / 2]) {
        float t[VW];
#pragma unroll
        for (int i = 0; i < VW / 2; ++i) {
            const float2 u = up2(f[i]);
            t[2 * i] = u.x;
            t[2 * i + 1] = u.y;
        }
        return pack(t);
    }
    static __device__ __forceinline__ P pack(const float (&f)[VW]) {
        P v;
        if constexpr (sizeof(T) == 2 && VW % 2 == 0) {  // two values per conversion
            uint32_t w[VW / 2];
#pragma unroll
            for (int i = 0; i < VW / 2; ++i) w[i] = IsBf16<T>::v ? bf16x2(f[2 * i], f[2 * i + 1]) : f16x2(f[2 * i], f[2 * i + 1]);
            memcpy(&v, w, sizeof(v));
        } else {
            T t[VW];
#pragma unroll
            for (int i = 0; i < VW; ++i) t[i] = narrow<T>(f[i]);
            memcpy(&v, t, sizeof(v));
        }
        return v;
    }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Calls f with a value of the C++ type of a sharq_dtype.
template <typename F>
static inline sharq_status with_dtype(int dtype, F f) {
    if (dtype == SHARQ_F16) return f(__half());
    if (dtype == SHARQ_BF16) return f(__nv_bfloat16());
    return f(float());
}

// Raises a kernel's dynamic shared memory limit, once per device.
#define SQ_SMEM_ONCE(kernel, bytes)                                                                              \
    do {                                                                                                         \
        static std::atomic<uint64_t> _done{0};                                                                   \
        int _dev = 0;                                                                                            \
        SQ_CUDA_TRY(cudaGetDevice(&_dev));                                                                       \
        if (!((_done.load() >> _dev) & 1u)) {                                                                    \
            SQ_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(bytes))); \
            _done.fetch_or(1ull << _dev);                                                                        \
        }                                                                                                        \
    } while (0)

// Launch with programmatic stream serialization (the kernels start with
// griddep_wait) and, for cluster > 1, a cluster dimension.
template <typename... A>
static sharq_status launch_pdl(LaunchCtx &ctx, void (*kernel)(A...), int64_t grid, int threads, size_t smem, int cluster,
                               std::common_type_t<A>... a) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    SQ_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, a...));
    ctx.launches++;
    return SHARQ_OK;
}

}  // namespace sq

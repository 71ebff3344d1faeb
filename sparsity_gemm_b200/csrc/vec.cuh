// Element types and 16-byte vectors of the operators that work in 16 or 32
// bits (normalization, adapters, token order): every value is widened to
// binary32 exactly on load and rounded once, to nearest even, on store.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "sq_internal.h"

namespace sq {

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

template <typename T, int VW>
struct Vec {
    using P = typename Packed<VW * (int)sizeof(T)>::type;
    static __device__ __forceinline__ P zero() {
        P p;
        memset(&p, 0, sizeof(p));
        return p;
    }
    static __device__ __forceinline__ P load(const T *p) { return __ldg(reinterpret_cast<const P *>(p)); }
    static __device__ __forceinline__ void store(T *p, P v) { *reinterpret_cast<P *>(p) = v; }
    static __device__ __forceinline__ void unpack(P v, float (&f)[VW]) {
        T t[VW];
        memcpy(t, &v, sizeof(v));
#pragma unroll
        for (int i = 0; i < VW; ++i) f[i] = widen(t[i]);
    }
    static __device__ __forceinline__ P pack(const float (&f)[VW]) {
        T t[VW];
#pragma unroll
        for (int i = 0; i < VW; ++i) t[i] = narrow<T>(f[i]);
        P v;
        memcpy(&v, t, sizeof(v));
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

// Launch with programmatic stream serialization (the kernels start with
// griddep_wait) and, for cluster > 1, a cluster dimension.
template <typename P, typename... A>
static sharq_status launch_pdl(LaunchCtx &ctx, void (*kernel)(P, A...), int64_t grid, int threads, size_t smem, int cluster,
                               P p, A... a) {
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
    SQ_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, p, a...));
    ctx.launches++;
    return SHARQ_OK;
}

}  // namespace sq

// Shared by the kernels of kda_layer.h: element types, 16-byte vectors, launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <atomic>

#include "kda_layer.h"

namespace kda_layer {

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// N consecutive elements moved as one access (N * sizeof(T) in {4, 8, 16}).
template <typename T, int N>
struct alignas(N * sizeof(T)) Vec {
    T v[N];
};

template <typename T, int N>
__device__ __forceinline__ Vec<T, N> ld_vec(const T *p) {
    return *reinterpret_cast<const Vec<T, N> *>(p);
}

template <typename T, int N>
__device__ __forceinline__ void st_vec(T *p, const Vec<T, N> &x) {
    *reinterpret_cast<Vec<T, N> *>(p) = x;
}

// The same 16 bytes without keeping them in L1: read once.
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> ld_stream(const T *p) {
    static_assert(sizeof(Vec<T, N>) == 16, "16-byte vectors");
    Vec<T, N> x;
    uint4 &u = *reinterpret_cast<uint4 *>(&x);
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p) : "memory");
    return x;
}

// Division by a divisor fixed for a launch: for 1 <= d < 2^31, l = ceil(log2 d)
// and m = floor(2^32 (2^l - d) / d) + 1, every n < 2^32 has n / d =
// (t + ((n - t) >> min(l, 1))) >> max(l - 1, 0) with t = umulhi(m, n) (Granlund and
// Montgomery, 1994).
struct FastDiv {
    uint32_t m;
    int s1, s2;
};

inline FastDiv make_fast_div(uint32_t d) {
    int l = 0;
    while ((uint64_t(1) << l) < d) ++l;
    FastDiv f;
    f.m = (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << l) - d)) / d + 1);
    f.s1 = l < 1 ? l : 1;
    f.s2 = l > 1 ? l - 1 : 0;
    return f;
}

__device__ __forceinline__ uint32_t fast_div(uint32_t n, FastDiv f) {
    const uint32_t t = __umulhi(f.m, n);
    return (t + ((n - t) >> f.s1)) >> f.s2;
}

// One element of a tensor whose type is known at run time (beta, per-head gates).
__device__ __forceinline__ float ld_dyn(const void *p, int64_t i, int dtype) {
    if (dtype == KDA_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    if (dtype == KDA_DTYPE_F16) return __half2float(static_cast<const __half *>(p)[i]);
    return static_cast<const float *>(p)[i];
}

// expf for its accuracy; the quotient by __fdividef (2 ulp; 0 for a denominator past 2^126).
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.0f, 1.0f + expf(-x)); }

// Every kernel starts with this: nothing is read before the preceding kernel's
// writes are visible, and the next kernel may be scheduled while this one runs.
__device__ __forceinline__ void dependency_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" :::);
}

inline bool aligned(const void *p, uintptr_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

inline int64_t dtype_bytes(int dtype) { return dtype == KDA_DTYPE_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype >= KDA_DTYPE_BF16 && dtype <= KDA_DTYPE_F32; }

char *error_buffer();  // the calling thread's text (256 bytes), kda_norm.cu
kda_status_t cuda_status(cudaError_t e);
int current_sms();

// Lets a kernel take `bytes` of dynamic shared memory, once per device (`done`: a bit
// each; threads that race set the same value).
inline cudaError_t allow_smem(const void *kernel, int bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// A launch as programmatic dependent of the preceding kernel (dependency_wait).
template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, unsigned threads, size_t smem,
                   kda_stream_t stream, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace kda_layer

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
